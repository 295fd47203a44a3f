// rnnt_distill.cu -- learning from a teacher: the top logits of a teacher's rows, and the loss of a
// student against them with its gradient.
//
// Row: the V logits x of one lattice node; s = x / tau for a temperature tau.
//
// Top logits.  The k largest of x with their ids, in order (ties: the lowest id first), and
// rest = log of the sum of exp(s_j) over the remaining j.
//
// Distillation.  The teacher's row is a distribution p over its places (softmax of their logits /
// tau), and, where a rest is given, one class more for all remaining outputs.  With q = softmax(s)
// and q_r the sum of q_j over the outputs that have no place,
//   loss = tau^2 [ sum_k p_k (log p_k - log q_id(k)) + p_r (log p_r - log q_r) ]
//   d loss / d x_j = tau (q_j - p_j)              where j has a place
//                  = tau q_j (1 - p_r / q_r)      where it has none (tau q_j without a rest).
// q_r is summed over its outputs, not taken as 1 - sum of the others, which would lose it where
// the student is sure of the teacher's places.  tau^2 keeps the gradient's size over temperatures.
#include "rnnt_rows.cuh"

using namespace rnnt_rows;

namespace {

constexpr float kMost = 3.40282347e38f;    // the largest float32: finite logits / tau stay finite
constexpr int kMostRows = 152 * 16;        // blocks of a kernel that takes a row a block

// The lattice's rows: all of them (no lengths), or those of the sequences, compact or padded.
struct Lattice {
    const int32_t* T;                      // logit lengths, or NULL: every row counts
    const int32_t* U;                      // target lengths
    int64_t rows;
    int32_t B, padded, max_T, max_U;

    // Rows of sequence b; `ok`: whether its lengths are in range.
    __device__ __forceinline__ int64_t of_sequence(int b, int& t, int& u, bool& ok) const {
        t = T[b];
        u = U[b];
        ok = t >= 0 && u >= 0 && u < INT32_MAX && (!padded || (t <= max_T && u <= max_U));
        t = max(t, 0);
        u = max(u, -1);
        if (padded) {
            t = min(t, max_T);
            u = min(u, max_U);
        }
        return (int64_t)t * ((int64_t)u + 1);
    }
    // Whether a row of the padded layout belongs to a sequence.
    __device__ __forceinline__ bool inside(int64_t row) const {
        const int64_t w = (int64_t)max_U + 1, q = row / w;
        const int u = (int)(row - q * w), b = (int)(q / max_T), t = (int)(q - (int64_t)b * max_T);
        return t < T[b] && u <= U[b];
    }
};

// ------------------------------------------------------------------ blocks
template <int TH>
__device__ __forceinline__ uint64_t block_largest(uint64_t x, uint64_t* space) {
    x = warp_largest(x);
    if ((threadIdx.x & 31) == 0) space[threadIdx.x >> 5] = x;
    __syncthreads();
    x = warp_largest((threadIdx.x & 31) < TH / 32 ? space[threadIdx.x & 31] : 0ull);
    __syncthreads();
    return x;
}
template <int TH, typename V>
__device__ __forceinline__ V block_sum(V x, V* space) {
    x = warp_sum(x);
    if ((threadIdx.x & 31) == 0) space[threadIdx.x >> 5] = x;
    __syncthreads();
    x = warp_sum((threadIdx.x & 31) < TH / 32 ? space[threadIdx.x & 31] : V(0));
    __syncthreads();
    return x;
}
template <int TH>
__device__ __forceinline__ float block_max(float x, float* space) {
    x = warp_max_nan(x);
    if ((threadIdx.x & 31) == 0) space[threadIdx.x >> 5] = x;
    __syncthreads();
    x = warp_max_nan((threadIdx.x & 31) < TH / 32 ? space[threadIdx.x & 31] : -INFINITY);
    __syncthreads();
    return x;
}

__device__ __forceinline__ void invalid(int32_t* status) {
    if (status) *status = RNNT_INVALID_VALUE;
}
template <int TH>
__device__ __forceinline__ void check_lengths(const Lattice& lat, int32_t* status) {
    for (int b = threadIdx.x; b < lat.B; b += TH) {
        int t, u;
        bool ok;
        lat.of_sequence(b, t, u, ok);
        if (!ok) invalid(status);
    }
}

// ------------------------------------------------------------- top logits
struct TopParams {
    const char* logits;
    Lattice lat;
    int32_t V, k;
    float scale;                           // log2 e / tau
    float inv_tau;
    void* values;
    int32_t* ids;
    float* rest;
    int32_t* status;
};

constexpr int kLongThreads = 256;
constexpr int kTopBuf = 1024;              // elements of a row that are ranked: 4 a thread

// The k + 1 best are selected: the last of them is the largest of the rest, to which its sum is
// relative (relative to the k-th best it could vanish).
//
// A row a block, read up to three times from the cache: for each thread's maximum, for the elements
// that reach the bound which these give (of every warp's largest maxima enough to make k + 1
// together; the least of them), and for the rest's sum.  A row in which too many reach it (a
// crowd of equal ones) gives its best one by one.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) k_top_long(const TopParams p) {
    constexpr int TH = kLongThreads, WARPS = TH / 32, E = 16 / (int)sizeof(T);
    __shared__ uint64_t buf[kTopBuf], best[RNNT_MAX_TOP + 1], space64[WARPS];
    __shared__ float space[WARPS];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, k = p.k, most = k + 1;
    if (blockIdx.x == 0 && p.lat.T) check_lengths<TH>(p.lat, p.status);
    for (int64_t row = blockIdx.x; row < p.lat.rows; row += gridDim.x) {
        bool live = !p.lat.T || p.lat.inside(row);
        int have = 0;
        float rest = -INFINITY;
        if (live) {
            const Row<T> r(reinterpret_cast<const T*>(p.logits) + row * p.V, p.V);
            if (tid == 0) count = 0;
            float mine = -INFINITY;
            for (int j = tid; j < r.n; j += TH) {
                const Pack<T, 16> v = r.load(j);
#pragma unroll
                for (int e = 0; e < E; ++e) mine = max_nan(mine, to_f32(v.e[e]));
            }
            const float top = block_max<TH>(mine, space);
            if (!(top < INFINITY)) {                       // NaN or +inf: the row is left empty
                if (tid == 0) invalid(p.status);
            } else if (top > -INFINITY) {
                // the bound: the warp's c-th largest maximum, the least of them over the warps
                const int c = (most + WARPS - 1) / WARPS;
                int above = 0;
                for (int o = 0; o < 32; ++o) {
                    const float y = __shfl_sync(kAll, mine, o);
                    above += y > mine || (y == mine && o < lane);
                }
                const unsigned at = __ballot_sync(kAll, above == c - 1);
                const float cth = __shfl_sync(kAll, mine, __ffs(at) - 1);
                if (lane == 0) space[tid >> 5] = -cth;
                __syncthreads();
                float bound = -space[0];
#pragma unroll
                for (int w = 1; w < WARPS; ++w) bound = fminf(bound, -space[w]);
                for (int j = tid; j < r.n; j += TH) {
                    const Pack<T, 16> v = r.load(j);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float y = to_f32(v.e[e]);
                        if (y >= bound && y > -INFINITY) {
                            const int i = atomicAdd(&count, 1);
                            if (i < kTopBuf) buf[i] = key_of(y, j * E + e - r.off);
                        }
                    }
                }
                __syncthreads();
                const int n = count;
                have = min(n, most);
                if (n <= kTopBuf) {
                    for (int i = tid; i < n; i += TH) {
                        int rank = 0;
                        for (int o = 0; o < n; ++o) rank += buf[o] > buf[i];
                        if (rank < most) best[rank] = buf[i];
                    }
                } else {
                    uint64_t last = ~0ull;
                    for (int i = 0; i < most; ++i) {
                        uint64_t next = 0;
                        for (int j = tid; j < r.n; j += TH) {
                            const Pack<T, 16> v = r.load(j);
#pragma unroll
                            for (int e = 0; e < E; ++e) {
                                const uint64_t key = key_of(to_f32(v.e[e]), j * E + e - r.off);
                                if (key < last && key > next) next = key;
                            }
                        }
                        last = block_largest<TH>(next, space64);
                        if (tid == 0) best[i] = last;
                    }
                }
                __syncthreads();
                // the rest: its largest, the elements below that, and those equal to it that
                // had no place
                if (have == most) {
                    const float first = value_of(best[k]);
                    float sum = 0.0f, equal = 0.0f;
                    for (int j = tid; j < r.n; j += TH) {
                        const Pack<T, 16> v = r.load(j);
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const float y = to_f32(v.e[e]);
                            sum += y < first ? ex2((y - first) * p.scale) : 0.0f;
                            equal += y == first ? 1.0f : 0.0f;
                        }
                    }
                    sum = block_sum<TH>(sum, space);
                    equal = block_sum<TH>(equal, space);
                    for (int i = 0; i < k; ++i) equal -= value_of(best[i]) == first ? 1.0f : 0.0f;
                    rest = fmaxf(logf(sum + equal) + first * p.inv_tau, -kMost);
                }
            }
        }
        for (int i = tid; i < k; i += TH) {
            const uint64_t key = i < have ? best[i] : 0;
            reinterpret_cast<T*>(p.values)[row * k + i] =
                from_f32<T>(i < have ? value_of(key) : -INFINITY);
            p.ids[row * k + i] = i < have ? element_of(key) : -1;
        }
        if (tid == 0) p.rest[row] = rest;
        __syncthreads();
    }
}

// ------------------------------------------------------------- distillation
struct DistillParams {
    const char* logits;
    const char* teacher;                   // logits of the places
    const int32_t* ids;
    const float* rest;                     // or NULL
    Lattice lat;
    int32_t V, k, teacher_dt;
    float scale;                           // log2 e / tau
    float inv_tau;
    float grad_scale;                      // tau * weight, over the batch for the mean
    double loss_scale;                     // tau^2 * weight
    char* grad;                            // or NULL
    float* row_loss;                       // [rows], 0 where a row does not count
    double* sample_loss;                   // [B]
    int32_t* done;                         // samples that k_distill_sum has finished
    int64_t* first_row;                    // [B + 1], of the compact layout
    float* loss;
    float* loss_reduced;
    int32_t mean;
    int32_t* status;
};

__device__ __forceinline__ float teacher_logit(const DistillParams& p, int64_t at) {
    if (p.teacher_dt == RNNT_F32) return reinterpret_cast<const float*>(p.teacher)[at];
    if (p.teacher_dt == RNNT_F16) return to_f32(reinterpret_cast<const __half*>(p.teacher)[at]);
    return to_f32(reinterpret_cast<const __nv_bfloat16*>(p.teacher)[at]);
}

// A teacher's row, two places a lane of a warp.
struct Teacher {
    int id[2];                             // -1: an empty place
    float t[2];                            // logit / tau, -inf in an empty place
    float rest;                            // -inf without one
    bool given;                            // a rest
    float p[2], log_p[2], p_rest, log_p_rest;
    bool some;                             // whether anything is in it

    __device__ __forceinline__ void load(const DistillParams& a, int64_t row) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int k = lane + 32 * q;
            id[q] = -1;
            t[q] = -INFINITY;
            if (k < a.k) {
                id[q] = a.ids[row * a.k + k];
                const float x = teacher_logit(a, row * a.k + k);
                t[q] = x * a.inv_tau;
                if (t[q] == -INFINITY && x != -INFINITY) t[q] = -kMost;
            }
        }
        given = a.rest != nullptr;
        rest = given ? a.rest[row] : -INFINITY;
    }
    // Empties places without an output of the vocabulary; says what is not allowed.
    __device__ __forceinline__ void check(const DistillParams& a) {
        bool bad = !(rest < INFINITY);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            bad |= id[q] >= a.V;
            if ((unsigned)id[q] >= (unsigned)a.V) {
                id[q] = -1;
                t[q] = -INFINITY;
            }
            bad |= !(t[q] < INFINITY);
        }
        if (bad) invalid(a.status);
    }
    // Empties a place whose id stands in one before it.
    __device__ __noinline__ void drop_repeated(const DistillParams& a) {
        const int lane = threadIdx.x & 31;
        const int id0 = id[0], id1 = id[1];
        for (int o = 0; o < 32; ++o) {
            const int x = __shfl_sync(kAll, id0, o), y = __shfl_sync(kAll, id1, o);
            if (id0 >= 0 && o < lane && x == id0) id[0] = -1;
            if (id1 >= 0 && (x == id1 || (o < lane && y == id1))) id[1] = -1;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (id[q] < 0) t[q] = -INFINITY;
        invalid(a.status);
    }
    __device__ __forceinline__ void softmax() {
        const float top = warp_max(fmaxf(fmaxf(t[0], t[1]), rest));
        some = top > -INFINITY;
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < 2; ++q) sum += t[q] == -INFINITY ? 0.0f : expf(t[q] - top);
        sum = warp_sum(sum) + (rest == -INFINITY ? 0.0f : expf(rest - top));
        const float log_sum = logf(sum);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            log_p[q] = (t[q] - top) - log_sum;
            p[q] = t[q] == -INFINITY ? 0.0f : expf(log_p[q]);
        }
        log_p_rest = (rest - top) - log_sum;
        p_rest = rest == -INFINITY ? 0.0f : expf(log_p_rest);
    }
};

// Zeros to a gradient row.
template <typename T, int TH>
__device__ __forceinline__ void zero_row(const DistillParams& p, int64_t row) {
    const Row<T> r(reinterpret_cast<const T*>(p.logits) + row * p.V, p.V);
    Pack<T, 16> z;
    z.raw = make_uint4(0, 0, 0, 0);
    T* y = reinterpret_cast<T*>(p.grad) + row * p.V;
    for (int j = (int)threadIdx.x % TH; j < r.n; j += TH) r.store(y, j, z);
}

// Rows of the sequences in the compact layout, at most all there are.
template <int TH>
__device__ __forceinline__ int64_t compact_rows(const Lattice& lat, int64_t* space) {
    int64_t n = 0;
    for (int b = threadIdx.x; b < lat.B; b += TH) {
        int t, u;
        bool ok;
        n += min(lat.of_sequence(b, t, u, ok), lat.rows);
    }
    return min(block_sum<TH>(n, space), lat.rows);
}

// A row a block, read twice (the second time from the cache).  The outputs that have a place are
// marked in a bitmap of the vocabulary.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) k_distill_long(const DistillParams p) {
    constexpr int TH = kLongThreads, WARPS = TH / 32, E = 16 / (int)sizeof(T);
    extern __shared__ uint32_t marks[];                    // of ids, (V + 31) / 32 words
    __shared__ int64_t space64[WARPS];
    __shared__ float tops[WARPS], sums[WARPS], s_base, s_coef;
    __shared__ int s_some;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    let_next_start();
    if (blockIdx.x == 0 && tid == 0) *p.done = 0;
    for (int i = tid; i < (p.V + 31) / 32; i += TH) marks[i] = 0;
    const int64_t rows = p.lat.padded ? p.lat.rows : compact_rows<TH>(p.lat, space64);
    __syncthreads();
    Teacher te;
    float at[2];
    for (int64_t row = blockIdx.x; row < p.lat.rows; row += gridDim.x) {
        const bool live = row < rows && (!p.lat.padded || p.lat.inside(row));
        if (warp == 0 && live) {
            te.load(p, row);
            te.check(p);
            bool again = false;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (te.id[q] >= 0) {
                    const uint32_t bit = 1u << (te.id[q] & 31);
                    again |= (atomicOr(&marks[te.id[q] >> 5], bit) & bit) != 0;
                }
            if (__any_sync(kAll, again)) te.drop_repeated(p);
            te.softmax();
            if (lane == 0) s_some = te.some;
        }
        __syncthreads();
        if (!live || !s_some) {
            if (p.grad) zero_row<T, TH>(p, row);
            if (tid == 0) p.row_loss[row] = 0.0f;
            if (live && warp == 0) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (te.id[q] >= 0) marks[te.id[q] >> 5] = 0;
            }
            __syncthreads();
            continue;
        }
        const Row<T> r(reinterpret_cast<const T*>(p.logits) + row * p.V, p.V);
        // the sum over the outputs without a place, relative to the largest so far
        float top = -INFINITY, sum = 0.0f;
        for (int j = tid; j < r.n; j += TH) {
            const Pack<T, 16> v = r.load(j);
            float y[E], m = -INFINITY;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = j * E + e - r.off;
                const bool marked =
                    (unsigned)i < (unsigned)p.V && (marks[i >> 5] >> (i & 31) & 1);
                y[e] = marked ? -INFINITY : to_f32(v.e[e]);
                m = max_nan(m, y[e]);
            }
            if (m == -INFINITY) continue;
            if (!(m <= top)) {
                sum = top == -INFINITY ? 0.0f : sum * ex2((top - m) * p.scale);
                top = m;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) sum += ex2((y[e] - top) * p.scale);
        }
        const float wtop = warp_max_nan(top);
        sum = top == -INFINITY ? 0.0f : sum * ex2((top - wtop) * p.scale);
        sum = warp_sum(sum);
        if (lane == 0) {
            tops[warp] = wtop;
            sums[warp] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            float m = -INFINITY;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                at[q] = te.id[q] >= 0 ? to_f32(r.x[te.id[q]]) : -INFINITY;
                m = max_nan(m, at[q]);
            }
            const float wt = lane < WARPS ? tops[lane] : -INFINITY;
            const float ws = lane < WARPS ? sums[lane] : 0.0f;
            // the terms of the outputs without a place are relative to their own largest
            // (relative to the whole row's they could vanish, with p_r > 0), the others to that of all
            const float outside = warp_max_nan(wt), base = warp_max_nan(max_nan(m, wt));
            const float left = warp_sum(wt == -INFINITY ? 0.0f : ws * ex2((wt - outside) * p.scale));
            const float shift = outside == -INFINITY ? 0.0f : ex2((outside - base) * p.scale);
            float e[2], mine = 0.0f;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                e[q] = te.id[q] >= 0 ? ex2((at[q] - base) * p.scale) : 0.0f;
                mine += e[q];
            }
            const float total = left * shift + warp_sum(mine);
            if (!(total > 0.0f && total < INFINITY)) invalid(p.status);    // NaN among them
            const float log_total = logf(total);
            float kl = 0.0f;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (te.p[q] != 0.0f)
                    kl += te.p[q] *
                          (te.log_p[q] - ((at[q] - base) * p.inv_tau - log_total));
            kl = warp_sum(kl);
            if (te.p_rest != 0.0f)
                kl += te.p_rest * (te.log_p_rest - (logf(left) + (outside - base) * p.inv_tau -
                                                    log_total));
            const float inv = 1.0f / total;
#pragma unroll
            for (int q = 0; q < 2; ++q) te.t[q] = e[q] * inv - te.p[q];    // of the places
            float coef = shift * inv;
            if (te.given && left > 0.0f) coef -= te.p_rest / left;
            if (lane == 0) {
                p.row_loss[row] = kl;
                s_base = outside == -INFINITY ? 0.0f : outside;
                s_coef = coef * p.grad_scale;
            }
        }
        __syncthreads();
        if (p.grad) {
            const float base = s_base, coef = s_coef;
            T* g = reinterpret_cast<T*>(p.grad) + row * p.V;
            for (int j = tid; j < r.n; j += TH) {
                Pack<T, 16> v = r.load(j);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    v.e[e] = from_f32<T>(ex2((to_f32(v.e[e]) - base) * p.scale) * coef);
                r.store(g, j, v);
            }
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (te.id[q] >= 0) g[te.id[q]] = from_f32<T>(te.t[q] * p.grad_scale);
            }
        }
        if (warp == 0) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (te.id[q] >= 0) marks[te.id[q] >> 5] = 0;
        }
        __syncthreads();
    }
}

// A block a sample: its rows' losses, added in float64 in an order that depends on the lengths
// alone; the last block adds the samples.  The compact layout's row offsets stay in the workspace
// for the gradient's scaling.
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) k_distill_sum(const DistillParams p) {
    constexpr int TH = kSumThreads, WARPS = TH / 32;
    __shared__ int64_t space64[WARPS];
    __shared__ double space[WARPS];
    __shared__ bool last;
    const int b = blockIdx.x, tid = threadIdx.x;
    int t, u;
    bool ok;
    const int64_t n = p.lat.of_sequence(b, t, u, ok);
    int64_t first = 0;
    if (!p.lat.padded) {
        for (int i = tid; i < b; i += TH) {
            int t0, u0;
            bool ok0;
            first += min(p.lat.of_sequence(i, t0, u0, ok0), p.lat.rows);
        }
        first = block_sum<TH>(first, space64);
        const int64_t end = first + min(n, p.lat.rows);
        if (b == p.lat.B - 1) ok &= end == p.lat.rows;
        if (tid == 0) {
            p.first_row[b] = first;
            if (b == p.lat.B - 1) p.first_row[b + 1] = end;
        }
    }
    if (!ok && tid == 0) invalid(p.status);
    wait_for_previous();
    double sum = 0.0;
    if (p.lat.padded) {
        const int64_t w = (int64_t)u + 1, row0 = (int64_t)b * p.lat.max_T * (p.lat.max_U + 1);
        for (int64_t i = tid; i < n; i += TH) {
            const int64_t q = i / w;
            sum += p.row_loss[row0 + q * (p.lat.max_U + 1) + (i - q * w)];
        }
    } else {
        const int64_t end = min(first + n, p.lat.rows);
        for (int64_t i = first + tid; i < end; i += TH) sum += p.row_loss[i];
    }
    sum = block_sum<TH>(sum, space) * p.loss_scale;
    if (tid == 0) {
        p.loss[b] = (float)sum;
        p.sample_loss[b] = sum;
        __threadfence();
        last = atomicAdd(p.done, 1) == p.lat.B - 1;
    }
    __syncthreads();
    if (!last || !p.loss_reduced) return;
    __threadfence();
    sum = 0.0;
    for (int i = tid; i < p.lat.B; i += TH)
        sum += *reinterpret_cast<volatile double*>(p.sample_loss + i);
    sum = block_sum<TH>(sum, space);
    if (tid == 0) *p.loss_reduced = (float)(p.mean ? sum / p.lat.B : sum);
}

// ------------------------------------------------- the gradient, times a factor
struct ScaleParams {
    char* grad;
    const float* factors;
    const int64_t* first_row;
    int64_t rows;
    int64_t each;                          // rows of a sample of the padded layout, 0: compact
    int32_t V, B, per_sample;
};

// Elements in float32, rounded once more.  A factor of 1 changes nothing and is not applied.
template <typename T>
__global__ void __launch_bounds__(256) k_distill_scale(const ScaleParams p) {
    const float one = p.per_sample ? 0.0f : p.factors[0];
    if (one == 1.0f) return;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float f = one;
        if (p.per_sample) {
            int b;
            if (p.each) {
                b = (int)(row / p.each);
            } else {
                int lo = 0, hi = p.B;                      // the last sample that begins at or before
                while (hi - lo > 1) {                      // the row
                    const int mid = (lo + hi) / 2;
                    (p.first_row[mid] <= row ? lo : hi) = mid;
                }
                b = lo;
            }
            f = p.factors[b];
            if (f == 1.0f) continue;
        }
        T* y = reinterpret_cast<T*>(p.grad) + row * p.V;
        const Row<T> r(y, p.V);
        for (int j = threadIdx.x; j < r.n; j += 256) {
            Pack<T, 16> v = r.load(j);
#pragma unroll
            for (int e = 0; e < Row<T>::E; ++e) v.e[e] = from_f32<T>(to_f32(v.e[e]) * f);
            r.store(y, j, v);
        }
    }
}

// ---------------------------------------------------------------------- host
bool lattice_ok(const Lattice& lat) {
    if (lat.rows < 1 || lat.rows > INT64_MAX / 8) return false;
    if (!lat.T != !lat.U) return false;
    if (!lat.T) return true;
    if (lat.B < 1 || ((uintptr_t)lat.T & 3) || ((uintptr_t)lat.U & 3)) return false;
    if (!lat.padded) return true;
    if (lat.max_T < 1 || lat.max_U < 0 || lat.max_U == INT32_MAX) return false;
    const int64_t w = (int64_t)lat.max_U + 1;
    return (int64_t)lat.max_T <= INT64_MAX / 8 / w / lat.B &&
           lat.rows == (int64_t)lat.B * lat.max_T * w;
}
// Bytes of `n` rows of `each` elements of `size`, or -1 beyond what an address holds.
int64_t bytes_of(int64_t n, int64_t each, int size) {
    return n <= (INT64_MAX >> 8) / each / size ? n * each * size : -1;
}
bool temperature_ok(double tau) { return tau >= 1e-4 && tau <= 1e4; }
dim3 row_grid(int64_t rows) { return dim3((unsigned)std::min<int64_t>(rows, kMostRows)); }

struct DistillLayout {
    size_t row_loss, sample_loss, first_row, done, total;
};
DistillLayout distill_layout(int32_t B, int64_t rows) {
    DistillLayout L;
    L.first_row = 0;                       // first: what rnnt_distill_grad_scale reads
    L.sample_loss = align256(L.first_row + ((size_t)B + 1) * sizeof(int64_t));
    L.done = align256(L.sample_loss + (size_t)B * sizeof(double));
    L.row_loss = L.done + 256;
    L.total = align256(L.row_loss + (size_t)rows * sizeof(float));
    return L;
}

bool distill_prepared() {
    static std::atomic<bool> done[64];
    return prepared_once(done, [] {
        const auto raise = [](auto kernel) {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        RNNT_MAX_TOP_VOCAB / 8) == cudaSuccess;
        };
        return raise(k_distill_long<float>) && raise(k_distill_long<__half>) &&
               raise(k_distill_long<__nv_bfloat16>);
    });
}

}  // namespace

extern "C" rnnt_status_t rnnt_top_logits(const void* logits, rnnt_dtype_t dt, int64_t rows,
                                         int32_t V, const int32_t* logit_lengths,
                                         const int32_t* target_lengths, int32_t B, int32_t max_T,
                                         int32_t max_U, int32_t k, double temperature,
                                         void* values, int32_t* ids, float* rest,
                                         int32_t* status_dev, rnnt_stream_t stream) {
    TopParams p{};
    p.lat = Lattice{logit_lengths, target_lengths, rows, B, 1, max_T, max_U};
    if (!logits || !values || !ids || !rest || !valid_dtype(dt) || V < 1 ||
        V > RNNT_MAX_TOP_VOCAB || k < 1 || k > RNNT_MAX_TOP || k > V ||
        !temperature_ok(temperature) || !lattice_ok(p.lat))
        return RNNT_INVALID_VALUE;
    const int es = elem_size(dt);
    const int64_t in = bytes_of(rows, V, es), out = bytes_of(rows, k, 4);
    if (in < 0 || out < 0 || ((uintptr_t)logits | (uintptr_t)values) % es ||
        ((uintptr_t)ids | (uintptr_t)rest | (uintptr_t)status_dev) & 3)
        return RNNT_INVALID_VALUE;
    const void* outs[3] = {values, ids, rest};
    const uint64_t sizes[3] = {(uint64_t)rows * k * es, (uint64_t)out, (uint64_t)rows * 4};
    for (int i = 0; i < 3; ++i) {
        if (overlaps(outs[i], sizes[i], logits, in)) return RNNT_INVALID_VALUE;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], sizes[i], outs[j], sizes[j])) return RNNT_INVALID_VALUE;
    }
    p.logits = static_cast<const char*>(logits);
    p.V = V;
    p.k = k;
    p.scale = (float)(kLog2e / temperature);
    p.inv_tau = (float)(1.0 / temperature);
    p.values = values;
    p.ids = ids;
    p.rest = rest;
    p.status = status_dev;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    with_type(dt, [&](auto t) {
        k_top_long<decltype(t)><<<row_grid(rows), kLongThreads, 0, st>>>(p);
    });
    return launched();
}

extern "C" rnnt_status_t rnnt_distill_workspace_size(int32_t B, int64_t rows, size_t* bytes) {
    if (!bytes || B < 1 || rows < 1 || rows > (INT64_MAX >> 8)) return RNNT_INVALID_VALUE;
    *bytes = distill_layout(B, rows).total;
    return RNNT_OK;
}

extern "C" rnnt_status_t rnnt_distill_loss(
    const void* logits, rnnt_dtype_t dt, int64_t rows, int32_t V, const void* teacher_logits,
    rnnt_dtype_t teacher_dt, const int32_t* teacher_ids, const float* teacher_rest, int32_t k,
    const int32_t* logit_lengths, const int32_t* target_lengths, int32_t B, int32_t padded,
    int32_t max_T, int32_t max_U, double temperature, double weight, rnnt_reduction_t reduction,
    float* loss, float* loss_reduced, void* grad, void* workspace, size_t workspace_bytes,
    int32_t* status_dev, rnnt_stream_t stream) {
    DistillParams p{};
    p.lat = Lattice{logit_lengths, target_lengths, rows, B, padded ? 1 : 0, max_T, max_U};
    if (!logits || !teacher_logits || !teacher_ids || !logit_lengths || !target_lengths || !loss ||
        !workspace || !valid_dtype(dt) || !valid_dtype(teacher_dt) || V < 1 ||
        V > RNNT_MAX_TOP_VOCAB || k < 1 || k > RNNT_MAX_TOP || !temperature_ok(temperature) ||
        !(weight > -1e30 && weight < 1e30) || (int)reduction < 0 ||
        (int)reduction > RNNT_RED_MEAN || !lattice_ok(p.lat))
        return RNNT_INVALID_VALUE;
    const int es = elem_size(dt);
    const int64_t in = bytes_of(rows, V, es), places = bytes_of(rows, k, 4);
    if (in < 0 || places < 0 || ((uintptr_t)logits | (uintptr_t)grad) & 15 ||
        (uintptr_t)teacher_logits % elem_size(teacher_dt) || ((uintptr_t)workspace & 255) ||
        ((uintptr_t)teacher_ids | (uintptr_t)teacher_rest | (uintptr_t)loss |
         (uintptr_t)loss_reduced | (uintptr_t)status_dev) & 3)
        return RNNT_INVALID_VALUE;
    const DistillLayout L = distill_layout(B, rows);
    if (workspace_bytes < L.total) return RNNT_WORKSPACE_TOO_SMALL;
    const void* outs[4] = {loss, workspace, grad, loss_reduced};
    const uint64_t out_sizes[4] = {(uint64_t)B * 4, L.total, (uint64_t)in, 4};
    const void* ins[6] = {logits, teacher_logits, teacher_ids, teacher_rest, logit_lengths,
                          target_lengths};
    const uint64_t in_sizes[6] = {(uint64_t)in, (uint64_t)rows * k * elem_size(teacher_dt),
                                  (uint64_t)places, (uint64_t)rows * 4, (uint64_t)B * 4,
                                  (uint64_t)B * 4};
    for (int i = 0; i < 4; ++i) {
        if (!outs[i]) continue;
        for (int j = 0; j < 6; ++j)
            if (ins[j] && overlaps(outs[i], out_sizes[i], ins[j], in_sizes[j]))
                return RNNT_INVALID_VALUE;
        for (int j = 0; j < i; ++j)
            if (outs[j] && overlaps(outs[i], out_sizes[i], outs[j], out_sizes[j]))
                return RNNT_INVALID_VALUE;
    }
    char* const ws = static_cast<char*>(workspace);
    p.logits = static_cast<const char*>(logits);
    p.teacher = static_cast<const char*>(teacher_logits);
    p.teacher_dt = teacher_dt;
    p.ids = teacher_ids;
    p.rest = teacher_rest;
    p.V = V;
    p.k = k;
    p.scale = (float)(kLog2e / temperature);
    p.inv_tau = (float)(1.0 / temperature);
    p.mean = reduction == RNNT_RED_MEAN;
    p.grad_scale = (float)(temperature * weight / (p.mean ? B : 1));
    p.loss_scale = temperature * temperature * weight;
    p.grad = static_cast<char*>(grad);
    p.row_loss = reinterpret_cast<float*>(ws + L.row_loss);
    p.sample_loss = reinterpret_cast<double*>(ws + L.sample_loss);
    p.first_row = reinterpret_cast<int64_t*>(ws + L.first_row);
    p.done = reinterpret_cast<int32_t*>(ws + L.done);
    p.loss = loss;
    p.loss_reduced = loss_reduced;
    p.status = status_dev;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!distill_prepared() || !clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    with_type(dt, [&](auto t) {
        k_distill_long<decltype(t)>
            <<<row_grid(rows), kLongThreads, (size_t)(V + 31) / 32 * 4, st>>>(p);
    });
    if (launched() != RNNT_OK) return RNNT_LAUNCH_FAILED;
    if (!launch_after(k_distill_sum, dim3((unsigned)B), kSumThreads, 0, st, p)) {
        cudaGetLastError();
        return RNNT_LAUNCH_FAILED;
    }
    return RNNT_OK;
}

extern "C" rnnt_status_t rnnt_distill_grad_scale(void* grad, rnnt_dtype_t dt, int64_t rows,
                                                 int32_t V, int32_t B, int64_t rows_each,
                                                 const void* workspace, size_t workspace_bytes,
                                                 const float* factors, int32_t per_sample,
                                                 rnnt_stream_t stream) {
    if (!grad || !workspace || !factors || !valid_dtype(dt) || rows < 1 || V < 1 ||
        V > RNNT_MAX_TOP_VOCAB || B < 1 || rows_each < 0 ||
        (rows_each && (rows_each > rows || rows % rows_each || rows / rows_each != B)) ||
        bytes_of(rows, V, 4) < 0 || ((uintptr_t)grad & 15) || ((uintptr_t)workspace & 255) ||
        ((uintptr_t)factors & 3))
        return RNNT_INVALID_VALUE;
    if (workspace_bytes < distill_layout(B, rows).total) return RNNT_WORKSPACE_TOO_SMALL;
    ScaleParams p{};
    p.grad = static_cast<char*>(grad);
    p.factors = factors;
    p.first_row = static_cast<const int64_t*>(workspace);
    p.rows = rows;
    p.each = rows_each;
    p.V = V;
    p.B = B;
    p.per_sample = per_sample ? 1 : 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    with_type(dt, [&](auto t) {
        k_distill_scale<decltype(t)><<<row_grid(rows), 256, 0, st>>>(p);
    });
    return launched();
}
