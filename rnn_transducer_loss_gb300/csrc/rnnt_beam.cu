// rnnt_beam.cu -- beam search: selection over beams and vocabulary, and the
// reordering of states by the selected beams.
//
// Selection.  A live beam k with score s_k and logits x_k offers, for every
// output v with x_kv > -inf, the candidate s_k + x_kv - lse(x_k) (lse = 0 for
// log-probabilities); a finished beam offers itself, with its score and token
// -1; a beam of score -inf offers nothing.  The Ko best of a batch item are
// selected, ties going to the lowest beam and then the lowest token.
#include "rnnt_labels.cuh"

using namespace rnnt_labels;

namespace {

// ------------------------------------------------- order-preserving integers
__device__ __forceinline__ uint32_t ordered(float x) {      // -0 counts as 0
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double unordered(uint64_t o) {
    return __longlong_as_double((long long)(o ^ ((o >> 63) ? 1ull << 63 : ~0ull)));
}

// ------------------------------------------------------ segments of the rows
// A row is cut into segments of at most kRowThreads * kRowVecs 16-byte vectors
// (counted from the row's first address rounded down to 16); a CTA holds one
// segment in registers, and writes its maximum, its sum of exponentials and its
// n best elements in order.
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowVecs = 8;
constexpr int kBuf = 4096;                 // > (RNNT_MAX_BEAM - 1) * 64 + 1, see below

struct SelectParams {
    const char* logits;
    int64_t batch_stride, beam_stride;     // bytes
    const float* scores;
    const uint8_t* finished;
    int32_t B, K, V, Ko, fused;
    int32_t segs, seg_vecs;                // segments of a row, vectors of a segment
    int32_t n;                             // elements a segment lists: min(Ko, V)
    double2* stat;                         // [row][seg]: maximum, sum of exp(x - maximum)
    uint64_t* list;                        // [row][seg][n]: ordered value << 32 | ~element
    float* out_scores;
    int32_t* out_tokens;
    int32_t* out_parents;
    int32_t* status;
};

// Whether beam `row` offers its logits' candidates.
__device__ __forceinline__ bool reads_logits(const SelectParams& p, int64_t row) {
    if (p.finished && p.finished[row]) return false;
    const float s = p.scores[row];
    return s > -INFINITY && s < INFINITY;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_rows(const SelectParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    __shared__ uint64_t buf[kBuf];
    __shared__ uint64_t tops[kRowWarps][32];
    __shared__ float wmax[kRowWarps];
    __shared__ double wsum[kRowWarps];
    __shared__ int bads, count;
    __shared__ uint64_t bound;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / p.segs;
    const int seg = (int)(blockIdx.x - row * p.segs);
    if (!reads_logits(p, row)) return;
    const int64_t b = row / p.K;
    const char* first = p.logits + b * p.batch_stride + (row - b * p.K) * p.beam_stride;
    const int head = (int)((uintptr_t)first & 15) / (int)sizeof(T);
    const T* x0 = reinterpret_cast<const T*>(first);

    // Elements outside the row read as -inf; a vector that is partly outside
    // is read element by element.
    Pack<T, 16> v[kRowVecs];
    const int vec0 = seg * p.seg_vecs;
    const int vecs = min(p.seg_vecs, (p.V + head + E - 1) / E - vec0);
#pragma unroll
    for (int i = 0; i < kRowVecs; ++i) {
        const int j = i * kRowThreads + tid;
        const int e0 = (vec0 + j) * E - head;
        if (j < vecs && e0 >= 0 && e0 + E <= p.V) {
            v[i].raw = __ldg(reinterpret_cast<const uint4*>(x0 + e0));
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[i].e[e] = j < vecs && e0 + e >= 0 && e0 + e < p.V ? x0[e0 + e]
                                                                     : from_f32<T>(-INFINITY);
        }
    }
    if (tid == 0) {
        bads = 0;
        count = 0;
        bound = 1;      // every element above -inf
    }
    // The thread's best element, ties to the lowest.
    bool bad = false;
    uint32_t best = 0;
    int where = 0;
#pragma unroll
    for (int i = 0; i < kRowVecs; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float x = to_f32(v[i].e[e]);
            bad |= !(x < INFINITY);
            const uint32_t o = ordered(x);
            if (x > -INFINITY && o > best) {
                best = o;
                where = (vec0 + i * kRowThreads + tid) * E - head + e;
            }
        }
    }
    uint64_t key = best ? (uint64_t)best << 32 | (uint32_t)~where : 0;
    float m = best ? unordered(best) : -INFINITY;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // The warp's bests in descending order (bitonic), then each one's rank
    // among all warps': the n-th best of the threads' bests bounds the n-th
    // best element from below, and at most (n - 1) * 64 + 1 elements reach it.
#pragma unroll
    for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
        for (int o = size / 2; o; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
            const bool larger = ((lane & o) == 0) == ((lane & size) == 0 || size == 32);
            if (larger == (other > key)) key = other;
        }
    }
    tops[warp][lane] = key;
    if (lane == 0) wmax[warp] = m;
    __syncthreads();
    if (bad) bads = 1;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) m = fmaxf(m, wmax[w]);
    if (key) {
        int rank = lane;
        for (int w = 0; w < kRowWarps; ++w) {
            if (w == warp) continue;
            int lo = 0;      // tops[w] entries above key
#pragma unroll
            for (int step = 16; step; step >>= 1)
                if (tops[w][lo + step - 1] > key) lo += step;
            if (lo == 31 && tops[w][31] > key) lo = 32;
            rank += lo;
        }
        if (rank == p.n - 1) bound = key;
    }
    // Sum of exponentials.
    double s = 0.0;
    if (p.fused && m > -INFINITY) {
#pragma unroll
        for (int i = 0; i < kRowVecs; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = to_f32(v[i].e[e]);
                if (x > -INFINITY) s += exp((double)x - (double)m);
            }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) wsum[warp] = s;
    }
    __syncthreads();
    const uint64_t at_least = bound;
#pragma unroll
    for (int i = 0; i < kRowVecs; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float x = to_f32(v[i].e[e]);
            const int at = (vec0 + i * kRowThreads + tid) * E - head + e;
            const uint64_t c = (uint64_t)ordered(x) << 32 | (uint32_t)~at;
            if (x > -INFINITY && c >= at_least) {
                const int to = atomicAdd(&count, 1);
                if (to < kBuf) buf[to] = c;
            }
        }
    __syncthreads();
    const int64_t unit = row * p.segs + seg;
    if (tid == 0) {
        double sum = 0.0;
        if (p.fused && m > -INFINITY)
            for (int w = 0; w < kRowWarps; ++w) sum += wsum[w];
        p.stat[unit] = make_double2(bads ? nan("") : (double)m, sum);
    }
    const int c = min(count, kBuf);
    uint64_t* list = p.list + unit * p.n;
    for (int i = tid; i < c; i += kRowThreads) {
        const uint64_t mine = buf[i];
        int rank = 0;
        for (int j = 0; j < c; ++j) rank += buf[j] > mine;
        if (rank < p.n) list[rank] = mine;
    }
    for (int i = c + tid; i < p.n; i += kRowThreads) list[i] = 0;
}

// --------------------------------------------------------- the Ko best of all
// One CTA per batch item: every (beam, segment) list is in order, so the best
// candidate is among the lists' heads; Ko rounds of a maximum over them.
constexpr int kPickThreads = 256;
constexpr int kPickWarps = kPickThreads / 32;

__global__ void __launch_bounds__(kPickThreads) k_pick(const SelectParams p) {
    extern __shared__ uint8_t taken[];                 // [K * segs]: candidates used
    __shared__ double lse[RNNT_MAX_BEAM];
    __shared__ float score[RNNT_MAX_BEAM];
    __shared__ uint8_t kind[RNNT_MAX_BEAM];            // 0 nothing, 1 logits, 2 finished
    __shared__ uint64_t wval[kPickWarps];
    __shared__ uint32_t wid[kPickWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.x;
    const int lists = p.K * p.segs;
    if (tid < p.K) {
        const int64_t row = b * p.K + tid;
        const float s = p.scores[row];
        const bool done = p.finished && p.finished[row];
        bool bad = !(s < INFINITY);
        int what = bad || s == -INFINITY ? 0 : done ? 2 : 1;
        double l = 0.0;
        if (what == 1) {
            const double2* st = p.stat + row * p.segs;
            double top = -INFINITY, sum = 0.0;
            bool nans = false;
            for (int g = 0; g < p.segs; ++g) {
                nans |= st[g].x != st[g].x;
                top = fmax(top, st[g].x);
            }
            if (nans || top == -INFINITY) {
                what = 0;
                bad |= nans;
            } else if (p.fused) {
                for (int g = 0; g < p.segs; ++g)
                    if (st[g].x > -INFINITY) sum += st[g].y * exp(st[g].x - top);
                l = top + log(sum);
            }
        }
        if (bad && p.status) *p.status = RNNT_INVALID_VALUE;
        lse[tid] = l;
        score[tid] = s;
        kind[tid] = (uint8_t)what;
    }
    for (int i = tid; i < lists; i += kPickThreads) taken[i] = 0;
    __syncthreads();
    // Value (0: none) and number (beam * V + token) of list i's head.
    auto headof = [&](int i, uint64_t& val, uint32_t& id) {
        const int k = i / p.segs, g = i - k * p.segs, at = taken[i];
        val = 0;
        id = 0xffffffffu;
        if (kind[k] == 2) {
            if (g == 0 && at == 0) {
                val = ordered((double)score[k]);
                id = (uint32_t)k * (uint32_t)p.V;
            }
        } else if (kind[k] == 1 && at < p.n) {
            const uint64_t c = __ldcg(p.list + ((b * p.K + k) * p.segs + g) * p.n + at);
            if (c) {
                val = ordered((double)score[k] + ((double)unordered((uint32_t)(c >> 32)) - lse[k]));
                id = (uint32_t)k * (uint32_t)p.V + ~(uint32_t)c;
            }
        }
    };
    uint64_t val = 0;
    uint32_t id = 0xffffffffu;
    int list = -1;
    auto best = [&]() {
        val = 0;
        id = 0xffffffffu;
        list = -1;
        for (int i = tid; i < lists; i += kPickThreads) {
            uint64_t v;
            uint32_t d;
            headof(i, v, d);
            if (v > val || (v == val && d < id)) {
                val = v;
                id = d;
                list = i;
            }
        }
    };
    best();
    for (int r = 0; r < p.Ko; ++r) {
        uint64_t v = val;
        uint32_t d = id;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const uint64_t ov = __shfl_xor_sync(0xffffffffu, v, o);
            const uint32_t od = __shfl_xor_sync(0xffffffffu, d, o);
            if (ov > v || (ov == v && od < d)) {
                v = ov;
                d = od;
            }
        }
        if (lane == 0) {
            wval[warp] = v;
            wid[warp] = d;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kPickWarps; ++w)
            if (wval[w] > v || (wval[w] == v && wid[w] < d)) {
                v = wval[w];
                d = wid[w];
            }
        if (v && v == val && d == id) {
            const int k = list / p.segs;
            const int64_t o = b * p.Ko + r;
            p.out_scores[o] = (float)unordered(v);
            p.out_tokens[o] = kind[k] == 2 ? -1 : (int)(d - (uint32_t)k * (uint32_t)p.V);
            p.out_parents[o] = k;
            ++taken[list];
            best();
        } else if (!v && tid == 0) {
            const int64_t o = b * p.Ko + r;
            p.out_scores[o] = -INFINITY;
            p.out_tokens[o] = -1;
            p.out_parents[o] = -1;
        }
        __syncthreads();
    }
}

struct SelectLayout {
    size_t stat, list, total;
    int32_t segs, seg_vecs, n;
};
SelectLayout select_layout(int32_t B, int32_t K, int32_t V, int32_t Ko, int dt) {
    SelectLayout L;
    const int E = 16 / elem_size(dt);
    const int64_t vecs = ((int64_t)V + 2 * (E - 1)) / E;      // the most, whatever the alignment
    L.seg_vecs = kRowThreads * kRowVecs;
    L.segs = (int32_t)((vecs + L.seg_vecs - 1) / L.seg_vecs);
    L.n = std::min(Ko, V);
    const size_t units = (size_t)B * K * L.segs;
    L.stat = 0;
    L.list = align256(units * sizeof(double2));
    L.total = align256(L.list + units * L.n * sizeof(uint64_t));
    return L;
}
bool select_ok(int32_t B, int32_t K, int32_t V, int32_t Ko, int dt) {
    return B >= 1 && K >= 1 && K <= RNNT_MAX_BEAM && Ko >= 1 && Ko <= RNNT_MAX_BEAM && V >= 1 &&
           V <= RNNT_MAX_BEAM_VOCAB && valid_dtype(dt) &&
           (int64_t)B * K * select_layout(B, K, V, Ko, dt).segs <= INT32_MAX;
}

// ------------------------------------------------------------------ reorder
// Every state is a set of rows (three outer axes, batch, new beam) of
// contiguous bytes.  A CTA copies kCopyUnits units: several short rows, or a
// piece of a long one.
constexpr int kCopyThreads = 256;
constexpr int kCopyEach = 4;
constexpr int kCopyUnits = kCopyThreads * kCopyEach;

struct CopyState {
    rnnt_state_t s;
    int64_t rows_all;        // rows of the state
    int32_t nunits;          // units of a row
    int32_t unit;            // bytes of a unit
    int32_t rows, pieces;    // rows of a CTA, CTAs of a row
    uint32_t inv;
    uint32_t cta0;           // first CTA
};
struct CopyParams {
    CopyState st[RNNT_MAX_STATES];
    int32_t states, B, K, Ko;
    const int32_t* parents;
    int32_t* status;
};

template <int UB>
__device__ __forceinline__ void copy_tile(const CopyState& s, int total, int u0, int rows1,
                                          const int64_t* from, const int64_t* to) {
    using U = typename Unit<UB>::type;
    U v[kCopyEach];
#pragma unroll
    for (int i = 0; i < kCopyEach; ++i) {
        const int u = u0 + threadIdx.x + i * kCopyThreads;
        v[i] = U{};
        if (u < total) {
            const int r = rows1 ? 0 : s.nunits == 1 ? u : (int)__umulhi((uint32_t)u, s.inv);
            if (from[r] >= 0)
                v[i] = __ldg(reinterpret_cast<const U*>(static_cast<const char*>(s.s.src) +
                                                        from[r]) + (u - r * s.nunits));
        }
    }
#pragma unroll
    for (int i = 0; i < kCopyEach; ++i) {
        const int u = u0 + threadIdx.x + i * kCopyThreads;
        if (u >= total) break;
        const int r = rows1 ? 0 : s.nunits == 1 ? u : (int)__umulhi((uint32_t)u, s.inv);
        reinterpret_cast<U*>(static_cast<char*>(s.s.dst) + to[r])[u - r * s.nunits] = v[i];
    }
}

__global__ void __launch_bounds__(kCopyThreads) k_reorder(const __grid_constant__ CopyParams p) {
    __shared__ int64_t from[kCopyThreads], to[kCopyThreads];
    int i = 0;
    while (i + 1 < p.states && blockIdx.x >= p.st[i + 1].cta0) ++i;
    const CopyState& s = p.st[i];
    const uint32_t cta = blockIdx.x - s.cta0;
    const int64_t tile = cta / (uint32_t)s.pieces;
    const int piece = (int)(cta - tile * s.pieces);
    const int64_t row0 = tile * s.rows;
    const int rows = (int)min((int64_t)s.rows, s.rows_all - row0);
    if (threadIdx.x < rows) {
        int64_t r = row0 + threadIdx.x;                // ((n0, n1), batch, beam, n2) row-major
        int64_t q = r / s.s.n[2];
        const int64_t i2 = r - q * s.s.n[2];
        r = q / p.Ko;
        const int64_t k = q - r * p.Ko;
        q = r / p.B;
        const int64_t b = r - q * p.B;
        const int64_t i0 = q / s.s.n[1], i1 = q - i0 * s.s.n[1];
        const int parent = __ldg(p.parents + b * p.Ko + k);
        if ((parent < -1 || parent >= p.K) && p.status) *p.status = RNNT_INVALID_VALUE;
        from[threadIdx.x] = parent < 0 || parent >= p.K ? -1
            : i0 * s.s.src_stride[0] + i1 * s.s.src_stride[1] + i2 * s.s.src_stride[2] +
              b * s.s.src_batch + parent * s.s.src_beam;
        to[threadIdx.x] = i0 * s.s.dst_stride[0] + i1 * s.s.dst_stride[1] +
                          i2 * s.s.dst_stride[2] + b * s.s.dst_batch + k * s.s.dst_beam;
    }
    __syncthreads();
    const int total = s.pieces > 1 ? s.nunits : rows * s.nunits;
    const int u0 = piece * kCopyUnits;
    const int rows1 = s.rows == 1;
    switch (s.unit) {
        case 16: copy_tile<16>(s, total, u0, rows1, from, to); break;
        case 8: copy_tile<8>(s, total, u0, rows1, from, to); break;
        case 4: copy_tile<4>(s, total, u0, rows1, from, to); break;
        case 2: copy_tile<2>(s, total, u0, rows1, from, to); break;
        default: copy_tile<1>(s, total, u0, rows1, from, to); break;
    }
}

// Bytes from the first to the last that a state's rows reach (strides are not negative).
uint64_t extent(const rnnt_state_t& s, const int64_t* stride, int64_t batch, int64_t beam,
                int64_t B, int64_t beams) {
    uint64_t n = (uint64_t)s.row_bytes + (uint64_t)(B - 1) * batch + (uint64_t)(beams - 1) * beam;
    for (int i = 0; i < 3; ++i) n += (uint64_t)(s.n[i] - 1) * stride[i];
    return n;
}

}  // namespace

extern "C" rnnt_status_t rnnt_beam_workspace_size(int32_t B, int32_t K, int32_t V, int32_t Ko,
                                                  rnnt_dtype_t dt, size_t* bytes) {
    if (!bytes || !select_ok(B, K, V, Ko, dt)) return RNNT_INVALID_VALUE;
    *bytes = select_layout(B, K, V, Ko, dt).total;
    return RNNT_OK;
}

extern "C" rnnt_status_t rnnt_beam_select(const void* logits, rnnt_dtype_t dt, int32_t B, int32_t K,
                                          int32_t V, int64_t batch_stride, int64_t beam_stride,
                                          const float* scores, const uint8_t* finished, int32_t Ko,
                                          int32_t fused_log_softmax, float* out_scores,
                                          int32_t* out_tokens, int32_t* out_parents,
                                          void* workspace, size_t workspace_bytes,
                                          int32_t* status_dev, rnnt_stream_t stream) {
    if (!logits || !scores || !out_scores || !out_tokens || !out_parents || !workspace)
        return RNNT_INVALID_VALUE;
    if (!select_ok(B, K, V, Ko, dt) || batch_stride < 0 || beam_stride < 0)
        return RNNT_INVALID_VALUE;
    const int es = elem_size(dt);
    if (((uintptr_t)logits & (es - 1)) || ((uintptr_t)workspace & 255)) return RNNT_INVALID_VALUE;
    const SelectLayout L = select_layout(B, K, V, Ko, dt);
    if (workspace_bytes < L.total) return RNNT_WORKSPACE_TOO_SMALL;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    SelectParams p{};
    p.logits = static_cast<const char*>(logits);
    p.batch_stride = batch_stride * es;
    p.beam_stride = beam_stride * es;
    p.scores = scores;
    p.finished = finished;
    p.B = B;
    p.K = K;
    p.V = V;
    p.Ko = Ko;
    p.fused = fused_log_softmax ? 1 : 0;
    p.segs = L.segs;
    p.seg_vecs = L.seg_vecs;
    p.n = L.n;
    p.stat = reinterpret_cast<double2*>(ws + L.stat);
    p.list = reinterpret_cast<uint64_t*>(ws + L.list);
    p.out_scores = out_scores;
    p.out_tokens = out_tokens;
    p.out_parents = out_parents;
    p.status = status_dev;
    if (!clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    with_type(dt, [&](auto tag) {
        k_rows<decltype(tag)><<<(unsigned)(B * K * L.segs), kRowThreads, 0, st>>>(p);
        return 0;
    });
    k_pick<<<(unsigned)B, kPickThreads, (size_t)K * L.segs, st>>>(p);
    return launched();
}

extern "C" rnnt_status_t rnnt_beam_reorder(const rnnt_state_t* states, int32_t n_states,
                                           const int32_t* parents, int32_t B, int32_t K, int32_t Ko,
                                           int32_t* status_dev, rnnt_stream_t stream) {
    if (!states || n_states < 1 || n_states > RNNT_MAX_STATES || !parents || B < 1 || K < 1 ||
        Ko < 1)
        return RNNT_INVALID_VALUE;
    CopyParams p;
    int64_t ctas = 0;
    for (int i = 0; i < n_states; ++i) {
        const rnnt_state_t& s = states[i];
        if (!s.src || !s.dst || s.row_bytes < 1 || s.src_batch < 0 || s.src_beam < 0 ||
            s.dst_batch < 0 || s.dst_beam < 0)
            return RNNT_INVALID_VALUE;
        if ((B > 1 && s.dst_batch == 0) || (Ko > 1 && s.dst_beam == 0)) return RNNT_INVALID_VALUE;
        uint64_t bits = (uintptr_t)s.src | (uintptr_t)s.dst | (uint64_t)s.row_bytes;
        // an axis of one element has no stride
        if (B > 1) bits |= (uint64_t)s.src_batch | (uint64_t)s.dst_batch;
        if (K > 1) bits |= (uint64_t)s.src_beam;
        if (Ko > 1) bits |= (uint64_t)s.dst_beam;
        int64_t rows = (int64_t)B * Ko;
        for (int a = 0; a < 3; ++a) {
            if (s.n[a] < 1 || s.src_stride[a] < 0 || s.dst_stride[a] < 0) return RNNT_INVALID_VALUE;
            if (s.n[a] > 1 && s.dst_stride[a] == 0) return RNNT_INVALID_VALUE;
            if (s.n[a] > 1) bits |= (uint64_t)s.src_stride[a] | (uint64_t)s.dst_stride[a];
            if (rows > INT64_MAX / s.n[a]) return RNNT_INVALID_VALUE;
            rows *= s.n[a];
        }
        CopyState& c = p.st[i];
        c.s = s;
        c.rows_all = rows;
        c.unit = unit_of(bits);
        if (s.row_bytes / c.unit > INT32_MAX - kCopyUnits) return RNNT_INVALID_VALUE;
        c.nunits = (int32_t)(s.row_bytes / c.unit);
        c.rows = std::max(1, std::min(kCopyThreads, kCopyUnits / c.nunits));
        c.pieces = (c.nunits + kCopyUnits - 1) / kCopyUnits;
        c.inv = (uint32_t)(((1ull << 32) + c.nunits - 1) / c.nunits);
        c.cta0 = (uint32_t)ctas;
        const int64_t tiles = (rows + c.rows - 1) / c.rows;
        if (tiles > INT32_MAX / c.pieces) return RNNT_INVALID_VALUE;
        ctas += tiles * c.pieces;
        if (ctas > INT32_MAX) return RNNT_INVALID_VALUE;
    }
    for (int i = 0; i < n_states; ++i)
        for (int j = 0; j < n_states; ++j) {
            const rnnt_state_t &d = states[i], &s = states[j];
            const uint64_t dn = extent(d, d.dst_stride, d.dst_batch, d.dst_beam, B, Ko);
            if (overlaps(d.dst, dn, s.src,
                         extent(s, s.src_stride, s.src_batch, s.src_beam, B, K)))
                return RNNT_INVALID_VALUE;
        }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    p.states = n_states;
    p.B = B;
    p.K = K;
    p.Ko = Ko;
    p.parents = parents;
    p.status = status_dev;
    if (!clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    k_reorder<<<(unsigned)ctas, kCopyThreads, 0, st>>>(p);
    return launched();
}
