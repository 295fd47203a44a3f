// rnnt_beam.cu -- beam search: selection over beams and vocabulary, and the
// reordering of states by the selected beams.
//
// Selection.  A live beam k with score s_k and logits x_k offers, for every
// output v with x_kv > -inf, the candidate s_k + x_kv - lse(x_k) (lse = 0 for
// log-probabilities); a finished beam offers itself, with its score and token
// -1; a beam of score -inf offers nothing.  The Ko best of a batch item are
// selected, ties going to the lowest beam and then the lowest token.
#include <atomic>

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

// ------------------------------------------------------------- rows of logits
// A row is cut into splits of 16-byte vectors (counted from the row's first
// address rounded down to 16); a CTA streams one split through registers in tiles
// of kRowThreads * NV vectors, the next tile's loads in flight, and writes
//   - the sum of exp(x - r) over the split and its reference r.  r is the first tile's
//     maximum and changes only when a thread meets a value more than 16 above it, so
//     that the running sum is (almost) never rescaled.
//   - the n best elements in order.  The first tile's n-th best of the threads' bests
//     bounds the n-th best element from below; later tiles only look for elements above
//     the bound (one comparison a thread and tile, with the tile's maximum).
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr float kLog2e = 1.44269504f;      // log2 e to 2^-26
constexpr float kRescale = 16.0f;
constexpr float kMostRef = 1e30f;          // larger references: computed again by exact_lse
constexpr int kMaxLists = 256;             // splits of a batch item's rows
constexpr int kBuf = 2560;                 // > RNNT_MAX_BEAM + (RNNT_MAX_BEAM - 1) * 32 + 1
constexpr int kCrowd = 256;                // elements from which the buffer is cut to the n best

struct SelectParams {
    const char* logits;
    int64_t batch_stride, beam_stride;     // bytes
    const float* scores;
    const uint8_t* finished;
    int32_t B, K, V, Ko, fused;
    int32_t splits, split_vecs;            // splits of a row, vectors of a split
    int32_t n;                             // elements a split lists: min(Ko, V)
    double2* stat;                         // [row][split]: reference, sum of exp(x - reference)
                                           // (negative if it was rescaled)
    uint64_t* list;                        // [row][split][n]: ordered value << 32 | ~element
    float* out_scores;
    int32_t* out_tokens;
    int32_t* out_parents;
    int32_t* status;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A pair of floats whose exact sum is the value: about 47 bits, on float32 units (of which
// there are 64 times as many as of float64 ones).
struct Pair { float h, l; };
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair fast_two_sum(float a, float b) {       // |a| >= |b|
    const float s = a + b;
    return {s, b - (s - a)};
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    const float h = a.h * b.h;
    return fast_two_sum(h, __fmaf_rn(a.h, b.h, -h) + (a.h * b.l + a.l * b.h));
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const Pair s = two_sum(a.h, b.h);
    return fast_two_sum(s.h, s.l + (a.l + b.l));
}

// Whether beam `row` offers its logits' candidates.
__device__ __forceinline__ bool reads_logits(const SelectParams& p, int64_t row) {
    if (p.finished && p.finished[row]) return false;
    const float s = p.scores[row];
    return s > -INFINITY && s < INFINITY;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const SelectParams& p, int64_t row) {
    const int64_t b = row / p.K;
    return reinterpret_cast<const T*>(p.logits + b * p.batch_stride +
                                      (row - b * p.K) * p.beam_stride);
}

// Rank of the thread's key among the block's (0: none, returns kRowThreads): the warps sort
// theirs (bitonic) and each key is searched for in the other warps' orders.
__device__ __forceinline__ int block_rank(uint64_t key, uint64_t (*order)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
        for (int o = size / 2; o; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
            const bool larger = ((lane & o) == 0) == ((lane & size) == 0 || size == 32);
            if (larger == (other > key)) key = other;
        }
    }
    order[warp][lane] = key;      // descending: this thread now stands for another's key
    __syncthreads();
    if (!key) return kRowThreads;
    int rank = lane;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
        if (w == warp) continue;
        int lo = 0;
#pragma unroll
        for (int step = 16; step; step >>= 1)
            if (order[w][lo + step - 1] > key) lo += step;
        if (lo == 31 && order[w][31] > key) lo = 32;
        rank += lo;
    }
    return rank;
}

// Keeps the n best of the buffer's keys, in order; all threads call it.
__device__ __noinline__ void keep_best(uint64_t* buf, uint64_t* best, int* count, int n) {
    const int c = *count;
    for (int i = threadIdx.x; i < c; i += kRowThreads) {
        const uint64_t mine = buf[i];
        int rank = 0;
        for (int j = 0; j < c; ++j) rank += buf[j] > mine;
        if (rank < n) best[rank] = mine;
    }
    __syncthreads();
    const int m = min(c, n);
    if (threadIdx.x < m) buf[threadIdx.x] = best[threadIdx.x];
    if (threadIdx.x == 0) *count = m;
    __syncthreads();
}

// Elements [e0, e0 + 16 bytes) of a row of V; those outside it are -inf.
template <typename T>
__device__ __noinline__ uint4 load_partly(const T* x0, int e0, int V) {
    constexpr int E = 16 / (int)sizeof(T);
    Pack<T, 16> v;
#pragma unroll
    for (int e = 0; e < E; ++e)
        v.e[e] = e0 + e >= 0 && e0 + e < V ? x0[e0 + e] : from_f32<T>(-INFINITY);
    return v.raw;
}

// Largest element of a vector (NaN is passed over).
__device__ __forceinline__ float vec_max(const Pack<float, 16>& v) {
    return fmaxf(fmaxf(v.e[0], v.e[1]), fmaxf(v.e[2], v.e[3]));
}
__device__ __forceinline__ float vec_max(const Pack<__half, 16>& v) {
    const __half2* h = reinterpret_cast<const __half2*>(&v.raw);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float vec_max(const Pack<__nv_bfloat16, 16>& v) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v.raw);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}

template <typename T, int NV, bool FUSED>
__global__ void __launch_bounds__(kRowThreads, 4) k_rows(const SelectParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    constexpr int kTileVecs = kRowThreads * NV;
    __shared__ uint64_t buf[kBuf], best[RNNT_MAX_BEAM];
    __shared__ uint64_t order[kRowWarps][32];
    __shared__ Pair wsum[kRowWarps];
    __shared__ float wmax[kRowWarps];
    __shared__ int count;
    __shared__ uint64_t bound;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / p.splits;
    const int split = (int)(blockIdx.x - row * p.splits);
    if (!reads_logits(p, row)) return;
    const T* x0 = row_of<T>(p, row);
    const int head = (int)((uintptr_t)x0 & 15) / (int)sizeof(T);
    const int vec0 = split * p.split_vecs;
    const int vecs = max(0, min(p.split_vecs, (p.V + head + E - 1) / E - vec0));
    Pack<T, 16> none;
#pragma unroll
    for (int e = 0; e < E; ++e) none.e[e] = from_f32<T>(-INFINITY);

    // Vector j of the split; elements outside the row and the split read as -inf.
    auto load = [&](Pack<T, 16>& v, int j) {
        const int e0 = (vec0 + j) * E - head;
        v.raw = none.raw;
        if (j < vecs) {
            if (e0 >= 0 && e0 + E <= p.V) v.raw = __ldg(reinterpret_cast<const uint4*>(x0 + e0));
            else v.raw = load_partly(x0, e0, p.V);
        }
    };
    Pack<T, 16> v[NV], next[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) load(v[i], i * kRowThreads + tid);
    if (tid == 0) count = 0;

    float ref = 0.0f, sum = 0.0f, low = 0.0f;      // sum + low: the running sum
    float above = -INFINITY;                       // only elements above it can be listed
    bool bad = false, rescaled = false;
    for (int t0 = 0; t0 < vecs || t0 == 0; t0 += kTileVecs) {
        if (t0 + kTileVecs < vecs) {
#pragma unroll
            for (int i = 0; i < NV; ++i) load(next[i], t0 + kTileVecs + i * kRowThreads + tid);
        }
        const int e0 = (vec0 + t0 + tid) * E - head;         // of the tile's vector 0
        float tops[NV], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            tops[i] = vec_max(v[i]);
            top = fmaxf(top, tops[i]);
            if (!FUSED) {
#pragma unroll
                for (int e = 0; e < E; ++e) bad |= !(to_f32(v[i].e[e]) < INFINITY);
            }
        }
        // Lists the elements of the tile whose key reaches least.
        auto collect = [&](uint64_t least) {
            const float from = unordered((uint32_t)(least >> 32));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!(tops[i] >= from)) continue;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float x = to_f32(v[i].e[e]);
                    if (x >= from) {
                        const uint64_t c = (uint64_t)ordered(x) << 32 |
                                           (uint32_t)~(e0 + i * kRowThreads * E + e);
                        if (c >= least) buf[atomicAdd(&count, 1)] = c;
                    }
                }
            }
        };
        // Selection.  Every path leaves `count` settled behind a barrier.
        bool all = t0 == 0;          // select within the tile first
        if (!all) {
            const int have = count;                // settled until the barrier
            const int hits = __syncthreads_count(top > above);
            if (hits && have + hits * NV * E > kBuf) {
                keep_best(buf, best, &count, p.n);
                all = true;
            } else if (hits) {
                if (top > above) collect(((uint64_t)ordered(above) + 1) << 32);
                __syncthreads();
            }
        }
        if (all) {
            // The thread's best element (its maximum's first place).
            int where = -1;
            if (top > above) {
#pragma unroll
                for (int i = NV - 1; i >= 0; --i)
#pragma unroll
                    for (int e = E - 1; e >= 0; --e)
                        if (to_f32(v[i].e[e]) == top) where = e0 + i * kRowThreads * E + e;
            }
            const uint64_t key = where >= 0 ? (uint64_t)ordered(top) << 32 | (uint32_t)~where : 0;
            if (tid == 0) bound = 0;
            if (t0 == 0) {
                float m = top;
#pragma unroll
                for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (lane == 0) wmax[warp] = m;
            }
            const int rank = block_rank(key, order);
            if (rank == p.n - 1) bound = order[warp][lane];
            __syncthreads();
            if (t0 == 0) {
                ref = wmax[0];
#pragma unroll
                for (int w = 1; w < kRowWarps; ++w) ref = fmaxf(ref, wmax[w]);
                if (!(fabsf(ref) < kMostRef)) ref = 0.0f;
            }
            const uint64_t reach = bound;
            if (key && key >= reach)
                collect(max(reach, ((uint64_t)ordered(above) + 1) << 32));
            __syncthreads();
            if (reach) above = fmaxf(above, unordered((uint32_t)(reach >> 32)));
        }
        if (count > kCrowd) {
            keep_best(buf, best, &count, p.n);
            above = fmaxf(above, unordered((uint32_t)(buf[p.n - 1] >> 32)));   // n < kCrowd
        }
        if (FUSED) {
            if (top - ref > kRescale) {
                const float to = fminf(top, kMostRef), f = ex2((ref - to) * kLog2e);
                sum *= f;
                low *= f;
                ref = to;
                rescaled = true;
            }
            const float shift = -ref * kLog2e;
            float s[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                s[i] = 0.0f;
                if (i && t0 + i * kRowThreads >= vecs) continue;     // for the whole block
                float y[E];
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = ex2(__fmaf_rn(to_f32(v[i].e[e]), kLog2e, shift));
#pragma unroll
                for (int o = E / 2; o; o /= 2)
#pragma unroll
                    for (int e = 0; e < o; ++e) y[e] += y[e + o];
                s[i] = y[0];
            }
#pragma unroll
            for (int o = NV / 2; o; o /= 2)
#pragma unroll
                for (int i = 0; i < o; ++i) s[i] += s[i + o];
            const float to = sum + s[0], part = to - sum;       // the sum's rounding error
            low += (sum - (to - part)) + (s[0] - part);
            sum = to;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i].raw = next[i].raw;
    }
    // The threads' sums at the largest of their references.
    float at = ref;
    if (FUSED) {
        const int any = __syncthreads_or(rescaled);
        if (any) {
            float m = ref;
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) wmax[warp] = m;
            __syncthreads();
            at = wmax[0];
#pragma unroll
            for (int w = 1; w < kRowWarps; ++w) at = fmaxf(at, wmax[w]);
            const float f = at != ref ? ex2((ref - at) * kLog2e) : 1.0f;
            sum *= f;
            low *= f;
        }
        rescaled = any;
        Pair total = two_sum(sum, low);
#pragma unroll
        for (int o = 16; o; o >>= 1)
            total = add(total, Pair{__shfl_xor_sync(0xffffffffu, total.h, o),
                                    __shfl_xor_sync(0xffffffffu, total.l, o)});
        if (lane == 0) wsum[warp] = total;
    }
    const int bads = __syncthreads_or(bad);
    const int64_t unit = row * p.splits + split;
    if (tid == 0) {
        double r = (double)at, t = 0.0;
        if (FUSED) {
            Pair total = wsum[0];
#pragma unroll
            for (int w = 1; w < kRowWarps; ++w) total = add(total, wsum[w]);
            // x * log2e - round(at * log2e) = (x - r) * log2e
            const float shift = -at * kLog2e;
            r -= (double)__fmaf_rn(at, kLog2e, shift) * (1.0 / (double)kLog2e);
            t = (double)total.h + (double)total.l;
            if (rescaled) t = -t;
        }
        p.stat[unit] = make_double2(bads ? nan("") : r, t);
    }
    const int c = count;
    uint64_t* list = p.list + unit * p.n;
    for (int i = tid; i < c; i += kRowThreads) {
        const uint64_t mine = buf[i];
        int rank = 0;
        for (int j = 0; j < c; ++j) rank += buf[j] > mine;
        if (rank < p.n) list[rank] = mine;
    }
    for (int i = c + tid; i < p.n; i += kRowThreads) list[i] = 0;
}

// ------------------------------------------------------- the logarithm, exactly
// exp(x - ref) for x <= ref, relative error below 2^-43 down to e^-60: with
// x - ref = n ln 2 + g (Cody and Waite's reduction: ln 2 in three parts, the first with few
// bits so that n times it is exact), e^(g/16) - 1 by its Taylor series and four times
// (1 + q)^2 - 1.
__device__ __forceinline__ Pair exp_pair(float x, float ref) {
    const Pair d = two_sum(x, -ref);
    if (!(d.h > -104.0f)) return {0.0f, 0.0f};
    const float n = rintf(d.h * kLog2e);
    constexpr double ln2 = 0.69314718055994530942;
    constexpr float ln2a = 11356.0f / 16384.0f;            // 14 bits: n * ln2a is exact
    constexpr float ln2b = (float)(ln2 - (double)ln2a);
    constexpr float ln2c = (float)(ln2 - (double)ln2a - (double)ln2b);
    const Pair a = two_sum(__fmaf_rn(-n, ln2a, d.h), d.l);
    const float p = n * ln2b;
    const float pl = __fmaf_rn(n, ln2b, -p) + n * ln2c;
    Pair g = add(a, Pair{-p, -pl});
    g = Pair{g.h * 0.0625f, g.l * 0.0625f};                // |g| < 0.0217
    const Pair g2 = mul(g, g);
    float tail = __fmaf_rn(g.h, 1.0f / 5040.0f, 1.0f / 720.0f);
    tail = __fmaf_rn(tail, g.h, 1.0f / 120.0f);
    tail = __fmaf_rn(tail, g.h, 1.0f / 24.0f);
    tail = tail * g.h * g.h * g2.h;                        // g^4/24 + ...: below 1e-8
    const Pair g3 = mul(g2, g);
    const Pair sixth{1.0f / 6.0f, (float)(1.0 / 6.0 - (double)(1.0f / 6.0f))};
    Pair q = add(g, add(Pair{0.5f * g2.h, 0.5f * g2.l}, add(mul(g3, sixth), Pair{tail, 0.0f})));
#pragma unroll
    for (int i = 0; i < 4; ++i) q = add(Pair{2.0f * q.h, 2.0f * q.l}, mul(q, q));
    const Pair e = add(Pair{1.0f, 0.0f}, q);
    const float s1 = __int_as_float(((int)n / 2 + 127) << 23);       // 2^n in two factors
    const float s2 = __int_as_float(((int)n - (int)n / 2 + 127) << 23);
    return {e.h * s1 * s2, e.l * s1 * s2};
}

// log s for 1 <= s < 2^140, off by less than 1e-12: one Newton step from the float32
// logarithm y, y + (s e^-y - 1).
__device__ __forceinline__ double log_pair(double s) {
    const float y = logf((float)s);
    const Pair e = exp_pair(0.0f, y);
    return (double)y + (s * ((double)e.h + (double)e.l) - 1.0);
}

// --------------------------------------------------------- the Ko best of all
// One CTA per batch item; a list (beam, split) has four threads.  Lists whose head is not
// among the Ko best heads hold nothing; of the others the elements from the Ko-th best
// head on are ranked by counting.
//
// The fast sums leave a log-sum-exp off by error[k]: 2^-22 of ex2.approx; 5 roundings of
// a tile's sum (a tree over up to 32 elements), tiles being added with the rounding error
// carried along; half a rounding of the exponent t = (x - r) log2 e and 2^-26 of log2 e,
// both relative to t, whose mean size over the distribution is at most
// log2 V - log2 S + 2 t_max (its entropy is at most log2 V).  Where the order of two
// candidates of different beams is closer than that, the beams' log-sum-exps are computed
// again to 40 bits and the selection is repeated.  With 50000 outputs the bound is about
// 1e-6, and 1 call in 15 of 64 items x 16 beams meets such a pair.
constexpr float kTermError = 2.4e-7f + 5 * 6e-8f;
constexpr float kExponentError = 5.2e-8f;          // 1.25 * 2^-24 * ln 2
constexpr float kRescaleError = 1e-6f;
constexpr int kPickThreads = 1024;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kCand = RNNT_MAX_BEAM * (RNNT_MAX_BEAM + 1) / 2;

// log sum exp of a row by the whole block, the same for equal rows wherever they lie.
template <typename T>
__device__ __noinline__ double exact_lse(const T* x, int V, Pair* sums, float* tops) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float top = -INFINITY;
    for (int i = tid; i < V; i += kPickThreads) top = fmaxf(top, to_f32(x[i]));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = tops[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    Pair s{0.0f, 0.0f};
#pragma unroll 2
    for (int i = tid; i < V; i += kPickThreads) s = add(s, exp_pair(to_f32(x[i]), top));
#pragma unroll
    for (int o = 16; o; o >>= 1)
        s = add(s, Pair{__shfl_xor_sync(0xffffffffu, s.h, o), __shfl_xor_sync(0xffffffffu, s.l, o)});
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    s = sums[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        s = add(s, Pair{__shfl_xor_sync(0xffffffffu, s.h, o), __shfl_xor_sync(0xffffffffu, s.l, o)});
    __syncthreads();
    return (double)top + log_pair((double)s.h + (double)s.l);
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) k_pick(const SelectParams p) {
    extern __shared__ uint64_t lists[];                // [K * splits][n]
    __shared__ uint64_t cval[kCand];                   // candidates: ordered value, number
    __shared__ uint32_t cid[kCand];
    __shared__ uint64_t heads[kMaxLists];
    __shared__ uint64_t oval[RNNT_MAX_BEAM];           // the best, in order
    __shared__ uint32_t oid[RNNT_MAX_BEAM];
    __shared__ double2 stat[kMaxLists];
    __shared__ double lse[RNNT_MAX_BEAM];
    __shared__ float score[RNNT_MAX_BEAM];
    __shared__ double error[RNNT_MAX_BEAM];
    __shared__ uint8_t kind[RNNT_MAX_BEAM];            // 0 nothing, 1 logits, 2 finished
    __shared__ unsigned long long doubt, border;       // beams, a bit each
    __shared__ Pair sums[kPickWarps];
    __shared__ float tops[kPickWarps];
    __shared__ int count, outside;
    __shared__ uint64_t bound;
    const int tid = threadIdx.x;
    const int64_t b = blockIdx.x;
    const int nlists = p.K * p.splits;
    if (tid < nlists) stat[tid] = p.stat[b * nlists + tid];
    for (int i = tid; i < nlists * p.n; i += kPickThreads) lists[i] = p.list[b * nlists * p.n + i];
    float s = 0.0f;
    bool done = false;
    if (tid < p.K) {
        s = p.scores[b * p.K + tid];
        done = p.finished && p.finished[b * p.K + tid];
    }
    if (tid == 0) doubt = 0;
    __syncthreads();
    if (tid < p.K) {
        bool bad = !(s < INFINITY);
        int what = bad || s == -INFINITY ? 0 : done ? 2 : 1;
        double l = 0.0, err = 0.0;
        if (what == 1) {
            const double2* st = stat + tid * p.splits;
            double top = -INFINITY, sum = 0.0;
            float high = -INFINITY;
            for (int g = 0; g < p.splits; ++g) {
                const uint64_t c = lists[(tid * p.splits + g) * p.n];
                if (c) high = fmaxf(high, unordered((uint32_t)(c >> 32)));
                bad |= st[g].x != st[g].x || st[g].y != st[g].y;
                if (st[g].y != 0.0) top = fmax(top, st[g].x);
            }
            bad |= high == INFINITY;
            if (bad || high == -INFINITY) {
                what = 0;
            } else if (p.fused) {
                const float logv = 1e-3f + __log2f((float)p.V);
                bool sure = top > -INFINITY;
                float worst = 0.0f;
                for (int g = 0; g < p.splits; ++g) {
                    const double y = fabs(st[g].y);
                    if (y == 0.0) continue;
                    sure &= y < 1e30 && y > 1e-30;
                    sum += st[g].x == top ? y : y * exp(st[g].x - top);
                    const uint64_t c = lists[(tid * p.splits + g) * p.n];
                    const float over = fmaxf(0.0f, unordered((uint32_t)(c >> 32)) - (float)st[g].x);
                    worst = fmaxf(worst, kTermError + (st[g].y < 0.0 ? kRescaleError : 0.0f) +
                                  kExponentError * (logv - __log2f((float)y) + 2.9f * over));
                }
                sure &= sum >= 1.0 && sum < 1e40;
                if (sure) {
                    l = top + log_pair(sum);
                    err = (double)worst + 1e-9;
                } else {
                    atomicOr(&doubt, 1ull << tid);     // out of the fast sum's range
                }
            }
        }
        if (bad && p.status) *p.status = RNNT_INVALID_VALUE;
        lse[tid] = l;
        score[tid] = s;
        error[tid] = err;
        kind[tid] = (uint8_t)what;
    }
    __syncthreads();
    const int list = tid >> 2, k = list / p.splits;    // of this thread
    for (unsigned long long again = doubt;;) {
        for (; again; again &= again - 1) {
            const int kk = __ffsll((long long)again) - 1;
            const double l = exact_lse(row_of<T>(p, b * p.K + kk), p.V, sums, tops);
            if (tid == 0) {
                lse[kk] = l;
                error[kk] = 0.0;
            }
        }
        if (tid == 0) {
            count = outside = 0;
            doubt = border = 0;
            bound = 1;
        }
        __syncthreads();
        const int what = list < nlists ? kind[k] : 0;
        // Ordered value of the list's element j, 0 if there is none.
        auto value = [&](int j) -> uint64_t {
            if (what == 2) return list == k * p.splits && j == 0 ? ordered((double)score[k]) : 0;
            const uint64_t c = what == 1 && j < p.n ? lists[list * p.n + j] : 0;
            return c ? ordered((double)score[k] + ((double)unordered((uint32_t)(c >> 32)) - lse[k]))
                     : 0;
        };
        auto number = [&](int j) {
            return (uint32_t)k * (uint32_t)p.V + (what == 2 ? 0u : ~(uint32_t)lists[list * p.n + j]);
        };
        const uint64_t first = value(0);
        if ((tid & 3) == 0 && list < nlists) heads[list] = first;
        __syncthreads();
        int rank = 0;
        if (list < nlists)
            for (int j = tid & 3; j < nlists; j += 4)
                rank += heads[j] > first || (heads[j] == first && j < list);
        rank += __shfl_xor_sync(0xffffffffu, rank, 1);
        rank += __shfl_xor_sync(0xffffffffu, rank, 2);
        if (first && rank == p.Ko - 1) bound = first;
        __syncthreads();
        // element j of the list of rank r has j + r better ones
        if (first && rank < p.Ko)
            for (int j = tid & 3; j + rank < p.Ko; j += 4) {
                const uint64_t v = value(j);
                if (v < bound) break;
                const int to = atomicAdd(&count, 1);
                cval[to] = v;
                cid[to] = number(j);
            }
        __syncthreads();
        const int c = count, found = min(c, p.Ko);
        for (int i0 = 0; i0 < c; i0 += kPickThreads / 4) {
            const int i = i0 + (tid >> 2);
            const uint64_t v = i < c ? cval[i] : 0;
            const uint32_t d = i < c ? cid[i] : 0;
            int r = 0;
            for (int j = tid & 3; j < c; j += 4)
                r += cval[j] > v || (cval[j] == v && cid[j] < d);
            r += __shfl_xor_sync(0xffffffffu, r, 1);
            r += __shfl_xor_sync(0xffffffffu, r, 2);
            if (i < c && r < p.Ko && (tid & 3) == 0) {
                oval[r] = v;
                oid[r] = d;
            }
        }
        __syncthreads();
        if (!p.fused || found == 0) break;
        // Neighbours of different beams whose order is in doubt.
        if (tid + 1 < found) {
            const int k0 = oid[tid] / p.V, k1 = oid[tid + 1] / p.V;
            if (k0 != k1 &&
                unordered(oval[tid]) - unordered(oval[tid + 1]) < error[k0] + error[k1])
                atomicOr(&doubt, (error[k0] > 0.0 ? 1ull << k0 : 0) |
                                 (error[k1] > 0.0 ? 1ull << k1 : 0));
        }
        // Beams with candidates as near to the last one, some of them left out.
        if (found == p.Ko && first) {
            const double last = unordered(oval[found - 1]);
            const double within = error[k] + error[oid[found - 1] / p.V];
            const uint64_t lo = ordered(last - within), hi = ordered(last + within);
            for (int j = tid & 3; j < p.n; j += 4) {
                const uint64_t v = value(j);
                if (!v || v < lo) break;
                if (v > hi) continue;
                atomicOr(&border, 1ull << k);
                if (v < oval[found - 1] || (v == oval[found - 1] && number(j) > oid[found - 1]))
                    outside = 1;
            }
        }
        __syncthreads();
        again = doubt;
        if (outside && __popcll(border) > 1)
            for (unsigned long long left = border; left; left &= left - 1) {
                const int kk = __ffsll((long long)left) - 1;
                if (error[kk] > 0.0) again |= 1ull << kk;
            }
        __syncthreads();       // `doubt` and `border` have been read
        if (!again) break;
    }
    for (int r = tid; r < p.Ko; r += kPickThreads) {
        const int64_t o = b * p.Ko + r;
        const int from = r < min(count, p.Ko) ? (int)(oid[r] / p.V) : -1;
        p.out_scores[o] = from < 0 ? -INFINITY : (float)unordered(oval[r]);
        p.out_tokens[o] = from < 0 || kind[from] == 2 ? -1 : (int)(oid[r] - from * p.V);
        p.out_parents[o] = from;
    }
}

struct SelectLayout {
    size_t stat, list, total;
    int32_t splits, split_vecs, n;
};
SelectLayout select_layout(int32_t B, int32_t K, int32_t V, int32_t Ko, int dt) {
    SelectLayout L;
    const int E = 16 / elem_size(dt);
    const int64_t vecs = ((int64_t)V + 2 * (E - 1)) / E;      // the most, whatever the alignment
    constexpr int64_t kWanted = 152 * 4;                      // CTAs that fill the device
    int64_t splits = (kWanted + (int64_t)B * K - 1) / ((int64_t)B * K);
    splits = std::min(splits, (vecs + kRowThreads - 1) / kRowThreads);
    splits = std::max<int64_t>(1, std::min<int64_t>(splits, kMaxLists / K));
    L.split_vecs = (int32_t)((vecs + splits - 1) / splits);
    L.splits = (int32_t)((vecs + L.split_vecs - 1) / L.split_vecs);
    L.n = std::min(Ko, V);
    const size_t units = (size_t)B * K * L.splits;
    L.stat = 0;
    L.list = align256(units * sizeof(double2));
    L.total = align256(L.list + units * L.n * sizeof(uint64_t));
    return L;
}
bool select_ok(int32_t B, int32_t K, int32_t V, int32_t Ko, int dt) {
    return B >= 1 && K >= 1 && K <= RNNT_MAX_BEAM && Ko >= 1 && Ko <= RNNT_MAX_BEAM && V >= 1 &&
           V <= RNNT_MAX_BEAM_VOCAB && valid_dtype(dt) &&
           (int64_t)B * K * select_layout(B, K, V, Ko, dt).splits <= INT32_MAX;
}

template <typename T>
void launch_select(const SelectParams& p, cudaStream_t st) {
    const unsigned grid = (unsigned)(p.B * p.K * p.splits);
    auto rows = [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        if (p.fused) k_rows<T, NV, true><<<grid, kRowThreads, 0, st>>>(p);
        else k_rows<T, NV, false><<<grid, kRowThreads, 0, st>>>(p);
    };
    if (p.split_vecs <= kRowThreads) rows(std::integral_constant<int, 1>{});
    else if (p.split_vecs <= 2 * kRowThreads) rows(std::integral_constant<int, 2>{});
    else rows(std::integral_constant<int, 4>{});
    const size_t shared = sizeof(uint64_t) * p.K * p.splits * p.n;
    k_pick<T><<<(unsigned)p.B, kPickThreads, shared, st>>>(p);
}

// k_pick's shared memory limit, raised once per device.
bool pick_prepared() {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return false;
    if (done[dev].load(std::memory_order_acquire)) return true;
    const int most = (int)(sizeof(uint64_t) * kMaxLists * RNNT_MAX_BEAM);
    bool ok = true;
    for (int dt = 0; dt < 3 && ok; ++dt)
        ok = with_type(dt, [&](auto tag) {
            return cudaFuncSetAttribute(k_pick<decltype(tag)>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        }) == cudaSuccess;
    if (ok) done[dev].store(true, std::memory_order_release);
    else cudaGetLastError();
    return ok;
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
    p.splits = L.splits;
    p.split_vecs = L.split_vecs;
    p.n = L.n;
    p.stat = reinterpret_cast<double2*>(ws + L.stat);
    p.list = reinterpret_cast<uint64_t*>(ws + L.list);
    p.out_scores = out_scores;
    p.out_tokens = out_tokens;
    p.out_parents = out_parents;
    p.status = status_dev;
    if (!pick_prepared() || !clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    with_type(dt, [&](auto tag) {
        launch_select<decltype(tag)>(p, st);
        return 0;
    });
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
