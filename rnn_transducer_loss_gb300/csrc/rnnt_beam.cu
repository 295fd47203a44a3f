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
// ------------------------------------------------------------- rows of logits
// A row is cut into splits of whole aligned 16-byte vectors (the few elements ahead of them
// and behind them go to threads of split 0 one by one); a CTA streams one split through
// registers and writes
//   - the sum of exp(x - r) over the split and its reference r.  r is the first tile's
//     maximum and changes only when a thread meets a value more than 16 above it, so
//     that a sum is (almost) never rescaled.
//   - the n best elements in order.  The stream keeps each thread's maximum of every
//     tile and nothing else.  Every warp's ceil(n / 8)-th largest thread maximum bounds the
//     n-th best element from below (the least of the eight does); the few tiles of a
//     thread that reach the bound are read once more, from the cache, and their elements
//     that reach it are ranked by counting.  Rows with a crowd of equal elements at the
//     bound go through best_of_row instead, tile by tile.
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr float kLog2e = 1.44269504f;      // log2 e to 2^-26
constexpr float kRescale = 16.0f;
constexpr float kMostRef = 1e30f;          // larger references: computed again by exact_lse
// Bound of a sum's relative error: 2^-22 of ex2.approx and 6 roundings of a tile's sum (a tree
// over up to 33 elements; tiles are added with the rounding error carried along); half a
// rounding of the exponent t = (x - ref) log2 e and 2^-26 of log2 e, both relative to t, whose
// mean size over the distribution is at most log2 V - log2 S + 2 max(t, 0) (its entropy is at
// most log2 V); rescalings, of which only the last two weigh anything.
constexpr float kTermError = 2.4e-7f + 6 * 6e-8f;
constexpr float kExponentError = 5.2e-8f;          // 1.25 * 2^-24 * ln 2
constexpr float kRescaleError = 1e-6f;
constexpr int kMaxLists = 256;             // splits of a batch item's rows
constexpr int kSlots = 8;                  // of tiles, whose maxima a thread keeps
constexpr int kBuf = 1024;                 // elements ranked: > RNNT_MAX_BEAM * 9 (best_of_row)

struct SelectParams {
    const char* logits;
    int64_t batch_stride, beam_stride;     // bytes
    const float* scores;
    const uint8_t* finished;
    int32_t B, K, V, Ko, fused;
    int32_t splits, split_vecs;            // splits of a row, vectors of a split
    int32_t n;                             // elements a split lists: min(Ko, V)
    float4* stat;                          // [row][split]: reference, sum of exp(x - reference) as
                                           // a pair, bound of the sum's relative error
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

// Two float32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d)
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
          "l"(reinterpret_cast<uint64_t&>(c)));
    return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d)
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return reinterpret_cast<float2&>(d);
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

__device__ __forceinline__ Pair shuffled(Pair a, int o) {
    return {__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
}
// Without the last step of add: for sums of positive terms.
__device__ __forceinline__ Pair add_loosely(Pair a, Pair b) {
    const Pair s = two_sum(a.h, b.h);
    return {s.h, s.l + (a.l + b.l)};
}
// Pairs in the order of their values: for |l| <= half a step of h, as add leaves them.
__device__ __forceinline__ uint64_t ordered(Pair a) {
    return (uint64_t)ordered(a.h) << 32 | ordered(a.l);
}
__device__ __forceinline__ float difference(uint64_t a, uint64_t b) {
    return (unordered((uint32_t)(a >> 32)) - unordered((uint32_t)(b >> 32))) +
           (unordered((uint32_t)a) - unordered((uint32_t)b));
}

// Whether beam `row` offers its logits' candidates.
__device__ __forceinline__ bool reads_logits(const SelectParams& p, uint32_t row) {
    if (p.finished && p.finished[row]) return false;
    const float s = p.scores[row];
    return s > -INFINITY && s < INFINITY;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const SelectParams& p, uint32_t row) {
    const uint32_t b = row / (uint32_t)p.K;
    return reinterpret_cast<const T*>(p.logits + b * p.batch_stride +
                                      (row - b * p.K) * p.beam_stride);
}

// Sorts the warp's keys in descending order (bitonic).
template <typename Key>
__device__ __forceinline__ Key warp_sorted(Key key) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
        for (int o = size / 2; o; o >>= 1) {
            const Key other = __shfl_xor_sync(0xffffffffu, key, o);
            const bool larger = ((lane & o) == 0) == ((lane & size) == 0 || size == 32);
            if (larger == (other > key)) key = other;
        }
    }
    return key;
}

// Ranks the buffer's c different keys: best[r] = the r-th for r < n.  Four threads count for a
// key.  Ends without a barrier.
__device__ __forceinline__ void rank_keys(const uint64_t* buf, int c, uint64_t* best, int n) {
    const int part = threadIdx.x & 3;
    for (int i0 = 0; i0 < c; i0 += kRowThreads / 4) {
        const int i = i0 + (threadIdx.x >> 2);
        const uint64_t mine = i < c ? buf[i] : ~0ull;
        int rank = 0;
        if (i < c)
            for (int j = part; j < c; j += 4) rank += buf[j] > mine;
        rank += __shfl_xor_sync(0xffffffffu, rank, 1);
        rank += __shfl_xor_sync(0xffffffffu, rank, 2);
        if (i < c && rank < n && part == 0) best[rank] = mine;
    }
}

// Keeps the n best of the buffer's keys, in order; all threads call it.
__device__ __noinline__ void keep_best(uint64_t* buf, uint64_t* best, int* count, int n) {
    const int c = *count, m = min(c, n);
    rank_keys(buf, c, best, n);
    __syncthreads();
    if (threadIdx.x < m) buf[threadIdx.x] = best[threadIdx.x];
    if (threadIdx.x == 0) *count = m;
    __syncthreads();
}

// The elements of a vector, two by two.
__device__ __forceinline__ void unpack(const Pack<float, 16>& v, float2* y) {
    y[0] = make_float2(v.e[0], v.e[1]);
    y[1] = make_float2(v.e[2], v.e[3]);
}
__device__ __forceinline__ void unpack(const Pack<__half, 16>& v, float2* y) {
    const __half2* h = reinterpret_cast<const __half2*>(&v.raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __half22float2(h[i]);
}
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, 16>& v, float2* y) {
    const uint32_t w[4] = {v.raw.x, v.raw.y, v.raw.z, v.raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
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

__device__ __forceinline__ uint64_t key_of(float x, int element) {
    return (uint64_t)ordered(x) << 32 | (uint32_t)~element;
}

__device__ __forceinline__ uint4 load_stream(const uint4* at) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at));
    return v;
}

// A split: `vecs` vectors from `aligned` on, the first of them at element `first` of the row.
template <typename T>
struct Split {
    static constexpr int E = 16 / (int)sizeof(T);
    const uint4* aligned;
    int first, vecs;

    __device__ __forceinline__ Split(const SelectParams& p, uint32_t row, int split) {
        const T* x0 = row_of<T>(p, row);
        const int ahead = min(p.V, (int)(-(uintptr_t)x0 & 15) / (int)sizeof(T));
        const int vec0 = split * p.split_vecs;
        vecs = max(0, min(p.split_vecs, (p.V - ahead) / E - vec0));
        first = ahead + vec0 * E;
        aligned = reinterpret_cast<const uint4*>(x0 + ahead) + vec0;
    }
    // Vector j, -inf from vecs on.
    __device__ __forceinline__ Pack<T, 16> at(int j) const {
        Pack<T, 16> v;
#pragma unroll
        for (int e = 0; e < E; ++e) v.e[e] = from_f32<T>(-INFINITY);
        if (j < vecs) v.raw = load_stream(aligned + j);
        return v;
    }
};

// The element ahead of the row's whole vectors or behind them that is this thread's, or -1.
template <typename T>
__device__ __forceinline__ int odd_element(const SelectParams& p, uint32_t row, int split) {
    constexpr int E = 16 / (int)sizeof(T);
    if (split || threadIdx.x >= 2 * E) return -1;
    const int ahead = min(p.V, (int)(-(uintptr_t)row_of<T>(p, row) & 15) / (int)sizeof(T));
    const int behind = ahead + (p.V - ahead) / E * E;
    const int at = threadIdx.x < E ? threadIdx.x : behind + threadIdx.x - E;
    return at < (threadIdx.x < E ? ahead : p.V) ? at : -1;
}

// The n best of a split to best: every tile of kRowThreads vectors gives its elements above the
// bound, the n-th best so far; a tile that has too many gives them element by element of each
// thread's vector.
template <typename T>
__device__ __noinline__ void best_of_row(const SelectParams& p, uint32_t row, int split,
                                         uint64_t* buf, uint64_t* best, int* count) {
    constexpr int E = 16 / (int)sizeof(T);
    const Split<T> sp(p, row, split);
    const int tid = threadIdx.x, n = p.n;
    __syncthreads();
    if (tid == 0) *count = 0;
    uint64_t least = (uint64_t)(ordered(-INFINITY) + 1) << 32;     // keys below it do not matter
    __syncthreads();
    const int odd = odd_element<T>(p, row, split);
    if (odd >= 0) {
        const float x = to_f32(row_of<T>(p, row)[odd]);
        if (x > -INFINITY) buf[atomicAdd(count, 1)] = key_of(x, odd);
    }
    for (int t0 = 0; t0 < sp.vecs; t0 += kRowThreads) {
        const Pack<T, 16> v = sp.at(t0 + tid);
        const int at = sp.first + (t0 + tid) * E;
        for (int e0 = 0; e0 < E;) {
            // as many elements of each thread as surely fit
            __syncthreads();
            const int have = *count;
            int hits = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = to_f32(v.e[e]);
                hits += e >= e0 && x > -INFINITY && key_of(x, at + e) >= least;
            }
            const int threads = __syncthreads_count(hits > 0);
            if (!threads) break;
            const int e1 = have + threads * (E - e0) <= kBuf ? E : e0 + 1;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = to_f32(v.e[e]);
                const uint64_t c = key_of(x, at + e);
                if (e >= e0 && e < e1 && x > -INFINITY && c >= least)
                    buf[atomicAdd(count, 1)] = c;
            }
            e0 = e1;
            __syncthreads();
            if (*count > kRowThreads) {
                keep_best(buf, best, count, n);
                least = max(least, buf[n - 1]);        // n < kRowThreads
            }
        }
    }
    __syncthreads();
    rank_keys(buf, *count, best, n);
    __syncthreads();
}

template <typename T, int NV, bool FUSED>
__global__ void __launch_bounds__(kRowThreads, NV == 1 ? 6 : 4) k_rows(const SelectParams p) {
    constexpr int E = 16 / (int)sizeof(T);
    constexpr int kTileVecs = kRowThreads * NV;
    __shared__ uint64_t buf[kBuf], best[RNNT_MAX_BEAM];
    __shared__ Pair wsum[kRowWarps];
    __shared__ float wref[kRowWarps], wleast[kRowWarps], wover[kRowWarps];
    __shared__ float tops[kSlots][kRowThreads];
    __shared__ int hit[kSlots * kRowThreads];      // slots to be read once more
    __shared__ int hits, count, bads, rescales;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t row = blockIdx.x / (uint32_t)p.splits;
    const int split = (int)(blockIdx.x - row * (uint32_t)p.splits);
    const Split<T> sp(p, row, split);
    const int vecs = sp.vecs;
    auto load_tile = [&](Pack<T, 16>* v, int t0) {
        if (t0 + kTileVecs <= vecs) {                        // for the whole block
#pragma unroll
            for (int i = 0; i < NV; ++i)
                v[i].raw = load_stream(sp.aligned + t0 + i * kRowThreads + tid);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = sp.at(t0 + i * kRowThreads + tid);
        }
    };
    Pack<T, 16> v[NV], next[NV];
    load_tile(v, 0);
    const int odd = odd_element<T>(p, row, split);
    const float odd_x = odd >= 0 ? to_f32(row_of<T>(p, row)[odd]) : -INFINITY;
    if (!reads_logits(p, row)) return;             // asked for while the loads are in flight
    if (tid == 0) hits = count = bads = rescales = 0;

    float ref = 0.0f, sum = 0.0f, low = 0.0f;      // sum + low: the running sum
    float most = odd_x;                            // the thread's maximum
    bool bad = !FUSED && !(odd_x < INFINITY), rescaled = false;
    int shift_slot = 0;                            // tiles of a slot: 1 << shift_slot
    while ((vecs - 1) / kTileVecs >> shift_slot >= kSlots) ++shift_slot;
    float slot_top = -INFINITY;
    for (int t0 = 0; t0 < vecs || t0 == 0; t0 += kTileVecs) {
        if (t0 + kTileVecs < vecs) load_tile(next, t0 + kTileVecs);
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            top = fmaxf(top, vec_max(v[i]));
            if (!FUSED) {
#pragma unroll
                for (int e = 0; e < E; ++e) bad |= !(to_f32(v[i].e[e]) < INFINITY);
            }
        }
        most = fmaxf(most, top);
        slot_top = fmaxf(slot_top, top);
        const int tile = t0 / kTileVecs;
        if (((tile + 1) & ((1 << shift_slot) - 1)) == 0 || t0 + kTileVecs >= vecs) {
            tops[tile >> shift_slot][tid] = slot_top;
            slot_top = -INFINITY;
        }
        if (FUSED) {
            if (t0 == 0) {
                top = fmaxf(top, odd_x);
                float m = top;
#pragma unroll
                for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (lane == 0) wref[warp] = m;
                __syncthreads();
                ref = wref[0];
#pragma unroll
                for (int w = 1; w < kRowWarps; ++w) ref = fmaxf(ref, wref[w]);
                if (!(fabsf(ref) < kMostRef)) ref = 0.0f;
            }
            if (top - ref > kRescale) {
                const float to = fminf(top, kMostRef), f = ex2(__fmul_rn(ref, kLog2e) - __fmul_rn(to, kLog2e));
                sum *= f;
                low *= f;
                ref = to;
                rescaled = true;
            }
            const float shift = -__fmul_rn(ref, kLog2e);
            const float2 scale2 = make_float2(kLog2e, kLog2e), shift2 = make_float2(shift, shift);
            float s[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                s[i] = 0.0f;
                if (i && t0 + i * kRowThreads >= vecs) continue;     // for the whole block
                float2 y[E / 2];
                unpack(v[i], y);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    const float2 t = fma2(y[e], scale2, shift2);
                    y[e] = make_float2(ex2(t.x), ex2(t.y));
                }
#pragma unroll
                for (int o = E / 4; o; o /= 2)
#pragma unroll
                    for (int e = 0; e < o; ++e) y[e] = add2(y[e], y[e + o]);
                s[i] = y[0].x + y[0].y;
            }
#pragma unroll
            for (int o = NV / 2; o; o /= 2)
#pragma unroll
                for (int i = 0; i < o; ++i) s[i] += s[i + o];
            if (t0 == 0) s[0] += ex2(__fmaf_rn(odd_x, kLog2e, shift));
            const float to = sum + s[0], part = to - sum;       // the sum's rounding error
            low += (sum - (to - part)) + (s[0] - part);
            sum = to;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i].raw = next[i].raw;
    }
    // The bound.
    const int whole = min(vecs / 32, kRowWarps);       // warps whose threads all have a maximum
    const int nth = (p.n - 1) / max(whole, 1);         // of each one's, from 0
    float least = most;
    if (nth == 0) {
#pragma unroll
        for (int o = 16; o; o >>= 1) least = fmaxf(least, __shfl_xor_sync(0xffffffffu, least, o));
    } else {
        least = unordered(__shfl_sync(0xffffffffu, warp_sorted(ordered(most)), nth & 31));
    }
    if (lane == 0) wleast[warp] = least;
    if (bad) bads = 1;
    if (rescaled) rescales = 1;
    __syncthreads();
    least = whole && nth < 32 ? INFINITY : -INFINITY;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w)
        if (w < whole) least = fminf(least, wleast[w]);
    const int span = kTileVecs << shift_slot;
    for (int t = 0; t * span < vecs; ++t) {
        const bool reaches = tops[t][tid] >= least && tops[t][tid] > -INFINITY;
        const unsigned who = __ballot_sync(0xffffffffu, reaches);
        if (!who) continue;
        int to = 0;
        if (lane == 0) to = atomicAdd(&hits, __popc(who));
        to = __shfl_sync(0xffffffffu, to, 0) + __popc(who & ((1u << lane) - 1));
        if (reaches) hit[to] = t * kRowThreads + tid;
    }
    float at = ref;                                // the largest of the threads' references
    if (FUSED) {
        Pair total{sum, low};
        float over = sum * fmaxf(0.0f, most - ref);
        if (rescales) {
            float m = ref;
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) wref[warp] = m;
            __syncthreads();
            at = wref[0];
#pragma unroll
            for (int w = 1; w < kRowWarps; ++w) at = fmaxf(at, wref[w]);
            const float f = at != ref ? ex2(__fmul_rn(ref, kLog2e) - __fmul_rn(at, kLog2e)) : 1.0f;
            total = Pair{total.h * f, total.l * f};
            over *= f;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            total = add_loosely(total, shuffled(total, o));
            over += __shfl_xor_sync(0xffffffffu, over, o);
        }
        if (lane == 0) {
            wsum[warp] = total;
            wover[warp] = over;
        }
    }
    __syncthreads();
    // Those slots' vectors once more: their elements that reach the bound.
    const int per = NV << shift_slot;              // vectors of a slot
    for (int i = tid; i < hits * per; i += kRowThreads) {
        const int slot = hit[i / per];
        const int j = slot / kRowThreads * span + i % per * kRowThreads + slot % kRowThreads;
        const Pack<T, 16> w = sp.at(j);
        unsigned which = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float x = to_f32(w.e[e]);
            which |= (x >= least && x > -INFINITY ? 1u : 0u) << e;
        }
        if (which) {
            int to = atomicAdd(&count, __popc(which));
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (which >> e & 1) {
                    if (to < kBuf) buf[to] = key_of(to_f32(w.e[e]), sp.first + j * E + e);
                    ++to;
                }
        }
    }
    if (odd_x >= least && odd_x > -INFINITY) {
        const int to = atomicAdd(&count, 1);
        if (to < kBuf) buf[to] = key_of(odd_x, odd);
    }
    __syncthreads();
    const bool crowd = count > kBuf;
    const uint32_t unit = blockIdx.x;
    if (warp == kRowWarps - 1) {                   // the keys are ranked by the first ones
        Pair total{0.0f, 0.0f};
        float over = 0.0f, err = 0.0f;
        if (FUSED) {
            if (lane < kRowWarps) {
                total = wsum[lane];
                over = wover[lane];
            }
#pragma unroll
            for (int o = kRowWarps / 2; o; o >>= 1) {
                total = add(total, shuffled(total, o));
                over += __shfl_xor_sync(0xffffffffu, over, o);
            }
            // x log2e - round(at log2e) = (x - at) log2e + off
            const float off = __fmaf_rn(at, kLog2e, -__fmul_rn(at, kLog2e)) * (-1.0f / kLog2e);
            if (fabsf(off) > 1e-3f) total = Pair{NAN, NAN};        // |at| above 10^4 or so
            total = mul(total, two_sum(1.0f, off + 0.5f * off * off));
            err = kTermError + (rescales ? kRescaleError : 0.0f) +
                  kExponentError * (1e-3f + __log2f((float)p.V) - __log2f(total.h) +
                                    2.9f * over / total.h);
        }
        if (lane == 0)
            p.stat[unit] = make_float4(FUSED ? at : bads ? NAN : 0.0f, total.h, total.l, err);
    }
    if (!crowd) rank_keys(buf, count, best, p.n);
    __syncthreads();
    if (crowd) best_of_row<T>(p, row, split, buf, best, &count);
    for (int i = tid; i < p.n; i += kRowThreads)
        p.list[(int64_t)unit * p.n + i] = i < min(count, p.n) ? best[i] : 0;
}

// ------------------------------------------------------- the logarithm, exactly
// exp(x - ref) for x <= ref, relative error below 2^-40 down to e^-60: with
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

// log s for 1 <= s < 2^140, off by less than 2^-40: one Newton step from the float32
// logarithm y, y + (s e^-y - 1).
__device__ __forceinline__ Pair log_pair(Pair s) {
    const float y = logf(s.h);
    const Pair e = add(mul(s, exp_pair(0.0f, y)), Pair{-1.0f, 0.0f});
    return add(Pair{y, 0.0f}, e);
}

// --------------------------------------------------------- the Ko best of all
// One CTA per batch item; a list (beam, split) has kParts threads.  Lists whose head is not
// among the Ko best heads hold nothing; of the others the elements from the Ko-th best
// head on are ranked by counting.
//
// The streamed sums leave a log-sum-exp off by error[k] (see kTermError).  Where the order of
// two candidates of different beams is closer than that, the beams' log-sum-exps are computed
// again to 40 bits and the selection is repeated.  With 50000 outputs the bound is about
// 1e-6, and 1 call in 15 of 64 items x 16 beams meets such a pair.
constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kParts = kPickThreads / kMaxLists;     // threads of a list
constexpr int kTokenBits = 20;              // a candidate's number: beam, then token
constexpr uint32_t kTokenMask = (1u << kTokenBits) - 1;
static_assert(RNNT_MAX_BEAM_VOCAB <= 1 << kTokenBits, "a token fits");
constexpr int kCand = RNNT_MAX_BEAM * (RNNT_MAX_BEAM + 1) / 2;

// log sum exp of a row by the whole block, the same for equal rows wherever they lie; NaN
// where the row holds NaN or +inf.
template <typename T>
__device__ __noinline__ Pair exact_lse(const T* x, int V, Pair* sums, float* tops) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float top = -INFINITY;
    for (int i = tid; i < V; i += kPickThreads) top = fmaxf(top, to_f32(x[i]));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = tops[lane & (kPickWarps - 1)];
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    Pair s{0.0f, 0.0f};
#pragma unroll 2
    for (int i = tid; i < V; i += kPickThreads) {
        const float y = to_f32(x[i]);
        s = add(s, y < INFINITY ? exp_pair(y, top) : Pair{NAN, NAN});
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s = add(s, shuffled(s, o));
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    s = lane < kPickWarps ? sums[lane] : Pair{0.0f, 0.0f};
#pragma unroll
    for (int o = 16; o; o >>= 1) s = add(s, shuffled(s, o));
    __syncthreads();
    return add(Pair{top, 0.0f}, log_pair(s));
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) k_pick(const SelectParams p) {
    extern __shared__ uint64_t lists[];                // [K * splits][n]
    __shared__ uint64_t cval[kCand];                   // candidates: ordered value, number
    __shared__ uint32_t cid[kCand];
    __shared__ uint64_t heads[kMaxLists];
    __shared__ uint64_t oval[RNNT_MAX_BEAM];           // the best, in order
    __shared__ uint32_t oid[RNNT_MAX_BEAM];
    __shared__ float4 stat[kMaxLists];
    __shared__ Pair lse[RNNT_MAX_BEAM];
    __shared__ float score[RNNT_MAX_BEAM], error[RNNT_MAX_BEAM];
    __shared__ uint8_t kind[RNNT_MAX_BEAM];            // 0 nothing, 1 logits, 2 finished
    __shared__ unsigned long long doubt, border;       // beams, a bit each
    __shared__ Pair sums[kPickWarps];
    __shared__ float tops[kPickWarps];
    __shared__ int count, outside;
    __shared__ uint64_t bound;
    const int tid = threadIdx.x;
    const uint32_t b = blockIdx.x;
    const int nlists = p.K * p.splits;
    const float4* all_stat = p.stat + (int64_t)b * nlists;
    const uint64_t* all_list = p.list + (int64_t)b * nlists * p.n;
    float s = 0.0f;
    bool done = false;
    if (tid < p.K) {
        s = p.scores[b * p.K + tid];
        done = p.finished && p.finished[b * p.K + tid];
    }
    if (tid == 0) doubt = 0;
    if (tid < nlists) stat[tid] = all_stat[tid];
    for (int i = tid; i < nlists * p.n; i += kPickThreads) lists[i] = all_list[i];
    __syncthreads();
    if (tid < p.K) {
        bool bad = !(s < INFINITY);
        int what = bad || s == -INFINITY ? 0 : done ? 2 : 1;
        Pair l{0.0f, 0.0f};
        float err = 0.0f;
        if (what == 1) {
            const float4* st = stat + tid * p.splits;
            const uint64_t* first = lists + tid * p.splits * p.n;
            float top = -INFINITY, high = -INFINITY;
            for (int g = 0; g < p.splits; ++g) {
                const uint64_t c = first[g * p.n];
                if (c) high = fmaxf(high, unordered((uint32_t)(c >> 32)));
                bad |= st[g].x != st[g].x;
                if (st[g].y != 0.0f) top = fmaxf(top, st[g].x);
            }
            bad |= high == INFINITY;
            if (p.fused && !bad) {
                bool sure = top > -INFINITY;
                Pair sum{0.0f, 0.0f};                  // at the reference `top`
                for (int g = 0; g < p.splits; ++g) {
                    const float4 q = st[g];
                    if (q.y == 0.0f) continue;
                    sure &= q.y < 1e30f && q.y > 1e-30f;           // not NaN either
                    const Pair part{q.y, q.z};
                    sum = add(sum, q.x == top ? part : mul(part, exp_pair(q.x, top)));
                    err = fmaxf(err, q.w);
                }
                sure &= sum.h >= 1.0f && sum.h < 1e30f;
                if (sure) {
                    l = add(Pair{top, 0.0f}, log_pair(sum));
                } else if (high > -INFINITY || sum.h != sum.h) {
                    atomicOr(&doubt, 1ull << tid);     // NaN, or out of the streamed sum's range
                    high = 0.0f;
                }
            }
            if (bad || high == -INFINITY) what = 0;
        }
        if (bad && p.status) *p.status = RNNT_INVALID_VALUE;
        lse[tid] = l;
        score[tid] = s;
        error[tid] = err;
        kind[tid] = (uint8_t)what;
    }
    __syncthreads();
    const int list = tid / kParts, part = tid % kParts, k = list / p.splits;    // of this thread
    for (unsigned long long again = doubt;;) {
        for (; again; again &= again - 1) {
            const int kk = __ffsll((long long)again) - 1;
            const Pair l = exact_lse(row_of<T>(p, b * p.K + kk), p.V, sums, tops);
            if (tid == 0) {
                lse[kk] = l;
                error[kk] = 0.0f;
                if (l.h != l.h) {                      // it holds NaN
                    kind[kk] = 0;
                    if (p.status) *p.status = RNNT_INVALID_VALUE;
                }
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
            if (what == 2) return list == k * p.splits && j == 0 ? ordered(Pair{score[k], 0.0f}) : 0;
            const uint64_t c = what == 1 && j < p.n ? lists[list * p.n + j] : 0;
            if (!c) return 0;
            const Pair v = two_sum(score[k], unordered((uint32_t)(c >> 32)));
            return ordered(add(v, Pair{-lse[k].h, -lse[k].l}));
        };
        auto number = [&](int j) {
            return (uint32_t)k << kTokenBits | (what == 2 ? 0u : ~(uint32_t)lists[list * p.n + j]);
        };
        const uint64_t first = value(0);
        if (part == 0 && list < nlists) heads[list] = first;
        __syncthreads();
        int rank = 0;
        if (first)
            for (int j = part; j < nlists; j += kParts)
                rank += heads[j] > first || (heads[j] == first && j < list);
#pragma unroll
        for (int o = 1; o < kParts; o *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
        if (first && rank == p.Ko - 1) bound = first;
        __syncthreads();
        // element j of the list of rank r has j + r better ones
        if (first && rank < p.Ko)
            for (int j = part; j + rank < p.Ko; j += kParts) {
                const uint64_t v = value(j);
                if (v < bound) break;
                const int to = atomicAdd(&count, 1);
                cval[to] = v;
                cid[to] = number(j);
            }
        __syncthreads();
        const int c = count, found = min(c, p.Ko);
        constexpr int kCount = 4;                      // threads that count for a candidate
        for (int i0 = 0; i0 < c; i0 += kPickThreads / kCount) {
            const int i = i0 + tid / kCount;
            const uint64_t v = i < c ? cval[i] : ~0ull;
            const uint32_t d = i < c ? cid[i] : 0;
            int r = 0;
            if (i < c)
                for (int j = tid % kCount; j < c; j += kCount)
                    r += cval[j] > v || (cval[j] == v && cid[j] < d);
#pragma unroll
            for (int o = 1; o < kCount; o *= 2) r += __shfl_xor_sync(0xffffffffu, r, o);
            if (i < c && r < p.Ko && tid % kCount == 0) {
                oval[r] = v;
                oid[r] = d;
            }
        }
        __syncthreads();
        if (!p.fused || found == 0) break;
        // Neighbours of different beams whose order is in doubt.
        if (tid + 1 < found) {
            const int k0 = oid[tid] >> kTokenBits, k1 = oid[tid + 1] >> kTokenBits;
            if (k0 != k1 && difference(oval[tid], oval[tid + 1]) < error[k0] + error[k1])
                atomicOr(&doubt, (error[k0] > 0.0f ? 1ull << k0 : 0) |
                                 (error[k1] > 0.0f ? 1ull << k1 : 0));
        }
        // Beams with candidates as near to the last one, some of them left out.
        if (found == p.Ko && first) {
            const uint64_t last = oval[found - 1];
            const float within = error[k] + error[oid[found - 1] >> kTokenBits];
            for (int j = part; j < p.n; j += kParts) {
                const uint64_t v = value(j);
                if (!v) break;
                const float d = difference(v, last);
                if (d < -within) break;
                if (d > within) continue;
                atomicOr(&border, 1ull << k);
                if (v < last || (v == last && number(j) > oid[found - 1])) outside = 1;
            }
        }
        __syncthreads();
        again = doubt;
        if (outside && __popcll(border) > 1)
            for (unsigned long long left = border; left; left &= left - 1) {
                const int kk = __ffsll((long long)left) - 1;
                if (error[kk] > 0.0f) again |= 1ull << kk;
            }
        if (!again) break;
        __syncthreads();       // `doubt` and `border` have been read
    }
    for (int r = tid; r < p.Ko; r += kPickThreads) {
        const int64_t o = (int64_t)b * p.Ko + r;
        const int from = r < min(count, p.Ko) ? (int)(oid[r] >> kTokenBits) : -1;
        p.out_scores[o] = from < 0 ? -INFINITY : unordered((uint32_t)(oval[r] >> 32));
        p.out_tokens[o] = from < 0 || kind[from] == 2 ? -1 : (int)(oid[r] & kTokenMask);
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
    const int64_t vecs = std::max(1, V / E);                 // the most, whatever the alignment
    // one tile a CTA where that gives no more than a wave of 6 CTAs an SM, else a wave of 4
    const int64_t rows = (int64_t)B * K, tiles = (vecs + kRowThreads - 1) / kRowThreads;
    int64_t splits = rows * tiles <= 152 * 6 ? tiles : std::min(tiles, 152 * 4 / rows);
    splits = std::max<int64_t>(1, std::min<int64_t>(splits, kMaxLists / K));
    L.split_vecs = (int32_t)((vecs + splits - 1) / splits);
    L.splits = (int32_t)((vecs + L.split_vecs - 1) / L.split_vecs);
    L.n = std::min(Ko, V);
    const size_t units = (size_t)B * K * L.splits;
    L.stat = 0;
    L.list = align256(units * sizeof(float4));
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
    p.stat = reinterpret_cast<float4*>(ws + L.stat);
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
