// rnnt_beam.cu -- beam search: selection over beams and vocabulary, and the
// reordering of states by the selected beams.
//
// Selection.  A live beam k with score s_k and logits x_k offers, for every
// output v with x_kv > -inf, the candidate s_k + x_kv - lse(x_k) (lse = 0 for
// log-probabilities); a finished beam offers itself, with its score and token
// -1; a beam of score -inf offers nothing.  The Ko best of a batch item are
// selected, ties going to the lowest beam and then the lowest token.
#include <cooperative_groups.h>

#include <atomic>

#include "rnnt_labels.cuh"

namespace cg = cooperative_groups;
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
// A row is cut into splits of whole aligned 16-byte vectors (the few elements ahead of them go to
// threads of the first split one by one, those behind them to the last split's, so that the splits
// are in the order of the tokens); a CTA streams one split through registers and writes
//   - the sum of exp(x - r) over the split and its reference r.  r is the first tile's
//     maximum and changes only when a thread meets a value more than 16 above it, so
//     that a sum is (almost) never rescaled.
//   - the n best elements in order.  The stream keeps each thread's maximum of every
//     tile and nothing else.  Of every warp's largest thread maxima enough to make n together
//     bound the n-th best element from below (the least of them does); the few tiles of a
//     thread that reach the bound are read once more, from the cache, and their elements
//     that reach it are ranked by counting.  Rows with a crowd of equal elements at the
//     bound go through best_of_row instead, tile by tile.
// Memory bounds it where rows are long (one read of the logits): 1024 rows of 200000 bfloat16, all
// at once, take 87 us with k_pick (4.7 TB/s; the ex2 units are busy for 23 % of it, the issue slots
// for 48 %), of 50000 28 us and 6 more for k_pick, of which 13 do not depend on the length:
// the first loads and, behind the stream, a chain of barriers (bound, second look, ranking).
constexpr int kRowThreads = 128;           // of k_rows: 8 CTAs an SM hold 1024 rows at once (256
                                           // threads, 4 CTAs: a second wave, 32 against 28 us)
constexpr int kClusterThreads = 128;       // of k_search
constexpr int kMaxCluster = 16;            // where the device runs clusters of so many blocks
constexpr int kAnyCluster = 8;             // which every device runs
constexpr int kClusterBytes = 32 << 10;    // of a row that a CTA of a cluster takes, at most
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
constexpr int kMaxLists = 128;             // splits of a batch item's rows
constexpr int kBuf = 1024;                 // elements ranked at a time: > 3 TH (best_of_row)
// Slots of tiles, whose maxima a thread keeps: a slot that reaches the bound is read once more as a
// whole.  Blocks with fewer than 4 vectors a thread have one tile.  (64 x 16 rows of 200000
// bfloat16: 96 us with 8 slots, 89 with 16, 87 with 32; no difference up to 50000.)
template <int NV, int MOST> constexpr int kSlots = NV == 4 ? MOST : 1;

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
// Keys of values beyond float32's range, in their order and outside the keys of finite values, from a
// quarter of each (2^126 <= |a| <= 3 2^126).  They take the patterns that read as NaN, of which there
// are half as many as such pairs: the last bit goes, of about 47.  Never 0.
constexpr float kMost = 3.40282347e38f;                // the largest float32
constexpr uint32_t kOrderedMost = 0xff7fffffu, kOrderedLeast = 0x00800000u;   // of kMost, -kMost
__device__ __forceinline__ uint64_t ordered_beyond(Pair a) {
    const uint64_t least = a.h < 0.0f ? (uint64_t)0x00bfffffu << 32        // ordered(-3 2^126)
                                      : (uint64_t)0xfe800000u << 32;       // ordered(2^126)
    const uint64_t base = a.h < 0.0f ? 1ull << 32 : (uint64_t)(kOrderedMost + 1) << 32;
    return base + ((ordered(a) - least) >> 1);
}
// What is returned for a key: the value's float32 rounding.
__device__ __forceinline__ float score_of(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return o < kOrderedLeast ? -INFINITY : o > kOrderedMost ? INFINITY : unordered(o);
}
// NaN or infinite where a key is of a value beyond float32's range, whose step is more than any
// log-sum-exp's error.
__device__ __forceinline__ float difference(uint64_t a, uint64_t b) {
    return (unordered((uint32_t)(a >> 32)) - unordered((uint32_t)(b >> 32))) +
           (unordered((uint32_t)a) - unordered((uint32_t)b));
}

// The key of score + x - lse.  Where one of the steps passes float32's range (masks of the type's
// lowest value in two steps of a search do), the sum is taken of quarters, which is exact.
__device__ __noinline__ uint64_t key_of_far(float score, float x, Pair lse) {
    const Pair q = add(two_sum(0.25f * score, 0.25f * x), Pair{-0.25f * lse.h, -0.25f * lse.l});
    const Pair v{4.0f * q.h, 4.0f * q.l};
    return fabsf(v.h) <= kMost ? ordered(v) : ordered_beyond(q);
}
__device__ __forceinline__ uint64_t key_of_sum(float score, float x, Pair lse) {
    const Pair v = add(two_sum(score, x), Pair{-lse.h, -lse.l});
    return fabsf(v.h) + fabsf(v.l) <= kMost ? ordered(v) : key_of_far(score, x, lse);   // not NaN
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
template <int TH>
__device__ __forceinline__ void rank_keys(const uint64_t* buf, int c, uint64_t* best, int n) {
    const int part = threadIdx.x & 3;
    for (int i0 = 0; i0 < c; i0 += TH / 4) {
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
template <int TH>
__device__ __noinline__ void keep_best(uint64_t* buf, uint64_t* best, int* count, int n) {
    const int c = *count, m = min(c, n);
    rank_keys<TH>(buf, c, best, n);
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

// Largest element of a tile's vectors (NaN is passed over).
template <int NV>
__device__ __forceinline__ float tile_max(const Pack<float, 16> (&v)[NV]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        m = fmaxf(m, fmaxf(fmaxf(v[i].e[0], v[i].e[1]), fmaxf(v[i].e[2], v[i].e[3])));
    return m;
}
template <typename T, int NV>
__device__ __forceinline__ float tile_max(const Pack<T, 16> (&v)[NV]) {
    using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    T2 m[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const T2* h = reinterpret_cast<const T2*>(&v[i].raw);
        m[i] = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    }
#pragma unroll
    for (int o = NV / 2; o; o /= 2)
#pragma unroll
        for (int i = 0; i < o; ++i) m[i] = __hmax2(m[i], m[i + o]);
    return fmaxf(__low2float(m[0]), __high2float(m[0]));
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

// The element ahead of the row's whole vectors (of the first split) or behind them (of the last)
// that is this thread's, or -1.
template <typename T>
__device__ __forceinline__ int odd_element(const SelectParams& p, uint32_t row, int split) {
    constexpr int E = 16 / (int)sizeof(T);
    const bool front = threadIdx.x < E;
    if (threadIdx.x >= 2 * E || split != (front ? 0 : p.splits - 1)) return -1;
    const int ahead = min(p.V, (int)(-(uintptr_t)row_of<T>(p, row) & 15) / (int)sizeof(T));
    const int behind = ahead + (p.V - ahead) / E * E;
    const int at = front ? threadIdx.x : behind + threadIdx.x - E;
    return at < (front ? ahead : p.V) ? at : -1;
}

// The n best of a split to best: every tile of TH vectors gives its elements above the
// bound, the n-th best so far; a tile that has too many gives them element by element of each
// thread's vector.
template <typename T, int TH>
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
    for (int t0 = 0; t0 < sp.vecs; t0 += TH) {
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
            if (*count > TH) {
                keep_best<TH>(buf, best, count, n);
                least = max(least, buf[n - 1]);        // n < TH
            }
        }
    }
    __syncthreads();
    rank_keys<TH>(buf, *count, best, n);
    __syncthreads();
}

template <int TH, int SLOTS>
struct RowShared {
    union {
        float tops[SLOTS][TH];            // each thread's maxima of the slots
        uint64_t buf[kBuf];               // keys to be ranked, once the tops have been read
    };
    uint64_t best[RNNT_MAX_BEAM];         // the split's list
    float4 stat;
    Pair wsum[(TH / 32)];
    float wref[(TH / 32)], wleast[(TH / 32)], wover[(TH / 32)];
    uint16_t hit[kBuf];                   // slots to be read once more: each has an element that is
                                          // ranked, so more of them are a crowd
    int hits, count, bads, rescales;
};

// Leaves the split's statistics and list (zeros behind its end) in sh, behind a barrier; returns
// false, at once, for a beam that offers no logits.
template <typename T, int NV, bool FUSED, int TH, int SLOTS>
__device__ __forceinline__ bool row_pass(const SelectParams& p, uint32_t row, int split,
                                         RowShared<TH, SLOTS>& sh) {
    constexpr int E = 16 / (int)sizeof(T);
    constexpr int kTileVecs = TH * NV;
    auto& buf = sh.buf;
    auto& best = sh.best;
    auto& wsum = sh.wsum;
    auto& wref = sh.wref;
    auto& wleast = sh.wleast;
    auto& wover = sh.wover;
    auto& tops = sh.tops;
    auto& hit = sh.hit;
    int &hits = sh.hits, &count = sh.count, &bads = sh.bads, &rescales = sh.rescales;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Split<T> sp(p, row, split);
    const int vecs = sp.vecs;
    auto load_tile = [&](Pack<T, 16>* v, int t0) {
        if (t0 + kTileVecs <= vecs) {                        // for the whole block
#pragma unroll
            for (int i = 0; i < NV; ++i)
                v[i].raw = load_stream(sp.aligned + t0 + i * TH + tid);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = sp.at(t0 + i * TH + tid);
        }
    };
    Pack<T, 16> v[NV], next[NV];
    load_tile(v, 0);
    const int odd = odd_element<T>(p, row, split);
    const float odd_x = odd >= 0 ? to_f32(row_of<T>(p, row)[odd]) : -INFINITY;
    if (!reads_logits(p, row)) return false;       // asked for while the loads are in flight
    if (tid == 0) hits = count = bads = rescales = 0;
    __syncthreads();

    float ref = 0.0f, sum = 0.0f, low = 0.0f;      // sum + low: the running sum
    float most = odd_x;                            // the thread's maximum
    bool bad = !FUSED && !(odd_x < INFINITY), rescaled = false;
    int shift_slot = 0;                            // tiles of a slot: 1 << shift_slot
    while ((vecs - 1) / kTileVecs >> shift_slot >= SLOTS) ++shift_slot;
    float slot_top = -INFINITY;
    for (int t0 = 0; t0 < vecs || t0 == 0; t0 += kTileVecs) {
        if (t0 + kTileVecs < vecs) load_tile(next, t0 + kTileVecs);
        float top = tile_max(v);
        if (!FUSED) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) bad |= !(to_f32(v[i].e[e]) < INFINITY);
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
                for (int w = 1; w < (TH / 32); ++w) ref = fmaxf(ref, wref[w]);
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
                if (i && t0 + i * TH >= vecs) continue;     // for the whole block
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
    const int whole = min(vecs / 32, (TH / 32));       // warps whose threads all have a maximum
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
    for (int w = 0; w < (TH / 32); ++w)
        if (w < whole) least = fminf(least, wleast[w]);
    const int span = kTileVecs << shift_slot;
    for (int t = 0; t * span < vecs; ++t) {
        const bool reaches = tops[t][tid] >= least && tops[t][tid] > -INFINITY;
        const unsigned who = __ballot_sync(0xffffffffu, reaches);
        if (!who) continue;
        int to = 0;
        if (lane == 0) to = atomicAdd(&hits, __popc(who));
        to = __shfl_sync(0xffffffffu, to, 0) + __popc(who & ((1u << lane) - 1));
        if (reaches && to < kBuf) hit[to] = (uint16_t)(t * TH + tid);
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
            for (int w = 1; w < (TH / 32); ++w) at = fmaxf(at, wref[w]);
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
    for (int i = tid; i < min(hits, kBuf) * per; i += TH) {
        const int slot = hit[i / per];
        const int j = slot / TH * span + i % per * TH + slot % TH;
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
    const bool crowd = hits > kBuf || count > kBuf;
    if (warp == (TH / 32) - 1) {                   // the keys are ranked by the first ones
        Pair total{0.0f, 0.0f};
        float over = 0.0f, err = 0.0f;
        if (FUSED) {
            if (lane < (TH / 32)) {
                total = wsum[lane];
                over = wover[lane];
            }
#pragma unroll
            for (int o = (TH / 32) / 2; o; o >>= 1) {
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
            sh.stat = make_float4(FUSED ? at : bads ? NAN : 0.0f, total.h, total.l, err);
    }
    if (!crowd) rank_keys<TH>(buf, count, best, p.n);
    __syncthreads();
    if (crowd) best_of_row<T, TH>(p, row, split, buf, best, &count);
    for (int i = count + tid; i < p.n; i += TH) best[i] = 0;
    __syncthreads();
    return true;
}


template <typename T, int NV, bool FUSED>
__global__ void __launch_bounds__(kRowThreads, NV == 1 ? 12 : 8) k_rows(const SelectParams p) {
    __shared__ RowShared<kRowThreads, kSlots<NV, 32>> sh;
    let_next_start();
    const uint32_t row = blockIdx.x / (uint32_t)p.splits;
    const int split = (int)(blockIdx.x - row * (uint32_t)p.splits);
    if (!row_pass<T, NV, FUSED>(p, row, split, sh)) return;
    uint64_t* list = p.list + (int64_t)blockIdx.x * p.n;
    if (threadIdx.x < p.n) list[threadIdx.x] = sh.best[threadIdx.x];
    if (threadIdx.x == 0) p.stat[blockIdx.x] = sh.stat;
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
// One CTA per batch item.  Every (beam, split) list is in order, so the best candidate is among
// the lists' heads: one warp holds them, up to 4 a lane, and takes Ko times the largest.  Latency
// bounds it: 6 us behind k_rows for 64 items of 16 lists (5 less in the whole call with one warp's
// selection than with ranks by counting, which compares all candidates with all).
//
// The streamed sums leave a log-sum-exp off by error[k] (see kTermError).  Where the order of
// two candidates of different beams is closer than that, the beams' log-sum-exps are computed
// again to 40 bits and the selection is repeated.  With 50000 outputs the bound is about
// 1e-6, and 1 call in 15 of 64 items x 16 beams meets such a pair.
constexpr int kPickThreads = 512;          // of k_pick
// a[i] of an array in registers.
template <int L>
__device__ __forceinline__ int sel(const int (&a)[L], int i) {
    int x = a[0];
#pragma unroll
    for (int q = 1; q < L; ++q) x = i == q ? a[q] : x;
    return x;
}

// log sum exp of a row by the whole block, the same for equal rows wherever they lie; NaN
// where the row holds NaN or +inf.
template <typename T, int THREADS>
__device__ __noinline__ Pair exact_lse(const T* x, int V, Pair* sums, float* tops) {
    constexpr int kPickThreads = THREADS, kPickWarps = THREADS / 32;
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

struct PickShared {
    uint64_t oval[RNNT_MAX_BEAM];           // the best, in order: ordered value, list << 8 | element
    uint32_t oid[RNNT_MAX_BEAM];
    uint8_t obeam[RNNT_MAX_BEAM];
    Pair lse[RNNT_MAX_BEAM];
    float score[RNNT_MAX_BEAM], error[RNNT_MAX_BEAM];
    uint8_t kind[RNNT_MAX_BEAM];            // 0 nothing, 1 logits, 2 finished
    unsigned long long again;               // beams whose log-sum-exp is wanted exactly
    Pair sums[32];
    float tops[32];
    int found;
};

__device__ __forceinline__ unsigned long long or_lanes(unsigned long long x) {
    return (unsigned long long)__reduce_or_sync(0xffffffffu, (uint32_t)(x >> 32)) << 32 |
           __reduce_or_sync(0xffffffffu, (uint32_t)x);
}

// An item's beams from their scores, whether they are finished (or null), and their lists
// ([K * splits][n]) and statistics, in shared memory already (behind the barrier here); leaves in
// sh.again the beams whose log-sum-exp is wanted exactly.
template <int THREADS>
__device__ __forceinline__ void weigh(const SelectParams& p, const float* scores,
                                      const uint8_t* finished, const uint64_t* lists,
                                      const float4* stat, PickShared& sh) {
    const int tid = threadIdx.x;
    if (tid == 0) sh.again = 0;
    __syncthreads();
    // A beam's log-sum-exp from its splits: by one thread, or a warp's lanes together.
    const int group = p.splits == 1 ? 1 : 32;
    for (int k = tid / group; k < p.K; k += THREADS / group) {
        const float score = scores[k];
        const bool done = finished && finished[k];
        const float4* st = stat + k * p.splits;
        const uint64_t* first = lists + k * p.splits * p.n;
        bool bad = !(score < INFINITY);
        int what = bad || score == -INFINITY ? 0 : done ? 2 : 1;
        Pair l{0.0f, 0.0f};
        float err = 0.0f;
        if (what == 1) {
            float top = -INFINITY, high = -INFINITY;
            bool nan = false;
            for (int g = tid & (group - 1); g < p.splits; g += group) {
                const uint64_t c = first[g * p.n];
                if (c) high = fmaxf(high, unordered((uint32_t)(c >> 32)));
                nan |= st[g].x != st[g].x;
                if (st[g].y != 0.0f) top = fmaxf(top, st[g].x);
            }
            for (int o = group / 2; o; o >>= 1) {
                high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                nan |= __shfl_xor_sync(0xffffffffu, (int)nan, o) != 0;
            }
            bad = nan || high == INFINITY;
            if (p.fused && !bad) {
                bool sure = top > -INFINITY;
                Pair sum{0.0f, 0.0f};                  // at the reference `top`
                for (int g = tid & (group - 1); g < p.splits; g += group) {
                    const float4 q = st[g];
                    if (q.y == 0.0f) continue;
                    sure &= q.y < 1e30f && q.y > 1e-30f;           // not NaN either
                    const Pair part{q.y, q.z};
                    sum = add(sum, q.x == top ? part : mul(part, exp_pair(q.x, top)));
                    err = fmaxf(err, q.w);
                }
                for (int o = group / 2; o; o >>= 1) {
                    sum = add(sum, shuffled(sum, o));
                    err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, o));
                    sure &= __shfl_xor_sync(0xffffffffu, (int)sure, o) != 0;
                }
                sure &= sum.h >= 1.0f && sum.h < 1e30f;
                if (sure) {
                    l = add(Pair{top, 0.0f}, log_pair(sum));
                } else if (high > -INFINITY || sum.h != sum.h) {
                    // NaN, or out of the streamed sum's range
                    if ((tid & (group - 1)) == 0) atomicOr(&sh.again, 1ull << k);
                    high = 0.0f;
                }
            }
            if (bad || high == -INFINITY) what = 0;
        }
        if ((tid & (group - 1)) == 0) {
            if (bad && p.status) *p.status = RNNT_INVALID_VALUE;
            sh.lse[k] = l;
            sh.score[k] = score;
            sh.error[k] = err;
            sh.kind[k] = (uint8_t)what;
        }
    }
    __syncthreads();
}

// What a beam's exact log-sum-exp changes, by one thread.
__device__ __forceinline__ void settle(const SelectParams& p, PickShared& sh, int k, Pair l) {
    sh.lse[k] = l;
    sh.error[k] = 0.0f;
    if (l.h != l.h) {                      // the row holds NaN
        sh.kind[k] = 0;
        if (p.status) *p.status = RNNT_INVALID_VALUE;
    }
}

// The selection by the log-sum-exps at hand; leaves in sh.again the beams whose log-sum-exp it
// wants exactly before it can be sure.  `values` is as large as the lists, of which there are 32 L
// at most.
template <int THREADS, int L>
__device__ __forceinline__ void choose(const SelectParams& p, const uint64_t* lists,
                                       uint64_t* values, PickShared& sh) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int nlists = p.K * p.splits;
    // Ordered values of the lists' elements, 0: none.
    for (int m = tid; m < nlists * p.n; m += THREADS) {
        const int i = m / p.n, k = i / p.splits, what = sh.kind[k];
        uint64_t v = 0;
        if (what == 2) {
            if (m == k * p.splits * p.n) v = ordered(Pair{sh.score[k], 0.0f});
        } else if (const uint64_t c = what == 1 ? lists[m] : 0) {
            v = key_of_sum(sh.score[k], unordered((uint32_t)(c >> 32)), sh.lse[k]);
        }
        values[m] = v;
    }
    __syncthreads();
    if (tid < 32) {
        uint64_t head[L];
        int at[L];
#pragma unroll
        for (int q = 0; q < L; ++q) {
            const int i = q * 32 + lane;
            at[q] = 0;
            head[q] = i < nlists ? values[i * p.n] : 0;
        }
        int found = 0;
        bool lost = false;                         // the same for the whole warp
        for (; found < p.Ko; ++found) {
            uint64_t v = head[0];
            int q0 = 0;
#pragma unroll
            for (int q = 1; q < L; ++q)
                if (head[q] > v) {                 // equal: the lower list
                    v = head[q];
                    q0 = q;
                }
            const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
            if (!hi) break;
            const uint32_t lo = __reduce_max_sync(
                0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
            // of equal values the lowest list: the lowest beam, and token, as its lists are in
            // the order of the tokens and each one's equal elements are
            const uint32_t list = __reduce_min_sync(
                0xffffffffu, v == ((uint64_t)hi << 32 | lo) ? (uint32_t)(q0 * 32 + lane)
                                                            : 0xffffffffu);
            // No lane's, which cannot be: nothing is indexed by it, and no result stays.
            const bool some = list < (uint32_t)nlists;
            lost |= !some;
            if (some && (list & 31) == lane) {
                sh.oval[found] = v;
                sh.oid[found] = list << 8 | sel(at, q0);
#pragma unroll
                for (int q = 0; q < L; ++q)
                    if (q == q0) {
                        ++at[q];
                        head[q] = at[q] < p.n ? values[list * p.n + at[q]] : 0;
                    }
            }
            __syncwarp();
        }
        if (lost) {
            found = 0;
            if (lane == 0 && p.status) *p.status = RNNT_LAUNCH_FAILED;
        }
        __syncwarp();
        for (int r = lane; r < found; r += 32) sh.obeam[r] = (uint8_t)((sh.oid[r] >> 8) / p.splits);
        __syncwarp();
        unsigned long long doubt = 0;
        if (p.fused && found) {
            // Neighbours of different beams whose order is in doubt.
            for (int r = lane; r + 1 < found; r += 32) {
                const int k0 = sh.obeam[r], k1 = sh.obeam[r + 1];
                const float e0 = sh.error[k0], e1 = sh.error[k1];
                if (k0 != k1 && difference(sh.oval[r], sh.oval[r + 1]) < e0 + e1)
                    doubt |= (e0 > 0.0f ? 1ull << k0 : 0) | (e1 > 0.0f ? 1ull << k1 : 0);
            }
            // Beams as near to the last one with candidates left out, and the selected ones
            // there: where that is more than one beam, any of them may belong.
            const uint64_t last = sh.oval[found - 1];
            const float own = sh.error[sh.obeam[found - 1]];
            unsigned long long out = 0, in = 0;
#pragma unroll
            for (int q = 0; q < L; ++q) {
                const int i = q * 32 + lane, k = i < nlists ? i / p.splits : 0;
                if (i < nlists && head[q] && difference(last, head[q]) <= own + sh.error[k])
                    out |= 1ull << k;
            }
            for (int r = lane; r < found; r += 32) {
                const int k = sh.obeam[r];
                if (difference(sh.oval[r], last) <= own + sh.error[k]) in |= 1ull << k;
            }
            out = or_lanes(out);
            in = or_lanes(in);
            doubt = or_lanes(doubt);
            if (out && __popcll(in | out) > 1)
                for (unsigned long long left = in | out; left; left &= left - 1) {
                    const int k = __ffsll((long long)left) - 1;
                    if (sh.error[k] > 0.0f) doubt |= 1ull << k;
                }
        }
        if (lane == 0) {
            sh.again = doubt;
            sh.found = found;
        }
    }
    __syncthreads();
}

template <int THREADS>
__device__ __forceinline__ void report(const SelectParams& p, uint32_t b, const uint64_t* lists,
                                       const PickShared& sh) {
    for (int r = threadIdx.x; r < p.Ko; r += THREADS) {
        const int64_t o = (int64_t)b * p.Ko + r;
        const int from = r < sh.found ? sh.obeam[r] : -1;
        p.out_scores[o] = from < 0 ? -INFINITY : score_of(sh.oval[r]);
        p.out_tokens[o] = from < 0 || sh.kind[from] == 2
                              ? -1 : (int)~(uint32_t)lists[(sh.oid[r] >> 8) * p.n + (sh.oid[r] & 255)];
        p.out_parents[o] = from;
    }
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) k_pick(const SelectParams p) {
    extern __shared__ uint64_t lists[];                // [K * splits][n], twice
    __shared__ float4 stat[kMaxLists];
    __shared__ PickShared sh;
    __shared__ float scores[RNNT_MAX_BEAM];
    __shared__ uint8_t finished[RNNT_MAX_BEAM];
    const uint32_t b = blockIdx.x;
    if (threadIdx.x < p.K) {                           // inputs: k_rows does not write them
        scores[threadIdx.x] = p.scores[b * p.K + threadIdx.x];
        finished[threadIdx.x] = p.finished && p.finished[b * p.K + threadIdx.x];
    }
    wait_for_previous();
    const int nlists = p.K * p.splits;
    const uint64_t* from = p.list + (int64_t)b * nlists * p.n;
    if (threadIdx.x < nlists) stat[threadIdx.x] = p.stat[(int64_t)b * nlists + threadIdx.x];
    for (int i = threadIdx.x; i < nlists * p.n; i += kPickThreads) lists[i] = from[i];
    weigh<kPickThreads>(p, scores, finished, lists, stat, sh);
    for (int turn = 0; turn <= RNNT_MAX_BEAM; ++turn) {        // each settles a beam at least
        for (unsigned long long again = sh.again; again; again &= again - 1) {
            const int k = __ffsll((long long)again) - 1;
            const Pair l = exact_lse<T, kPickThreads>(row_of<T>(p, b * p.K + k), p.V, sh.sums,
                                                      sh.tops);
            if (threadIdx.x == 0) settle(p, sh, k, l);
        }
        __syncthreads();
        if (nlists <= 32) choose<kPickThreads, 1>(p, lists, lists + nlists * p.n, sh);
        else choose<kPickThreads, kMaxLists / 32>(p, lists, lists + nlists * p.n, sh);
        if (!sh.again) break;
    }
    report<kPickThreads>(p, b, lists, sh);
}

// ------------------------------------------------------- both, by a cluster an item
// A cluster takes a batch item: each CTA streams a row and leaves its list and statistics in the
// first CTA's shared memory, which picks; where that wants exact log-sum-exps, each CTA
// computes its own row's.  One launch and no workspace.  Latency bounds it, a chain of the row's
// barriers, two cluster barriers and one maximum of the heads a selected hypothesis: 7.9 to 8.3 us
// in a graph for 1 x 4 x 1024 float16 (from one GPU to another), 10.6 for 32 x 10 x 29 float32, 8.0
// for 16 x 8 x 5000 float32 log-probabilities (two launches: 3 us more for the last, and 5 us more of the host's time).
template <int NV>
struct ClusterShared {
    union {
        RowShared<kClusterThreads, kSlots<NV, kClusterBytes / 16 / (4 * kClusterThreads)>> rows;
        PickShared pick;
    };
    float4 stat[kMaxCluster];
};

template <typename T, int NV, bool FUSED>
__global__ void __launch_bounds__(kClusterThreads, 8) k_search(const SelectParams p) {
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(16) char search_space[];
    using Shared = ClusterShared<NV>;
    Shared& sh = *reinterpret_cast<Shared*>(search_space);
    uint64_t* lists = reinterpret_cast<uint64_t*>(search_space + sizeof(Shared));
    const int rank = (int)cluster.block_rank();
    const uint32_t b = blockIdx.x / (uint32_t)p.K;
    cluster.barrier_arrive();                          // that every CTA has started:
    Shared& first = *cluster.map_shared_rank(&sh, 0);
    uint64_t* to_lists = cluster.map_shared_rank(lists, 0);
    const bool reads = row_pass<T, NV, FUSED>(p, b * p.K + rank, 0, sh.rows);
    cluster.barrier_wait();                            // here it is to be known
    if (reads) {
        if (threadIdx.x < p.n) to_lists[rank * p.n + threadIdx.x] = sh.rows.best[threadIdx.x];
        if (threadIdx.x == 0) first.stat[rank] = sh.rows.stat;
    }
    cluster.sync();
    if (rank == 0)
        weigh<kClusterThreads>(p, p.scores + b * p.K, p.finished ? p.finished + b * p.K : nullptr,
                               lists, sh.stat, sh.pick);
    for (int turn = 0; turn <= kMaxCluster; ++turn) {          // each settles a beam at least
        if (rank == 0) {
            if (turn || !sh.pick.again)
                choose<kClusterThreads, 1>(p, lists, lists + p.K * p.n, sh.pick);
        }
        if (!p.fused) break;                           // exact as it is
        cluster.sync();
        const unsigned long long again = first.pick.again;
        if (!again) break;
        if (again >> rank & 1) {
            const Pair l = exact_lse<T, kClusterThreads>(row_of<T>(p, b * p.K + rank), p.V,
                                                         sh.pick.sums, sh.pick.tops);
            if (threadIdx.x == 0) settle(p, first.pick, rank, l);
        }
        cluster.sync();
    }
    if (rank == 0) report<kClusterThreads>(p, b, lists, sh.pick);
    if (p.fused) cluster.sync();                       // its memory has been read
}

struct SelectLayout {
    size_t stat, list, total;
    int32_t splits, split_vecs, n;
    int32_t cluster;                       // CTAs of an item's cluster, or 0: two launches
};
// `widest`: the blocks of the largest cluster that the device runs.
SelectLayout select_layout(int32_t B, int32_t K, int32_t V, int32_t Ko, int dt, int widest) {
    SelectLayout L{};
    const int es = elem_size(dt), E = 16 / es;
    const int64_t vecs = std::max(1, V / E);                 // the most, whatever the alignment
    L.n = std::min(Ko, V);
    L.splits = 1;
    L.split_vecs = (int32_t)vecs;
    // A cluster's CTAs take a row each, whole, against splits over the whole device and a second
    // launch.  On the GPU they are level where rows are short (items of 4 and 16 rows of 5000
    // float16: 9.9 and 13.2 us against 9.7 and 14.1), and the one launch without a workspace
    // costs the host 5 us less; long rows (of 50000: 15.3 and 19.5 against 9.5 and 15.4) are
    // faster split, and their exact sums by k_pick's larger block.
    if (K <= widest && (int64_t)V * es <= kClusterBytes) {
        L.cluster = K;
        return L;
    }
    // one tile a CTA where that gives no more than a wave of 12 CTAs an SM, else a wave of 8
    const int64_t rows = (int64_t)B * K, tiles = (vecs + kRowThreads - 1) / kRowThreads;
    int64_t splits = rows * tiles <= 152 * 12 ? tiles : std::min(tiles, 152 * 8 / rows);
    splits = std::max<int64_t>(1, std::min<int64_t>(splits, kMaxLists / K));
    L.split_vecs = (int32_t)((vecs + splits - 1) / splits);
    L.splits = (int32_t)((vecs + L.split_vecs - 1) / L.split_vecs);
    const size_t units = (size_t)B * K * L.splits;
    L.stat = 0;
    L.list = align256(units * sizeof(float4));
    L.total = align256(L.list + units * L.n * sizeof(uint64_t));
    return L;
}
bool select_ok(int32_t B, int32_t K, int32_t V, int32_t Ko, int dt) {
    return B >= 1 && K >= 1 && K <= RNNT_MAX_BEAM && Ko >= 1 && Ko <= RNNT_MAX_BEAM && V >= 1 &&
           V <= RNNT_MAX_BEAM_VOCAB && valid_dtype(dt) &&
           (int64_t)B * K <= INT32_MAX / kMaxLists;
}

template <typename T>
bool launch_select(const SelectParams& p, int cluster, cudaStream_t st) {
    auto launch = [&](auto nv, auto fused) {
        constexpr int NV = decltype(nv)::value;
        constexpr bool FUSED = decltype(fused)::value;
        if (!cluster) {
            k_rows<T, NV, FUSED><<<(unsigned)(p.B * p.K * p.splits), kRowThreads, 0, st>>>(p);
            return true;
        }
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(p.B * cluster));
        cfg.blockDim = dim3(kClusterThreads);
        cfg.dynamicSmemBytes = sizeof(ClusterShared<NV>) + 2 * sizeof(uint64_t) * p.K * p.n;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, k_search<T, NV, FUSED>, p) == cudaSuccess;
    };
    auto by_size = [&](auto fused) {
        const int threads = cluster ? kClusterThreads : kRowThreads;
        if (p.split_vecs <= threads) return launch(std::integral_constant<int, 1>{}, fused);
        if (p.split_vecs <= 2 * threads) return launch(std::integral_constant<int, 2>{}, fused);
        return launch(std::integral_constant<int, 4>{}, fused);
    };
    if (!(p.fused ? by_size(std::true_type{}) : by_size(std::false_type{}))) {
        cudaGetLastError();
        return false;
    }
    if (cluster) return true;
    if (launch_after(k_pick<T>, dim3((unsigned)p.B), kPickThreads,
                     2 * sizeof(uint64_t) * p.K * p.splits * p.n, st, p))
        return true;
    cudaGetLastError();
    return false;
}

// The kernels' shared memory limits, raised once per device.
template <typename T>
bool raise_limits() {
    const auto raise = [](auto kernel, size_t most) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)most) == cudaSuccess &&
               cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                   cudaSuccess;
    };
    const size_t lists = 2 * sizeof(uint64_t) * kMaxCluster * RNNT_MAX_BEAM;
    const size_t most = sizeof(ClusterShared<4>) + lists;
    return raise(k_pick<T>, 2 * sizeof(uint64_t) * kMaxLists * RNNT_MAX_BEAM) &&
           raise(k_search<T, 1, true>, most) && raise(k_search<T, 1, false>, most) &&
           raise(k_search<T, 2, true>, most) && raise(k_search<T, 2, false>, most) &&
           raise(k_search<T, 4, true>, most) && raise(k_search<T, 4, false>, most);
}
bool select_prepared() {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return false;
    if (done[dev].load(std::memory_order_acquire)) return true;
    const bool ok = raise_limits<float>() && raise_limits<__half>() && raise_limits<__nv_bfloat16>();
    if (ok) done[dev].store(true, std::memory_order_release);
    else cudaGetLastError();
    return ok;
}

// Blocks of the largest cluster that each of k_search's forms gets on the current device: 16, or
// 8 where some does not fit (a part of a device, say) and where there is no device to ask. Asked
// once per device, and only where K and V leave it open.
template <typename T>
bool widest_fits() {
    const auto fits = [](auto kernel) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(kMaxCluster);
        cfg.blockDim = dim3(kClusterThreads);
        cfg.dynamicSmemBytes =
            sizeof(ClusterShared<4>) + 2 * sizeof(uint64_t) * kMaxCluster * RNNT_MAX_BEAM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kMaxCluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
    };
    return fits(k_search<T, 1, true>) && fits(k_search<T, 1, false>) &&
           fits(k_search<T, 2, true>) && fits(k_search<T, 2, false>) &&
           fits(k_search<T, 4, true>) && fits(k_search<T, 4, false>);
}
int widest_cluster(int32_t K, int32_t V, int dt) {
    if (K <= kAnyCluster || K > kMaxCluster || (int64_t)V * elem_size(dt) > kClusterBytes)
        return kAnyCluster;
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices || !select_prepared()) {
        cudaGetLastError();
        return kAnyCluster;
    }
    int v = known[dev].load(std::memory_order_acquire);
    if (!v) {
        v = widest_fits<float>() && widest_fits<__half>() && widest_fits<__nv_bfloat16>()
                ? kMaxCluster : kAnyCluster;
        cudaGetLastError();
        known[dev].store(v, std::memory_order_release);
    }
    return v;
}

// ------------------------------------------------------------------ reorder
// Every state is a set of rows (three outer axes, batch, new beam) of
// contiguous bytes.  A CTA copies kCopyUnits units: several short rows, or a
// piece of a long one; all states of a call go in one launch.  Bound by memory: four caches of
// 32 x 8 hypotheses, 8 heads and 401 of 512 places of 64 float16 (280 MB read, 421 written) take
// 114 us, 6.1 TB/s; two LSTM states and the labels of 16 x 8 hypotheses (2.3 MB) 3.2 us in a graph.
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
    *bytes = select_layout(B, K, V, Ko, dt, widest_cluster(K, V, dt)).total;
    return RNNT_OK;
}

extern "C" rnnt_status_t rnnt_beam_select(const void* logits, rnnt_dtype_t dt, int32_t B, int32_t K,
                                          int32_t V, int64_t batch_stride, int64_t beam_stride,
                                          const float* scores, const uint8_t* finished, int32_t Ko,
                                          int32_t fused_log_softmax, float* out_scores,
                                          int32_t* out_tokens, int32_t* out_parents,
                                          void* workspace, size_t workspace_bytes,
                                          int32_t* status_dev, rnnt_stream_t stream) {
    if (!logits || !scores || !out_scores || !out_tokens || !out_parents) return RNNT_INVALID_VALUE;
    if (!select_ok(B, K, V, Ko, dt) || batch_stride < 0 || beam_stride < 0)
        return RNNT_INVALID_VALUE;
    const int es = elem_size(dt);
    if (((uintptr_t)logits & (es - 1)) || ((uintptr_t)workspace & 255)) return RNNT_INVALID_VALUE;
    const SelectLayout L = select_layout(B, K, V, Ko, dt, widest_cluster(K, V, dt));
    if (L.total && !workspace) return RNNT_INVALID_VALUE;
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
    if (!select_prepared() || !clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    if (!with_type(dt, [&](auto tag) { return launch_select<decltype(tag)>(p, L.cluster, st); }))
        return RNNT_LAUNCH_FAILED;
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
            if (i != j && d.dst == s.dst) return RNNT_INVALID_VALUE;
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
