// rnnt_sample.cu -- drawing labels: of every hypothesis one extension, from a random number that is
// given.
//
// With logits x, e_j = exp(x_j / tau) and a number u in [0, 1): outputs are ordered by logit (equal
// ones by id); of the first top_k the shortest beginning with a sum of e of at least top_p of
// theirs is kept, and of it what has e_j >= min_p max e.  All three keep a beginning of the order,
// so what is kept is what reaches one key (value and id).  The token is the first kept id at
// which the running sum of e, by id, exceeds u times the kept sum.
//
// Whether a sum reaches a border decides a whole number, so sums are taken as if held to 40 bits:
// fast ones, of float32 exponentials, come with a bound of their error, and where a border is nearer
// than that they are taken again in pairs of floats, of exponentials that are pairs themselves.
#include <cmath>

#include "rnnt_rows.cuh"

using namespace rnnt_rows;

namespace {

// ------------------------------------------------------------ pairs of floats
// Knuth's sum of two, Dekker's where one is the larger.  Their exact sum is the value: about 47 bits on
// float32 units, of which there are 64 times as many as of float64 ones.  The compiler neither reorders nor
// contracts what is spelt with intrinsics.
struct Pair { float h, l; };
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair fast_two_sum(float a, float b) {       // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const Pair s = two_sum(a.h, b.h);
    return fast_two_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    const float h = __fmul_rn(a.h, b.h);
    return fast_two_sum(h, __fadd_rn(__fmaf_rn(a.h, b.h, -h),
                                     __fmaf_rn(a.h, b.l, __fmul_rn(a.l, b.h))));
}
__device__ __forceinline__ bool less(Pair a, Pair b) {     // of pairs as add leaves them
    return a.h < b.h || (a.h == b.h && a.l < b.l);
}
__device__ __forceinline__ Pair shuffled(Pair a, int o) {
    return {__shfl_xor_sync(kAll, a.h, o), __shfl_xor_sync(kAll, a.l, o)};
}
__device__ __forceinline__ Pair shuffled_up(Pair a, int o) {
    return {__shfl_up_sync(kAll, a.h, o), __shfl_up_sync(kAll, a.l, o)};
}
inline Pair pair_of(double x) {
    const float h = (float)x;
    return {h, (float)(x - (double)h)};
}

// 2^(i / 16) as pairs.
__device__ const float2 kRoots[16] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}};
// 2^(d c) for d <= 0, relative error below 2^-40 down to 2^-120: d c = n + i / 16 + g, and 2^g = e^z,
// z = g ln 2, by its Taylor series (|z| < 0.0217: the first two terms in pairs, what follows is
// below 2e-6).  About 50 operations.
__device__ __forceinline__ Pair exp2_pair(Pair d, Pair c) {
    float th = __fmul_rn(d.h, c.h);
    const bool some = th > -120.0f;
    if (!some) {
        d = Pair{0.0f, 0.0f};
        th = 0.0f;
    }
    const float tl = __fadd_rn(__fmaf_rn(d.h, c.h, -th),
                               __fmaf_rn(d.h, c.l, __fmul_rn(d.l, c.h)));
    const float at = rintf(th * 16.0f);                    // in sixteenths
    const int k = (int)at, n = k >> 4;                     // rounded down
    const float gh = __fmaf_rn(at, -0.0625f, th);          // exact
    constexpr double ln2 = 0.69314718055994530942;
    constexpr float lh = (float)ln2, ll = (float)(ln2 - (double)lh);
    const float zh = __fmul_rn(gh, lh);
    const float zl = __fadd_rn(__fmaf_rn(gh, lh, -zh), __fmaf_rn(gh, ll, __fmul_rn(tl, lh)));
    const float qh = __fmul_rn(zh, zh);                    // z^2
    const float ql = __fmaf_rn(2.0f * zh, zl, __fmaf_rn(zh, zh, -qh));
    float tail = __fmaf_rn(zh, 1.0f / 120.0f, 1.0f / 24.0f);
    tail = __fmaf_rn(tail, zh, 1.0f / 6.0f);
    tail = __fmul_rn(tail, __fmul_rn(qh, zh));
    const Pair q = fast_two_sum(zh, 0.5f * qh);
    const float low = __fadd_rn(q.l, __fadd_rn(__fmaf_rn(0.5f, ql, zl), tail));
    const float2 r = __ldg(&kRoots[k & 15]);
    const float ph = __fmul_rn(r.x, q.h);
    const float pl = __fadd_rn(__fmaf_rn(r.x, q.h, -ph), __fmaf_rn(r.x, low, __fmul_rn(r.y, q.h)));
    const Pair e = fast_two_sum(r.x, ph);
    const Pair f = fast_two_sum(e.h, __fadd_rn(e.l, __fadd_rn(r.y, pl)));
    const float s = some ? __int_as_float((n + 127) << 23) : 0.0f;     // n >= -120
    return {f.h * s, f.l * s};
}

// --------------------------------------------------------------------- rows
struct SampleParams {
    const char* logits;
    int64_t batch_stride, beam_stride;     // bytes
    const float* scores;
    const float* random;
    const uint8_t* finished;
    int32_t B, K, V, top_k, fused;
    int32_t unit_tau;                      // temperature 1
    float scale, scale_low;                // log2 e / tau, in two parts
    float one, one_low;                    // log2 e
    float bin_scale;                       // bins of a logit's unit
    Pair exact_scale, top_p;               // log2 e / tau; top_p.h >= 1: not used
    double min_gap;                        // tau log min_p, or -inf
    float* out_scores;
    int32_t* out_tokens;
    int32_t* status;
};

// Keys of elements: their order as integers of 52 bits.
constexpr int kIdBits = 20;
static_assert(RNNT_MAX_TOP_VOCAB == 1 << kIdBits, "ids fill their bits of a key");
__device__ __forceinline__ uint64_t short_key(float x, int element) {
    return (uint64_t)ordered(x) << kIdBits | (uint32_t)((1 << kIdBits) - 1 - element);
}
constexpr uint64_t kFinite = (uint64_t)0x00800000u << kIdBits;   // the least key of a finite value

// A mass that is kept is above 0 however far it lies: u = 0 draws the first id.
constexpr float kLeastMass = 1.17549435e-38f;

// Fast sums are of float32 terms, added as trees of a vector's and then as pairs.  A border is u of a
// whole sum W, and a running sum R beside it is compared with u W.  A term is a function of its logit:
// relative to a factor that all share (and that cancels) it is off by at most kTerm and kStep for each
// of its exponent's binary orders.  ex2.approx is off by -1.44e-7 to 1.05e-7 (all float32 from -126 to 0,
// against exp2 in float64), so by 1.25e-7 from the middle; x - top and the exponent are rounded once each.
// The term counts 1 - u times in R - u W where it is in R, and -u times where it is not; the terms of R
// have a mean order of at most log2 V - log2 R (their entropy is at most log2 V), the others likewise.
// With R = u W and c = u (1 - u) that is
//   |error of R - u W| <= W [ c (2 kTerm + kStep (2 (log2 V - log2 W) - log2 c)) + kSum ],
// kSum for the pairs' own additions (below 2^-30 for the longest rows).  A vector's tree is off by
// kAdd of its sum, in R and in W alike where both add the same trees.  Nothing is assumed of how the
// errors are spread: equal logits share theirs, and 16-bit rows are full of them.  A border nearer
// to a sum than the bound is decided on sums of pairs: of 50000 normal logits (bfloat16) one row in 11 with
// top_p 0.9, one in 38 without filters; a row then takes 10 to 30 us more.
constexpr float kTerm = 1.27e-7f, kStep = 8.3e-8f, kSum = 2e-9f;
template <typename T>
constexpr float kAdd = (sizeof(T) == 4 ? 2.0f : 3.0f) * 5.97e-8f;              // additions, one after another
__device__ __forceinline__ float error_at(float u, float sum, int V, float term) {     // absolute
    const float c = fmaxf(u * (1.0f - u), 1e-12f);
    return sum * (c * (2.0f * term +
                       kStep * (2.0f * (__log2f((float)V) - __log2f(sum)) - __log2f(c))) + kSum);
}
// Where R and W add different trees: of a list's elements, one by one, and of the row's vectors.
template <typename T>
__device__ __forceinline__ float error_of_list(float u, float sum, int V) {
    return error_at(u, sum, V, kTerm) + 2.0f * u * kAdd<T> * sum;
}
__device__ __forceinline__ Pair add_loosely(Pair a, float b) {     // of sums of positive terms
    const Pair s = two_sum(a.h, b);
    return {s.h, __fadd_rn(s.l, a.l)};
}
__device__ __forceinline__ float difference(Pair a, Pair b) {
    return __fadd_rn(__fsub_rn(a.h, b.h), __fsub_rn(a.l, b.l));
}

constexpr int kBins = 1024;
constexpr float kBinsPerOrder = 32.0f;     // of the first histogram: bins of 2^(1/32)
constexpr int kList = 512;                 // elements that are put in order

template <int TH>
struct Shared {
    static constexpr int WARPS = TH / 32;
    union {
        uint32_t bins[kBins];
        uint64_t order[kList];
    };
    union {
        uint64_t list[kList];
        Pair masses[kList + 32];
    };
    uint32_t groups[32];                   // sums of 32 bins each
    Pair pairs[2][WARPS];
    float floats[WARPS];
    int ints[WARPS];
    unsigned long long low, high;          // keys
    uint64_t bar;                          // of the row's copy
    uint32_t before;
    int bin, count, token, kept;
    bool unsure;
};

// What is kept: values above `value`, and equal ones up to an id.
template <typename T>
struct Floor {
    T value;
    int last;
    __device__ __forceinline__ explicit Floor(uint64_t key) {
        const float f = unordered((uint32_t)(key >> kIdBits));
        value = not_below<T>(fmaxf(f, lowest<T>()));
        last = (1 << kIdBits) - 1 -
               (to_f32(value) == f ? (int)(key & ((1 << kIdBits) - 1)) : 0);
    }
    // The kept elements of a vector whose first has this id.
    __device__ __forceinline__ uint32_t kept(const Pack<T, 16>& v, int id) const {
        const uint32_t ge = reaching(v, value);
        if (!ge) return 0;
        const int more = last - id;        // ids up to last
        const uint32_t ids = more < 0 ? 0u : more > 30 ? ~0u : (2u << more) - 1u;
        return ge & (ids | reaching<true>(v, value));
    }
};

// A draw by a block of TH threads; the row lies in shared memory (HERE) or is read from the cache.
// Blocks of 128, 256 and 512 threads for rows of up to 4 KB, 32 KB and beyond.  Latency bounds short
// rows (4 of 1024 float16 with top_k 40: 9 us, one chain of barriers); issue slots and barriers long
// ones, of which two fit an SM: 1024 rows of 50000 bfloat16 take 110 us unfiltered, 147 with
// top_p 0.9 and min_p 0.002, 66 where few elements are kept.  What is seldom run is not inlined and gets a
// copy of this object: 200 to 290 bytes of a thread's stack, in the L1, beside 64 to 80 registers.
template <typename T, int TH, bool HERE>
struct Draw {
    static constexpr int E = 16 / (int)sizeof(T), WARPS = TH / 32;
    Shared<TH>& sh;
    const Row<T> r;
    uint4* const here;
    const float scale, scale_low, bin_scale;
    const Pair exact_scale, top_p;
    float top;
    bool unsure;                           // of the last result: the fast sums leave it open

    __device__ __forceinline__ Draw(const SampleParams& p, Shared<TH>& s, const T* x, uint4* stage)
        : sh(s), r(x, p.V), here(stage), scale(p.scale), scale_low(p.scale_low),
          bin_scale(p.bin_scale), exact_scale(p.exact_scale), top_p(p.top_p), top(0.0f), unsure(false) {}

    __device__ __forceinline__ Pack<T, 16> at(int j) const {
        if constexpr (HERE) {
            Pack<T, 16> v;
            v.raw = here[j];
            return v;
        } else {
            return r.load(j);
        }
    }
    __device__ __forceinline__ int id_of(int j, int e) const { return j * E + e - r.off; }

    // ---- masses: of pairs (exact), or float32
    __device__ __forceinline__ Pair mass(float x) const {
        const Pair e = exp2_pair(two_sum(x, -top), exact_scale);
        return e.h >= kLeastMass ? e : Pair{kLeastMass, 0.0f};
    }
    __device__ __forceinline__ float fast_mass(float x) const {
        return fmaxf(Exponent(top, scale, scale_low)(x), kLeastMass);
    }
    // One copy of the code: it is seldom run, and then mostly waits to be fetched.
    __device__ __noinline__ Pair exact_masses(uint4 raw, uint32_t kept) const {
        Pair s{0.0f, 0.0f};
        uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll 1
        for (int i = 0; i < 4 && kept; ++i) {              // a word's elements side by side
            float x, y = -INFINITY;
            if constexpr (sizeof(T) == 4) {
                x = __uint_as_float(w[0]);
            } else {
                const uint16_t a = (uint16_t)w[0], b = (uint16_t)(w[0] >> 16);
                x = to_f32(reinterpret_cast<const T&>(a));
                y = to_f32(reinterpret_cast<const T&>(b));
            }
            const Pair m = mass(x), n = sizeof(T) == 4 ? Pair{0.0f, 0.0f} : mass(y);
            s = add(s, add(kept & 1 ? m : Pair{0.0f, 0.0f},
                           sizeof(T) == 2 && (kept & 2) ? n : Pair{0.0f, 0.0f}));
            kept >>= sizeof(T) == 4 ? 1 : 2;
            w[0] = w[1], w[1] = w[2], w[2] = w[3];
        }
        return s;
    }
    template <bool EXACT>
    __device__ __forceinline__ Pair masses(const Pack<T, 16>& v, uint32_t kept) const {
        Pair s{0.0f, 0.0f};
        if constexpr (EXACT) {
            s = exact_masses(v.raw, kept);
        } else {
            const Exponent f(top, scale, scale_low);
            float2 e[E / 2];
            if (kept == (1u << E) - 1u) {
                s.h = fmaxf(terms_of(v, f, e), kLeastMass);
                return s;
            }
            unpack(v, e);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                e[i] = f(e[i]);
                e[i].x = kept >> (2 * i) & 1 ? fmaxf(e[i].x, kLeastMass) : 0.0f;
                e[i].y = kept >> (2 * i + 1) & 1 ? fmaxf(e[i].y, kLeastMass) : 0.0f;
            }
#pragma unroll
            for (int o = E / 4; o; o /= 2)
#pragma unroll
                for (int i = 0; i < o; ++i) e[i] = add2(e[i], e[i + o]);
            s.h = e[0].x + e[0].y;
        }
        return s;
    }
    template <bool EXACT>
    __device__ __forceinline__ Pair mass_of_vector(int j, const Floor<T>& f) const {
        const Pack<T, 16> v = at(j);
        const uint32_t kept = f.kept(v, id_of(j, 0));
        return kept ? masses<EXACT>(v, kept) : Pair{0.0f, 0.0f};
    }

    // ---- over the block
    __device__ __forceinline__ void sum2(Pair& a, Pair& b) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            a = add(a, shuffled(a, o));
            b = add(b, shuffled(b, o));
        }
        if (lane == 0) {
            sh.pairs[0][threadIdx.x >> 5] = a;
            sh.pairs[1][threadIdx.x >> 5] = b;
        }
        __syncthreads();
        a = lane < WARPS ? sh.pairs[0][lane] : Pair{0.0f, 0.0f};
        b = lane < WARPS ? sh.pairs[1][lane] : Pair{0.0f, 0.0f};
#pragma unroll
        for (int o = WARPS / 2; o; o >>= 1) {
            a = add(a, shuffled(a, o));
            b = add(b, shuffled(b, o));
        }
        a = Pair{__shfl_sync(kAll, a.h, 0), __shfl_sync(kAll, a.l, 0)};
        b = Pair{__shfl_sync(kAll, b.h, 0), __shfl_sync(kAll, b.l, 0)};
        __syncthreads();
    }
    // Sums of pairs over the keys from `least` and from `above` on.
    __device__ __noinline__ void exact_sums(uint64_t least, uint64_t above, Pair& whole,
                                            Pair& upper) const {
        Draw(*this).exact_sums_of(least, above, whole, upper);     // a copy, for registers
    }
    __device__ __forceinline__ void exact_sums_of(uint64_t least, uint64_t above, Pair& whole,
                                                  Pair& upper) {
        const Floor<T> f(least), g(above);
        Pair a{0.0f, 0.0f}, b{0.0f, 0.0f};
        for (int j = threadIdx.x; j < r.n; j += TH) {
            const Pack<T, 16> v = at(j);
            const uint32_t kept = f.kept(v, id_of(j, 0));
            if (!kept) continue;
            const uint32_t over = g.kept(v, id_of(j, 0));  // of those: above >= least
            if (over) b = add(b, masses<true>(v, over));
            if (kept != over) a = add(a, masses<true>(v, kept ^ over));
        }
        sum2(a, b);
        whole = add(a, b);
        upper = b;
    }
    // The least key, from `least` on, above which lies less than the target: by bisection.
    __device__ __noinline__ uint64_t bisect(uint64_t least, Pair target) {
        uint64_t lo = least, hi = short_key(top, 0);
        while (lo < hi) {
            const uint64_t mid = lo + (hi - lo) / 2;
            Pair whole, upper;
            exact_sums(mid + 1, mid + 1, whole, upper);
            if (less(whole, target)) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    }

    // ---- the first histogram's bins: by the exponent
    __device__ __forceinline__ int bin_of(float x) const {
        return (int)fminf((top - x) * bin_scale, (float)(kBins - 1));
    }
    // The bin at whose end `target` is reached (the last filled one if it is not), and what is in
    // those before it.
    __device__ __forceinline__ void find_bin(uint32_t target) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        for (int g = warp; g < kBins / 32; g += WARPS) {
            const uint32_t n = __reduce_add_sync(kAll, sh.bins[g * 32 + lane]);
            if (lane == 0) sh.groups[g] = n;
        }
        __syncthreads();
        if (warp == 0) {
            const auto find = [&](uint32_t mine, uint32_t& before) {   // the lane that reaches it
                uint32_t run = mine;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const uint32_t y = __shfl_up_sync(kAll, run, o);
                    if (lane >= o) run += y;
                }
                const unsigned at = __ballot_sync(kAll, mine && before + run >= target);
                const unsigned some = __ballot_sync(kAll, mine != 0);
                const int g = at ? __ffs(at) - 1 : some ? 31 - __clz(some) : 0;
                before += __shfl_sync(kAll, run - mine, g);
                return g;
            };
            uint32_t before = 0;
            const int g = find(sh.groups[lane], before);
            const int b = g * 32 + find(sh.bins[g * 32 + lane], before);
            if (lane == 0) {
                sh.bin = b;
                sh.before = before;
            }
        }
        __syncthreads();
    }

    // Puts a list in order that holds the border of `count` elements (MASS: of `target`, by fast
    // sums) among the keys from `least` on; returns its length, and in `above` (MASS) the sum of
    // the masses above the list or (else) `before`, the number of elements above it.
    // Each turn counts the elements of a range by bins and takes the bin in which the
    // border lies for the next range, until it holds few enough: first by their
    // exponents, then by the bits of their keys, which are all different.
    // With `few` the whole range is tried as a list first.
    template <bool MASS>
    __device__ __noinline__ int list_at(bool few, uint64_t least, uint32_t count, float target,
                                        float whole, Pair& above, uint32_t& before) const {
        return Draw(*this).template list_of<MASS>(few, least, count, target, whole, above, before);
    }
    template <bool MASS>
    __device__ __forceinline__ int list_of(bool few, uint64_t least, uint32_t count, float target,
                                           float whole, Pair& above, uint32_t& before) {
        const Floor<T> f(least);
        uint64_t low = 0, high = ~0ull;    // the range; whole at first
        int shift = -1;                    // of keys to bins; -1: by exponents
        uint32_t base = 0;                 // elements above the range
        float mass_above = 0.0f, mass_in = whole;
        above = Pair{0.0f, 0.0f};
        for (int turn = 0; turn < 12; ++turn) {
            const bool binned = !few || turn;
            if (binned)
                for (int i = threadIdx.x; i < kBins; i += TH) sh.bins[i] = 0;
            if (threadIdx.x == 0) {
                sh.count = 0;
                sh.low = ~0ull;
                sh.high = 0;
            }
            __syncthreads();
            const float unit = MASS ? 2147483648.0f / mass_in : 0.0f;
            const auto bin = [&](float x, uint64_t key) {
                return shift < 0 ? bin_of(x) : (int)((high - key) >> shift);
            };
            for (int j = binned ? (int)threadIdx.x : r.n; j < r.n; j += TH) {
                const Pack<T, 16> v = at(j);
                const uint32_t kept = f.kept(v, id_of(j, 0));
                if (!kept) continue;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (!(kept >> e & 1)) continue;
                    const float x = to_f32(v.e[e]);
                    uint64_t key = 0;
                    if (shift >= 0) {
                        key = short_key(x, id_of(j, e));
                        if (key < low || key > high) continue;
                    }
                    atomicAdd(&sh.bins[bin(x, key)],
                              MASS ? __float2uint_rn(fminf(fast_mass(x) * unit, 2147483648.0f)) : 1u);
                }
            }
            if (binned) {
                __syncthreads();
                find_bin(MASS ? (uint32_t)fminf(fmaxf((target - mass_above) * unit, 1.0f), 4.0e9f)
                              : count - base);
            }
            const int b = binned ? sh.bin : kBins;
            Pair over{0.0f, 0.0f}, in{0.0f, 0.0f};
            uint64_t mine_low = ~0ull, mine_high = 0;
            for (int j = threadIdx.x; j < r.n; j += TH) {
                const Pack<T, 16> v = at(j);
                const uint32_t kept = f.kept(v, id_of(j, 0));
                if (!kept) continue;
                uint32_t higher = 0;       // of those, the ones above the bin
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (!(kept >> e & 1)) continue;
                    const float x = to_f32(v.e[e]);
                    uint64_t key = 0;
                    int at_bin = kBins;
                    if (!binned) {
                    } else if (shift < 0) {
                        at_bin = bin_of(x);
                    } else {
                        key = short_key(x, id_of(j, e));
                        at_bin = key > high ? -1 : key < low ? kBins : bin(x, key);
                    }
                    higher |= at_bin < b ? 1u << e : 0u;
                    if (at_bin != b) continue;
                    key = short_key(x, id_of(j, e));
                    if (MASS) in = add_loosely(in, fast_mass(x));
                    const int i = atomicAdd(&sh.count, 1);
                    if (i < kList) sh.list[i] = key;
                    mine_low = key < mine_low ? key : mine_low;
                    mine_high = key > mine_high ? key : mine_high;
                }
                if (MASS && higher) over = add_loosely(over, masses<false>(v, higher).h);
            }
            if (binned && mine_high) {
                atomicMin(&sh.low, (unsigned long long)mine_low);
                atomicMax(&sh.high, (unsigned long long)mine_high);
            }
            if (MASS) sum2(over, in);
            else __syncthreads();
            const int n = sh.count;
            above = over;
            if (!MASS && binned) base += sh.before;
            if (n <= kList) {
                for (int i = threadIdx.x; i < n; i += TH) {
                    const uint64_t key = sh.list[i];
                    int rank = 0;
#pragma unroll 2
                    for (int o = 0; o < n; ++o) rank += sh.list[o] > key;
                    sh.order[rank] = key;              // where the bins were
                }
                __syncthreads();
                before = base;
                return n;
            }
            if (binned) {
                low = sh.low;
                high = sh.high;
                mass_above = over.h;
                mass_in = in.h;
                shift = 0;
                while ((high - low) >> shift >= kBins) ++shift;
            }
            __syncthreads();
        }
        before = base;
        return 0;                          // not reached: a turn leaves 1/1024 of a range of 52 bits
    }

    // The least key of the first k; `bound`: a value that k elements reach, or -inf.
    __device__ __forceinline__ uint64_t floor_of_count(int k, float bound) {
        Pair above;
        uint32_t before;
        const bool bounded = bound > -INFINITY;
        const int n = list_at<false>(bounded || r.V <= kList,
                                     bounded ? (uint64_t)ordered(bound) << kIdBits : kFinite,
                                     (uint32_t)k, 0.0f, 0.0f, above, before);
        const int at = min(k - 1 - (int)before, n - 1);    // fewer than k finite ones: the last
        const uint64_t key = at >= 0 ? sh.order[at] : kFinite;
        __syncthreads();
        return key;
    }

    // How many of the list's n elements are kept: those before which, with what is above the list,
    // less than the target lies.  -1: less than the target lies before its end, -2: more before its begin.
    template <bool EXACT>
    __device__ __noinline__ int kept_of_list(int n, Pair above, Pair target, float error) {
        Draw d(*this);
        const int kept = d.template kept_of<EXACT>(n, above, target, error);
        unsure = d.unsure;
        return kept;
    }
    template <bool EXACT>
    __device__ __forceinline__ int kept_of(int n, Pair above, Pair target, float error) {
        const int lane = threadIdx.x & 31;
        for (int i = threadIdx.x; i < n; i += TH) {        // in the place of the unordered list
            const float x = unordered((uint32_t)(sh.order[i] >> kIdBits));
            sh.masses[i] = EXACT ? mass(x) : Pair{fast_mass(x), 0.0f};
        }
        __syncthreads();
        if (threadIdx.x < 32) {
            const int each = (n + 31) / 32, i0 = min(n, lane * each), i1 = min(n, i0 + each);
            Pair s{0.0f, 0.0f};
            for (int i = i0; i < i1; ++i) s = add(s, sh.masses[i]);
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const Pair y = shuffled_up(s, o);
                if (lane >= o) s = add(s, y);
            }
            Pair run = shuffled_up(s, 1);
            run = lane ? add(above, run) : above;
            int kept = 0;
            bool close = false;
            for (int i = i0; i < i1; ++i) {
                kept += less(run, target);
                close |= fabsf(difference(run, target)) <= error;
                run = add(run, sh.masses[i]);
            }
            // behind the list's end
            const Pair end = add(above, Pair{__shfl_sync(kAll, s.h, 31), __shfl_sync(kAll, s.l, 31)});
            kept = __reduce_add_sync(kAll, kept);
            if (less(end, target)) kept = -1;
            else if (!less(above, target)) kept = -2;
            close |= fabsf(difference(end, target)) <= error;
            close = __any_sync(kAll, close);
            if (lane == 0) {
                sh.kept = kept;
                sh.unsure = close;
            }
        }
        __syncthreads();
        const int kept = sh.kept;
        unsure = sh.unsure;
        __syncthreads();
        return kept;
    }
    // The least key of the first ones, from `least` on, whose masses reach top_p of theirs (`whole`), or
    // `from` if that is higher; `few`: no more than a list holds are there.
    __device__ __forceinline__ uint64_t floor_of_mass(bool few, uint64_t least, uint64_t from,
                                                      Pair whole) {
        Pair above;
        uint32_t before;
        Pair target = mul(whole, top_p);
        const int n = list_at<true>(few, from, 0, target.h, whole.h, above, before);
        int kept = kept_of_list<false>(n, above, target, error_of_list<T>(top_p.h, whole.h, r.V));
        const bool again = unsure && n;
        Pair exact, upper;
        if (again) {
            // the sums again, to 40 bits, over the same list
            exact_sums(least, sh.order[0] + 1, exact, upper);
            target = mul(exact, top_p);
            kept = kept_of_list<true>(n, upper, target, 0.0f);
        }
        uint64_t key = kept > 0 && n ? sh.order[kept - 1] : 0;
        if (!key && kept == -1 && few) key = from;         // all from `from` on
        __syncthreads();
        if (key) return key;
        // a border outside the list, which the histogram's rounded masses did not place: the bisection
        // compares sums of pairs, so its target has to be one
        if (!again) {
            exact_sums(least, least, exact, upper);
            target = mul(exact, top_p);
        }
        return bisect(from, target);
    }

    // The first id of a key from `least` on at which the running sum exceeds u of the whole.
    // A warp takes a piece of the row; the one in whose piece the border lies goes through it.
    template <bool EXACT>
    __device__ __noinline__ int token_from(uint64_t least, float u) {
        Draw d(*this);
        const int token = d.template token_of<EXACT>(least, u);
        unsure = d.unsure;
        return token;
    }
    template <bool EXACT>
    __device__ __forceinline__ int token_of(uint64_t least, float u) {
        const Floor<T> f(least);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int each = (r.n + WARPS - 1) / WARPS, j0 = min(r.n, warp * each);
        const int j1 = min(r.n, j0 + each);
        Pair s{0.0f, 0.0f};
        for (int j = j0 + lane; j < j1; j += 32)
            s = EXACT ? add(s, mass_of_vector<true>(j, f))
                      : add_loosely(s, mass_of_vector<false>(j, f).h);
#pragma unroll
        for (int o = 16; o; o >>= 1) s = add(s, shuffled(s, o));
        if (lane == 0) sh.pairs[0][warp] = s;
        __syncthreads();
        // every warp adds up the pieces before each, by its lanes
        const Pair piece = lane < WARPS ? sh.pairs[0][lane] : Pair{0.0f, 0.0f};
        Pair upto_piece = piece;
#pragma unroll
        for (int o = 1; o < WARPS; o *= 2) {
            const Pair y = shuffled_up(upto_piece, o);
            if (lane >= o) upto_piece = add(upto_piece, y);
        }
        const Pair whole{__shfl_sync(kAll, upto_piece.h, WARPS - 1),
                         __shfl_sync(kAll, upto_piece.l, WARPS - 1)};
        const Pair border = mul(whole, Pair{u, 0.0f});
        const float error = EXACT ? 0.0f : error_at(u, whole.h, r.V, kTerm + kAdd<T>);
        // the first piece at whose end the border is passed, else the last with a mass
        const unsigned filled = __ballot_sync(kAll, piece.h > 0.0f);
        const unsigned passed = __ballot_sync(kAll, piece.h > 0.0f && less(border, upto_piece));
        const int found = passed ? __ffs(passed) - 1 : filled ? 31 - __clz(filled) : 0;
        const int ahead_of = max(found - 1, 0);
        Pair run{__shfl_sync(kAll, upto_piece.h, ahead_of), __shfl_sync(kAll, upto_piece.l, ahead_of)};
        if (found == 0) run = Pair{0.0f, 0.0f};
        // the piece again, in steps of 32 vectors that all warps share; every warp then looks for the
        // step with the border
        const int k0 = min(r.n, found * each), k1 = min(r.n, k0 + each);
        const int steps = (k1 - k0 + 31) / 32;             // up to kList + 1
        for (int i = warp; i < steps; i += WARPS) {
            const int j = k0 + i * 32 + lane;
            Pair m = j < k1 ? mass_of_vector<EXACT>(j, f) : Pair{0.0f, 0.0f};
#pragma unroll
            for (int o = 16; o; o >>= 1) m = add(m, shuffled(m, o));
            if (lane == 0) sh.masses[i] = m;
        }
        __syncthreads();
        const auto reached = [&](Pair mine, Pair upto, unsigned& past) {   // by which lane
            past = __ballot_sync(kAll, mine.h > 0.0f && less(border, upto));
            const unsigned some = __ballot_sync(kAll, mine.h > 0.0f);
            return past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
        };
        const auto scanned = [&](Pair m) {
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const Pair y = shuffled_up(m, o);
                if (lane >= o) m = add(m, y);
            }
            return m;
        };
        const auto from_lane = [&](Pair m, int l) {
            return Pair{__shfl_sync(kAll, m.h, l), __shfl_sync(kAll, m.l, l)};
        };
        const auto ahead = [&](Pair upto) {                // of what the lane before has reached
            const Pair y = shuffled_up(upto, 1);
            return lane ? add(run, y) : run;
        };
        int step = 0;
        {
            const int some = (steps + 31) / 32, i0 = min(steps, lane * some), i1 = min(steps, i0 + some);
            Pair m{0.0f, 0.0f};
            for (int i = i0; i < i1; ++i) m = add(m, sh.masses[i]);
            const Pair upto = scanned(m);
            unsigned past;
            const int l = reached(m, add(run, upto), past);
            Pair at_step = ahead(upto), next = at_step;
            for (int i = i0; i < i1; ++i) {
                const Pair t = sh.masses[i];
                if (!(t.h > 0.0f)) continue;
                step = i;
                at_step = next;
                next = add(next, t);
                if (past && less(border, next)) break;
            }
            step = __shfl_sync(kAll, step, l);
            run = from_lane(at_step, l);
        }
        if (warp == step % WARPS) {
            const int j = k0 + step * 32 + lane;
            const Pair m = j < k1 ? mass_of_vector<EXACT>(j, f) : Pair{0.0f, 0.0f};
            const Pair upto = scanned(m);
            unsigned past;
            const int l = reached(m, add(run, upto), past);
            Pair before = ahead(upto), after = before;     // of the token
            if (lane == l) {
                int token = -1;
                const Pack<T, 16> v = at(min(j, r.n - 1));
                const uint32_t kept = j < k1 ? f.kept(v, id_of(j, 0)) : 0u;
                bool open = true;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (!open || !(kept >> e & 1)) continue;
                    const float x = to_f32(v.e[e]);
                    token = id_of(j, e);
                    before = after;
                    after = add(after, EXACT ? mass(x) : Pair{fast_mass(x), 0.0f});
                    if (past && less(border, after)) open = false;
                }
                // certain where nothing is kept before the token, and on its other side as u < 1
                // (the elements of this vector are added one by one here, as a tree in the whole)
                const float near = error + (EXACT ? 0.0f : kAdd<T> * m.h);
                const bool low = before.h > 0.0f && difference(border, before) <= near;
                const bool high = difference(after, border) <= near;
                sh.token = token;
                sh.unsure = low || high;
            }
        }
        __syncthreads();
        unsure = sh.unsure;
        const int token = sh.token;
        __syncthreads();
        return token;
    }
};

// score + x - (top + lse), rounded once but for lse; without the log-sum-exp score + x.
__device__ __forceinline__ float score_of(float score, float x, float top, float lse, bool fused) {
    if (!fused) return score + x;
    const float plain = score + ((x - top) - lse);
    if (!(fabsf(x) + fabsf(score) < 1e37f)) return plain;  // beyond what pairs hold
    return add(add(two_sum(x, -top), Pair{-lse, 0.0f}), Pair{score, 0.0f}).h;
}

template <typename T, int TH, bool HERE>
__global__ void __launch_bounds__(TH) k_sample(const SampleParams p) {
    constexpr int E = 16 / (int)sizeof(T), WARPS = TH / 32;
    extern __shared__ uint4 stage[];
    __shared__ Shared<TH> sh;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int b = row / p.K, k = row - b * p.K;
    const float score = p.scores[row], u = p.random[row];
    const bool finished = p.finished && p.finished[row];
    float out = finished ? score : -INFINITY;
    int token = -1;
    bool bad = !(score < INFINITY) || (!finished && !(u >= 0.0f && u < 1.0f));
    if (bad) out = -INFINITY;
    if (!bad && !finished && score > -INFINITY) {
        const T* x = reinterpret_cast<const T*>(p.logits + b * p.batch_stride + k * p.beam_stride);
        Draw<T, TH, HERE> d(p, sh, x, stage);
        Pack<T, 16> most = all_minus_inf<T>();
        if constexpr (HERE) {
            // one bulk copy; the units it shares with what is not the row's element by element
            const Staged<T, TH> row_here(x, p.V, stage, x, x + p.V);
            if (tid == 0) {
                mbar_init(&sh.bar);
                fence_mbar_init();
                row_here.fetch(&sh.bar);
            }
            __syncthreads();                               // the barrier is there
            int polls = kWaitPolls;
            mbar_wait(&sh.bar, 0, polls, p.status);
            row_here.complete();
#pragma unroll 4
            for (int j = tid; j < d.r.n; j += TH) most = larger(most, row_here.at(j));
        } else {
#pragma unroll 4
            for (int j = tid; j < d.r.n; j += TH) most = larger(most, d.r.load(j));
        }
        const float2 both = half_maxima(most);
        const float mine = max_nan(both.x, both.y);        // the thread's largest
        float m = warp_max_nan(mine);
        if (lane == 0) sh.floats[tid >> 5] = m;
        __syncthreads();
        m = warp_max_nan(lane < WARPS ? sh.floats[lane] : -INFINITY);
        bad = !(m < INFINITY);
        if (!bad && m > -INFINITY) {
            d.top = m;
            // the whole row's sums at the temperature and at 1, where they are wanted
            const bool at_tau = p.top_p.h < 1.0f || (p.fused && p.unit_tau);
            const bool at_one = p.fused && !p.unit_tau;
            Pair s{0.0f, 0.0f}, s1{0.0f, 0.0f};
            if (at_tau || at_one) {
                const Exponent f(m, p.scale, p.scale_low), f1(m, p.one, p.one_low);
                for (int j = tid; j < d.r.n; j += TH) {
                    const Pack<T, 16> v = d.at(j);
                    float2 e[E / 2];
                    if (at_one) s1 = add_loosely(s1, terms_of(v, f1, e));
                    if (at_tau) s = add_loosely(s, terms_of(v, f, e));
                }
                d.sum2(s, s1);
            }
            const float lse = p.fused ? logf(p.unit_tau ? s.h : s1.h) : 0.0f;
            uint64_t least = kFinite;
            const bool some_k = p.top_k && p.top_k < p.V;
            if (some_k) {
                // of every warp's threads' largest elements its share of top_k, the least of them: a
                // bound that so many elements reach
                const int c = (p.top_k + WARPS - 1) / WARPS;
                float bound = -INFINITY;
                if (c <= 32) {
                    const float cth = __shfl_sync(kAll, warp_sorted(mine), c - 1);
                    __syncthreads();
                    if (lane == 0) sh.floats[tid >> 5] = -cth;
                    __syncthreads();
                    bound = -warp_max(lane < WARPS ? sh.floats[lane] : -INFINITY);
                }
                least = d.floor_of_count(p.top_k, bound);
            }
            uint64_t by_gap = 0;
            if (p.min_gap > -INFINITY) {
                // the least float32 that is not below top + tau log min_p
                const float f = __double2float_ru((double)m + p.min_gap);
                if (f > -INFINITY) by_gap = (uint64_t)ordered(f) << kIdBits;
            }
            uint64_t floor = least;
            if (p.top_p.h < 1.0f) {
                const uint64_t from = by_gap > least ? by_gap : least;
                bool few = p.V <= kList || (some_k && p.top_k <= kList);
                if (some_k) {                              // of what top_k has left
                    const Floor<T> f(least);
                    s = s1 = Pair{0.0f, 0.0f};
                    for (int j = tid; j < d.r.n; j += TH)
                        s = add_loosely(s, d.template mass_of_vector<false>(j, f).h);
                    d.sum2(s, s1);
                }
                bool within = true;                        // the border lies above `from`
                if (from > least) {
                    const Floor<T> f(from);
                    Pair upper{0.0f, 0.0f};
                    s1 = Pair{0.0f, 0.0f};
                    int n = 0;
                    for (int j = tid; j < d.r.n; j += TH) {
                        const Pack<T, 16> v = d.at(j);
                        const uint32_t kept = f.kept(v, d.id_of(j, 0));
                        if (!kept) continue;
                        upper = add_loosely(upper, d.template masses<false>(v, kept).h);
                        n += __popc(kept);
                    }
                    s1.h = (float)n;
                    d.sum2(upper, s1);
                    few |= s1.h <= (float)kList;
                    // where that is open, by what the exact sums say of the whole list, or of all
                    within = !(difference(mul(s, p.top_p), upper) >
                               error_of_list<T>(p.top_p.h, s.h, p.V));
                }
                floor = within ? d.floor_of_mass(few, least, from, s) : from;
            }
            floor = by_gap > floor ? by_gap : floor;
            token = d.template token_from<false>(floor, u);
            if (d.unsure) token = d.template token_from<true>(floor, u);
            if (token >= 0) out = score_of(score, to_f32(x[token]), m, lse, p.fused);
        }
    }
    if (tid == 0) {
        p.out_scores[row] = out;
        p.out_tokens[row] = token;
        if (bad && p.status) *p.status = RNNT_INVALID_VALUE;
    }
}

constexpr size_t kHere = 200 << 10;        // bytes of a row that a block holds in shared memory

void fill_params(SampleParams& p, int32_t V, double temperature, int32_t top_k, double top_p,
                 double min_p, bool fused) {
    p.V = V;
    p.top_k = top_k;
    p.fused = fused;
    p.unit_tau = temperature == 1.0;
    parts_below(kLog2e / temperature, p.scale, p.scale_low);
    parts_below(kLog2e, p.one, p.one_low);
    p.bin_scale = (float)(kLog2e / temperature) * kBinsPerOrder;
    p.exact_scale = pair_of(kLog2e / temperature);
    p.top_p = top_p < 1.0 ? pair_of(top_p) : Pair{2.0f, 0.0f};
    p.min_gap = min_p > 0.0 ? temperature * std::log(min_p) : -INFINITY;
}

template <typename T>
void launch_sample(const SampleParams& p, cudaStream_t st) {
    const unsigned rows = (unsigned)(p.B * p.K);
    const size_t bytes = ((size_t)p.V * sizeof(T) + 30) / 16 * 16;         // at any alignment
    // Fewer threads have shorter chains of barriers, more read a row sooner.  float16, us of unfiltered draws /
    // top_k 40 / top_p 0.9, of 4 and of 1024 rows, by 128, 256 and 512 threads:
    //   4000 bytes   7/10/15 and 16/19/27   7/10/14 and 17/27/35   8/12/14 and 32/47/61
    //   8000         8/13/19 and 21/23/42   7/12/16 and 23/31/49   8/13/15 and 33/55/73
    //  32000         12/18/47 and 48/45/146  10/16/54 and 45/43/131  10/16/25 and 53/69/138
    if (bytes <= 4 << 10) k_sample<T, 128, true><<<rows, 128, bytes, st>>>(p);
    else if (bytes <= 32 << 10) k_sample<T, 256, true><<<rows, 256, bytes, st>>>(p);
    else if (bytes <= kHere) k_sample<T, 512, true><<<rows, 512, bytes, st>>>(p);
    else k_sample<T, 512, false><<<rows, 512, 0, st>>>(p);
}
template <typename T>
bool raise_sample() {
    return cudaFuncSetAttribute(k_sample<T, 512, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)kHere) == cudaSuccess;
}
bool sample_prepared() {
    static std::atomic<bool> done[64];
    return prepared_once(done, [] {
        return raise_sample<float>() && raise_sample<__half>() && raise_sample<__nv_bfloat16>();
    });
}

}  // namespace

extern "C" rnnt_status_t rnnt_sample(const void* logits, rnnt_dtype_t dt, int32_t B, int32_t K,
                                     int32_t V, int64_t batch_stride, int64_t beam_stride,
                                     const float* scores, const float* random,
                                     const uint8_t* finished, double temperature, int32_t top_k,
                                     double top_p, double min_p, int32_t fused_log_softmax,
                                     float* out_scores, int32_t* out_tokens, int32_t* status_dev,
                                     rnnt_stream_t stream) {
    if (!logits || !scores || !random || !out_scores || !out_tokens || !valid_dtype(dt) || B < 1 ||
        K < 1 || V < 1 || V > RNNT_MAX_TOP_VOCAB || (int64_t)B * K > INT32_MAX ||
        batch_stride < 0 || beam_stride < 0 || !(temperature >= 1e-4 && temperature <= 1e4) ||
        top_k < 0 || !(top_p > 0.0 && top_p <= 1.0) || !(min_p >= 0.0 && min_p <= 1.0))
        return RNNT_INVALID_VALUE;
    const int es = elem_size(dt);
    if (batch_stride > (INT64_MAX >> 4) / B || beam_stride > (INT64_MAX >> 4) / K ||
        (uintptr_t)logits % es ||
        ((uintptr_t)scores | (uintptr_t)random | (uintptr_t)out_scores | (uintptr_t)out_tokens |
         (uintptr_t)status_dev) & 3)
        return RNNT_INVALID_VALUE;
    const uint64_t n = (uint64_t)B * K;
    const void* ins[4] = {logits, scores, random, finished};
    const uint64_t in_sizes[4] = {
        (uint64_t)((B - 1) * batch_stride + (K - 1) * beam_stride + V) * es, n * 4, n * 4, n};
    const void* outs[2] = {out_scores, out_tokens};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 4; ++j)
            if (ins[j] && overlaps(outs[i], n * 4, ins[j], in_sizes[j])) return RNNT_INVALID_VALUE;
    if (overlaps(outs[0], n * 4, outs[1], n * 4)) return RNNT_INVALID_VALUE;
    SampleParams p{};
    p.logits = static_cast<const char*>(logits);
    p.batch_stride = batch_stride * es;
    p.beam_stride = beam_stride * es;
    p.scores = scores;
    p.random = random;
    p.finished = finished;
    p.B = B;
    p.K = K;
    fill_params(p, V, temperature, top_k, top_p, min_p, fused_log_softmax != 0);
    p.out_scores = out_scores;
    p.out_tokens = out_tokens;
    p.status = status_dev;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!sample_prepared() || !clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    with_type(dt, [&](auto t) { launch_sample<decltype(t)>(p, st); });
    return launched();
}
