// rnnt_sample.cu -- drawing labels: of every hypothesis one extension, from a random number that is
// given.
//
// With logits x, e_j = exp(x_j / tau) and a number u in [0, 1): outputs are ordered by logit (equal
// ones by id); of the first top_k the shortest beginning with a sum of e of at least top_p of
// theirs is kept, and of it what has e_j >= min_p max e.  All three keep a beginning of the order,
// so what is kept is what reaches one key (value and id).  The token is the first kept id at
// which the running sum of e, by id, exceeds u times the kept sum.
//
// Whether a sum reaches a border decides a whole number, so sums are taken as if held to 40 bits: in
// pairs of floats, of exponentials that are pairs of floats themselves.
#include <cmath>

#include "rnnt_rows.cuh"

using namespace rnnt_rows;

namespace {

// ------------------------------------------------------------ pairs of floats
// Their exact sum is the value: about 47 bits on float32 units, of which there are 64 times as many
// as of float64 ones.  The compiler neither reorders nor contracts what is spelt with intrinsics.
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

// exp(d) for d <= 0, relative error below 2^-40 down to e^-60: with d = n ln 2 + g (Cody and
// Waite's reduction: ln 2 in three parts, the first with few bits so that n times it is exact),
// e^(g/16) - 1 by its Taylor series and four times (1 + q)^2 - 1.
__device__ __forceinline__ Pair exp_pair(Pair d) {
    if (!(d.h > -86.0f)) return {0.0f, 0.0f};
    const float n = rintf(d.h * (float)kLog2e);
    constexpr double ln2 = 0.69314718055994530942;
    constexpr float ln2a = 11356.0f / 16384.0f;            // 14 bits: n * ln2a is exact
    constexpr float ln2b = (float)(ln2 - (double)ln2a);
    constexpr float ln2c = (float)(ln2 - (double)ln2a - (double)ln2b);
    const Pair a = two_sum(__fmaf_rn(-n, ln2a, d.h), d.l);
    const float p = __fmul_rn(n, ln2b);
    const float pl = __fadd_rn(__fmaf_rn(n, ln2b, -p), __fmul_rn(n, ln2c));
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
    const float s = __int_as_float(((int)n + 127) << 23);  // n >= -125
    return {e.h * s, e.l * s};
}

// --------------------------------------------------------------------- rows
struct SampleParams {
    const char* logits;
    int64_t batch_stride, beam_stride;     // bytes
    const float* scores;
    const float* random;
    const uint8_t* finished;
    int32_t B, K, V, top_k, fused;
    Pair inv_tau, top_p;                   // top_p.h >= 1: not used
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

template <int TH>
struct Shared {
    static constexpr int WARPS = TH / 32;
    Pair pairs[WARPS], prefix[WARPS + 1];
    float floats[WARPS];
    int ints[WARPS];
    int token, found;
};

template <typename T, int TH>
struct Draw {
    static constexpr int E = 16 / (int)sizeof(T), WARPS = TH / 32;
    const SampleParams& p;
    Shared<TH>& sh;
    const Row<T> r;
    float top;

    __device__ __forceinline__ Draw(const SampleParams& a, Shared<TH>& s, const T* x)
        : p(a), sh(s), r(x, a.V), top(0.0f) {}

    __device__ __forceinline__ Pair mass(float x) const {
        const Pair d = two_sum(x, -top);
        const Pair e = exp_pair(mul(d, p.inv_tau));
        return e.h >= kLeastMass ? e : Pair{kLeastMass, 0.0f};
    }
    __device__ __forceinline__ Pair sum(Pair s) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int o = 16; o; o >>= 1) s = add(s, shuffled(s, o));
        if (lane == 0) sh.pairs[threadIdx.x >> 5] = s;
        __syncthreads();
        s = lane < WARPS ? sh.pairs[lane] : Pair{0.0f, 0.0f};
#pragma unroll
        for (int o = 16; o; o >>= 1) s = add(s, shuffled(s, o));
        __syncthreads();
        return s;
    }
    // Of the elements whose keys are at least `least`.
    __device__ __noinline__ Pair mass_from(uint64_t least) {
        Pair s{0.0f, 0.0f};
        for (int j = threadIdx.x; j < r.n; j += TH) {
            const Pack<T, 16> v = r.load(j);
#pragma unroll 1
            for (int e = 0; e < E; ++e) {
                const float x = to_f32(v.e[e]);
                if (short_key(x, j * E + e - r.off) >= least && x > -INFINITY) s = add(s, mass(x));
            }
        }
        return sum(s);
    }
    __device__ __noinline__ int count_from(uint64_t least) {
        int n = 0;
        for (int j = threadIdx.x; j < r.n; j += TH) {
            const Pack<T, 16> v = r.load(j);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = to_f32(v.e[e]);
                n += short_key(x, j * E + e - r.off) >= least && x > -INFINITY;
            }
        }
        n = __reduce_add_sync(kAll, n);
        if ((threadIdx.x & 31) == 0) sh.ints[threadIdx.x >> 5] = n;
        __syncthreads();
        n = __reduce_add_sync(kAll, (threadIdx.x & 31) < WARPS ? sh.ints[threadIdx.x & 31] : 0);
        __syncthreads();
        return n;
    }
    // The least key of the first k: fewer than k lie above it.
    __device__ __noinline__ uint64_t floor_of_count(int k) {
        uint64_t lo = kFinite, hi = short_key(top, 0);
        while (lo < hi) {
            const uint64_t mid = lo + (hi - lo) / 2;
            if (count_from(mid + 1) < k) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    }
    // The least key, from `least` on, above which lies less than the target.
    __device__ __noinline__ uint64_t floor_of_mass(uint64_t least, Pair target) {
        uint64_t lo = least, hi = short_key(top, 0);
        while (lo < hi) {
            const uint64_t mid = lo + (hi - lo) / 2;
            if (less(mass_from(mid + 1), target)) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    }
    // The first id of a key from `least` on at which the running sum exceeds u of the whole.
    // A warp takes a piece of the row; the one in whose piece the border lies goes through it.
    __device__ __noinline__ int token_from(uint64_t least, float u) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int each = (r.n + WARPS - 1) / WARPS, j0 = warp * each, j1 = min(r.n, j0 + each);
        Pair s{0.0f, 0.0f};
        for (int j = j0 + lane; j < j1; j += 32) s = add(s, mass_of_vector(j, least));
#pragma unroll
        for (int o = 16; o; o >>= 1) s = add(s, shuffled(s, o));
        if (lane == 0) sh.pairs[warp] = s;
        if (threadIdx.x == 0) sh.found = WARPS;
        __syncthreads();
        if (threadIdx.x == 0) {
            Pair run{0.0f, 0.0f};
            int last = 0;
            for (int w = 0; w < WARPS; ++w) {
                sh.prefix[w] = run;
                run = add(run, sh.pairs[w]);
                if (sh.pairs[w].h > 0.0f) last = w;
            }
            const Pair border = mul(run, Pair{u, 0.0f});
            sh.prefix[WARPS] = border;
            int w = 0;                     // the first piece at whose end the border is passed
            while (w < last && !less(border, add(sh.prefix[w], sh.pairs[w]))) ++w;
            sh.found = w;
        }
        __syncthreads();
        if (warp == sh.found) {
            const Pair border = sh.prefix[WARPS];
            Pair run = sh.prefix[warp];
            int token = -1;
            for (int j = j0; j < j1; j += 32) {
                Pair s = j + lane < j1 ? mass_of_vector(j + lane, least) : Pair{0.0f, 0.0f};
                const Pair mine = s;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const Pair y = shuffled_up(s, o);
                    if (lane >= o) s = add(s, y);
                }
                const Pair end = add(run, s);
                const unsigned some = __ballot_sync(kAll, mine.h > 0.0f);
                const unsigned past = __ballot_sync(kAll, mine.h > 0.0f && less(border, end));
                // the vector that passes the border, or (where the sums' last bits differ) the last
                // that holds a kept element so far
                const int at = past ? __ffs(past) - 1 : 31 - __clz(some);
                if (some) {
                    Pair before = shuffled_up(s, 1);
                    before = lane ? add(run, before) : run;
                    int got = -1;
                    if (lane == at) {
                        const Pack<T, 16> v = r.load(j + lane);
#pragma unroll 1
                        for (int e = 0; e < E; ++e) {
                            const float x = to_f32(v.e[e]);
                            const int id = (j + lane) * E + e - r.off;
                            if (x > -INFINITY && short_key(x, id) >= least) {
                                got = id;
                                before = add(before, mass(x));
                                if (past && less(border, before)) break;
                            }
                        }
                    }
                    token = __shfl_sync(kAll, got, at);
                }
                if (past) break;
                run = Pair{__shfl_sync(kAll, end.h, 31), __shfl_sync(kAll, end.l, 31)};
            }
            if (lane == 0) sh.token = token;
        }
        __syncthreads();
        return sh.token;
    }
    __device__ __noinline__ Pair mass_of_vector(int j, uint64_t least) {
        const Pack<T, 16> v = r.load(j);
        Pair s{0.0f, 0.0f};
#pragma unroll 1
        for (int e = 0; e < E; ++e) {
            const float x = to_f32(v.e[e]);
            if (x > -INFINITY && short_key(x, j * E + e - r.off) >= least) s = add(s, mass(x));
        }
        return s;
    }
};

// score + x - (top + lse), rounded once but for lse; without the log-sum-exp score + x.
__device__ __forceinline__ float score_of(float score, float x, float top, float lse, bool fused) {
    if (!fused) return score + x;
    const float plain = score + ((x - top) - lse);
    if (!(fabsf(x) + fabsf(score) < 1e37f)) return plain;  // beyond what pairs hold
    return add(add(two_sum(x, -top), Pair{-lse, 0.0f}), Pair{score, 0.0f}).h;
}

template <typename T, int TH>
__global__ void __launch_bounds__(TH) k_sample(const SampleParams p) {
    constexpr int E = 16 / (int)sizeof(T), WARPS = TH / 32;
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
        Draw<T, TH> d(p, sh, x);
        float m = -INFINITY;
        for (int j = tid; j < d.r.n; j += TH) {
            const Pack<T, 16> v = d.r.load(j);
#pragma unroll
            for (int e = 0; e < E; ++e) m = max_nan(m, to_f32(v.e[e]));
        }
        m = warp_max_nan(m);
        if (lane == 0) sh.floats[tid >> 5] = m;
        __syncthreads();
        m = warp_max_nan(lane < WARPS ? sh.floats[lane] : -INFINITY);
        __syncthreads();
        bad = !(m < INFINITY);
        if (!bad && m > -INFINITY) {
            d.top = m;
            float lse = 0.0f;
            if (p.fused) {
                Pair s{0.0f, 0.0f};
                for (int j = tid; j < d.r.n; j += TH) {
                    const Pack<T, 16> v = d.r.load(j);
                    float part = 0.0f;
#pragma unroll
                    for (int e = 0; e < E; ++e) part += ex2((to_f32(v.e[e]) - m) * (float)kLog2e);
                    s = add(s, Pair{part, 0.0f});
                }
                lse = logf(d.sum(s).h);
            }
            uint64_t least = kFinite;
            if (p.top_k && p.top_k < p.V) least = d.floor_of_count(p.top_k);
            uint64_t floor = least;
            if (p.top_p.h < 1.0f) floor = d.floor_of_mass(least, mul(d.mass_from(least), p.top_p));
            if (p.min_gap > -INFINITY) {
                // the least float32 that is not below top + tau log min_p
                const double border = (double)m + p.min_gap;
                const float f = __double2float_ru(border);
                if (f > -INFINITY) {
                    const uint64_t by_gap = (uint64_t)ordered(f) << kIdBits;
                    floor = by_gap > floor ? by_gap : floor;
                }
            }
            token = d.token_from(floor, u);
            out = score_of(score, to_f32(x[token]), m, lse, p.fused);
        }
    }
    if (tid == 0) {
        p.out_scores[row] = out;
        p.out_tokens[row] = token;
        if (bad && p.status) *p.status = RNNT_INVALID_VALUE;
    }
}

template <typename T>
void launch_sample(const SampleParams& p, cudaStream_t st) {
    const unsigned rows = (unsigned)(p.B * p.K);
    if ((int64_t)p.V * (int64_t)sizeof(T) <= 16 << 10) k_sample<T, 128><<<rows, 128, 0, st>>>(p);
    else k_sample<T, 1024><<<rows, 1024, 0, st>>>(p);
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
    p.V = V;
    p.top_k = top_k;
    p.fused = fused_log_softmax != 0;
    p.inv_tau = pair_of(1.0 / temperature);
    p.top_p = top_p < 1.0 ? pair_of(top_p) : Pair{2.0f, 0.0f};
    p.min_gap = min_p > 0.0 ? temperature * std::log(min_p) : -INFINITY;
    p.out_scores = out_scores;
    p.out_tokens = out_tokens;
    p.status = status_dev;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    with_type(dt, [&](auto t) { launch_sample<decltype(t)>(p, st); });
    return launched();
}
