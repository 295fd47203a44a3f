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
constexpr int kSMs = 152;
constexpr int kMostRows = kSMs * 16;        // blocks of a kernel that takes a row a block

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
        if (rows <= INT32_MAX) {                           // 32-bit divisions
            const uint32_t w = (uint32_t)max_U + 1, q = (uint32_t)row / w, b = q / (uint32_t)max_T;
            return (int)(q - b * max_T) < T[b] && (int)((uint32_t)row - q * w) <= U[b];
        }
        const int64_t w = (int64_t)max_U + 1, q = row / w;
        const int u = (int)(row - q * w), b = (int)(q / max_T), t = (int)(q - (int64_t)b * max_T);
        return t < T[b] && u <= U[b];
    }
};

// Whether the rows first, first + step, ... count: rows below `rows` and, in the padded layout, inside
// their sequence.  A warp's lanes look 32 rows up at a time, up to 64 rows ahead.
struct Window {
    uint32_t now, later;
    int32_t i;
    __device__ static __forceinline__ uint32_t look(const Lattice& lat, int64_t first, int64_t step,
                                                    int64_t rows) {
        const int64_t row = first + (threadIdx.x & 31) * step;
        return __ballot_sync(kAll, row < rows && (!lat.T || !lat.padded || lat.inside(row)));
    }
    __device__ __forceinline__ Window(const Lattice& lat, int64_t first, int64_t step, int64_t rows)
        : now(look(lat, first, step, rows)), later(look(lat, first + 32 * step, step, rows)), i(0) {}
    // Of the row `ahead` (below 32) behind the present one.
    __device__ __forceinline__ bool operator[](int ahead) const {
        return __funnelshift_r(now, later, i) >> ahead & 1;
    }
    __device__ __forceinline__ void advance(const Lattice& lat, int64_t next, int64_t step,
                                            int64_t rows) {
        if (++i < 32) return;
        i = 0;
        now = later;
        later = look(lat, next + 32 * step, step, rows);
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
    float scale, scale_low;                // log2 e / tau, in two parts
    float inv_tau, inv_tau_low;            // 1 / tau, in two parts
    void* values;
    int32_t* ids;
    float* rest;
    int32_t* status;
};

// a + b + c for a c below a step of a + b, rounded once (Knuth's sum): added to a rounded a + b, a low
// part of a product would be lost, in all rows the same way.
__device__ __forceinline__ float sum_of(float a, float b, float c) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    if (!(fabsf(s) < INFINITY)) return s;
    return __fadd_rn(s, __fadd_rn(__fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)), c));
}

// The logarithm of a rest whose largest is `first` and whose sum relative to it is `sum`; finite, and
// rounded once: by a reciprocal rounded to one float32 all of a call's rests would be off the same way.
__device__ __forceinline__ float rest_of(const TopParams& p, float sum, float first) {
    const float hi = first * p.inv_tau;
    if (!(fabsf(hi) < kMost)) return copysignf(kMost, hi);
    const float low = __fmaf_rn(first, p.inv_tau_low, __fmaf_rn(first, p.inv_tau, -hi));
    return fminf(fmaxf(sum_of(logf(sum), hi, low), -kMost), kMost);
}

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
                    const Exponent f(first, p.scale, p.scale_low);
                    float sum = 0.0f, equal = 0.0f;
                    for (int j = tid; j < r.n; j += TH) {
                        const Pack<T, 16> v = r.load(j);
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const float y = to_f32(v.e[e]);
                            sum += y < first ? f(y) : 0.0f;
                            equal += y == first ? 1.0f : 0.0f;
                        }
                    }
                    sum = block_sum<TH>(sum, space);
                    equal = block_sum<TH>(equal, space);
                    for (int i = 0; i < k; ++i) equal -= value_of(best[i]) == first ? 1.0f : 0.0f;
                    rest = rest_of(p, sum + equal, first);
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

// The stages of a group's ring, and what a group needs beside them.
struct Ring {
    int32_t stages;
    uint32_t stage_bytes, group_bytes;
};
constexpr int kMostStages = 2;            // more cost blocks an SM: 3 and 4 measured slower

// Keys of a row's elements in the order of their values, the lower element first where they are equal:
// in 32 bits where a value has 16 and a row at most 65536.
template <typename T, int G>
struct Keys {
    static constexpr bool kShort = sizeof(T) == 2 && G == 32;
    using Key = std::conditional_t<kShort, uint32_t, uint64_t>;
    __device__ static __forceinline__ Key of(T x, int element) {
        if constexpr (kShort) {
            uint32_t b = reinterpret_cast<const uint16_t&>(x);
            b = b == 0x8000u ? 0u : b;                     // -0 counts as 0
            return (b ^ (b >> 15 ? 0xffffu : 0x8000u)) << 16 | (uint32_t)(0xffff - element);
        } else {
            return key_of(to_f32(x), element);
        }
    }
    __device__ static __forceinline__ float value(Key key) {
        if constexpr (kShort) {
            const uint32_t o = key >> 16;
            const uint16_t b = (uint16_t)(o ^ (o >> 15 ? 0x8000u : 0xffffu));
            return to_f32(reinterpret_cast<const T&>(b));
        } else {
            return value_of(key);
        }
    }
    __device__ static __forceinline__ int element(Key key) {
        if constexpr (kShort) return 0xffff - (int)(key & 0xffffu);
        else return element_of(key);
    }
};

template <typename T, int G>
struct TopScratch {
    static constexpr int BUF = G == 32 ? 128 : 512;        // elements that are ranked
    using Key = typename Keys<T, G>::Key;
    uint64_t bar[kMostStages];
    __align__(16) Key buf[BUF + 4];
    Key best[RNNT_MAX_TOP + 1];
    typename Group<G>::Space space;
    float bounds[G / 32];
    int count;
};

// The c-th largest of the warp's values: one by one, or sorted, which costs the same for c = 7 or so
// (100000 rows of 1024 float16: c = 5 84 us and 86, c = 9 93 and 90, c = 12 100 and 93, c = 21 133
// and 116).
__device__ __forceinline__ float warp_cth(float x, int c) {
    if (c > 7) return __shfl_sync(kAll, warp_sorted(x), c - 1);
    for (int n = 0;;) {
        const float m = warp_max(x);
        n += __popc(__ballot_sync(kAll, x == m));
        if (n >= c) return m;
        x = x == m ? -INFINITY : x;
    }
}

// Rows through a ring of shared memory, a group of threads each.  The k best of a row: the
// largest maxima of its threads (of both halves of their vectors where k needs more than there are
// threads in a warp) bound the k + 1-st best from below; the few elements that reach the bound are
// ranked by counting.  They are then taken out of the row, which leaves the rest: its largest
// element (the k + 1-st best, if it reached the bound) and the sum relative to it.
//
// Issue slots bound it: 480000 rows of 1024 float16 with k = 8 take 414 us (2.4 TB/s; 834 warp
// instructions a row, of which 200 touch elements, in 76 % of the slots), 226000 of 5000 float32 with
// k = 32 1766 us (3.0 TB/s).  Rows of up to 4 KB by warps, longer ones by blocks: a warp has
// no barriers, but its ring of longer rows would leave an SM with few warps.
template <typename T, int TH, int G, bool WHOLE>
__global__ void __launch_bounds__(TH, 5) k_top(const TopParams p, const Ring ring) {
    using Gr = Group<G>;
    using Scratch = TopScratch<T, G>;
    using K = Keys<T, G>;
    using Key = typename K::Key;
    constexpr int WARPS = G / 32, E = 16 / (int)sizeof(T), GROUPS = TH / G;
    extern __shared__ __align__(16) char space[];
    char* const mine = space + (G == 32 ? threadIdx.x / G : 0) * ring.group_bytes;
    Scratch& sh = *reinterpret_cast<Scratch*>(mine + ring.stages * ring.stage_bytes);
    const int me = Gr::rank(), lane = me & 31, k = p.k;
    const int64_t groups = (int64_t)gridDim.x * GROUPS;
    const int64_t first_row = (int64_t)blockIdx.x * GROUPS + (G == 32 ? threadIdx.x / G : 0);
    const T* const logits = reinterpret_cast<const T*>(p.logits);
    const T* const end = logits + p.lat.rows * p.V;
    const auto staged = [&](int64_t row, int st) {
        return Staged<T, G, WHOLE>(logits + row * p.V, p.V,
                                   reinterpret_cast<uint4*>(mine + st * ring.stage_bytes), logits,
                                   end);
    };
    if (blockIdx.x == 0 && p.lat.T) check_lengths<TH>(p.lat, p.status);
    if (me == 0) {
        for (int st = 0; st < ring.stages; ++st) mbar_init(&sh.bar[st]);
        fence_mbar_init();
        sh.count = 0;
    }
    Gr::sync();
    Window live(p.lat, first_row, groups, p.lat.rows);
    if (me == 0)
        for (int st = 0; st < ring.stages; ++st)
            if (live[st]) staged(first_row + st * groups, st).fetch(&sh.bar[st]);
    int polls = kWaitPolls, st = 0;
    uint32_t phases = 0;                                   // a bit a stage
    for (int64_t row = first_row; row < p.lat.rows; row += groups) {
        float rest = -INFINITY;
        int have = 0;
        if (live[0]) {
            const Staged<T, G, WHOLE> x = staged(row, st);
            mbar_wait(&sh.bar[st], phases >> st & 1, polls, p.status);
            phases ^= 1u << st;
            x.complete();
            Pack<T, 16> m = all_minus_inf<T>();
#pragma unroll 4
            for (int j = me; j < x.r.n; j += G) m = larger(m, x.at(j));
            float2 both = half_maxima(m);
            const float top = Gr::max(max_nan(both.x, both.y), sh.space);
            if (!(top < INFINITY)) {                       // NaN or +inf: the row is left empty
                if (me == 0) invalid(p.status);
            } else if (top > -INFINITY) {
                const int c = min((k + WARPS) / WARPS, 64 / WARPS);    // a warp's share of k + 1
                float bound;
                if (c <= 32) {
                    bound = warp_cth(fmaxf(both.x, both.y), c);
                } else {
                    const int h = (c + 1) / 2;
                    bound = fminf(warp_cth(both.x, h), warp_cth(both.y, h));
                }
                if constexpr (G > 32) {
                    if (lane == 0) sh.bounds[threadIdx.x >> 5] = bound;
                    Gr::sync();
#pragma unroll
                    for (int w = 0; w < WARPS; ++w) bound = fminf(bound, sh.bounds[w]);
                }
                // -inf reaches no bound
                bound = fmaxf(bound, lowest<T>());
                const T at_least = from_f32<T>(bound);     // a value of the type
                int n = 0;
                constexpr int B = 32 / E;                  // vectors whose elements have a bit each
                for (int j0 = 0; j0 < x.r.n; j0 += B * G) {
                    uint32_t hits = 0;
#pragma unroll
                    for (int i = 0; i < B; ++i)
                        if (j0 + me + i * G < x.r.n)
                            hits |= reaching(x.at(j0 + me + i * G), at_least) << (i * E);
                    if constexpr (G == 32) {
                        for (unsigned some; (some = __ballot_sync(kAll, hits != 0)) != 0;) {
                            const int at = n + __popc(some & ((1u << lane) - 1u));
                            if (hits) {
                                const int bit = __ffs(hits) - 1;
                                const int i = (j0 + me + bit / E * G) * E + bit % E - x.r.off;
                                if (at < Scratch::BUF) sh.buf[at] = K::of(x.element(i), i);
                            }
                            hits &= hits - 1;
                            n += __popc(some);
                        }
                    } else {
                        while (hits) {
                            const int bit = __ffs(hits) - 1;
                            const int i = (j0 + me + bit / E * G) * E + bit % E - x.r.off;
                            hits &= hits - 1;
                            const int at = atomicAdd(&sh.count, 1);
                            if (at < Scratch::BUF) sh.buf[at] = K::of(x.element(i), i);
                        }
                    }
                }
                if constexpr (G == 32) {
                    if (lane < 4 && n <= Scratch::BUF) sh.buf[n + lane] = 0;   // to fours
                }
                Gr::sync();
                if constexpr (G > 32) n = sh.count;
                have = min(n, k);
                if (n <= Scratch::BUF) {
                    for (int i = me; i < n; i += G) {
                        const Key key = sh.buf[i];
                        int rank = 0;
                        if constexpr (K::kShort) {
                            for (int o = 0; o < n; o += 4) {
                                const uint4 four = *reinterpret_cast<const uint4*>(&sh.buf[o]);
                                rank += (four.x > key) + (four.y > key) + (four.z > key) +
                                        (four.w > key);
                            }
                        } else {
                            for (int o = 0; o < n; ++o) rank += sh.buf[o] > key;
                        }
                        if (rank <= k) sh.best[rank] = key;
                    }
                } else {                                   // a crowd: one by one
                    Key last = (Key)~0ull;
                    for (int i = 0; i <= k; ++i) {
                        Key next = 0;
                        for (int j = me; j < x.r.n; j += G) {
                            const Pack<T, 16> v = x.at(j);
#pragma unroll
                            for (int e = 0; e < E; ++e) {
                                const Key key = K::of(v.e[e], max(j * E + e - x.r.off, 0));
                                if (key < last && key > next) next = key;
                            }
                        }
                        next = warp_largest(next);
                        if constexpr (G > 32) {
                            if (lane == 0) sh.buf[threadIdx.x >> 5] = next;
                            Gr::sync();
                            for (int w = 0; w < WARPS; ++w) next = max(next, sh.buf[w]);
                            Gr::sync();
                        }
                        last = next;
                        if (me == 0) sh.best[i] = last;
                    }
                }
                Gr::sync();
                if (G > 32 && me == 0) sh.count = 0;
                for (int i = me; i < have; i += G)
                    x.element(K::element(sh.best[i])) = from_f32<T>(-INFINITY);
                Gr::sync();
                float first = n > k ? K::value(sh.best[k]) : -INFINITY;
                if (n == k && bound > lowest<T>()) {
                    Pack<T, 16> m = all_minus_inf<T>();
                    for (int j = me; j < x.r.n; j += G) m = larger(m, x.at(j));
                    both = half_maxima(m);
                    first = Gr::max(max_nan(both.x, both.y), sh.space);
                }
                if (first > -INFINITY) {
                    const Exponent f(first, p.scale, p.scale_low);
                    float sum = 0.0f;
#pragma unroll 4
                    for (int j = me; j < x.r.n; j += G) {
                        float2 e[E / 2];
                        sum += terms_of(x.at(j), f, e);
                    }
                    sum = Gr::sum(sum, sh.space);
                    if (G == 32 || me < 32) rest = rest_of(p, sum, first);         // thread 0 stores it
                }
            }
        }
        const int64_t out = row * k;
        for (int i = me; i < k; i += G) {
            const Key key = i < have ? sh.best[i] : 0;
            reinterpret_cast<T*>(p.values)[out + i] =
                from_f32<T>(i < have ? K::value(key) : -INFINITY);
            p.ids[out + i] = i < have ? K::element(key) : -1;
        }
        if (me == 0) p.rest[row] = rest;
        Gr::sync();                                        // the stage has been read
        if (me == 0 && live[ring.stages]) {
            fence_proxy_async();
            staged(row + ring.stages * groups, st).fetch(&sh.bar[st]);
        }
        live.advance(p.lat, row + groups, groups, p.lat.rows);
        st = st + 1 == ring.stages ? 0 : st + 1;
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
    float scale, scale_low;                // log2 e / tau, in two parts
    float tau, inv_tau, inv_tau_low;       // the reciprocal in two parts
    float grad_scale;                      // tau * weight, over the batch for the mean
    double loss_scale;                     // of a row's loss, which is tau times its divergence
    char* grad;                            // or NULL
    float* row_loss;                       // [rows], 0 where a row does not count
    double* part_loss;                     // [B][splits]
    int32_t splits;                        // blocks of k_distill_sum a sample
    int32_t* done;                         // those that have finished
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

// d / tau of a difference of logits.  By a reciprocal rounded to one float32 all rows would be off the
// same way, by 3e-8 of their exponents.  (Both parts are above 0, so that -inf stays it.)
__device__ __forceinline__ float over_tau(const DistillParams& p, float d) {
    return __fmaf_rn(d, p.inv_tau, d * p.inv_tau_low);
}
// rest - logit / tau; logit / tau outside float32's range is the nearer end of it (as in a rest), and so is
// a difference above it.
__device__ __forceinline__ float rest_above(const DistillParams& p, float rest, float logit) {
    const float hi = logit * p.inv_tau, far = rest - copysignf(kMost, hi);
    const float low = __fmaf_rn(logit, p.inv_tau_low, __fmaf_rn(logit, p.inv_tau, -hi));
    const float d = fabsf(hi) >= kMost ? far : sum_of(rest, -hi, -low);
    return rest < INFINITY ? fminf(d, kMost) : rest;
}

// tau times what a class adds to a row's divergence, for probabilities p of the teacher and q:
// p (x + exp(-x) - 1) with x = log p - log q, which adds up to sum p x as p and q add up to 1 each.
// Every class's part is positive, and an error of x counts p - q times only: the sum of p x would lose
// a small divergence among its rounded logarithms, and keep what of their errors points one way.
// d: x times tau, but for what is small beside 1e30, where x may leave float32; +inf where q is 0.
__device__ __forceinline__ float divergence(const DistillParams& a, float w, float p, float q, float x,
                                            float d) {
    float y = __fmaf_rn(x, 1.0f / 40320.0f, -1.0f / 5040.0f);          // the series, to 3e-8 of the value
    y = __fmaf_rn(x, y, 1.0f / 720.0f);
    y = __fmaf_rn(x, y, -1.0f / 120.0f);
    y = __fmaf_rn(x, y, 1.0f / 24.0f);
    y = __fmaf_rn(x, y, -1.0f / 6.0f);
    y = __fmaf_rn(x, y, 0.5f);
    y = a.tau * (fabsf(x) <= 0.5f ? p * (x * x * y) : __fmaf_rn(p, x - 1.0f, q));
    if (d > 1e30f) y = d == INFINITY ? d : p * d;
    return w == 0.0f ? a.tau * q : y;                      // (p may be rounded to 0 before w is)
}

// Which of the warp's ids (of places 0 to 31, and 32 to 63) stand in a place before theirs: bits 0, 1.
__device__ __noinline__ unsigned repeated(int id0, int id1) {
    const int lane = threadIdx.x & 31;
    unsigned again = 0;
    for (int o = 0; o < 32; ++o) {
        const int x = __shfl_sync(kAll, id0, o), y = __shfl_sync(kAll, id1, o);
        if (id0 >= 0 && x == id0 && o < lane) again |= 1;
        if (id1 >= 0 && (x == id1 || (y == id1 && o < lane))) again |= 2;
    }
    return again;
}


// A teacher's row, P places a lane of a warp.
template <int P>
struct Teacher {
    int id[P];                             // -1: an empty place
    float t[P];                            // its logit, -inf in an empty place
    float rest;                            // -inf without one

    __device__ __forceinline__ void load(const DistillParams& a, int64_t row, int64_t place0) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const int k = lane + 32 * q;
            id[q] = -1;
            t[q] = -INFINITY;
            if (k < a.k) {
                id[q] = a.ids[place0 + k];
                t[q] = teacher_logit(a, place0 + k);
            }
        }
        rest = a.rest ? a.rest[row] : -INFINITY;
    }
    // Empties places without an output of the vocabulary; says what is not allowed.
    __device__ __forceinline__ void check(const DistillParams& a) {
        bool bad = !(rest < INFINITY);
#pragma unroll
        for (int q = 0; q < P; ++q) {
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
    __device__ __forceinline__ void drop_repeated(const DistillParams& a) {
        const unsigned again = repeated(id[0], P > 1 ? id[P - 1] : -1);
#pragma unroll
        for (int q = 0; q < P; ++q)
            if (again >> q & 1) {
                id[q] = -1;
                t[q] = -INFINITY;
            }
        invalid(a.status);
    }
    // Whether anything is in it (NaN counts: the loss says so).
    __device__ __forceinline__ bool some() const {
        bool any = rest != -INFINITY;
#pragma unroll
        for (int q = 0; q < P; ++q) any |= t[q] != -INFINITY;
        return __any_sync(kAll, any);
    }
};

// A row's places, relative to the largest of their teacher's logits and of their student's (`t_top`,
// `top`), the teacher's also to the rest where that is larger (`shift`, over tau):
// w = exp((t - t_top) / tau - shift), e = exp((x - top) / tau), gap = (t - t_top) - (x - top).  With W the
// sum of all w and total the row's sum relative to `base`, a place has
// p = w / W and log p - log q = (gap + base - top) / tau + log (total / W) - shift.
template <int P>
struct Places {
    float at[P], w[P], e[P], gap[P], top, w_rest, shift;
    float log_w_rest;                      // -inf without a rest
    float w_sum, sum;                      // of this lane's, then of the warp's
    float inv_all;                         // 1 / W

    __device__ __forceinline__ void terms(const DistillParams& a, const Teacher<P>& te) {
        float m = -INFINITY, x = -INFINITY;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            m = max_nan(m, te.t[q]);
            x = max_nan(x, at[q]);
        }
        const float t_top = warp_max_nan(m);
        top = warp_max_nan(x);
        const float above = te.rest == -INFINITY || t_top == -INFINITY
                                ? te.rest : rest_above(a, te.rest, t_top);
        shift = t_top == -INFINITY ? above : fmaxf(above, 0.0f);
        log_w_rest = above == -INFINITY ? above : above - shift;
        // few terms, of which the largest is exactly 1: by expf, which ex2.approx's corrected mean is
        // not good enough for
        w_rest = te.rest == -INFINITY ? 0.0f : expf(log_w_rest);
        w_sum = sum = 0.0f;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const float t = te.t[q] - t_top, x = at[q] - top;
            w[q] = te.t[q] == -INFINITY ? 0.0f : expf(over_tau(a, t) - shift);
            e[q] = at[q] == -INFINITY ? 0.0f : expf(over_tau(a, x));
            gap[q] = at[q] == -INFINITY ? INFINITY : t - x;
            w_sum += w[q];
            sum += e[q];
        }
    }
    __device__ __forceinline__ void finish(float& left) {              // left: a third sum
        const float4 s = warp_sum4(w_sum, sum, left, 0.0f);
        w_sum = s.x, sum = s.y, left = s.z;
        inv_all = rounded_reciprocal(w_sum + w_rest);
    }
};

// The sum of a row whose outputs without a place have their largest at `outside` and a sum `left`
// relative to it, and whose places have `top` and `sum`.
struct Whole {
    float base, outer, inner;              // exp((outside - base) / tau), exp((top - base) / tau)
    float total, inv_total;
    __device__ __forceinline__ Whole(const DistillParams& a, float outside, float left, float top,
                                     float sum) {
        base = max_nan(outside, top);
        const bool out = outside >= top;                   // one of the two is 1
        const float other = expf(over_tau(a, (out ? top : outside) - base));
        outer = out ? 1.0f : other;
        inner = out ? other : 1.0f;
        total = left * outer + sum * inner;
        inv_total = rounded_reciprocal(total);
    }
    __device__ __forceinline__ bool good() const { return total > 0.0f && total < INFINITY; }
    // of the terms relative to `outside`
    __device__ __forceinline__ float factor(const DistillParams& a, float left,
                                            float p_rest) const {
        float c = outer * inv_total;
        if (a.rest && left > 0.0f) c -= p_rest * reciprocal(left);
        return c * a.grad_scale;
    }
    // Classes of the divergence: a place's, and that of all outputs without one.  With the sums' logarithms
    // log_ratio (of total / W) and log_left a class has w, e, q = e * unit and
    // log p - log q = d / tau + offset.
    struct Part {
        float w, e, unit, d, offset;
    };
    __device__ __forceinline__ Part part_of_place(float w, float e, float gap, float top, float shift,
                                                  float log_ratio) const {
        return {w, e, inner * inv_total, gap + (base - top), log_ratio - shift};
    }
    __device__ __forceinline__ Part part_of_rest(float w, float log_w, float outside, float left,
                                                 float log_ratio, float log_left) const {
        return {w, left, outer * inv_total, left > 0.0f ? base - outside : INFINITY,
                log_w + (log_ratio - log_left)};
    }
    __device__ __forceinline__ float divergence_of(const DistillParams& a, const Part& c,
                                                   float inv_all) const {
        return divergence(a, c.w, c.w * inv_all, c.e * c.unit, over_tau(a, c.d) + c.offset, c.d);
    }
    // tau times the row's divergence, of the warp's sums (the same in all lanes).
    template <int P>
    __device__ __forceinline__ float loss(const DistillParams& a, const Places<P>& pl, float outside,
                                          float left) const {
        const int lane = threadIdx.x & 31;
        const float mine = logf((lane & 1) ? left : total * pl.inv_all);   // the two logarithms by two lanes
        const float ratio = __shfl_sync(kAll, mine, 0), log_left = __shfl_sync(kAll, mine, 1);
        const Part rest = part_of_rest(pl.w_rest, pl.log_w_rest, outside, left, ratio, log_left);
        const bool spare = a.k < 32 * P;                   // a lane without a place takes the rest
        float sum = 0.0f;
        if (!spare && lane == 0) sum = divergence_of(a, rest, pl.inv_all);
#pragma unroll
        for (int q = 0; q < P; ++q) {
            Part c = part_of_place(pl.w[q], pl.e[q], pl.gap[q], pl.top, pl.shift, ratio);
            if (lane + 32 * q == a.k) c = rest;
            sum += divergence_of(a, c, pl.inv_all);
        }
        return warp_sum(sum);
    }
    template <int P>
    __device__ __forceinline__ float place(const DistillParams& a, const Places<P>& pl,
                                           int q) const {
        return (pl.e[q] * (inner * inv_total) - pl.w[q] * pl.inv_all) * a.grad_scale;
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
    Teacher<2> te;
    Places<2> pl;
    for (int64_t row = blockIdx.x; row < p.lat.rows; row += gridDim.x) {
        const bool live = row < rows && (!p.lat.padded || p.lat.inside(row));
        if (warp == 0 && live) {
            te.load(p, row, row * p.k);
            te.check(p);
            bool again = false;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (te.id[q] >= 0) {
                    const uint32_t bit = 1u << (te.id[q] & 31);
                    again |= (atomicOr(&marks[te.id[q] >> 5], bit) & bit) != 0;
                }
            if (__any_sync(kAll, again)) te.drop_repeated(p);
            const bool some = te.some();
            if (lane == 0) s_some = some;
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
                sum = top == -INFINITY ? 0.0f : sum * Exponent(m, p.scale, p.scale_low)(top);
                top = m;
            }
            const Exponent f(top, p.scale, p.scale_low);
#pragma unroll
            for (int e = 0; e < E; ++e) sum += f(y[e]);
        }
        const float wtop = warp_max_nan(top);
        sum = top == -INFINITY ? 0.0f : sum * Exponent(wtop, p.scale, p.scale_low)(top);
        sum = warp_sum(sum);
        if (lane == 0) {
            tops[warp] = wtop;
            sums[warp] = sum;
        }
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                pl.at[q] = te.id[q] >= 0 ? to_f32(r.x[te.id[q]]) : -INFINITY;
            pl.terms(p, te);
            const float wt = lane < WARPS ? tops[lane] : -INFINITY;
            const float ws = lane < WARPS ? sums[lane] : 0.0f;
            const float outside = warp_max_nan(wt);
            float left = wt == -INFINITY ? 0.0f : ws * Exponent(outside, p.scale, p.scale_low)(wt);
            pl.finish(left);
            const Whole w(p, outside, left, pl.top, pl.sum);
            if (!w.good()) invalid(p.status);              // NaN among them
            const float kl = w.loss(p, pl, outside, left);
#pragma unroll
            for (int q = 0; q < 2; ++q) te.t[q] = w.place(p, pl, q);
            if (lane == 0) {
                p.row_loss[row] = w.good() ? kl : NAN;
                s_base = outside == -INFINITY ? 0.0f : outside;
                s_coef = w.good() ? w.factor(p, left, pl.w_rest * pl.inv_all) : NAN;
            }
        }
        __syncthreads();
        if (p.grad) {
            const Exponent f(s_base, p.scale, p.scale_low);
            const float coef = s_coef;
            T* g = reinterpret_cast<T*>(p.grad) + row * p.V;
            for (int j = tid; j < r.n; j += TH) {
                Pack<T, 16> v = r.load(j);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    v.e[e] = from_f32<T>(f(to_f32(v.e[e])) * coef);
                r.store(g, j, v);
            }
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (te.id[q] >= 0) g[te.id[q]] = from_f32<T>(te.t[q]);
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

// What a block's last warp needs of a row's places for its loss.
struct Kept {
    float w[RNNT_MAX_TOP], e[RNNT_MAX_TOP], gap[RNNT_MAX_TOP];
    float inv_all, w_rest, shift, log_w_rest, outside, left;
    template <int P>
    __device__ __forceinline__ void put(const Places<P>& pl) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            w[lane + 32 * q] = pl.w[q];
            e[lane + 32 * q] = pl.e[q];
            gap[lane + 32 * q] = pl.gap[q];
        }
        if (lane == 0) {
            inv_all = pl.inv_all;
            w_rest = pl.w_rest;
            shift = pl.shift;
            log_w_rest = pl.log_w_rest;
        }
    }
    template <int P>
    __device__ __forceinline__ void get(Places<P>& pl) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            pl.w[q] = w[lane + 32 * q];
            pl.e[q] = e[lane + 32 * q];
            pl.gap[q] = gap[lane + 32 * q];
        }
        pl.inv_all = inv_all;
        pl.w_rest = w_rest;
        pl.shift = shift;
        pl.log_w_rest = log_w_rest;
    }
};
struct None {};

template <int G>
struct DistillScratch {
    uint64_t bar[kMostStages];
    typename Group<G>::Space space;
    float top, sum, p_rest;                // of the places, for a block
    int some;
    std::conditional_t<(G > 32), Kept, None> kept;
};

// Rows through a ring of shared memory, a group of threads each, one read and one write.  The places'
// logits are picked out of the staged row and -inf is left in their stead, so that what the threads
// then read is the rest alone; its terms stay in registers from their sum to the gradient (NV vectors
// a thread; NV = 0: rows too long for that are read from the stage again).  A group's first warp
// looks after the teacher, a block's last one after the loss, while the first is at the next row.
//
// Long rows are bound by memory: 226000 of 5000 float32 with 32 places take 1.66 ms (6.3 TB/s, 0.93
// of the copy's); rows of 1024 by issue slots: 480000 of float16 with 8 places 480 us (4.1 TB/s; 858
// warp instructions a row, 220 of them on elements, in 68 % of the slots).  3 blocks an SM of 80 registers
// against 2 of 87, at an earlier step: 487 and 579 us.  Two stages a warp: more would cost blocks.
template <typename T, int TH, int G, int NV, int P, bool WHOLE>
__global__ void __launch_bounds__(TH, NV == 8 && sizeof(T) == 2 ? 2 : NV == 0 || NV == 1 ? 4 : 3)
    k_distill(const DistillParams p, const Ring ring) {
    using Gr = Group<G>;
    using Scratch = DistillScratch<G>;
    using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
    constexpr int E = 16 / (int)sizeof(T), GROUPS = TH / G;
    extern __shared__ __align__(16) char space[];
    __shared__ int64_t space64[TH / 32];
    char* const mine = space + (G == 32 ? threadIdx.x / G : 0) * ring.group_bytes;
    Scratch& sh = *reinterpret_cast<Scratch*>(mine + ring.stages * ring.stage_bytes);
    const int me = Gr::rank(), lane = me & 31;
    const bool leads = G == 32 || threadIdx.x < 32;        // the teacher's warp
    const int64_t groups = (int64_t)gridDim.x * GROUPS;
    const int64_t first_row = (int64_t)blockIdx.x * GROUPS + (G == 32 ? threadIdx.x / G : 0);
    let_next_start();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
    const int64_t rows = p.lat.padded ? p.lat.rows : compact_rows<TH>(p.lat, space64);
    const T* const logits = reinterpret_cast<const T*>(p.logits);
    const T* const end = logits + p.lat.rows * p.V;
    const auto staged = [&](int64_t row, int st) {
        return Staged<T, G, WHOLE>(logits + row * p.V, p.V,
                                   reinterpret_cast<uint4*>(mine + st * ring.stage_bytes), logits,
                                   end);
    };
    if (me == 0) {
        for (int st = 0; st < ring.stages; ++st) mbar_init(&sh.bar[st]);
        fence_mbar_init();
    }
    Gr::sync();
    Window live(p.lat, first_row, groups, rows);
    if (me == 0)
        for (int st = 0; st < ring.stages; ++st)
            if (live[st]) staged(first_row + st * groups, st).fetch(&sh.bar[st]);
    int polls = kWaitPolls, st = 0;
    uint32_t phases = 0;                                   // a bit a stage
    Teacher<P> te, ahead;
    Places<P> pl;
    int64_t place0 = first_row * p.k;                      // of the row's places
    const int64_t place_step = groups * p.k;
    if (leads && live[0]) ahead.load(p, first_row, place0);
    for (int64_t row = first_row; row < p.lat.rows; row += groups) {
        const bool counts = live[0];
        bool weighed = false;
        te = ahead;
        place0 += place_step;
        if (leads && live[1]) ahead.load(p, row + groups, place0);     // one row ahead
        T* const g = reinterpret_cast<T*>(p.grad) + row * p.V;
        if (counts) {
            const Staged<T, G, WHOLE> x = staged(row, st);
            mbar_wait(&sh.bar[st], phases >> st & 1, polls, p.status);
            phases ^= 1u << st;
            x.complete();
            bool some = true;
            if (leads) {
                te.check(p);
#pragma unroll
                for (int q = 0; q < P; ++q)
                    pl.at[q] = te.id[q] >= 0 ? to_f32(x.element(te.id[q])) : -INFINITY;
                __syncwarp();
                // each place leaves its number; one that finds another's has its id in common
#pragma unroll
                for (int q = 0; q < P; ++q)
                    if (te.id[q] >= 0)
                        reinterpret_cast<volatile Bits&>(x.element(te.id[q])) =
                            (Bits)(lane + 32 * q);
                __syncwarp();
                bool again = false;
#pragma unroll
                for (int q = 0; q < P; ++q)
                    again |= te.id[q] >= 0 &&
                             reinterpret_cast<volatile Bits&>(x.element(te.id[q])) !=
                                 (Bits)(lane + 32 * q);
                if (__any_sync(kAll, again)) {
                    te.drop_repeated(p);
#pragma unroll
                    for (int q = 0; q < P; ++q)
                        if (te.id[q] < 0) pl.at[q] = -INFINITY;
                }
#pragma unroll
                for (int q = 0; q < P; ++q)
                    if (te.id[q] >= 0) x.element(te.id[q]) = from_f32<T>(-INFINITY);
                some = te.some();
                if (G > 32 && lane == 0) sh.some = some;
            }
            Gr::sync();
            if (G > 32) some = sh.some;
            if (!some) {
                if (p.grad) zero_row<T, G>(p, row);
                if (me == 0) p.row_loss[row] = 0.0f;
            } else {
                Pack<T, 16> m = all_minus_inf<T>();
#pragma unroll 4
                for (int j = me; j < x.r.n; j += G) m = larger(m, x.at(j));
                if (leads) {
                    pl.terms(p, te);
                    if constexpr (G > 32) {
                        float none = 0.0f;
                        pl.finish(none);
                        sh.kept.put(pl);
                        if (lane == 0) {
                            sh.top = pl.top;
                            sh.sum = pl.sum;
                            sh.p_rest = pl.w_rest * pl.inv_all;
                        }
                    }
                }
                const float2 both = half_maxima(m);
                const float outside = Gr::max(max_nan(both.x, both.y), sh.space);
                const Exponent f(outside == -INFINITY ? 0.0f : outside, p.scale, p.scale_low);
                float2 e[NV ? NV : 1][E / 2];
                float left = 0.0f;
                if constexpr (NV > 0) {
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (me + i * G < x.r.n) left += terms_of(x.at(me + i * G), f, e[i]);
                } else {
                    for (int j = me; j < x.r.n; j += G) left += terms_of(x.at(j), f, e[0]);
                }
                if constexpr (G > 32) left = Gr::sum(left, sh.space);
                else pl.finish(left);
                const float top = G > 32 ? sh.top : pl.top, sum = G > 32 ? sh.sum : pl.sum;
                const Whole w(p, outside, left, top, sum);
                if (p.grad) {
                    const float c = w.good() ? w.factor(p, left,
                                                       G > 32 ? sh.p_rest
                                                              : pl.w_rest * pl.inv_all) : NAN;
                    const float2 c2 = make_float2(c, c);
                    const auto put = [&](int j, float2 (&y)[E / 2]) {
                        Pack<T, 16> v;
#pragma unroll
                        for (int i = 0; i < E / 2; ++i) y[i] = mul2(y[i], c2);
                        pack(v, y);
                        x.r.store(g, j, v);
                    };
                    if constexpr (NV > 0) {
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            if (me + i * G < x.r.n) put(me + i * G, e[i]);
                    } else {
                        for (int j = me; j < x.r.n; j += G) {
                            terms_of(x.at(j), f, e[0]);
                            put(j, e[0]);
                        }
                    }
                }
                if (leads && !w.good()) invalid(p.status); // NaN among them
                if constexpr (G == 32) {
                    const float kl = w.loss(p, pl, outside, left);
                    if (lane == 0) p.row_loss[row] = w.good() ? kl : NAN;
                } else {
                    weighed = true;
                    if (me == 0) {
                        sh.kept.outside = outside;
                        sh.kept.left = left;
                    }
                }
                if (p.grad) {
                    Gr::sync();                            // behind the rest's stores
                    if (leads) {
#pragma unroll
                        for (int q = 0; q < P; ++q)
                            if (te.id[q] >= 0) g[te.id[q]] = from_f32<T>(w.place(p, pl, q));
                    }
                }
            }
        } else {
            if (p.grad) zero_row<T, G>(p, row);
            if (me == 0) p.row_loss[row] = 0.0f;
        }
        Gr::sync();                                        // the stage has been read
        if (me == 0 && live[ring.stages]) {
            fence_proxy_async();
            staged(row + ring.stages * groups, st).fetch(&sh.bar[st]);
        }
        if constexpr (G > 32) {
            // the loss by the last warp, while the first one looks at the next row's teacher (whose
            // places take the place of these behind a barrier)
            if (weighed && threadIdx.x >= TH - 32) {
                sh.kept.get(pl);
                pl.top = sh.top;
                const float outside = sh.kept.outside, left = sh.kept.left;
                const Whole w(p, outside, left, pl.top, sh.sum);
                const float kl = w.loss(p, pl, outside, left);
                if (lane == 0) p.row_loss[row] = w.good() ? kl : NAN;
            }
        }
        live.advance(p.lat, row + groups, groups, rows);
        st = st + 1 == ring.stages ? 0 : st + 1;
    }
}

// ------------------------------------------------------------------ short rows
// A warp takes 32 consecutive rows, which are one aligned piece of memory whatever V is, through its
// part of shared memory (unless none of them counts), and a thread each of them: no reductions, no idle
// lanes.  172000 rows of 29 float32 with 8 places take 27 us with the gradient (a warp a row: 130); 1.9
// TB/s, bound by latency: a thread's looks at its row follow one another.
struct ShortBatch {
    int32_t stage_bytes, warp_bytes;       // of a warp: the rows; with what is behind them
};
constexpr int kShortThreads = 128;
constexpr int kShortRow = 512;             // bytes of a row, at most: 16 KB a warp

// A thread's row in shared memory.  Its elements are gone through from `start` on, which turns with
// the thread so that a warp's accesses lie in different banks where V is even.
template <typename T>
struct ShortRow {
    using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
    static constexpr Bits kTaken = (Bits)~0u;              // a NaN; rows with one are left out before
    T* s;
    int V, start;
    __device__ __forceinline__ ShortRow(T* rows, int size) : V(size) {
        const int lane = threadIdx.x & 31;
        s = rows + lane * V;
        start = sizeof(T) == 4 ? (V % 2 ? 0 : lane) : (V % 4 ? 0 : 2 * lane);
        start %= V;
    }
    __device__ __forceinline__ Bits& bits(int i) const { return reinterpret_cast<Bits*>(s)[i]; }
    template <typename F>
    __device__ __forceinline__ void each(F&& f) const {
#pragma unroll 4
        for (int i = start; i < V; ++i) f(i, s[i]);
#pragma unroll 4
        for (int i = 0; i < start; ++i) f(i, s[i]);
    }
};

// Brings `n` rows from row0 on; all lanes call it.
template <typename T>
__device__ __forceinline__ void fetch_short(const char* logits, int64_t row0, int n, int V, T* stage,
                                            uint64_t* bar, uint32_t& phase, int& polls,
                                            int32_t* status) {
    const int lane = threadIdx.x & 31;
    const T* x = reinterpret_cast<const T*>(logits) + row0 * V;
    const uint32_t bytes = (uint32_t)(n * V) * (uint32_t)sizeof(T), whole = bytes & ~15u;
    if (lane == 0) {
        fence_proxy_async();
        bulk_load(stage, x, whole, bar);
    }
    const int i = (int)(whole / sizeof(T)) + lane;         // behind the last whole unit
    if (i < n * V) stage[i] = x[i];
    mbar_wait(bar, phase, polls, status);
    phase ^= 1;
    __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(kShortThreads) k_top_short(const TopParams p, const ShortBatch sb) {
    extern __shared__ __align__(16) char space[];
    __shared__ uint64_t bars[kShortThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = p.k;
    char* const mine = space + warp * sb.warp_bytes;
    T* const stage = reinterpret_cast<T*>(mine);
    T* const values = reinterpret_cast<T*>(mine + sb.stage_bytes);
    int32_t* const ids = reinterpret_cast<int32_t*>(mine + sb.stage_bytes + 128 * k);
    uint64_t* const bar = &bars[warp];
    if (blockIdx.x == 0 && p.lat.T) check_lengths<kShortThreads>(p.lat, p.status);
    if (lane == 0) {
        mbar_init(bar);
        fence_mbar_init();
    }
    __syncwarp();
    int polls = kWaitPolls;
    uint32_t phase = 0;
    const int64_t step = (int64_t)gridDim.x * (kShortThreads / 32) * 32;
    for (int64_t row0 = ((int64_t)blockIdx.x * (kShortThreads / 32) + warp) * 32; row0 < p.lat.rows;
         row0 += step) {
        const int n = (int)min((int64_t)32, p.lat.rows - row0);
        const int64_t row = row0 + lane;
        const bool counts = lane < n && (!p.lat.T || p.lat.inside(row));
        if (__any_sync(kAll, counts))
            fetch_short(p.logits, row0, n, p.V, stage, bar, phase, polls, p.status);
        const ShortRow<T> r(stage, p.V);
        float rest = -INFINITY;
        int have = 0;
        if (counts) {
            float top = -INFINITY;
            r.each([&](int, T x) { top = max_nan(top, to_f32(x)); });
            if (!(top < INFINITY)) {                       // NaN or +inf: the row is left empty
                invalid(p.status);
            } else {
                float best = -INFINITY;
                for (int q = 0; q <= k; ++q) {             // the last is the largest of the rest
                    best = -INFINITY;
                    int at = p.V;
                    r.each([&](int i, T x) {
                        const float y = to_f32(x);
                        if (y > best || (y == best && i < at)) {
                            best = y;
                            at = i;
                        }
                    });
                    if (best == -INFINITY || q == k) break;
                    values[lane * k + q] = from_f32<T>(best);
                    ids[lane * k + q] = at;
                    have = q + 1;
                    r.s[at] = from_f32<T>(-INFINITY);
                }
                if (best > -INFINITY) {
                    const Exponent f(best, p.scale, p.scale_low);
                    float sum = 0.0f;
                    r.each([&](int, T x) { sum += f(to_f32(x)); });
                    rest = rest_of(p, sum, best);
                }
            }
        }
        if (lane < n) {
            for (int q = have; q < k; ++q) {
                values[lane * k + q] = from_f32<T>(-INFINITY);
                ids[lane * k + q] = -1;
            }
            p.rest[row] = rest;
        }
        __syncwarp();
        for (int i = lane; i < n * k; i += 32) {
            reinterpret_cast<T*>(p.values)[row0 * k + i] = values[i];
            p.ids[row0 * k + i] = ids[i];
        }
        __syncwarp();
    }
}

template <typename T>
__global__ void __launch_bounds__(kShortThreads) k_distill_short(const DistillParams p,
                                                                 const ShortBatch sb) {
    extern __shared__ __align__(16) char space[];
    __shared__ uint64_t bars[kShortThreads / 32];
    __shared__ int64_t space64[kShortThreads / 32];
    using Bits = typename ShortRow<T>::Bits;
    constexpr Bits kTaken = ShortRow<T>::kTaken;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    char* const mine = space + warp * sb.warp_bytes;
    T* const stage = reinterpret_cast<T*>(mine);
    float* const ats = reinterpret_cast<float*>(mine + sb.stage_bytes);    // [k][32]
    uint64_t* const bar = &bars[warp];
    let_next_start();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
    const int64_t rows = p.lat.padded ? p.lat.rows : compact_rows<kShortThreads>(p.lat, space64);
    if (lane == 0) {
        mbar_init(bar);
        fence_mbar_init();
    }
    __syncwarp();
    int polls = kWaitPolls;
    uint32_t phase = 0;
    const int64_t step = (int64_t)gridDim.x * (kShortThreads / 32) * 32;
    for (int64_t row0 = ((int64_t)blockIdx.x * (kShortThreads / 32) + warp) * 32; row0 < p.lat.rows;
         row0 += step) {
        const int n = (int)min((int64_t)32, p.lat.rows - row0);
        const int64_t row = row0 + lane, first = row * p.k;
        const bool counts = lane < n && row < rows && (!p.lat.padded || p.lat.inside(row));
        if (__any_sync(kAll, counts))
            fetch_short(p.logits, row0, n, p.V, stage, bar, phase, polls, p.status);
        const ShortRow<T> r(stage, p.V);
        float loss = 0.0f, outside = -INFINITY, t_top = -INFINITY, top = -INFINITY;
        bool some = false;
        if (counts) {
            bool bad = false;
            float most = -INFINITY;
            r.each([&](int, T x) { most = max_nan(most, to_f32(x)); });
            const bool fine = most < INFINITY;
            // the places: their logits are put aside, and what they leave is marked; +inf: an empty one
            for (int q = 0; q < p.k; ++q) {
                const int id = p.ids[first + q];
                float at = INFINITY;
                bad |= id >= p.V;
                if ((unsigned)id < (unsigned)p.V) {
                    if (r.bits(id) == kTaken && fine) {
                        bad = true;                        // an id again
                    } else {
                        const float t = teacher_logit(p, first + q);
                        bad |= !(t < INFINITY);
                        at = fine ? to_f32(r.s[id]) : -INFINITY;
                        r.bits(id) = kTaken;
                        t_top = max_nan(t_top, t);
                        top = fmaxf(top, at);
                    }
                }
                ats[q * 32 + lane] = at;
            }
            const float rest = p.rest ? p.rest[row] : -INFINITY;
            bad |= !(rest < INFINITY);
            some = t_top != -INFINITY || rest != -INFINITY;        // NaN counts
            const float above = rest == -INFINITY || t_top == -INFINITY
                                    ? rest : rest_above(p, rest, t_top);
            const float shift = t_top == -INFINITY ? above : fmaxf(above, 0.0f);
            if (some) {
                r.each([&](int i, T x) {
                    if (r.bits(i) != kTaken) outside = fmaxf(outside, to_f32(x));
                });
                const Exponent f(outside == -INFINITY ? 0.0f : outside, p.scale, p.scale_low);
                float left = 0.0f;
                r.each([&](int i, T x) { left += r.bits(i) != kTaken ? f(to_f32(x)) : 0.0f; });
                const auto weight = [&](int q) {           // of a place
                    const float x = teacher_logit(p, first + q);
                    return x == -INFINITY ? 0.0f : expf(over_tau(p, x - t_top) - shift);
                };
                const auto term = [&](float at) {
                    return at == -INFINITY ? 0.0f : expf(over_tau(p, at - top));
                };
                float sum = 0.0f, w_sum = 0.0f;
                for (int q = 0; q < p.k; ++q) {
                    const float at = ats[q * 32 + lane];
                    if (at == INFINITY) continue;
                    sum += term(at);
                    w_sum += weight(q);
                }
                const float log_w_rest = above - shift;
                const float w_rest = rest == -INFINITY ? 0.0f : expf(log_w_rest);
                const Whole w(p, outside, left, top, sum);
                const bool good = fine && w.good();
                bad |= !good;
                const float all = w_sum + w_rest, inv_all = rounded_reciprocal(all);
                const float ratio = logf(w.total * inv_all);
                loss = w.divergence_of(
                    p, w.part_of_rest(w_rest, log_w_rest, outside, left, ratio, logf(left)), inv_all);
                if (p.grad) {
                    const float c = good ? w.factor(p, left, w_rest * inv_all) : NAN;
                    r.each([&](int i, T x) {
                        if (r.bits(i) != kTaken || c != c) r.s[i] = from_f32<T>(f(to_f32(x)) * c);
                    });
                }
                for (int q = 0; q < p.k; ++q) {
                    const float at = ats[q * 32 + lane];
                    if (at == INFINITY) continue;
                    const float e = term(at), wq = weight(q);
                    const float gap = at == -INFINITY
                                          ? INFINITY
                                          : (teacher_logit(p, first + q) - t_top) - (at - top);
                    loss += w.divergence_of(p, w.part_of_place(wq, e, gap, top, shift, ratio), inv_all);
                    if (p.grad)
                        r.s[p.ids[first + q]] = from_f32<T>(
                            good ? (e * (w.inner * w.inv_total) - wq * inv_all) * p.grad_scale : NAN);
                }
                if (!good) loss = NAN;
            }
            if (bad) invalid(p.status);
        }
        if (lane < n) p.row_loss[row] = loss;
        if (!p.grad) {
            __syncwarp();
            continue;
        }
        if (lane < n && !some)
            for (int i = 0; i < p.V; ++i) r.s[i] = from_f32<T>(0.0f);
        fence_proxy_async();
        __syncwarp();
        T* const y = reinterpret_cast<T*>(p.grad) + row0 * p.V;
        const uint32_t bytes = (uint32_t)(n * p.V) * (uint32_t)sizeof(T), whole = bytes & ~15u;
        const int i = (int)(whole / sizeof(T)) + lane;     // behind the last whole unit
        if (i < n * p.V) y[i] = stage[i];
        if (lane == 0) {
            if (whole) bulk_store(y, stage, whole);
            bulk_commit();
            bulk_wait_read<0>();                           // the stage is free again
        }
        __syncwarp();
    }
    if (lane == 0) bulk_wait_all();
}

// Rows' losses to samples' and the batch's, added in float64 in an order that depends on the sizes
// alone: `splits` blocks a sample take a part of its rows each, and the last block of all adds what
// they leave.  (One block a sample took 36 us for 16 samples of 30000 rows, and 106 in the padded
// layout, beside rows of 450 and 400.)  The compact layout's row offsets stay in the workspace for
// the gradient's scaling.
constexpr int kSumThreads = 256;
constexpr int kMostSplits = 64;
__global__ void __launch_bounds__(kSumThreads) k_distill_sum(const DistillParams p) {
    constexpr int TH = kSumThreads, WARPS = TH / 32;
    __shared__ int64_t space64[WARPS];
    __shared__ double space[WARPS];
    __shared__ bool last;
    const int b = (int)(blockIdx.x / (unsigned)p.splits), tid = threadIdx.x;
    const int part = (int)(blockIdx.x - (unsigned)b * p.splits);
    int t, u;
    bool ok;
    const int64_t n = p.lat.of_sequence(b, t, u, ok);
    int64_t first = 0;
    if (!p.lat.padded) {
        const int64_t most = p.lat.rows + 1;               // so that one too many shows in the sum
        for (int i = tid; i < b; i += TH) {
            int t0, u0;
            bool ok0;
            first += min(p.lat.of_sequence(i, t0, u0, ok0), most);
        }
        first = block_sum<TH>(first, space64);
        const int64_t end = first + min(n, most);
        if (b == p.lat.B - 1) ok &= end == p.lat.rows;
        if (tid == 0 && part == 0) {
            p.first_row[b] = first;
            if (b == p.lat.B - 1) p.first_row[b + 1] = end;
        }
    }
    if (!ok && tid == 0) invalid(p.status);
    wait_for_previous();
    double sum = 0.0;
    if (p.lat.padded) {
        const int64_t each = (n + p.splits - 1) / p.splits, end = min(n, (part + 1) * each);
        const float* rows = p.row_loss + (int64_t)b * p.lat.max_T * (p.lat.max_U + 1);
        const uint32_t w = (uint32_t)u + 1;
        for (int64_t i = part * each + tid; i < end; i += TH) {
            const int64_t q = n <= INT32_MAX ? (int64_t)((uint32_t)i / w) : i / w;
            sum += rows[q * (p.lat.max_U + 1) + (i - q * w)];
        }
    } else {
        const int64_t here = max((int64_t)0, min(n, p.lat.rows - first));
        const int64_t each = (here + p.splits - 1) / p.splits, end = min(here, (part + 1) * each);
        for (int64_t i = part * each + tid; i < end; i += TH) sum += p.row_loss[first + i];
    }
    sum = block_sum<TH>(sum, space);
    if (tid == 0) {
        p.part_loss[blockIdx.x] = sum;
        __threadfence();
        last = atomicAdd(p.done, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = 0.0;
    for (int i = tid; i < p.lat.B; i += TH) {
        const volatile double* parts = p.part_loss + (int64_t)i * p.splits;
        double sample = 0.0;
        for (int k = 0; k < p.splits; ++k) sample += parts[k];
        sample *= p.loss_scale;
        p.loss[i] = (float)sample;
        sum += sample;
    }
    sum = block_sum<TH>(sum, space);
    if (tid == 0 && p.loss_reduced) *p.loss_reduced = (float)(p.mean ? sum / p.lat.B : sum);
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
    size_t row_loss, part_loss, first_row, done, total;
};
// Blocks a sample of the sums: about four an SM, each with a few thousand rows at least.
int32_t splits_of(int32_t B, int64_t rows) {
    return (int32_t)std::max<int64_t>(
        1, std::min<int64_t>({kMostSplits, 4 * kSMs / B, rows / B / 2048}));
}
DistillLayout distill_layout(int32_t B, int64_t rows) {
    DistillLayout L;
    L.first_row = 0;                       // first: what rnnt_distill_grad_scale reads
    L.part_loss = align256(L.first_row + ((size_t)B + 1) * sizeof(int64_t));
    L.done = align256(L.part_loss + (size_t)B * splits_of(B, rows) * sizeof(double));
    L.row_loss = L.done + 256;
    L.total = align256(L.row_loss + (size_t)rows * sizeof(float));
    return L;
}

// How rows of V elements are taken: by a warp or a block, through how many stages.
constexpr int kWarpThreads = 256;          // of blocks whose warps take a row each
constexpr int kBlockThreads = 256;         // of blocks that take a row each
constexpr size_t kShared = 226 << 10;      // of a block, at most (1 KB is left for what is static)
struct Shape {
    int group;                             // 32, kBlockThreads, or 0: the kernels of long rows
    Ring ring;
    size_t shared;
    int64_t blocks;
};
Shape shape_of(const void* logits, int64_t rows, int32_t V, int es, size_t warp_scratch,
               size_t block_scratch) {
    Shape s{};
    // at any alignment where rows are not whole units
    const size_t row = (size_t)V * es, units =
        row % 16 || ((uintptr_t)logits & 15) ? (row + 30) / 16 * 16 : row;
    const bool warp = units <= 4096;
    const int groups = warp ? kWarpThreads / 32 : 1;
    const size_t scratch = ((warp ? warp_scratch : block_scratch) + 15) & ~size_t(15);
    int stages = kMostStages;
    while (stages > 1 && groups * (stages * units + scratch) > kShared / 2) --stages;
    if (groups * (stages * units + scratch) > kShared) return s;
    s.group = warp ? 32 : kBlockThreads;
    s.ring.stages = stages;
    s.ring.stage_bytes = (uint32_t)units;
    s.ring.group_bytes = (uint32_t)(stages * units + scratch);
    s.shared = (size_t)groups * s.ring.group_bytes;
    s.blocks = (rows + groups - 1) / groups;
    return s;
}
// One wave of blocks, each taking its rows in turn.
template <typename K>
unsigned grid_of(const Shape& s, K kernel, int threads) {
    int per_sm = 1;
    if (s.blocks > kSMs &&
        (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, s.shared) !=
             cudaSuccess || per_sm < 1)) {
        cudaGetLastError();
        per_sm = 1;
    }
    return (unsigned)std::min<int64_t>(s.blocks, (int64_t)kSMs * per_sm);
}

// Rows that are short enough for a thread each.
bool short_rows(const void* logits, int32_t V, int es) {
    return (size_t)V * es <= kShortRow && ((uintptr_t)logits & 15) == 0;
}
ShortBatch short_batch(int32_t V, int es, size_t behind) {
    ShortBatch sb;
    sb.stage_bytes = 32 * V * es;
    sb.warp_bytes = (int32_t)(((size_t)sb.stage_bytes + behind + 127) & ~size_t(127));
    return sb;
}
template <typename K>
unsigned short_grid(K kernel, int64_t rows, size_t shared) {
    Shape s{};
    s.shared = shared;
    s.blocks = (rows + kShortThreads - 1) / kShortThreads;
    return grid_of(s, kernel, kShortThreads);
}

template <typename T>
bool raise_top() {
    const auto raise = [](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kShared) == cudaSuccess;
    };
    return raise(k_top<T, kWarpThreads, 32, true>) && raise(k_top<T, kWarpThreads, 32, false>) &&
           raise(k_top<T, kBlockThreads, kBlockThreads, true>) &&
           raise(k_top<T, kBlockThreads, kBlockThreads, false>) &&
           raise(k_top_short<T>) && raise(k_distill_short<T>);
}
// Calls f(k_distill's form for rows of n vectors and k places).
template <typename T, typename F>
auto distill_form(int group, int n, int k, bool whole, F&& f) {
    const auto by_places = [&](auto g, auto nv) {
        constexpr int G = decltype(g)::value, NV = decltype(nv)::value;
        constexpr int TH = G == 32 ? kWarpThreads : G;
        if (whole)
            return k <= 32 ? f(k_distill<T, TH, G, NV, 1, true>, TH)
                           : f(k_distill<T, TH, G, NV, 2, true>, TH);
        return k <= 32 ? f(k_distill<T, TH, G, NV, 1, false>, TH)
                       : f(k_distill<T, TH, G, NV, 2, false>, TH);
    };
    using std::integral_constant;
    if (group == 32) {
        constexpr integral_constant<int, 32> g{};
        if (n <= 32) return by_places(g, integral_constant<int, 1>{});
        if (n <= 128) return by_places(g, integral_constant<int, 4>{});
        return by_places(g, integral_constant<int, 8>{});
    }
    constexpr integral_constant<int, kBlockThreads> g{};
    constexpr int most = sizeof(T) == 4 ? 8 : 4;           // vectors in 32 registers
    if (n <= most * kBlockThreads) return by_places(g, integral_constant<int, most>{});
    return by_places(g, integral_constant<int, 0>{});
}
template <typename T>
bool raise_distill() {
    bool ok = true;
    const auto raise = [](auto kernel, int) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kShared) == cudaSuccess;
    };
    for (bool whole : {false, true})
        for (int k : {1, 64}) {
            for (int n : {1, 100, 200}) ok &= distill_form<T>(32, n, k, whole, raise);
            for (int n : {1, 1 << 20}) ok &= distill_form<T>(kBlockThreads, n, k, whole, raise);
        }
    return ok;
}
bool distill_prepared() {
    static std::atomic<bool> done[64];
    return prepared_once(done, [] {
        const auto raise = [](auto kernel) {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        RNNT_MAX_TOP_VOCAB / 8) == cudaSuccess;
        };
        return raise_top<float>() && raise_top<__half>() && raise_top<__nv_bfloat16>() &&
               raise_distill<float>() && raise_distill<__half>() &&
               raise_distill<__nv_bfloat16>() &&
               raise(k_distill_long<float>) && raise(k_distill_long<__half>) &&
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
    parts_below(kLog2e / temperature, p.scale, p.scale_low);
    parts_below(1.0 / temperature, p.inv_tau, p.inv_tau_low);
    p.values = values;
    p.ids = ids;
    p.rest = rest;
    p.status = status_dev;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!distill_prepared() || !clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    with_type(dt, [&](auto t) {
        using T = decltype(t);
        // the best are taken one by one, in k + 1 looks at the row.  172000 rows by a thread and by a warp
        // each, us: float32 V = 29, k = 8 20 and 174; 64, 4 100 and 107; 64, 8 158 and 127; 96, 16 298 and 163;
        // 128, 1 73 and 95; 128, 16 (a warp's from here on) 417 and 155; float16 48, 16 132 and 220; 80, 16
        // 179 and 312; 96, 4 97 and 115; 128, 8 269 and 132; 256, 8 (a warp's) 341 and 125.  A warp is slow
        // where a row has fewer vectors than k + 1, a thread where V is a power of 2; over 60 pairs of
        // V and k up to the border the rule's choice took 8 % more than the better one.
        if (short_rows(logits, V, es) && (k + 1) * V <= 2048) {
            const ShortBatch sb = short_batch(V, es, (size_t)256 * k);
            const size_t shared = (size_t)sb.warp_bytes * (kShortThreads / 32);
            k_top_short<T><<<short_grid(k_top_short<T>, rows, shared), kShortThreads, shared, st>>>(
                p, sb);
            return;
        }
        const Shape s = shape_of(logits, rows, V, es, sizeof(TopScratch<T, 32>),
                                 sizeof(TopScratch<T, kBlockThreads>));
        const auto launch = [&](auto kernel, int threads) {
            kernel<<<grid_of(s, kernel, threads), threads, s.shared, st>>>(p, s.ring);
        };
        const bool whole = (size_t)V * es % 16 == 0 && ((uintptr_t)logits & 15) == 0;
        if (s.group == 32 && whole) launch(k_top<T, kWarpThreads, 32, true>, kWarpThreads);
        else if (s.group == 32) launch(k_top<T, kWarpThreads, 32, false>, kWarpThreads);
        else if (s.group && whole)
            launch(k_top<T, kBlockThreads, kBlockThreads, true>, kBlockThreads);
        else if (s.group) launch(k_top<T, kBlockThreads, kBlockThreads, false>, kBlockThreads);
        else
            k_top_long<T><<<row_grid(rows), kLongThreads, 0, st>>>(p);
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
    parts_below(kLog2e / temperature, p.scale, p.scale_low);
    parts_below(1.0 / temperature, p.inv_tau, p.inv_tau_low);
    p.mean = reduction == RNNT_RED_MEAN;
    p.grad_scale = (float)(temperature * weight / (p.mean ? B : 1));
    p.tau = (float)temperature;
    p.loss_scale = temperature * temperature * weight / p.tau;
    p.grad = static_cast<char*>(grad);
    p.row_loss = reinterpret_cast<float*>(ws + L.row_loss);
    p.part_loss = reinterpret_cast<double*>(ws + L.part_loss);
    p.splits = splits_of(B, rows);
    p.first_row = reinterpret_cast<int64_t*>(ws + L.first_row);
    p.done = reinterpret_cast<int32_t*>(ws + L.done);
    p.loss = loss;
    p.loss_reduced = loss_reduced;
    p.status = status_dev;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!distill_prepared() || !clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    with_type(dt, [&](auto t) {
        using T = decltype(t);
        // A thread's time goes with its looks at the row and at the places, a warp's is nearly the same for any
        // row up to 512 bytes, longer where rows are not whole units; V of a power of 2 costs a thread bank
        // conflicts.  172000 rows, by a thread and by a warp each, us.  Loss alone: float32 V = 29, k = 4 27
        // and 122; 64, 16 105 and 106; 128, 16 129 and 107; 33, 32 200 and 125; float16 128, 4 93 and 114;
        // 205, 16 92 and 132; 256, 16 152 and 117; 184, 32 167 and 119.  With the gradient: float32 29, 8 42
        // and 137; 96, 4 115 and 118; 64, 16 138 and 117; 33, 32 242 and 140; float16 160, 4 113 and 130;
        // 192, 1 178 and 130; 205, 16 147 and 156; 251, 4 130 and 202; 256, 64 688 and 165.  Over 210 such
        // pairs the choice took 1.6 % (loss alone) and 3 % more than the better one.  It is the same with and
        // without a gradient, and so are the loss's bits.
        const int most = (size_t)V * es % 16 ? 384 : 248;
        if (short_rows(logits, V, es) && V + 8 * k <= most) {
            const ShortBatch sb = short_batch(V, es, (size_t)128 * k);
            const size_t shared = (size_t)sb.warp_bytes * (kShortThreads / 32);
            k_distill_short<T>
                <<<short_grid(k_distill_short<T>, rows, shared), kShortThreads, shared, st>>>(p, sb);
            return;
        }
        const Shape s = shape_of(logits, rows, V, es, sizeof(DistillScratch<32>),
                                 sizeof(DistillScratch<kBlockThreads>));
        if (s.group)
            distill_form<T>(s.group, (int)(s.ring.stage_bytes / 16), k, (size_t)V * es % 16 == 0,
                            [&](auto kernel, int th) {
                                kernel<<<grid_of(s, kernel, th), th, s.shared, st>>>(p, s.ring);
                                return 0;
                            });
        else
            k_distill_long<T><<<row_grid(rows), kLongThreads, (size_t)(V + 31) / 32 * 4, st>>>(p);
    });
    if (launched() != RNNT_OK) return RNNT_LAUNCH_FAILED;
    if (!launch_after(k_distill_sum, dim3((unsigned)B * (unsigned)p.splits), kSumThreads, 0, st, p)) {
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
