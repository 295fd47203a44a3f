// rnnt_embed.cu -- label embedding (lookup with scaling) and its gradient.
//
// Positions: B sequences of P = S + has_start places.  Place 0 holds the start
// symbol when has_start, place has_start + j holds tokens[b, j]; places whose
// token is negative, or lies at or past lengths[b], are padding.
//   forward   out[b, p, :] = round(scale * weight[tok(b, p), :]), padding 0
//   gradient  grad_weight[v, :] = round(scale * sum over places with tok = v of
//             grad_out[b, p, :]), in float32 sums of a fixed order
#include <cooperative_groups.h>

#include <atomic>

#include "rnnt_labels.cuh"

namespace cg = cooperative_groups;
using namespace rnnt_labels;

namespace {

constexpr int32_t kMaxWidth = 1 << 24;    // of a row: keeps unit numbers in 32 bits

struct Places {
    const int32_t* tokens;
    int64_t stride;
    const int32_t* lengths;   // or null: all S tokens count
    int32_t B, S, first, start, V;
};

// The id at place i (row-major over (B, P)), -1 for padding; `bad` is set for
// an id that is no row of the table and a length outside [0, S].
__device__ __forceinline__ int place_id(const Places& p, int64_t i, bool& bad) {
    const int P = p.S + p.first;
    const int64_t b = i / P;
    const int j = (int)(i - b * P) - p.first;
    if (j < 0) return p.start;
    if (p.lengths) {
        const int n = __ldg(p.lengths + b);
        bad |= n < 0 || n > p.S;
        if (j >= n) return -1;
    }
    const int t = __ldg(p.tokens + b * p.stride + j);
    bad |= t >= p.V;
    return t < 0 || t >= p.V ? -1 : t;
}

// ------------------------------------------------------------------ forward
constexpr int kEmbedThreads = 256;
constexpr int kEmbedUnits = 4;                               // units a thread has in flight
constexpr int kEmbedTile = kEmbedThreads * kEmbedUnits;      // units of a CTA

struct EmbedParams {
    Places pl;
    const char* weight;
    int64_t weight_stride;   // bytes
    char* out;
    int64_t N;               // places
    int32_t nunits;          // units of a row
    int32_t rows;            // rows of a CTA
    int32_t pieces;          // CTAs of a row that is longer than a CTA's tile
    uint32_t inv;            // ceil(2^32 / nunits): u / nunits = (u * inv) >> 32 for u < kEmbedTile
    float scale;
    int32_t* status;
};

// A CTA writes kEmbedTile units: several short rows, or a piece of a long one.
template <typename T, int UB>
__global__ void __launch_bounds__(kEmbedThreads) k_embed(const EmbedParams p) {
    using U = typename Unit<UB>::type;
    constexpr int E = UB / (int)sizeof(T);
    __shared__ int ids[kEmbedThreads];
    const int64_t tile = blockIdx.x / p.pieces;
    const int piece = (int)(blockIdx.x - tile * p.pieces);
    const int64_t row0 = tile * p.rows;
    const int rows = (int)min((int64_t)p.rows, p.N - row0);
    if (threadIdx.x < rows) {
        bool bad = false;
        ids[threadIdx.x] = place_id(p.pl, row0 + threadIdx.x, bad);
        if (bad && p.status) *p.status = RNNT_INVALID_VALUE;
    }
    __syncthreads();
    const int u0 = piece * kEmbedTile;
    const int total = p.pieces > 1 ? p.nunits : rows * p.nunits;
    U* out = reinterpret_cast<U*>(p.out) + row0 * p.nunits;
    Pack<T, UB> v[kEmbedUnits];
    bool some[kEmbedUnits];
#pragma unroll
    for (int i = 0; i < kEmbedUnits; ++i) {
        const int u = u0 + threadIdx.x + i * kEmbedThreads;
        some[i] = false;
        if (u < total) {
            const int r = p.rows == 1 ? 0 : p.nunits == 1 ? u : (int)__umulhi((uint32_t)u, p.inv);
            const int id = ids[r];
            some[i] = id >= 0;
            if (id >= 0)
                v[i].raw = __ldg(reinterpret_cast<const U*>(p.weight + id * p.weight_stride) +
                                 (u - r * p.nunits));
        }
    }
#pragma unroll
    for (int i = 0; i < kEmbedUnits; ++i) {
        const int u = u0 + threadIdx.x + i * kEmbedThreads;
        if (u >= total) break;
        Pack<T, UB> o;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o.e[e] = from_f32<T>(some[i] ? to_f32(v[i].e[e]) * p.scale : 0.0f);
        out[u] = o.raw;
    }
}

// ----------------------------------------------------- gradient: sorted places
// One cluster sorts the places by id (stable, so places of an id stay in
// order): least-significant-digit radix sort, one to three digits of up to 11
// bits.  A CTA owns a contiguous range of the input; per digit it counts its
// range, the CTAs exchange counts through distributed shared memory, and each
// writes its places behind those of smaller digits and of earlier CTAs.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 8;                             // places of a thread and chunk
constexpr int kSortChunk = kSortThreads * kSortItems;
constexpr int kMaxBits = 11;
constexpr int kMaxBins = 1 << kMaxBits;

struct SortParams {
    Places pl;
    int64_t N;
    int32_t bits, passes;      // digits of `bits` bits
    int32_t* key[2];           // pass i writes key[i & 1] / place[i & 1]
    int32_t* place[2];
    uint8_t* present;          // [V]: id occurs
    int32_t* count;            // places that are not padding
    int32_t* status;
};

constexpr size_t kSortShared = sizeof(uint16_t) * kSortWarps * kMaxBins;

__global__ void __launch_bounds__(kSortThreads) k_sort(const SortParams p) {
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ uint16_t wh[];          // [warp][bin]: counts, then starts
    __shared__ int32_t total[kMaxBins];       // this CTA's count of each digit
    __shared__ int32_t base[kMaxBins];        // where its next place of a digit goes
    __shared__ int32_t chunk[kMaxBins];       // the current chunk's count of each digit
    __shared__ int32_t scan[kSortWarps];
    const int bins = 1 << p.bits;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();

    for (int64_t v = rank * kSortThreads + tid; v < p.pl.V; v += (int64_t)C * kSortThreads)
        p.present[v] = 0;

    int64_t n = p.N;
    for (int pass = 0; pass < p.passes; ++pass) {
        const bool last = pass + 1 == p.passes;
        const int shift = pass * p.bits;
        const int64_t per = (n + C - 1) / C;
        const int64_t lo = min(n, per * rank), hi = min(n, lo + per);
        int key[kSortItems], place[kSortItems];
        int ahead[kSortItems];                // places of the same warp and digit ahead
        // The chunk at c0: its items, their order within the warp, the warp's counts.
        auto rank_chunk = [&](int64_t c0) {
            __syncthreads();                  // readers of the previous counts are done
            for (int i = tid; i < bins * kSortWarps / 2; i += kSortThreads)
                reinterpret_cast<uint32_t*>(wh)[i] = 0;
            __syncthreads();
            uint16_t* mine = wh + warp * bins;
#pragma unroll
            for (int i = 0; i < kSortItems; ++i) {
                const int64_t at = c0 + warp * (32 * kSortItems) + i * 32 + lane;
                key[i] = -1;
                place[i] = (int)at;
                if (at < hi) {
                    if (pass == 0) {
                        bool bad = false;
                        key[i] = place_id(p.pl, at, bad);
                        if (bad && p.status) *p.status = RNNT_INVALID_VALUE;
                    } else {
                        key[i] = __ldcg(p.key[(pass & 1) ^ 1] + at);
                        place[i] = __ldcg(p.place[(pass & 1) ^ 1] + at);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kSortItems; ++i) {
                const int d = (key[i] >> shift) & (bins - 1);
                const unsigned same = __match_any_sync(0xffffffffu, key[i] < 0 ? -1 : d);
                const int before = mine[d];
                ahead[i] = before + __popc(same & ((1u << lane) - 1));
                __syncwarp();
                if (key[i] >= 0 && lane == __ffs(same) - 1)
                    mine[d] = (uint16_t)(before + __popc(same));
                __syncwarp();
            }
            __syncthreads();
        };
        for (int b = tid; b < bins; b += kSortThreads) total[b] = 0;
        for (int64_t c0 = lo; c0 < hi; c0 += kSortChunk) {
            rank_chunk(c0);
            for (int b = tid; b < bins; b += kSortThreads) {
                int s = 0;
                for (int w = 0; w < kSortWarps; ++w) s += wh[w * bins + b];
                total[b] += s;
            }
        }
        cluster.sync();
        // base[b] = places of smaller digits + places of digit b in earlier CTAs.
        int all[kMaxBins / kSortThreads], mineb[kMaxBins / kSortThreads];
        int sum = 0;
#pragma unroll
        for (int q = 0; q < kMaxBins / kSortThreads; ++q) {
            const int b = tid * (kMaxBins / kSortThreads) + q;
            all[q] = mineb[q] = 0;
            if (b < bins)
                for (int r = 0; r < C; ++r) {
                    const int c = *cluster.map_shared_rank(total + b, r);
                    if (r < rank) mineb[q] += c;
                    all[q] += c;
                }
            sum += all[q];
        }
        int incl = sum;
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        int off = 0, full = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            if (w < warp) off += scan[w];
            full += scan[w];
        }
        off += incl - sum;
#pragma unroll
        for (int q = 0; q < kMaxBins / kSortThreads; ++q) {
            const int b = tid * (kMaxBins / kSortThreads) + q;
            if (b < bins) base[b] = off + mineb[q];
            off += all[q];
        }
        if (rank == 0 && tid == 0 && pass == 0) *p.count = full;
        for (int64_t c0 = lo; c0 < hi; c0 += kSortChunk) {
            if (hi - lo > kSortChunk) rank_chunk(c0);     // one chunk: still at hand
            __syncthreads();
            for (int b = tid; b < bins; b += kSortThreads) {
                int s = 0;
                for (int w = 0; w < kSortWarps; ++w) {
                    const int c = wh[w * bins + b];
                    wh[w * bins + b] = (uint16_t)s;
                    s += c;
                }
                chunk[b] = s;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kSortItems; ++i) {
                if (key[i] < 0) continue;
                const int d = (key[i] >> shift) & (bins - 1);
                const int to = base[d] + wh[warp * bins + d] + ahead[i];
                p.key[pass & 1][to] = key[i];
                p.place[pass & 1][to] = place[i];
                if (last) p.present[key[i]] = 1;
            }
            __syncthreads();
            for (int b = tid; b < bins; b += kSortThreads) base[b] += chunk[b];
        }
        n = full;
        cluster.sync();
    }
}

// -------------------------------------------------- gradient: sums of sorted rows
// The sorted places are cut into tiles of kTile; a group of threads adds a
// tile's rows, one unit of columns a thread, and stores each id that begins
// and ends inside its tile.  The rows of an id that crosses tiles go as
// float32 partial sums to the workspace (slot 0: begun in an earlier tile,
// slot 1: goes on in a later one), which k_join adds in order.
constexpr int kTile = 32;
constexpr int kSumThreads = 128;
constexpr int kAhead = 8;                 // rows a thread has in flight
constexpr int kZeroRows = 64;             // ids of a CTA that zeroes the rows of absent ids

struct SumParams {
    const char* grad_out;
    char* grad_weight;
    const int32_t* key;
    const int32_t* place;
    const uint8_t* present;
    const int32_t* count;
    float* partial;          // [tile][2][D]
    int64_t tiles;           // upper bound: tiles of all places
    int32_t V, D, nunits, group;   // group: threads of a tile, a power of two
    float scale;
    unsigned sum_ctas;       // CTAs that add; the others zero
};

template <typename T, int UB>
__device__ __forceinline__ void store_row_unit(const SumParams& p, int64_t id, int unit,
                                               const float* acc) {
    constexpr int E = UB / (int)sizeof(T);
    Pack<T, UB> o;
#pragma unroll
    for (int e = 0; e < E; ++e) o.e[e] = from_f32<T>(acc[e] * p.scale);
    reinterpret_cast<typename Unit<UB>::type*>(p.grad_weight)[id * p.nunits + unit] = o.raw;
}

template <typename T, int UB>
__global__ void __launch_bounds__(kSumThreads) k_sum(const SumParams p) {
    using U = typename Unit<UB>::type;
    constexpr int E = UB / (int)sizeof(T);
    if (blockIdx.x >= p.sum_ctas) {
        const int64_t v0 = (int64_t)(blockIdx.x - p.sum_ctas) * kZeroRows;
        const int n = (int)min((int64_t)kZeroRows, p.V - v0);
        Pack<T, UB> zero;
#pragma unroll
        for (int e = 0; e < E; ++e) zero.e[e] = from_f32<T>(0.0f);
        __shared__ uint8_t present[kZeroRows];
        if (threadIdx.x < n) present[threadIdx.x] = p.present[v0 + threadIdx.x];
        __syncthreads();
        for (int r = 0; r < n; ++r) {
            if (present[r]) continue;
            U* row = reinterpret_cast<U*>(p.grad_weight) + (v0 + r) * p.nunits;
            for (int u = blockIdx.y * kSumThreads + threadIdx.x; u < p.nunits;
                 u += gridDim.y * kSumThreads)
                row[u] = zero.raw;
        }
        return;
    }
    const int g = threadIdx.x / p.group, groups = kSumThreads / p.group;
    const int64_t t = (int64_t)blockIdx.x * groups + g;
    const int unit = blockIdx.y * p.group + (threadIdx.x & (p.group - 1));
    const int64_t n = *p.count, j0 = t * kTile;
    if (j0 >= n || unit >= p.nunits) return;
    const int cnt = (int)min((int64_t)kTile, n - j0);
    float acc[E] = {};
    int cur = p.key[j0];
    bool head = j0 > 0 && p.key[j0 - 1] == cur;
    float* part = p.partial + t * 2 * p.D + unit * E;
    const U* src = reinterpret_cast<const U*>(p.grad_out) + unit;
    for (int j = 0; j < cnt; j += kAhead) {
        Pack<T, UB> v[kAhead];
        int next[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (j + i < cnt) {
                v[i].raw = __ldg(src + (int64_t)p.place[j0 + j + i] * p.nunits);
                next[i] = j0 + j + i + 1 < n ? p.key[j0 + j + i + 1] : -1;
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (j + i >= cnt) break;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += to_f32(v[i].e[e]);
            if (next[i] != cur || j + i + 1 == cnt) {
                const bool ends = next[i] != cur;
                if (head || !ends) {
                    float* to = part + (head ? 0 : p.D);
#pragma unroll
                    for (int e = 0; e < E; ++e) to[e] = acc[e];
                } else {
                    store_row_unit<T, UB>(p, cur, unit, acc);
                }
                head = false;
                cur = next[i];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = 0.0f;
            }
        }
    }
}

// The id that begins in tile t and goes on: its partial sums, tile after tile.
template <typename T, int UB>
__global__ void __launch_bounds__(kSumThreads) k_join(const SumParams p) {
    constexpr int E = UB / (int)sizeof(T);
    const int g = threadIdx.x / p.group, groups = kSumThreads / p.group;
    int64_t t = (int64_t)blockIdx.x * groups + g;
    const int unit = blockIdx.y * p.group + (threadIdx.x & (p.group - 1));
    const int64_t n = *p.count;
    if ((t + 1) * kTile >= n || unit >= p.nunits) return;    // no later tile
    const int id = p.key[(t + 1) * kTile - 1];
    if (p.key[(t + 1) * kTile] != id || (t > 0 && p.key[t * kTile - 1] == id)) return;
    float acc[E];
    const float* part = p.partial + unit * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = part[(t * 2 + 1) * p.D + e];
    do {
        ++t;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += part[t * 2 * p.D + e];
    } while ((t + 1) * kTile < n && p.key[(t + 1) * kTile] == id);
    store_row_unit<T, UB>(p, id, unit, acc);
}

// Calls f(T{}, unit) with the unit's width as a constant; units are never
// narrower than an element.
template <typename F>
void with_unit(int dt, int unit, F&& f) {
    with_type(dt, [&](auto tag) {
        using T = decltype(tag);
        if (unit >= 16) f(tag, std::integral_constant<int, 16>{});
        else if (unit == 8) f(tag, std::integral_constant<int, 8>{});
        else if (unit == 4 || sizeof(T) == 4) f(tag, std::integral_constant<int, 4>{});
        else f(tag, std::integral_constant<int, sizeof(T) == 4 ? 4 : 2>{});
        return 0;
    });
}

bool places_ok(const Places& p) {
    return p.B >= 1 && p.S >= 0 && p.S < INT32_MAX && p.S + p.first >= 1 && p.V >= 1 &&
           (p.S == 0 || (p.tokens && p.stride >= p.S)) &&
           (!p.first || (p.start >= 0 && p.start < p.V)) &&
           (int64_t)p.B * (p.S + p.first) <= INT32_MAX;
}

// k_sort's shared memory limit, raised once per device.
bool sort_prepared() {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return false;
    if (done[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(k_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kSortShared) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    done[dev].store(true, std::memory_order_release);
    return true;
}

struct GradLayout {
    size_t key[2], place[2], present, count, partial, total;
    int64_t tiles;
};
GradLayout grad_layout(int64_t N, int32_t V, int32_t D) {
    GradLayout L;
    size_t at = 0;
    for (int i = 0; i < 2; ++i) {
        L.key[i] = at;   at = align256(at + sizeof(int32_t) * (size_t)N);
        L.place[i] = at; at = align256(at + sizeof(int32_t) * (size_t)N);
    }
    L.present = at; at = align256(at + (size_t)V);
    L.count = at;   at = align256(at + sizeof(int32_t));
    L.tiles = (N + kTile - 1) / kTile;
    L.partial = at; at = align256(at + sizeof(float) * 2 * (size_t)L.tiles * (size_t)D);
    L.total = at;
    return L;
}

}  // namespace

extern "C" rnnt_status_t rnnt_embed(const void* weight, rnnt_dtype_t dt, int32_t V, int32_t D,
                                    int64_t weight_stride, const int32_t* tokens,
                                    int64_t tokens_stride, const int32_t* lengths, int32_t B,
                                    int32_t S, int32_t has_start, int32_t start, float scale,
                                    void* out, int32_t* status_dev, rnnt_stream_t stream) {
    if (!weight || !out || !valid_dtype(dt) || V < 1 || D < 1 || D > kMaxWidth ||
        weight_stride < D)
        return RNNT_INVALID_VALUE;
    Places pl{tokens, tokens_stride, lengths, B, S, has_start ? 1 : 0,
              start < 0 ? start + V : start, V};
    if (!places_ok(pl) || !(scale == scale)) return RNNT_INVALID_VALUE;
    const int es = elem_size(dt);
    const int64_t N = (int64_t)B * (S + pl.first);
    if (((uintptr_t)weight | (uintptr_t)out) & (es - 1)) return RNNT_INVALID_VALUE;
    if (overlaps(weight, ((uint64_t)(V - 1) * weight_stride + D) * es, out, (uint64_t)N * D * es))
        return RNNT_INVALID_VALUE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int unit = unit_of((uintptr_t)weight | (uintptr_t)out | (uint64_t)weight_stride * es |
                             (uint64_t)D * es);
    EmbedParams p{};
    p.pl = pl;
    p.weight = static_cast<const char*>(weight);
    p.weight_stride = weight_stride * es;
    p.out = static_cast<char*>(out);
    p.N = N;
    p.nunits = (int32_t)((int64_t)D * es / unit);
    p.rows = std::max(1, std::min(kEmbedThreads, kEmbedTile / p.nunits));
    p.pieces = (int32_t)((p.nunits + (int64_t)kEmbedTile - 1) / kEmbedTile);
    p.inv = (uint32_t)(((1ull << 32) + p.nunits - 1) / p.nunits);
    p.scale = scale;
    p.status = status_dev;
    const int64_t grid = (N + p.rows - 1) / p.rows * p.pieces;
    if (grid > INT32_MAX) return RNNT_INVALID_VALUE;
    if (!clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    with_unit(dt, unit, [&](auto tag, auto ub) {
        k_embed<decltype(tag), decltype(ub)::value>
            <<<(unsigned)grid, kEmbedThreads, 0, st>>>(p);
    });
    return launched();
}

extern "C" rnnt_status_t rnnt_embed_grad_workspace_size(int32_t B, int32_t S, int32_t has_start,
                                                        int32_t V, int32_t D, size_t* bytes) {
    const int first = has_start ? 1 : 0;
    if (!bytes || B < 1 || S < 0 || S == INT32_MAX || S + first < 1 || V < 1 || D < 1 ||
        D > kMaxWidth ||        (int64_t)B * (S + first) > INT32_MAX)
        return RNNT_INVALID_VALUE;
    *bytes = grad_layout((int64_t)B * (S + first), V, D).total;
    return RNNT_OK;
}

extern "C" rnnt_status_t rnnt_embed_grad(const void* grad_out, rnnt_dtype_t dt,
                                         const int32_t* tokens, int64_t tokens_stride,
                                         const int32_t* lengths, int32_t B, int32_t S,
                                         int32_t has_start, int32_t start, int32_t V, int32_t D,
                                         float scale, void* grad_weight, void* workspace,
                                         size_t workspace_bytes, int32_t* status_dev,
                                         rnnt_stream_t stream) {
    if (!grad_out || !grad_weight || !workspace || !valid_dtype(dt) || V < 1 || D < 1 ||
        D > kMaxWidth)
        return RNNT_INVALID_VALUE;
    Places pl{tokens, tokens_stride, lengths, B, S, has_start ? 1 : 0,
              start < 0 ? start + V : start, V};
    if (!places_ok(pl) || !(scale == scale)) return RNNT_INVALID_VALUE;
    const int es = elem_size(dt);
    const int64_t N = (int64_t)B * (S + pl.first);
    if ((((uintptr_t)grad_out | (uintptr_t)grad_weight) & (es - 1)) || ((uintptr_t)workspace & 255))
        return RNNT_INVALID_VALUE;
    if (overlaps(grad_out, (uint64_t)N * D * es, grad_weight, (uint64_t)V * D * es))
        return RNNT_INVALID_VALUE;
    const GradLayout L = grad_layout(N, V, D);
    if (workspace_bytes < L.total) return RNNT_WORKSPACE_TOO_SMALL;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);

    SortParams s{};
    s.pl = pl;
    s.N = N;
    int k = 1;
    while (k < 31 && ((int64_t)1 << k) < V) ++k;
    s.passes = (k + kMaxBits - 1) / kMaxBits;
    s.bits = (k + s.passes - 1) / s.passes;
    for (int i = 0; i < 2; ++i) {
        s.key[i] = reinterpret_cast<int32_t*>(ws + L.key[i]);
        s.place[i] = reinterpret_cast<int32_t*>(ws + L.place[i]);
    }
    s.present = reinterpret_cast<uint8_t*>(ws + L.present);
    s.count = reinterpret_cast<int32_t*>(ws + L.count);
    s.status = status_dev;
    SumParams q{};
    const int unit = unit_of((uintptr_t)grad_out | (uintptr_t)grad_weight | (uint64_t)D * es);
    q.grad_out = static_cast<const char*>(grad_out);
    q.grad_weight = static_cast<char*>(grad_weight);
    q.key = s.key[(s.passes - 1) & 1];
    q.place = s.place[(s.passes - 1) & 1];
    q.present = s.present;
    q.count = s.count;
    q.partial = reinterpret_cast<float*>(ws + L.partial);
    q.tiles = L.tiles;
    q.V = V;
    q.D = D;
    q.nunits = (int32_t)((int64_t)D * es / unit);
    q.group = 1;
    while (q.group < kSumThreads && q.group < q.nunits) q.group *= 2;
    q.scale = scale;
    const int groups = kSumThreads / q.group;
    q.sum_ctas = (unsigned)((L.tiles + groups - 1) / groups);
    const unsigned zero_ctas = (unsigned)(((int64_t)V + kZeroRows - 1) / kZeroRows);
    const unsigned cols = (unsigned)((q.nunits + q.group - 1) / q.group);
    if (cols > 65535 || (uint64_t)q.sum_ctas + zero_ctas > INT32_MAX) return RNNT_INVALID_VALUE;

    if (!clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    const size_t shared = sizeof(uint16_t) * kSortWarps * ((size_t)1 << s.bits);
    if (!sort_prepared()) return RNNT_LAUNCH_FAILED;
    int C = 1;
    while (C < 8 && (int64_t)C * kSortChunk < N) C *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_sort, s) != cudaSuccess) {
        cudaGetLastError();
        return RNNT_LAUNCH_FAILED;
    }
    with_unit(dt, unit, [&](auto tag, auto ub) {
        k_sum<decltype(tag), decltype(ub)::value>
            <<<dim3(q.sum_ctas + zero_ctas, cols), kSumThreads, 0, st>>>(q);
        if (L.tiles > 1)
            k_join<decltype(tag), decltype(ub)::value>
                <<<dim3(q.sum_ctas, cols), kSumThreads, 0, st>>>(q);
    });
    return launched();
}
