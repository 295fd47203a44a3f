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

constexpr int32_t kMaxWidth = 1 << 20;    // of a row: column slices fit a grid's second axis

struct Places {
    const int32_t* tokens;
    int64_t stride;
    const int32_t* lengths;   // or null: all S tokens count
    int32_t B, S, first, start, V;
};

// The ids at I places (row-major over (B, P)), -1 for padding and from place `end` on; `bad` is
// set for an id that is no row of the table and a length outside [0, S].  The I lengths are
// asked for together, then the I tokens.
template <int I>
__device__ __forceinline__ void place_ids(const Places& p, const uint32_t* place, uint32_t end,
                                          int* id, bool& bad) {
    const uint32_t P = (uint32_t)p.S + (uint32_t)p.first;
    uint32_t b[I];
    int j[I], n[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        b[i] = place[i] / P;
        j[i] = (int)(place[i] - b[i] * P) - p.first;
        n[i] = p.S;
        // where S = 0 no place but the start symbol's sees a length
        if (p.lengths && place[i] < end && (j[i] >= 0 || p.S == 0)) n[i] = __ldg(p.lengths + b[i]);
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
        bad |= n[i] < 0 || n[i] > p.S;
        id[i] = -1;
        if (place[i] < end && j[i] < min(max(n[i], 0), p.S))
            id[i] = j[i] < 0 ? p.start : __ldg(p.tokens + (int64_t)b[i] * p.stride + j[i]);
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
        bad |= id[i] >= p.V;
        if (id[i] < 0 || id[i] >= p.V) id[i] = -1;
    }
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

// A CTA writes kEmbedTile units: several short rows, or a piece of a long one.  It looks its rows'
// ids up once, a row a thread, and then has four units a thread in flight.  Bound by writing:
// 64 x 1023 places of 1024 bfloat16 out of 50000 rows, 134 MB written and 24 MB read, take
// 28 us (5.6 TB/s); fewer and more units a thread, and streaming stores, measured the same or
// slower.  Four rows take 1.8 us in a graph, a launch's time.
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
        const uint32_t place = (uint32_t)row0 + threadIdx.x;
        place_ids<1>(p.pl, &place, (uint32_t)p.N, ids + threadIdx.x, bad);
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
// order): least-significant-digit radix sort, one to four digits of up to 10
// bits.  A CTA owns a contiguous range of the input; per digit it counts its
// range, the CTAs exchange counts through distributed shared memory, and each
// writes its places, brought into order in shared memory first so that the writes are
// runs, behind those of smaller digits and of earlier CTAs.
//
// Latency bounds it (64000 places of 50000 ids are 0.25 MB to read), so the rest of the
// device spends the time on zeroing grad_weight, whose rows without places k_sum does not
// come to (finding those rows first, so as to zero no others, took 15 us longer than it saved
// for 50000 ids of which a third occur).  65472 places of 50000 ids, two digits of 8 bits: 20 us by
// 16 CTAs without the zeroing, 24 beside the 102 MB of it; 46 with atomics for the counts and
// scattered writes.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 4;                             // places of a thread and chunk, at most
constexpr int kMaxBits = 10;
constexpr int kMaxBins = 1 << kMaxBits;                   // a thread each
constexpr int kMaxCluster = 16;
static_assert(kMaxBins <= kSortThreads, "a digit has a thread");
constexpr int kCountStride = kSortWarps + 2;              // 17 words: neighbouring digits' counts
                                                          // lie in different banks
struct SortParams {
    Places pl;
    int64_t N;
    int32_t bits, passes;      // digits of `bits` bits
    int2* out[2];              // {id, place}: pass i writes out[i & 1]
    int32_t* count;            // places that are not padding
    int32_t* heavy;            // number of long ids, which k_sum lists: set to 0
    int32_t* status;
    char* grad_weight;         // zeroed by the clusters behind the first
    int64_t bytes;
    int32_t unit;
};

// The chunk's places in order, its counts, and every CTA's totals; at least so much that a CTA
// has an SM to itself.
constexpr size_t sort_shared(int bits) {
    return std::max<size_t>(120 << 10, ((sizeof(uint16_t) * kCountStride +
                                             sizeof(int32_t) * kMaxCluster) << bits) +
                                           sizeof(int2) * kSortThreads * kSortItems);
}

template <int UB>
__device__ __forceinline__ void zero_fill(char* at, int64_t bytes, int64_t i, int64_t step) {
    using U = typename Unit<UB>::type;
    for (; i < bytes / UB; i += step) reinterpret_cast<U*>(at)[i] = U{};
}

// x and y become the sums of the earlier threads' x and y; returns the block's sum of x, and of y
// in all_y.
__device__ __forceinline__ int exclusive_scan(int& x, int& y, int& all_y, int2* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 incl = make_int2(x, y);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, incl.x, o);
        const int b = __shfl_up_sync(0xffffffffu, incl.y, o);
        if (lane >= o) {
            incl.x += a;
            incl.y += b;
        }
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int2 upto = scratch[lane];                          // the warps' sums, once more
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, upto.x, o);
        const int b = __shfl_up_sync(0xffffffffu, upto.y, o);
        if (lane >= o) {
            upto.x += a;
            upto.y += b;
        }
    }
    const int before = max(warp, 1) - 1;
    const int bx = __shfl_sync(0xffffffffu, upto.x, before);
    const int by = __shfl_sync(0xffffffffu, upto.y, before);
    x = incl.x - x + (warp ? bx : 0);
    y = incl.y - y + (warp ? by : 0);
    all_y = __shfl_sync(0xffffffffu, upto.y, 31);
    return __shfl_sync(0xffffffffu, upto.x, 31);
}

__global__ void __launch_bounds__(kSortThreads) k_sort(const SortParams p) {
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(16) char sort_space[];
    int2* ordered = reinterpret_cast<int2*>(sort_space);      // the chunk's places
    // [digit][warp], 16 bits: counts, then starts
    uint32_t* counts32 = reinterpret_cast<uint32_t*>(ordered + kSortThreads * kSortItems);
    uint16_t* counts = reinterpret_cast<uint16_t*>(counts32);
    __shared__ int32_t total[kMaxBins];       // this CTA's count of each digit
    __shared__ int32_t base[kMaxBins];        // where its next place of a digit goes
    __shared__ int32_t chunk[kMaxBins];       // the current chunk's count of each digit, and where
    __shared__ int32_t start[kMaxBins];       // the digit starts in `ordered`
    __shared__ int2 scan[kSortWarps];
    static_assert(kSortWarps == 32, "exclusive_scan takes a warp's sums by a warp");
    const int bins = 1 << p.bits;
    int32_t* given = reinterpret_cast<int32_t*>(counts32 + bins * kCountStride / 2);   // [CTA][digit]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    if ((int)blockIdx.x >= C) {
        const int64_t i = (int64_t)(blockIdx.x - C) * kSortThreads + tid;
        const int64_t step = (int64_t)(gridDim.x - C) * kSortThreads;
        if (p.unit == 16) zero_fill<16>(p.grad_weight, p.bytes, i, step);
        else if (p.unit >= 4) zero_fill<4>(p.grad_weight, p.bytes, i, step);
        else zero_fill<2>(p.grad_weight, p.bytes, i, step);
        return;
    }
    cluster.barrier_arrive();

    uint32_t n = (uint32_t)p.N;
    for (int pass = 0; pass < p.passes; ++pass) {
        const bool last = pass + 1 == p.passes;
        const int shift = pass * p.bits;
        const uint32_t per = (n + C - 1) / C;
        const uint32_t lo = min(n, per * rank), hi = min(n, lo + per);
        // a warp's places are adjacent: 32 * items of them
        const int items = (int)min((uint32_t)kSortItems, (hi - lo + kSortThreads - 1) / kSortThreads);
        const uint32_t step = (uint32_t)items * kSortThreads;
        const int2* in = pass & 1 ? p.out[0] : p.out[1];
        int key[kSortItems], ahead[kSortItems];     // ahead: places of the same warp and digit
        uint32_t place[kSortItems];                 // ahead of it
        // The chunk at c0: its items, their order within the warp, per digit the warps'
        // starts and the count.
        auto rank_chunk = [&](uint32_t c0) {
            __syncthreads();                        // readers of the previous counts are done
            for (int i = tid; i < bins * kCountStride / 2; i += kSortThreads) counts32[i] = 0;
            __syncthreads();
            const uint32_t at = c0 + warp * 32 * items + lane;
#pragma unroll
            for (int i = 0; i < kSortItems; ++i) {
                place[i] = at + i * 32;
                key[i] = -1;
            }
            if (pass == 0) {
                bool bad = false;
                place_ids<kSortItems>(p.pl, place, min(hi, at - lane + 32 * items), key, bad);
                if (bad && p.status) *p.status = RNNT_INVALID_VALUE;
            } else {
#pragma unroll
                for (int i = 0; i < kSortItems; ++i)
                    if (i < items && place[i] < hi) {
                        const int2 v = __ldcg(in + place[i]);
                        key[i] = v.x;
                        place[i] = (uint32_t)v.y;
                    }
            }
#pragma unroll
            for (int i = 0; i < kSortItems; ++i) {
                if (i >= items) break;
                const int d = (key[i] >> shift) & (bins - 1);
                unsigned same = __ballot_sync(0xffffffffu, key[i] >= 0);
                for (int bit = 0; bit < p.bits; ++bit) {
                    const bool one = d >> bit & 1;
                    const unsigned ones = __ballot_sync(0xffffffffu, one);
                    same &= one ? ones : ~ones;
                }
                uint16_t* mine = counts + d * kCountStride + warp;
                const int before = key[i] >= 0 ? *mine : 0;
                ahead[i] = before + __popc(same & ((1u << lane) - 1));
                __syncwarp();
                if (key[i] >= 0 && lane == __ffs(same) - 1)
                    *mine = (uint16_t)(before + __popc(same));
                __syncwarp();
            }
            __syncthreads();
            for (int b = tid; b < bins; b += kSortThreads) {
                uint32_t* row = counts32 + b * (kCountStride / 2);
                uint32_t c[kSortWarps / 2], s = 0;
#pragma unroll
                for (int w = 0; w < kSortWarps / 2; ++w) c[w] = row[w];
#pragma unroll
                for (int w = 0; w < kSortWarps / 2; ++w) {
                    const uint32_t a = c[w] & 0xffffu, z = c[w] >> 16;
                    row[w] = s | (s + a) << 16;
                    s += a + z;
                }
                chunk[b] = (int)s;
            }
            __syncthreads();
        };
        for (int b = tid; b < bins; b += kSortThreads) total[b] = 0;
        for (uint32_t c0 = lo; c0 < hi; c0 += step) {
            rank_chunk(c0);
            for (int b = tid; b < bins; b += kSortThreads) total[b] += chunk[b];
        }
        __syncthreads();
        if (pass == 0) cluster.barrier_wait();          // every CTA has started
        // Every CTA hands its counts to the others.  base[b] = places of smaller digits, and of
        // digit b in earlier CTAs; start[b] likewise within the first chunk.
        for (int i = tid; i < bins * C; i += kSortThreads) {
            const int r = i >> p.bits, b = i & (bins - 1);
            *cluster.map_shared_rank(given + rank * bins + b, r) = total[b];
        }
        cluster.sync();
        int all = 0, ours = 0, held = 0, first = 0;
        if (tid < bins) {
            for (int r = 0; r < C; ++r) {
                const int c = given[r * bins + tid];
                if (r < rank) ours += c;
                all += c;
            }
            first = lo < hi ? chunk[tid] : 0;
        }
        const int full = exclusive_scan(all, first, held, scan);
        if (tid < bins) {
            base[tid] = all + ours;
            start[tid] = first;
        }
        if (rank == 0 && tid == 0 && pass == 0) {
            *p.count = full;
            *p.heavy = 0;
        }
        __syncthreads();
        int2* out = p.out[pass & 1];
        for (uint32_t c0 = lo; c0 < hi; c0 += step) {
            if (hi - lo > step) rank_chunk(c0);         // one chunk: still at hand, with its starts
            if (hi - lo > step) {
                int none = 0;
                first = tid < bins ? chunk[tid] : 0;
                exclusive_scan(none, first, held, scan);
                if (tid < bins) start[tid] = first;
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < kSortItems; ++i) {
                if (i >= items || key[i] < 0) continue;
                const int d = (key[i] >> shift) & (bins - 1);
                ordered[start[d] + counts[d * kCountStride + warp] + ahead[i]] =
                    make_int2(key[i], (int)place[i]);
            }
            __syncthreads();
            for (int i = tid; i < held; i += kSortThreads) {
                const int2 v = ordered[i];
                const int d = (v.x >> shift) & (bins - 1);
                out[base[d] + i - start[d]] = v;
            }
            if (c0 + step < hi) {
                __syncthreads();
                for (int b = tid; b < bins; b += kSortThreads) base[b] += chunk[b];
            }
        }
        n = (uint32_t)full;
        if (!last) cluster.sync();
    }
}

// -------------------------------------------------- gradient: sums of sorted rows
// The sorted places are cut into tiles of kTile; a group of threads adds a tile's rows, one
// unit of columns a thread.  An id belongs to the tile that it begins in: where it ends less
// than kTile places behind that tile its group goes on to its end, and the next tile's
// group begins behind it.  A longer one's rows are added tile by tile, to float32 partial
// sums in the workspace (slot 0 of a tile: begun in an earlier one, slot 1: begun in it),
// which k_join adds in order.
//
// Every row is read once and every id of up to kTile places is written once, by one group, so it
// is bound by memory: 42000 places of 1024 bfloat16 (86 MB) and 16000 ids' rows (34 MB) take 26 us
// (4.7 TB/s, while 22 MB of the sort's zeroes still leave the L2), 3 less than with the rows in
// registers.  Tiles of 16 places make more partial sums than they balance (2 us slower).
constexpr int kTile = 32;
constexpr int kSumThreads = 128;
constexpr int kRing = 8;                  // rows a thread has in flight, a power of two

struct SumParams {
    const char* grad_out;
    char* grad_weight;
    const int2* sorted;      // {id, place}
    const int32_t* count;
    int32_t* heavy;          // number of long ids, then the tiles that they begin in, in no order
    float* partial;          // [tile][2][D]
    int64_t tiles;           // upper bound: tiles of all places
    int32_t V, D, nunits, group;   // group: threads of a tile, a power of two
    float scale;
};

template <typename T, int UB>
__device__ __forceinline__ void store_unit(char* grad_weight, int64_t id, int nunits, int unit,
                                           const float* acc, float scale) {
    constexpr int E = UB / (int)sizeof(T);
    Pack<T, UB> o;
#pragma unroll
    for (int e = 0; e < E; ++e) o.e[e] = from_f32<T>(acc[e] * scale);
    reinterpret_cast<typename Unit<UB>::type*>(grad_weight)[id * nunits + unit] = o.raw;
}

// E float32 sums of a unit, in the workspace.
template <int E>
__device__ __forceinline__ void put_sums(float* to, const float* acc) {
    if constexpr (E % 4 == 0) {
#pragma unroll
        for (int e = 0; e < E; e += 4)
            *reinterpret_cast<float4*>(to + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) to[e] = acc[e];
    }
}
template <int E>
__device__ __forceinline__ void add_sums(const float* from, float* acc) {
    if constexpr (E % 4 == 0) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(from + e);
            acc[e] += v.x;
            acc[e + 1] += v.y;
            acc[e + 2] += v.z;
            acc[e + 3] += v.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += from[e];
    }
}

// One unit from global to shared memory, behind the thread's back: it reads it after
// copies_left lets it (two-byte units, which have no such copy, at once).
template <int UB>
__device__ __forceinline__ void copy_unit(void* to, const void* from) {
    if constexpr (UB == 2) {
        *reinterpret_cast<uint16_t*>(to) = __ldg(reinterpret_cast<const uint16_t*>(from));
    } else if constexpr (UB == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                     :: "r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;"
                     :: "r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "n"(UB) : "memory");
    }
}
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_left() {
    asm volatile("cp.async.wait_group %0;" :: "n"(LEFT) : "memory");
}

template <typename T, int UB>
__global__ void __launch_bounds__(kSumThreads, 12) k_sum(const SumParams p) {
    using U = typename Unit<UB>::type;
    constexpr int E = UB / (int)sizeof(T);
    constexpr int kEntries = 2 * kTile;
    extern __shared__ int2 entries[];              // of each group's tile, and of the next
    const int g = threadIdx.x / p.group, in_group = threadIdx.x & (p.group - 1);
    const int groups = kSumThreads / p.group;
    const int64_t t = (int64_t)blockIdx.x * groups + g;
    const int unit = blockIdx.y * p.group + in_group;
    wait_for_previous();
    let_next_start();
    const int64_t n = *p.count, j0 = t * kTile;
    int2* mine = entries + g * kEntries;
    for (int i = in_group; i < kEntries; i += p.group)
        mine[i] = j0 + i < n ? __ldg(p.sorted + j0 + i) : make_int2(-1, 0);
    int before = -1, before2 = -1;                 // the last ids of the two tiles ahead
    if (j0 > 0 && j0 < n) before = __ldg(&p.sorted[j0 - 1].x);
    if (j0 > kTile && j0 < n) before2 = __ldg(&p.sorted[j0 - kTile - 1].x);
    __syncthreads();
    if (j0 >= n || unit >= p.nunits) return;
    const int last = (int)min((int64_t)kTile, n - j0) - 1;
    int j = 0, end = last + 1;
    bool head = mine[0].x == before;               // the first id began earlier
    if (head && before2 != before && mine[kTile - 1].x != before) {
        while (j < kTile && mine[j].x == before) ++j;        // and ends here: not this tile's
        head = false;
        if (j == end) return;
    }
    // the last id goes on: to its end if that is near (mine[2 kTile - 1] is another's)
    const bool goes_on = mine[last + 1].x == mine[last].x;
    const bool begun_here = !(head && mine[last].x == before);
    if (goes_on && begun_here && mine[kEntries - 1].x != mine[last].x)
        while (mine[end].x == mine[last].x) ++end;
    float acc[E] = {};
    int cur = mine[j].x;
    float* part = p.partial + t * 2 * p.D + unit * E;
    const U* src = reinterpret_cast<const U*>(p.grad_out) + unit;
    // the rows go through a ring in shared memory, a slot a row, each thread its own unit: it
    // waits for its own copies only
    __shared__ U ring[kRing][kSumThreads];
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
        if (j + i < end)
            copy_unit<UB>(&ring[(j + i) & (kRing - 1)][threadIdx.x],
                          src + (int64_t)mine[j + i].y * p.nunits);
        copy_group();
    }
    for (; j < end; ++j) {
        copies_left<kRing - 1>();
        Pack<T, UB> v;
        v.raw = ring[j & (kRing - 1)][threadIdx.x];
        if (j + kRing < end)
            copy_unit<UB>(&ring[j & (kRing - 1)][threadIdx.x],
                          src + (int64_t)mine[j + kRing].y * p.nunits);
        copy_group();
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += to_f32(v.e[e]);
        // the tile's last place may be followed by more of its id, which other tiles add
        const int next = j + 1 < kEntries ? mine[j + 1].x : -1;
        const bool ends = next != cur;
        if (ends || j + 1 == end) {
            if (!head && !ends && unit == 0) p.heavy[1 + atomicAdd(p.heavy, 1)] = (int)t;
            if (head || !ends) put_sums<E>(part + (head ? 0 : p.D), acc);
            else store_unit<T, UB>(p.grad_weight, cur, p.nunits, unit, acc, p.scale);
            head = false;
            cur = next;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        }
    }
}

// The long ids' partial sums, tile after tile.  A CTA takes every gridDim.x-th id and a slice of
// columns.  Ids of up to kShortRun further tiles are a warp's each; the others are the whole
// CTA's, one by one: its groups of threads add stretches of the id's tiles, which are then added
// in order.  Bound by the longest id's chain of additions: 9 us by itself, less behind k_sum's
// end, where the longest of the long ids has 85 tiles; with one stretch an id, 62.  One id at all
// of 65472 places of 512 float16, 2045 tiles: 82 us for the whole gradient (128 with CTAs of 128
// threads).
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kShortRun = 12;
template <typename T, int UB>
__global__ void __launch_bounds__(kJoinThreads) k_join(const SumParams p) {
    constexpr int E = UB / (int)sizeof(T);
    __shared__ float partly[kJoinThreads * E];
    __shared__ int runs[kJoinWarps];
    __shared__ bool is_long[kJoinWarps];
    const int group = min(p.group, 32), groups = kJoinThreads / group;
    const int g = threadIdx.x / group, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_previous();
    const int64_t n = *p.count;
    const int heavy = *p.heavy;
    for (int64_t first = blockIdx.x; first < heavy; first += (int64_t)gridDim.x * kJoinWarps) {
        const int64_t own = first + (int64_t)gridDim.x * warp;
        bool many = false;
        if (own < heavy) {
            const int64_t t = p.heavy[1 + own];
            const int id = p.sorted[(t + 1) * kTile - 1].x;
            // Tiles t + 1 .. t + m hold more of it: the first that ends with another id is the last.
            const int64_t at = (t + 2 + lane) * kTile;             // the tile behind
            const unsigned go = __ballot_sync(0xffffffffu, at < n && p.sorted[at].x == id);
            const int m = go == 0xffffffffu ? 33 : __ffs(~go);
            many = m > kShortRun;
            for (int unit = blockIdx.y * 32 + lane; !many && unit < p.nunits; unit += gridDim.y * 32) {
                const float* part = p.partial + (t + 1) * 2 * p.D + unit * E;
                float acc[E] = {};
                add_sums<E>(part - p.D, acc);                      // of tile t, slot 1
                for (int i0 = 0; i0 < m; i0 += 4) {
                    float next[4][E] = {};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i0 + i < m) add_sums<E>(part + (i0 + i) * 2 * (int64_t)p.D, next[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < E; ++e) acc[e] += next[i][e];
                }
                store_unit<T, UB>(p.grad_weight, id, p.nunits, unit, acc, p.scale);
            }
        }
        __syncthreads();
        if (lane == 0) is_long[warp] = many;
        __syncthreads();
        for (int w = 0; w < kJoinWarps; ++w) {
            if (!is_long[w]) continue;
            const int64_t t = p.heavy[1 + first + (int64_t)gridDim.x * w];
            const int id = p.sorted[(t + 1) * kTile - 1].x;
            int64_t m = 0;
            for (;;) {
                const int64_t at = (t + 2 + m + threadIdx.x) * kTile;
                const unsigned go = __ballot_sync(0xffffffffu, at < n && p.sorted[at].x == id);
                __syncthreads();
                if (lane == 0) runs[warp] = go == 0xffffffffu ? 32 : __ffs(~go) - 1;
                __syncthreads();
                int run = 0;
                for (int i = 0; i < kJoinWarps && run == 32 * i; ++i) run += runs[i];
                m += run < kJoinThreads ? run + 1 : run;
                if (run < kJoinThreads) break;
            }
            const int64_t each = (m + groups - 1) / groups;        // a group's stretch
            for (int u0 = blockIdx.y * group; u0 < p.nunits; u0 += gridDim.y * group) {
                const int unit = u0 + (threadIdx.x & (group - 1));
                float acc[E] = {};
                if (unit < p.nunits) {
                    const float* part = p.partial + (t + 1) * 2 * p.D + unit * E;
                    if (g == 0) add_sums<E>(part - p.D, acc);
                    const int64_t end = min(m, (g + 1) * each);
#pragma unroll 8
                    for (int64_t i = g * each; i < end; ++i) add_sums<E>(part + i * 2 * p.D, acc);
                }
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e) partly[threadIdx.x * E + e] = acc[e];
                __syncthreads();
                if (g == 0 && unit < p.nunits) {
                    for (int i = 1; i < groups; ++i)
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            acc[e] += partly[(i * group + threadIdx.x) * E + e];
                    store_unit<T, UB>(p.grad_weight, id, p.nunits, unit, acc, p.scale);
                }
            }
        }
    }
}

// ------------------------------------------------- gradient: few places, one launch
// With up to kFewPlaces places every CTA looks at all of them.  It takes a range of ids and a
// slice of columns: it collects the places of its ids, sorts them by id (stable) in shared
// memory, gives each group of kFewLanes threads an equal stretch of them to add, joins the sums
// of ids that cross stretches in order, and zeroes the rows of ids without places.
//
// Latency bounds it, and where one id has most places the CTAs that own it: 1312 places of 29
// ids x 301 float32 take 6.7 us in a graph; 2032 places of 512 float16, evenly over 1024 ids, 6.4, all
// of one id 14.5.  Sort, sums and join by three launches took 17 for the first, and take 17 to 20
// for 4096 places, where this takes 8 to 23.  A bitonic sort in the place of the ballots took 5000
// cycles for 23 keys and 46000 for 4080 (18 us of 41).  Slices of 8 units: 1 us slower for even ids, 1
// to 4 faster for one id; of 32: 1 us faster and 5 to 10 slower.
constexpr int kFewPlaces = 4096;
constexpr int kFewBits = 12;              // of a place in a key; the rest is the id's number
constexpr int kFewThreads = 512;
constexpr int kFewLanes = 16;             // units of a CTA's slice of columns
constexpr int kFewGroups = kFewThreads / kFewLanes;
constexpr int kFewIds = 4096;             // ids of a CTA, at most
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewDigit = 6;              // bits of a digit, at most
constexpr int kFewItems = kFewPlaces / kFewThreads;
constexpr int kFewStride = kFewWarps + 1; // of a digit's counts: lanes' digits lie in different banks

struct FewParams {
    Places pl;
    const char* grad_out;
    char* grad_weight;
    int32_t N, ids, nunits, slices;
    int32_t passes, bits;      // of the sort: digits of `bits` bits
    float scale;
    int32_t* status;
};

// A ring of rows, as k_sum's (before it, every other pass's keys); each group's sum of an id that
// began in an earlier stretch; the keys.
template <typename T, int UB>
struct FewShared {
    union {
        typename Unit<UB>::type ring[kRing][kFewThreads];
        uint32_t other[kFewPlaces];
    };
    float partly[kFewGroups][kFewLanes * (UB / (int)sizeof(T))];
    uint32_t key[kFewPlaces];
    uint32_t present[kFewIds / 32];
    int counts[kFewStride << kFewDigit];      // [digit][warp]: counts, then starts
    int sums[kFewWarps];
};

template <typename T, int UB>
__global__ void __launch_bounds__(kFewThreads, 2) k_few(const FewParams p) {
    using U = typename Unit<UB>::type;
    constexpr int E = UB / (int)sizeof(T);
    extern __shared__ __align__(16) char few_space[];
    auto& sh = *reinterpret_cast<FewShared<T, UB>*>(few_space);
    auto& key = sh.key;
    auto& present = sh.present;
    auto& partly = sh.partly;
    auto& ring = sh.ring;
    const int tid = threadIdx.x, lane = tid % kFewLanes, group = tid / kFewLanes;
    const int warp = tid / 32, in_warp = tid & 31;
    const unsigned below = (1u << in_warp) - 1;
    const int range = (int)(blockIdx.x / (unsigned)p.slices);
    const int v0 = range * p.ids, ids = min(p.ids, p.pl.V - v0);
    const int unit = (int)(blockIdx.x - (unsigned)(range * p.slices)) * kFewLanes + lane;
    for (int i = tid; i < (ids + 31) / 32; i += kFewThreads) present[i] = 0;
    // The places of the CTA's ids, in order; the last pass is to end in `key`.
    int n = 0;
    for (int c = 0; c < p.N; c += 4 * kFewThreads) {
        uint32_t* to = p.passes & 1 ? sh.other : key;
        uint32_t place[4];
        int id[4];
        unsigned who[4];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) place[i] = c + (warp * 4 + i) * 32 + in_warp;
        place_ids<4>(p.pl, place, p.N, id, bad);
        if (bad && p.status) *p.status = RNNT_INVALID_VALUE;
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            who[i] = __ballot_sync(0xffffffffu, id[i] >= v0 && id[i] - v0 < ids);
            mine += __popc(who[i]);
        }
        if (in_warp == 0) sh.sums[warp] = mine;
        __syncthreads();
        const int of_warp = in_warp < kFewWarps ? sh.sums[in_warp] : 0;
        int at = n + __reduce_add_sync(0xffffffffu, in_warp < warp ? of_warp : 0);
        n += __reduce_add_sync(0xffffffffu, of_warp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (who[i] >> in_warp & 1)
                to[at + __popc(who[i] & below)] = (uint32_t)(id[i] - v0) << kFewBits | place[i];
            at += __popc(who[i]);
        }
        __syncthreads();
    }
    // Stable radix sort by id.  A warp's keys are adjacent, each one's rank among them by ballots.
    const int per = (n + kFewThreads - 1) / kFewThreads;         // keys of a lane
    for (int pass = 0; pass < p.passes; ++pass) {
        const bool back = (p.passes - pass) & 1;
        const uint32_t* from = back ? sh.other : key;
        uint32_t* to = back ? key : sh.other;
        const int shift = kFewBits + pass * p.bits, bins = 1 << p.bits;
        for (int i = tid; i < bins * kFewStride; i += kFewThreads) sh.counts[i] = 0;
        __syncthreads();
        uint32_t k[kFewItems];
        int ahead[kFewItems];
#pragma unroll
        for (int s = 0; s < kFewItems; ++s) {
            if (s >= per) break;
            const int i = (warp * per + s) * 32 + in_warp;
            k[s] = i < n ? from[i] : 0;
            const int d = (int)(k[s] >> shift) & (bins - 1);
            unsigned same = __ballot_sync(0xffffffffu, i < n);
            for (int bit = 0; bit < p.bits; ++bit) {
                const bool one = d >> bit & 1;
                const unsigned ones = __ballot_sync(0xffffffffu, one);
                same &= one ? ones : ~ones;
            }
            int* count = &sh.counts[d * kFewStride + warp];
            const int before = *count;
            ahead[s] = i < n ? before + __popc(same & below) : -1;
            __syncwarp();
            if (i < n && in_warp == __ffs(same) - 1) *count = before + __popc(same);
            __syncwarp();
        }
        __syncthreads();
        // Each count becomes the sum of those ahead of it, digit by digit and warp by warp: two a
        // thread.
        int* two = &sh.counts[tid / (kFewWarps / 2) * kFewStride + tid % (kFewWarps / 2) * 2];
        const bool some = tid < bins * kFewWarps / 2;
        const int x = some ? two[0] : 0, y = some ? two[1] : 0;
        int upto = x + y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (in_warp >= o) upto += v;
        }
        if (in_warp == 31) sh.sums[warp] = upto;
        __syncthreads();
        const int of_warp = in_warp < kFewWarps ? sh.sums[in_warp] : 0;
        upto += __reduce_add_sync(0xffffffffu, in_warp < warp ? of_warp : 0);
        if (some) {
            two[0] = upto - x - y;
            two[1] = upto - y;
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kFewItems; ++s) {
            if (s >= per) break;
            if (ahead[s] >= 0)
                to[sh.counts[((int)(k[s] >> shift) & (bins - 1)) * kFewStride + warp] + ahead[s]] = k[s];
        }
        __syncthreads();
    }
    for (int i = tid; i < n; i += kFewThreads) {
        const int mine = (int)(key[i] >> kFewBits);
        if (i == 0 || (int)(key[i - 1] >> kFewBits) != mine)
            atomicOr(&present[mine >> 5], 1u << (mine & 31));
    }
    // A group's stretch: ids that begin and end in it are stored, the others' sums kept.
    const int each = (n + kFewGroups - 1) / kFewGroups;
    const int lo = min(n, group * each), hi = min(n, lo + each);
    float acc[E] = {};                       // in the end, of the id that goes on behind hi
    if (unit < p.nunits && lo < hi) {
        const U* src = reinterpret_cast<const U*>(p.grad_out) + unit;
        int cur = (int)(key[lo] >> kFewBits);
        bool head = lo > 0 && (int)(key[lo - 1] >> kFewBits) == cur;
        auto fetch = [&](int j) {
            if (j < hi)
                copy_unit<UB>(&ring[j & (kRing - 1)][tid],
                              src + (int64_t)(key[j] & (kFewPlaces - 1)) * p.nunits);
            copy_group();
        };
#pragma unroll
        for (int i = 0; i < kRing; ++i) fetch(lo + i);
        auto take = [&](int j) {
            copies_left<kRing - 1>();
            Pack<T, UB> v;
            v.raw = ring[j & (kRing - 1)][tid];
            fetch(j + kRing);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += to_f32(v.e[e]);
        };
        for (int j = lo; j < hi; ++j) {
            // eight rows of an id at a time while it goes on behind them, then one by one
            for (; j + 8 < hi && (int)(key[j + 8] >> kFewBits) == cur; j += 8)
#pragma unroll
                for (int i = 0; i < 8; ++i) take(j + i);
            take(j);
            const int next = j + 1 < n ? (int)(key[j + 1] >> kFewBits) : -1;
            if (next != cur || (head && j + 1 == hi)) {
                if (head) {
#pragma unroll
                    for (int e = 0; e < E; ++e) partly[group][lane * E + e] = acc[e];
                } else {
                    store_unit<T, UB>(p.grad_weight, v0 + cur, p.nunits, unit, acc, p.scale);
                }
                head = false;
                cur = next;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = 0.0f;
            }
        }
    }
    __syncthreads();
    if (unit < p.nunits && lo < hi && hi < n) {
        const int id = (int)(key[hi - 1] >> kFewBits);
        const bool begun = lo == 0 || (int)(key[lo - 1] >> kFewBits) != id;
        if (begun && (int)(key[hi] >> kFewBits) == id) {
            for (int w = group + 1; w * each < n && (int)(key[w * each] >> kFewBits) == id; ++w)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += partly[w][lane * E + e];
            store_unit<T, UB>(p.grad_weight, v0 + id, p.nunits, unit, acc, p.scale);
        }
    }
    if (unit < p.nunits) {
        float zero[E] = {};
        for (int r = group; r < ids; r += kFewGroups)
            if (!(present[r >> 5] >> (r & 31) & 1))
                store_unit<T, UB>(p.grad_weight, v0 + r, p.nunits, unit, zero, 1.0f);
    }
}

// k_few's limits, raised once per device.
template <typename T, int UB>
bool few_prepared() {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return false;
    if (done[dev].load(std::memory_order_acquire)) return true;
    const bool ok = cudaFuncSetAttribute(k_few<T, UB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(FewShared<T, UB>)) == cudaSuccess;
    if (ok) done[dev].store(true, std::memory_order_release);
    else cudaGetLastError();
    return ok;
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

// The CTAs of k_sort's largest cluster (16 where the device runs such clusters, else 8) and how
// many of these clusters run at once; size 0 on an error.  k_sort's own limits are raised
// once per device.
struct SortLimits {
    int size, fit;
};
int clusters_of(int size) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sort_shared(kMaxBits);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, k_sort, &cfg) == cudaSuccess ? n : 0;
}
SortLimits sort_limits() {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];           // size << 16 | fit
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return {0, 0};
    int v = known[dev].load(std::memory_order_acquire);
    if (!v) {
        if (cudaFuncSetAttribute(k_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sort_shared(kMaxBits)) == cudaSuccess &&
            cudaFuncSetAttribute(k_sort, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                cudaSuccess) {
            for (int size = 16; size >= 8 && !v; size /= 2)
                if (const int n = clusters_of(size)) v = size << 16 | n;
        }
        cudaGetLastError();
        if (v) known[dev].store(v, std::memory_order_release);
    }
    return {v >> 16, v & 0xffff};
}

struct GradLayout {
    size_t out[2], count, heavy, partial, total;
    int64_t tiles;
};
bool few_places(int64_t N) { return N <= kFewPlaces; }
GradLayout grad_layout(int64_t N, int32_t D) {
    GradLayout L{};
    size_t at = 0;
    if (few_places(N)) return L;             // needs none
    for (int i = 0; i < 2; ++i) {
        L.out[i] = at;
        at = align256(at + sizeof(int2) * (size_t)N);
    }
    L.count = at;   at = align256(at + sizeof(int32_t));
    L.tiles = (N + kTile - 1) / kTile;
    L.heavy = at;   at = align256(at + sizeof(int32_t) * (size_t)(1 + L.tiles));
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
        D > kMaxWidth || (int64_t)B * (S + first) > INT32_MAX)
        return RNNT_INVALID_VALUE;
    *bytes = grad_layout((int64_t)B * (S + first), D).total;
    return RNNT_OK;
}

extern "C" rnnt_status_t rnnt_embed_grad(const void* grad_out, rnnt_dtype_t dt,
                                         const int32_t* tokens, int64_t tokens_stride,
                                         const int32_t* lengths, int32_t B, int32_t S,
                                         int32_t has_start, int32_t start, int32_t V, int32_t D,
                                         float scale, void* grad_weight, void* workspace,
                                         size_t workspace_bytes, int32_t* status_dev,
                                         rnnt_stream_t stream) {
    if (!grad_out || !grad_weight || !valid_dtype(dt) || V < 1 || D < 1 ||
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
    const GradLayout L = grad_layout(N, D);
    if (L.total && !workspace) return RNNT_INVALID_VALUE;
    if (workspace_bytes < L.total) return RNNT_WORKSPACE_TOO_SMALL;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const int unit = unit_of((uintptr_t)grad_out | (uintptr_t)grad_weight | (uint64_t)D * es);
    const int64_t nunits = (int64_t)D * es / unit;
    if (few_places(N)) {
        FewParams f{};
        f.pl = pl;
        f.grad_out = static_cast<const char*>(grad_out);
        f.grad_weight = static_cast<char*>(grad_weight);
        f.N = (int32_t)N;
        f.nunits = (int32_t)nunits;
        f.scale = scale;
        f.status = status_dev;
        const int64_t slices = (nunits + kFewLanes - 1) / kFewLanes;
        // two CTAs an SM, or one an id
        const int64_t ctas = std::max<int64_t>(1, 152 * 2 / slices);
        f.ids = (int32_t)std::min<int64_t>(kFewIds, (V + ctas - 1) / ctas);
        f.slices = (int32_t)slices;
        int bits = 0;
        while (1 << bits < f.ids) ++bits;
        f.passes = (bits + kFewDigit - 1) / kFewDigit;
        f.bits = f.passes ? (bits + f.passes - 1) / f.passes : 0;
        const int64_t grid = ((int64_t)V + f.ids - 1) / f.ids * slices;
        if (grid > INT32_MAX) return RNNT_INVALID_VALUE;
        if (!clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
        bool ok = true;
        with_unit(dt, unit, [&](auto tag, auto ub) {
            using T = decltype(tag);
            constexpr int UB = decltype(ub)::value;
            ok = few_prepared<T, UB>();
            if (ok)
                k_few<T, UB><<<(unsigned)grid, kFewThreads, sizeof(FewShared<T, UB>), st>>>(f);
        });
        return ok ? launched() : RNNT_LAUNCH_FAILED;
    }

    SortParams s{};
    s.pl = pl;
    s.N = N;
    int k = 1;
    while (k < 31 && ((int64_t)1 << k) < V) ++k;
    s.passes = (k + kMaxBits - 1) / kMaxBits;
    s.bits = (k + s.passes - 1) / s.passes;
    for (int i = 0; i < 2; ++i) s.out[i] = reinterpret_cast<int2*>(ws + L.out[i]);
    s.count = reinterpret_cast<int32_t*>(ws + L.count);
    s.status = status_dev;
    SumParams q{};
    q.grad_out = static_cast<const char*>(grad_out);
    q.grad_weight = static_cast<char*>(grad_weight);
    q.sorted = s.out[(s.passes - 1) & 1];
    q.count = s.count;
    q.heavy = s.heavy = reinterpret_cast<int32_t*>(ws + L.heavy);
    q.partial = reinterpret_cast<float*>(ws + L.partial);
    q.tiles = L.tiles;
    q.V = V;
    q.D = D;
    q.nunits = (int32_t)nunits;
    q.group = 4;             // at least: the groups' entries fit shared memory
    while (q.group < kSumThreads && q.group < q.nunits) q.group *= 2;
    q.scale = scale;
    const int groups = kSumThreads / q.group;
    const int64_t sum_ctas = (L.tiles + groups - 1) / groups;
    const unsigned cols = (unsigned)((q.nunits + q.group - 1) / q.group);
    if (sum_ctas > INT32_MAX) return RNNT_INVALID_VALUE;

    if (!clear_status(status_dev, st)) return RNNT_LAUNCH_FAILED;
    s.grad_weight = q.grad_weight;
    s.bytes = (int64_t)V * D * es;
    s.unit = unit >= 16 ? 16 : unit >= 4 ? 4 : 2;
    int C = 1;
    const SortLimits limits = sort_limits();
    if (!limits.size) return RNNT_LAUNCH_FAILED;
    while (C < limits.size && (int64_t)C * kSortThreads < N) C *= 2;
    // The clusters that zero: no more than run beside the first at once (a cluster that has to
    // wait for another's end costs its whole time: 102 MB take 31 us by 8 clusters of 16
    // where 7 fit, 19 by 7).
    const int64_t fit = C == limits.size ? limits.fit : 128 / C;
    const int64_t units = (s.bytes / s.unit + kSortThreads - 1) / kSortThreads;
    const int64_t zero = std::min<int64_t>(std::max<int64_t>(fit - 1, 1), (units + C - 1) / C);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(C * (1 + zero)));
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sort_shared(s.bits);
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
    bool ok = true;
    with_unit(dt, unit, [&](auto tag, auto ub) {
        using T = decltype(tag);
        constexpr int UB = decltype(ub)::value;
        ok = launch_after(k_sum<T, UB>, dim3((unsigned)sum_ctas, cols), kSumThreads,
                          sizeof(int2) * groups * 2 * kTile, st, q) &&
             (L.tiles == 1 ||
              launch_after(k_join<T, UB>,
                           dim3((unsigned)std::min<int64_t>(L.tiles / 2 + 1, 304),
                                std::min(cols * ((unsigned)q.group + 31) / 32, 65535u)),
                           kJoinThreads, 0, st, q));
    });
    if (!ok) {
        cudaGetLastError();
        return RNNT_LAUNCH_FAILED;
    }
    return launched();
}
