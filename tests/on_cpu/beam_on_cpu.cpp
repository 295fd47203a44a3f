// The selection's kernels, compiled from their source for the CPU (device.inc, cut out of
// rnnt_beam.cu), on cases read from standard input: int32 header {dtype, K, V, Ko, fused, splits
// (0: as the host chooses, -1: as it does where the largest cluster has 8 blocks), skip, finished
// given, no minimum}, float scores[K], uint8 finished[K], `skip` elements and the K * V logits.
// Writes int32 {status, found a way out}, float scores[Ko], int32 tokens[Ko], parents[Ko].
#include "cuda_on_cpu.h"

#include "rnnt_gb300.h"

inline int elem_size(int dt) { return dt == RNNT_F32 ? 4 : 2; }

#include "device.inc"

template <typename T, bool FUSED> bool rows(const SelectParams& p, int threads, bool cluster, int K) {
    const auto run = [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        if (cluster)
            return run_blocks(K, threads, 0, sizeof(ClusterShared<NV>) + 16 * (size_t)p.K * p.n,
                              [&] { k_search<T, NV, FUSED>(p); });
        for (int b = 0; b < p.K * p.splits; ++b)
            if (!run_blocks(1, threads, b, 16, [&] { k_rows<T, NV, FUSED>(p); })) return false;
        return true;
    };
    if (p.split_vecs <= threads) return run(std::integral_constant<int, 1>{});
    if (p.split_vecs <= 2 * threads) return run(std::integral_constant<int, 2>{});
    return run(std::integral_constant<int, 4>{});
}

template <typename T> bool select(SelectParams& p, int cluster) {
    const int threads = cluster ? kClusterThreads : kRowThreads;
    if (!(p.fused ? rows<T, true>(p, threads, cluster, p.K) : rows<T, false>(p, threads, cluster, p.K)))
        return false;
    return cluster || run_blocks(1, kPickThreads, 0, 16 * (size_t)p.K * p.splits * p.n,
                                 [&] { k_pick<T>(p); });
}

int main() {
    for (int32_t h[9]; fread(h, sizeof h, 1, stdin) == 1;) {
        const auto [dt, K, V, Ko, fused, splits, skip, has_finished, no_minimum] = h;
        std::vector<float> scores(K);
        std::vector<uint8_t> finished(K);
        const size_t es = elem_size(dt), bytes = ((size_t)skip + (size_t)K * V) * es;
        std::unique_ptr<char[]> space(new char[bytes + 16]);
        char* logits = space.get() + (-(uintptr_t)space.get() & 15);
        if (fread(scores.data(), 4, K, stdin) != (size_t)K ||
            fread(finished.data(), 1, K, stdin) != (size_t)K ||
            fread(logits, 1, bytes, stdin) != bytes)
            return 2;
        SelectLayout L =
            select_layout(1, K, V, Ko, dt, splits < 0 ? kAnyCluster : kMaxCluster);
        if (splits > 0) {
            const int vecs = std::max(1, V / (16 / (int)es));
            L.cluster = 0;
            L.split_vecs = (vecs + splits - 1) / splits;
            L.splits = (vecs + L.split_vecs - 1) / L.split_vecs;
        }
        if (!L.splits) L.splits = 1;
        std::vector<float4> stat(K * L.splits);
        std::vector<uint64_t> list((size_t)K * L.splits * L.n);
        std::vector<float> out_scores(Ko);
        std::vector<int32_t> out_tokens(Ko), out_parents(Ko);
        int32_t status[2] = {0, 0};
        SelectParams p{};
        p.logits = logits + skip * es;
        p.batch_stride = (int64_t)K * V * es;
        p.beam_stride = (int64_t)V * es;
        p.scores = scores.data();
        p.finished = has_finished ? finished.data() : nullptr;
        p.B = 1;
        p.K = K;
        p.V = V;
        p.Ko = Ko;
        p.fused = fused;
        p.splits = L.splits;
        p.split_vecs = L.split_vecs;
        p.n = L.n;
        p.stat = stat.data();
        p.list = list.data();
        p.out_scores = out_scores.data();
        p.out_tokens = out_tokens.data();
        p.out_parents = out_parents.data();
        p.status = status;
        g_no_minimum = no_minimum;
        status[1] = dt == RNNT_F32   ? select<float>(p, L.cluster)
                    : dt == RNNT_F16 ? select<__half>(p, L.cluster)
                                     : select<__nv_bfloat16>(p, L.cluster);
        fwrite(status, sizeof status, 1, stdout);
        fwrite(out_scores.data(), 4, Ko, stdout);
        fwrite(out_tokens.data(), 4, Ko, stdout);
        fwrite(out_parents.data(), 4, Ko, stdout);
        fflush(stdout);
    }
}
