// Rows in a stage (rnnt_rows.cuh's Staged) on the CPU: arguments {dtype, V, rows, skip}.  Every row of a tensor
// that begins `skip` elements behind a 16-byte boundary is copied and completed by a warp; fails where a
// copy reaches past the tensor's ends, or the stage does not hold the row with -inf around it.
#define main draw_main
#include "sample_on_cpu.cpp"
#undef main

template <typename T> int check(int V, int rows, int skip) {
    constexpr int E = 16 / (int)sizeof(T);
    const size_t n = (size_t)rows * V;
    std::vector<char> space((skip + n + 2 * E) * sizeof(T) + 32);
    T* const begin = reinterpret_cast<T*>(space.data() + (-(uintptr_t)space.data() & 15)) + skip;
    T* const end = begin + n;
    for (size_t i = 0; i < n; ++i) begin[i] = from_f32<T>((float)(i % 97));
    int bad = 0;
    for (int row = 0; row < rows; ++row) {
        const bool done = run_blocks(1, 32, 0, ((size_t)V * sizeof(T) + 30) / 16 * 16, [&] {
            uint4* const stage = reinterpret_cast<uint4*>(g_fiber->cta->dynamic);
            const Staged<T, 32> s(begin + (size_t)row * V, V, stage, begin, end);
            if (threadIdx.x == 0) {
                const uintptr_t at = (uintptr_t)(s.r.x - s.r.off);
                if (s.hi > s.lo && (at + 16 * s.lo < (uintptr_t)begin || at + 16 * s.hi > (uintptr_t)end)) bad |= 1;
                s.fetch(nullptr);
            }
            __syncwarp();
            s.complete();
            for (int i = threadIdx.x; i < s.r.n * E; i += 32) {
                const int e = i - s.r.off;
                const float want = e >= 0 && e < V ? to_f32(s.r.x[e]) : -INFINITY;
                if (to_f32(reinterpret_cast<const T*>(stage)[i]) != want) bad |= 2;
            }
        });
        if (!done) bad |= 4;
    }
    return bad;
}

int main(int n, char** a) {
    if (n != 5) return 64;
    const int dt = atoi(a[1]), V = atoi(a[2]), rows = atoi(a[3]), skip = atoi(a[4]);
    return dt == 0 ? check<float>(V, rows, skip) : dt == 1 ? check<__half>(V, rows, skip)
                                                           : check<__nv_bfloat16>(V, rows, skip);
}
