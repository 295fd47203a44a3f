// The drawing kernel, compiled from its source for the CPU (sample_device.inc, cut out of rnnt_rows.cuh
// and rnnt_sample.cu), on one case read from standard input: int32 header {dtype, B, K, V, top_k,
// fused, skip, threads, here}, double {temperature, top_p, min_p}, float scores[B K], random[B K],
// `skip` elements and the B * K * V logits.  Writes int32 {status, found a way out}, float scores[B K],
// int32 tokens[B K].
#include "cuda_on_cpu.h"

#include "rnnt_gb300.h"

template <class T> T __shfl_up_sync(unsigned, T x, int o) {
    const int l = threadIdx.x & 31;
    return from_bits<T>(warp_op(bits_of(x), [&](uint64_t* v) { return v[l < o ? l : l - o]; }));
}
inline uint32_t __reduce_add_sync(unsigned, uint32_t x) {
    return (uint32_t)warp_op(x, [](uint64_t* v) {
        uint64_t s = 0;
        for (int i = 0; i < 32; ++i) s += v[i];
        return s;
    });
}
template <class F> float warp_reduced(float x, F f) {
    return from_bits<float>(warp_op(bits_of(x), [&](uint64_t* v) {
        float m = from_bits<float>(v[0]);
        for (int i = 1; i < 32; ++i) m = f(m, from_bits<float>(v[i]));
        return bits_of(m);
    }));
}
inline bool __any_sync(unsigned m, bool p) { return __ballot_sync(m, p) != 0; }
inline int __clz(unsigned x) { return x ? __builtin_clz(x) : 32; }
inline uint32_t atomicAdd(uint32_t* p, uint32_t x) { const uint32_t o = *p; *p += x; return o; }
inline int atomicMin(int* p, int x) { const int o = *p; *p = std::min(o, x); return o; }
inline void atomicMin(unsigned long long* p, unsigned long long x) { *p = std::min(*p, x); }
inline void atomicMax(unsigned long long* p, unsigned long long x) { *p = std::max(*p, x); }
inline float __fadd_rn(float a, float b) { return a + b; }
inline float __fsub_rn(float a, float b) { return a - b; }
inline uint32_t __float2uint_rn(float x) { return (uint32_t)std::llrint(x); }
inline float __int_as_float_(int x) { return std::bit_cast<float>(x); }
inline float __double2float_ru(double x) {
    const float f = (float)x;
    return (double)f < x ? std::nextafterf(f, INFINITY) : f;
}
inline __half __float2half_ru(float x) {
    _Float16 h = (_Float16)x;
    if ((float)h < x) {
        const uint16_t b = std::bit_cast<uint16_t>(h);
        h = std::bit_cast<_Float16>((uint16_t)(b == 0x8000 ? 1 : b & 0x8000 ? b - 1 : b + 1));
    }
    return {h};
}
inline __nv_bfloat16 __float2bfloat16_ru(float x) {
    uint32_t b = __float_as_uint(x);
    if ((b & 0xffff) && !(b >> 31)) b += 0x10000;
    return {(uint16_t)(b >> 16)};
}
template <class T2> T2 __hmax2_nan(T2 a, T2 b) {
    using T = decltype(a.x);
    const auto most = [](T x, T y) {
        const float f = to_f32(x), g = to_f32(y);
        return f != f ? x : g != g ? y : f > g ? x : y;
    };
    return {most(a.x, b.x), most(a.y, b.y)};
}
template <class T2> unsigned __hge2_mask(T2 a, T2 b) {
    return (to_f32(a.x) >= to_f32(b.x) ? 0xffffu : 0u) | (to_f32(a.y) >= to_f32(b.y) ? 0xffff0000u : 0u);
}
template <class T2> unsigned __hgt2_mask(T2 a, T2 b) {
    return (to_f32(a.x) > to_f32(b.x) ? 0xffffu : 0u) | (to_f32(a.y) > to_f32(b.y) ? 0xffff0000u : 0u);
}

inline void mbar_init(uint64_t*) {}
inline void fence_mbar_init() {}
inline void mbar_wait(uint64_t*, uint32_t, int&, int32_t*) {}
inline void bulk_load(void* to, const void* from, uint32_t bytes, uint64_t*) {
    if ((uintptr_t)to % 16 || (uintptr_t)from % 16 || bytes % 16) abort();
    memcpy(to, from, bytes);
}

#include "sample_device.inc"

template <typename T, int TH, bool HERE> bool draw(const SampleParams& p) {
    for (int row = 0; row < p.B * p.K; ++row)
        if (!run_blocks(1, TH, row, HERE ? ((size_t)p.V * sizeof(T) + 30) / 16 * 16 : 16,
                        [&] { k_sample<T, TH, HERE>(p); }))
            return false;
    return true;
}
template <typename T> bool draw(const SampleParams& p, int threads, int here) {
    if (threads == 128) return draw<T, 128, true>(p);
    if (threads == 256) return draw<T, 256, true>(p);
    return here ? draw<T, 512, true>(p) : draw<T, 512, false>(p);
}

int main() {
    int32_t h[9];
    double d[3];
    if (fread(h, sizeof h, 1, stdin) != 1 || fread(d, sizeof d, 1, stdin) != 1) return 2;
    const auto [dt, B, K, V, top_k, fused, skip, threads, here] = h;
    const int es = dt == RNNT_F32 ? 4 : 2, n = B * K;
    std::vector<float> scores(n), random(n), out(n);
    std::vector<int32_t> tokens(n);
    const size_t bytes = ((size_t)skip + (size_t)n * V) * es;
    std::unique_ptr<char[]> space(new char[bytes + 16]);
    char* logits = space.get() + (-(uintptr_t)space.get() & 15);
    if (fread(scores.data(), 4, n, stdin) != (size_t)n || fread(random.data(), 4, n, stdin) != (size_t)n ||
        fread(logits, 1, bytes, stdin) != bytes)
        return 2;
    int32_t status[2] = {0, 0};
    SampleParams p{};
    fill_params(p, V, d[0], top_k, d[1], d[2], fused);
    p.logits = logits + (size_t)skip * es;
    p.batch_stride = (int64_t)K * V * es;
    p.beam_stride = (int64_t)V * es;
    p.scores = scores.data();
    p.random = random.data();
    p.B = B;
    p.K = K;
    p.out_scores = out.data();
    p.out_tokens = tokens.data();
    p.status = status;
    status[1] = dt == RNNT_F32   ? draw<float>(p, threads, here)
                : dt == RNNT_F16 ? draw<__half>(p, threads, here)
                                 : draw<__nv_bfloat16>(p, threads, here);
    fwrite(status, sizeof status, 1, stdout);
    fwrite(out.data(), 4, n, stdout);
    fwrite(tokens.data(), 4, n, stdout);
}
