// softmax_tile.cuh -- the online softmax of a tile of 128 query rows by 128
// keys in tensor memory, and the handling of 16-bit values that are not finite,
// shared by the attention kernels on the 5th-generation tensor cores whose
// query rows are the lanes.
#pragma once

#include "tcgen05.cuh"

namespace pkv {

// A pair of 16-bit floats: bit 0 (1) set where the low (high) one is an infinity or NaN.
template <bool kBF16>
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
    constexpr uint32_t e = kBF16 ? 0x7f80u : 0x7c00u;
    return ((w & e) == e ? 1u : 0u) | ((w >> 16 & e) == e ? 2u : 0u);
}
// ... with those put to zero.
template <bool kBF16>
__device__ __forceinline__ uint32_t finite_or_zero2(uint32_t w) {
    const uint32_t bad = not_finite2<kBF16>(w);
    return w & ~((bad & 1u ? 0xffffu : 0u) | (bad & 2u ? 0xffff0000u : 0u));
}

template <bool kBF16>
__device__ __forceinline__ float widen16(uint16_t h) {
    if constexpr (kBF16)
        return __uint_as_float((uint32_t)h << 16);
    else
        return __half2float(__ushort_as_half(h));
}

// 2^x (results below fp32's normal range become zero).
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The running maximum is raised, and the sums rescaled, only when a score passes it by more than this (log2 units):
// weights up to 2^8 against the old one are as good.
constexpr float kRaise = 8.f;

// One tile of S (128 columns from s_addr on; this thread's lane is its query row) into the row's running maximum m_run
// (log2 domain) and sum l, and into P, 16 bits, over the first 64 columns of S; the row's O (128 columns from o_addr on, if
// `begun`) is rescaled where the maximum is raised.  The row's sum is that of the rounded weights, so that the weights that
// the products see add up to one.  scaled: the tile has masks, seen(c) says which of keys c .. c + 31 the row attends, or
// the scale is not above zero; else every key counts and the scale is applied on the way into the exponential.
//
// Twice over S, 32 columns at a time, the largest score and then the weights: a row kept in registers between the two does
// not fit beside the rest (168 registers a thread; 640 bytes of spills a thread), and tensor memory hands 32 columns over in
// some 32 cycles.
template <bool kBF16, typename Seen>
__device__ __forceinline__ void softmax_tile(uint32_t s_addr, uint32_t o_addr, bool scaled, float scale_log2, bool begun,
                                             float& m_run, float& l, Seen seen) {
    const float f = scaled ? 1.f : scale_log2;
    const auto scores = [&](int c, float (&s)[32]) {
        tmem_ld_wait32(s);
        if (scaled) {
            const uint32_t bits = seen(32 * c);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = bits >> i & 1 ? s[i] * scale_log2 : -INFINITY;
        }
    };
    float s[2][32];
    float mx = -INFINITY;
    tmem_ld32_start(s_addr, s[0]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        scores(c, s[c & 1]);
        if (c < 3) tmem_ld32_start(s_addr + 32 * (c + 1), s[(c + 1) & 1]);
#pragma unroll
        for (int i = 0; i < 32; i += 2) mx = fmaxf(mx, fmaxf(s[c & 1][i], s[c & 1][i + 1]));
    }
    tmem_ld32_start(s_addr, s[0]);
    mx *= f;
    const bool raise = mx > m_run + kRaise;
    float alpha = 1.f;
    if (raise) {
        alpha = m_run == -INFINITY ? 0.f : exp2f(m_run - mx);
        m_run = mx;
        l *= alpha;
    }
    if (begun && __any_sync(0xffffffffu, raise)) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            float o[32];
            tmem_ld32_start(o_addr + 32 * c, o);
            tmem_ld_wait32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= alpha;
            tmem_st32(o_addr + 32 * c, o);
        }
    }
    const float ms = m_run == -INFINITY ? 0.f : m_run;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float(&v)[32] = s[c & 1];
        scores(c, v);
        if (c < 3) tmem_ld32_start(s_addr + 32 * (c + 1), s[(c + 1) & 1]);
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float a, b;
            w[i] = pack2<kBF16>(fast_exp2(fmaf(v[2 * i], f, -ms)), fast_exp2(fmaf(v[2 * i + 1], f, -ms)), a, b);
            l += a + b;
        }
        tmem_st16_start(s_addr + 16 * c, w);  // over columns that have been read
    }
    tmem_st_wait();
}

}  // namespace pkv
