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

// The values of one token in shared memory, 16 * n bytes at the places at(i): zeros for a token that is not there, else those
// that are not finite are put to zero; whether there were any.  Looked for by a product with zero, which is NaN for them.
template <bool kBF16, typename At>
__device__ __forceinline__ bool scrub(int n, bool there, At at) {
    if (!there) {
#pragma unroll 4
        for (int i = 0; i < n; ++i) *at(i) = make_uint4(0, 0, 0, 0);
        return false;
    }
    uint32_t acc = 0;
    const auto see = [&](uint32_t w) {
        if constexpr (kBF16)
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0u));
        else
            asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0u));
    };
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const uint4 w = *at(i);
        see(w.x), see(w.y), see(w.z), see(w.w);
    }
    if (!not_finite2<kBF16>(acc)) return false;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        uint4 w = *at(i);
        w.x = finite_or_zero2<kBF16>(w.x), w.y = finite_or_zero2<kBF16>(w.y);
        w.z = finite_or_zero2<kBF16>(w.z), w.w = finite_or_zero2<kBF16>(w.w);
        *at(i) = w;
    }
    return true;
}

template <bool kBF16>
__device__ __forceinline__ float widen16(uint16_t h) {
    if constexpr (kBF16)
        return __uint_as_float((uint32_t)h << 16);
    else
        return __half2float(__ushort_as_half(h));
}

// Adds to `n` sums (fp32 partials, or outputs of the 16-bit type) the values at v that are not finite.
template <bool kBF16>
__device__ __noinline__ void add_not_finite(float* part, uint16_t* out, const uint16_t* v, int n) {
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        if (!not_finite2<kBF16>(v[i])) continue;
        const float x = widen16<kBF16>(v[i]);
        if (part)
            part[i] += x;
        else
            out[i] = (uint16_t)pack2<kBF16>(widen16<kBF16>(out[i]) + x, 0.f);
    }
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

// Weights are 2^(score - maximum + this) on their way to 16 bits.  fp16 ends at 2^16 and the weights at 2^kRaise, so its steps
// of 2^-24 near zero are used seven binades further down: what a weight loses there is at most 2^-32 of the largest, so that 2^21
// tokens of the smallest weights are held to the output's own half step (without it 131072 tokens 18 below one other in the
// exponent, 2^-9 of the output, would be zeros).  The factor is in the row's sum and its products alike, and every part of a
// divided context has it.  bf16 has fp32's range.
template <bool kBF16>
constexpr float kWeightExponent = kBF16 ? 0.f : 7.f;

// Two fp32 values in a register pair, and their arithmetic.
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 pack_f32x2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack_f32x2(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma_f32x2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add_f32x2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Raises the row's maximum to mx where that passes it, and rescales what the row has summed.
__device__ __forceinline__ void raise_maximum(float mx, uint32_t o_addr, float& m_run, float& l) {
    const bool raise = mx > m_run + kRaise;
    if (!__any_sync(0xffffffffu, raise)) return;
    float alpha = 1.f;
    if (raise) {
        alpha = m_run == -INFINITY ? 0.f : exp2f(m_run - mx);
        m_run = mx;
        l *= alpha;
    }
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

// 32 scores v to weights 2^(v f + neg_ms): 16 pairs to `w`, their sum added to `sum`.
template <bool kBF16>
__device__ __forceinline__ void weights32(const float (&v)[32], f32x2 f, f32x2 neg_ms, uint32_t (&w)[16], f32x2& sum) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 x = unpack_f32x2(fma_f32x2(pack_f32x2(v[2 * i], v[2 * i + 1]), f, neg_ms));
        const float a = fast_exp2(x.x), b = fast_exp2(x.y);
        w[i] = pack2<kBF16>(a, b);
        sum = add_f32x2(sum, pack_f32x2(a, b));
    }
}

// One tile of S (128 columns from s_addr on; this thread's lane is its query row) into the row's running maximum m_run
// (log2 domain) and sum l, and into P, 16 bits, over the first 64 columns of S; the row's O (128 columns from o_addr on, if
// `begun`) is rescaled where the maximum is raised.  masked: the tile has masks, seen(c) says which of keys c .. c + 31 the row
// attends; else every key counts.
//
// Twice over S, 32 columns at a time, the largest score and then the weights: a row kept in registers between the two does not
// fit beside the rest (168 registers a thread).  Taking a tile against the maxima of the tiles before, in one pass whose
// weights wait in registers, is 500 of 1500 cycles shorter for one warp and 5% slower for the prompts' kernel; eight warps to
// a stream, with half a row's registers each, are slower yet.  Masks are written into S first, so that a tile with masks goes
// the same way as the others: code that runs once in a unit waits for its instructions, and a loop of its own for such tiles
// took 5200 cycles where the way of all tiles takes 1500.
template <bool kBF16, typename Seen>
__device__ __forceinline__ void softmax_tile(uint32_t s_addr, uint32_t o_addr, bool masked, float scale_log2, bool begun,
                                             float& m_run, float& l, Seen seen) {
    // Where the scale is above zero, it is applied on the way into the exponential; else the scores are scaled in S, since
    // their order is another then.
    const bool scaled = !(scale_log2 > 0.f);
    const float f = scaled ? 1.f : scale_log2;
    if (masked || scaled) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            const uint32_t bits = masked ? seen(32 * c) : ~0u;
            if (!scaled && __all_sync(0xffffffffu, bits == ~0u)) continue;
            float s[32];
            tmem_ld32_start(s_addr + 32 * c, s);
            tmem_ld_wait32(s);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = bits >> i & 1 ? (scaled ? s[i] * scale_log2 : s[i]) : -INFINITY;
            tmem_st32(s_addr + 32 * c, s);
        }
    }
    f32x2 sum = pack_f32x2(0.f, 0.f);
    float s[2][32];
    float mx = -INFINITY;
    tmem_ld32_start(s_addr, s[0]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        tmem_ld_wait32(s[c & 1]);
        tmem_ld32_start(s_addr + 32 * ((c + 1) & 3), s[(c + 1) & 1]);
#pragma unroll
        for (int i = 0; i < 32; i += 2) mx = fmaxf(mx, fmaxf(s[c & 1][i], s[c & 1][i + 1]));
    }
    mx *= f;
    if (begun)
        raise_maximum(mx, o_addr, m_run, l);
    else
        m_run = fmaxf(m_run, mx);
    const float neg_ms = kWeightExponent<kBF16> - (m_run == -INFINITY ? 0.f : m_run);
    const f32x2 ff = pack_f32x2(f, f), neg = pack_f32x2(neg_ms, neg_ms);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        tmem_ld_wait32(s[c & 1]);
        if (c < 3) tmem_ld32_start(s_addr + 32 * (c + 1), s[(c + 1) & 1]);
        uint32_t w[16];
        weights32<kBF16>(s[c & 1], ff, neg, w, sum);
        tmem_st16_start(s_addr + 16 * c, w);  // over columns that have been read
    }
    const float2 both = unpack_f32x2(sum);
    l += both.x + both.y;
    tmem_st_wait();
}

}  // namespace pkv
