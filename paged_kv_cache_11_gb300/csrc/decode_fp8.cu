// decode_fp8.cu -- paged decode attention over an e4m3 pool with one scale
// for each (block, KV head) (paged_attention_decode_fp8).
//
// The mathematics is the decode kernel's (decode.cu) with K[t] = ks K8[t] and
// V[t] = vs V8[t], ks and vs constant over a block: ks multiplies the scores
// of the block's tokens, vs its share of the output, both in 32 bits, and the
// products see the e4m3 values themselves, exact as fp16:
//   S^T = K8 Q^T, p = 2^(sl2 ks S - m), O^T += vs (V8^T P^T), l += p.
// q enters as fp16 too, each head row divided by the power of two that brings
// its largest value to [1, 2): bf16 has 8 significant bits and fp16 11, so
// nothing is lost but below 2^-25 of the row's largest value.  P is split into
// an fp16 value and an fp16 residual (22 bits), and lifted by 2^kF8Lift, so
// that p reaches up to 2^15 and fp16's smallest step, 2^-24, lies 2^-31 below
// the largest weight: a context's many small weights keep their bits beside a
// few large ones.
//
// vs enters through P as well: a warp keeps O in units of a reference scale
// vref and multiplies p by vs / vref, which fp16 holds without loss while the
// ratio is in [2^-6, 1].  Only a scale outside of that moves O to a new
// reference (a test that the whole warp passes together), so the products
// need no scale after them.  (Adding each unit's product, times vs, to O took
// 32 more multiply-adds per unit: 83 us against 78 for 64 sequences.)
//
// A unit of work is 16 tokens of one (block, KV head) tile: 2 KiB of K and 2
// KiB of V.  The warps of a CTA take units in turn, each through a ring of its
// own in shared memory, filled by 16-byte asynchronous copies of whole rows
// (copies of half rows, each lane its own bytes, held the stream to 5.2 TB/s).
// A lane (g = lane / 4, t = lane % 4) reads 16-byte chunks of them:
//   K: rows g and g + 8, chunks 2t and 2t + 1: with the query held in the same
//      order of dims, word j of a chunk is the A operand of one k-step;
//   V: tokens 2t, 2t + 1, 2t + 8, 2t + 9, chunk g: byte pairs of two tokens
//      are interleaved (PRMT) to make the A operand of V^T, and a lane ends up
//      with 16 neighbouring dims of the output.
// TMA copies would be 2 KiB each here, which the SM's TMA unit takes some 75
// cycles for, 150 of the about 180 that a unit may cost at full bandwidth.
//
// Bytes bound long contexts: 8 sequences of 131072 tokens, 64/8 heads (2.15 GB)
// in 327 us, 6.6 TB/s.  Short ones lose to each CTA's start and end, some 6 us:
// 64 of 512 to 4096 tokens, 32/8 heads (304 MB) in 59.8 us, 5.1 TB/s.  Other
// shapes of the CTA were slower there (warps, stages, CTAs per SM: 2, 2, 6
// 64.2 us; 2, 3, 4 67.5; 4, 3, 2 71.5; 3, 2, 4 65.0 against 62.4 then).
#include <atomic>

#include "decode_common.cuh"

namespace pkv {

constexpr int kF8Warps = 4;             // warps per CTA, each with a ring of its own
constexpr int kF8Stages = 2;            // pairs of units: one in use, the others in flight
constexpr int kF8CtasPerSm = kDecodeFp8CtasPerSm;
constexpr float kF8Lift = 7.f;          // log2; kLazyMargin + kF8Lift stays below fp16's 2^16
constexpr int kF8UnitBytes = 2 * 16 * kHeadDim;       // 16 tokens of K and V
constexpr int kF8StageBytes = 2 * kF8UnitBytes + 16;  // two units and their scales: ks, vs, ks, vs

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^x, results below 2^-126 flushed to zero: the weights have no use for them.
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The four e4m3 values of a word as two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// d = a b, the first product of a sum.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// d += a b
__device__ __forceinline__ void mma_next(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// a += b, two values in one instruction.
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\t"
        "mov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}

template <int HT>
struct DecodeFp8Smem {
    static constexpr int kRing = kF8Warps * kF8Stages * kF8StageBytes;
    // per-warp rows, per-warp (m, l, vref), per-row merge weights and lse
    static constexpr int kRed = kF8Warps * HT * kRedStride * 4 + kF8Warps * HT * 3 * 4 + HT * (kF8Warps + 1) * 4;
    static constexpr int kFlags = ((kRing > kRed ? kRing : kRed) + 15) / 16 * 16;
    static constexpr int kTotal = kFlags + 16;
};

// NH: 8-head n-tiles per CTA (1: up to 8 query heads of a group, 2: up to 16).
// kRound: for fp32 outputs.  The tensor cores round towards zero with every
// step, by a part of what they add to; products added to O at once shrink it
// by 1e-6 over 2048 tokens (7 sequences of 12859 tokens: 1.2e-6 off in all,
// nothing beside a 16-bit output's rounding).  Summed pair by pair and added to
// nearest they leave 5.5e-7, for 63.3 us against 59.8 (64 sequences of 512 to
// 4096 tokens).
template <int NH, bool kRound>
__global__ void __launch_bounds__(kF8Warps * 32, NH == 1 ? kF8CtasPerSm : kF8CtasPerSm - 1)
    decode_fp8_kernel(const __grid_constant__ DecodeFp8Params fp) {
    const DecodeParams& p = fp.d;
    constexpr int D = kHeadDim, HT = 8 * NH, NW = kF8Warps, NST = kF8Stages;
    using S = DecodeFp8Smem<HT>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

    // Grid as the decode kernel's: (head group, sequence, partition counted
    // from the end of the sequence), or (partition, head group, sequence) for
    // more partitions than the slowest dimension holds.
    const int ygrp = p.parts_in_x ? blockIdx.y : blockIdx.x;
    const int kvh = ygrp / p.head_tiles;
    const int ht = ygrp - kvh * p.head_tiles;
    const int s = p.parts_in_x ? blockIdx.z : blockIdx.y;
    const int from_end = p.parts_in_x ? blockIdx.x : blockIdx.z;
    const int h0 = kvh * p.group + ht * HT;
    const int rows = min(HT, p.group - ht * HT);

    pdl_launch_dependents();
    pdl_wait();
    const int L = p.context_lens[s];
    const bool bad_len = L < 0 || L > p.len_limit;
    const int nparts = bad_len || L == 0 ? 1 : (L - 1) / p.partition_size + 1;
    if (from_end >= nparts) return;
    const int part = nparts - 1 - from_end;
    if (bad_len || L == 0) {  // nothing to attend: zeros
        if (bad_len && tid == 0) record_error(p.err, PKV_DEVERR_CONTEXT_LEN);
        for (int i = tid; i < rows * D; i += blockDim.x) store_out(p, s, h0 + i / D, i % D, 0.f);
        return;
    }
    // The row's blocks in nparts even parts: no part is longer than
    // partition_size, and none is a short rest that leaves the others waiting.
    // (part < nparts, and nparts - 1 full parts hold less than the row, so
    // every part has a token.)
    const bool whole = p.block_size == 32;  // a pair is one block (else two of 16)
    const int sh = whole ? 5 : 4;
    const int per_blocks = (((L - 1) >> sh) + nparts) / nparts, first_block = part * per_blocks;
    const int len = min(L - (first_block << sh), per_blocks << sh);  // tokens of this part
    const int npairs = (len + 31) / 32;
    const bool write_partial = p.split && nparts > 1;

    // ---- this warp's pairs: warp, warp + NW, ...
    const int mine = npairs > warp ? (npairs - 1 - warp) / NW + 1 : 0;
    const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks_per_seq + first_block;
    const int nblk = ((len - 1) >> sh) + 1;  // blocks of this partition
    const uint64_t policy = l2_policy_evict_first();
    uint8_t* ring = smem + warp * (NST * kF8StageBytes);
    const uint32_t ring_sa = smem_addr(ring);

    int ids0 = 0, ids1 = 0;
    bool bad_id = false;
    // Block ids of the warp's n-th pair: 32 pairs are read at a time, a lane
    // each.  A pair without a second unit names its first block twice (its
    // tokens are masked).
    auto load_ids = [&](int n0) {
        const int n = n0 + lane;
        bool bad = false;
        if (n < mine) {
            const int pr = warp + n * NW;
            const int b0 = whole ? pr : 2 * pr, b1 = whole ? pr : min(2 * pr + 1, nblk - 1);
            ids0 = __ldg(table + b0);
            ids1 = __ldg(table + b1);
            bad = ids0 < 0 || (int64_t)ids0 >= p.num_blocks || ids1 < 0 || (int64_t)ids1 >= p.num_blocks;
            if (bad) ids0 = ids1 = 0;  // the output is zeroed below
        }
        if (bad) {
            bad_id = true;
            record_error(p.err, PKV_DEVERR_BLOCK_ID);
        }
    };
    // A copy instruction brings four whole rows; lane l has chunk l % 8 of row
    // l / 8.  Chunk c of row r goes to chunk c ^ (r % 8) of its row in shared
    // memory, which keeps the reads below free of bank conflicts.
    const int own = kvh * (p.block_size * D) + lane * 16;  // of the KV head's tile in a block, and of the lane in it
    const int r8 = lane >> 3, put = (lane >> 3) * D;
    const uint32_t put0 = put + (((lane & 7) ^ r8) << 4), put1 = put + (((lane & 7) ^ (r8 + 4)) << 4) + 4 * D;
    const int second = whole ? 16 * D : 0;  // where a pair's second unit starts in its block
    auto issue = [&](int n, int st) {       // pair n into stage st
        if (n < mine) {
            if ((n & 31) == 0) load_ids(n);
            const int id0 = __shfl_sync(0xffffffffu, ids0, n & 31), id1 = __shfl_sync(0xffffffffu, ids1, n & 31);
            const uint32_t sa = ring_sa + st * kF8StageBytes;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t off = (u ? id1 : id0) * fp.block_bytes + (own + (u ? second : 0));
                const uint8_t* kr = fp.k8 + off;
                const uint8_t* vr = fp.v8 + off;
                const uint32_t dst = sa + u * kF8UnitBytes;
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // rows 8i .. 8i + 7 of K and of V
                    cp_async16(dst + put0 + 8 * D * i, kr + 8 * D * i, policy);
                    cp_async16(dst + put1 + 8 * D * i, kr + 8 * D * i + 4 * D, policy);
                    cp_async16(dst + put0 + 8 * D * i + 16 * D, vr + 8 * D * i, policy);
                    cp_async16(dst + put1 + 8 * D * i + 16 * D, vr + 8 * D * i + 4 * D, policy);
                }
            }
            if (lane < 4)
                cp_async4(sa + 2 * kF8UnitBytes + 4 * lane, ((lane & 1) ? fp.v_scales : fp.k_scales) +
                                                                (int64_t)(lane < 2 ? id0 : id1) * p.num_kv_heads + kvh);
            __syncwarp();
        }
        cp_async_commit();
    };
#pragma unroll
    for (int n = 0; n < NST - 1; ++n) issue(n, n);

    // ---- the query: head 8n + g, dims of chunk 2t (k-steps 0-3) and 2t + 1 (4-7)
    uint32_t qf[NH][8][2];
    float qs[NH][2];  // what a product of the heads 8n + 2t, 8n + 2t + 1 is multiplied by
#pragma unroll
    for (int n = 0; n < NH; ++n) {
        const int hr = 8 * n + g;
        float x[32];
        float mx = 0.f;
        if (hr < rows) {
            const uint16_t* qr = static_cast<const uint16_t*>(p.q) + ((int64_t)s * p.num_q_heads + h0 + hr) * D;
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // 8 values each
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(qr + 32 * t + 8 * c));
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lo, hi;
                    if (fp.q_bf16) {
                        lo = __uint_as_float(ww[j] << 16);
                        hi = __uint_as_float(ww[j] & 0xffff0000u);
                    } else {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[j]));
                        lo = f.x, hi = f.y;
                    }
                    x[8 * c + 2 * j] = lo;
                    x[8 * c + 2 * j + 1] = hi;
                    mx = fmaxf(mx, fmaxf(fabsf(lo), fabsf(hi)));
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = 0.f;
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // 2^e <= mx < 2^(e+1) (e is held to what has a normal reciprocal);
        // rows of zeros, and rows with an infinity, keep their values
        const int e = mx > 0.f && mx < INFINITY ? min(max((int)(__float_as_uint(mx) >> 23), 2) - 127, 126) : 0;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int b = 0; b < 2; ++b)
                qf[n][ks][b] = pack2<false>(x[4 * ks + 2 * b] * down, x[4 * ks + 2 * b + 1] * down);
        const float f = p.scale_log2 * up;
        qs[n][0] = __shfl_sync(0xffffffffu, f, 8 * t);      // lane 4 (2t): head 8n + 2t
        qs[n][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);  // lane 4 (2t + 1)
    }

    WarpAcc<NH> a;  // o[mt][n]: dims 16g + 2mt (0, 1) and 16g + 2mt + 1 (2, 3) of heads 8n + 2t, 8n + 2t + 1
    acc_reset(a);
    float vref = 0.f, vinv = 0.f;  // O's unit and its reciprocal; 0: O is zero and has none

    // O^T += V8^T P^T: tokens 2t, 2t + 1 (k 0-7), 2t + 8, 2t + 9 of a unit
    using V = uint32_t[4][4];
    using P = uint32_t[NH][2];
    const auto v_operand = [](const V& vw, int mt, uint32_t (&af)[4]) {
        const int j = mt >> 1;
        const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;  // bytes 2, 3 or 0, 1 of both tokens, paired
        e4m3x4_to_f16(__byte_perm(vw[0][j], vw[1][j], sel), af[0], af[1]);
        e4m3x4_to_f16(__byte_perm(vw[2][j], vw[3][j], sel), af[2], af[3]);
    };
    const auto pv = [&](const V& vw, const P& ph, const P& pl) {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            uint32_t af[4];
            v_operand(vw, mt, af);
#pragma unroll
            for (int m = 0; m < NH; ++m) {
                mma_16816<false>(a.o[mt][m], af, ph[m][0], ph[m][1]);
                mma_16816<false>(a.o[mt][m], af, pl[m][0], pl[m][1]);
            }
        }
    };
    // ... kRound: both units of a pair, summed by themselves, two sums side by
    // side, and added to O to nearest.
    const auto pv_pair = [&](const V (&vw)[2], const P (&ph)[2], const P (&pl)[2]) {
#pragma unroll
        for (int mt = 0; mt < 8; mt += 2) {
            uint32_t af[2][2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u) v_operand(vw[u], mt + k, af[k][u]);
#pragma unroll
            for (int m = 0; m < NH; ++m) {
                float sum[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) mma_first(sum[k], af[k][0], pl[0][m][0], pl[0][m][1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) mma_next(sum[k], af[k][1], pl[1][m][0], pl[1][m][1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) mma_next(sum[k], af[k][0], ph[0][m][0], ph[0][m][1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) mma_next(sum[k], af[k][1], ph[1][m][0], ph[1][m][1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float(&o)[4] = a.o[mt + k][m];
                    add2(o[0], o[1], sum[k][0], sum[k][1]);
                    add2(o[2], o[3], sum[k][2], sum[k][3]);
                }
            }
        }
    };
    // P^T of one unit as two B operands: the fp16 value and the fp16 residual
    auto split = [&](const float (&x)[NH][4], float ratio, uint32_t (&ph)[NH][2], uint32_t (&pl)[NH][2]) {
#pragma unroll
        for (int m = 0; m < NH; ++m) {
            const float p0 = x[m][0] * ratio, p1 = x[m][1] * ratio, p2 = x[m][2] * ratio, p3 = x[m][3] * ratio;
            float r0, r1, r2, r3;
            const uint32_t h01 = pack2<false>(p0, p1, r0, r1), h23 = pack2<false>(p2, p3, r2, r3);
            ph[m][0] = movmatrix_trans(h01);
            ph[m][1] = movmatrix_trans(h23);
            pl[m][0] = movmatrix_trans(pack2<false>(p0 - r0, p1 - r1));
            pl[m][1] = movmatrix_trans(pack2<false>(p2 - r2, p3 - r3));
        }
    };
    // where the lane's chunks lie in a unit: K row g, chunks 2t and 2t + 1; V
    // rows 2t and 2t + 1, chunk g (rows 8 further on are 8 D further on)
    const uint32_t get_k0 = g * D + (((2 * t) ^ g) << 4), get_k1 = g * D + (((2 * t + 1) ^ g) << 4);
    const uint32_t get_v0 = 16 * D + 2 * t * D + ((g ^ (2 * t)) << 4);
    const uint32_t get_v1 = 16 * D + (2 * t + 1) * D + ((g ^ (2 * t + 1)) << 4);
    // V8 of one unit: tokens 2t, 2t + 1, 2t + 8, 2t + 9, dims 16g .. 16g + 15;
    // rows past the context may hold anything (even NaN): zeros, chosen by masks
    // and not by branches, as the products that follow need the whole warp
    auto load_v = [&](const uint8_t* unit, int valid, uint32_t (&vw)[4][4]) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint4 w = *reinterpret_cast<const uint4*>(unit + ((r & 1) ? get_v1 : get_v0) + (r >> 1) * (8 * D));
            vw[r][0] = w.x, vw[r][1] = w.y, vw[r][2] = w.z, vw[r][3] = w.w;
        }
        if (valid < 16) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t in = 2 * t + (r & 1) + 8 * (r >> 1) < valid ? 0xffffffffu : 0u;
                vw[r][0] &= in, vw[r][1] &= in, vw[r][2] &= in, vw[r][3] &= in;
            }
            __syncwarp();
        }
    };
    // What P is multiplied by for a unit of 16 tokens of scale vs, where a scale
    // of the pair is not in [2^-6, 1] of O's unit; O moves to a new unit where it
    // has to.  A larger scale becomes O's unit.  A smaller one does, too, if O,
    // as it is, stays below 2^110 in it: the scales alone do not tell, as a block
    // of large scale may have no weight, and moves add up.  (Sums of 2^20 tokens
    // stay below 2^44 of the largest scale among them, so that scales within 2^64
    // of one another always move.)  Else it is folded in the unit that O has, and
    // fp16 keeps of it what it can.
    auto take_scale = [&](float vs) {
        if (vs == 0.f) return 0.f;  // adds nothing and sets nothing
        const float r = vs / vref;
        float f = vref / vs;
        if (vref == 0.f || fabsf(r) > 1.f) {
        } else if (fabsf(r) >= 0x1p-6f) {
            return r;
        } else {
            float top = 0.f;
#pragma unroll
            for (int m = 0; m < NH; ++m)
#pragma unroll
                for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(a.o[mt][m][e]));
            top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
            if (top == 0.f)
                f = 1.f;
            else if (!(top * fabsf(f) <= 0x1p110f))
                return r;
        }
#pragma unroll
        for (int m = 0; m < NH; ++m)
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.o[mt][m][e] *= f;
        vref = vs;
        vinv = 1.f / vs;
        return 1.f;
    };

    int st = 0, st_in = NST - 1;  // stage of pair n and of pair n + NST - 1
    for (int n = 0; n < mine; ++n) {
        cp_async_wait<NST - 2>();
        __syncwarp();  // the scales' copies of lanes 0 to 3
        issue(n + NST - 1, st_in);
        const uint8_t* stage = ring + st * kF8StageBytes;
        st_in = st;  // this pair's stage is free when it has been used
        st = st + 1 == NST ? 0 : st + 1;
        const float4 scl = *reinterpret_cast<const float4*>(stage + 2 * kF8UnitBytes);  // ks, vs of both units
        const int valid = len - 32 * (warp + n * NW);  // >= 1

        // ---- S^T = K8 Q^T: tokens g, g + 8 of each unit x heads 2t, 2t + 1
        float sc[2][NH][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int m = 0; m < NH; ++m) sc[u][m][0] = sc[u][m][1] = sc[u][m][2] = sc[u][m][3] = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint4 ka[2], kb[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* at = stage + u * kF8UnitBytes + (c ? get_k1 : get_k0);
                ka[u] = *reinterpret_cast<const uint4*>(at);
                kb[u] = *reinterpret_cast<const uint4*>(at + 8 * D);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t af[4];
                    e4m3x4_to_f16(reinterpret_cast<const uint32_t*>(&ka[u])[j], af[0], af[2]);
                    e4m3x4_to_f16(reinterpret_cast<const uint32_t*>(&kb[u])[j], af[1], af[3]);
#pragma unroll
                    for (int m = 0; m < NH; ++m)
                        mma_16816<false>(sc[u][m], af, qf[m][4 * c + j][0], qf[m][4 * c + j][1]);
                }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int m = 0; m < NH; ++m) {
                const float f0 = qs[m][0] * (u ? scl.z : scl.x), f1 = qs[m][1] * (u ? scl.z : scl.x);
                sc[u][m][0] *= f0, sc[u][m][1] *= f1, sc[u][m][2] *= f0, sc[u][m][3] *= f1;
            }
        if (valid < 32) {  // tokens past the context do not count
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int m = 0; m < NH; ++m) {
                    if (16 * u + g >= valid) sc[u][m][0] = sc[u][m][1] = -INFINITY;
                    if (16 * u + g + 8 >= valid) sc[u][m][2] = sc[u][m][3] = -INFINITY;
                }
        }
        // ---- online softmax; the maximum is raised, and O and l rescaled,
        // only when a score passes it by more than kLazyMargin
        bool need = false;
        float mx[NH][2];
#pragma unroll
        for (int m = 0; m < NH; ++m)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                mx[m][c] = fmaxf(fmaxf(sc[0][m][c], sc[0][m][c + 2]), fmaxf(sc[1][m][c], sc[1][m][c + 2]));
                need |= mx[m][c] > a.m[m][c] + kLazyMargin;
            }
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int m = 0; m < NH; ++m)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x = mx[m][c];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                    const float mn = fmaxf(a.m[m][c], x);
                    const float al = mn == -INFINITY ? 1.f : exp2_ftz(a.m[m][c] - mn);
                    a.m[m][c] = mn;
                    a.l[m][c] *= al;
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt) {
                        a.o[mt][m][c] *= al;
                        a.o[mt][m][c + 2] *= al;
                    }
                }
        }
#pragma unroll
        for (int m = 0; m < NH; ++m)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float m0 = a.m[m][c] == -INFINITY ? 0.f : a.m[m][c];
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        sc[u][m][c + 2 * r] = exp2_ftz(sc[u][m][c + 2 * r] - m0 + kF8Lift);
                        sum += sc[u][m][c + 2 * r];
                    }
                a.l[m][c] += sum;
            }
        // ---- O^T += vs V8^T P^T
        if (vref == 0.f) {  // the first unit that has one: the larger of the pair's, so that both ratios fit
            const float big = fmaxf(fabsf(scl.y), fabsf(scl.w));
            if (big > 0.f && big < INFINITY) vref = big, vinv = 1.f / big;
        }
        float r0 = scl.y * vinv, r1 = scl.w * vinv;
        const bool keep = fabsf(r0) <= 1.f && fabsf(r0) >= 0x1p-6f && fabsf(r1) <= 1.f && fabsf(r1) >= 0x1p-6f;
        P ph[2], pl[2];
        if constexpr (kRound) {
            V vw[2];
            load_v(stage, valid, vw[0]);
            load_v(stage + kF8UnitBytes, valid - 16, vw[1]);
#pragma unroll 1
            for (int pass = keep ? 1 : 0; pass < 2; ++pass) {  // (not keep: the units one after the other)
                if (!keep) {
                    r0 = pass == 0 ? take_scale(scl.y) : 0.f;
                    r1 = pass == 1 && valid > 16 ? take_scale(scl.w) : 0.f;
                }
                split(sc[0], r0, ph[0], pl[0]);
                split(sc[1], r1, ph[1], pl[1]);
                pv_pair(vw, ph, pl);
            }
        } else {
            V vw;
            if (!keep) {  // the first unit by itself, at the unit that its scale sets
                r0 = take_scale(scl.y);
                split(sc[0], r0, ph[0], pl[0]);
                load_v(stage, valid, vw);
                pv(vw, ph[0], pl[0]);
#pragma unroll
                for (int m = 0; m < NH; ++m) sc[0][m][0] = sc[0][m][1] = sc[0][m][2] = sc[0][m][3] = 0.f;
                r1 = valid > 16 ? take_scale(scl.w) : 0.f;
                r0 = 0.f;
            }
            split(sc[0], r0, ph[0], pl[0]);
            split(sc[1], r1, ph[1], pl[1]);
            load_v(stage, valid, vw);
            pv(vw, ph[0], pl[0]);
            load_v(stage + kF8UnitBytes, valid - 16, vw);
            pv(vw, ph[1], pl[1]);
        }
    }
    acc_finish(a);
    cp_async_wait<0>();
    // every ring is free: its memory takes the warps' states
    const int fl = __syncthreads_or(bad_id);

    // ---- merge the warps' states, as the decode kernel does
    float* red = reinterpret_cast<float*>(smem);  // [NW][HT][kRedStride]
    float* ml = red + NW * HT * kRedStride;       // [NW][HT][3]: m, l, vref
    float* wts = ml + NW * HT * 3;                // [HT][NW + 1]: weights, then the row's lse
#pragma unroll
    for (int m = 0; m < NH; ++m)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int hr = 8 * m + 2 * t + c;
            if (hr < rows) {
                float* row = red + (warp * HT + hr) * kRedStride + 16 * g;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<float4*>(row + 4 * q) =
                        make_float4(a.o[2 * q][m][c], a.o[2 * q][m][c + 2], a.o[2 * q + 1][m][c],
                                    a.o[2 * q + 1][m][c + 2]);
                if (g == 0) {
                    ml[(warp * HT + hr) * 3] = a.m[m][c];
                    ml[(warp * HT + hr) * 3 + 1] = a.l[m][c];
                    ml[(warp * HT + hr) * 3 + 2] = vref;
                }
            }
        }
    __syncthreads();
    if (tid < rows) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[(w * HT + tid) * 3]);
        const float Mf = M == -INFINITY ? 0.f : M;
        float f[NW], sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            f[w] = exp2f(ml[(w * HT + tid) * 3] - Mf);  // a warp without units: 0
            sum += f[w] * ml[(w * HT + tid) * 3 + 1];
        }
        const float inv = 1.f / sum;
#pragma unroll
        for (int w = 0; w < NW; ++w) wts[tid * (NW + 1) + w] = f[w] * inv;
        // A NaN among the scores makes the outputs NaN; the merge would pass
        // over a partition whose lse is one, so it gets a finite lse.
        const float lse = M + log2f(sum) - kF8Lift;
        wts[tid * (NW + 1) + NW] = lse == lse ? lse : 0.f;
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 4); i += blockDim.x) {
        const int hr = i / (D / 4), c4 = i - hr * (D / 4);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!fl) {
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                // (weight and unit one after the other: their product may leave fp32's range where the output does not)
                const float ww = wts[hr * (NW + 1) + w], vr = ml[(w * HT + hr) * 3 + 2];
                const float4 r = *reinterpret_cast<const float4*>(red + (w * HT + hr) * kRedStride + 4 * c4);
                o.x += vr * (ww * r.x);
                o.y += vr * (ww * r.y);
                o.z += vr * (ww * r.z);
                o.w += vr * (ww * r.w);
            }
        }
        if (write_partial) {
            const int64_t idx = ((int64_t)s * p.num_q_heads + h0 + hr) * p.max_parts + part;
            *reinterpret_cast<float4*>(p.part_o + idx * D + 4 * c4) = o;
            // +inf marks a partition whose metadata was bad: the merge zeroes the output.
            if (c4 == 0) p.part_lse[idx] = fl ? INFINITY : wts[hr * (NW + 1) + NW];
        } else {
            store_out4(p, s, h0 + hr, 4 * c4, o);
        }
    }
    if (write_partial && p.fuse_merge) {
        int* verdict = reinterpret_cast<int*>(smem + S::kFlags);  // is this the last to arrive
        __syncthreads();
        if (tid == 0) {
            fence_acq_rel_gpu();
            const bool last =
                arrive_last(p.merge_ctr + (int64_t)s * p.num_kv_heads * p.head_tiles + ygrp, p.epoch, nparts);
            if (last) fence_acq_rel_gpu();
            *verdict = last ? 1 : 0;
        }
        __syncthreads();
        if (*verdict) merge_row_partials(p, s, h0, rows, nparts, reinterpret_cast<float*>(smem));
    }
}

template <int NH, bool kRound>
static cudaError_t launch_decode_fp8_t(const DecodeFp8Params& fp, cudaStream_t stream, int* launches) {
    const DecodeParams& p = fp.d;
    constexpr int kSmem = DecodeFp8Smem<8 * NH>::kTotal;
    auto kern = decode_fp8_kernel<NH, kRound>;
    // the attribute is a device's and stays: set on the first call there
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(set.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        set |= bit;
    }
    const unsigned heads = p.num_kv_heads * p.head_tiles;
    const dim3 grid = p.parts_in_x ? dim3(p.max_parts, heads, p.num_seqs) : dim3(heads, p.num_seqs, p.max_parts);
    e = launch_pdl(kern, grid, dim3(kF8Warps * 32), kSmem, stream, fp);
    if (e != cudaSuccess) return e;
    ++*launches;
    return p.split && !p.fuse_merge ? launch_reduce(p, stream, launches) : cudaSuccess;
}

cudaError_t launch_decode_fp8(const DecodeFp8Params& p, cudaStream_t stream, int* launches) {
    const bool wide = decode_head_tile(p.d.group) == 16;
    if (p.d.out_dtype == PKV_FP32)
        return wide ? launch_decode_fp8_t<2, true>(p, stream, launches) : launch_decode_fp8_t<1, true>(p, stream, launches);
    return wide ? launch_decode_fp8_t<2, false>(p, stream, launches) : launch_decode_fp8_t<1, false>(p, stream, launches);
}

}  // namespace pkv
