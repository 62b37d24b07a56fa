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
// accumulate in O directly.  (Adding each unit's product, times vs, to O took
// 32 more multiply-adds per unit, and a wait for the products' end.)
//
// A unit of work is 16 tokens of one (block, KV head) tile: 2 KiB of K and 2
// KiB of V.  The warps of a CTA take units in turn, each through a ring of its
// own in shared memory, filled by 16-byte asynchronous copies.  Every lane
// copies the very bytes that it will use, so a stage needs no barrier between
// lanes but for its two scales:
//   K: rows g and g + 8 (g = lane / 4), 16-byte chunks t and t + 4 of the row
//      (t = lane % 4): full 32-byte sectors, and with the query held in the
//      same order of dims, word j of a chunk is the A operand of k-step j;
//   V: tokens 2t, 2t + 1, 2t + 8, 2t + 9, chunk g of the row: byte pairs of
//      two tokens are interleaved (PRMT) to make the A operand of V^T, and a
//      lane ends up with 16 neighbouring dims of the output.
// TMA copies would be 2 KiB each here, which the SM's TMA unit takes some 75
// cycles for, 150 of the about 180 that a unit may cost at full bandwidth.
#include "decode_common.cuh"

namespace pkv {

constexpr int kF8Warps = 4;             // consumer warps per CTA, each with a ring of its own
constexpr int kF8Stages = 3;            // units in flight per warp
constexpr int kF8CtasPerSm = 4;
constexpr float kF8Lift = 7.f;          // log2; kLazyMargin + kF8Lift stays below fp16's 2^16
constexpr int kF8UnitBytes = 2 * 16 * kHeadDim;       // 16 tokens of K and V
constexpr int kF8StageBytes = kF8UnitBytes + 16;      // and their two scales

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

template <int HT>
struct DecodeFp8Smem {
    static constexpr int kRing = kF8Warps * kF8Stages * kF8StageBytes;
    // per-warp rows, per-warp (m, l, vref), per-row merge weights and lse
    static constexpr int kRed = kF8Warps * HT * kRedStride * 4 + kF8Warps * HT * 3 * 4 + HT * (kF8Warps + 1) * 4;
    static constexpr int kFlags = ((kRing > kRed ? kRing : kRed) + 15) / 16 * 16;
    static constexpr int kTotal = kFlags + 16;
};

// NH: 8-head n-tiles per CTA (1: up to 8 query heads of a group, 2: up to 16).
template <int NH>
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
    const int tok0 = part * p.partition_size;
    const int len = min(L - tok0, p.partition_size);  // tokens of this partition
    const int nunits = (len + 15) / 16;
    const int subs = p.block_size >> 4;  // units per block: 1 or 2
    const bool write_partial = p.split && nparts > 1;

    int* flags = reinterpret_cast<int*>(smem + S::kFlags);  // [0]: bad block id, [1]: last-arrival verdict
    if (tid == 0) flags[0] = 0;
    __syncthreads();

    // ---- this warp's units: warp, warp + NW, ...
    const int mine = nunits > warp ? (nunits - 1 - warp) / NW + 1 : 0;
    const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks_per_seq + tok0 / p.block_size;
    const uint64_t policy = l2_policy_evict_first();
    const int64_t tile_bytes = (int64_t)p.block_size * D;
    uint8_t* ring = smem + warp * (NST * kF8StageBytes);
    const uint32_t ring_sa = smem_addr(ring);

    int ids = 0;
    // Block id of the warp's n-th unit: 32 are read at a time, a lane each.
    auto load_ids = [&](int n0) {
        const int n = n0 + lane;
        int id = 0;
        bool bad = false;
        if (n < mine) {
            id = __ldg(table + (warp + n * NW) / subs);
            bad = id < 0 || (int64_t)id >= p.num_blocks;
            if (bad) id = 0;  // the output is zeroed below
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) {
            atomicOr(flags, 1);
            record_error(p.err, PKV_DEVERR_BLOCK_ID);
        }
        ids = id;
    };
    const uint8_t* kbase = fp.k8 + kvh * tile_bytes + g * D + t * 16;
    const uint8_t* vbase = fp.v8 + kvh * tile_bytes + 2 * t * D + g * 16;
    const float* sbase = (lane ? fp.v_scales : fp.k_scales) + kvh;
    const int64_t block_bytes = p.num_kv_heads * tile_bytes;
    auto issue = [&](int n, int st) {  // unit n into stage st
        if (n < mine) {
            if ((n & 31) == 0) load_ids(n);
            const int id = __shfl_sync(0xffffffffu, ids, n & 31);
            const int sub = (warp + n * NW) & (subs - 1);
            const int64_t off = id * block_bytes + sub * (16 * D);
            const uint8_t* kr = kbase + off;
            const uint8_t* vr = vbase + off;
            const uint32_t sa = ring_sa + st * kF8StageBytes;
            const uint32_t dst = sa + lane * 16;
            cp_async16(dst, kr, policy);
            cp_async16(dst + 512, kr + 64, policy);
            cp_async16(dst + 1024, kr + 8 * D, policy);
            cp_async16(dst + 1536, kr + 8 * D + 64, policy);
            cp_async16(dst + 2048, vr, policy);
            cp_async16(dst + 2560, vr + D, policy);
            cp_async16(dst + 3072, vr + 8 * D, policy);
            cp_async16(dst + 3584, vr + 9 * D, policy);
            if (lane < 2) cp_async4(sa + kF8UnitBytes + 4 * lane, sbase + (int64_t)id * p.num_kv_heads);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int n = 0; n < NST - 1; ++n) issue(n, n);

    // ---- the query: head 8n + g, dims of chunk t (k-steps 0-3) and t + 4 (4-7)
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
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(qr + (c >> 1) * 64 + 16 * t + (c & 1) * 8));
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

    int st = 0, st_in = NST - 1;  // stage of unit n and of unit n + NST - 1
    for (int n = 0; n < mine; ++n) {
        cp_async_wait<NST - 2>();
        __syncwarp();  // the scales' copies of lanes 0 and 1
        issue(n + NST - 1, st_in);
        const uint8_t* stage = ring + st * kF8StageBytes;
        st_in = st;  // this unit's stage is free when it has been used
        st = st + 1 == NST ? 0 : st + 1;
        const uint4* own = reinterpret_cast<const uint4*>(stage) + lane;
        const float2 scl = *reinterpret_cast<const float2*>(stage + kF8UnitBytes);  // ks, vs
        const int valid = min(16, len - 16 * (warp + n * NW));  // >= 1

        // ---- S^T = K8 Q^T: tokens g, g + 8 x heads 2t, 2t + 1, in two sums
        float sc[NH][4], sc2[NH][4];
#pragma unroll
        for (int m = 0; m < NH; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[m][e] = sc2[m][e] = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint4 ka = own[32 * c], kb = own[32 * (c + 2)];
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t af[4];
                e4m3x4_to_f16(wa[j], af[0], af[2]);
                e4m3x4_to_f16(wb[j], af[1], af[3]);
#pragma unroll
                for (int m = 0; m < NH; ++m)
                    mma_16816<false>((j & 1) ? sc2[m] : sc[m], af, qf[m][4 * c + j][0], qf[m][4 * c + j][1]);
            }
        }
        uint32_t vw[4][4];  // V8: tokens 2t, 2t + 1, 2t + 8, 2t + 9, dims 16g .. 16g + 15
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint4 w = own[32 * (4 + r)];
            vw[r][0] = w.x, vw[r][1] = w.y, vw[r][2] = w.z, vw[r][3] = w.w;
        }
#pragma unroll
        for (int m = 0; m < NH; ++m) {
            const float f0 = qs[m][0] * scl.x, f1 = qs[m][1] * scl.x;
            sc[m][0] = (sc[m][0] + sc2[m][0]) * f0;
            sc[m][1] = (sc[m][1] + sc2[m][1]) * f1;
            sc[m][2] = (sc[m][2] + sc2[m][2]) * f0;
            sc[m][3] = (sc[m][3] + sc2[m][3]) * f1;
        }
        if (valid < 16) {
            // rows past the context may hold anything (even NaN): their
            // scores become -inf, their V rows zeros
#pragma unroll
            for (int m = 0; m < NH; ++m) {
                if (g >= valid) sc[m][0] = sc[m][1] = -INFINITY;
                if (g + 8 >= valid) sc[m][2] = sc[m][3] = -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (2 * t + (r & 1) + 8 * (r >> 1) >= valid) vw[r][0] = vw[r][1] = vw[r][2] = vw[r][3] = 0u;
        }
        // ---- online softmax; the maximum is raised, and O and l rescaled,
        // only when a score passes it by more than kLazyMargin
        bool need = false;
#pragma unroll
        for (int m = 0; m < NH; ++m)
            need |= fmaxf(sc[m][0], sc[m][2]) > a.m[m][0] + kLazyMargin ||
                    fmaxf(sc[m][1], sc[m][3]) > a.m[m][1] + kLazyMargin;
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int m = 0; m < NH; ++m)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = fmaxf(sc[m][c], sc[m][c + 2]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const float mn = fmaxf(a.m[m][c], mx);
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
        float ratio = scl.y * vinv;  // the same in every lane
        if (!(fabsf(ratio) <= 1.f && fabsf(ratio) >= 0x1p-6f)) {
            if (vref == 0.f) {
                vref = scl.y;  // a scale of zero adds nothing and sets nothing
                vinv = vref == 0.f ? 0.f : 1.f / vref;
                ratio = vref == 0.f ? 0.f : 1.f;
            } else if (!(fabsf(ratio) < 0x1p-60f)) {
                // (a scale 2^-60 times the unit or less is folded as it is:
                // what it adds is lost beside the unit, and O times the
                // inverse could leave fp32's range)
                const float f = vref / scl.y;
#pragma unroll
                for (int m = 0; m < NH; ++m)
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) a.o[mt][m][e] *= f;
                vref = scl.y;
                vinv = 1.f / vref;
                ratio = 1.f;
            }
        }
        uint32_t ph[NH][2], pl[NH][2];
#pragma unroll
        for (int m = 0; m < NH; ++m) {
            const float m0 = a.m[m][0] == -INFINITY ? 0.f : a.m[m][0], m1 = a.m[m][1] == -INFINITY ? 0.f : a.m[m][1];
            float p0 = exp2_ftz(sc[m][0] - m0 + kF8Lift), p1 = exp2_ftz(sc[m][1] - m1 + kF8Lift);
            float p2 = exp2_ftz(sc[m][2] - m0 + kF8Lift), p3 = exp2_ftz(sc[m][3] - m1 + kF8Lift);
            a.l[m][0] += p0 + p2;
            a.l[m][1] += p1 + p3;
            p0 *= ratio, p1 *= ratio, p2 *= ratio, p3 *= ratio;
            float r0, r1, r2, r3;
            const uint32_t h01 = pack2<false>(p0, p1, r0, r1), h23 = pack2<false>(p2, p3, r2, r3);
            ph[m][0] = movmatrix_trans(h01);
            ph[m][1] = movmatrix_trans(h23);
            pl[m][0] = movmatrix_trans(pack2<false>(p0 - r0, p1 - r1));
            pl[m][1] = movmatrix_trans(pack2<false>(p2 - r2, p3 - r3));
        }
        // ---- O^T += V8^T P^T: tokens 2t, 2t + 1 (k 0-7), 2t + 8, 2t + 9
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            const int j = mt >> 1;
            const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;  // bytes 2, 3 or 0, 1 of both tokens, paired
            uint32_t af[4];
            e4m3x4_to_f16(__byte_perm(vw[0][j], vw[1][j], sel), af[0], af[1]);
            e4m3x4_to_f16(__byte_perm(vw[2][j], vw[3][j], sel), af[2], af[3]);
#pragma unroll
            for (int m = 0; m < NH; ++m) {
                mma_16816<false>(a.o[mt][m], af, ph[m][0], ph[m][1]);
                mma_16816<false>(a.o[mt][m], af, pl[m][0], pl[m][1]);
            }
        }
    }
    acc_finish(a);
    cp_async_wait<0>();
    __syncthreads();  // every ring is free: its memory takes the warps' states

    // ---- merge the warps' states, as the decode kernel does
    const int fl = flags[0];
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
        for (int w = 0; w < NW; ++w) wts[tid * (NW + 1) + w] = f[w] * inv * ml[(w * HT + tid) * 3 + 2];
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
                const float ww = wts[hr * (NW + 1) + w];
                const float4 r = *reinterpret_cast<const float4*>(red + (w * HT + hr) * kRedStride + 4 * c4);
                o.x += ww * r.x;
                o.y += ww * r.y;
                o.z += ww * r.z;
                o.w += ww * r.w;
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
        __syncthreads();
        if (tid == 0) {
            fence_acq_rel_gpu();
            const bool last =
                arrive_last(p.merge_ctr + (int64_t)s * p.num_kv_heads * p.head_tiles + ygrp, p.epoch, nparts);
            if (last) fence_acq_rel_gpu();
            flags[1] = last ? 1 : 0;
        }
        __syncthreads();
        if (flags[1]) merge_row_partials(p, s, h0, rows, nparts, reinterpret_cast<float*>(smem));
    }
}

template <int NH>
static cudaError_t launch_decode_fp8_t(const DecodeFp8Params& fp, cudaStream_t stream, int* launches) {
    const DecodeParams& p = fp.d;
    constexpr int kSmem = DecodeFp8Smem<8 * NH>::kTotal;
    auto kern = decode_fp8_kernel<NH>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const unsigned heads = p.num_kv_heads * p.head_tiles;
    const dim3 grid = p.parts_in_x ? dim3(p.max_parts, heads, p.num_seqs) : dim3(heads, p.num_seqs, p.max_parts);
    e = launch_pdl(kern, grid, dim3(kF8Warps * 32), kSmem, stream, fp);
    if (e != cudaSuccess) return e;
    ++*launches;
    return p.split && !p.fuse_merge ? launch_reduce(p, stream, launches) : cudaSuccess;
}

cudaError_t launch_decode_fp8(const DecodeFp8Params& p, cudaStream_t stream, int* launches) {
    return decode_head_tile(p.d.group) == 16 ? launch_decode_fp8_t<2>(p, stream, launches)
                                             : launch_decode_fp8_t<1>(p, stream, launches);
}

}  // namespace pkv
