// rope_append.cu -- the block write with the position rotation, and the norms
// of query and key heads, on the way (paged_kv_append_rope), into 16-bit
// pools and into e4m3 pools with a scale for each (block, KV head).
//
// A 16-lane half-warp holds one head row of 128 values, 8 per lane, as two
// quads of neighbouring values.  In the lanes that rotate, quad A and quad B
// hold the four pairs whose angles are 4i .. 4i+3 of lane i: values 4i .. and
// rot_dim / 2 + 4i .. for pairs (i, i + rot_dim / 2), values 8i .. 8i+7 for
// neighbouring pairs.  Either way a lane has both members of its pairs, so the
// turn needs no exchange, and its cosines and sines are one 16-byte load each.
// The norm's sum of squares is the only exchange, over the 16 lanes.
//
// Bytes, not arithmetic, bound it: each row is read once and written once.
#include <cuda_fp8.h>

#include "pkv_internal.cuh"

namespace pkv {

// Where a lane's two quads sit in a head row.
struct QuadPos {
    int a, b;      // first element of quad A and of quad B
    bool rotates;  // its four pairs are turned
};

template <bool kInter>  // pairs (2i, 2i + 1), else (i, i + rot_dim / 2)
__device__ __forceinline__ QuadPos quad_pos(const RopeParams& p, int i) {
    QuadPos r;
    r.rotates = i < p.rot_dim / 8;
    const bool split = r.rotates && !kInter;
    r.a = split ? 4 * i : 8 * i;
    r.b = split ? p.rot_dim / 2 + 4 * i : 8 * i + 4;
    return r;
}

// Two fp32 values in a register pair, and their arithmetic (one instruction
// for both: with scalar instructions the issue slots, not the memory, bounded
// the write: 97 instructions per row, 67% of the slots, at 4.4 TB/s).
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 pack_f32x2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack_f32x2(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 swapped(f32x2 v) {
    float lo, hi;
    unpack_f32x2(v, lo, hi);
    return pack_f32x2(hi, lo);
}

// A lane's eight values of a head row: quad A in v[0], v[1], quad B in v[2], v[3].
struct Row {
    f32x2 v[4];
};

template <bool kBF16>
__device__ __forceinline__ f32x2 widen(uint32_t w) {
    if constexpr (kBF16) {
        return pack_f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        return pack_f32x2(f.x, f.y);
    }
}

template <bool kBF16>
__device__ __forceinline__ Row widen_row(uint2 a, uint2 b) {
    Row x;
    x.v[0] = widen<kBF16>(a.x), x.v[1] = widen<kBF16>(a.y);
    x.v[2] = widen<kBF16>(b.x), x.v[3] = widen<kBF16>(b.y);
    return x;
}

__device__ __forceinline__ uint2 ldg8(const uint16_t* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }

// What turns the lane's values: y[k] = v[k] c[k] + (the other members of the
// pairs) s[k], the sines negative for the first members.
struct Turn {
    f32x2 c[4], s[4];
};

template <bool kInter>
__device__ __forceinline__ Turn load_turn(const RopeParams& p, const QuadPos& qp, int64_t pos, int i) {
    Turn t;
    if (qp.rotates) {
        const float* row = p.cos_sin + pos * p.rot_dim + 4 * i;
        const float4 c = __ldg(reinterpret_cast<const float4*>(row));
        const float4 s = __ldg(reinterpret_cast<const float4*>(row + p.rot_dim / 2));
        if constexpr (kInter) {
            t.c[0] = pack_f32x2(c.x, c.x), t.c[1] = pack_f32x2(c.y, c.y);
            t.c[2] = pack_f32x2(c.z, c.z), t.c[3] = pack_f32x2(c.w, c.w);
            t.s[0] = pack_f32x2(-s.x, s.x), t.s[1] = pack_f32x2(-s.y, s.y);
            t.s[2] = pack_f32x2(-s.z, s.z), t.s[3] = pack_f32x2(-s.w, s.w);
        } else {
            t.c[0] = t.c[2] = pack_f32x2(c.x, c.y), t.c[1] = t.c[3] = pack_f32x2(c.z, c.w);
            t.s[0] = pack_f32x2(-s.x, -s.y), t.s[1] = pack_f32x2(-s.z, -s.w);
            t.s[2] = pack_f32x2(s.x, s.y), t.s[3] = pack_f32x2(s.z, s.w);
        }
    }
    return t;
}

// Norm (where there is a weight) and turn of a head row, in 32 bits.  All 16
// lanes of the row's half-warp take part (`half` is their mask).
template <bool kInter>
__device__ __forceinline__ void norm_turn(const RopeParams& p, const QuadPos& qp, bool norm, const Row& weight,
                                          const Turn& t, uint32_t half, Row& x) {
    if (norm) {
        f32x2 s2 = mul2(x.v[0], x.v[0]);
#pragma unroll
        for (int k = 1; k < 4; ++k) s2 = fma2(x.v[k], x.v[k], s2);
        float lo, hi;
        unpack_f32x2(s2, lo, hi);
        float ss = lo + hi;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(half, ss, o);
        const float r = rsqrtf(ss * (1.f / kHeadDim) + p.norm_eps);
        const f32x2 rr = pack_f32x2(r, r);
#pragma unroll
        for (int k = 0; k < 4; ++k) x.v[k] = mul2(mul2(x.v[k], rr), weight.v[k]);
    }
    if (qp.rotates) {
        Row y;
        if constexpr (kInter) {
#pragma unroll
            for (int k = 0; k < 4; ++k) y.v[k] = fma2(swapped(x.v[k]), t.s[k], mul2(x.v[k], t.c[k]));
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) y.v[k] = fma2(x.v[k ^ 2], t.s[k], mul2(x.v[k], t.c[k]));
        }
        x = y;
    }
}

// The one rounding of a row to 16 bits.
template <bool kBF16>
__device__ __forceinline__ uint32_t narrow(f32x2 v) {
    float lo, hi;
    unpack_f32x2(v, lo, hi);
    return pack2<kBF16>(lo, hi);
}

template <bool kBF16>
__device__ __forceinline__ void store_row(uint16_t* row, const QuadPos& qp, const Row& x) {
    *reinterpret_cast<uint2*>(row + qp.a) = make_uint2(narrow<kBF16>(x.v[0]), narrow<kBF16>(x.v[1]));
    *reinterpret_cast<uint2*>(row + qp.b) = make_uint2(narrow<kBF16>(x.v[2]), narrow<kBF16>(x.v[3]));
}

// What becomes of a token: padding, an error (recorded once by the caller), or
// its slot and position.
struct Token {
    int64_t slot, pos;
    int err;  // PKV_DEVERR_*, 0: none
};

__device__ __forceinline__ Token token_at(const RopeParams& p, int64_t t) {
    Token k;
    k.slot = __ldg(p.slot_mapping + t);
    k.pos = p.rot_dim > 0 ? __ldg(p.positions + t) : 0;  // loaded beside the slot; padding's is not used
    k.err = 0;
    if (k.slot >= p.num_slots)
        k.err = PKV_DEVERR_SLOT;
    else if (k.slot >= 0 && p.rot_dim > 0 && (k.pos < 0 || k.pos >= p.max_position))
        k.err = PKV_DEVERR_POSITION;
    return k;
}

// slot -> (block, row); 32-bit arithmetic where the slot allows it
__device__ __forceinline__ void split_slot(const RopeParams& p, int64_t slot, int64_t& blk, int& off) {
    if (slot <= 0xffffffffll) {
        const uint32_t b = (uint32_t)slot / (uint32_t)p.block_size;
        blk = b;
        off = (int)((uint32_t)slot - b * (uint32_t)p.block_size);
    } else {
        blk = slot / p.block_size;
        off = (int)(slot - blk * p.block_size);
    }
}

// kRowsPerUnit neighbouring head rows of one token and one kind (queries,
// keys or values), by one half-warp: the rows are loaded together, and share
// the token's slot, angles and weights.  With an 8-bit pool (kQOnly) only the
// queries are done here.
constexpr int kRowsPerUnit = 4;

__host__ __device__ __forceinline__ uint32_t row_units(int heads) { return (heads + kRowsPerUnit - 1) / kRowsPerUnit; }

template <bool kBF16, bool kInter, bool kQOnly>
__device__ __forceinline__ void do_rows(const RopeParams& p, uint32_t unit) {
    const int i = threadIdx.x & 15;
    const uint32_t half = 0xffffu << (threadIdx.x & 16);
    const uint32_t uq = row_units(p.num_q_heads), uk = kQOnly ? 0 : row_units(p.num_kv_heads);
    const uint32_t per_token = uq + 2 * uk;
    const uint32_t tt = unit / per_token;
    uint32_t c = unit - tt * per_token;
    const int64_t t = tt;
    if (t >= p.num_tokens) return;  // uniform over the half-warp
    const int kind = kQOnly || c < uq ? 0 : c < uq + uk ? 1 : 2;  // queries, keys, values
    c -= kind == 0 ? 0 : kind == 1 ? uq : uq + uk;
    const int h0 = (int)c * kRowsPerUnit;
    const int n = min(kRowsPerUnit, (kind == 0 ? p.num_q_heads : p.num_kv_heads) - h0);
    const uint16_t* from = (kind == 0   ? p.q + t * p.q_stride
                            : kind == 1 ? p.k + t * p.k_stride
                                        : p.v + t * p.v_stride) +
                           h0 * kHeadDim;
    const Token tok = token_at(p, t);
    const QuadPos qp = quad_pos<kInter>(p, i);
    // the rows are loaded beside the slot and the position, not after them
    uint2 ra[kRowsPerUnit], rb[kRowsPerUnit];
#pragma unroll
    for (int r = 0; r < kRowsPerUnit; ++r)
        if (r < n) {
            // read once, and q_out may be q: not through the read-only path
            ra[r] = *reinterpret_cast<const uint2*>(from + r * kHeadDim + qp.a);
            rb[r] = *reinterpret_cast<const uint2*>(from + r * kHeadDim + qp.b);
        }
    const uint16_t* wp = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : nullptr;
    Row weight;
    if (wp) weight = widen_row<kBF16>(ldg8(wp + qp.a), ldg8(wp + qp.b));
    if (tok.slot < 0) return;
    uint16_t* to = p.q_out + (t * p.num_q_heads + h0) * kHeadDim;
    int64_t to_step = kHeadDim;
    if (tok.err) {
        if (unit == tt * per_token && i == 0) record_error(p.err, tok.err);
        if (kind == 0)
            for (int r = 0; r < n; ++r) {
                *reinterpret_cast<uint2*>(to + r * kHeadDim + qp.a) = make_uint2(0u, 0u);
                *reinterpret_cast<uint2*>(to + r * kHeadDim + qp.b) = make_uint2(0u, 0u);
            }
        return;
    }
    if (!kQOnly && kind > 0) {
        int64_t blk;
        int off;
        split_slot(p, tok.slot, blk, off);
        to_step = (int64_t)p.block_size * kHeadDim;
        to = static_cast<uint16_t*>(kind == 1 ? p.k_cache : p.v_cache) + (blk * p.num_kv_heads + h0) * to_step +
             off * kHeadDim;
    }
    if (kQOnly || kind < 2) {
        const Turn turn = load_turn<kInter>(p, qp, tok.pos, i);
#pragma unroll
        for (int r = 0; r < kRowsPerUnit; ++r)
            if (r < n) {
                Row x = widen_row<kBF16>(ra[r], rb[r]);
                norm_turn<kInter>(p, qp, wp != nullptr, weight, turn, half, x);
                store_row<kBF16>(to + r * to_step, qp, x);
            }
    } else {  // values pass through as they are
#pragma unroll
        for (int r = 0; r < kRowsPerUnit; ++r)
            if (r < n) {
                *reinterpret_cast<uint2*>(to + r * to_step + qp.a) = ra[r];
                *reinterpret_cast<uint2*>(to + r * to_step + qp.b) = rb[r];
            }
    }
}

constexpr int kRopeThreads = 128;

// Tokens per window of the 8-bit write: one while the warps are fewer than
// this (a step's tokens each start a run of their own), then more, so that
// few warps find nothing to start in a long chunk.
constexpr int64_t kRunWarps = 4096;

template <bool kBF16, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const RopeParams p) {
    pdl_launch_dependents();
    pdl_wait();
    do_rows<kBF16, kInter, false>(p, (uint32_t)((blockIdx.x * (uint32_t)kRopeThreads + threadIdx.x) >> 4));
}

// ---------------------------------------------------------------- 8-bit pool
// The smallest power of two >= a / 448, 2^-64 at least (a >= 0, finite).  448
// = 1.75 * 2^8: the exponent of a less 8, one more when its mantissa is above
// 1.75.
__device__ __forceinline__ float power_scale(float a) {
    const int e = (int)((__float_as_uint(a) + 0x1fffffu) >> 23) - 127 - 8;
    return __uint_as_float((uint32_t)(max(e, -64) + 127) << 23);
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// Two values (at most 448 in magnitude, but for the last bit, or NaN) to two
// e4m3 bytes, nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3_pair(f32x2 v) {
    float lo, hi;
    unpack_f32x2(v, lo, hi);
    uint16_t w;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w) : "f"(hi), "f"(lo));
    return w;
}

__device__ __forceinline__ uint32_t e4m3_quad(f32x2 a, f32x2 b, f32x2 inv) {
    return e4m3_pair(mul2(a, inv)) | (e4m3_pair(mul2(b, inv)) << 16);
}

// The move of a block's held rows 0 .. first - 1 to another scale, by a warp:
// 8 lanes per row, 16 bytes each.
__device__ __forceinline__ void move_rows(uint8_t* tile, int first, float ratio, int lane) {
#pragma unroll 1
    for (int r = lane >> 3; r < first; r += 4) {
        uint4* at = reinterpret_cast<uint4*>(tile + r * kHeadDim) + (lane & 7);
        uint4 v = *at;
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = __half2float(
                    __half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)((w[j] >> (8 * e)) & 0xffu), __NV_E4M3)));
            w[j] = e4m3_quad(pack_f32x2(f[0], f[1]), pack_f32x2(f[2], f[3]), pack_f32x2(ratio, ratio));
        }
        *at = v;
    }
}

// What a run's rows are written with: the block's scale for the largest
// magnitude `a` of rows from row `first` on.  Raises the scale, and moves the
// held rows, where the rule asks for it; returns the scale.  By a whole warp.
__device__ __forceinline__ float settle_scale(const RopeParams& p, float* scale, uint8_t* tile, float a, int first,
                                              int lane) {
    float s = power_scale(a);
    if (first > 0) {
        const float old = *scale;
        if (!(old > 0.f && finite(old))) {
            if (lane == 0) record_error(p.err, PKV_DEVERR_SCALE);
        } else if (a <= 448.f * old) {
            return old;
        } else {
            move_rows(tile, first, old / s, lane);
        }
    }
    __syncwarp();
    if (lane == 0) *scale = s;
    return s;
}

// max(a, the magnitudes of a row); NaN counts for nothing, an infinity does.
__device__ __forceinline__ float top(float a, const Row& x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo, hi;
        unpack_f32x2(x.v[k], lo, hi);
        a = fmaxf(a, fmaxf(fabsf(lo), fabsf(hi)));
    }
    return a;
}

__device__ __forceinline__ float warp_max(float a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

__device__ __forceinline__ void store_e4m3(uint8_t* row, const QuadPos& qp, const Row& x, float inv) {
    const f32x2 ii = pack_f32x2(inv, inv);
    *reinterpret_cast<uint32_t*>(row + qp.a) = e4m3_quad(x.v[0], x.v[1], ii);
    *reinterpret_cast<uint32_t*>(row + qp.b) = e4m3_quad(x.v[2], x.v[3], ii);
}

// Infinities of a row to NaN, as they are stored (and counted).
__device__ __forceinline__ void infinite_to_nan(Row& x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo, hi;
        unpack_f32x2(x.v[k], lo, hi);
        x.v[k] = pack_f32x2(finite(lo) ? lo : NAN, finite(hi) ? hi : NAN);
    }
}

// A run of any shape (padding inside, refused tokens, a slot twice,
// infinities among its values), of keys
// (is_k) or values of KV head h, from its first token t0 on: two passes over
// its tokens, the largest magnitudes, then the bytes.  The common runs take
// write_run below.
template <bool kBF16, bool kInter>
__device__ __noinline__ void write_any_run(const RopeParams& p, int64_t t0, int64_t blk, int h, bool is_k) {
    const int lane = threadIdx.x & 31, i = lane & 15, hf = lane >> 4;
    const uint32_t half = 0xffffu << (lane & 16);
    const QuadPos qp = quad_pos<kInter>(p, i);
    uint8_t* tile = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) +
                    (blk * p.num_kv_heads + h) * p.block_size * kHeadDim;
    Row weight;
    if (p.k_norm) weight = widen_row<kBF16>(ldg8(p.k_norm + qp.a), ldg8(p.k_norm + qp.b));
    float a = 0.f;              // pass 0: the largest finite magnitude; pass 1: the reciprocal of the scale
    int first = p.block_size;  // first row written
    for (int pass = 0; pass < 2; ++pass) {
        for (int64_t c = t0; c < p.num_tokens; c += 32) {
            Token tok;
            tok.slot = -1;
            tok.pos = 0;
            tok.err = 0;
            if (c + lane < p.num_tokens) tok = token_at(p, c + lane);
            const bool real = tok.slot >= 0 && tok.slot < p.num_slots;
            const bool mine = real && tok.slot / p.block_size == blk;
            const uint32_t other = __ballot_sync(0xffffffffu, real && !mine);
            const uint32_t before = other ? (1u << (__ffs(other) - 1)) - 1u : 0xffffffffu;
            if (mine && tok.err && ((before >> lane) & 1u) && pass == 0 && h == 0 && is_k) record_error(p.err, tok.err);
            uint32_t rows = __ballot_sync(0xffffffffu, mine && !tok.err) & before;
            while (rows) {
                const int r0 = __ffs(rows) - 1;
                rows &= rows - 1;
                const int r1 = rows ? __ffs(rows) - 1 : -1;
                rows &= rows - 1;
                const int r = hf ? r1 : r0;
                const int64_t slot = __shfl_sync(0xffffffffu, tok.slot, max(r, 0));
                const int64_t pos = __shfl_sync(0xffffffffu, tok.pos, max(r, 0));
                if (r >= 0) {  // uniform over the half-warp
                    const int64_t t = c + r;
                    const int off = (int)(slot - blk * p.block_size);
                    const uint16_t* row =
                        is_k ? p.k + t * p.k_stride + h * kHeadDim : p.v + t * p.v_stride + h * kHeadDim;
                    Row x = widen_row<kBF16>(ldg8(row + qp.a), ldg8(row + qp.b));
                    if (is_k) {
                        const Turn turn = load_turn<kInter>(p, qp, pos, i);
                        norm_turn<kInter>(p, qp, p.k_norm != nullptr, weight, turn, half, x);
                    }
                    infinite_to_nan(x);
                    if (pass == 0) {
                        first = min(first, off);
                        a = top(a, x);
                    } else {
                        store_e4m3(tile + off * kHeadDim, qp, x, a);
                    }
                }
                __syncwarp();
            }
            if (other) break;
        }
        if (pass == 1) break;
        a = warp_max(a);
        first = __reduce_min_sync(0xffffffffu, first);
        if (first == p.block_size) return;  // every token of the run was refused
        a = 1.f / settle_scale(p, (is_k ? p.k_scales : p.v_scales) + blk * p.num_kv_heads + h, tile, a, first, lane);
    }
}

// A run of `count` neighbouring tokens from t0 on, all of them good; `slot`
// and `pos` are lane l's token t0 + l's.  False, and nothing written, where a
// value is infinite.  Two passes over the rows, kPairs
// pairs of them in flight at a time; the second finds them in the L1.  (All
// rows of a run held in registers took 128 of them at 16 rows and 210 at 32,
// which left too few warps to keep the memory busy.)
template <bool kBF16, bool kInter, int BS>
__device__ __forceinline__ bool write_run(const RopeParams& p, int64_t t0, int count, int64_t slot, int64_t pos,
                                          int64_t blk, int h, bool is_k) {
    constexpr int kPairs = 2;
    const int lane = threadIdx.x & 31, i = lane & 15, hf = lane >> 4;
    const uint32_t half = 0xffffu << (lane & 16);
    QuadPos qp = quad_pos<kInter>(p, i);
    if (!is_k) qp.rotates = false;
    const uint16_t* wp = is_k ? p.k_norm : nullptr;
    Row weight;
    if (wp) weight = widen_row<kBF16>(ldg8(wp + qp.a), ldg8(wp + qp.b));
    const int64_t stride = is_k ? p.k_stride : p.v_stride;
    const uint16_t* from = (is_k ? p.k : p.v) + t0 * stride + h * kHeadDim;
    uint8_t* tile = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) +
                    (blk * p.num_kv_heads + h) * (int64_t)(BS * kHeadDim);
    const int off_l = (int)(slot & (BS - 1));
    const int first = __reduce_min_sync(0xffffffffu, lane < count ? off_l : BS);
    float a = 0.f, inv = 0.f;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int j0 = 0; j0 < count; j0 += 2 * kPairs) {
            uint2 ra[kPairs], rb[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const int r = j0 + 2 * j + hf;
                if (r < count) {
                    ra[j] = ldg8(from + r * stride + qp.a);
                    rb[j] = ldg8(from + r * stride + qp.b);
                }
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                if (j0 + 2 * j < count) {  // uniform over the warp
                    const int r = j0 + 2 * j + hf, rr = min(r, count - 1);
                    const int64_t ps = __shfl_sync(0xffffffffu, pos, rr);
                    const int off = __shfl_sync(0xffffffffu, off_l, rr);
                    if (r < count) {  // uniform over the half-warp
                        Row x = widen_row<kBF16>(ra[j], rb[j]);
                        const Turn turn = load_turn<kInter>(p, qp, ps, i);
                        norm_turn<kInter>(p, qp, wp != nullptr, weight, turn, half, x);
                        if (pass == 0)
                            a = top(a, x);
                        else
                            store_e4m3(tile + off * kHeadDim, qp, x, inv);
                    }
                    __syncwarp();
                }
            }
        }
        if (pass == 0) {
            a = warp_max(a);
            if (a == INFINITY) return false;
            inv = 1.f / settle_scale(p, (is_k ? p.k_scales : p.v_scales) + blk * p.num_kv_heads + h, tile, a, first,
                                     lane);
        }
    }
    return true;
}

// The keys (is_k) or values of KV head h of the runs that start among the
// tokens t0 .. t0 + window - 1, by one warp.  A run is the tokens of one
// block, which stand together in slot_mapping but for padding.
template <bool kBF16, bool kInter, int BS>
__device__ __forceinline__ void do_runs(const RopeParams& p, int64_t t0, int window, int h, bool is_k) {
    const int lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1u;
    Token tok;
    auto look = [&](int64_t t) {  // lane l's token t + l
        tok.slot = -1;
        tok.pos = 0;
        tok.err = 0;
        if (t + lane < p.num_tokens) tok = token_at(p, t + lane);
    };
    auto real = [&] { return tok.slot >= 0 && tok.slot < p.num_slots; };
    const int64_t back = t0 - 1 - lane >= 0 ? __ldg(p.slot_mapping + (t0 - 1 - lane)) : -1;
    look(t0);
    if (lane < window && tok.slot >= p.num_slots && h == 0 && is_k) record_error(p.err, PKV_DEVERR_SLOT);
    uint32_t in = __ballot_sync(0xffffffffu, real());
    if (!(in & (window < 32 ? (1u << window) - 1u : 0xffffffffu))) return;
    // the block of the last token in the pool before t0, over any padding
    int64_t before = -1;
    for (int64_t s = back, c = t0 - 1;;) {
        const uint32_t m = __ballot_sync(0xffffffffu, s >= 0 && s < p.num_slots);
        if (m) {
            before = __shfl_sync(0xffffffffu, s, __ffs(m) - 1) / BS;
            break;
        }
        c -= 32;
        if (c < 0) break;
        s = c - lane >= 0 ? __ldg(p.slot_mapping + (c - lane)) : -1;
    }
    int64_t blk = tok.slot / BS;  // of tokens in the pool
    const uint32_t prior = in & below;
    const int64_t prev = __shfl_sync(0xffffffffu, blk, prior ? 31 - __clz(prior) : 0);
    uint32_t leaders = __ballot_sync(0xffffffffu, lane < window && real() && blk != (prior ? prev : before));
    int at = 0;  // the window in the registers starts at token t0 + at
    while (leaders) {
        const int l = __ffs(leaders) - 1;
        leaders &= leaders - 1;
        const int64_t b = __shfl_sync(0xffffffffu, blk, l - at);
        uint32_t mine, other;
        for (;;) {
            mine = __ballot_sync(0xffffffffu, real() && blk == b);
            other = __ballot_sync(0xffffffffu, real() && blk != b) & ~((1u << (l - at)) - 1u);
            if (other || l == at) break;
            // the run may go on past the window: start it at the run
            at = l;
            look(t0 + at);
            blk = tok.slot / BS;
        }
        mine &= ~((1u << (l - at)) - 1u);
        if (other) mine &= (1u << (__ffs(other) - 1)) - 1u;
        const uint32_t run = mine >> (l - at);
        const int count = __popc(run);
        const bool good = __all_sync(0xffffffffu, !((mine >> lane) & 1u) || tok.err == 0);
        // all tokens of the run are seen: another block follows, or none
        // does, or every row of the block is there (more could only repeat)
        const uint32_t rows =
            __reduce_or_sync(0xffffffffu, (mine >> lane) & 1u ? 1u << (uint32_t)(tok.slot & (BS - 1)) : 0u);
        const bool whole = other || t0 + at + 32 >= p.num_tokens || __popc(rows) == BS;
        // tokens that follow one another, each to a row of its own
        bool done = false;
        if (good && whole && run == (count < 32 ? (1u << count) - 1u : 0xffffffffu) && __popc(rows) == count) {
            const int src = min(lane + l - at, 31);
            done = write_run<kBF16, kInter, BS>(p, t0 + l, count, __shfl_sync(0xffffffffu, tok.slot, src),
                                        __shfl_sync(0xffffffffu, tok.pos, src), b, h, is_k);
        }
        if (!done) write_any_run<kBF16, kInter>(p, t0 + l, b, h, is_k);
        // a leader later in this window is found from its own slot again
        if (leaders && at > 0) {
            at = 0;
            look(t0);
            blk = tok.slot / BS;
        }
    }
}

// kv_blocks of the CTAs write keys and values, a warp for each (window of
// tokens, KV head, keys or values); the others turn the query heads.  The two
// kinds are spread evenly over the grid: the first wait on a chain of loads
// (slots, rows, the scale, rows again), the second stream, and side by side
// they fill each other's pauses.  kv_rate = ceil(kv_blocks 2^32 / CTAs).
template <bool kBF16, bool kInter, int BS>
__global__ void __launch_bounds__(kRopeThreads) rope_fp8_kernel(const RopeParams p, uint64_t kv_rate, int window) {
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t kv = (uint32_t)((blockIdx.x * kv_rate) >> 32);  // CTAs of the first kind before this one
    if ((uint32_t)(((blockIdx.x + 1ull) * kv_rate) >> 32) > kv) {
        const uint32_t w = (kv * (uint32_t)kRopeThreads + threadIdx.x) >> 5;
        const uint32_t lanes = 2 * (uint32_t)p.num_kv_heads;
        const uint32_t win = w / lanes, k = w - win * lanes;
        const int64_t t0 = (int64_t)win * window;
        if (t0 < p.num_tokens) do_runs<kBF16, kInter, BS>(p, t0, window, (int)(k >> 1), (k & 1u) == 0);
    } else {
        do_rows<kBF16, kInter, true>(p, ((blockIdx.x - kv) * (uint32_t)kRopeThreads + threadIdx.x) >> 4);
    }
}

template <bool kBF16, bool kInter>
static cudaError_t launch_rope_append_t(const RopeParams& p, bool fp8, cudaStream_t stream) {
    const int64_t units =
        p.num_tokens * ((int64_t)row_units(p.num_q_heads) + (fp8 ? 0 : 2 * (int64_t)row_units(p.num_kv_heads)));
    const int64_t row_blocks = (units + kRopeThreads / 16 - 1) / (kRopeThreads / 16);
    if (!fp8) return launch_pdl(rope_rows_kernel<kBF16, kInter>, dim3((unsigned)row_blocks), dim3(kRopeThreads), 0, stream, p);
    int window = 1;
    while (window < 16 && p.num_tokens * p.num_kv_heads / window > kRunWarps) window *= 2;
    const int64_t warps = (p.num_tokens + window - 1) / window * 2 * p.num_kv_heads;
    const int64_t kv_blocks = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    auto kern = p.block_size == 16 ? rope_fp8_kernel<kBF16, kInter, 16> : rope_fp8_kernel<kBF16, kInter, 32>;
    const uint64_t blocks = (uint64_t)(kv_blocks + row_blocks);
    const uint64_t kv_rate = (((uint64_t)kv_blocks << 32) + blocks - 1) / blocks;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(kRopeThreads), 0, stream, p, kv_rate, window);
}

cudaError_t launch_rope_append(const RopeParams& p, int dtype, bool fp8, cudaStream_t stream, int* launches) {
    const cudaError_t e =
        dtype == PKV_BF16
            ? (p.interleaved ? launch_rope_append_t<true, true>(p, fp8, stream) : launch_rope_append_t<true, false>(p, fp8, stream))
            : (p.interleaved ? launch_rope_append_t<false, true>(p, fp8, stream) : launch_rope_append_t<false, false>(p, fp8, stream));
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace pkv
