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
// Bytes bound the 16-bit write: each row is read once and written once, 16384
// normed tokens of 64/8 heads (680 MB) in 103.8 us, 6.5 TB/s.  The 8-bit write
// waits on more: a block's scale needs all of its new rows before the first
// byte, a chain of loads and exchanges for each run of tokens: 16384 tokens of
// 32/8 heads (378 MB) in 70.5 us, 5.4 TB/s.
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
// its slot and position (32 bits hold both: the host refuses larger pools and
// tables).
struct Token {
    int slot, pos;  // slot -1: not in the pool
    int err;        // PKV_DEVERR_*, 0: none
};

__device__ __forceinline__ Token token_at(const RopeParams& p, int64_t t) {
    const int64_t slot = __ldg(p.slot_mapping + t);
    const int64_t pos = p.rot_dim > 0 ? __ldg(p.positions + t) : 0;  // loaded beside the slot; padding's is not used
    Token k;
    k.slot = (int)slot;
    k.pos = (int)pos;
    k.err = 0;
    if (slot >= p.num_slots) {
        k.slot = -1;
        k.err = PKV_DEVERR_SLOT;
    } else if (slot < 0) {
        k.slot = -1;
    } else if (p.rot_dim > 0 && (pos < 0 || pos >= p.max_position)) {
        k.err = PKV_DEVERR_POSITION;
    }
    return k;
}

// R neighbouring head rows of one token and one kind (queries,
// keys or values), by one half-warp: the rows are loaded together, and share
// the token's slot, angles and weights.  With an 8-bit pool (kQOnly) only the
// queries are done here.  R = 8 rows ask more of the memory at a time, 4 fill
// the GPU with less work: 103.8 against 117.0 us for 16384 tokens of 64/8
// heads, 16.1 against 15.8 us for 1537 of 40/40, 2.6 against 2.0 us for 64 of
// 32/8.
__host__ __device__ __forceinline__ uint32_t row_units(int heads, int R) { return (heads + R - 1) / R; }
constexpr int64_t kManyUnits = 65536;  // units of 8 rows from which on R = 8

template <bool kBF16, bool kInter, bool kQOnly, int R>
__device__ __forceinline__ void do_rows(const RopeParams& p, uint32_t unit) {
    const int i = threadIdx.x & 15;
    const uint32_t half = 0xffffu << (threadIdx.x & 16);
    const uint32_t uq = row_units(p.num_q_heads, R), uk = kQOnly ? 0 : row_units(p.num_kv_heads, R);
    const uint32_t per_token = uq + 2 * uk;
    const uint32_t tt = unit / per_token;
    uint32_t c = unit - tt * per_token;
    const int64_t t = tt;
    if (t >= p.num_tokens) return;  // uniform over the half-warp
    const int kind = kQOnly || c < uq ? 0 : c < uq + uk ? 1 : 2;  // queries, keys, values
    c -= kind == 0 ? 0 : kind == 1 ? uq : uq + uk;
    const int h0 = (int)c * R;
    const int n = min(R, (kind == 0 ? p.num_q_heads : p.num_kv_heads) - h0);
    const uint16_t* from = (kind == 0   ? p.q + t * p.q_stride
                            : kind == 1 ? p.k + t * p.k_stride
                                        : p.v + t * p.v_stride) +
                           h0 * kHeadDim;
    const int64_t slot = __ldg(p.slot_mapping + t);
    const int64_t pos = p.rot_dim > 0 ? __ldg(p.positions + t) : 0;
    const QuadPos qp = quad_pos<kInter>(p, i);
    // the rows are loaded beside the slot and the position, not after them
    uint2 ra[R], rb[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r < n) {
            // read once, and q_out may be q: not through the read-only path
            ra[r] = *reinterpret_cast<const uint2*>(from + r * kHeadDim + qp.a);
            rb[r] = *reinterpret_cast<const uint2*>(from + r * kHeadDim + qp.b);
        }
    const uint16_t* wp = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : nullptr;
    Row weight;
    if (wp) weight = widen_row<kBF16>(ldg8(wp + qp.a), ldg8(wp + qp.b));
    if (slot < 0) return;  // padding
    uint16_t* to = p.q_out + (t * p.num_q_heads + h0) * kHeadDim;
    int64_t to_step = kHeadDim;
    const bool out = slot >= p.num_slots;
    if (out || (p.rot_dim > 0 && (pos < 0 || pos >= p.max_position))) {
        if (unit == tt * per_token && i == 0) record_error(p.err, out ? PKV_DEVERR_SLOT : PKV_DEVERR_POSITION);
        if (kind == 0)
            for (int r = 0; r < n; ++r) {
                *reinterpret_cast<uint2*>(to + r * kHeadDim + qp.a) = make_uint2(0u, 0u);
                *reinterpret_cast<uint2*>(to + r * kHeadDim + qp.b) = make_uint2(0u, 0u);
            }
        return;
    }
    if (!kQOnly && kind > 0) {
        const uint32_t blk = (uint32_t)slot / (uint32_t)p.block_size, off = (uint32_t)slot - blk * p.block_size;
        to_step = (int64_t)p.block_size * kHeadDim;
        to = static_cast<uint16_t*>(kind == 1 ? p.k_cache : p.v_cache) + ((int64_t)blk * p.num_kv_heads + h0) * to_step +
             off * kHeadDim;
    }
    if (kQOnly || kind < 2) {
        const Turn turn = load_turn<kInter>(p, qp, pos, i);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r < n) {
                Row x = widen_row<kBF16>(ra[r], rb[r]);
                norm_turn<kInter>(p, qp, wp != nullptr, weight, turn, half, x);
                store_row<kBF16>(to + r * to_step, qp, x);
            }
    } else {  // values pass through as they are
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r < n) {
                *reinterpret_cast<uint2*>(to + r * to_step + qp.a) = ra[r];
                *reinterpret_cast<uint2*>(to + r * to_step + qp.b) = rb[r];
            }
    }
}

constexpr int kRopeThreads = 128;

template <bool kBF16, bool kInter, int R>
__global__ void __launch_bounds__(kRopeThreads, R == 8 ? 7 : 8) rope_rows_kernel(const RopeParams p) {
    pdl_launch_dependents();
    pdl_wait();
    do_rows<kBF16, kInter, false, R>(p, blockIdx.x * (kRopeThreads / 16) + (threadIdx.x >> 4));
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
// magnitude `a` of rows from row `first` on, `old` being the scale so far.  By
// a whole warp; the one with `writes` sets the scale, and moves the held rows
// where it is raised.
__device__ __forceinline__ float settle_scale(const RopeParams& p, float* scale, float old, uint8_t* tile, float a,
                                              int first, bool writes) {
    const int lane = threadIdx.x & 31;
    const float s = power_scale(a);
    if (first > 0) {
        if (!(old >= 0x1p-126f && finite(old))) {  // (a smaller one has no finite reciprocal)
            if (writes && lane == 0) record_error(p.err, PKV_DEVERR_SCALE);
        } else if (a <= 448.f * old) {
            return old;
        } else if (writes) {
            move_rows(tile, first, old / s, lane);
        }
    }
    if (writes && lane == 0) *scale = s;
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

// A run of any shape (padding inside, refused tokens, a slot twice, infinities
// among its values), of keys (is_k) or values of KV head h, from its first
// token t0 on: two passes over its tokens, the largest magnitude, then the
// bytes.  The common runs take write_run below.
template <bool kBF16, bool kInter>
__device__ __noinline__ void write_any_run(const RopeParams& p, int64_t t0, int blk, int h, bool is_k) {
    const int lane = threadIdx.x & 31, i = lane & 15, hf = lane >> 4;
    const uint32_t half = 0xffffu << (lane & 16);
    const QuadPos qp = quad_pos<kInter>(p, i);
    uint8_t* tile = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) +
                    ((int64_t)blk * p.num_kv_heads + h) * p.block_size * kHeadDim;
    Row weight;
    if (p.k_norm) weight = widen_row<kBF16>(ldg8(p.k_norm + qp.a), ldg8(p.k_norm + qp.b));
    float a = 0.f;              // pass 0: the largest finite magnitude; pass 1: the reciprocal of the scale
    int first = p.block_size;  // first row written
    for (int pass = 0; pass < 2; ++pass) {
        for (int64_t c = t0; c < p.num_tokens; c += 32) {
            Token tok;
            tok.slot = -1, tok.pos = 0, tok.err = 0;
            if (c + lane < p.num_tokens) tok = token_at(p, c + lane);
            const bool real = tok.slot >= 0;
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
                const int slot = __shfl_sync(0xffffffffu, tok.slot, max(r, 0));
                const int pos = __shfl_sync(0xffffffffu, tok.pos, max(r, 0));
                if (r >= 0) {  // uniform over the half-warp
                    const int64_t t = c + r;
                    const int off = slot - blk * p.block_size;
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
        float* scale = (is_k ? p.k_scales : p.v_scales) + (int64_t)blk * p.num_kv_heads + h;
        const float old = first > 0 ? *scale : 0.f;
        __syncwarp();  // read by all before it is set
        a = 1.f / settle_scale(p, scale, old, tile, a, first, true);
    }
}

// A run of `count` <= BS neighbouring tokens from t0 on, all of them good, of
// keys (kKeys) or values of KV head h; `off` and `pos` are lane l's token t0 +
// l's row and position.  False, and nothing written, where a value is
// infinite.
//
// A warp has 16 rows of a run at most.  They are copied to shared memory
// (`stage`, the warp's own 8 KiB) together, turned there into 32-bit values,
// which take the place of the rows, and become bytes once the largest
// magnitude is known.  (Turning them twice cost 17 us more for 16384 tokens of
// 8 KV heads; kept in registers they spilled; a CTA for each window, its runs'
// magnitudes meeting in shared memory, took 61 us for keys and values against
// 45.)  The two warps of a 32-row block meet at a barrier, `meet` is where they
// leave their magnitudes.
template <bool kBF16, bool kInter, bool kKeys, int BS>
__device__ __forceinline__ bool write_run(const RopeParams& p, uint4* stage, float* meet, int64_t t0, int count,
                                          int off_l, int pos_l, int first, int blk, int h) {
    const int lane = threadIdx.x & 31, i = lane & 15, hf = lane >> 4, warp = threadIdx.x >> 5;
    const int r0 = BS == 32 ? 16 * (warp & 1) : 0;  // the warp's first row
    const int mine = min(count - r0, 16);           // its rows (none: <= 0)
    QuadPos qp = quad_pos<kInter>(p, i);
    if (!kKeys) qp.rotates = false, qp.a = 8 * i, qp.b = 8 * i + 4;
    const int64_t stride = kKeys ? p.k_stride : p.v_stride;
    const uint16_t* from = (kKeys ? p.k : p.v) + (t0 + r0 + hf) * stride + h * kHeadDim + 8 * i;
    const uint32_t to = smem_addr(stage + lane);
    __syncwarp();  // the warp is done with what the stage held
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (2 * j + hf < mine)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 512 * j), "l"(from + 2 * j * stride)
                         : "memory");
    float* scale = (kKeys ? p.k_scales : p.v_scales) + (int64_t)blk * p.num_kv_heads + h;
    const float old = first > 0 ? *scale : 0.f;
    const bool norm = kKeys && p.k_norm;
    Row weight;
    if (norm) weight = widen_row<kBF16>(ldg8(p.k_norm + qp.a), ldg8(p.k_norm + qp.b));
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();  // every lane has read `old`, too
    // Pair j of rows lies in bytes 512j .. 512j + 511 of the stage, its 32-bit
    // values go to 1024j .. 1024j + 1023: from the last pair down, over rows
    // that are done.  An odd last row is done by both halves.
    float a = 0.f;
#pragma unroll 1
    for (int j = (mine - 1) >> 1; j >= 0; --j) {
        const int r = min(2 * j + hf, mine - 1);
        const uint16_t* row = reinterpret_cast<const uint16_t*>(stage) + r * kHeadDim;
        Row y = widen_row<kBF16>(*reinterpret_cast<const uint2*>(row + qp.a),
                                 *reinterpret_cast<const uint2*>(row + qp.b));
        if constexpr (kKeys) {
            const Turn turn = load_turn<kInter>(p, qp, __shfl_sync(0xffffffffu, pos_l, r0 + r), i);
            norm_turn<kInter>(p, qp, norm, weight, turn, 0xffffffffu, y);
        }
        a = top(a, y);
        __syncwarp();
        ulonglong2* at = reinterpret_cast<ulonglong2*>(stage + 64 * j + lane);
        at[0] = make_ulonglong2(y.v[0], y.v[1]);
        at[32] = make_ulonglong2(y.v[2], y.v[3]);
        __syncwarp();
    }
    a = warp_max(a);
    if constexpr (BS == 32) {
        if (lane == 0) meet[warp & 1] = a;
        asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");
        a = fmaxf(meet[0], meet[1]);
    }
    if (a == INFINITY) return false;
    uint8_t* tile = static_cast<uint8_t*>(kKeys ? p.k_cache : p.v_cache) +
                    ((int64_t)blk * p.num_kv_heads + h) * (BS * kHeadDim);
    const float inv = 1.f / settle_scale(p, scale, old, tile, a, first, r0 == 0);
#pragma unroll 1
    for (int j = 0; 2 * j < mine; ++j) {
        const ulonglong2* at = reinterpret_cast<const ulonglong2*>(stage + 64 * j + lane);
        const ulonglong2 lo = at[0], hi = at[32];
        Row y;
        y.v[0] = lo.x, y.v[1] = lo.y, y.v[2] = hi.x, y.v[3] = hi.y;
        store_e4m3(tile + __shfl_sync(0xffffffffu, off_l, r0 + min(2 * j + hf, mine - 1)) * kHeadDim, qp, y, inv);
    }
    return true;
}

// The keys and values of some KV heads (items item0 .. item1 - 1, 32 at most:
// item 2h is the keys of head h, 2h + 1 its values) of the runs that start
// among the tokens t0 .. t0 + window - 1 (window <= 31), by one warp (BS = 16)
// or two that go through it together.  A run is the tokens of one block, which
// stand together in slot_mapping but for padding.  The warp looks at 64 tokens,
// from the one before t0 on, so that a run ends among them (but for long
// padding inside, or slots named twice).  The search takes 3 us of a call.
template <bool kBF16, bool kInter, int BS>
__device__ __forceinline__ void do_runs(const RopeParams& p, uint4* stage, float (*meet)[2], int64_t t0, int window,
                                        int item0, int item1) {
    const int lane = threadIdx.x & 31;
    const bool second = BS == 32 && ((threadIdx.x >> 5) & 1);  // the second warp of two: leaves the rest to the first
    int turn = 0;                                              // which of the meeting places is next
    Token tok[2];  // tokens t0 - 1 + lane and t0 + 31 + lane: bits lane and 32 + lane below
    uint32_t in[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int64_t t = t0 - 1 + 32 * u + lane;
        tok[u].slot = -1, tok[u].pos = 0, tok[u].err = 0;
        if (t >= 0 && t < p.num_tokens) tok[u] = token_at(p, t);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) in[u] = __ballot_sync(0xffffffffu, tok[u].slot >= 0);
    if (tok[0].err == PKV_DEVERR_SLOT && lane >= 1 && lane <= window && item0 == 0 && !second)
        record_error(p.err, PKV_DEVERR_SLOT);
    const uint32_t inside = (2u << window) - 2u;
    if (!(in[0] & inside)) return;
    // the block of the last token in the pool before t0, over any padding
    int before = __shfl_sync(0xffffffffu, tok[0].slot, 0) / BS;
    if (!(in[0] & 1u)) {
        before = -1;
        for (int64_t c = t0 - 2; c >= 0; c -= 32) {
            const int64_t s = c - lane >= 0 ? __ldg(p.slot_mapping + (c - lane)) : -1;
            const uint32_t m = __ballot_sync(0xffffffffu, s >= 0 && s < p.num_slots);
            if (m) {
                before = __shfl_sync(0xffffffffu, (int)s, __ffs(m) - 1) / BS;
                break;
            }
        }
    }
    uint32_t starts[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int blk = tok[u].slot / BS;
        const uint32_t prior = in[u] & ((1u << lane) - 1u);
        const int prev = __shfl_sync(0xffffffffu, blk, prior ? 31 - __clz(prior) : 0);
        starts[u] = __ballot_sync(0xffffffffu, tok[u].slot >= 0 && blk != (prior ? prev : before) && (u || lane));
        if (in[u]) before = __shfl_sync(0xffffffffu, blk, 31 - __clz(in[u]));
    }
    const uint64_t leaders = starts[0] | (uint64_t)starts[1] << 32, present = in[0] | (uint64_t)in[1] << 32;
    for (uint32_t own = starts[0] & inside; own; own &= own - 1u) {
        const int x = __ffs(own) - 1;
        const uint64_t later = leaders & ~((2ull << x) - 1ull);
        const uint64_t upto = later ? (later & (0ull - later)) - 1ull : ~0ull;  // bits below the next run's first
        const uint64_t run = (present & upto) >> x;
        const int count = __popcll(run);
        // lane l: the run's token l
        const int src = (x + lane) & 31;
        const bool hi = x + lane >= 32;
        const int sl0 = __shfl_sync(0xffffffffu, tok[0].slot, src), sl1 = __shfl_sync(0xffffffffu, tok[1].slot, src);
        const int ps0 = __shfl_sync(0xffffffffu, tok[0].pos, src), ps1 = __shfl_sync(0xffffffffu, tok[1].pos, src);
        const int er0 = __shfl_sync(0xffffffffu, tok[0].err, src), er1 = __shfl_sync(0xffffffffu, tok[1].err, src);
        const bool good = __all_sync(0xffffffffu, lane >= count || (hi ? er1 : er0) == 0);
        const int slot = hi ? sl1 : sl0, pos = hi ? ps1 : ps0, off = slot & (BS - 1);
        const int blk = __shfl_sync(0xffffffffu, slot, 0) / BS;
        uint32_t left = 0xffffffffu;  // items that write_any_run has to do
        // neighbouring tokens, the run's end in sight
        if (good && count <= BS && run == (1ull << count) - 1ull && (later || t0 + 63 >= p.num_tokens)) {
            const int first = __reduce_min_sync(0xffffffffu, lane < count ? off : BS);
#pragma unroll 1
            for (int item = item0; item < item1; ++item) {
                turn ^= 1;  // one meeting's barrier lies between two uses of a place
                const bool done =
                    (item & 1) ? write_run<kBF16, kInter, false, BS>(p, stage, meet[turn], t0 + x - 1, count, off, pos,
                                                                     first, blk, item >> 1)
                               : write_run<kBF16, kInter, true, BS>(p, stage, meet[turn], t0 + x - 1, count, off, pos,
                                                                    first, blk, item >> 1);
                if (done) left &= ~(1u << (item - item0));
            }
        }
        for (int item = item0; item < item1; ++item)
            if (((left >> (item - item0)) & 1u) && !second)
                write_any_run<kBF16, kInter>(p, t0 + x - 1, blk, item >> 1, (item & 1) == 0);
    }
}

// kv_blocks of the CTAs write keys and values, a warp for each window of
// tokens and `items` items; the others turn the query heads.  The two kinds
// are spread evenly over the grid: the first wait on a chain of loads (slots,
// rows and scale), the second stream, and side by side they fill each other's
// pauses.  kv_rate = ceil(kv_blocks 2^32 / CTAs).
template <bool kBF16, bool kInter, int BS, int R>
__global__ void __launch_bounds__(kRopeThreads, BS == 16 ? 5 : 4)
    rope_fp8_kernel(const RopeParams p, uint64_t kv_rate, int window, int items) {
    __shared__ uint4 stage[kRopeThreads / 32][16 * kHeadDim / 4];  // 16 rows of 32-bit values for each warp
    __shared__ float meet[kRopeThreads / 64][2][2];                // for each pair of warps
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t kv = (uint32_t)((blockIdx.x * kv_rate) >> 32);  // CTAs of the first kind before this one
    if ((uint32_t)(((blockIdx.x + 1ull) * kv_rate) >> 32) > kv) {
        const uint32_t w = kv * (kRopeThreads / (2 * BS)) + threadIdx.x / (2 * BS);  // one or two warps together
        const uint32_t all = 2 * (uint32_t)p.num_kv_heads, per_window = (all + items - 1) / items;
        const uint32_t win = w / per_window;
        const int item0 = (int)((w - win * per_window) * items);
        const int64_t t0 = (int64_t)win * window;
        if (t0 < p.num_tokens)
            do_runs<kBF16, kInter, BS>(p, stage[threadIdx.x >> 5], meet[threadIdx.x >> 6], t0, window, item0,
                                       min(item0 + items, (int)all));
    } else {
        do_rows<kBF16, kInter, true, R>(p, (blockIdx.x - kv) * (kRopeThreads / 16) + (threadIdx.x >> 4));
    }
}

constexpr int64_t kRunWarps = 6080;  // warps for keys and values that a long call keeps (40 per SM)

template <bool kBF16, bool kInter, int R>
static cudaError_t launch_rope_append_t(const RopeParams& p, bool fp8, cudaStream_t stream) {
    const int64_t units = p.num_tokens * ((int64_t)row_units(p.num_q_heads, R) +
                                          (fp8 ? 0 : 2 * (int64_t)row_units(p.num_kv_heads, R)));
    const int64_t row_blocks = (units + kRopeThreads / 16 - 1) / (kRopeThreads / 16);
    if (!fp8)
        return launch_pdl(rope_rows_kernel<kBF16, kInter, R>, dim3((unsigned)row_blocks), dim3(kRopeThreads), 0, stream,
                          p);
    // Few tokens: a warp for each token and item, so that every SM has some.
    // Many: windows of a block, then items in one warp, which share the search
    // for the runs and their angles, while kRunWarps are left: 16384 tokens of
    // 8 KV heads took 80.0 us with 4096 warps, 73.3 with 8192, 777 tokens of
    // 40 heads 20.0 with 7840, 26.1 with 15680.
    const int64_t all = 2 * (int64_t)p.num_kv_heads, pair = p.block_size / 16;
    int window = 1, items = 1;
    const auto warps = [&](int w, int n) { return (p.num_tokens + w - 1) / w * ((all + n - 1) / n) * pair; };
    while (window < 16 && warps(2 * window, 1) >= kRunWarps) window *= 2;
    while (items < 32 && warps(window, 2 * items) >= kRunWarps) items *= 2;
    const int64_t kv_blocks = (warps(window, items) + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    auto kern = p.block_size == 16 ? rope_fp8_kernel<kBF16, kInter, 16, R> : rope_fp8_kernel<kBF16, kInter, 32, R>;
    const uint64_t blocks = (uint64_t)(kv_blocks + row_blocks);
    const uint64_t kv_rate = (((uint64_t)kv_blocks << 32) + blocks - 1) / blocks;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(kRopeThreads), 0, stream, p, kv_rate, window, items);
}

template <bool kBF16, bool kInter>
static cudaError_t launch_rope_append_r(const RopeParams& p, bool fp8, cudaStream_t stream) {
    const int64_t rows = (int64_t)p.num_q_heads + (fp8 ? 0 : 2 * (int64_t)p.num_kv_heads);
    return p.num_tokens * rows >= 8 * kManyUnits ? launch_rope_append_t<kBF16, kInter, 8>(p, fp8, stream)
                                                 : launch_rope_append_t<kBF16, kInter, 4>(p, fp8, stream);
}

cudaError_t launch_rope_append(const RopeParams& p, int dtype, bool fp8, cudaStream_t stream, int* launches) {
    const bool bf16 = dtype == PKV_BF16;
    const cudaError_t e = bf16 ? (p.interleaved ? launch_rope_append_r<true, true>(p, fp8, stream)
                                                : launch_rope_append_r<true, false>(p, fp8, stream))
                               : (p.interleaved ? launch_rope_append_r<false, true>(p, fp8, stream)
                                                : launch_rope_append_r<false, false>(p, fp8, stream));
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace pkv
