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
// normed tokens of 64/8 heads (680 MB) in 104 us, 6.5 TB/s.  The 8-bit write
// waits on more: a block's scale needs all of its new rows before the first
// byte, a chain of loads and exchanges for each run of tokens: 16384 tokens of
// 32/8 heads (378 MB) in 64.4 us, 5.9 TB/s; 777 normed ones of 40/40 heads (40
// MB) in 14.7 us (issue slots some 35 to 40% used, three or four warps to a
// scheduler); a step of 256 sequences in 3.0 us.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

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
// A lane's eight values of a head row: the first members of its four pairs in
// v[0], v[1], the second members in v[2], v[3], so that both kinds of pairs
// are turned alike (quad A and quad B, or their even and odd values).
struct Row {
    f32x2 v[4];
};

// ... from and to the order of quad A, quad B.
template <bool kInter>
__device__ __forceinline__ Row row_of(const float (&f)[8]) {
    Row x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int lo = kInter ? 4 * (k & 1) + (k >> 1) : 2 * k;
        x.v[k] = pack_f32x2(f[lo], f[lo + (kInter ? 2 : 1)]);
    }
    return x;
}
template <bool kInter>
__device__ __forceinline__ void values_of(const Row& x, float (&f)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int lo = kInter ? 4 * (k & 1) + (k >> 1) : 2 * k;
        unpack_f32x2(x.v[k], f[lo], f[lo + (kInter ? 2 : 1)]);
    }
}

template <bool kBF16>
__device__ __forceinline__ void widen8(uint4 x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (kBF16) {
            f[2 * k] = __uint_as_float(w[k] << 16);
            f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
            f[2 * k] = h.x, f[2 * k + 1] = h.y;
        }
    }
}

template <bool kBF16, bool kInter>
__device__ __forceinline__ Row widen_row(uint2 a, uint2 b) {
    float f[8];
    widen8<kBF16>(make_uint4(a.x, a.y, b.x, b.y), f);
    return row_of<kInter>(f);
}

__device__ __forceinline__ uint2 ldg8(const uint16_t* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }

// The cosines and sines of a lane's four angles, and the sines' negatives.
struct Turn {
    f32x2 c[2], s[2], n[2];
};

__device__ __forceinline__ Turn load_turn(const RopeParams& p, const QuadPos& qp, int64_t pos, int i) {
    Turn t;
    if (qp.rotates) {
        const float* row = p.cos_sin + pos * p.rot_dim + 4 * i;
        const float4 c = __ldg(reinterpret_cast<const float4*>(row));
        const float4 s = __ldg(reinterpret_cast<const float4*>(row + p.rot_dim / 2));
        t.c[0] = pack_f32x2(c.x, c.y), t.c[1] = pack_f32x2(c.z, c.w);
        t.s[0] = pack_f32x2(s.x, s.y), t.s[1] = pack_f32x2(s.z, s.w);
        t.n[0] = pack_f32x2(-s.x, -s.y), t.n[1] = pack_f32x2(-s.z, -s.w);
    }
    return t;
}

// Norm (where there is a weight) and turn of a head row, in 32 bits.  All 16
// lanes of the row's half-warp take part (`half` is their mask).
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
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            y.v[k] = fma2(x.v[k + 2], t.n[k], mul2(x.v[k], t.c[k]));
            y.v[k + 2] = fma2(x.v[k], t.s[k], mul2(x.v[k + 2], t.c[k]));
        }
        x = y;
    }
}

// The one rounding of a row to 16 bits.
template <bool kBF16, bool kInter>
__device__ __forceinline__ void store_row(uint16_t* row, const QuadPos& qp, const Row& x) {
    float f[8];
    values_of<kInter>(x, f);
    *reinterpret_cast<uint2*>(row + qp.a) = make_uint2(pack2<kBF16>(f[0], f[1]), pack2<kBF16>(f[2], f[3]));
    *reinterpret_cast<uint2*>(row + qp.b) = make_uint2(pack2<kBF16>(f[4], f[5]), pack2<kBF16>(f[6], f[7]));
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
// the GPU with less work: 103.9 against 114.9 us for 16384 tokens of 64/8
// heads, 16.1 against 15.8 us for 1537 of 40/40, 2.5 against 1.9 us for 64 of
// 32/8.
__host__ __device__ __forceinline__ uint32_t row_units(int heads, int R) { return (heads + R - 1) / R; }
constexpr int64_t kManyRows = 524288;  // from which on R = 8

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
    if (wp) weight = widen_row<kBF16, kInter>(ldg8(wp + qp.a), ldg8(wp + qp.b));
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
        const Turn turn = load_turn(p, qp, pos, i);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r < n) {
                Row x = widen_row<kBF16, kInter>(ra[r], rb[r]);
                norm_turn(p, qp, wp != nullptr, weight, turn, half, x);
                store_row<kBF16, kInter>(to + r * to_step, qp, x);
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

// Four values (at most 448 in magnitude, but for the last bit, or NaN) to e4m3
// bytes, nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return lo | ((uint32_t)hi << 16);
}

// A 32-bit value x and the sign of what is missing to the exact one: the value
// rounded to odd, which rounds to e4m3 as the exact one does.  (The nearest
// 32-bit value may be a tie of e4m3 where the exact one is none.)  Values that
// become zero either way, and NaN, stay.
__device__ __forceinline__ float to_odd(float x, float rest) {
    const uint32_t b = __float_as_uint(x);
    if (!(fabsf(x) >= 0x1p-12f) || rest == 0.f || (b & 1u)) return x;
    return __uint_as_float((rest < 0.f) == (x < 0.f) ? b + 1u : b - 1u);
}

__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0u; }  // s >= 2^-126
// ... and its reciprocal, exact (that of 2^127 is subnormal)
__device__ __forceinline__ float reciprocal_of_power(float s) {
    return __uint_as_float(max(0x7f000000u - __float_as_uint(s), 0x00400000u));
}

// Does a scale hold rows of magnitude a: a <= 448 s?  (One rounding, which
// keeps the sign: exact.)
__device__ __forceinline__ bool holds(float s, float a) { return fmaf(448.f, s, -a) >= 0.f; }

// The move of a block's held rows 0 .. first - 1 to another scale, by `kLanes`
// lanes: 8 per row, 16 bytes each.
template <int kLanes>
__device__ __noinline__ void move_rows(uint8_t* tile, int first, float ratio, int lane) {
#pragma unroll 1
    for (int r = lane >> 3; r < first; r += kLanes / 8) {
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
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = f[e] * ratio;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = to_odd(y[e], fmaf(f[e], ratio, -y[e]));
            w[j] = e4m3_quad(y[0], y[1], y[2], y[3]);
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
        } else if (holds(old, a)) {
            return old;
        } else if (writes) {
            move_rows<32>(tile, first, old / s, lane);
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

// Quotients y / scale of a scale that is no power of two, to odd: y times the
// rounded reciprocal may fall on the other side of a border between two e4m3
// values, so what is missing is found (exactly, by one rounding) and added, and
// its sign found once more.  (Under such scales 256 tokens' step takes 3.45 us,
// 3.02 under powers of two, the chunk of 777 15.4 us for 14.6.)
struct Divisor {
    float up, d, inv;  // scale d / up, so that no remainder falls below fp32's smallest step
};
__device__ __forceinline__ Divisor divisor(float scale) {
    Divisor r;
    r.up = scale < 0x1p-60f ? 0x1p64f : 1.f;
    r.d = scale * r.up;
    r.inv = 1.f / r.d;
    return r;
}
template <int N>
__device__ __forceinline__ void divide_to_odd(float (&f)[N], const Divisor& v) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float y = f[k] * v.up, q0 = y * v.inv, q = fmaf(fmaf(-q0, v.d, y), v.inv, q0);
        f[k] = to_odd(q, fmaf(-q, v.d, y));
    }
}

template <bool kInter>
__device__ __forceinline__ void store_quotients(uint8_t* row, const QuadPos& qp, const Row& x, const Divisor& v) {
    float f[8];
    values_of<kInter>(x, f);
    divide_to_odd(f, v);
    *reinterpret_cast<uint32_t*>(row + qp.a) = e4m3_quad(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<uint32_t*>(row + qp.b) = e4m3_quad(f[4], f[5], f[6], f[7]);
}

template <bool kInter>
__device__ __forceinline__ void store_e4m3(uint8_t* row, const QuadPos& qp, Row x, float inv) {
    const f32x2 ii = pack_f32x2(inv, inv);
#pragma unroll
    for (int k = 0; k < 4; ++k) x.v[k] = mul2(x.v[k], ii);
    float f[8];
    values_of<kInter>(x, f);
    *reinterpret_cast<uint32_t*>(row + qp.a) = e4m3_quad(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<uint32_t*>(row + qp.b) = e4m3_quad(f[4], f[5], f[6], f[7]);
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
    if (p.k_norm) weight = widen_row<kBF16, kInter>(ldg8(p.k_norm + qp.a), ldg8(p.k_norm + qp.b));
    float a = 0.f;              // the largest finite magnitude
    float s = 1.f;              // pass 1: the scale
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
                    Row x = widen_row<kBF16, kInter>(ldg8(row + qp.a), ldg8(row + qp.b));
                    if (is_k) {
                        const Turn turn = load_turn(p, qp, pos, i);
                        norm_turn(p, qp, p.k_norm != nullptr, weight, turn, half, x);
                    }
                    infinite_to_nan(x);
                    if (pass == 0) {
                        first = min(first, off);
                        a = top(a, x);
                    } else {
                        if (power_of_two(s))
                            store_e4m3<kInter>(tile + off * kHeadDim, qp, x, reciprocal_of_power(s));
                        else
                            store_quotients<kInter>(tile + off * kHeadDim, qp, x, divisor(s));
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
        s = settle_scale(p, scale, old, tile, a, first, true);
    }
}

// The largest magnitude among a warp's eight words of 16-bit pairs so far: NaN
// counts for nothing, an infinity does.
template <bool kBF16>
__device__ __forceinline__ uint32_t top16(uint32_t a, uint32_t w) {
    uint32_t r;
    if constexpr (kBF16)
        asm("{\n\t.reg .b32 m;\n\tabs.bf16x2 m, %2;\n\tmax.bf16x2 %0, %1, m;\n\t}" : "=r"(r) : "r"(a), "r"(w));
    else
        asm("{\n\t.reg .b32 m;\n\tabs.f16x2 m, %2;\n\tmax.f16x2 %0, %1, m;\n\t}" : "=r"(r) : "r"(a), "r"(w));
    return r;
}

// A lane's 16 bytes of every other row of `rows` to shared memory, 512 bytes
// apart, asynchronously.
__device__ __forceinline__ void copy_rows(uint32_t to, const uint16_t* from, int64_t step, int rows) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (2 * j < rows)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 512 * j), "l"(from + j * step) : "memory");
}

// The larger of the magnitudes that the two warps of a 32-row block found.
__device__ __forceinline__ float meet_max(float a, float (*meet)[2], int& turn) {
    const int warp = threadIdx.x >> 5;
    turn ^= 1;  // one meeting's barrier lies between two uses of a place
    if ((threadIdx.x & 31) == 0) meet[turn][warp & 1] = a;
    __syncwarp();  // bar.sync takes whole warps
    asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");
    return fmaxf(meet[turn][0], meet[turn][1]);
}

// A run of `count` <= BS neighbouring tokens from t0 on, all of them good, its
// keys (do_k), its values (do_v) or both, of KV head h; `off_l` and `pos_l` are
// lane l's token t0 + l's row and position.  Returns which are left to
// write_any_run, nothing written (bit 0: keys, 1: values): those with an
// infinity.
//
// A warp has 16 rows of a run at most.  Values and keys are copied to the two
// halves of `stage`, the warp's own 8 KiB, at once; the values become bytes as
// they are while the keys are still on the way.  The keys are turned into
// 32-bit values, which take the whole stage, and become bytes once the largest
// magnitude is known.  (One after the other through the same code, values as
// 32-bit too: 777 tokens of 40 heads 16.5 us against 14.5, 16384 of 8 heads
// 68.0 against 64.2.  Turning keys twice cost 17 us more for the latter; kept
// in registers they spilled; a CTA for each window, its runs' magnitudes
// meeting in shared memory, took 61 us for keys and values against 45.)  The two warps of a 32-row block meet at a
// barrier, `meet` is where they leave their magnitudes.
template <bool kBF16, bool kInter, int BS>
__device__ __forceinline__ uint32_t write_run(const RopeParams& p, uint4* stage, float (*meet)[2], int& turn,
                                              int64_t t0, int count, int off_l, int pos_l, int first, int blk, int h,
                                              bool do_k, bool do_v) {
    const int lane = threadIdx.x & 31, i = lane & 15, hf = lane >> 4, warp = threadIdx.x >> 5;
    const int r0 = BS == 32 ? 16 * (warp & 1) : 0;  // the warp's first row
    const int mine = min(count - r0, 16);           // its rows (none: <= 0)
    const int64_t tile_no = (int64_t)blk * p.num_kv_heads + h;
    uint32_t left = 0;
    __syncwarp();  // the warp is done with what the stage held
    const uint32_t to = smem_addr(stage + lane);
    if (do_v) copy_rows(to, p.v + (t0 + r0 + hf) * p.v_stride + h * kHeadDim + 8 * i, 2 * p.v_stride, mine - hf);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (do_k) copy_rows(to + 4096, p.k + (t0 + r0 + hf) * p.k_stride + h * kHeadDim + 8 * i, 2 * p.k_stride, mine - hf);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (do_v) {
        float* scale = p.v_scales + tile_no;
        const float old = first > 0 ? *scale : 0.f;
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();  // every lane has read `old`, too
        uint32_t m = 0u;
#pragma unroll 1
        for (int j = 0; 2 * j < mine; ++j) {
            const uint4 x = stage[16 * min(2 * j + hf, mine - 1) + i];
            m = top16<kBF16>(top16<kBF16>(top16<kBF16>(top16<kBF16>(m, x.x), x.y), x.z), x.w);
        }
        float f[8];
        widen8<kBF16>(make_uint4(m, 0u, 0u, 0u), f);
        float a = warp_max(fmaxf(f[0], f[1]));
        if constexpr (BS == 32) a = meet_max(a, meet, turn);
        uint8_t* tile = static_cast<uint8_t*>(p.v_cache) + tile_no * (BS * kHeadDim) + 8 * i;
        const float s = a == INFINITY ? a : settle_scale(p, scale, old, tile - 8 * i, a, first, r0 == 0);
        if (a == INFINITY) {
            left = 2u;
        } else if (power_of_two(s)) {
            const float inv = reciprocal_of_power(s);
            const f32x2 ii = pack_f32x2(inv, inv);
#pragma unroll 1
            for (int j = 0; 2 * j < mine; ++j) {
                const int r = min(2 * j + hf, mine - 1);
                widen8<kBF16>(stage[16 * r + i], f);
#pragma unroll
                for (int e = 0; e < 8; e += 2) unpack_f32x2(mul2(pack_f32x2(f[e], f[e + 1]), ii), f[e], f[e + 1]);
                *reinterpret_cast<uint2*>(tile + __shfl_sync(0xffffffffu, off_l, r0 + r) * kHeadDim) =
                    make_uint2(e4m3_quad(f[0], f[1], f[2], f[3]), e4m3_quad(f[4], f[5], f[6], f[7]));
            }
        } else {
            const Divisor v = divisor(s);
#pragma unroll 1
            for (int j = 0; 2 * j < mine; ++j) {
                const int r = min(2 * j + hf, mine - 1);
                widen8<kBF16>(stage[16 * r + i], f);
                divide_to_odd(f, v);
                *reinterpret_cast<uint2*>(tile + __shfl_sync(0xffffffffu, off_l, r0 + r) * kHeadDim) =
                    make_uint2(e4m3_quad(f[0], f[1], f[2], f[3]), e4m3_quad(f[4], f[5], f[6], f[7]));
            }
        }
        __syncwarp();  // the keys' values may take the rows' place
    }
    if (do_k) {
        const QuadPos qp = quad_pos<kInter>(p, i);
        float* scale = p.k_scales + tile_no;
        const float old = first > 0 ? *scale : 0.f;
        Row weight;
        if (p.k_norm) weight = widen_row<kBF16, kInter>(ldg8(p.k_norm + qp.a), ldg8(p.k_norm + qp.b));
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();  // every lane has read `old`, too
        // Pair j of rows lies in bytes 512j .. 512j + 511 of the stage's second
        // half, its 32-bit values go to 1024j .. 1024j + 1023 of the whole: over
        // the values' rows and pairs that are done.  An odd last row is done
        // by both halves.
        float a = 0.f;
#pragma unroll 1
        for (int j = 0; 2 * j < mine; ++j) {
            const int r = min(2 * j + hf, mine - 1);
            const uint16_t* row = reinterpret_cast<const uint16_t*>(stage + 256) + r * kHeadDim;
            Row y = widen_row<kBF16, kInter>(*reinterpret_cast<const uint2*>(row + qp.a),
                                             *reinterpret_cast<const uint2*>(row + qp.b));
            const Turn tn = load_turn(p, qp, __shfl_sync(0xffffffffu, pos_l, r0 + r), i);
            norm_turn(p, qp, p.k_norm != nullptr, weight, tn, 0xffffffffu, y);
            a = top(a, y);
            __syncwarp();
            ulonglong2* at = reinterpret_cast<ulonglong2*>(stage + 64 * j + lane);
            at[0] = make_ulonglong2(y.v[0], y.v[1]);
            at[32] = make_ulonglong2(y.v[2], y.v[3]);
            __syncwarp();
        }
        a = warp_max(a);
        if constexpr (BS == 32) a = meet_max(a, meet, turn);
        if (a == INFINITY) return left | 1u;
        uint8_t* tile = static_cast<uint8_t*>(p.k_cache) + tile_no * (BS * kHeadDim);
        const float s = settle_scale(p, scale, old, tile, a, first, r0 == 0);
        const auto turned = [&](int j) {
            const ulonglong2* at = reinterpret_cast<const ulonglong2*>(stage + 64 * j + lane);
            const ulonglong2 lo = at[0], hi = at[32];
            Row y;
            y.v[0] = lo.x, y.v[1] = lo.y, y.v[2] = hi.x, y.v[3] = hi.y;
            return y;
        };
        const auto place = [&](int j) {
            return tile + __shfl_sync(0xffffffffu, off_l, r0 + min(2 * j + hf, mine - 1)) * kHeadDim;
        };
        if (power_of_two(s)) {
            const float inv = reciprocal_of_power(s);
#pragma unroll 1
            for (int j = 0; 2 * j < mine; ++j) store_e4m3<kInter>(place(j), qp, turned(j), inv);
        } else {
            const Divisor v = divisor(s);
#pragma unroll 1
            for (int j = 0; 2 * j < mine; ++j) store_quotients<kInter>(place(j), qp, turned(j), v);
        }
    }
    return left;
}

// A run of one token, as a decode step has: its keys of KV head h by the warp's
// first half, its values by the second, in registers (write_run, one after the
// other, took 6.0 us for 256 sequences of 8 KV heads, this 3.0).  Returns which of the two are left to
// write_any_run (bit 0: keys, 1: values), as write_run does.
template <bool kBF16, bool kInter, int BS>
__device__ __forceinline__ uint32_t write_one(const RopeParams& p, int64_t t, int off, int pos, int blk, int h) {
    const int lane = threadIdx.x & 31, i = lane & 15;
    const bool is_v = lane >> 4;
    const QuadPos qp = quad_pos<kInter>(p, i);
    const uint16_t* row = (is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride) + h * kHeadDim;
    const int64_t tile_no = (int64_t)blk * p.num_kv_heads + h;
    float* scale = (is_v ? p.v_scales : p.k_scales) + tile_no;
    uint8_t* tile = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + tile_no * (BS * kHeadDim);
    const float old = off > 0 ? *scale : 0.f;
    Row y = widen_row<kBF16, kInter>(ldg8(row + qp.a), ldg8(row + qp.b)), weight;
    if (p.k_norm) weight = widen_row<kBF16, kInter>(ldg8(p.k_norm + qp.a), ldg8(p.k_norm + qp.b));
    const Row as_is = y;
    norm_turn(p, qp, p.k_norm != nullptr, weight, load_turn(p, qp, pos, i), 0xffffffffu, y);
    if (is_v) y = as_is;
    float a = top(0.f, y);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    __syncwarp();  // every lane has read `old`
    const bool joins = off > 0 && old >= 0x1p-126f && finite(old), keeps = joins && holds(old, a);
    if (a < INFINITY) {
        const float s = keeps ? old : power_scale(a);
        if (joins && !keeps) move_rows<16>(tile, off, old / s, i);
        if (off > 0 && !joins && i == 0) record_error(p.err, PKV_DEVERR_SCALE);
        if (i == 0) *scale = s;
        if (power_of_two(s))
            store_e4m3<kInter>(tile + off * kHeadDim, qp, y, reciprocal_of_power(s));
        else
            store_quotients<kInter>(tile + off * kHeadDim, qp, y, divisor(s));
    }
    const uint32_t rest = __ballot_sync(0xffffffffu, !(a < INFINITY));
    return (rest & 1u) | ((rest >> 15) & 2u);
}

// The keys and values of some KV heads (items item0 .. item1 - 1, 32 at most:
// item 2h is the keys of head h, 2h + 1 its values) of the runs that start
// among the tokens t0 .. t0 + window - 1, by one warp (BS = 16) or two that go
// through it together.  A run is the tokens of one block, which stand together
// in slot_mapping but for padding.  The warp looks at the 2 BS tokens from the
// one before t0 on; window < BS, so that a run's end is among them (but for
// padding inside, or slots named twice).
template <bool kBF16, bool kInter, int BS>
__device__ __forceinline__ void do_runs(const RopeParams& p, uint4* stage, float (*meet)[2], int64_t t0, int window,
                                        int item0, int item1) {
    constexpr int W = BS / 16;  // words of 32 tokens
    using Bits = typename std::conditional<W == 1, uint32_t, uint64_t>::type;
    const int lane = threadIdx.x & 31;
    const bool second = BS == 32 && ((threadIdx.x >> 5) & 1);  // the second warp of two: leaves the rest to the first
    int turn = 0;                                              // which of the meeting places is next
    Token tok[W];  // token t0 - 1 + 32u + lane: bit 32u + lane below
    Bits present = 0, wrong = 0, leaders = 0;
#pragma unroll
    for (int u = 0; u < W; ++u) {
        const int64_t t = t0 - 1 + 32 * u + lane;
        tok[u].slot = -1, tok[u].pos = 0, tok[u].err = 0;
        if (t >= 0 && t < p.num_tokens) tok[u] = token_at(p, t);
    }
#pragma unroll
    for (int u = 0; u < W; ++u) {
        present |= (Bits)__ballot_sync(0xffffffffu, tok[u].slot >= 0) << (32 * u);
        wrong |= (Bits)__ballot_sync(0xffffffffu, tok[u].err != 0) << (32 * u);
    }
    if (tok[0].err == PKV_DEVERR_SLOT && lane >= 1 && lane <= window && item0 == 0 && !second)
        record_error(p.err, PKV_DEVERR_SLOT);
    const uint32_t inside = (2u << window) - 2u;
    if (!((uint32_t)present & inside)) return;
    // the block of the last token in the pool before t0, over any padding
    int before = __shfl_sync(0xffffffffu, tok[0].slot, 0) / BS;
    if (!(present & 1u)) {
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
#pragma unroll
    for (int u = 0; u < W; ++u) {
        const int blk = tok[u].slot / BS;
        const uint32_t in = (uint32_t)(present >> (32 * u)), prior = in & ((1u << lane) - 1u);
        const int prev = __shfl_sync(0xffffffffu, blk, prior ? 31 - __clz(prior) : 0);
        leaders |= (Bits)__ballot_sync(0xffffffffu, tok[u].slot >= 0 && blk != (prior ? prev : before) && (u || lane))
                   << (32 * u);
        if (u + 1 < W && in) before = __shfl_sync(0xffffffffu, blk, 31 - __clz(in));
    }
    uint32_t undone = 0;  // lane x: items of the run that starts at bit x, left to write_any_run
    for (uint32_t own = (uint32_t)leaders & inside; own; own &= own - 1u) {
        const int x = __ffs(own) - 1;
        const Bits later = leaders & ~(((Bits)2 << x) - 1u);
        const Bits upto = later ? (later & (0u - later)) - 1u : (Bits)0 - 1u;  // bits below the next run's first
        const Bits run = (present & upto) >> x;
        const int count = W == 1 ? __popc((uint32_t)run) : __popcll(run);
        // lane l: the run's token l
        int slot = __shfl_sync(0xffffffffu, tok[0].slot, (x + lane) & 31);
        int pos = __shfl_sync(0xffffffffu, tok[0].pos, (x + lane) & 31);
        if constexpr (W == 2) {
            const int s1 = __shfl_sync(0xffffffffu, tok[W - 1].slot, (x + lane) & 31);
            const int p1 = __shfl_sync(0xffffffffu, tok[W - 1].pos, (x + lane) & 31);
            if (x + lane >= 32) slot = s1, pos = p1;
        }
        const int off = slot & (BS - 1);
        const int blk = __shfl_sync(0xffffffffu, slot, 0) / BS;
        uint32_t left = item1 - item0 < 32 ? (1u << (item1 - item0)) - 1u : 0xffffffffu;
        // neighbouring tokens, all good, the run's end in sight
        if (count <= BS && run == ((Bits)1 << count) - 1u && !(wrong & (run << x)) &&
            (later || t0 + 32 * W - 1 >= p.num_tokens)) {
            left = 0;
            if (count == 1) {  // a head's keys and values fall to who has its keys
                const int off0 = __shfl_sync(0xffffffffu, off, 0), pos0 = __shfl_sync(0xffffffffu, pos, 0);
#pragma unroll 1
                for (int item = (item0 + 1) & ~1; item < item1; item += 2)
                    if (BS == 16 || second == ((item >> 1) & 1))
                        left |= write_one<kBF16, kInter, BS>(p, t0 + x - 1, off0, pos0, blk, item >> 1) << (item - item0);
            } else {
                const int first = __reduce_min_sync(0xffffffffu, lane < count ? off : BS);
#pragma unroll 1
                for (int item = item0; item < item1;) {
                    const bool do_k = !(item & 1), do_v = !do_k || item + 1 < item1;
                    const uint32_t rest = write_run<kBF16, kInter, BS>(p, stage, meet, turn, t0 + x - 1, count, off, pos,
                                                                       first, blk, item >> 1, do_k, do_v);
                    if (!second) left |= (do_k ? rest : rest >> 1) << (item - item0);
                    item += do_k && do_v ? 2 : 1;
                }
            }
        } else if (second) {
            left = 0;
        }
        if (lane == x) undone = left;
    }
    for (uint32_t runs = __ballot_sync(0xffffffffu, undone != 0); runs; runs &= runs - 1u) {
        const int x = __ffs(runs) - 1, blk = __shfl_sync(0xffffffffu, tok[0].slot, x) / BS;
        for (uint32_t left = __shfl_sync(0xffffffffu, undone, x); left; left &= left - 1u) {
            const int item = item0 + __ffs(left) - 1;
            write_any_run<kBF16, kInter>(p, t0 + x - 1, blk, item >> 1, (item & 1) == 0);
        }
    }
}

// kv_blocks of the CTAs write keys and values, a warp (or two) for each window
// of tokens and `items` items; the others turn the query heads.  Of the first
// CTAs kv_rate / 2^32 are of the first kind, until there are no more: these
// wait on a chain of loads (slots, rows and scale), the others stream, and
// side by side they fill each other's pauses.
template <bool kBF16, bool kInter, int BS, int R>
__global__ void __launch_bounds__(kRopeThreads, BS == 16 ? 5 : 4)
    rope_fp8_kernel(const RopeParams p, uint32_t kv_blocks, uint64_t kv_rate, int window, int items) {
    __shared__ uint4 stage[kRopeThreads / 32][16 * kHeadDim / 4];  // 16 rows of 32-bit values for each warp
    __shared__ float meet[kRopeThreads / 64][2][2];                // for each pair of warps
    pdl_launch_dependents();
    pdl_wait();
    // CTAs of the first kind before this one and before the next
    const uint32_t kv = min(kv_blocks, (uint32_t)((blockIdx.x * kv_rate) >> 32));
    if (min(kv_blocks, (uint32_t)(((blockIdx.x + 1ull) * kv_rate) >> 32)) > kv) {
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

template <bool kBF16, bool kInter>
static cudaError_t launch_rope_fp8(const RopeParams& p, cudaStream_t stream) {
    // Eight rows of queries at a time whatever the call's size: keys and
    // values hold most of the places, and half the loads in flight cost 36.7 -> 42.0
    // us for 5000 tokens of 64/8 heads, 64.4 -> 72.6 for 16384 of 32/8 (3.0 either
    // way for 256).
    constexpr int R = 8;
    const int64_t q_units = p.num_tokens * (int64_t)row_units(p.num_q_heads, R);
    const int64_t q_blocks = (q_units + kRopeThreads / 16 - 1) / (kRopeThreads / 16);
    // Teams of a warp, or of two, for keys and values.  As long as all are
    // resident at once (16 warps on an SM), one for each token and item.  With
    // more, a head's keys and values share one (256 sequences' next tokens: 3.0
    // us, 4.4 without; but 5.3 us, 6.4 with, for a chunk of 100 tokens, which has
    // few runs); then windows grow towards a block's tokens, and items again,
    // while enough teams are left, 30 to an SM, or 10 of two warps: half as many
    // as the bound cost 777 tokens of 40 heads in blocks of 32 14.7 -> 16.0 us,
    // 16384 normed ones of 8 heads there 82.4 -> 98.1, 5000 of 8 heads in blocks
    // of 16 36.7 -> 37.5; twice as many 17.4, 82.9 and 37.9, and 64.4 -> 67.1 for
    // 16384 of 8 heads in blocks of 16.  (Short chunks in blocks of 32 would take
    // half as many: 256 and 512 tokens of 8 heads 7.9 -> 7.1 and 8.1 -> 7.2.)
    const int64_t resident = 16 * (int64_t)p.sms, enough = (p.block_size == 16 ? 30 : 10) * (int64_t)p.sms;
    const int64_t all = 2 * (int64_t)p.num_kv_heads, pair = p.block_size / 16;
    const auto teams = [&](int w, int n) { return (p.num_tokens + w - 1) / w * ((all + n - 1) / n); };
    int window = 1, items = teams(1, 1) * pair > resident ? 2 : 1;
    for (int w = 2; w < 2 * (int)p.block_size; w *= 2) {
        const int most = std::min(w, (int)p.block_size - 1);
        if (teams(most, items) >= enough) window = most;
    }
    while (items < 32 && teams(window, 2 * items) >= enough) items *= 2;
    const int64_t kv_blocks = (teams(window, items) * pair + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    const uint64_t blocks = (uint64_t)(kv_blocks + q_blocks);
    // Keys and values are spread over the first two thirds of the grid: their
    // teams take longest, and none should start last.  (Spread over all of it
    // 65.4, 16.5 and 40.8 us for 16384, 777 and 5000 tokens; so 64.4, 14.7,
    // 36.7; all of them first 70.0, 14.7, 38.3.)
    const uint64_t even = (((uint64_t)kv_blocks << 32) + blocks - 1) / blocks;
    const uint64_t kv_rate = std::min<uint64_t>(even + even / 2, 1ull << 32);
    auto kern = p.block_size == 16 ? rope_fp8_kernel<kBF16, kInter, 16, R> : rope_fp8_kernel<kBF16, kInter, 32, R>;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(kRopeThreads), 0, stream, p, (uint32_t)kv_blocks, kv_rate, window,
                      items);
}

template <bool kBF16, bool kInter, int R>
static cudaError_t launch_rope_rows(const RopeParams& p, cudaStream_t stream) {
    const int64_t units =
        p.num_tokens * ((int64_t)row_units(p.num_q_heads, R) + 2 * (int64_t)row_units(p.num_kv_heads, R));
    const int64_t blocks = (units + kRopeThreads / 16 - 1) / (kRopeThreads / 16);
    return launch_pdl(rope_rows_kernel<kBF16, kInter, R>, dim3((unsigned)blocks), dim3(kRopeThreads), 0, stream, p);
}

template <bool kBF16, bool kInter>
static cudaError_t launch_rope_append_t(const RopeParams& p, bool fp8, cudaStream_t stream) {
    if (fp8) return launch_rope_fp8<kBF16, kInter>(p, stream);
    const int64_t rows = (int64_t)p.num_q_heads + 2 * (int64_t)p.num_kv_heads;
    return p.num_tokens * rows >= kManyRows ? launch_rope_rows<kBF16, kInter, 8>(p, stream)
                                            : launch_rope_rows<kBF16, kInter, 4>(p, stream);
}

cudaError_t launch_rope_append(const RopeParams& p, int dtype, bool fp8, cudaStream_t stream, int* launches) {
    const bool bf16 = dtype == PKV_BF16;
    const cudaError_t e = bf16 ? (p.interleaved ? launch_rope_append_t<true, true>(p, fp8, stream)
                                                : launch_rope_append_t<true, false>(p, fp8, stream))
                               : (p.interleaved ? launch_rope_append_t<false, true>(p, fp8, stream)
                                                : launch_rope_append_t<false, false>(p, fp8, stream));
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace pkv
