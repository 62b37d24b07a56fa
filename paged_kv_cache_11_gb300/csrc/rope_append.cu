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

__device__ __forceinline__ QuadPos quad_pos(const RopeParams& p, int i) {
    QuadPos r;
    r.rotates = i < p.rot_dim / 8;
    const bool split = r.rotates && !p.interleaved;
    r.a = split ? 4 * i : 8 * i;
    r.b = split ? p.rot_dim / 2 + 4 * i : 8 * i + 4;
    return r;
}

template <bool kBF16>
__device__ __forceinline__ float to_f32(uint16_t x) {
    if constexpr (kBF16)
        return __uint_as_float((uint32_t)x << 16);
    else
        return __half2float(__ushort_as_half(x));
}

template <bool kBF16>
__device__ __forceinline__ void unpack4(uint2 w, float* x) {
    x[0] = to_f32<kBF16>((uint16_t)(w.x & 0xffffu));
    x[1] = to_f32<kBF16>((uint16_t)(w.x >> 16));
    x[2] = to_f32<kBF16>((uint16_t)(w.y & 0xffffu));
    x[3] = to_f32<kBF16>((uint16_t)(w.y >> 16));
}

__device__ __forceinline__ uint2 ldg8(const uint16_t* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }

// A lane's eight values of a head row: quad A in x[0..3], quad B in x[4..7].
template <bool kBF16>
__device__ __forceinline__ void load_row(const uint16_t* row, const QuadPos& qp, float* x) {
    unpack4<kBF16>(ldg8(row + qp.a), x);
    unpack4<kBF16>(ldg8(row + qp.b), x + 4);
}

// Cosines and sines of the lane's four pairs.
struct Turn {
    float c[4], s[4];
};

__device__ __forceinline__ Turn load_turn(const RopeParams& p, const QuadPos& qp, int64_t pos, int i) {
    Turn t;
    if (qp.rotates) {
        const float* row = p.cos_sin + pos * p.rot_dim + 4 * i;
        const float4 c = __ldg(reinterpret_cast<const float4*>(row));
        const float4 s = __ldg(reinterpret_cast<const float4*>(row + p.rot_dim / 2));
        t.c[0] = c.x, t.c[1] = c.y, t.c[2] = c.z, t.c[3] = c.w;
        t.s[0] = s.x, t.s[1] = s.y, t.s[2] = s.z, t.s[3] = s.w;
    }
    return t;
}

// Norm (weight != nullptr) and turn of a head row, in 32 bits.  All 16 lanes
// of the row's half-warp take part (`half` is their mask).
template <bool kBF16>
__device__ __forceinline__ void norm_turn(const RopeParams& p, const QuadPos& qp, const uint16_t* weight,
                                          const Turn& t, uint32_t half, float* x) {
    if (weight) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(half, ss, o);
        const float r = 1.f / sqrtf(ss * (1.f / kHeadDim) + p.norm_eps);
        float w[8];
        load_row<kBF16>(weight, qp, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
    }
    if (qp.rotates) {
        if (p.interleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = x[2 * j], b = x[2 * j + 1];
                x[2 * j] = a * t.c[j] - b * t.s[j];
                x[2 * j + 1] = b * t.c[j] + a * t.s[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = x[j], b = x[j + 4];
                x[j] = a * t.c[j] - b * t.s[j];
                x[j + 4] = b * t.c[j] + a * t.s[j];
            }
        }
    }
}

// The one rounding of a row to 16 bits.
template <bool kBF16>
__device__ __forceinline__ void store_row(uint16_t* row, const QuadPos& qp, const float* x) {
    *reinterpret_cast<uint2*>(row + qp.a) = make_uint2(pack2<kBF16>(x[0], x[1]), pack2<kBF16>(x[2], x[3]));
    *reinterpret_cast<uint2*>(row + qp.b) = make_uint2(pack2<kBF16>(x[4], x[5]), pack2<kBF16>(x[6], x[7]));
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
    k.pos = 0;
    k.err = 0;
    if (k.slot < 0) return k;
    if (p.rot_dim > 0) k.pos = __ldg(p.positions + t);
    if (k.slot >= p.num_slots)
        k.err = PKV_DEVERR_SLOT;
    else if (p.rot_dim > 0 && (k.pos < 0 || k.pos >= p.max_position))
        k.err = PKV_DEVERR_POSITION;
    return k;
}

// Rows of the 16-bit path: for each token its query heads, key heads, value
// heads.  With an 8-bit pool only the query heads are done here.
template <bool kBF16, bool kQOnly>
__global__ void __launch_bounds__(256) rope_rows_kernel(const RopeParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int i = threadIdx.x & 15;
    const uint32_t half = 0xffffu << (threadIdx.x & 16);
    const int rows = p.num_q_heads + (kQOnly ? 0 : 2 * p.num_kv_heads);
    const int64_t r = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 4;
    const int64_t t = r / rows;
    if (t >= p.num_tokens) return;  // uniform over the half-warp
    const int h = (int)(r - t * rows);
    const Token tok = token_at(p, t);
    if (tok.slot < 0) return;
    const QuadPos qp = quad_pos(p, i);
    if (tok.err) {
        if (h == 0 && i == 0) record_error(p.err, tok.err);
        if (h < p.num_q_heads) {
            const float z[8] = {};
            store_row<kBF16>(p.q_out + (t * p.num_q_heads + h) * kHeadDim, qp, z);
        }
        return;
    }
    const int64_t blk = tok.slot / p.block_size, off = tok.slot - blk * p.block_size;
    if (h < p.num_q_heads + (kQOnly ? 0 : p.num_kv_heads)) {
        const bool is_q = h < p.num_q_heads;
        const int hk = h - p.num_q_heads;
        float x[8];
        load_row<kBF16>(is_q ? p.q + t * p.q_stride + h * kHeadDim : p.k + t * p.k_stride + hk * kHeadDim, qp, x);
        const Turn turn = load_turn(p, qp, tok.pos, i);
        norm_turn<kBF16>(p, qp, is_q ? p.q_norm : p.k_norm, turn, half, x);
        uint16_t* to = is_q ? p.q_out + (t * p.num_q_heads + h) * kHeadDim
                            : static_cast<uint16_t*>(p.k_cache) +
                                  ((blk * p.num_kv_heads + hk) * p.block_size + off) * kHeadDim;
        store_row<kBF16>(to, qp, x);
    } else {
        const int hv = h - p.num_q_heads - p.num_kv_heads;
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p.v + t * p.v_stride + hv * kHeadDim) + i);
        uint16_t* to = static_cast<uint16_t*>(p.v_cache) +
                       ((blk * p.num_kv_heads + hv) * p.block_size + off) * kHeadDim;
        reinterpret_cast<uint4*>(to)[i] = w;
    }
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

// Two values to two e4m3 bytes, nearest, ties to even; what is not finite
// becomes NaN.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint32_t w = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
    if (!finite(lo)) w |= 0x007fu;
    if (!finite(hi)) w |= 0x7f00u;
    return w;
}

__device__ __forceinline__ uint32_t e4m3_quad(const float* x, float inv) {
    return e4m3_pair(x[0] * inv, x[1] * inv) | (e4m3_pair(x[2] * inv, x[3] * inv) << 16);
}

// One warp per (token that starts a block's run, KV head).  A run is the
// tokens of one block, which stand together in slot_mapping but for padding.
// Two passes over its rows: the largest magnitudes, then the scaled bytes.
template <bool kBF16>
__global__ void __launch_bounds__(256) rope_kv8_kernel(const RopeParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, i = lane & 15, hf = lane >> 4;
    const int64_t t0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int h = blockIdx.y;
    if (t0 >= p.num_tokens) return;
    const int64_t slot0 = __ldg(p.slot_mapping + t0);
    if (slot0 < 0) return;
    if (slot0 >= p.num_slots) {
        if (h == 0 && lane == 0) record_error(p.err, PKV_DEVERR_SLOT);
        return;
    }
    const int64_t blk = slot0 / p.block_size;
    // Does an earlier token of the run exist?  Look back over what is not in the pool.
    for (int64_t b = t0 - 1; b >= 0; b -= 32) {
        const int64_t s = b - lane >= 0 ? __ldg(p.slot_mapping + b - lane) : -1;
        const bool real = s >= 0 && s < p.num_slots;
        const uint32_t m = __ballot_sync(0xffffffffu, real);
        if (m) {
            const int64_t prev = __shfl_sync(0xffffffffu, s, __ffs(m) - 1);
            if (prev / p.block_size == blk) return;
            break;
        }
    }
    const QuadPos qp = quad_pos(p, i);
    const uint32_t half = 0xffffu << (lane & 16);
    const int64_t tile = (blk * p.num_kv_heads + h) * p.block_size * kHeadDim;
    uint8_t* kt = static_cast<uint8_t*>(p.k_cache) + tile;
    uint8_t* vt = static_cast<uint8_t*>(p.v_cache) + tile;
    float ka = 0.f, va = 0.f;  // pass 0: largest finite magnitudes; pass 1: reciprocals of the scales
    int first = p.block_size;  // first row written
    for (int pass = 0; pass < 2; ++pass) {
        for (int64_t c = t0; c < p.num_tokens; c += 32) {
            const bool in = c + lane < p.num_tokens;
            Token tok;
            tok.slot = -1;
            tok.pos = 0;
            tok.err = 0;
            if (in) tok = token_at(p, c + lane);
            const bool real = tok.slot >= 0 && tok.slot < p.num_slots;
            const bool mine = real && tok.slot / p.block_size == blk;
            uint32_t other = __ballot_sync(0xffffffffu, real && !mine);
            const uint32_t before = other ? (1u << (__ffs(other) - 1)) - 1u : 0xffffffffu;
            if (mine && tok.err && ((before >> lane) & 1u) && pass == 0 && h == 0) record_error(p.err, tok.err);
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
                    float x[8], y[8];
                    load_row<kBF16>(p.k + t * p.k_stride + h * kHeadDim, qp, x);
                    load_row<kBF16>(p.v + t * p.v_stride + h * kHeadDim, qp, y);
                    const Turn turn = load_turn(p, qp, pos, i);
                    norm_turn<kBF16>(p, qp, p.k_norm, turn, half, x);
                    if (pass == 0) {
                        first = min(first, off);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (finite(x[j])) ka = fmaxf(ka, fabsf(x[j]));
                            if (finite(y[j])) va = fmaxf(va, fabsf(y[j]));
                        }
                    } else {
                        uint8_t* kr = kt + off * kHeadDim;
                        uint8_t* vr = vt + off * kHeadDim;
                        *reinterpret_cast<uint32_t*>(kr + qp.a) = e4m3_quad(x, ka);
                        *reinterpret_cast<uint32_t*>(kr + qp.b) = e4m3_quad(x + 4, ka);
                        *reinterpret_cast<uint32_t*>(vr + qp.a) = e4m3_quad(y, va);
                        *reinterpret_cast<uint32_t*>(vr + qp.b) = e4m3_quad(y + 4, va);
                    }
                }
                __syncwarp();
            }
            if (other) break;
        }
        if (pass == 1) break;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
            va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
            first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
        }
        if (first == p.block_size) return;  // every token of the run was refused
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float* sp = (w ? p.v_scales : p.k_scales) + blk * p.num_kv_heads + h;
            const float a = w ? va : ka;
            float s = power_scale(a);
            if (first > 0) {
                const float old = *sp;
                if (!(old > 0.f && finite(old))) {
                    if (lane == 0) record_error(p.err, PKV_DEVERR_SCALE);
                } else if (a <= 448.f * old) {
                    s = old;
                } else {
                    // move the held rows: 8 lanes per row, 16 bytes each
                    uint8_t* bytes = (w ? vt : kt) + (lane & 7) * 16;
                    const float ratio = old / s;
                    for (int r = lane >> 3; r < first; r += 4) {
                        uint4* at = reinterpret_cast<uint4*>(bytes + r * kHeadDim);
                        uint4 v = *at;
                        uint32_t* ww = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float f[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                f[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(
                                    (__nv_fp8_storage_t)((ww[j] >> (8 * e)) & 0xffu), __NV_E4M3)));
                            ww[j] = e4m3_quad(f, ratio);
                        }
                        *at = v;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) *sp = s;
            (w ? va : ka) = 1.f / s;
        }
    }
}

cudaError_t launch_rope_append(const RopeParams& p, int dtype, bool fp8, cudaStream_t stream, int* launches) {
    const bool bf16 = dtype == PKV_BF16;
    cudaError_t e = cudaSuccess;
    const int rows = p.num_q_heads + (fp8 ? 0 : 2 * p.num_kv_heads);
    if (rows > 0) {
        const int64_t blocks = (p.num_tokens * rows + 15) / 16;
        auto kern = fp8 ? (bf16 ? rope_rows_kernel<true, true> : rope_rows_kernel<false, true>)
                        : (bf16 ? rope_rows_kernel<true, false> : rope_rows_kernel<false, false>);
        e = launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, stream, p);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    if (fp8) {
        const dim3 grid((unsigned)((p.num_tokens + 7) / 8), (unsigned)p.num_kv_heads);
        auto kern = bf16 ? rope_kv8_kernel<true> : rope_kv8_kernel<false>;
        e = launch_pdl(kern, grid, dim3(256), 0, stream, p);
        if (e == cudaSuccess) ++*launches;
    }
    return e;
}

}  // namespace pkv
