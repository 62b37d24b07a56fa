// latent_append.cu -- paged_latent_append_rope: the write of new tokens into a
// paged latent cache.  A token's row is a latent of 512 values, divided by its
// root mean square and weighted where weights are given, and a key part of 64
// values turned by the token's position; every query head's 64 values are
// turned by the same angles on the way.
//
// Bytes bound it: each row is read once and written once (twice with kv_out).
// A warp takes one token's row, 16 values of the latent to a lane, so the
// norm's sum is one exchange over the warp; or 16 of a token's query heads,
// eight lanes to a head, whose four loads are all on their way before the
// first is used: 16384 tokens with 16 heads (128 MB) take 24.2 us, 5.3 TB/s, and
// a step of 64 tokens with 128 heads 2.0 us, a launch.  (More warps on an SM at
// fewer registers: 25.1 and 28.6 us; CTAs of 256 threads: 25.2.)  Pairs (i, i +
// 32) sit in lanes 4 apart and cost one exchange; neighbouring pairs sit in one
// lane.
#include "latent.cuh"

namespace pkv {
namespace {

constexpr int kLatent = kLatentDim, kRot = kLatentRope, kRow = kLatentRow;
constexpr int kThreads = 128;
constexpr int kHeadsPerWarp = 16;

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
template <bool kBF16>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
    return make_uint4(pack2<kBF16>(f[0], f[1]), pack2<kBF16>(f[2], f[3]), pack2<kBF16>(f[4], f[5]),
                      pack2<kBF16>(f[6], f[7]));
}

// The cosines and sines that lane i of eight needs for its values 8 i .. 8 i + 7.
struct Angles {
    float c[8], s[8];
};
template <bool kInter>
__device__ __forceinline__ void load_angles(Angles& a, const float* row, int i) {
    // pairs (2 j, 2 j + 1): angles 4 i .. 4 i + 3, each for two values; pairs (j, j + 32): angles 8 (i % 4) ..
    const float4* c = reinterpret_cast<const float4*>(row + (kInter ? 4 * i : 8 * (i & 3)));
    const float4* s = c + kRot / 8;
#pragma unroll
    for (int h = 0; h < (kInter ? 1 : 2); ++h) {
        const float4 x = __ldg(c + h), y = __ldg(s + h);
        a.c[4 * h] = x.x, a.c[4 * h + 1] = x.y, a.c[4 * h + 2] = x.z, a.c[4 * h + 3] = x.w;
        a.s[4 * h] = y.x, a.s[4 * h + 1] = y.y, a.s[4 * h + 2] = y.z, a.s[4 * h + 3] = y.w;
    }
}
// (y_a, y_b) = (x_a c - x_b s, x_b c + x_a s)
template <bool kInter>
__device__ __forceinline__ void turn(float (&x)[8], const Angles& a, int i) {
    if constexpr (kInter) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float u = x[2 * k], v = x[2 * k + 1];
            x[2 * k] = u * a.c[k] - v * a.s[k];
            x[2 * k + 1] = v * a.c[k] + u * a.s[k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float other = __shfl_xor_sync(0xffffffffu, x[k], 4);
            x[k] = i < 4 ? x[k] * a.c[k] - other * a.s[k] : x[k] * a.c[k] + other * a.s[k];
        }
    }
}

template <bool kBF16, bool kInter>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const LatentAppendParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t task = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    if (task >= p.num_tokens * (1 + p.head_tasks)) return;  // (whole warps)
    const bool row_task = task < p.num_tokens;
    const int64_t rest = task - p.num_tokens;
    const int64_t t = row_task ? task : rest / p.head_tasks;
    const int64_t slot = __ldg(p.slot_mapping + t);
    const int64_t pos = p.cos_sin ? __ldg(p.positions + t) : 0;
    const int i = lane & 7;  // lane of eight
    // the rows' loads do not wait for the token's slot and position
    uint4 in[4];
    const int h0 = row_task ? 0 : (int)(rest - t * p.head_tasks) * kHeadsPerWarp;
    const uint16_t* kv = p.kv + t * p.kv_stride;
    if (row_task) {
        in[0] = __ldg(reinterpret_cast<const uint4*>(kv) + lane);
        in[1] = __ldg(reinterpret_cast<const uint4*>(kv) + 32 + lane);
        in[2] = __ldg(reinterpret_cast<const uint4*>(kv + kLatent) + i);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int h = h0 + 4 * k + (lane >> 3);
            in[k] = h < p.num_heads
                        ? __ldg(reinterpret_cast<const uint4*>(p.q + t * p.q_stride + h * p.q_head_stride) + i)
                        : make_uint4(0, 0, 0, 0);
        }
    }
    if (slot < 0) return;  // padding
    int err = 0;
    if (slot >= p.num_slots)
        err = PKV_DEVERR_SLOT;
    else if (p.cos_sin && (pos < 0 || pos >= p.max_position))
        err = PKV_DEVERR_POSITION;
    if (err && lane == 0) record_error(p.err, err);
    Angles ang;
    if (p.cos_sin) load_angles<kInter>(ang, p.cos_sin + (err ? 0 : pos) * kRot, i);
    if (!row_task) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int h = h0 + 4 * k + (lane >> 3);
            if (p.cos_sin) {
                float x[8];
                widen8<kBF16>(in[k], x);
                turn<kInter>(x, ang, i);
                in[k] = narrow8<kBF16>(x);
            }
            if (err) in[k] = make_uint4(0, 0, 0, 0);
            if (h < p.num_heads)
                *(reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + h * p.q_out_head_stride) + i) = in[k];
        }
        return;
    }
    if (p.kv_norm) {
        float x[2][8], sum = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            widen8<kBF16>(in[k], x[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += x[k][e] * x[k][e];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = 1.f / sqrtf(sum * (1.f / kLatent) + p.norm_eps);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float w[8];
            widen8<kBF16>(__ldg(reinterpret_cast<const uint4*>(p.kv_norm) + 32 * k + lane), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] = x[k][e] * r * w[e];
            in[k] = narrow8<kBF16>(x[k]);
        }
    }
    if (p.cos_sin) {
        float x[8];
        widen8<kBF16>(in[2], x);
        turn<kInter>(x, ang, i);
        in[2] = narrow8<kBF16>(x);
    }
    const auto store = [&](uint16_t* row) {
        reinterpret_cast<uint4*>(row)[lane] = in[0];
        reinterpret_cast<uint4*>(row)[32 + lane] = in[1];
        if (lane < 8) reinterpret_cast<uint4*>(row + kLatent)[lane] = in[2];
    };
    if (err) in[0] = in[1] = in[2] = make_uint4(0, 0, 0, 0);
    if (!err) store(p.cache + slot * kRow);
    if (p.kv_out) store(p.kv_out + t * kRow);
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendParams& in, int dtype, cudaStream_t stream, int* launches) {
    LatentAppendParams p = in;
    p.head_tasks = (p.num_heads + kHeadsPerWarp - 1) / kHeadsPerWarp;
    const int64_t warps = p.num_tokens * (1 + p.head_tasks), ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
    auto kern = dtype == PKV_BF16 ? (p.interleaved ? latent_append_kernel<true, true> : latent_append_kernel<true, false>)
                                  : (p.interleaved ? latent_append_kernel<false, true> : latent_append_kernel<false, false>);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), 0, stream, p);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace pkv
