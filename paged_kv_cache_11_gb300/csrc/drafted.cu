// drafted.cu -- joins the pieces of units that were divided between CTAs
// (drafted.cuh): with (o_p, m_p, l_p) the unnormalised sums, maximum (log2
// domain) and weight of piece p,
//     out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,  M = max_p m_p.
// A row whose pieces hold no weight is zeros; a piece of negative weight (bad
// metadata) zeroes its rows; what is not finite in any piece stays so.  The
// pieces lie in L2, where the main kernel left them; a chain of latencies bounds
// the merge (which unit, where it ends, its weights, its sums): 4 to 5 us for 18
// MB in pairs of pieces, 13 us for 36 MB, and 13 for eight units of 19 pieces.
#include "drafted.cuh"

namespace pkv {

constexpr int kMergeThreads = 256;
constexpr int kMergeParts = 128;   // pieces at a time

// A CTA merges a slice of a unit, kMergeItems float4 to a thread.
template <bool kBF16, int D, int kUnitRows, int kMergeItems>
__global__ void __launch_bounds__(kMergeThreads) draft_merge_kernel(const DraftParams p) {
    constexpr int kRows = kMergeThreads * kMergeItems / (D / 4);  // of a slice, at most
    static_assert(kUnitRows % kRows == 0, "whole slices");
    __shared__ float weight[kRows][kMergeParts];
    __shared__ float top[kRows], total[kRows];
    __shared__ int last_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = blockIdx.x;
    if (tid == 0) last_s = p.pieces - 1;
    __syncthreads();
    pdl_wait();
    const int4 d = __ldcg(p.part_desc + (c * 2 + 1) * 2);
    const int kvh = __ldcg(p.part_desc + (c * 2 + 1) * 2 + 1).x;
    const int state = d.x, tok0 = d.y, row0 = d.z, rows = d.w;
    // the CTA that holds the unit's last tile: the first behind this one that ends a unit which it did not begin
    for (int k = c + 1 + tid; k < p.pieces; k += kMergeThreads)
        if (__ldcg(p.part_desc + k * 4).x & kPartEnds) {
            atomicMin(&last_s, k);
            break;
        }
    if (!(state & kPartValid) || (state & kPartEnds)) return;  // no unit begins here and ends elsewhere
    const int r0 = blockIdx.y * kRows, n = min(kRows, rows - r0);
    if (n <= 0) return;
    __syncthreads();
    const int parts = last_s - c + 1;
    const auto at = [&](int k, int r) { return (int64_t)((c + k) * 2 + (k == 0)) * kUnitRows + r0 + r; };
    // the first two pieces (there are two at least) are on their way beside their weights
    float4 early[2][kMergeItems];
    const auto fetch = [&](int k, float4 (&v)[kMergeItems]) {
#pragma unroll
        for (int i = 0; i < kMergeItems; ++i) {
            const int e = tid + i * kMergeThreads, r = e / (D / 4);
            v[i] = r < n ? __ldcg(reinterpret_cast<const float4*>(p.part_o + at(k, r) * D) + e % (D / 4))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    fetch(0, early[0]);
    fetch(1, early[1]);
    // each row's largest maximum and its weight in all, a warp to a row
#pragma unroll 2
    for (int r = warp; r < n; r += kMergeThreads / 32) {
        const float2 none = make_float2(-INFINITY, 0.f);
        const float2 mine = lane < parts ? __ldcg(p.part_ml + at(lane, r)) : none;  // (the rest, if any, is read twice)
        float m = mine.x;
        bool bad = mine.y < 0.f;
        for (int k = lane + 32; k < parts; k += 32) {
            const float2 ml = __ldcg(p.part_ml + at(k, r));
            m = fmaxf(m, ml.x);
            bad |= ml.y < 0.f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float l = 0.f;
        for (int k = lane; k < parts; k += 32) {
            const float2 ml = k < 32 ? mine : __ldcg(p.part_ml + at(k, r));
            const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);  // (nothing there for this row)
            l += w * ml.y;  // (a sum that is NaN stays, of a weight of zero too)
            if (k < kMergeParts) weight[r][k] = w;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
            top[r] = m;
            total[r] = bad || l == 0.f ? 0.f : 1.f / l;  // (NaN stays)
        }
    }
    float4 o[kMergeItems];
#pragma unroll
    for (int i = 0; i < kMergeItems; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < parts; k0 += kMergeParts) {
        const int np = min(kMergeParts, parts - k0);
        __syncthreads();
        if (k0 > 0) {  // (more pieces than weights are held at once)
            for (int i = tid; i < n * np; i += kMergeThreads) {
                const int r = i / np, k = i - r * np;
                const float m = __ldcg(p.part_ml + at(k0 + k, r)).x;
                weight[r][k] = m == -INFINITY ? 0.f : exp2f(m - top[r]);
            }
            __syncthreads();
        }
        const auto add = [&](int k, const float4 (&v)[kMergeItems]) {
#pragma unroll
            for (int i = 0; i < kMergeItems; ++i) {
                const int r = (tid + i * kMergeThreads) / (D / 4);
                const float w = r < n ? weight[r][k] : 0.f;
                o[i].x += w * v[i].x, o[i].y += w * v[i].y, o[i].z += w * v[i].z, o[i].w += w * v[i].w;
            }
        };
        int k = 0;
        if (k0 == 0) {
            add(0, early[0]);
            add(1, early[1]);
            k = 2;
        }
#pragma unroll 4
        for (; k < np; ++k) {
            float4 v[kMergeItems];
            fetch(k0 + k, v);
            add(k, v);
        }
    }
#pragma unroll
    for (int i = 0; i < kMergeItems; ++i) {
        const int e = tid + i * kMergeThreads, r = e / (D / 4), d4 = e % (D / 4);
        if (r >= n) continue;
        const float inv = total[r];
        const int row = row0 + r0 + r, token = row / p.group, h = kvh * p.group + row - token * p.group;
        uint16_t* dst = static_cast<uint16_t*>(p.out) + ((int64_t)(tok0 + token) * p.num_q_heads + h) * D + 4 * d4;
        *reinterpret_cast<uint2*>(dst) = inv == 0.f ? make_uint2(0, 0)
                                                    : make_uint2(pack2<kBF16>(o[i].x * inv, o[i].y * inv),
                                                                 pack2<kBF16>(o[i].z * inv, o[i].w * inv));
    }
}

template <int D, int kUnitRows>
static cudaError_t launch_merge_t(const DraftParams& p, bool bf16, bool few, cudaStream_t stream) {
    auto kern = few ? (bf16 ? draft_merge_kernel<true, D, kUnitRows, 1> : draft_merge_kernel<false, D, kUnitRows, 1>)
                    : (bf16 ? draft_merge_kernel<true, D, kUnitRows, 2> : draft_merge_kernel<false, D, kUnitRows, 2>);
    const int rows = kMergeThreads * (few ? 1 : 2) / (D / 4);
    return launch_pdl(kern, dim3(p.pieces, kUnitRows / rows), dim3(kMergeThreads), 0, stream, p);
}

cudaError_t launch_draft_merge(const DraftParams& p, int dtype, int value_dims, int unit_rows, cudaStream_t stream,
                               int* launches) {
    // Few units are divided into many pieces each, and their slices are made small enough to give every SM some; many
    // units fill the SMs as they are, and smaller slices would only be more CTAs to start (of 152 x 32, and all but the
    // divided units' have nothing to do).
    const int64_t rows = ((int64_t)p.num_tokens + p.num_seqs - 1) / p.num_seqs * p.group;
    const int64_t units = p.num_seqs * (int64_t)p.num_kv_heads * ((rows + unit_rows - 1) / unit_rows);
    const bool few = units * 16 < 2 * p.pieces, bf16 = dtype == PKV_BF16;
    const cudaError_t e = value_dims == 128 ? launch_merge_t<128, kTreeRows>(p, bf16, few, stream)
                                               : launch_merge_t<512, kLatentRows>(p, bf16, few, stream);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace pkv
