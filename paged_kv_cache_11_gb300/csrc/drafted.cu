// drafted.cu -- joins the pieces of units that were divided between CTAs
// (drafted.cuh): with (o_p, m_p, l_p) the unnormalised sums, maximum (log2
// domain) and weight of piece p,
//     out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,  M = max_p m_p.
// A row whose pieces hold no weight is zeros; a piece of negative
// weight (bad metadata) zeroes its rows.  Bytes bound it: the pieces lie in L2, where the
// main kernel left them.
#include "drafted.cuh"

namespace pkv {

constexpr int kMergeThreads = 128;
constexpr int kMergeSlices = 16;  // CTAs of one unit

template <bool kBF16, int D>
__global__ void __launch_bounds__(kMergeThreads) draft_merge_kernel(const DraftParams p, int unit_rows) {
    pdl_wait();
    const int c = blockIdx.x;
    const int4 d = __ldcg(p.part_desc + (c * 2 + 1) * 2);
    const int state = d.x, tok0 = d.y, row0 = d.z, rows = d.w;
    if (!(state & kPartValid) || (state & kPartEnds)) return;  // no unit begins here and ends elsewhere
    const int kvh = __ldcg(p.part_desc + (c * 2 + 1) * 2 + 1).x;
    int last = c + 1;  // the CTA that holds the unit's last tile
    while (last < p.ctas - 1 && !(__ldcg(p.part_desc + last * 4).x & kPartEnds)) ++last;
    const int per = (rows + kMergeSlices - 1) / kMergeSlices, r0 = blockIdx.y * per, r1 = min(rows, r0 + per);
    for (int i = r0 * (D / 4) + threadIdx.x; i < r1 * (D / 4); i += kMergeThreads) {
        const int r = i / (D / 4), d4 = i - r * (D / 4);
        float M = -INFINITY;
        bool bad = false;
        for (int k = c; k <= last; ++k) {
            const float2 ml = __ldcg(p.part_ml + (int64_t)(k * 2 + (k == c)) * unit_rows + r);
            M = fmaxf(M, ml.x);
            bad |= ml.y < 0.f;
        }
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        if (!bad && M != -INFINITY) {
            for (int k = c; k <= last; ++k) {
                const int64_t at = (int64_t)(k * 2 + (k == c)) * unit_rows + r;
                const float2 ml = __ldcg(p.part_ml + at);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D) + d4);
                if (ml.x == -INFINITY) continue;  // nothing there for this row
                const float w = exp2f(ml.x - M);
                l += w * ml.y;
                o.x += w * v.x, o.y += w * v.y, o.z += w * v.z, o.w += w * v.w;
            }
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;  // (NaN stays)
        const int token = (row0 + r) / p.group, h = kvh * p.group + (row0 + r) - token * p.group;
        uint16_t* dst = static_cast<uint16_t*>(p.out) + ((int64_t)(tok0 + token) * p.num_q_heads + h) * D + 4 * d4;
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack2<kBF16>(o.x * inv, o.y * inv), pack2<kBF16>(o.z * inv, o.w * inv));
    }
}

cudaError_t launch_draft_merge(const DraftParams& p, int dtype, int value_dims, int unit_rows, cudaStream_t stream,
                               int* launches) {
    const bool bf16 = dtype == PKV_BF16;
    auto kern = value_dims == 128 ? (bf16 ? draft_merge_kernel<true, 128> : draft_merge_kernel<false, 128>)
                                  : (bf16 ? draft_merge_kernel<true, 512> : draft_merge_kernel<false, 512>);
    const cudaError_t e = launch_pdl(kern, dim3(p.ctas, kMergeSlices), dim3(kMergeThreads), 0, stream, p, unit_rows);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace pkv
