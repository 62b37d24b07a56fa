// latent.cu -- paged_latent_decode: attention over a paged cache of one latent
// row a token (512 values and a 64-value key part that all heads share), in
// its absorbed form: with every head's query taken through the key expansion
// beforehand, its score against a token is a product over all 576 values of
// the token's row, and the first 512 are the token's value as well.
//
// Bytes against operations: a token's row is read once (1152 bytes) for 2 (576
// + 512) operations of every query row, 121 operations a byte at the 64 rows of
// a unit, where the card has 288.  A sequence of more rows is walked once for
// every 64 of them (its copies are marked as the first to leave L2 all the same:
// without the mark 64 of 512 to 4096 with 128 heads take 3 us more).
//
// The sums of 64 rows x 512 values are 256 columns of tensor memory when the
// values are the lanes, so the second product is transposed; the first is not,
// so that a query row's scores lie in one lane:
//   S = Q K^T        M = 64 query rows, N = 64 keys, 36 steps of 16 values;
//                    Q and K in shared memory, K-major
//   O^T += V^T P^T   M = 4 x 128 values, N = query rows, 4 steps of 16 keys;
//                    V = the same tile of rows, read value-major; P in shared
//                    memory, 16 bits, K-major
// (With the query rows as lanes 128 rows would fill all of tensor memory and
// leave no room for S, and 64 rows half of each lane quarter.)
//
// The ring holds two tiles of 64 keys as eight slots of 16; a slot is given
// back as soon as the last of its products has ended, so that copies go on
// while a tile is at work.  A slot is one TMA copy: 8-key groups of 9 KiB, the
// nine 64-value parts of the 8 rows one after the other, so that the groups of
// a tile stand 9 KiB apart for both products whatever the block size.
//
// Warps: 0-3 the softmax (16 rows each) and the output, 4 the copies of rows, 5
// the products, 6 the copies of queries.  The maximum is raised lazily, as in
// tree.cu; a weight is rounded to the cache's 16-bit type for its product (fp16's
// at seven binades more, softmax_tile.cuh), the row's sum is that of the weights
// before.  Masked places are replaced, not added to, and values that are not
// finite are kept out of the products of tiles with masks, as there.
//
// What bounds it.  A tile costs the tensor core 36 x 32 + 16 x 48 cycles (the
// latter by shared memory reads, 128 bytes a cycle), 1920 in all; its copy 3200
// at the memory's pace.  The ring holds two tiles, and a tile is held from its
// copy to its last product, so the latencies of both (copy 1700 cycles, softmax
// 1000) add up to some 3750 cycles a tile.  8 contexts of 131072 tokens, 16
// heads, 1 to 4 drafted tokens (1.2 GB): 236 us, 5.1 TB/s, 13 us of it the
// merge; 64 of 512 to 4096 with 128 heads (190 MB): 96 us, 430 TFLOP/s, of it 13
// the merge of 36 MB of divided sums, and two or three outputs of 3 us a CTA.
// Tiles of 32 keys, four in the ring, were slower (269, 103): products with N =
// 32 take 34 cycles to issue and not 16.  (Pairs of CTAs that copied each row
// into both rings at once took 92 us for the 96; such copies are not used here,
// since nothing keeps them to memory of this GPU.)
#include "copies.cuh"
#include "drafted.cuh"
#include "latent.cuh"
#include "softmax_tile.cuh"

namespace pkv {
namespace {

constexpr int kRow = kLatentRow, kValue = kLatentDim;  // values of a row, of them the token's value
constexpr int kSoftWarps = 4;
constexpr int kCopyWarp = 4, kProductWarp = 5, kQueryWarp = 6;
constexpr int kThreads = 7 * 32;
constexpr int kTile = 64;                 // keys
constexpr int kParts = kRow / 64;         // 64-value (128-byte) parts of a row
constexpr int kGroup = kParts * 1024;     // bytes of 8 keys
constexpr int kSlotKeys = 16;
constexpr int kSlot = 2 * kGroup;
constexpr int kSlots = kTile / kSlotKeys; // of a tile
constexpr int kRing = 2 * kSlots;
constexpr int kLeast = 8;                 // tiles of a piece
constexpr uint32_t kTmemCols = 512;       // O^T: four parts of 64 columns; S: [256, 320), [320, 384)

struct LatentSmem {
    static constexpr int kQ = 0;  // [9 parts][64 rows][128 B]
    static constexpr int kKV = kQ + kParts * kLatentRows * 128;
    static constexpr int kP = kKV + kRing * kSlot;  // [64 rows][64 keys]
    static constexpr int kAlpha = kP + kLatentRows * kTile * 2;  // [2][64]
    static constexpr int kFin = kAlpha + 2 * kLatentRows * 4;    // [64]
    static constexpr int kBar = kFin + kLatentRows * 4;
    // full[kRing], empty[kRing], sfull[2], qfull, qempty, pfull, odone
    static constexpr int kNumBars = 2 * kRing + 6;
    static constexpr int kLost = kBar + kNumBars * 8;  // [3]
    static constexpr int kAddr = kLost + 3 * 8;        // tensor memory address
    static constexpr int kBad = kAddr + 8;             // [2] a block id outside the pool, [2]: a bad row set of the unit
    static constexpr int kTotal = kBad + 4 * 4;
    static_assert(kTotal <= 227 * 1024 && kBar % 8 == 0, "shared memory of one CTA");
};

// 16 lanes x 64 columns: thread l has columns 8 i + 2 (l % 4) + {0, 1} of lanes l / 4 (r[4 i], r[4 i + 1]) and l / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
    tmem_ld_wait32(r);
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)mine)
        : "memory");
    return r != 0;
}

template <bool kBF16, int BS>
__global__ void __launch_bounds__(kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmc, const DraftParams p) {
    using S = LatentSmem;
    using Cursor = DraftCursor<kLatentRows, kTile>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_addr(smem);
    const uint32_t full0 = sbase + S::kBar, empty0 = full0 + 8 * kRing, sfull0 = empty0 + 8 * kRing, qfull = sfull0 + 16,
                   qempty = qfull + 8, pfull = qempty + 8, odone = pfull + 8;
    unsigned long long* lost = reinterpret_cast<unsigned long long*>(smem + S::kLost);
    volatile int* bad = reinterpret_cast<volatile int*>(smem + S::kBad);

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        mbar_init(sfull0, 1);
        mbar_init(sfull0 + 8, 1);
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        mbar_init(pfull, kSoftWarps);
        mbar_init(odone, 1);
        for (int i = 0; i < 3; ++i) lost[i] = 0;
        bad[0] = bad[1] = 0;
        fence_barrier_init();
    }
    if (warp == kCopyWarp && lane == 0) {
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmc);
    }
    if (warp == kProductWarp) tmem_alloc(sbase + S::kAddr, kTmemCols);
    pdl_wait();
    pdl_launch_dependents();  // (the merge kernel waits for this one's end)
    if (tid == 0) {           // no partials yet
        p.part_desc[blockIdx.x * 4] = make_int4(0, 0, 0, 0);
        p.part_desc[blockIdx.x * 4 + 2] = make_int4(0, 0, 0, 0);
    }
    Cursor cur;
    draft_schedule<kLatentRows, kTile, kThreads, kLeast>(p, blockIdx.x, kValue, smem + S::kAlpha, cur);
    static_assert(draft_scratch<kThreads>() <= 2 * kLatentRows * 4, "the schedule's scratch");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + S::kAddr);
    DraftItem it;
    bool ok = true;  // no wait has run out

    if (warp == kCopyWarp) {
        // -------------------------------------------------------------- copies
        const uint64_t policy = l2_policy_evict_first();
        const uint32_t el = issuing_lane();
        int c = 0;  // tiles
        while (ok && cur.next(p, it)) {
            const int32_t* table = p.block_tables + (int64_t)it.s * p.max_blocks_per_seq;
            const int units = (it.q.L + kSlotKeys - 1) / kSlotKeys;
            int ids = 0;  // block ids of 32 slots, 8 tiles
            for (int t = it.t0; t < it.t1 && ok; ++t, ++c) {
                const int at = (t - it.t0) % (32 / kSlots) * kSlots;
                if (at == 0) {
                    const int j = t * kSlots + lane;
                    ids = j < units ? __ldg(table + j * kSlotKeys / BS) : 0;
                }
                int id = __shfl_sync(0xffffffffu, ids, at + lane % kSlots);
                const int j = t * kSlots + lane;
                const bool there = lane < kSlots && j < units;
                const bool wrong = there && (id < 0 || id >= p.num_blocks);
                if (wrong) id = 0;  // keep the shape; the unit's rows become zeros
                const bool any = __any_sync(0xffffffffu, wrong);
                if (any && lane == 0) record_error(p.err, PKV_DEVERR_BLOCK_ID);
                const uint32_t b = c & 1;
                if (c >= 2) ok = mbar_wait_warp(empty0 + 8 * b * kSlots, (c / 2 - 1) & 1);
                if (el && ok) bad[b] = any;
#pragma unroll
                for (int i = 0; i < kSlots; ++i) {
                    const uint32_t slot = b * kSlots + i, bar = full0 + 8 * slot;
                    if (c >= 2 && i > 0) ok = ok && mbar_wait_warp(empty0 + 8 * slot, (c / 2 - 1) & 1);
                    if (!ok) break;
                    const int jj = t * kSlots + i;
                    const int group = __shfl_sync(0xffffffffu, id, i) * (BS / 8) + (jj * kSlotKeys % BS) / 8;
                    if (jj < units) {
                        if (el) {
                            mbar_arrive_expect_tx(bar, kSlot);
                            tma_load_4d(sbase + S::kKV + slot * kSlot, &tmc, bar, 0, 0, 0, group, policy);
                        }
                    } else if (el) {
                        mbar_arrive(bar);  // behind the context: whatever lies there is masked
                    }
                }
            }
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
        // every copy has landed before the CTA ends
        if (lane == 0)
            for (int i = max(0, c - 2); i < c; ++i)
                for (int k = 0; k < kSlots; ++k) wait_bar(full0 + 8 * ((i & 1) * kSlots + k), (i / 2) & 1);
    } else if (warp == kQueryWarp) {
        // ------------------------------------------------------------- queries
        if (lane == 0) {
            int k = 0;
            while (ok && cur.next(p, it)) {
                if (k > 0) ok = wait_bar(qempty, (k - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(qfull, kParts * kLatentRows * 128);
                const int row = it.q.tok0 * p.num_q_heads + it.row0;
                for (int i = 0; i < kParts; ++i)
                    tma_load_2d(sbase + S::kQ + i * kLatentRows * 128, &tmq, qfull, 64 * i, row);
                ++k;
            }
            if (!ok) record_error(p.err, PKV_DEVERR_TIMEOUT);
            if (k > 0) wait_bar(qfull, (k - 1) & 1);
        }
    } else if (warp == kProductWarp) {
        // ------------------------------------------------------------ products
        // Whichever is ready goes first, P V (which frees slots) before Q K (of at most two tiles ahead): a fixed order
        // would have the one wait for copies that the other makes room for.
        const uint32_t el = issuing_lane(), tm = __shfl_sync(0xffffffffu, tmem, 0), sb = __shfl_sync(0xffffffffu, sbase, 0);
        const uint32_t id_s = umma_idesc(kBF16, kLatentRows, kTile, false, false);
        const uint64_t q_desc = umma_desc_sw128(sb + S::kQ, 16, 1024), k_desc = umma_desc_sw128(sb + S::kKV, 16, kGroup),
                       v_desc = umma_desc_sw128(sb + S::kKV, 1024, kGroup),
                       p_desc = umma_desc_sw128(sb + S::kP, 16, 1024);  // + (bytes / 16)
        constexpr uint32_t kTileStep = kSlots * kSlot / 16;
        uint32_t nk = 0, np = 0, nq = 0;        // tiles whose Q K, whose P V was issued; units begun
        int left = 0;                           // tiles of the unit whose Q K is still to come
        bool first = false, more = true;
        uint32_t pend_first = 0, pend_id[2];    // of the tiles between the two products: begins a unit (bits), P V's shape
        pend_id[0] = pend_id[1] = 0;
        uint32_t id_o = 0;
        uint32_t last_bar = 0, last_par = 0;
        uint64_t since = 0;  // of a wait
        while (ok) {
            if (left == 0 && more) {
                more = cur.next(p, it);
                left = __shfl_sync(0xffffffffu, more ? it.t1 - it.t0 : 0, 0);
                more = left > 0;
                id_o = umma_idesc(kBF16, 128, (__shfl_sync(0xffffffffu, it.rows, 0) + 15) / 16 * 16, true, false);
                first = true;
            }
            if (np < nk && mbar_test_warp(pfull, np & 1)) {
                tc_fence_after();
                const uint32_t b = np & 1, id = b ? pend_id[1] : pend_id[0], begins = pend_first >> b & 1;
                const uint64_t vd = v_desc + b * kTileStep;
#pragma unroll
                for (int ks = 0; ks < kSlots; ++ks) {
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
                        umma_f16_ss(el, tm + 64 * mt, vd + ks * (kSlot / 16) + mt * 128, p_desc + ks * 2, id, !begins || ks > 0);
                    umma_commit(el, empty0 + 8 * (b * kSlots + ks));
                }
                umma_commit(el, odone);
                last_bar = odone;
                last_par = np & 1;
                ++np;
                since = 0;
                continue;
            }
            if (left > 0 && nk - np < 2 && (!first || mbar_test_warp(qfull, nq & 1)) &&
                mbar_test_warp(full0 + 8 * ((nk & 1) * kSlots + kSlots - 1), (nk / 2) & 1)) {
                const uint32_t b = nk & 1;
                // (the slots before the last one landed before it, or soon will)
                for (int i = 0; i < kSlots - 1 && ok; ++i) ok = mbar_wait_warp(full0 + 8 * (b * kSlots + i), (nk / 2) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t kd = k_desc + b * kTileStep;
#pragma unroll 3
                for (int i = 0; i < kParts; ++i)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        umma_f16_ss(el, tm + 256 + 64 * b, q_desc + i * (kLatentRows * 128 / 16) + ks * 2,
                                    kd + i * 64 + ks * 2, id_s, i > 0 || ks > 0);
                --left;
                if (left == 0) umma_commit(el, qempty);
                umma_commit(el, sfull0 + 8 * b);
                last_bar = sfull0 + 8 * b;
                last_par = (nk / 2) & 1;
                pend_first = (pend_first & ~(1u << b)) | (uint32_t)first << b;
                if (b)
                    pend_id[1] = id_o;
                else
                    pend_id[0] = id_o;
                nq += first;
                first = false;
                ++nk;
                since = 0;
                continue;
            }
            if (!more && left == 0 && np == nk) break;
            const uint64_t now = global_timer_ns();
            if (since == 0) since = now;
            ok = __shfl_sync(0xffffffffu, now - since <= kWaitLimitNs, 0);
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
        // every product that was issued has ended before tensor memory is given back
        if (last_bar) wait_bar(last_bar, last_par);
    } else {
        // ------------------------------------------------------------- softmax
        const int ra = 16 * warp + (lane >> 2), rb = ra + 8;  // this thread's rows
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * warp) << 16);
        float* alpha = reinterpret_cast<float*>(smem + S::kAlpha);
        float* fin = reinterpret_cast<float*>(smem + S::kFin);
        int c = 0, k = 0;
        while (cur.next(p, it)) {
            const int base = it.q.L - it.q.n;
            const int ta = min((it.row0 + ra) / p.group, it.q.n - 1), tb = min((it.row0 + rb) / p.group, it.q.n - 1);
            const uint64_t mask_a = draft_mask(p, it.q, ta), mask_b = draft_mask(p, it.q, tb);
            float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
            bool wrong = false;
            for (int t = it.t0; t < it.t1; ++t, ++c) {
                const int b = c & 1;
                const bool guard = (t + 1) * kTile > base;
                // (the slot whose values this warp looks through below, and `bad` with it)
                ok = ok && wait_bar(sfull0 + 8 * b, (c / 2) & 1) && wait_bar(full0 + 8 * (b * kSlots + warp), (c / 2) & 1);
                ok = __all_sync(0xffffffffu, ok);
                float s[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] = 0.f;
                if (ok) {
                    wrong |= bad[b] != 0;
                    tc_fence_after();
                    tmem_ld_16x64(lane_addr + 256 + 64 * b, s);
                }
                const int pos0 = t * kTile + 2 * (lane & 3);
                const bool scaled = guard || !(p.scale_log2 > 0.f);
                const float f = scaled ? 1.f : p.scale_log2;
                if (scaled) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t sa = draft_visible(pos0 + 32 * h, base, mask_a),
                                       sb = draft_visible(pos0 + 32 * h, base, mask_b);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float& x = s[16 * h + 4 * i + e];
                                float& y = s[16 * h + 4 * i + 2 + e];
                                x = sa >> (8 * i + e) & 1 ? x * p.scale_log2 : -INFINITY;
                                y = sb >> (8 * i + e) & 1 ? y * p.scale_log2 : -INFINITY;
                            }
                    }
                }
                if (guard && ok) {
                    // the products of this tile's keys have ended: half of a token's value for each thread
                    const int key = tid >> 1, pos = t * kTile + key;
                    static_assert(kSlotKeys == 16 && kSlots == kSoftWarps, "a warp's keys are a slot's");
                    if (pos >= base) {
                        uint4* v = reinterpret_cast<uint4*>(smem + S::kKV + b * kSlots * kSlot + (key >> 3) * kGroup +
                                                            (key & 7) * 128 + (tid & 1) * 4096);
                        // (neighbouring threads start at different eighths of 128 bytes: the same would lie in the same banks)
                        if (scrub<kBF16>(32, pos < it.q.L, [&](int i) { return v + (i >> 3) * 64 + ((i + key) & 7); }))
                            atomicOr(lost + k % 3, 1ull << (pos - base));
                    }
                }
                float xa = -INFINITY, xb = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    xa = fmaxf(xa, fmaxf(s[4 * i], s[4 * i + 1]));
                    xb = fmaxf(xb, fmaxf(s[4 * i + 2], s[4 * i + 3]));
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, o));
                    xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, o));
                }
                xa *= f, xb *= f;
                float fa = 1.f, fb = 1.f;
                const bool raise_a = xa > ma + kRaise, raise_b = xb > mb + kRaise;
                if (raise_a) {
                    fa = ma == -INFINITY ? 0.f : exp2f(ma - xa);
                    ma = xa;
                    la *= fa;
                }
                if (raise_b) {
                    fb = mb == -INFINITY ? 0.f : exp2f(mb - xb);
                    mb = xb;
                    lb *= fb;
                }
                if ((lane & 3) == 0) {
                    alpha[b * kLatentRows + ra] = fa;
                    alpha[b * kLatentRows + rb] = fb;
                }
                const bool rescale = softmax_any(t > it.t0 && (raise_a || raise_b));
                const float na = kWeightExponent<kBF16> - (ma == -INFINITY ? 0.f : ma);
                const float nb = kWeightExponent<kBF16> - (mb == -INFINITY ? 0.f : mb);
                uint32_t wa[8], wb[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float a0 = fast_exp2(fmaf(s[4 * i], f, na)), a1 = fast_exp2(fmaf(s[4 * i + 1], f, na));
                    const float b0 = fast_exp2(fmaf(s[4 * i + 2], f, nb)), b1 = fast_exp2(fmaf(s[4 * i + 3], f, nb));
                    wa[i] = pack2<kBF16>(a0, a1);
                    wb[i] = pack2<kBF16>(b0, b1);
                    la += a0 + a1;
                    lb += b0 + b1;
                }
                // the product before has read P and is in O
                if (c > 0) ok = __all_sync(0xffffffffu, ok && wait_bar(odone, (c - 1) & 1));
                if (!ok) continue;
                if (rescale) {
                    tc_fence_after();
                    const float4* al = reinterpret_cast<const float4*>(alpha + b * kLatentRows);
#pragma unroll 1
                    for (int q = 0; q < 8; ++q) {  // 32 query rows of 128 values
                        float o[32];
                        tmem_ld32(lane_addr + 32 * q, o);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 a = al[(q & 1) * 8 + i];
                            o[4 * i] *= a.x, o[4 * i + 1] *= a.y, o[4 * i + 2] *= a.z, o[4 * i + 3] *= a.w;
                        }
                        tmem_st32(lane_addr + 32 * q, o);
                    }
                }
                // P: a row of 64 keys is 128 bytes, its 16-byte pieces swizzled by the row
                uint8_t* pb = smem + S::kP + ra * 128 + 4 * (lane & 3);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = (i ^ (ra & 7)) << 4;  // (rb % 8 is the same)
                    *reinterpret_cast<uint32_t*>(pb + at) = wa[i];
                    *reinterpret_cast<uint32_t*>(pb + 1024 + at) = wb[i];
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull);
            }
            // ---- the unit's end
            if (c > 0) ok = __all_sync(0xffffffffu, ok && wait_bar(odone, (c - 1) & 1));
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                la += __shfl_xor_sync(0xffffffffu, la, o);
                lb += __shfl_xor_sync(0xffffffffu, lb, o);
            }
            const bool part = it.partial(), zero = !ok || wrong;
            const int slot = blockIdx.x * 2 + (it.begins() ? 1 : 0);
            const int64_t prow = (int64_t)slot * kLatentRows;
            if ((lane & 3) == 0) {
                if (part) {
                    float2* ml = p.part_ml + prow;
                    if (ra < it.rows) ml[ra] = make_float2(ma, zero ? -1.f : la);
                    if (rb < it.rows) ml[rb] = make_float2(mb, zero ? -1.f : lb);
                    fin[ra] = fin[rb] = 1.f;
                } else {
                    fin[ra] = la != 0.f && !zero ? 1.f / la : 0.f;
                    fin[rb] = lb != 0.f && !zero ? 1.f / lb : 0.f;
                }
            }
            if (tid == 0) {
                lost[(k + 1) % 3] = 0;  // (read last before the barrier of the unit before)
                if (part) {
                    p.part_desc[slot * 2] =
                        make_int4(kPartValid | (it.ends() ? kPartEnds : 0), it.q.tok0, it.row0, it.rows);
                    p.part_desc[slot * 2 + 1] = make_int4(0, 0, 0, 0);
                }
            }
            softmax_sync();
            tc_fence_after();
            const unsigned long long gone = lost[k % 3];
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {  // 32 query rows of this lane's value d
                const int r0 = 32 * (q & 1), d = 128 * (q >> 1) + 32 * warp + lane;
                if (r0 >= it.rows) continue;
                float o[32];
                if (ok) {
                    tmem_ld32(lane_addr + 32 * q, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
                if (part) {
                    float* dst = p.part_o + (prow + r0) * kValue + d;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (r0 + i < it.rows) dst[(int64_t)i * kValue] = o[i];
                    continue;
                }
                // two neighbouring values of one row to a lane: lanes trade rows 2 i and 2 i + 1
                uint16_t* dst = static_cast<uint16_t*>(p.out) +
                                ((int64_t)it.q.tok0 * p.num_q_heads + it.row0 + r0 + (lane & 1)) * kValue + (d & ~1);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 in = *reinterpret_cast<const float2*>(fin + r0 + 2 * i);
                    const float x = in.x != 0.f ? o[2 * i] * in.x : 0.f, y = in.y != 0.f ? o[2 * i + 1] * in.y : 0.f;
                    const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? x : y, 1);
                    const uint32_t w = lane & 1 ? pack2<kBF16>(other, y) : pack2<kBF16>(x, other);
                    if (r0 + 2 * i + (lane & 1) < it.rows)
                        *reinterpret_cast<uint32_t*>(dst + (int64_t)2 * i * kValue) = w;
                }
            }
            if (gone) {
                // values that are not finite and were left out of the products, for the rows that attend them: a thread
                // takes four values of every row
                softmax_sync();
#pragma unroll 1
                for (unsigned long long at = zero ? 0 : gone; at; at &= at - 1) {
                    const int bit = __ffsll(at) - 1, pos = base + bit;
                    const int id = p.block_tables[(int64_t)it.s * p.max_blocks_per_seq + pos / BS];
#pragma unroll 1
                    for (int r = 0; r < it.rows; ++r)
                        if (draft_mask(p, it.q, (it.row0 + r) / p.group) >> bit & 1)
                            add_not_finite<kBF16>(
                                part ? p.part_o + (prow + r) * kValue + 4 * tid : nullptr,
                                static_cast<uint16_t*>(p.out) +
                                    ((int64_t)it.q.tok0 * p.num_q_heads + it.row0 + r) * kValue + 4 * tid,
                                static_cast<const uint16_t*>(p.values) + ((int64_t)id * BS + pos % BS) * kRow + 4 * tid, 4);
                }
            }
            tc_fence_before();
            ++k;
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kProductWarp) tmem_dealloc(tmem, kTmemCols);
}

template <bool kBF16, int BS>
cudaError_t launch_t(const DraftParams& p, const CUtensorMap& tmq, const CUtensorMap& tmc, cudaStream_t stream) {
    auto kern = latent_kernel<kBF16, BS>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LatentSmem::kTotal);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(p.pieces), dim3(kThreads), LatentSmem::kTotal, stream, tmq, tmc, p);
}

}  // namespace

cudaError_t launch_latent_decode(const DraftParams& in, int dtype, int block_size, const CUtensorMap& tmq, const CUtensorMap& tmc,
                                 cudaStream_t stream, int* launches) {
    DraftParams p = in;
    p.merged = draft_divides(p, kTile, kLatentRows, kLeast);
    const bool bf16 = dtype == PKV_BF16;
    const cudaError_t e =
        block_size == 16
            ? (bf16 ? launch_t<true, 16>(p, tmq, tmc, stream) : launch_t<false, 16>(p, tmq, tmc, stream))
            : (bf16 ? launch_t<true, 32>(p, tmq, tmc, stream) : launch_t<false, 32>(p, tmq, tmc, stream));
    if (e != cudaSuccess) return e;
    ++*launches;
    return p.merged ? launch_draft_merge(p, dtype, kValue, kLatentRows, stream, launches) : cudaSuccess;
}

}  // namespace pkv
