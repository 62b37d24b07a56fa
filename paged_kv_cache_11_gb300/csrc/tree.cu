// tree.cu -- paged_attention_tree: attention of the drafted tokens of each
// sequence (a tree or a chain, the last n positions of its context) over a
// paged K/V cache.
//
// The n x G query rows of a sequence and KV head (G query heads share it; row
// r is token r / G, head r % G) all read the same keys and values, so they are
// the M dimension of dense products on the 5th-generation tensor cores, 128
// keys at a time:
//   S = Q K^T   A = Q [128 rows x 128 dims] and B = K [128 keys x 128 dims],
//               both in shared memory, K-major, 128-byte swizzle
//   O += P V    A = P (16 bits, in tensor memory over the S that it was made
//               from), B = V, dims-major
// A unit takes up to 256 rows (256 rows of 2 x 2 x 128 operations a key and dim
// against 512 bytes of K and V a key: 256 operations a byte, near the 288 that
// the card has), so K and V leave HBM once for every 256 rows.
//
// Two streams, each with a buffer of Q, S and O and four softmax warps, keep
// the tensor core and the softmax at work at once.  A unit of more than 128
// rows gives each stream 128 of them, and both walk every tile of keys; one of
// fewer gives both streams all of its rows, and they walk the odd and the even
// tiles and join their sums at the end.
//
// Each thread of the softmax holds one row of S: the running maximum and sum
// need no exchange.  The maximum is raised, and O rescaled, only when a score
// passes it by 2^8 (weights up to 2^8 against the old one are as good).  A
// weight is rounded to the cache's 16-bit type for the product, half a step at
// most, 2^-8 (bf16), of each weight, some up and some down, where the output is
// rounded by as much (softmax_tile.cuh: fp16's range); the row's sum is that of
// the weights before, in 32 bits.
//
// Warps: 0-3 and 4-7 the streams' softmax, 8 the copies (one TMA copy for each
// block of K or V, as 8-token groups of 2 KiB, into a ring of five 32 KiB
// buffers that runs on across units), 9 the products, 10 and 11 the streams'
// queries.  Copies are marked as the first to leave L2, also where a sequence's
// next 256 rows walk them again (without the mark 8 x 32768 with 64/8 heads and 64
// tokens take 433 us for 428).
//
// Keys past the context, drafted tokens that a row does not descend from, and
// whatever the ring held before count nothing: their scores are replaced, not
// added to.  Their values meet weights of zero, which an infinity or NaN would
// turn into NaN; so in the tiles that any row masks, values past the context
// are zeroed and drafted values that are not finite are taken out, and added to
// the rows that do attend them when those are written.
//
// What bounds it.  Copies alone (the same kernel without products and softmax)
// run at 7.0 TB/s.  8 documents of 131072 tokens, 64/8 heads, 31 drafted tokens
// (4.3 GB): 870-930 us, 4.7 TB/s, 1.2 PFLOP/s, bound by the chain of a stream's
// tile, Q K, softmax, P V, of some 4100 cycles in which two tiles of rows are
// worked off (the copies' pace is 2800; without the softmax 775 us).  64
// contexts of 512 to 4096, 32/8 heads, 16 tokens (606 MB): 128-134 us, 4.6
// TB/s; 128 of up to 2048, 40 heads without sharing, 1 to 5 tokens (2.7 GB):
// 605-715 us from run to run, 3.8-4.5 TB/s: there the ends of units, when the
// last tile's softmax, product and output follow one another and the ring runs
// full, are what is left.  Tried and not kept: output by four warps of its own
// (they were as long as the chain they took over), twice the softmax warps, a
// loop for the products, the weights in one pass (softmax_tile.cuh), the first Q K
// of a unit before the last P V of the one before (what has to be remembered of a
// tile from one unit to the next costs more in every tile: 138 for 132 us).
#include "copies.cuh"
#include "drafted.cuh"
#include "softmax_tile.cuh"

namespace pkv {
namespace {

constexpr int kStreamWarps = 4;
constexpr int kCopyWarp = 2 * kStreamWarps;
constexpr int kProductWarp = kCopyWarp + 1;
constexpr int kQueryWarp = kProductWarp + 1;  // and the next: one for each stream
constexpr int kThreads = (kQueryWarp + 2) * 32;
constexpr int kTile = 128;                 // keys
constexpr int kRing = 5;                   // 32 KiB buffers of K or V, in turn
constexpr int kBuf = kTile * kHeadDim * 2;
constexpr int kLeast = 4;                  // tiles of a piece
constexpr uint32_t kTmemCols = 512;        // S and P of the streams: [0, 128), [128, 256); O: [256, 384), [384, 512)

struct TreeSmem {
    static constexpr int kQ = 0;  // [2 streams][2 dims halves][128 rows][128 B]
    static constexpr int kKV = kQ + 2 * kBuf;
    static constexpr int kXch = kKV + kRing * kBuf;  // [256] maximum and sum of each thread of the softmax
    static constexpr int kBar = kXch + 256 * 8;
    // full[kRing], empty[kRing], qfull[2], sfull[2], pfull[2], odone[2], qempty[2]
    static constexpr int kNumBars = 2 * kRing + 10;
    static constexpr int kLost = kBar + kNumBars * 8;   // [3] drafted tokens whose values were taken out
    static constexpr int kSlot = kLost + 3 * 8;         // tensor memory address
    static constexpr int kBad = kSlot + 8;              // [kRing] a block id outside the pool
    static constexpr int kTotal = kBad + kRing * 4 + 4;
    static_assert(kTotal <= 227 * 1024 && kBar % 8 == 0, "shared memory of one CTA");
    static_assert(draft_scratch<kThreads>() <= kBuf, "the schedule's scratch lies where Q will");
};

__device__ __forceinline__ void both_streams() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <bool kBF16, int BS>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const DraftParams p) {
    using S = TreeSmem;
    using Cursor = DraftCursor<kTreeRows, kTile>;
    constexpr int D = kHeadDim, kBlocks = kTile / BS;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_addr(smem);
    const uint32_t full0 = sbase + S::kBar, empty0 = full0 + 8 * kRing, qfull0 = empty0 + 8 * kRing, sfull0 = qfull0 + 16,
                   pfull0 = sfull0 + 16, odone0 = pfull0 + 16, qempty0 = odone0 + 16;
    unsigned long long* lost = reinterpret_cast<unsigned long long*>(smem + S::kLost);
    volatile int* bad = reinterpret_cast<volatile int*>(smem + S::kBad);

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
            bad[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(qfull0 + 8 * i, 1);
            mbar_init(qempty0 + 8 * i, 1);
            mbar_init(sfull0 + 8 * i, 1);
            mbar_init(pfull0 + 8 * i, kStreamWarps);
            mbar_init(odone0 + 8 * i, 1);
        }
        for (int i = 0; i < 3; ++i) lost[i] = 0;
        fence_barrier_init();
    }
    if (warp == kCopyWarp && lane == 0) {
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    if (warp == kProductWarp) tmem_alloc(sbase + S::kSlot, kTmemCols);
    pdl_wait();
    pdl_launch_dependents();  // (the merge kernel waits for this one's end)
    if (tid == 0) {           // no partials yet
        p.part_desc[blockIdx.x * 4] = make_int4(0, 0, 0, 0);
        p.part_desc[blockIdx.x * 4 + 2] = make_int4(0, 0, 0, 0);
    }
    Cursor cur;
    draft_schedule<kTreeRows, kTile, kThreads, kLeast>(p, blockIdx.x, D, smem + S::kQ, cur);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + S::kSlot);
    DraftItem it;
    bool ok = true;  // no wait has run out

    if (warp == kCopyWarp) {
        // -------------------------------------------------------------- copies
        const uint64_t policy = l2_policy_evict_first();
        int k = 0;  // buffers filled: K and V of each tile in turn
        while (ok && cur.next(p, it)) {
            const int32_t* table = p.block_tables + (int64_t)it.s * p.max_blocks_per_seq;
            const int nblk = (it.q.L + BS - 1) / BS;  // <= max_blocks_per_seq
            int ids = 0;                              // 32 block ids, of 32 / kBlocks tiles
            for (int t = it.t0; t < it.t1 && ok; ++t) {
                const int at = (t - it.t0) % (32 / kBlocks) * kBlocks;
                if (at == 0) {
                    const int j = t * kBlocks + lane;
                    ids = j < nblk ? __ldg(table + j) : 0;
                }
                int id = __shfl_sync(0xffffffffu, ids, at + lane % kBlocks);
                const int nb = min(kBlocks, nblk - t * kBlocks);
                const bool wrong = lane < nb && (id < 0 || id >= p.num_blocks);
                if (wrong) id = 0;  // keep the shape; the unit's rows become zeros
                const bool any = __any_sync(0xffffffffu, wrong);
                if (any && lane == 0) record_error(p.err, PKV_DEVERR_BLOCK_ID);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++k) {
                    const int b = k % kRing;
                    if (lane == 0 && k >= kRing) ok = wait_bar(empty0 + 8 * b, (k / kRing - 1) & 1);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == 0) {
                        bad[b] = any;
                        mbar_arrive_expect_tx(full0 + 8 * b, (uint32_t)nb * BS * D * 2);
                    }
                    __syncwarp();
                    if (lane < nb)
                        tma_load_4d(sbase + S::kKV + b * kBuf + lane * BS * D * 2, kv ? &tmv : &tmk, full0 + 8 * b, 0, 0, 0,
                                    (id * p.num_kv_heads + it.kvh) * (BS / 8), policy);
                }
            }
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
        // every copy has landed before the CTA ends
        if (lane == 0)
            for (int i = max(0, k - kRing); i < k; ++i) wait_bar(full0 + 8 * (i % kRing), (i / kRing) & 1);
    } else if (warp == kProductWarp) {
        // ------------------------------------------------------------ products
        const uint32_t el = issuing_lane(), tm = __shfl_sync(0xffffffffu, tmem, 0), sb = __shfl_sync(0xffffffffu, sbase, 0);
        const uint32_t id_s = umma_idesc(kBF16, 128, kTile, false, false), id_o = umma_idesc(kBF16, 128, D, false, true);
        const uint64_t q_desc = umma_desc_sw128(sb + S::kQ, 16, 1024), k_desc = umma_desc_sw128(sb + S::kKV, 16, 2048),
                       v_desc = umma_desc_sw128(sb + S::kKV, 1024, 2048);  // + (bytes / 16)
        uint32_t last_bar = 0, last_par = 0;
        uint32_t tile0 = 0, par0 = 0, units = 0;  // tiles so far; bits of the streams: their tiles, their units
        for (;;) {
            const bool more = cur.next(p, it);
            const int n = __shfl_sync(0xffffffffu, more && ok ? it.t1 - it.t0 : 0, 0);
            const bool two = __shfl_sync(0xffffffffu, it.rows, 0) > 128;
            if (n == 0) break;
            const int sh = two ? 0 : 1;  // a stream's tile t of the unit is its (t >> sh)-th
            // the tile whose P V is still to come: QK of the next tile goes first, so that the tensor core has
            // work while the softmax has its turn
            int pend_x = -1, pend_t = 0;
            const auto values = [&]() {
                const uint32_t x = pend_x, t = pend_t, pb = (2 * (tile0 + t) + 1) % kRing;
                pend_x = -1;
                ok = mbar_wait_warp(pfull0 + 8 * x, (par0 >> x ^ t >> sh) & 1);  // (the softmax has waited for V)
                if (!ok) return;
                tc_fence_after();
                const uint64_t vd = v_desc + pb * (kBuf / 16);
#pragma unroll
                for (int ks = 0; ks < kTile / 16; ++ks)
                    umma_f16_ts(el, tm + 256 + 128 * x, tm + 128 * x + 8 * ks, vd + ks * 256, id_o, t >> sh > 0 || ks > 0);
                if (!two || x == 1) umma_commit(el, empty0 + 8 * pb);
                if ((int)t + 1 + sh >= n) {  // the stream's last of the unit
                    umma_commit(el, odone0 + 8 * x);
                    last_bar = odone0 + 8 * x;
                    last_par = units >> x & 1;
                }
            };
            for (int t = 0; t < n && ok; ++t) {
                const uint32_t kk = 2 * (tile0 + t), kb = kk % kRing;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!two && x != (kk >> 1 & 1)) continue;
                    if (pend_x == x && ok) values();  // P of this stream lies where S goes
                    if (t >> sh == 0 && ok) ok = mbar_wait_warp(qfull0 + 8 * x, units >> x & 1);
                    ok = ok && mbar_wait_warp(full0 + 8 * kb, (kk / kRing) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t qd = q_desc + x * (kBuf / 16), kd = k_desc + kb * (kBuf / 16);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        umma_f16_ss(el, tm + 128 * x, qd + (ks >> 2) * 1024 + (ks & 3) * 2, kd + (ks >> 2) * 64 + (ks & 3) * 2,
                                    id_s, ks > 0);
                    if (!two || x == 1) umma_commit(el, empty0 + 8 * kb);
                    umma_commit(el, sfull0 + 8 * x);
                    last_bar = sfull0 + 8 * x;
                    last_par = (par0 >> x ^ t >> sh) & 1;
                    if (pend_x >= 0) values();
                    pend_x = x;
                    pend_t = t;
                }
            }
            if (!ok) break;
            // tiles of each stream
            const int x1 = tile0 & 1, c0 = two ? n : (n + 1 - x1) >> 1, c1 = two ? n : (n + x1) >> 1;
            // every Q K has been issued: the queries may be replaced when they have ended
            if (c0 > 0) umma_commit(el, qempty0);
            if (c1 > 0) umma_commit(el, qempty0 + 8);
            values();
            tile0 += n;
            par0 ^= (c0 & 1) | (c1 & 1) << 1;
            units ^= (c0 > 0) | (c1 > 0) << 1;
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
        // every product that was issued has ended before tensor memory is given back
        if (last_bar) wait_bar(last_bar, last_par);
    } else if (warp >= kQueryWarp) {
        // ------------------------------------------------------------- queries
        // Q of each unit into the stream's buffer, as soon as the unit before has no product with it left: 16 lanes to
        // a row of 256 bytes
        const int X = warp - kQueryWarp;
        int k = 0, j = 0;  // units of this stream, tiles
        while (ok && cur.next(p, it)) {
            const bool two = it.rows > 128;
            const int tiles = it.t1 - it.t0, j0 = j;
            j += tiles;
            if (!two && tiles == 1 && (j0 & 1) != X) continue;  // no tile of this unit is this stream's
            if (k > 0) ok = mbar_wait_warp(qempty0 + 8 * X, (k - 1) & 1);
            if (!ok) break;
            ++k;
            const int first = two ? 128 * X : 0, rows = min(128, it.rows - first), c = lane & 15;
            for (int r0 = 0; r0 < rows; r0 += 2) {
                const int r = r0 + (lane >> 4);
                if (r < rows) {
                    const int row = it.row0 + first + r, token = row / p.group, g = row - token * p.group;
                    cp_async16(sbase + S::kQ + X * kBuf + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                               static_cast<const uint16_t*>(p.q) +
                                   ((int64_t)(it.q.tok0 + token) * p.num_q_heads + it.kvh * p.group + g) * D + 8 * c);
                }
            }
            cp_async_wait_all();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull0 + 8 * X);
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
    } else {
        // ------------------------------------------------------------- softmax
        const int X = warp >> 2, r = tid & 127;  // stream, row of its tile (tensor memory lane)
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t s_addr = lane_addr + 128 * X, o_addr = lane_addr + 256;
        float2* xch = reinterpret_cast<float2*>(smem + S::kXch);
        int ns = 0, no[2] = {0, 0};  // tiles of this stream; units of both
        int j = 0, k = 0;            // tiles, items
        bool more = cur.next(p, it);
        const auto row_mask = [&](const DraftItem& n) -> uint64_t {
            const int row = (n.rows > 128 ? 128 * X : 0) + r;
            return row < n.rows ? draft_mask(p, n.q, (n.row0 + row) / p.group) : 0;
        };
        uint64_t mask = more ? row_mask(it) : 0;
        while (more) {
            const bool two = it.rows > 128;
            const int row = (two ? 128 * X : 0) + r;
            const bool live = (two ? 128 * X : 0) + 32 * (warp & 3) < it.rows;  // some row of the warp is real
            const int token = min((it.row0 + row) / p.group, it.q.n - 1);
            const int base = it.q.L - it.q.n;
            // (a lane without a row, whose scores are anything, never asks for a raise)
            float m_run = row < it.rows ? -INFINITY : INFINITY, l = 0.f;
            bool begun = false, wrong = false;
            for (int t = it.t0; t < it.t1; ++t, ++j) {
                const bool mine = two || (j & 1) == X;
                const bool guard = (t + 1) * kTile > base;
                const int vk = 2 * j + 1;
                if (mine) {
                    ok = __all_sync(0xffffffffu, ok && wait_bar(sfull0 + 8 * X, ns & 1));
                    ++ns;
                }
                if (live && ok && mine) {
                    tc_fence_after();
                    softmax_tile<kBF16>(s_addr, o_addr + 128 * X, guard, p.scale_log2, begun, m_run,
                                        l, [&](int c) { return draft_visible(t * kTile + c, base, mask); });
                    tc_fence_before();
                }
                if (mine) ok = __all_sync(0xffffffffu, ok && wait_bar(full0 + 8 * (vk % kRing), (vk / kRing) & 1));
                if (guard && ok && mine) {
                    // this thread's token of V: all of a tile that is the stream's own, half of one that both walk
                    const int tk = two ? 64 * X + (r >> 1) : r;
                    const int pos = t * kTile + tk;
                    if (pos >= base) {
                        uint4* v = reinterpret_cast<uint4*>(smem + S::kKV + (vk % kRing) * kBuf + (tk >> 3) * 2048 +
                                                            (tk & 7) * 128 + (two ? (r & 1) * 1024 : 0));
                        // (neighbouring threads start at different eighths of 128 bytes: the same would lie in the same banks)
                        if (scrub<kBF16>(two ? 8 : 16, pos < it.q.L, [&](int i) { return v + (i >> 3) * 64 + ((i + tk) & 7); }))
                            atomicOr(lost + k % 3, 1ull << (pos - base));
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                if (guard && two) both_streams();
                if (!mine || !ok) continue;
                begun = true;
                wrong |= bad[vk % kRing] != 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull0 + 8 * X);
            }
            // ---- the unit's end: the next unit's masks are fetched first
            const DraftItem done = it;
            more = cur.next(p, it);
            const uint64_t next_mask = more ? row_mask(it) : 0;  // (on its way during the output)
            xch[tid] = make_float2(m_run, wrong || !ok ? -1.f : l);
            if (tid == 0) lost[(k + 1) % 3] = 0;  // (read last before the barrier of the unit before)
            both_streams();
            const int x0 = two ? X : 0, x1 = two ? X + 1 : 2;
            // products whose sums are read: this stream's, or those of both where they walked a tile of the unit
            bool has[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                has[x] = x >= x0 && x < x1 && (two || done.t1 - done.t0 > 1 || ((j - 1) & 1) == x);
                if (has[x]) ok = ok && wait_bar(odone0 + 8 * x, no[x] & 1);
                no[x] += two || done.t1 - done.t0 > 1 || ((j - 1) & 1) == x;
            }
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            const unsigned long long gone = lost[k % 3];
            float m = m_run, f0 = 1.f, f1 = 1.f, sum = l;
            bool zero = !ok || wrong;
            if (!two) {
                const float2 a = xch[r], b = xch[128 + r];
                m = fmaxf(a.x, b.x);
                const float ms = m == -INFINITY ? 0.f : m;
                f0 = exp2f(a.x - ms), f1 = exp2f(b.x - ms);
                zero = !ok || a.y < 0.f || b.y < 0.f;
                sum = (has[0] ? a.y * f0 : 0.f) + (has[1] ? b.y * f1 : 0.f);
            }
            const bool part = done.partial();
            const int64_t prow = (int64_t)(blockIdx.x * 2 + (done.begins() ? 1 : 0)) * kTreeRows + row;
            // this thread's dims: all of its row, or with both streams on one row the stream's half; the streams go on to
            // their next tiles once both have read
            const int c0 = two ? 0 : 2 * X, c1 = two ? 4 : 2 * X + 2;
            const int head = done.kvh * p.group + done.row0 + row - token * p.group;
            const float g0 = two ? 1.f : f0, g1 = two ? 1.f : f1;
            const float inv = zero || sum == 0.f ? 0.f : 1.f / sum;  // (NaN stays)
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0.f;
                if (live && ok) {
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {
                        if (!(x ? has[1] : has[0])) continue;
                        const float g = x ? g1 : g0;
                        float v[32];
                        tmem_ld32_start(o_addr + 128 * x + 32 * c, v);
                        tmem_ld_wait32(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = fmaf(v[i], g, o[i]);
                    }
                }
                if (c + 1 == c1) {
                    tc_fence_before();
                    both_streams();
                    tc_fence_after();
                }
                if (row >= done.rows) continue;
                if (part) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + 32 * c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                                          ((int64_t)(done.q.tok0 + token) * p.num_q_heads + head) * D + 32 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = inv == 0.f ? 0u : pack2<kBF16>(o[8 * i + 2 * e] * inv, o[8 * i + 2 * e + 1] * inv);
                        dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            if (row < done.rows && !zero) {
                // values that are not finite and were left out of the products, of the tokens that this item walked
                for (unsigned long long at = gone & mask; at; at &= at - 1) {
                    const int pos = base + __ffsll(at) - 1;
                    if (pos / kTile < done.t0 || pos / kTile >= done.t1) continue;
                    const int id = p.block_tables[(int64_t)done.s * p.max_blocks_per_seq + pos / BS];
                    add_not_finite<kBF16>(part ? p.part_o + prow * D + 32 * c0 : nullptr,
                                          static_cast<uint16_t*>(p.out) +
                                              ((int64_t)(done.q.tok0 + token) * p.num_q_heads + head) * D + 32 * c0,
                                          static_cast<const uint16_t*>(p.values) +
                                              (((int64_t)id * p.num_kv_heads + done.kvh) * BS + pos % BS) * D + 32 * c0,
                                          32 * (c1 - c0));
                }
            }
            if (part && row < done.rows && (two || X == 0)) {
                p.part_ml[prow] = make_float2(m, zero ? -1.f : sum);
            }
            if (part && tid == 0) {
                int4* d = p.part_desc + (blockIdx.x * 2 + (done.begins() ? 1 : 0)) * 2;
                d[0] = make_int4(kPartValid | (done.ends() ? kPartEnds : 0), done.q.tok0, done.row0, done.rows);
                d[1] = make_int4(done.kvh, 0, 0, 0);
            }
            mask = next_mask;
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
cudaError_t launch_t(const DraftParams& p, const CUtensorMap& tmk, const CUtensorMap& tmv, cudaStream_t stream) {
    auto kern = tree_kernel<kBF16, BS>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeSmem::kTotal);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(p.pieces), dim3(kThreads), TreeSmem::kTotal, stream, tmk, tmv, p);
}

}  // namespace

cudaError_t launch_tree(const DraftParams& in, int dtype, int block_size, const CUtensorMap& tmk, const CUtensorMap& tmv,
                        cudaStream_t stream, int* launches) {
    DraftParams p = in;
    p.merged = draft_divides(p, kTile, kTreeRows, kLeast);
    const bool bf16 = dtype == PKV_BF16;
    const cudaError_t e = block_size == 16 ? (bf16 ? launch_t<true, 16>(p, tmk, tmv, stream) : launch_t<false, 16>(p, tmk, tmv, stream))
                                           : (bf16 ? launch_t<true, 32>(p, tmk, tmv, stream) : launch_t<false, 32>(p, tmk, tmv, stream));
    if (e != cudaSuccess) return e;
    ++*launches;
    return p.merged ? launch_draft_merge(p, dtype, kHeadDim, kTreeRows, stream, launches) : cudaSuccess;
}

}  // namespace pkv
