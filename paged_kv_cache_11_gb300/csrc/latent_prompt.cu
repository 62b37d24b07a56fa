// latent_prompt.cu -- latent_attention_prefill: causal attention of whole
// prompts in the expanded form of latent attention.  Each head has keys of 128
// values of its own beside the 64 that all heads share, and values of 128:
//   S = scale (Q_n K_n^T + Q_r K_r^T),  O = softmax(S) V
// 640 operations a (query, key, head): the tensor cores bound it.
//
// A CTA takes 256 queries of one head and walks the keys 128 at a time.  Two
// streams of 128 queries each, with their own Q (shared memory), S, P and O
// (tensor memory) and four softmax warps, take turns: while one's products run,
// the other is in its softmax (softmax_tile.cuh has its arithmetic).  Both
// streams use each tile of keys and values before it is given back.
//
// Shared memory is Q (2 x 48 KiB) and a ring of eight 16 KiB units of 128
// tokens x 64 values: a tile of keys is three units, a tile of values two, in
// turn.  Eight units back from those of keys t lie values t - 2, and from those
// of values t keys t - 1: that is all that a copy waits for, and a tile of
// either kind has one barrier.
//
// The strips of 256 queries of all prompts stand in a line, a prompt's last (and
// longest) first, and the grid is that line for every head.  The host knows an
// upper bound of its length, from the tokens, the prompts and the longest of them;
// a CTA counts the strips before each prompt (or before every so many, past 512
// prompts) when it starts, and a warp looks a place up, 32 prompts or counts at a
// time; up to 32 prompts it goes by their lengths alone.  (A place for each prompt
// and strip of the longest would be 1e9 places for the 2e5 strips of 16384 prompts
// whose longest is not known.  1024 prompts of 64 tokens with 8 heads take 225 us
// with and without a bound, so 220 with one and 6200 without; one prompt of 4000
// tokens among 200 of 40 takes 198, so 258; one of 100 alone 7.0, so 6.85.)  A
// place behind the line's end costs a claim, 1 us: 20000 sequences of which 50 have
// new tokens, 7 each, with 64 heads 250 us for the 50 sequences' 100.
//
// A CTA that has issued the copies of its queries' last tile takes the place of
// one that has not begun (a cluster launch control request) and goes on with that
// one's queries and keys, so that they are on their way while the last tiles are
// worked off, and barriers and tensor memory are set up once: 16 prompts of 256 tokens
// with 128 heads 137 us for 168, 8 of 1024 426 for 477, one of 16384 with 64
// heads 3.38 ms for 3.47.  (Claimed one item earlier, the grid's last items wait
// behind long ones: 7 ragged prompts 175 us for 169.)  Grids of one CTA an SM at
// most claim nothing.
//
// What bounds it: two prompts of 8192 tokens with 128 heads (5.5 TFLOP) take 3.79
// to 3.89 ms, 1.44 PFLOP/s, 75% of the card's peak and 82% of what it sustains
// under its power limit.  Without the softmax the products alone take 3.6 ms; the
// rest is the part of a stream's softmax that the other's products do not cover,
// and there every instruction of the product warp between a stream's P and its
// next S counts: flags of its tiles carried from one item to the next cost 5%, the
// loop over streams not unrolled 10%.  (A warp for each stream's products: 3.92
// against 3.90 ms.)  Seven prompts of 1 to 1537 tokens with 40 heads: 169 us.
#include <algorithm>

#include "copies.cuh"
#include "latent.cuh"
#include "softmax_tile.cuh"

namespace pkv {
namespace {

constexpr int kStreamWarps = 4;
constexpr int kCopyWarp = 2 * kStreamWarps, kProductWarp = kCopyWarp + 1;
constexpr int kThreads = (kProductWarp + 1) * 32;
constexpr int kTakers = 1 + 2 * kStreamWarps;  // the warps that read an item which the copies' has posted
constexpr int kRows = 256;               // queries of a CTA
constexpr int kTile = 128;               // keys
constexpr int kUnit = kTile * 128;       // bytes of a ring unit
constexpr int kKeyUnits = 3, kTileUnits = 5;
constexpr int kRing = 8;
constexpr int kMarks = 512;              // of the line of strips: where every so many prompts begin
constexpr int kLostTiles = 3;            // tiles that some of a CTA's queries mask: 255 keys and a part of one more
constexpr uint32_t kTmemCols = 512;      // S and P of the streams: [0, 128), [128, 256); O: [256, 384), [384, 512)

struct PromptSmem {
    static constexpr int kQ = 0;  // [2 streams][3 parts][128 rows][128 B]
    static constexpr int kKV = kQ + 2 * kKeyUnits * kUnit;
    static constexpr int kBar = kKV + kRing * kUnit;
    // keys landed[2], values landed[2], keys read[2], values read[2] (by the tile's parity), qfull[2], sfull[2], pfull[2],
    // odone[2], qempty[2]; ifull, iempty, claim
    static constexpr int kNumBars = 22;  // (one more keeps what follows 16-byte aligned)
    static constexpr int kAddr = kBar + kNumBars * 8;  // tensor memory address
    static constexpr int kItem = kAddr + 16;           // an Item
    static constexpr int kClaim = kItem + 32;          // the answer to a claim
    // [3 items in turn][12] keys whose values were taken out, from the first masked tile on
    static constexpr int kLost = kClaim + 16;
    static constexpr int kMark = kLost + 3 * kLostTiles * 4 * 4;  // [kMarks + 1]
    static constexpr int kSum = kMark + (kMarks + 1) * 4;         // [8] of the warps that count
    static constexpr int kTotal = kSum + 8 * 4;
    static_assert(kTotal <= 227 * 1024 && kBar % 16 == 0 && kClaim % 16 == 0, "shared memory of one CTA");
};

// Up to 256 queries of a prompt and a head.  Query i attends the first seen0 + i keys.
struct Item {
    int row, rows, head, seen0;  // first token in q; rows == 0: no more items
    int key, keys;               // first token in kv
    __device__ __forceinline__ int tiles(int x) const {  // of a stream
        const int n = min(rows, 128 * (x + 1));
        return n > 128 * x ? max(0, seen0 + n - 1 + kTile - 1) / kTile : 0;
    }
};

// Asks for a CTA of this grid that has not begun; the answer, 16 bytes, arrives at `dst` and on `bar`.
__device__ __forceinline__ void claim_cta(uint32_t dst, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
                 "r"(bar)
                 : "memory");
}
// Was there one, and its place in the grid.
__device__ __forceinline__ bool claimed_cta(uint32_t src, dim3& at) {
    uint32_t got, x, y, z;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%4];\n\t"
        "mov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, %3, _}, h;\n\t}"
        : "=&r"(got), "=&r"(x), "=&r"(y), "=&r"(z)
        : "r"(src)
        : "memory");
    at = dim3(x, y, z);
    return got != 0;
}

__device__ __forceinline__ void both_streams() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// 32 keys from c on as bits: those before `seen`.
__device__ __forceinline__ uint32_t before(int c, int seen) {
    return seen - c >= 32 ? ~0u : seen > c ? (1u << (seen - c)) - 1 : 0u;
}

// Strips of a prompt whose queries are tokens a0 .. a1 - 1: 0 where these are no rows.
__device__ __forceinline__ int strips_of(int a0, int a1, int num_queries, int max_query_len) {
    return a0 < 0 || a1 < a0 || a1 > num_queries ? 0 : (min(a1 - a0, max_query_len) + kRows - 1) / kRows;
}

__device__ __forceinline__ bool bad_prompt(const LatentPromptParams& p, int a0, int a1, int b0, int b1) {
    return a0 < 0 || a1 < a0 || a1 > p.num_queries || b0 < 0 || b1 < b0 || b1 > p.num_keys || a1 - a0 > p.max_query_len;
}

// marks[i] = strips of the prompts before i * per, up to i = used (a whole CTA; a barrier of the caller's follows).  Counts end
// at the grid's length, which only bad metadata (prompts over one another) passes; that is recorded here.
__device__ __noinline__ void mark_strips(const LatentPromptParams& p, int per, int used, int* marks, int* sums) {
    const int tid = threadIdx.x, lane = tid & 31, most = (int)gridDim.x;
    int mine[2] = {0, 0}, scan = 0;
    if (2 * (tid & ~31) < used) {  // (whole warps)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            for (int s = (2 * tid + h) * per; s < min((2 * tid + h + 1) * per, p.num_seqs); ++s) {
                const int a0 = p.query_starts[s], a1 = p.query_starts[s + 1], b0 = p.key_starts[s], b1 = p.key_starts[s + 1];
                if (bad_prompt(p, a0, a1, b0, b1)) record_error(p.err, PKV_DEVERR_QUERY);
                mine[h] = min(most, mine[h] + strips_of(a0, a1, p.num_queries, p.max_query_len));
            }
        scan = mine[0] + mine[1];  // inclusive over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
        }
        if (lane == 31) sums[tid >> 5] = min(most, scan);
    }
    if (used > 64) __syncthreads();
    if (2 * tid >= used) return;
    int before = scan - mine[0] - mine[1];
    for (int w = 0; w < tid >> 5; ++w) before += sums[w];
    if (tid == 0) marks[0] = 0;
    marks[2 * tid + 1] = min(most, before + mine[0]);
    marks[2 * tid + 2] = min(most, before + mine[0] + mine[1]);
}

// Strip x of the line: the prompt that it is in (-1: x is behind the line's end), and its number there.  A whole warp.
__device__ __noinline__ int2 find_strip(const LatentPromptParams& p, int per, int used, const int* marks, int x) {
    const int lane = threadIdx.x & 31;
    int s = 0, count = p.num_seqs;  // prompts that it is among
    if (count > 32) {
        if (x >= marks[used]) return make_int2(-1, 0);
        // the last mark that x has come to: of those sixteen apart, then of sixteen
        static_assert(kMarks == 32 * 16, "two looks");
        int i = 16 * lane;
        unsigned passed = __ballot_sync(0xffffffffu, i < used && marks[i] <= x);
        const int from = 16 * (31 - __clz(passed));
        i = from + (lane & 15);
        passed = __ballot_sync(0xffffffffu, lane < 16 && i < used && marks[i] <= x);
        i = from + 31 - __clz(passed);
        x -= marks[i];
        if (per == 1) return make_int2(i, x);
        s = i * per;
        count = min(per, count - s);
    }
    for (;; s += 32, count -= 32) {
        const int mine =
            lane < count ? strips_of(p.query_starts[s + lane], p.query_starts[s + lane + 1], p.num_queries, p.max_query_len) : 0;
        int scan = mine;  // inclusive over the warp
        for (int o = 1; o < min(32, count); o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
        }
        const unsigned in = __ballot_sync(0xffffffffu, lane < count && x < scan);
        if (in) return make_int2(s + __ffs(in) - 1, x - __shfl_sync(0xffffffffu, scan - mine, __ffs(in) - 1));
        if (count <= 32) return make_int2(-1, 0);
        x -= __shfl_sync(0xffffffffu, scan, 31);
    }
}

// The rows of a prompt with bad metadata become zeros, whatever their number: a head's, from query q0 on, 256 for each of its
// strips.
__device__ __noinline__ void zero_prompt(const LatentPromptParams& p, int a0, int a1, int q0, int strips, int head) {  // (a whole warp)
    const int lane = threadIdx.x & 31;
    uint16_t* out = static_cast<uint16_t*>(p.out);
    for (int64_t r = q0; r < a1 - a0; r += (int64_t)strips * kRows)
        for (int i = lane; i < min((int64_t)kRows, a1 - a0 - r) * 16; i += 32)
            *reinterpret_cast<uint4*>(out + ((a0 + r + i / 16) * p.num_heads + head) * 128 + i % 16 * 8) = make_uint4(0, 0, 0, 0);
}

// The wait for an item: the copies' lane may be looking through many empty places.
__device__ __noinline__ bool wait_item(uint32_t bar, uint32_t parity) { return mbar_wait_for(bar, parity, 32 * kWaitLimitNs); }

template <bool kBF16>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prompt_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmkv,
                         const __grid_constant__ CUtensorMap tmr, const __grid_constant__ LatentPromptParams p) {
    using S = PromptSmem;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_addr(smem);
    const uint32_t kfull0 = sbase + S::kBar, vfull0 = kfull0 + 16, kread0 = vfull0 + 16, vread0 = kread0 + 16,
                   qfull0 = vread0 + 16, sfull0 = qfull0 + 16, pfull0 = sfull0 + 16, odone0 = pfull0 + 16,
                   qempty0 = odone0 + 16, ifull = qempty0 + 16, iempty = ifull + 8, claim = iempty + 8;
    uint32_t* lost = reinterpret_cast<uint32_t*>(smem + S::kLost);
    uint16_t* out = static_cast<uint16_t*>(p.out);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(kfull0 + 8 * i, 1);
            mbar_init(vfull0 + 8 * i, 1);
            mbar_init(kread0 + 8 * i, 1);
            mbar_init(vread0 + 8 * i, 1);
            mbar_init(qfull0 + 8 * i, 1);
            mbar_init(sfull0 + 8 * i, 1);
            mbar_init(pfull0 + 8 * i, kStreamWarps);
            mbar_init(odone0 + 8 * i, 1);
            mbar_init(qempty0 + 8 * i, 1);
        }
        mbar_init(ifull, 1);
        mbar_init(iempty, kTakers);
        mbar_init(claim, 1);
        for (int i = 0; i < 3 * kLostTiles * 4; ++i) lost[i] = 0;
        fence_barrier_init();
    }
    if (warp == kCopyWarp && lane == 0) {
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmkv);
        prefetch_tensormap(&tmr);
    }
    if (warp == kProductWarp) tmem_alloc(sbase + S::kAddr, kTmemCols);
    pdl_wait();
    pdl_launch_dependents();
    int* marks = reinterpret_cast<int*>(smem + S::kMark);
    const int per = (p.num_seqs + kMarks - 1) / kMarks, used = (p.num_seqs + per - 1) / per;
    const auto starts_of = [&](int s, int2& q, int2& k) {
        q = make_int2(p.query_starts[s], p.query_starts[s + 1]);
        k = make_int2(p.key_starts[s], p.key_starts[s + 1]);
    };
    // A strip of the prompt whose queries and keys begin and end at q and k, and a head: the item (rows == 0: there is none).
    // zeroes: this warp sees to the rows of a prompt with bad metadata.
    const auto item_of = [&](int2 q, int2 k, int strip, int head, bool zeroes) -> Item {
        const int strips = strips_of(q.x, q.y, p.num_queries, p.max_query_len), q0 = (strips - 1 - strip) * kRows, n = q.y - q.x;
        if (strip < 0 || q0 < 0) return {0, 0, 0, 0, 0, 0};
        if (bad_prompt(p, q.x, q.y, k.x, k.y)) {
            if (zeroes) zero_prompt(p, q.x, q.y, q0, strips, head);
            return {0, 0, 0, 0, 0, 0};
        }
        return {q.x + q0, min(kRows, n - q0), head, q0 + 1 + (k.y - k.x) - n, k.x, k.y - k.x};
    };
    // The CTA's own place: what find_strip finds, with a load and a few exchanges less where there are few prompts.
    int2 q, k;
    int strip = blockIdx.x;
    if (p.num_seqs == 1) {
        starts_of(0, q, k);
    } else if (p.num_seqs <= 32) {
        starts_of(min(lane, p.num_seqs - 1), q, k);
        const int mine = lane < p.num_seqs ? strips_of(q.x, q.y, p.num_queries, p.max_query_len) : 0;
        int scan = mine;  // inclusive over the warp
        for (int o = 1; o < p.num_seqs; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
        }
        const unsigned in = __ballot_sync(0xffffffffu, strip < scan);
        const int at = in ? __ffs(in) - 1 : 0;
        strip = in ? strip - __shfl_sync(0xffffffffu, scan - mine, at) : -1;
        q = make_int2(__shfl_sync(0xffffffffu, q.x, at), __shfl_sync(0xffffffffu, q.y, at));
        k = make_int2(__shfl_sync(0xffffffffu, k.x, at), __shfl_sync(0xffffffffu, k.y, at));
    } else {
        mark_strips(p, per, used, marks, reinterpret_cast<int*>(smem + S::kSum));
        __syncthreads();
        const int2 at = find_strip(p, per, used, marks, strip);
        starts_of(max(at.x, 0), q, k);
        strip = at.x < 0 ? -1 : at.y;
    }
    Item it = item_of(q, k, strip, blockIdx.y, warp == kCopyWarp);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + S::kAddr);
    bool ok = true;  // no wait has run out
    // The next item, the CTA's own first (a whole warp).
    uint32_t taken = 0;
    bool own = __all_sync(0xffffffffu, it.rows > 0);
    const auto take = [&]() -> bool {
        if (own) {
            own = false;
            return true;
        }
        if (!p.claims) return false;
        ok = __all_sync(0xffffffffu, ok && wait_item(ifull, taken & 1));
        if (!ok) return false;
        ++taken;
        const int4 a = *reinterpret_cast<const int4*>(smem + S::kItem);
        const int2 b = *reinterpret_cast<const int2*>(smem + S::kItem + 16);
        it = {a.x, a.y, a.z, a.w, b.x, b.y};
        __syncwarp();
        if (lane == 0) mbar_arrive(iempty);
        return __all_sync(0xffffffffu, it.rows > 0);  // (a vote: known to be the same in all lanes)
    };

    if (warp == kCopyWarp) {
        // -------------------------------------------------------------- copies
        uint32_t nq[2] = {0, 0}, nk = 0, nv = 0;  // of each stream's Q, of tiles: those copied (by lane 0)
        uint32_t claims = 0, posted = 0;
        // The next item: the place of a CTA that has not begun, claimed when the copies of the item before have been
        // issued, two tiles before its end.
        const auto claimed = [&]() -> bool {
            if (own) {
                own = false;
                return true;
            }
            if (!p.claims) return false;
            it = {0, 0, 0, 0, 0, 0};
            for (bool more = true; more && it.rows == 0;) {
                dim3 at;
                if (lane == 0 && ok) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    mbar_arrive_expect_tx(claim, 16);
                    claim_cta(sbase + S::kClaim, claim);
                    ok = wait_bar(claim, claims++ & 1);
                    more = ok && claimed_cta(sbase + S::kClaim, at);
                } else if (lane == 0) {
                    more = false;
                }
                more = __shfl_sync(0xffffffffu, more, 0);
                if (more) {
                    const int2 found = find_strip(p, per, used, marks, __shfl_sync(0xffffffffu, (int)at.x, 0));
                    starts_of(max(found.x, 0), q, k);
                    it = item_of(q, k, found.x < 0 ? -1 : found.y, __shfl_sync(0xffffffffu, (int)at.y, 0), true);
                }
            }
            if (lane == 0) {
                // until the softmax, which may be at the item before, has taken it
                if (posted > 0) ok = ok && wait_bar(iempty, (posted - 1) & 1);
                if (!ok) it.rows = 0;  // (the others need not wait for more)
                *reinterpret_cast<int4*>(smem + S::kItem) = make_int4(it.row, it.rows, it.head, it.seen0);
                *reinterpret_cast<int2*>(smem + S::kItem + 16) = make_int2(it.key, it.keys);
                mbar_arrive(ifull);
            }
            ++posted;
            return __shfl_sync(0xffffffffu, it.rows, 0) > 0;
        };
        while (claimed()) {
            if (lane == 0) {
                const auto queries = [&](int x) {
                    if (nq[x] > 0) ok = ok && wait_bar(qempty0 + 8 * x, (nq[x] - 1) & 1);
                    if (!ok) return;
                    ++nq[x];
                    mbar_arrive_expect_tx(qfull0 + 8 * x, kKeyUnits * kUnit);
                    for (int i = 0; i < kKeyUnits; ++i)
                        tma_load_3d(sbase + S::kQ + (x * kKeyUnits + i) * kUnit, &tmq, qfull0 + 8 * x, 64 * i, it.head,
                                    it.row + 128 * x);
                };
                const int tiles_a = it.tiles(0), tiles_b = it.tiles(1), tiles = max(tiles_a, tiles_b);
                if (tiles_a > 0) queries(0);
                for (int t = 0; t < tiles; ++t) {
                    const uint32_t par = nk & 1;
                    const int y = it.key + t * kTile;
                    if (nk >= 2) ok = ok && wait_bar(vread0 + 8 * par, (nk / 2 - 1) & 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(kfull0 + 8 * par, kKeyUnits * kUnit);
                    for (int i = 0; i < kKeyUnits; ++i) {
                        const uint32_t dst = sbase + S::kKV + (nk * kTileUnits + i) % kRing * kUnit;
                        if (i < 2)
                            tma_load_3d(dst, &tmkv, kfull0 + 8 * par, 64 * i, it.head, y);
                        else
                            tma_load_2d(dst, &tmr, kfull0 + 8 * par, 0, y);
                    }
                    ++nk;
                    if (t == 0 && tiles_b > 0) queries(1);
                    if (nv >= 1) ok = ok && wait_bar(kread0 + 8 * (par ^ 1), ((nv - 1) / 2) & 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(vfull0 + 8 * par, 2 * kUnit);
                    for (int i = 0; i < 2; ++i)
                        tma_load_3d(sbase + S::kKV + (nv * kTileUnits + kKeyUnits + i) % kRing * kUnit, &tmkv, vfull0 + 8 * par,
                                    128 + 64 * i, it.head, y);
                    ++nv;
                }
            }
            __syncwarp();
        }
        if (lane == 0) {
            if (!ok) record_error(p.err, PKV_DEVERR_TIMEOUT);
            // every copy has landed before the CTA ends
            for (int x = 0; x < 2; ++x)
                if (nq[x] > 0) wait_bar(qfull0 + 8 * x, (nq[x] - 1) & 1);
            for (uint32_t i = max(nk, 2u) - 2; i < nk; ++i) wait_bar(kfull0 + 8 * (i & 1), (i / 2) & 1);
            for (uint32_t i = max(nv, 2u) - 2; i < nv; ++i) wait_bar(vfull0 + 8 * (i & 1), (i / 2) & 1);
        }
    } else if (warp == kProductWarp) {
        // ------------------------------------------------------------ products
        // (first what mark_strips does for more prompts, away from the copies' way)
        if (lane < p.num_seqs && p.num_seqs <= 32 &&
            bad_prompt(p, p.query_starts[lane], p.query_starts[lane + 1], p.key_starts[lane], p.key_starts[lane + 1]))
            record_error(p.err, PKV_DEVERR_QUERY);
        __syncwarp();
        const uint32_t el = issuing_lane(), tm = __shfl_sync(0xffffffffu, tmem, 0), sb = __shfl_sync(0xffffffffu, sbase, 0);
        const uint32_t id_s = umma_idesc(kBF16, 128, kTile, false, false);
        const uint32_t id_o = umma_idesc(kBF16, 128, 128, false, true), id_h = umma_idesc(kBF16, 128, 64, false, true);
        const uint64_t q_desc = umma_desc_sw128(sb + S::kQ, 16, 1024), k_desc = umma_desc_sw128(sb + S::kKV, 16, 1024),
                       v_desc = umma_desc_sw128(sb + S::kKV, kUnit, 1024);  // + (bytes / 16)
        uint32_t last_bar = 0, last_par = 0;
        uint32_t tile0 = 0, par0 = 0, items = 0;  // tiles of the items before; bits of the streams: those of each, their items
        while (take()) {
            const int ta = __shfl_sync(0xffffffffu, it.tiles(0), 0), tb = __shfl_sync(0xffffffffu, it.tiles(1), 0),
                      tn = max(ta, tb);
            int pend_x = -1, pend_t = 0;  // a tile whose second product is still to come
            const auto values = [&]() {
                const uint32_t x = pend_x, t = pend_t, g = tile0 + t, at = (g * kTileUnits + kKeyUnits) % kRing;
                pend_x = -1;
                ok = mbar_wait_warp(vfull0 + 8 * (g & 1), (g / 2) & 1) && mbar_wait_warp(pfull0 + 8 * x, (par0 >> x ^ t) & 1);
                if (!ok) return;
                tc_fence_after();
                const uint32_t o = tm + 256 + 128 * x, pp = tm + 128 * x;
                if (at + 1 < kRing) {
                    const uint64_t vd = v_desc + at * (kUnit / 16);
#pragma unroll
                    for (int ks = 0; ks < kTile / 16; ++ks) umma_f16_ts(el, o, pp + 8 * ks, vd + ks * 128, id_o, t > 0 || ks > 0);
                } else {  // the two halves of the values do not stand together in the ring
                    const uint64_t v0 = k_desc + at * (kUnit / 16), v1 = k_desc;
#pragma unroll 1
                    for (int ks = 0; ks < kTile / 16; ++ks) {
                        umma_f16_ts(el, o, pp + 8 * ks, v0 + ks * 128, id_h, t > 0 || ks > 0);
                        umma_f16_ts(el, o + 64, pp + 8 * ks, v1 + ks * 128, id_h, t > 0 || ks > 0);
                    }
                }
                if (x == 1 || t >= (uint32_t)tb) umma_commit(el, vread0 + 8 * (g & 1));  // the last to read it
                if (t + 1 == (uint32_t)(x ? tb : ta)) {
                    umma_commit(el, odone0 + 8 * x);
                    last_bar = odone0 + 8 * x;
                    last_par = items >> x & 1;
                }
            };
            for (int t = 0; t < tn && ok; ++t) {
                const uint32_t g = tile0 + t;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (t >= (x ? tb : ta) || !ok) continue;
                    if (pend_x == x) values();  // P of this stream lies where S goes
                    if (ok && t == 0) ok = mbar_wait_warp(qfull0 + 8 * x, items >> x & 1);
                    ok = ok && mbar_wait_warp(kfull0 + 8 * (g & 1), (g / 2) & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < kKeyUnits; ++i) {
                        const uint64_t qd = q_desc + (x * kKeyUnits + i) * (kUnit / 16),
                                       kd = k_desc + (g * kTileUnits + i) % kRing * (kUnit / 16);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            umma_f16_ss(el, tm + 128 * x, qd + 2 * ks, kd + 2 * ks, id_s, i > 0 || ks > 0);
                    }
                    if (x == 1 || t >= tb) umma_commit(el, kread0 + 8 * (g & 1));  // the last to read it
                    umma_commit(el, sfull0 + 8 * x);
                    last_bar = sfull0 + 8 * x;
                    last_par = (par0 >> x ^ t) & 1;
                    if (pend_x >= 0) values();
                    pend_x = x;
                    pend_t = t;
                }
            }
            if (!ok) break;
            // every Q K has been issued: the queries may be replaced when they have ended
            if (ta > 0) umma_commit(el, qempty0);
            if (tb > 0) umma_commit(el, qempty0 + 8);
            if (pend_x >= 0) values();
            if (!ok) break;
            tile0 += tn;
            par0 ^= (ta & 1) | (tb & 1) << 1;
            items ^= (ta > 0) | (tb > 0) << 1;
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
        // every product that was issued has ended before tensor memory is given back
        if (last_bar) wait_bar(last_bar, last_par);
    } else {
        // ------------------------------------------------------------- softmax
        const int X = warp >> 2, r = tid & 127, row = 128 * X + r;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t s_addr = lane_addr + 128 * X, o_addr = lane_addr + 256 + 128 * X;
        uint32_t items = 0, tile0 = 0, ns = 0, no = 0;  // items, and their tiles; of this stream: tiles, items
        while (take()) {
            const int tiles_a = it.tiles(0), tiles_b = it.tiles(1), mine = X ? tiles_b : tiles_a;
            const int masked = max(0, it.seen0) / kTile;  // tiles before it hold no key that any row masks
            const int mine_masked = max(0, it.seen0 + 128 * X) / kTile;  // ... that any row of the stream masks
            const int seen = min(it.keys, it.seen0 + row);  // keys that this row attends (rows past the prompt's end: whatever)
            const bool live = 128 * X + 32 * (warp & 3) < it.rows;
            uint32_t* mine_lost = lost + items % 3 * (kLostTiles * 4);
            // (a lane without a row, whose scores are anything, never asks for a raise)
            float m_run = row < it.rows ? -INFINITY : INFINITY, l = 0.f;
            for (int t = 0; t < mine; ++t) {
                const bool shared = t < tiles_a && t < tiles_b;
                const bool guard = t >= masked;
                ok = ok && wait_bar(sfull0 + 8 * X, ns & 1);
                ok = __all_sync(0xffffffffu, ok);
                ++ns;
                if (live && ok) {
                    tc_fence_after();
                    softmax_tile<kBF16>(s_addr, o_addr, t >= mine_masked, p.scale_log2, t > 0, m_run, l,
                                        [&](int c) { return before(t * kTile + c, seen); });
                    tc_fence_before();
                }
                if (guard) {
                    const uint32_t tile = tile0 + t, u = tile * kTileUnits + kKeyUnits;
                    ok = ok && wait_bar(vfull0 + 8 * (tile & 1), (tile / 2) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok) {
                        // this thread's key: its values past the prompt become zeros, and those not finite are taken out;
                        // where both streams use the tile each sees to half of it
                        const int key = shared ? 64 * X + (r >> 1) : r, pos = t * kTile + key;
                        const int h0 = shared ? r & 1 : 0;
                        const auto at = [&](int i) {  // (neighbouring threads start at different eighths of 128 bytes)
                            return reinterpret_cast<uint4*>(smem + S::kKV + ((u + h0 + (i >> 3)) % kRing) * kUnit + key * 128) +
                                   ((i + key) & 7);
                        };
                        if (scrub<kBF16>(shared ? 8 : 16, pos < it.keys, at))
                            atomicOr(mine_lost + (pos - masked * kTile) / 32, 1u << (pos & 31));
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    if (shared) both_streams();
                }
                if (!ok) continue;
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull0 + 8 * X);
            }
            // (read last before the barrier of the item before)
            if (tid < kLostTiles * 4) lost[(items + 1) % 3 * (kLostTiles * 4) + tid] = 0;
            both_streams();  // (what was taken out is known)
            if (mine > 0) ok = __all_sync(0xffffffffu, ok && wait_bar(odone0 + 8 * X, no & 1));
            no += mine > 0;
            tc_fence_after();
            const float inv = ok && l != 0.f ? 1.f / l : 0.f;
            uint16_t* dst = out + ((int64_t)(it.row + row) * p.num_heads + it.head) * 128;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0.f;
                if (live && ok && mine > 0) {
                    tmem_ld32_start(o_addr + 32 * c, o);
                    tmem_ld_wait32(o);
                }
                if (row >= it.rows) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = inv != 0.f ? pack2<kBF16>(o[8 * i + 2 * e] * inv, o[8 * i + 2 * e + 1] * inv) : 0u;
                    *reinterpret_cast<uint4*>(dst + 32 * c + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            tc_fence_before();
            if (row < it.rows && ok) {
                // values that are not finite and were left out of the products
#pragma unroll 1
                for (int w = 0; w < kLostTiles * 4; ++w)
                    for (uint32_t at = mine_lost[w]; at; at &= at - 1) {
                        const int pos = masked * kTile + 32 * w + __ffs(at) - 1;
                        if (pos < seen)
                            add_not_finite<kBF16>(nullptr, dst,
                                                  static_cast<const uint16_t*>(p.values) + (it.key + pos) * p.kv_stride +
                                                      it.head * p.kv_head_stride + 128,
                                                  128);
                    }
            }
            ++items;
            tile0 += max(tiles_a, tiles_b);
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kProductWarp) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_latent_prompt(const LatentPromptParams& in, int dtype, const CUtensorMap& tmq, const CUtensorMap& tmkv,
                                 const CUtensorMap& tmr, cudaStream_t stream, int* launches) {
    auto kern = dtype == PKV_BF16 ? latent_prompt_kernel<true> : latent_prompt_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptSmem::kTotal);
    if (e != cudaSuccess) return e;
    // No more strips than these, whatever the prompts' lengths: n tokens make at most (n + kRows - 1) / kRows, and a strip has a
    // token.
    const int64_t strips = std::min({in.num_seqs * (((int64_t)in.max_query_len + kRows - 1) / kRows),
                                     (in.num_queries + (int64_t)in.num_seqs * (kRows - 1)) / kRows, (int64_t)in.num_queries});
    const dim3 grid((unsigned)strips, in.num_heads);
    LatentPromptParams p = in;
    p.claims = strips * grid.y > p.sms;  // (more than one CTA an SM)
    e = launch_pdl(kern, grid, dim3(kThreads), PromptSmem::kTotal, stream, tmq, tmkv, tmr, p);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace pkv
