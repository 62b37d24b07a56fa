// drafted.cuh -- batches whose sequences have several query tokens each, the
// drafted tokens at the end of their contexts (tree.cu, latent.cu): what a
// sequence attends, how the work is dealt to a fixed grid, and where the
// halves of a divided unit meet.
//
// A unit of work is a sequence, a KV head and a group of its query rows; it
// is walked in tiles of keys.  All tiles of all units, one unit after the
// other, form one line that is cut into equal pieces, one for each CTA of a
// grid of one CTA per SM, so that long and short contexts load the SMs
// alike.  A CTA holds at most two units in part: the one that its piece begins
// inside (slot 0 of its partials) and the one that its piece ends inside
// (slot 1).  Their unnormalised sums go to the workspace with each row's
// running maximum and sum, and a merge kernel, which starts when this one has
// ended, joins the pieces.  So no CTA waits on another, nothing in the
// workspace is read that the same call has not written, and the result is the
// same from run to run.
#pragma once

#include "pkv_internal.cuh"

namespace pkv {

constexpr int kMaxDrafted = 64;  // query tokens of one sequence: a tree's mask has 64 bits

struct DraftParams {
    const void* q;                // [num_tokens][num_q_heads][q row]
    const int32_t* block_tables;  // [num_seqs][max_blocks_per_seq]
    const int32_t* context_lens;  // [num_seqs]
    const int32_t* query_starts;  // [num_seqs + 1]; nullptr: one token a sequence
    const int64_t* tree_masks;    // [num_tokens]; nullptr: chains
    void* out;                    // [num_tokens][num_q_heads][value dims], q's type
    const void* values;           // the pool that values are read from (rows that are not finite)
    float* part_o;                // [pieces][2][rows of a unit][value dims]
    float2* part_ml;              // [pieces][2][rows of a unit]: running maximum (log2 domain) and sum
    int4* part_desc;              // [pieces][2][2]: state, first token, first row, rows; KV head
    int* err;
    int64_t num_blocks;
    int num_seqs, num_tokens, num_q_heads, num_kv_heads;
    int group;                    // query heads of a KV head
    int max_blocks_per_seq;
    int len_limit;                // max_blocks_per_seq * block_size
    int pieces;                   // of the line: CTAs of the grid
    bool merged;                  // a merge follows (draft_divides)
    float scale_log2;             // scale * log2(e)
};

// State of a partial: it exists, it holds its unit's last tile.  (Its unit's first tile is in slot 1.)
enum { kPartValid = 1, kPartEnds = 2 };

// What sequence s asks for: n query tokens, rows tok0 .. of q, the last n of
// its L positions.  n == 0: no rows.  idle: its rows are zeros (an empty
// context, or, with err, bad metadata).
struct DraftSeq {
    int tok0, n, L, err;
    bool idle;
};

__device__ __forceinline__ DraftSeq draft_seq(const DraftParams& p, int s) {
    DraftSeq r;
    int tok1;
    if (p.query_starts) {
        r.tok0 = p.query_starts[s];
        tok1 = p.query_starts[s + 1];
    } else {
        r.tok0 = s;
        tok1 = s + 1;
    }
    r.err = 0;
    r.idle = false;
    r.L = 0;
    const int L = p.context_lens[s];  // (on its way beside the others)
    if (r.tok0 < 0 || tok1 < r.tok0 || tok1 > p.num_tokens) {  // no rows that could be written
        r.n = 0;
        r.err = PKV_DEVERR_QUERY;
        return r;
    }
    r.n = tok1 - r.tok0;
    if (r.n == 0) return r;
    r.L = L;
    if (r.n > kMaxDrafted)
        r.err = PKV_DEVERR_QUERY;
    else if (r.L < 0 || r.L > p.len_limit || (r.L > 0 && r.L < r.n))
        r.err = PKV_DEVERR_CONTEXT_LEN;
    r.idle = r.err != 0 || r.L == 0;
    return r;
}

// The shape of a kernel's units.
template <int kRows, int kTile>
struct UnitShape {
    static __device__ __forceinline__ int row_groups(const DraftParams& p, const DraftSeq& q) {
        return (q.n * p.group + kRows - 1) / kRows;
    }
    static __device__ __forceinline__ int tiles(const DraftSeq& q) { return (q.L + kTile - 1) / kTile; }
    static __device__ __forceinline__ int units(const DraftParams& p, const DraftSeq& q) {
        return q.n == 0 || q.idle ? 0 : row_groups(p, q) * p.num_kv_heads;
    }
};

// Part of a unit: tiles t0 .. t1-1 of `tiles`.  Rows row0 .. row0+rows-1 of
// the sequence's n * group (row r: token r / group, head r % group).
struct DraftItem {
    DraftSeq q;
    int s, kvh, row0, rows, t0, t1, tiles;
    __device__ __forceinline__ bool begins() const { return t0 == 0; }
    __device__ __forceinline__ bool ends() const { return t1 == tiles; }
    __device__ __forceinline__ bool partial() const { return !begins() || !ends(); }
};

// Walks a CTA's piece of the line, item by item.
template <int kRows, int kTile>
struct DraftCursor {
    using U = UnitShape<kRows, kTile>;
    int s, u, t;
    int64_t left;
    DraftSeq q;
    int units;

    // From tile t0 of unit u0 of sequence s0 on.
    __device__ __forceinline__ void start(const DraftParams& p, int s0, const DraftSeq& q0, int u0, int t0, int64_t count) {
        s = s0;
        q = q0;
        units = U::units(p, q);
        u = u0;
        t = t0;
        left = count;
    }
    __device__ __forceinline__ bool next(const DraftParams& p, DraftItem& it) {
        if (left <= 0) return false;
        while (u >= units) {  // (a sequence follows while tiles are left)
            ++s;
            q = draft_seq(p, s);
            units = U::units(p, q);
            u = 0;
        }
        it.q = q;
        it.s = s;
        it.tiles = U::tiles(q);
        const int groups = U::row_groups(p, q), all = q.n * p.group, per = (all + groups - 1) / groups;
        const int rg = u / p.num_kv_heads;
        it.kvh = u - rg * p.num_kv_heads;
        it.row0 = rg * per;
        it.rows = min(per, all - it.row0);
        it.t0 = t;
        it.t1 = (int)min((int64_t)it.tiles, t + left);
        left -= it.t1 - it.t0;
        t = 0;
        ++u;
        return true;
    }
};

// Zeroes the rows of a sequence that has nothing to attend (whole warp).
__device__ __forceinline__ void zero_rows(const DraftParams& p, int tok0, int n, int value_dims, int lane) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (int64_t)tok0 * p.num_q_heads * value_dims);
    const int64_t vecs = (int64_t)n * p.num_q_heads * value_dims / 8;
    for (int64_t i = lane; i < vecs; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
}

// Deals the line and starts `cur` on piece piece_id of it; every thread of the
// CTA calls it and gets the same piece.  A piece is the line's length over the
// CTAs, and kLeast tiles at least (or the longest unit, where that is shorter): a
// smaller one costs more in starting and merging than it spreads.  Where no unit is longer than that and each can have a CTA of its
// own, it has, and nothing is divided; nor where no merge follows, and only
// sequences that lie over one another (bad metadata) can make more units than
// CTAs: then a CTA has several, whole.  Each CTA reads all lengths, a run of
// sequences to a thread: 2 us for 1000 sequences, 20 (tree.cu) to 30 (latent.cu)
// for 10000 and 155 to 255 for 65535, at most a tenth of a call whose contexts
// are the shortest.  On the way the sequences that attend nothing get their
// zeros, and bad metadata is recorded, each by one CTA.
// scratch: (kThreads / 32) * 16 + 48 bytes of shared memory, 8-byte aligned.
template <int kThreads>
__host__ __device__ constexpr int draft_scratch() {
    return kThreads / 32 * 16 + 48;
}
template <int kRows, int kTile, int kThreads, int kLeast>
__device__ __forceinline__ void draft_schedule(const DraftParams& p, int piece_id, int value_dims, void* scratch,
                                               DraftCursor<kRows, kTile>& cur) {
    using U = UnitShape<kRows, kTile>;
    constexpr int kWarps = kThreads / 32;
    long long* warp_tiles = static_cast<long long*>(scratch);  // [kWarps]
    long long* warp_units = warp_tiles + kWarps;               // [kWarps]
    long long* count = warp_units + kWarps;
    int* longest = reinterpret_cast<int*>(count + 1);
    int* found = longest + 1;  // [6]: sequence, its first token, tokens, length; unit, tile
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) *longest = 0, *count = 0;
    __syncthreads();
    const int per = (p.num_seqs + kThreads - 1) / kThreads;
    const int first = tid * per;
    long long tiles = 0, units = 0;
    int most = 0;
    for (int k = 0; k < per; ++k) {
        const int s = first + k;
        DraftSeq q;
        q.n = 0, q.idle = false, q.err = 0, q.tok0 = 0, q.L = 0;
        if (s < p.num_seqs) {
            q = draft_seq(p, s);
            const int n = U::units(p, q);
            if (n > 0) {
                units += n;
                tiles += (long long)n * U::tiles(q);
                most = max(most, U::tiles(q));
            }
            if (q.err && s % p.pieces == piece_id) record_error(p.err, q.err);
        }
        unsigned idle = __ballot_sync(0xffffffffu, q.idle && s % p.pieces == piece_id);
        while (idle) {
            const int src = __ffs(idle) - 1;
            idle &= idle - 1;
            zero_rows(p, __shfl_sync(0xffffffffu, q.tok0, src), __shfl_sync(0xffffffffu, q.n, src), value_dims, lane);
        }
    }
    if (most > 0) atomicMax(longest, most);
    long long scan = tiles, scan_units = units;  // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, scan, o), w = __shfl_up_sync(0xffffffffu, scan_units, o);
        if (lane >= o) scan += v, scan_units += w;
    }
    if (lane == 31) warp_tiles[warp] = scan, warp_units[warp] = scan_units;
    __syncthreads();
    long long total = 0, before = 0, total_units = 0, before_units = 0;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_tiles[w], before_units += warp_units[w];
        total += warp_tiles[w];
        total_units += warp_units[w];
    }
    const bool whole = *longest <= kLeast && (total_units <= p.pieces || !p.merged);
    long long w0, w1;
    if (whole) {
        before = before_units + scan_units - units, tiles = units;
        const long long each = total_units <= p.pieces ? 1 : (total_units + p.pieces - 1) / p.pieces;
        w0 = min(total_units, each * piece_id), w1 = min(total_units, w0 + each);
    } else {
        const long long piece = max((total + p.pieces - 1) / p.pieces, (long long)min(kLeast, *longest));
        before += scan - tiles;
        w0 = min(total, piece * piece_id), w1 = min(total, w0 + piece);
    }
    if (w0 < w1 && before <= w0 && w0 < before + tiles) {  // this thread's sequences hold the piece's start
        long long at = before;
        for (int k = 0; k < per; ++k) {
            const int s = first + k;
            if (s >= p.num_seqs) break;
            DraftSeq q = draft_seq(p, s);
            const int n = U::units(p, q), len = n > 0 && !whole ? U::tiles(q) : 1;
            if (w0 < at + (long long)n * len) {
                const long long in = w0 - at;
                int u = (int)(in / len);
                found[0] = s, found[1] = q.tok0, found[2] = q.n, found[3] = q.L;
                found[4] = u, found[5] = (int)(in - (long long)u * len);
                *count = !whole ? w1 - w0 : U::tiles(q);
                if (whole && w1 - w0 > 1) {  // the tiles of so many units
                    long long more = w1 - w0, sum = 0;
                    for (int k = s;;) {
                        const long long take = min(more, (long long)(U::units(p, q) - u));
                        sum += take * U::tiles(q);
                        more -= take;
                        if (more == 0) break;
                        q = draft_seq(p, ++k);
                        u = 0;
                    }
                    *count = sum;
                }
                break;
            }
            at += (long long)n * len;
        }
    }
    __syncthreads();
    DraftSeq q;
    q.tok0 = found[1], q.n = found[2], q.L = found[3], q.err = 0, q.idle = false;
    cur.start(p, found[0], q, found[4], found[5], w0 < w1 ? *count : 0);
}

// Can a unit of this call be divided, so that a merge has to follow?  Not where all are short and each surely has a CTA of its
// own (see draft_schedule).
inline bool draft_divides(const DraftParams& p, int tile, int unit_rows, int least) {
    if (p.len_limit <= tile) return false;
    const int64_t units = p.num_kv_heads * (p.num_seqs + (int64_t)p.num_tokens * p.group / unit_rows);
    return p.len_limit > (int64_t)least * tile || units > p.pieces;
}
// The merge of divided units (drafted.cu): value_dims 128 (tree.cu) or 512 (latent.cu).
cudaError_t launch_draft_merge(const DraftParams& p, int dtype, int value_dims, int unit_rows, cudaStream_t stream,
                               int* launches);
// tree.cu
cudaError_t launch_tree(const DraftParams& p, int dtype, int block_size, const CUtensorMap& tmk, const CUtensorMap& tmv,
                        cudaStream_t stream, int* launches);
constexpr int kTreeRows = 256;   // query rows of a unit
// latent.cu
cudaError_t launch_latent_decode(const DraftParams& p, int dtype, int block_size, const CUtensorMap& tmq, const CUtensorMap& tmc,
                                 cudaStream_t stream, int* launches);
constexpr int kLatentRows = 64;  // query rows of a unit

// The position bits that a query row attends among its sequence's drafted tokens.
__device__ __forceinline__ uint64_t draft_mask(const DraftParams& p, const DraftSeq& q, int token) {
    const uint64_t whole = q.n >= 64 ? ~0ull : (1ull << q.n) - 1;
    const uint64_t m = p.tree_masks ? (uint64_t)p.tree_masks[q.tok0 + token]
                                    : (token >= 63 ? ~0ull : (2ull << token) - 1);
    return m & whole;
}

// 32 positions from pos on as bits: those before `base`, and behind it those of the mask.
__device__ __forceinline__ uint32_t draft_visible(int pos, int base, uint64_t mask) {
    const int ahead = base - pos;  // positions of the context proper
    if (ahead >= 32) return ~0u;
    if (ahead > 0) return ((1u << ahead) - 1) | (uint32_t)(mask << ahead);
    return ahead > -64 ? (uint32_t)(mask >> -ahead) : 0u;
}

}  // namespace pkv
