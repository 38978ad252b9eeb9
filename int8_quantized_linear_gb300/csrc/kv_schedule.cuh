// How the attention kernels share out their work.
//
// An item is a block of up to ROWS query rows of one cache head of one
// sequence (row r of a sequence: query token r / G, query head r % G of the
// head's group of G); it has as many tiles as its rows see TILE-token tiles
// of the cache, at least one, so that rows that see nothing are still
// written.  Items are ordered by sequence, row block and head; each counts as
// its tiles plus COST more in front of them (what a CTA spends on beginning
// and ending an item), and all items, end to end, are cut into one equal range
// per CTA: the work is even whatever the lengths, without the host knowing
// them.  An item cut
// between CTAs is finished from its parts (unnormalised sums, maximum and
// total of the softmax) by a second kernel, in the order of the CTAs, so the
// result does not depend on timing.  Every CTA derives its range from the
// lengths itself: one pass of block-wide sums over the sequences.
#pragma once

#include "kv_common.cuh"

namespace i8ql {

// Tiles of the kernel for many query rows (kv_prompt.cu).
constexpr int kKvPromptTile = 128;
constexpr int kKvPromptRows = 256;

struct KvAttnParams {
    KvCache cache;
    const uint16_t* q;
    int64_t q_stride;  // elements between query tokens
    const int32_t* table;
    int64_t table_width;  // pages per sequence in the table
    const int32_t* kv_lens;
    const int32_t* q_offsets;  // null: one query token per sequence
    uint16_t* out;
    int64_t B;
    int64_t T_q;
    int G;
    int64_t window;      // 0: none
    float scale_log2;    // softmax scale * log2 e
    float* part_o;       // [CTAs][2][ROWS][D]: slot 0 a part that continues an item, slot 1 one that begins it
    float* part_ml;      // [CTAs][2][ROWS][2]
    struct KvSplitItem* split;  // [CTAs]; null when no item can be cut
    unsigned* err;
};

// The item that begins in a CTA's range and ends in a later one's.
struct KvSplitItem {
    int64_t q_row;  // first query token of the sequence
    int32_t row0;   // first row of the block
    int32_t rows;   // 0: nothing to join
    int32_t h;
    int32_t last_cta;
    int64_t pad;
};

// The kernel for many query rows, without the join (D 64 or 128, bits 4 or 8).
cudaError_t launch_kv_prompt(const KvAttnParams& p, int64_t D, int64_t bits, int64_t ctas, const LaunchEnv& env);

namespace {

struct KvSeq {
    int64_t q0;   // first query token
    int32_t nq;   // query tokens
    int32_t len;  // cache tokens
};

// Reads a sequence's sizes, held to what the buffers have; what is out of
// their range is recorded.
__device__ __forceinline__ KvSeq kv_sequence(const KvAttnParams& p, int64_t b) {
    KvSeq s;
    const int64_t most = min(p.table_width << p.cache.page_shift, (int64_t)INT32_MAX - 65536);
    const int64_t len = p.kv_lens[b];
    int64_t q0 = b, q1 = b + 1;
    if (p.q_offsets) {
        q0 = p.q_offsets[b];
        q1 = p.q_offsets[b + 1];
    }
    if (len < 0 || len > most || q0 < 0 || q1 < q0 || q1 > p.T_q || (b == 0 && q0 != 0) ||
        (b == p.B - 1 && q1 != p.T_q))
        record_fault(p.err, kErrBitBadIndex);
    q0 = min(max(q0, (int64_t)0), p.T_q);
    q1 = min(max(q1, q0), p.T_q);
    s.q0 = q0;
    s.nq = (int32_t)(q1 - q0);
    s.len = (int32_t)min(max(len, (int64_t)0), most);
    return s;
}

// Row blocks of a sequence.  nq * G stays below 2^31 (checked on the host).
template <int ROWS>
__device__ __forceinline__ int kv_blocks(const KvAttnParams& p, const KvSeq& s) {
    return (int)(((int64_t)s.nq * p.G + ROWS - 1) / ROWS);
}

struct KvSpan {
    int first;  // first tile that any row of the block sees
    int tiles;  // >= 1
    int begin;  // tokens before this one are seen by no row,
    int end;    // and neither are those from here on (begin = end: none is seen)
};

// The tiles of row block rb.
template <int ROWS, int TILE>
__device__ __forceinline__ KvSpan kv_span(const KvAttnParams& p, const KvSeq& s, int rb) {
    const int row0 = rb * ROWS;
    const int row1 = min(row0 + ROWS, s.nq * p.G) - 1;
    const int base = s.len - s.nq;
    KvSpan t;
    t.end = max(base + row1 / p.G + 1, 0);
    const int64_t begin = p.window > 0 ? max((int64_t)(base + row0 / p.G) + 1 - p.window, (int64_t)0) : 0;
    t.begin = (int)min(begin, (int64_t)t.end);
    t.first = t.begin / TILE;
    t.tiles = max((t.end + TILE - 1) / TILE - t.first, 1);
    return t;
}

// A place in the order of the tiles.
struct KvCursor {
    int64_t b;
    KvSeq seq;
    int blocks;
    int rb;
    int h;
    KvSpan span;
    int tile;    // within the item
    int64_t at;  // where the item begins, in the order of all items
};

// Tiles of the cursor's item, from its tile on, that lie before `end`; 0: the
// range is done.
template <int COST>
__device__ __forceinline__ int kv_take(const KvAttnParams& p, const KvCursor& c, int64_t end) {
    if (c.b >= p.B) return 0;
    return (int)max(min((int64_t)c.span.tiles, end - c.at - COST) - c.tile, (int64_t)0);
}

template <int ROWS, int TILE, int COST>
__device__ __forceinline__ void kv_next_item(const KvAttnParams& p, KvCursor& c) {
    c.tile = 0;
    c.at += c.span.tiles + COST;
    if (++c.h < p.cache.H) return;
    c.h = 0;
    if (++c.rb >= c.blocks) {
        c.rb = 0;
        do {
            if (++c.b >= p.B) return;
            c.seq = kv_sequence(p, c.b);
            c.blocks = kv_blocks<ROWS>(p, c.seq);
        } while (c.blocks == 0);
    }
    c.span = kv_span<ROWS, TILE>(p, c.seq, c.rb);
}

// Tiles and costs of one head over all row blocks of the sequence that each
// lane holds: a lane alone when its sequence has few blocks, the warp together
// for sequences of many.
template <int ROWS, int TILE, int COST>
__device__ __forceinline__ int64_t kv_seq_tiles(const KvAttnParams& p, const KvSeq& s, int blocks) {
    constexpr int kAlone = 4;
    const int lane = threadIdx.x & 31;
    int64_t tiles = 0;
    if (blocks <= kAlone)
        for (int rb = 0; rb < blocks; ++rb) tiles += kv_span<ROWS, TILE>(p, s, rb).tiles + COST;
    unsigned many = __ballot_sync(0xffffffffu, blocks > kAlone);
    while (many) {
        const int src = __ffs(many) - 1;
        many &= many - 1;
        KvSeq o;
        o.q0 = 0;
        o.nq = __shfl_sync(0xffffffffu, s.nq, src);
        o.len = __shfl_sync(0xffffffffu, s.len, src);
        const int n = __shfl_sync(0xffffffffu, blocks, src);
        int64_t sum = 0;
        for (int rb = lane; rb < n; rb += 32) sum += kv_span<ROWS, TILE>(p, o, rb).tiles + COST;
#pragma unroll
        for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (lane == src) tiles = sum;
    }
    return tiles;
}

// Shared memory of kv_locate.
struct KvLocate {
    int64_t warp_sum[32];
    int64_t total;
    int64_t at;      // where sequence b begins
    int64_t b;
};

struct KvRange {
    int64_t total, begin, end;  // tiles and costs of all items; this CTA's range
    uint32_t ctas;              // CTAs that have a range (those behind have none)
};

// Where the ranges of n CTAs begin: CTA i's at each * i + more * i / n (i, n and
// more < n below 2^16: a 32-bit division).
struct KvCuts {
    int64_t each;
    uint32_t more, n;
    __device__ __forceinline__ KvCuts(int64_t total, uint32_t ctas) : n(ctas) {
        // (the 64-bit division alone takes as long as the rest of a short call's prologue)
        each = total < ((int64_t)1 << 32) ? (int64_t)((uint32_t)total / n) : total / n;
        more = (uint32_t)(total - each * n);
    }
    __device__ __forceinline__ int64_t at(uint32_t i) const { return each * i + more * i / n; }
};

// This CTA's range and the cursor at its beginning.  Called by all THREADS
// threads of the block (whole warps).
template <int ROWS, int TILE, int COST, int THREADS>
__device__ __forceinline__ KvRange kv_locate(const KvAttnParams& p, KvLocate& sm, KvCursor& c) {
    constexpr int kWarps = THREADS / 32;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int64_t carry = 0;
    KvRange r = {0, 0, 0, 1};
    // pass 0 sums all tiles; pass 1 finds the sequence that holds r.begin
    // (skipped sums: a batch that fits one pass keeps its counts)
    int64_t kept = 0;
    for (int pass = 0; pass < 2; ++pass) {
        carry = 0;
        for (int64_t base = 0; base < p.B; base += THREADS) {
            const int64_t b = base + threadIdx.x;
            int64_t tiles = kept;
            if (pass == 0 || p.B > THREADS) {
                KvSeq s = {0, 0, 0};
                int blocks = 0;
                if (b < p.B) {
                    s = kv_sequence(p, b);
                    blocks = kv_blocks<ROWS>(p, s);
                }
                tiles = kv_seq_tiles<ROWS, TILE, COST>(p, s, blocks) * p.cache.H;
                kept = tiles;
            }
            int64_t upto = tiles;  // inclusive sum over the warp
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, upto, m);
                if (lane >= m) upto += o;
            }
            __syncthreads();
            if (lane == 31) sm.warp_sum[warp] = upto;
            __syncthreads();
            int64_t before = carry, all = carry;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += sm.warp_sum[w];
                all += sm.warp_sum[w];
            }
            if (pass == 1 && r.begin >= before + upto - tiles && r.begin < before + upto) {
                sm.b = b;
                sm.at = before + upto - tiles;
            }
            carry = all;
        }
        if (pass == 0) {
            r.total = carry;
            r.ctas = (uint32_t)min((int64_t)gridDim.x, max(carry, (int64_t)1));
            const KvCuts cuts(carry, r.ctas);
            r.begin = cuts.at(min(blockIdx.x, r.ctas));
            r.end = cuts.at(min(blockIdx.x + 1, r.ctas));
        }
    }
    __syncthreads();
    c = {};
    c.b = p.B;
    if (r.begin >= r.end) return r;
    c.b = sm.b;
    c.seq = kv_sequence(p, c.b);
    c.blocks = kv_blocks<ROWS>(p, c.seq);
    // the row block: 32 at a time, every warp the same
    int64_t left = r.begin - sm.at;
    for (int rb0 = 0;; rb0 += 32) {
        const int rb = rb0 + lane;
        const int64_t tiles = rb < c.blocks ? (int64_t)(kv_span<ROWS, TILE>(p, c.seq, rb).tiles + COST) * p.cache.H : 0;
        int64_t upto = tiles;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, left < upto);
        if (hit) {
            const int at = __ffs(hit) - 1;
            c.rb = rb0 + at;
            left -= __shfl_sync(0xffffffffu, upto - tiles, at);
            break;
        }
        left -= __shfl_sync(0xffffffffu, upto, 31);
        if (rb0 + 32 >= c.blocks) {  // not reached: the sums above hold left below the sequence's tiles
            c.rb = c.blocks - 1;
            left = 0;
            break;
        }
    }
    c.span = kv_span<ROWS, TILE>(p, c.seq, c.rb);
    const int per_head = c.span.tiles + COST;
    c.h = left < ((int64_t)1 << 32) ? (int)((uint32_t)left / (uint32_t)per_head) : (int)(left / per_head);
    left -= (int64_t)c.h * per_head;
    c.at = r.begin - left;
    c.tile = (int)max(left - COST, (int64_t)0);
    return r;
}

// The CTA whose range holds place x, from CTA `from` on.
__device__ __forceinline__ int kv_owner(const KvRange& r, int64_t x, uint32_t from) {
    const KvCuts cuts(r.total, r.ctas);
    // an estimate from below, then the few steps that are left
    const float est = (float)x / (float)r.total * (float)r.ctas - 2.0f;
    uint32_t i = max(from, (uint32_t)fmaxf(est, 0.0f));
    while (i > from && cuts.at(i) > x) --i;
    while (i + 1 < r.ctas && cuts.at(i + 1) <= x) ++i;
    return (int)i;
}

}  // namespace

}  // namespace i8ql
