// Attention over the quantized key/value cache for few query rows (single
// tokens and short drafts): the codes are read once, in pages, and never
// written back wider.
//
//   a_j = c * sum_d q_d k_jd   (c = softmax scale * log2 e, j over the visible tokens)
//   o_d = sum_j w_j v_jd / sum_j w_j,   w_j = 2^(a_j - max a)
// with k_jd = low_j + s_j code_jd (and v the same), so that with centred
// codes c = code - z (z = 8 or 128)
//   sum_d q_d k_jd = s_j sum_d q_d c_jd + (low_j + z s_j) sum_d q_d
//   sum_j w_j v_jd = sum_j (w_j s_j) c_jd + sum_j w_j (low_j + z s_j):
// the products run on the codes themselves (small integers, exact in fp16)
// with the scales outside.  Centred, because sums of uncentred codes over a
// long context would be far larger than the result that is left of them.
//
// Precision: logits, totals and accumulators in fp32.  fp16 holds q exactly
// after a power of two per row has put its largest element near 2^8 (elements
// 2^32 times smaller round), and w_j s_j to 2^-11 after a power of two S per
// warp, raised as larger value scales appear, has put s_j / S below 1: eight
// times finer than bf16.  The weights are relative to a reference that a row's
// logits exceed by 2^5 at most (w_j s_j / S is held times 2^10, so it ends at
// 2^15); weights down to 2^-34 of the reference are kept, and to 2^-24 at 11
// bits, either times S / s_j less: S also counts the scales of tokens that only
// other rows of the block see.  References are held below 2^23 (shrink_reference).
// Keys of 2^110 and more can take the sums of the products past fp32.
//
// Bound by the bytes of the cache: 136 bytes a token and head (4 bits, 128
// channels, K and V).  Against them stands the unpacking, which is bound by
// the integer pipe (half rate), so the layout of the MMA operands is chosen
// to unpack with the fewest integer instructions:
//  * the cache is the 16-row A operand and the head group's queries are N (8
//    rows, or twice 8; a sequence with more takes several blocks): single
//    tokens of a group of up to 8 waste no MMA rows and no accumulators.
//    Q K^T comes out as tokens x queries, and one transpose of 8 x 8 halves
//    per 8 tokens makes it the B operand of P V;
//  * fp16 rather than bf16: its 10-bit mantissa takes a nibble at bits 0-3 or
//    4-7 as it lies (1024 + c, 1024 + 16 c), so a word of 8 codes needs one
//    shift, and the subtraction runs on the other (half-precision) pipe;
//  * the channel order of a sum over channels is free: a lane takes D / 4
//    neighbouring channels of a key row, and pairs code i with code i + 4,
//    which one mask yields (4 bits), or i + 1 (8 bits); q is permuted alike;
//  * values are paired across two tokens by byte permutes, and a lane's
//    channels of an output are neighbours (g D / 8 ..);
//  * a lane turns the scale and low value of one token into the four factors
//    the warp needs, and shares them through shared memory.
// A block is four such warps over 32 tokens of a 128-token tile each, with
// their own reference, and one warp that keeps 3 tiles of bulk copies
// in flight (61 KB a block at 4 bits and 128 channels, three blocks an SM).
//
// Measured, 32 query heads over 8 x 128, one token a sequence: 128 sequences of
// 16384 tokens in 440 us at 4 bits (5.2 TB/s, 77 % of a copy; warps wait on
// the chain unpack, product, softmax and for each other's issue slots), 64 of
// up to 4096 in 51 us with the join; at 8 bits, which unpack with fewer instructions
// a byte, 64 of 16384 in 345 us (6.4 TB/s, 94 %).  With pages of 16 tokens, whose
// tiles take 32 copies, these are 621 us (3.7 TB/s) and 427; short contexts do not
// mind (24 of up to 2047, 16 own heads, 8 bits: 31.3 us in pages of 16, 32.7 of 64).

#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kv_math.cuh"

namespace i8ql {
namespace {

constexpr int kTile = 128;                   // tokens per pipeline stage
constexpr int kWarps = 4;                    // consumer warps
constexpr int kWarpTokens = kTile / kWarps;  // tokens of a stage per warp
constexpr int kThreads = kWarps * 32 + 32;
constexpr float kSlack = 5.0f;    // a logit may exceed what the weights are relative to by this (log2)
constexpr int kValueShift = 10;   // w s / S is held times 2^this: at most 2^15 in fp16
// Tiles that beginning and ending an item counts (0 to 3 measure alike).
constexpr int kCost = 1;
// Query rows of a sequence's head group up to which this kernel runs.  Over 16
// sequences of 4096 tokens and 8 heads, 32 rows take it 64 us and the kernel for many
// rows 75 (4 bits, 128 channels; 75 and 94 at 8 bits, 40 and 67 with 64 channels); each
// 16 rows more read and unpack the cache once more here, about 22 us, and nothing there.
constexpr int64_t kFewRows = 32;

template <int D, int BITS, int ROWS>
struct Cfg {
    static constexpr int kBlocks = ROWS == 8 && BITS == 4 ? 3 : 2;  // resident blocks per SM
    static constexpr int kRowBytes = D * BITS / 8;
    static constexpr int kCodes = kTile * kRowBytes;
    static constexpr int kStageBytes = 2 * kCodes + 2 * kTile * 4;
    static constexpr int kStages = ROWS == 16 && BITS == 8 && D == 128 ? 2 : 3;  // (so that kBlocks fit an SM)
    // a merge row: D floats, 4 more after every 32 (spreads a warp's stores over the banks)
    static constexpr int kMergeRow = D + D / 8;
    static constexpr int kMergeBytes = 2 * ROWS * kMergeRow * 4;
    static constexpr int kSmem = kStages * kStageBytes + kMergeBytes;
    static_assert(kBlocks * (kSmem + 4608) <= 228 * 1024, "shared memory of the resident blocks");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of a warp's 8 x 8 matrix of halves (lane (g, t): row g, columns 2t and 2t + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

// S = 0: the work is shared out evenly (kv_schedule.cuh).  S > 0: a cluster of S
// CTAs takes one cache head of one sequence and joins its parts through
// distributed shared memory: one launch and no workspace, for calls of few and
// short contexts.
template <int D, int BITS, int HALVES, int S>
__global__ void __launch_bounds__(kThreads, Cfg<D, BITS, 8 * HALVES>::kBlocks)
    kv_attention_kernel(const KvAttnParams p) {
    constexpr int ROWS = 8 * HALVES;
    using C = Cfg<D, BITS, ROWS>;
    constexpr int kStages = C::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ KvLocate locate;
    __shared__ KvCursor cursors[kWarps];  // (kept out of the registers of the main loop)
    __shared__ KvRange range;
    __shared__ float merge_ml[kWarps][ROWS][2];
    __shared__ float shrunk[kWarps][ROWS];  // by how much a row's unit and reference have been shrunk, where any has
    __shared__ __align__(16) float cta_ml[ROWS][2];  // (S > 0) this CTA's part
    __shared__ float4 factors[kWarps][kWarpTokens];  // of a token: K scale and offset, V scale and offset
    __shared__ int abort_flag;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], kWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    pdl_launch_dependents();
    int stage = 0;
    uint32_t parity = 0;
    KvCursor start;
    KvRange found;
    const int rank = S > 0 ? (int)tc::cluster_rank() : 0;
    // A cursor's work: the tiles from its tile on that are this CTA's, and
    // whether there is any item left.  (S > 0: an item's tiles are cut evenly;
    // a CTA may have none of them.)
    auto part_begin = [&](const KvCursor& c) { return c.span.tiles * rank / max(S, 1); };
    auto work = [&](const KvCursor& c, int64_t end, int& n) {
        if constexpr (S == 0) {
            n = kv_take<kCost>(p, c, end);
            return n > 0;
        } else {
            if (c.rb >= c.blocks) return false;
            n = c.span.tiles * (rank + 1) / S - c.tile;
            return true;
        }
    };
    auto advance = [&](KvCursor& c) {
        if constexpr (S == 0) {
            kv_next_item<ROWS, kTile, kCost>(p, c);
        } else if (++c.rb < c.blocks) {
            c.span = kv_span<ROWS, kTile>(p, c.seq, c.rb);
            c.tile = part_begin(c);
        }
    };
    if constexpr (S == 0) {
        found = kv_locate<ROWS, kTile, kCost, kThreads>(p, locate, start);  // (its barriers also publish the mbarriers)
    } else {
        found = {};
        start = {};
        const int64_t item = blockIdx.x / S;
        start.b = item / p.cache.H;
        start.h = (int)(item - start.b * p.cache.H);
        start.seq = kv_sequence(p, start.b);
        start.blocks = kv_blocks<ROWS>(p, start.seq);
        if (start.blocks > 0) {
            start.span = kv_span<ROWS, kTile>(p, start.seq, 0);
            start.tile = part_begin(start);
        }
        __syncthreads();
    }

    if (warp == kWarps) {
        KvCursor& c = start;
        // ---------------------------------------------------------- producer
        // One lane per copy: four arrays (K and V codes and params) of up to
        // eight pieces of a tile (a piece is a page, or the tile's part of one).
        const int page_tokens = 1 << p.cache.page_shift;
        const int piece = min(page_tokens, kTile);
        const int kv = lane & 1, is_param = (lane >> 1) & 1;
        const int at = (lane >> 2) * piece;
        const uint32_t bytes = piece * (is_param ? 4 : C::kRowBytes);
        const int dst = is_param ? 2 * C::kCodes + kv * kTile * 4 + at * 4 : kv * C::kCodes + at * C::kRowBytes;
        int issued = 0;
        bool ok = true;
        int n = 0;
        while (work(c, found.end, n) && (ok || S > 0)) {
            const int32_t* table = p.table + c.b * p.table_width;
            const int first = (c.span.first + c.tile) * kTile + at;  // this lane's token of the item's next tile
            auto needed = [&](int i) {
                const int token = first + i * kTile;
                return i < n && at < kTile && token < c.span.end && token + piece > c.span.begin;
            };
            // pages are looked up two tiles ahead, so that no copy waits for its address
            int32_t ahead[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) ahead[i] = needed(i) ? __ldg(table + ((first + i * kTile) >> p.cache.page_shift)) : 0;
            for (int i = 0; i < n && ok; ++i) {
                const int token = first + i * kTile;
                const bool need = needed(i);
                int64_t page = ahead[0];
                ahead[0] = ahead[1];
                ahead[1] = needed(i + 2) ? __ldg(table + ((token + 2 * kTile) >> p.cache.page_shift)) : 0;
                const uint8_t* src = nullptr;
                if (need) {
                    if (page < 0 || page >= p.cache.pages) {
                        record_fault(p.err, kErrBitBadIndex);
                        page = 0;
                    }
                    const int64_t row = kv_row(p.cache, page, kv, c.h, token & (page_tokens - 1));
                    src = is_param ? reinterpret_cast<const uint8_t*>(p.cache.params + row)
                                   : p.cache.codes + row * C::kRowBytes;
                }
                const unsigned copies = __popc(__ballot_sync(0xffffffffu, need)) / 4;
                ok = tc::warp_wait(&empty[stage], parity ^ 1, &abort_flag, p.err);
                // a consumer that gave up says so before it frees a stage that it
                // did not wait for, whose copies may still be on their way
                ok = ok && !__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&abort_flag));
                if (!ok) break;
                if (lane == 0) tc::mbar_expect_tx(&full[stage], copies * piece * (2 * C::kRowBytes + 8));
                __syncwarp();
                if (need) bulk_load(smem + stage * C::kStageBytes + dst, src, bytes, &full[stage]);
                ++issued;
                if (++stage == kStages) {
                    stage = 0;
                    parity ^= 1;
                }
            }
            if constexpr (S > 0) {  // the barriers of the join
                __syncwarp();
                tc::cluster_sync_all();
                tc::cluster_sync_all();
            }
            advance(c);
        }
        // the last copies land before the block's shared memory can go to
        // another (the consumers may have given up on them)
        for (int i = 0; i < min(issued, kStages); ++i) {
            int none = 0;
            if (--stage < 0) {
                stage = kStages - 1;
                parity ^= 1;
            }
            tc::mbar_wait(&full[stage], parity, &none, p.err);
        }
        return;
    }

    // -------------------------------------------------------------- consumers
    constexpr int kKeyWords = D * BITS / 128;     // words of a key row per lane
    constexpr int kValWords = D * BITS / 256;     // words of a value row per lane
    constexpr int kOut = D / 16;                  // 16-channel tiles of the output
    constexpr int kPairs = 16 / BITS;             // pairs per word
    constexpr int kSteps = D / 16;
    const int g = lane / 4, t = lane % 4;
    const int row_g = g ^ ((g >> 1) & 1);  // the token of row g (of 8): rows of both parities in every load (banks)
    const int tok0 = (2 * t) ^ (t & 1), tok1 = (2 * t + 1) ^ (t & 1);  // the same for rows 2t and 2t + 1
    float* merge = reinterpret_cast<float*>(smem + kStages * C::kStageBytes);

    KvCursor& c = cursors[warp];
    if (lane == 0) c = start;
    if (threadIdx.x == 0) range = found;
    consumer_sync();
    bool split = false;
    int n = 0;
    while (work(c, range.end, n)) {
        const int row0 = c.rb * ROWS;
        const int rows = min(ROWS, c.seq.nq * p.G - row0);
        const int base = c.seq.len - c.seq.nq;
        // this lane's rows of Q (B operand: rows g, g + 8), permuted as the
        // keys' unpacking pairs channels, times 2^8 / (the power of two below
        // the row's largest element)
        uint32_t qf[kSteps][HALVES][2];
        // of the rows 2t and 2t + 1 (+ 8), whose logits the lane holds:
        float q_sum[HALVES][2];   // the scaled row's sum
        float q_unit[HALVES][2];  // what a scaled logit counts, in log2 units
        int hi[HALVES][2], lo[HALVES][2];  // the tokens the row sees: lo .. hi
#pragma unroll
        for (int x = 0; x < HALVES; ++x) {
            const int r = g + 8 * x;
            const bool live = r < rows;
            const int i = (row0 + (live ? r : 0)) / p.G;
            const int head = c.h * p.G + (row0 + (live ? r : 0)) - i * p.G;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (c.seq.q0 + i) * p.q_stride + (int64_t)head * D +
                                                              t * (D / 4));
            uint4 v[D / 32];
            uint32_t top = 0;  // largest finite magnitude, as bits
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                v[w] = live ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
                const uint32_t words[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a = words[j] & 0x7fff0000u, b = (words[j] << 16) & 0x7fff0000u;
                    top = max(top, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
                }
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = max((int)(top >> 23), 9) - 127;
            const float f = p.scale_log2 < 0.0f ? -pow2(8 - e) : pow2(8 - e);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const float y[8] = {lo_bf16(v[w].x) * f, hi_bf16(v[w].x) * f, lo_bf16(v[w].y) * f, hi_bf16(v[w].y) * f,
                                    lo_bf16(v[w].z) * f, hi_bf16(v[w].z) * f, lo_bf16(v[w].w) * f, hi_bf16(v[w].w) * f};
                sum += ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
                uint32_t (&f0)[2] = qf[2 * w][x], (&f1)[2] = qf[2 * w + 1][x];
                if constexpr (BITS == 4) {  // 8 channels: (0,4) (1,5) | (2,6) (3,7)
                    f0[0] = pack_f16(y[0], y[4]);
                    f0[1] = pack_f16(y[1], y[5]);
                    f1[0] = pack_f16(y[2], y[6]);
                    f1[1] = pack_f16(y[3], y[7]);
                } else {  // twice 4 channels: (0,1) (2,3)
                    f0[0] = pack_f16(y[0], y[1]);
                    f0[1] = pack_f16(y[2], y[3]);
                    f1[0] = pack_f16(y[4], y[5]);
                    f1[1] = pack_f16(y[6], y[7]);
                }
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const float unit = pow2(e - 8) * fabsf(p.scale_log2);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int from = 4 * (2 * t + y);  // a lane that loaded row 2t + y
                q_sum[x][y] = __shfl_sync(0xffffffffu, sum, from);
                q_unit[x][y] = __shfl_sync(0xffffffffu, unit, from);
                const int j = __shfl_sync(0xffffffffu, i, from);
                const bool there = 8 * x + 2 * t + y < rows;
                hi[x][y] = there ? base + j : INT32_MAX;
                lo[x][y] = there && p.window > 0 ? (int)max(base + j + 1 - p.window, (int64_t)0) : 0;
            }
        }
        const int seen_begin = c.span.begin, seen_end = c.span.end;
        const int first_token = (c.span.first + c.tile) * kTile + warp * kWarpTokens;
        // tokens [all_lo, all_hi] are seen by every row
        const int all_hi = base + row0 / p.G;
        const int all_lo = p.window > 0 ? (int)max(base + (row0 + rows - 1) / p.G + 1 - p.window, (int64_t)0) : 0;

        // O^T: channels g D/8 + 2i (+ 1) x rows 2t, 2t + 1 (+ 8)
        float o[kOut][HALVES][4];
        // what the weights are relative to (a logit; at most kSlack below the row's
        // maximum); this lane's share of the total and of sum w (low + z s)
        float m[HALVES][2], l[HALVES][2], z[HALVES][2];
        bool any_shrunk = false;
        int unit = kValueShift;  // S = 2^(unit - 126) is above every value scale so far
#pragma unroll
        for (int x = 0; x < HALVES; ++x) {
#pragma unroll
            for (int i = 0; i < kOut; ++i) o[i][x][0] = o[i][x][1] = o[i][x][2] = o[i][x][3] = 0.0f;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                m[x][y] = -INFINITY;
                l[x][y] = z[x][y] = 0.0f;
            }
        }

        // One warp's 32 tokens of a stage.  EDGE: some row does not see some of them.
        auto step = [&](const uint8_t* st, int token, auto edge_tag) {
            constexpr bool EDGE = decltype(edge_tag)::value;
            // this lane's token: its scales and low values
            {
                const uint32_t* params = reinterpret_cast<const uint32_t*>(st + 2 * C::kCodes) + warp * kWarpTokens + lane;
                uint32_t pk = params[0], pv = params[kTile];
                if (EDGE && (token + lane >= seen_end || token + lane < seen_begin)) pk = pv = 0;  // may be anything
                const float ks = kv_scale(pk), vs = kv_scale(pv);
                const uint32_t bits = __float_as_uint(vs);
                const int e = (int)(__reduce_max_sync(0xffffffffu, bits < 0x7f800000u ? bits : 0u) >> 23);
                if (e > unit) {
                    const float f = e - unit > 126 ? 0.0f : pow2(unit - e);
                    unit = e;
#pragma unroll
                    for (int j = 0; j < kOut; ++j)
#pragma unroll
                        for (int x = 0; x < HALVES; ++x)
#pragma unroll
                            for (int y = 0; y < 4; ++y) o[j][x][y] *= f;
                }
                factors[warp][lane] = make_float4(ks, fmaf(ks, kCentre<BITS>, kv_low(pk)), vs * pow2(kValueShift + 126 - unit),
                                                  fmaf(vs, kCentre<BITS>, kv_low(pv)));
                __syncwarp();
            }
            // logits: s[i]: tokens row_g + 16 i (+ 8) x rows 2t, 2t + 1
            float s[2][HALVES][4];
            const uint8_t* keys = st + (warp * kWarpTokens + row_g) * C::kRowBytes + t * (kKeyWords * 4);
            uint32_t kw[4][kKeyWords];
#pragma unroll
            for (int i = 0; i < 4; ++i) lds<kKeyWords>(keys + i * 8 * C::kRowBytes, kw[i]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < HALVES; ++x) s[i][x][0] = s[i][x][1] = s[i][x][2] = s[i][x][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < kKeyWords; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t a[kPairs], b[kPairs];
                    unpack_key<BITS, true>(kw[2 * i][k], a);
                    unpack_key<BITS, true>(kw[2 * i + 1][k], b);
#pragma unroll
                    for (int j = 0; j < kPairs; j += 2)
#pragma unroll
                        for (int x = 0; x < HALVES; ++x) {
                            const uint32_t (&q)[2] = qf[(k * kPairs + j) / 2][x];
                            mma_f16(s[i][x], a[j], b[j], a[j + 1], b[j + 1], q[0], q[1]);
                        }
                }
            float top[HALVES][2];
            float4 f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = factors[warp][row_g + 8 * i];
#pragma unroll
            for (int x = 0; x < HALVES; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    top[x][y] = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& a = s[i / 2][x][2 * (i & 1) + y];
                        a = fmaf(a, f[i].x, f[i].y * q_sum[x][y]);
                        const int tok = token + row_g + 8 * i;
                        if (EDGE && (tok > hi[x][y] || tok < lo[x][y])) a = -INFINITY;
                        top[x][y] = fmaxf(top[x][y], a);
                    }
                }
            // softmax weights; the reference is raised only when a logit exceeds
            // it by kSlack, which spares the other steps the sums' rescaling and
            // the exchange between the lanes of a row
            bool above = false;
#pragma unroll
            for (int x = 0; x < HALVES; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    top[x][y] *= q_unit[x][y];
                    above |= top[x][y] > m[x][y] + kSlack;  // (the first time: from -infinity)
                }
            if (__any_sync(0xffffffffu, above)) {
                bool large = false;
#pragma unroll
                for (int x = 0; x < HALVES; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) large |= fabsf(top[x][y]) >= 0x1p23f && top[x][y] != -INFINITY;
                large = __any_sync(0xffffffffu, large);
#pragma unroll
                for (int x = 0; x < HALVES; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
#pragma unroll
                        for (int k = 4; k < 32; k <<= 1)
                            top[x][y] = fmaxf(top[x][y], __shfl_xor_sync(0xffffffffu, top[x][y], k));
                    }
                if (__builtin_expect(large, 0)) {  // (rare)
#pragma unroll
                    for (int x = 0; x < HALVES; ++x)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float shrink = shrink_reference(fmaxf(m[x][y], top[x][y]));
                            m[x][y] *= shrink;
                            top[x][y] *= shrink;
                            q_unit[x][y] *= shrink;
                            float& all = shrunk[warp][8 * x + 2 * t + y];
                            if (g == 0) all = any_shrunk ? all * shrink : shrink;
                        }
                    any_shrunk = true;
                }
#pragma unroll
                for (int x = 0; x < HALVES; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float to = fmaxf(m[x][y], top[x][y]);
                        const float by = to == -INFINITY ? 1.0f : exp2_approx(m[x][y] - to);
                        m[x][y] = to;
                        l[x][y] *= by;
                        z[x][y] *= by;
#pragma unroll
                        for (int j = 0; j < kOut; ++j) {
                            o[j][x][y] *= by;
                            o[j][x][2 + y] *= by;
                        }
                    }
            }
            uint32_t pr[4][HALVES];  // P^T as B operand: tokens of rows 2t, 2t + 1 (+ 8 i) x row g
#pragma unroll
            for (int x = 0; x < HALVES; ++x) {
                float shift[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) shift[y] = m[x][y] == -INFINITY ? 0.0f : m[x][y];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float wgt[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float a = s[i / 2][x][2 * (i & 1) + y];
                        // a token a row does not see may hold anything: no product with it
                        const bool skip = EDGE && (token + row_g + 8 * i > hi[x][y] || token + row_g + 8 * i < lo[x][y]);
                        float w = exp2_approx(fmaf(a, q_unit[x][y], -shift[y]));
                        if (skip) w = 0.0f;
                        l[x][y] += w;
                        z[x][y] = skip ? z[x][y] : fmaf(w, f[i].w, z[x][y]);
                        wgt[y] = skip ? 0.0f : w * f[i].z;
                    }
                    pr[i][x] = transpose8(pack_f16(wgt[0], wgt[1]));
                }
            }
            // o += (w s 2^kValueShift / S) (codes of V)
            const uint8_t* vals = st + C::kCodes + warp * kWarpTokens * C::kRowBytes + g * (kValWords * 4);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t v[4][kValWords];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    lds<kValWords>(vals + (16 * half + 8 * (r >> 1) + ((r & 1) ? tok1 : tok0)) * C::kRowBytes, v[r]);
#pragma unroll
                for (int k = 0; k < kValWords; ++k) {
                    uint32_t a[2 * kPairs], b[2 * kPairs];
                    unpack_values<BITS, true>(v[0][k], v[1][k], a);
                    unpack_values<BITS, true>(v[2][k], v[3][k], b);
#pragma unroll
                    for (int j = 0; j < 2 * kPairs; j += 2)
#pragma unroll
                        for (int x = 0; x < HALVES; ++x)
                            mma_f16(o[k * kPairs + j / 2][x], a[j], a[j + 1], b[j], b[j + 1], pr[2 * half][x],
                                    pr[2 * half + 1][x]);
                }
            }
        };

        for (int i = 0; i < n; ++i) {
            const bool ok = tc::warp_wait(&full[stage], parity, &abort_flag, p.err);
            const uint8_t* st = smem + stage * C::kStageBytes;
            const int token = first_token + i * kTile;
            // (a warp whose tokens no row sees has nothing to do)
            if (ok && token < seen_end && token + kWarpTokens > seen_begin) {
                if (token + kWarpTokens - 1 > all_hi || token < all_lo)
                    step(st, token, std::true_type{});
                else
                    step(st, token, std::false_type{});
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[stage]);
            if (++stage == kStages) {
                stage = 0;
                parity ^= 1;
            }
        }

        if (__builtin_expect(any_shrunk, 0))
#pragma unroll
            for (int x = 0; x < HALVES; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) m[x][y] /= shrunk[warp][8 * x + 2 * t + y];
        // join the four warps: totals over the lanes of a row, then one common maximum
#pragma unroll
        for (int x = 0; x < HALVES; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) {
                    l[x][y] += __shfl_xor_sync(0xffffffffu, l[x][y], k);
                    z[x][y] += __shfl_xor_sync(0xffffffffu, z[x][y], k);
                }
                if (g == 0) {
                    merge_ml[warp][8 * x + 2 * t + y][0] = m[x][y];
                    merge_ml[warp][8 * x + 2 * t + y][1] = l[x][y];
                }
            }
        consumer_sync();
#pragma unroll
        for (int x = 0; x < HALVES; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int r = 8 * x + 2 * t + y;
                float top = merge_ml[0][r][0];
                for (int w = 1; w < kWarps; ++w) top = fmaxf(top, merge_ml[w][r][0]);
                const float f = l[x][y] == 0.0f ? 0.0f : exp2_approx(m[x][y] - top);  // (0: saw nothing)
#pragma unroll
                for (int j = 0; j < kOut; ++j)
#pragma unroll
                    for (int k = y; k < 4; k += 2)
                        o[j][x][k] = f == 0.0f ? 0.0f : fmaf(o[j][x][k], pow2(unit - 126 - kValueShift), z[x][y]) * f;
            }
        // a lane holds D / 8 channels from g D / 8 on of rows 2t and 2t + 1 (+ 8)
        const int at = g * (D / 8) + 4 * (g * (D / 8) / 32);
        for (int turn = 0; turn < 2; ++turn) {
            if (warp / 2 == 1 - turn) {
#pragma unroll
                for (int x = 0; x < HALVES; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int j = 0; j < kOut; j += 2) {
                            float4* dst = reinterpret_cast<float4*>(
                                merge + ((warp & 1) * ROWS + 8 * x + 2 * t + y) * C::kMergeRow + at + 2 * j);
                            float4 v = make_float4(o[j][x][y], o[j][x][2 + y], o[j + 1][x][y], o[j + 1][x][2 + y]);
                            if (turn == 1) {
                                const float4 u = *dst;
                                v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                            }
                            *dst = v;
                        }
            }
            consumer_sync();
        }
        const int tid = threadIdx.x;
        auto local_sum = [&](int r, int d, float (&v)[8]) {  // of the two halves of the block's warps
            const float* src = merge + r * C::kMergeRow + d + 4 * (d / 32);
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const float4 a = *reinterpret_cast<const float4*>(src + j);
                const float4 b = *reinterpret_cast<const float4*>(src + ROWS * C::kMergeRow + j);
                v[j] = a.x + b.x;
                v[j + 1] = a.y + b.y;
                v[j + 2] = a.z + b.z;
                v[j + 3] = a.w + b.w;
            }
        };
        auto local_ml = [&](int r) {
            float top = merge_ml[0][r][0], total = 0.0f;
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, merge_ml[w][r][0]);
            for (int w = 0; w < kWarps; ++w)
                total += merge_ml[w][r][1] == 0.0f ? 0.0f : merge_ml[w][r][1] * exp2_approx(merge_ml[w][r][0] - top);
            return make_float2(top, total);
        };
        auto write_out = [&](int r, int d, const float (&v)[8], float total) {
            const int i = (row0 + r) / p.G;
            const int head = c.h * p.G + row0 + r - i * p.G;
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
            *reinterpret_cast<uint4*>(p.out + ((c.seq.q0 + i) * ((int64_t)p.cache.H * p.G) + head) * D + d) =
                make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                           pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
        };
        const bool store = *reinterpret_cast<volatile int*>(&abort_flag) == 0;
        if constexpr (S > 0) {
            // this CTA's part in the first merge rows; then each CTA joins its share of the outputs
            for (int k = tid; k < ROWS * (D / 8); k += kWarps * 32) {
                const int r = k / (D / 8), d = (k % (D / 8)) * 8;
                float v[8];
                local_sum(r, d, v);
                float4* dst = reinterpret_cast<float4*>(merge + r * C::kMergeRow + d + 4 * (d / 32));
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                if (d == 0) *reinterpret_cast<float2*>(cta_ml[r]) = local_ml(r);
            }
            __syncwarp();
            tc::cluster_sync_all();
            for (int k = tid * S + rank; k < rows * (D / 8) && store; k += kWarps * 32 * S) {
                const int r = k / (D / 8), d = (k % (D / 8)) * 8;
                const uint32_t ml_at = tc::smem_u32(cta_ml[r] - (r & 1) * 2);  // (pairs of rows: 16-byte loads)
                const uint32_t v_at = tc::smem_u32(merge + r * C::kMergeRow + d + 4 * (d / 32));
                float2 ml[S];
                float top = -INFINITY, total = 0.0f, v[8] = {};
#pragma unroll
                for (int y = 0; y < S; ++y) {
                    const int4 x = tc::ld_dsmem_v4(ml_at, y);
                    ml[y] = (r & 1) ? make_float2(__int_as_float(x.z), __int_as_float(x.w))
                                    : make_float2(__int_as_float(x.x), __int_as_float(x.y));
                    top = fmaxf(top, ml[y].x);
                }
#pragma unroll
                for (int y = 0; y < S; ++y) {
                    const float f = ml[y].y == 0.0f ? 0.0f : exp2_approx(ml[y].x - top);
                    total += ml[y].y * f;
                    const int4 a = tc::ld_dsmem_v4(v_at, y), b = tc::ld_dsmem_v4(v_at + 16, y);
                    const int x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = fmaf(__int_as_float(x[j]), f, v[j]);
                }
                write_out(r, d, v, total);
            }
            __syncwarp();
            tc::cluster_sync_all();  // no CTA's rows are overwritten or gone while others read them
        } else {
            const bool begins = c.tile == 0, ends = c.tile + n == c.span.tiles;
            for (int k = tid; k < rows * (D / 8) && store; k += kWarps * 32) {
                const int r = k / (D / 8), d = (k % (D / 8)) * 8;
                float v[8];
                local_sum(r, d, v);
                const float2 ml = local_ml(r);
                if (begins && ends) {
                    write_out(r, d, v, ml.y);
                } else {
                    const int64_t slot = ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * ROWS + r;
                    float4* dst = reinterpret_cast<float4*>(p.part_o + slot * D + d);
                    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                    if (d == 0) *reinterpret_cast<float2*>(p.part_ml + slot * 2) = ml;
                }
            }
            if (begins && !ends && store) {
                split = true;
                if (tid == 0) {
                    KvSplitItem it;
                    it.q_row = c.seq.q0;
                    it.row0 = row0;
                    it.rows = rows;
                    it.h = c.h;
                    it.last_cta = kv_owner(range, c.at + kCost + c.span.tiles - 1, blockIdx.x);
                    it.pad = 0;
                    p.split[blockIdx.x] = it;
                }
            }
        }
        __syncwarp();
        if (lane == 0) advance(c);
        consumer_sync();  // the cursor is at the next item, and the merge rows are free again
    }
    if (threadIdx.x == 0 && p.split != nullptr && !split) p.split[blockIdx.x].rows = 0;
}

// Joins the parts of an item cut between CTAs, always in the same order.  A
// block takes 8 rows: of an item of few parts a warp each, of more the warps
// share the parts (each warp all 8 rows of a part, so that 8 loads are under
// way) and then add up.  (Blocks of 8 warps: most CTAs have an item of two or
// three parts or none, and small blocks run side by side.)  Bound by the latency
// of its chain of loads: with cold caches 5 us for 64 sequences of 4096 tokens, 9.5 for 2
// of 131072, 27 for two prompt chunks of 2048, whose parts are 35 MB.
constexpr int kJoinWarps = 8;

template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32) kv_join_kernel(const KvAttnParams p) {
    constexpr int kVec = D / 32;  // channels per lane
    __shared__ float sums[kJoinWarps][kJoinWarps][D];  // [warp][row]
    __shared__ float totals[kJoinWarps][kJoinWarps];
    pdl_wait();
    if constexpr (ROWS <= 16) pdl_launch_dependents();  // (one wave)
    const KvSplitItem it = p.split[blockIdx.x];
    const int r0 = blockIdx.y * kJoinWarps;
    if (r0 >= it.rows) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int first = blockIdx.x, count = it.last_cta - first + 1;
    // part k: the beginning (slot 1 of the first CTA), then slot 0 of the following ones
    auto slot = [&](int k, int r) { return ((int64_t)(first + k) * 2 + (k == 0 ? 1 : 0)) * ROWS + r; };
    auto ml = [&](int k, int r) { return *reinterpret_cast<const float2*>(p.part_ml + slot(k, r) * 2); };
    auto store = [&](int r, const float (&x)[kVec], float inv) {
        const int i = (it.row0 + r) / p.G;
        const int head = it.h * p.G + it.row0 + r - i * p.G;
        uint16_t* dst = p.out + ((it.q_row + i) * ((int64_t)p.cache.H * p.G) + head) * D + lane * kVec;
        if constexpr (kVec == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv));
        else
            *reinterpret_cast<uint32_t*>(dst) = pack_bf16(x[0] * inv, x[1] * inv);
    };
    auto fetch = [&](int k, int r, float (&x)[kVec]) {
        const float* src = p.part_o + slot(k, r) * D + lane * kVec;
        if constexpr (kVec == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            x[0] = v.x;
            x[1] = v.y;
            x[2] = v.z;
            x[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            x[0] = v.x;
            x[1] = v.y;
        }
    };
    // a part's weight; 0 where it saw nothing
    auto weigh = [](float2 x, float top) { return x.y == 0.0f ? 0.0f : exp2_approx(x.x - top); };
    if (count <= kJoinWarps) {
        const int r = r0 + warp;
        if (r >= it.rows) return;
        float2 x[kJoinWarps];
        float top = -INFINITY, total = 0.0f, acc[kVec] = {};
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) {
            x[k] = k < count ? ml(k, r) : make_float2(-INFINITY, 0.0f);
            top = fmaxf(top, x[k].x);
        }
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) {
            if (k >= count) break;
            const float f = weigh(x[k], top);
            total += x[k].y * f;
            float v[kVec];
            fetch(k, r, v);
#pragma unroll
            for (int i = 0; i < kVec; ++i) acc[i] = fmaf(v[i], f, acc[i]);
        }
        store(r, acc, total == 0.0f ? 0.0f : 1.0f / total);
        return;
    }
    // the rows' references: lane l looks at row r0 + l % 8, parts l / 8, l / 8 + 4, ..
    const int my_row = r0 + lane % kJoinWarps;
    float top = -INFINITY;
    if (my_row < it.rows)
        for (int k = lane / kJoinWarps; k < count; k += 4) top = fmaxf(top, ml(k, my_row).x);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
    float acc[kJoinWarps][kVec] = {}, total = 0.0f;  // (the total: of row my_row)
    for (int k = warp; k < count; k += kJoinWarps) {
        float weight = 0.0f;  // of the part in row my_row
        if (my_row < it.rows) {
            const float2 x = ml(k, my_row);
            weight = weigh(x, top);
            total += x.y * weight;
        }
        float v[kJoinWarps][kVec];
#pragma unroll
        for (int j = 0; j < kJoinWarps; ++j) {
            if (r0 + j < it.rows) fetch(k, r0 + j, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kJoinWarps; ++j) {
            const float f = __shfl_sync(0xffffffffu, weight, j);
            if (r0 + j >= it.rows) continue;
#pragma unroll
            for (int i = 0; i < kVec; ++i) acc[j][i] = fmaf(v[j][i], f, acc[j][i]);
        }
    }
#pragma unroll
    for (int j = 0; j < kJoinWarps; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) sums[warp][j][lane * kVec + i] = acc[j][i];
    if (lane < kJoinWarps) totals[warp][lane] = total;
    __syncthreads();
    const int r = r0 + warp;
    if (r >= it.rows) return;
    float out[kVec] = {}, all = 0.0f;
    for (int w = 0; w < kJoinWarps; ++w) {
        all += totals[w][warp];
#pragma unroll
        for (int i = 0; i < kVec; ++i) out[i] += sums[w][warp][lane * kVec + i];
    }
    store(r, out, all == 0.0f ? 0.0f : 1.0f / all);
}

template <int D, int ROWS>
cudaError_t launch_join(const KvAttnParams& p, int64_t ctas, const LaunchEnv& env) {
    return launch_kernel(kv_join_kernel<D, ROWS>, dim3((unsigned)ctas, ROWS / kJoinWarps), dim3(kJoinWarps * 32), 0,
                         env.stream, kNoCluster, p);
}

// How a call runs: the query rows of a block, the CTAs, whether an item may be
// cut between CTAs (and is joined by a second kernel), and whether it runs as
// clusters that join by themselves.
struct Plan {
    int rows;
    int64_t ctas;
    bool split;
    bool cluster;
};

// Contexts of up to this many tiles run as clusters when all clusters fit the device
// at once.  (By the page table's width, since only the device knows the lengths: short
// contexts behind a wide table run in the other form.)  One sequence of 517 tokens takes 10.9
// us so, 14.9 in two launches (events around the call; 5.3 us on the device), one
// of 16000 23.2 against 25.2, one of 32000 39.6 against 29.3.
constexpr int kClusterSize = 8;
constexpr int64_t kClusterTiles = 128;

Plan make_plan(int64_t B, int64_t T_q, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int64_t bits, int sms) {
    Plan pl;
    pl.rows = max_q * G <= 8 ? 8 : max_q * G <= kFewRows ? 16 : kKvPromptRows;
    const int64_t per_sm = pl.rows == kKvPromptRows ? 1 : pl.rows == 8 && bits == 4 ? 3 : 2;
    // no more CTAs than there can be tiles
    const int64_t tile = pl.rows == kKvPromptRows ? kKvPromptTile : kTile;
    const int64_t item_tiles = std::max<int64_t>((max_kv + tile - 1) / tile, 1);
    const int64_t items = (T_q * G / pl.rows + B) * H;
    pl.ctas = items > sms * per_sm ? sms * per_sm : std::min<int64_t>(sms * per_sm, items * item_tiles);
    pl.split = item_tiles > 1;
    pl.cluster = pl.rows != kKvPromptRows && item_tiles > 1 && item_tiles <= kClusterTiles &&
                 B * H * kClusterSize <= sms * per_sm;
    if (pl.cluster) {
        pl.ctas = B * H * kClusterSize;
        pl.split = false;
    }
    return pl;
}

size_t part_bytes(int64_t ctas, int64_t rows, int64_t D) { return (size_t)(ctas * 2 * rows * (D + 2) * 4); }

template <int D, int BITS, int HALVES, int S>
cudaError_t launch_size(const KvAttnParams& p, const Plan& pl, const LaunchEnv& env) {
    using C = Cfg<D, BITS, 8 * HALVES>;
    const cudaError_t e = allow_smem<kv_attention_kernel<D, BITS, HALVES, S>>(C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kv_attention_kernel<D, BITS, HALVES, S>, dim3((unsigned)pl.ctas), dim3(kThreads), C::kSmem,
                         env.stream, S > 0 ? dim3(S, 1, 1) : kNoCluster, p);
}

template <int D, int BITS, int HALVES>
cudaError_t launch_form(const KvAttnParams& p, const Plan& pl, const LaunchEnv& env) {
    return pl.cluster ? launch_size<D, BITS, HALVES, kClusterSize>(p, pl, env)
                      : launch_size<D, BITS, HALVES, 0>(p, pl, env);
}

template <int D>
cudaError_t launch_dim(const KvAttnParams& p, int64_t bits, const Plan& pl, const LaunchEnv& env) {
    cudaError_t e;
    if (pl.rows == kKvPromptRows)
        e = launch_kv_prompt(p, D, bits, pl.ctas, env);
    else if (bits == 4)
        e = pl.rows == 8 ? launch_form<D, 4, 1>(p, pl, env) : launch_form<D, 4, 2>(p, pl, env);
    else
        e = pl.rows == 8 ? launch_form<D, 8, 1>(p, pl, env) : launch_form<D, 8, 2>(p, pl, env);
    if (e != cudaSuccess || !pl.split) return e;
    if (pl.rows == kKvPromptRows) return launch_join<D, kKvPromptRows>(p, pl.ctas, env);
    return pl.rows == 8 ? launch_join<D, 8>(p, pl.ctas, env) : launch_join<D, 16>(p, pl.ctas, env);
}

}  // namespace

size_t kv_attention_workspace(int64_t B, int64_t T_q, int64_t G, int64_t H, int64_t D, int64_t bits, int64_t max_kv,
                              int64_t max_q, int sms) {
    const Plan pl = make_plan(B, T_q, G, H, max_kv, max_q, bits, sms);
    if (!pl.split) return 0;
    return part_bytes(pl.ctas, pl.rows, D) + (size_t)pl.ctas * sizeof(KvSplitItem);
}

cudaError_t launch_kv_attention(KvAttnParams p, int64_t D, int64_t bits, int64_t max_q, void* workspace,
                                const LaunchEnv& env) {
    const Plan pl = make_plan(p.B, p.T_q, p.G, p.cache.H, p.table_width << p.cache.page_shift, max_q, bits,
                              env.sm_count);
    p.part_o = nullptr;
    p.part_ml = nullptr;
    p.split = nullptr;
    if (pl.split) {
        const int64_t slots = pl.ctas * 2 * pl.rows;
        p.part_o = static_cast<float*>(workspace);
        p.part_ml = p.part_o + slots * D;
        p.split = reinterpret_cast<KvSplitItem*>(p.part_ml + slots * 2);
    }
    return D == 64 ? launch_dim<64>(p, bits, pl, env) : launch_dim<128>(p, bits, pl, env);
}

}  // namespace i8ql
