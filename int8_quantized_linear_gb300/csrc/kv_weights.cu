// Attention weights summed per cached token: how much attention the query rows
// of a call give each token of the quantized cache, for eviction.
//
//   a_ij = c * sum_d q_id k_jd   (c = softmax scale * log2 e, j over the tokens that row i sees)
//   w_j  = previous_j + sum_i 2^(a_ij - m_i) / l_i,   m_i = max_j a_ij, l_i = sum_j 2^(a_ij - m_i)
// over the query rows of a cache head (its group's heads, all query tokens).
// With k_jd = low_j + s_j code_jd the products run on the codes themselves, and the
// scales are applied outside:
//   sum_d q_d k_jd = s_j sum_d q_d code_jd + low_j sum_d q_d.
// A code is an fp16 number as it lies: the integer c in the low bits of a half is
// 2^-24 c (subnormal, exact), and a nibble one place up 2^-24 16 c, which the query's
// element makes up for by a 16th.  So unpacking is masks alone, five instructions for
// eight 4-bit codes (and nine to make centred integers of them: see kv_math.cuh).
// q is scaled by a power of two per row that brings its largest element to 2^14;
// elements 2^-28 of that round.  Logits, maxima and sums are fp32.  What a product counts is
// a power of two: c's mantissa is multiplied into the scales and the sum of q.  So a maximum
// is a logit without rounding, and an exponent a - m, taken in one step from the product, is 0
// for the largest, however large the logits are.  (With the mantissa in that step an exponent
// misses what m was rounded by, which leaves fp32 where logits reach 2^31.)  Maximum and sum are
// kept apart (2^(a - m) / l, not 2^(a - m - log2 l)): beside a large m the logarithm
// would lose its bits.
//
// A weight needs its row's maximum and sum, which need all keys.  While a cluster's
// shared memory holds the logits of a cache head (one token's rows, contexts up to 32768
// with four query heads), one launch reads the keys once: 96 sequences of 16384 tokens, 8 x
// 128 channels, 4 bits, 248 us, of 143 for the bytes (3.8 TB/s; the products, the
// exchange and the sums of a block follow each other, and four blocks an SM cover for it).
// Otherwise two kernels both go over the keys.  The first leaves each row's (m, l) over
// a part of the tokens, the second joins them and sums the weights of its tokens over all
// rows, in order; no atomics.  16 sequences of up to 8191 tokens with 64 rows a
// head (16 heads x 64 channels, 8 bits): 58 and 52 us, bound by the instructions beside
// the products (unpacking per 32 rows, an exponential a logit and pass; issue slots 40 and 50 %,
// 8 and 11 warps an SM) and by the beginnings and ends of blocks.
// Tokens that no row sees keep what they have.
//
// The layout of the products is that of kv_attention.cu: 16 tokens are the M rows
// of an MMA (A: codes as they lie, a lane taking D / 4 neighbouring channels of
// a token), 8 query rows its columns.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv_tc.cuh"
#include "kv_weights.cuh"

namespace i8ql {
namespace {

// The two kernels:
constexpr int kTile = 128;   // tokens a block works on at a time
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 16;   // most tiles of a block of the second kernel
template <int D, int BITS>
constexpr int kStages = D * BITS == 128 * 8 ? 3 : 4;
// All in one:
constexpr int kOneTile = 256;
constexpr int kOneWarps = 8;
constexpr int kOneThreads = kOneWarps * 32;
constexpr int kOneStages = 1;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A sequence's sizes; more query tokens than max_q are recorded and left out.
__device__ __forceinline__ KvSeq weights_sequence(const KvWeightsParams& p, int64_t b) {
    KvSeq s = kv_sequence(p.a, b);
    if (s.nq > p.max_q) {
        record_fault(p.a.err, kErrBitBadIndex);
        s.nq = (int32_t)p.max_q;
    }
    return s;
}

// What a product counts, in log2 units, where the row's largest element has the exponent e.
// (Not 0: what is not seen, -inf, times 0 would be no number.)
__device__ __forceinline__ float product_unit(const KvScale& scale, int e) {
    return pow2(min(max(e - 14 + 24 + scale.exponent, -126), 127));
}

// A lane's share of 8 HALVES query rows.
template <int D, int BITS, int HALVES>
struct Queries {
    uint32_t f[D / 16][HALVES][2];  // B operand: rows g + 8 x, permuted as the keys' unpacking pairs channels
    // of rows 2t + y + 8 x, whose logits the lane holds:
    float sum[HALVES][2];          // the scaled row's sum, times 2^-24 and c's mantissa
    float unit[HALVES][2];         // what a product counts, in log2 units: a power of two
    int hi[HALVES][2], lo[HALVES][2];  // the tokens the row sees: lo .. hi (none: hi < lo)

    __device__ __forceinline__ void load(const KvAttnParams& p, const KvScale& scale, const KvSeq& seq, int h, int row0,
                                         int rows) {
        const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
        const int base = seq.len - seq.nq;
#pragma unroll
        for (int x = 0; x < HALVES; ++x) {
            const int r = g + 8 * x;
            const bool live = r < rows;
            const int i = (row0 + (live ? r : 0)) / p.G;
            const int head = h * p.G + (row0 + (live ? r : 0)) - i * p.G;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (seq.q0 + i) * p.q_stride + (int64_t)head * D +
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
            const int e = max((int)(top >> 23), 15) - 127;
            const float by = p.scale_log2 < 0.0f ? -pow2(14 - e) : pow2(14 - e);
            float total = 0.0f;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const float y[8] = {lo_bf16(v[w].x) * by, hi_bf16(v[w].x) * by, lo_bf16(v[w].y) * by,
                                    hi_bf16(v[w].y) * by, lo_bf16(v[w].z) * by, hi_bf16(v[w].z) * by,
                                    lo_bf16(v[w].w) * by, hi_bf16(v[w].w) * by};
                total += ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
                uint32_t (&f0)[2] = f[2 * w][x], (&f1)[2] = f[2 * w + 1][x];
                if constexpr (BITS == 4) {  // 8 channels: (0,4) (1,5) | (2,6) (3,7)
                    f0[0] = pack_f16(y[0], y[4]);
                    f0[1] = pack_f16(y[1] * 0.0625f, y[5] * 0.0625f);
                    f1[0] = pack_f16(y[2], y[6]);
                    f1[1] = pack_f16(y[3] * 0.0625f, y[7] * 0.0625f);
                } else {  // twice 4 channels: (0,1) (2,3)
                    f0[0] = pack_f16(y[0], y[1]);
                    f0[1] = pack_f16(y[2], y[3]);
                    f1[0] = pack_f16(y[4], y[5]);
                    f1[1] = pack_f16(y[6], y[7]);
                }
            }
            total += __shfl_xor_sync(0xffffffffu, total, 1);
            total += __shfl_xor_sync(0xffffffffu, total, 2);
            const float u = product_unit(scale, e);
            total *= 0x1p-24f * scale.mantissa;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int from = 4 * (2 * t + y);  // a lane that loaded row 2t + y
                sum[x][y] = __shfl_sync(0xffffffffu, total, from);
                unit[x][y] = __shfl_sync(0xffffffffu, u, from);
                const int j = __shfl_sync(0xffffffffu, i, from);
                const bool there = 8 * x + 2 * t + y < rows;
                hi[x][y] = there ? base + j : -1;
                lo[x][y] = p.window > 0 ? (int)max(base + j + 1 - p.window, (int64_t)0) : 0;
            }
        }
    }
};

// Query rows ready for the lanes, made once per block: a warp a row.
template <int D, int BITS, int ROWS>
struct SharedQueries {
    static constexpr int kChunks = D / 8;
    uint4 row[ROWS][kChunks + 1];  // (one more: banks)
    float sum[ROWS], unit[ROWS];
    int hi[ROWS], lo[ROWS];

    template <int WARPS>
    __device__ __forceinline__ void make(const KvAttnParams& p, const KvScale& scale, const KvSeq& seq, int h, int rows) {
        const int lane = threadIdx.x % 32;
#pragma unroll
        for (int r = threadIdx.x / 32; r < ROWS; r += WARPS) {
            const bool live = r < rows;
            const int i = live ? r / p.G : 0;
            const int head = h * p.G + (live ? r - i * p.G : 0);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (live && lane < kChunks)
                v = __ldg(reinterpret_cast<const uint4*>(p.q + (seq.q0 + i) * p.q_stride + (int64_t)head * D) + lane);
            const uint32_t words[4] = {v.x, v.y, v.z, v.w};
            uint32_t top = 0;  // largest finite magnitude, as bits
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a = words[j] & 0x7fff0000u, b = (words[j] << 16) & 0x7fff0000u;
                top = max(top, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
            }
            top = __reduce_max_sync(0xffffffffu, top);
            const int e = max((int)(top >> 23), 15) - 127;
            const float by = p.scale_log2 < 0.0f ? -pow2(14 - e) : pow2(14 - e);
            const float y[8] = {lo_bf16(v.x) * by, hi_bf16(v.x) * by, lo_bf16(v.y) * by, hi_bf16(v.y) * by,
                                lo_bf16(v.z) * by, hi_bf16(v.z) * by, lo_bf16(v.w) * by, hi_bf16(v.w) * by};
            float total = ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
            if (lane < kChunks) {
                row[r][lane] = BITS == 4 ? make_uint4(pack_f16(y[0], y[4]), pack_f16(y[1] * 0.0625f, y[5] * 0.0625f),
                                                      pack_f16(y[2], y[6]), pack_f16(y[3] * 0.0625f, y[7] * 0.0625f))
                                         : make_uint4(pack_f16(y[0], y[1]), pack_f16(y[2], y[3]), pack_f16(y[4], y[5]),
                                                      pack_f16(y[6], y[7]));
            }
            if (lane == 0) {
                sum[r] = total * (0x1p-24f * scale.mantissa);
                unit[r] = product_unit(scale, e);
                const int at = seq.len - seq.nq + i;
                hi[r] = live ? at : -1;
                lo[r] = p.window > 0 ? (int)max(at + 1 - p.window, (int64_t)0) : 0;
            }
        }
    }

    template <int HALVES>
    __device__ __forceinline__ void load(Queries<D, BITS, HALVES>& q) const {
        const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
#pragma unroll
        for (int x = 0; x < HALVES; ++x) {
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint4 v = row[g + 8 * x][t * (D / 32) + w];
                q.f[2 * w][x][0] = v.x;
                q.f[2 * w][x][1] = v.y;
                q.f[2 * w + 1][x][0] = v.z;
                q.f[2 * w + 1][x][1] = v.w;
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int r = 8 * x + 2 * t + y;
                q.sum[x][y] = sum[r];
                q.unit[x][y] = unit[r];
                q.hi[x][y] = hi[r];
                q.lo[x][y] = lo[r];
            }
        }
    }
};

// A warp's 32 tokens of a tile: token g + 8 i, a lane's quarter of each row.
template <int D, int BITS>
struct Keys {
    static constexpr int kWords = D * BITS / 128;
    uint32_t w[4][kWords];
    uint32_t param[4];

    // Logits, in units of their rows, of tokens g + 16 i (+ 8) and rows 2t, 2t + 1 (+ 8 x).
    // EDGE: some row does not see some token: -inf there.
    template <bool EDGE, int HALVES>
    __device__ __forceinline__ void logits(const Queries<D, BITS, HALVES>& q, float mantissa, int token,
                                           float (&s)[2][HALVES][4]) const {
        constexpr int kPairs = 16 / BITS;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < HALVES; ++x) s[i][x][0] = s[i][x][1] = s[i][x][2] = s[i][x][3] = 0.0f;
#pragma unroll
        for (int k = 0; k < kWords; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t a[kPairs], b[kPairs];
                kv_small_codes<BITS>(w[2 * i][k], a);
                kv_small_codes<BITS>(w[2 * i + 1][k], b);
#pragma unroll
                for (int j = 0; j < kPairs; j += 2)
#pragma unroll
                    for (int x = 0; x < HALVES; ++x) {
                        const uint32_t (&f)[2] = q.f[(k * kPairs + j) / 2][x];
                        mma_f16(s[i][x], a[j], b[j], a[j + 1], b[j + 1], f[0], f[1]);
                    }
            }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const float scale = kv_scale(param[2 * i + z]) * mantissa, low = kv_low(param[2 * i + z]);
                const uint64_t scale2 = pair_f32(scale, scale), low2 = pair_f32(low, low);
                const int j = token + 16 * i + 8 * z;
#pragma unroll
                for (int x = 0; x < HALVES; ++x) {
                    float* v = s[i][x] + 2 * z;
                    split_f32(fma_f32x2(scale2, pair_f32(v[0], v[1]), mul_f32x2(low2, pair_f32(q.sum[x][0], q.sum[x][1]))),
                              v[0], v[1]);
                    if (EDGE) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) v[y] = j >= q.lo[x][y] && j <= q.hi[x][y] ? v[y] : -INFINITY;
                    }
                }
            }
    }
};

// A warp's tokens on their way: a ring of STAGES steps of 32 tokens, WARPS * 32 tokens
// (the block's tile) apart, each lane copying (cp.async) what it will itself unpack, and one token's scale
// and low value, so that no barrier beyond the warp is needed and no register waits
// for memory.  Pages are looked up a step before they are copied from.
template <int D, int BITS, int WARPS, int STAGES>
struct KeyRing {
    static constexpr int kRow = D * BITS / 8;
    static constexpr int kLaneBytes = kRow / 4;
    static constexpr int kStageBytes = 32 * 4 * kLaneBytes + 32 * 4;
    static constexpr int kBytes = WARPS * STAGES * kStageBytes;

    const KvAttnParams& p;
    const int32_t* table;
    uint8_t* mine;          // this warp's part
    const uint8_t* codes;   // this lane's part of page 0's first rows of the head, and its parameter
    const uint32_t* params;
    int begin, end;
    int next, last;  // the warp's next step's first token; tokens from `last` on are not wanted
    int page[2];     // of the next step (of its second 16 tokens, where pages have 16)
    int put, get;    // stages
    uint32_t page_rows;

    __device__ __forceinline__ void look_up() {
        if (next >= last) return;
        // (the first tokens may lie before `begin`, in a page that may be anything, or all of
        // them behind `end`)
        const int32_t* at = table + (next >> p.cache.page_shift);
        page[0] = next < end ? __ldg(at) : -1;
        if (p.cache.page_shift == 4) page[1] = next + 16 < end ? __ldg(at + 1) : -1;
    }

    // Tiles t0 .. t1 - 1; tokens outside begin .. end come as zeros.
    __device__ __forceinline__ KeyRing(const KvAttnParams& p, const int32_t* table, uint8_t* ring, int h, int t0, int t1,
                                       int begin, int end)
        : p(p), table(table), begin(begin), end(end), put(0), get(0) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        mine = ring + warp * (STAGES * kStageBytes);
        const int64_t row = (int64_t)h << p.cache.page_shift;
        codes = p.cache.codes + (row + lane / 4) * kRow + lane % 4 * kLaneBytes;
        params = p.cache.params + row + lane % 16;
        next = t0 * (WARPS * 32) + warp * 32;
        last = t1 * (WARPS * 32);
        page_rows = (uint32_t)(2 * p.cache.H) << p.cache.page_shift;  // < 2^25
        look_up();
#pragma unroll 1
        for (int i = 0; i < max(STAGES - 1, 1); ++i) issue();
    }

    static constexpr int kCopy = kLaneBytes < 16 ? kLaneBytes : 16;
    __device__ __forceinline__ static void copy(uint32_t dst, const void* src) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kCopy) : "memory");
    }
    __device__ __forceinline__ static void copy(uint32_t dst, const void* src, bool there) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kCopy), "r"(there ? kCopy : 0)
                     : "memory");
    }

    // A step whose tokens lie in one page and are all wanted: addresses are constants apart.
    __device__ __forceinline__ void issue_whole(uint32_t stage) {
        const int lane = threadIdx.x % 32;
        const uint32_t off = (uint32_t)next & ((1u << p.cache.page_shift) - 1u);
        const uint64_t row = (uint64_t)(uint32_t)page[0] * page_rows + off;
        const uint8_t* src = codes + row * kRow;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kLaneBytes == 32) {
                // (16 bytes of all lanes, then the other 16: banks)
                copy(stage + i * 32 * kLaneBytes + lane * 16, src + i * (8 * kRow));
                copy(stage + i * 32 * kLaneBytes + lane * 16 + 512, src + i * (8 * kRow) + 16);
            } else {
                copy(stage + (i * 32 + lane) * kLaneBytes, src + i * (8 * kRow));
            }
        }
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(stage + 128 * kLaneBytes + lane * 4),
                     "l"(params + row + (lane & 16))
                     : "memory");
    }

    // Any step: tokens that are not wanted come as zeros (and nothing is read for them).
    // (Rare, so a function; of values, so that the ring stays in registers.)
    static __device__ __noinline__ void issue_parts(const uint8_t* codes, const uint32_t* params, int64_t pages,
                                                    int page_shift, uint32_t page_rows, int page0, int page1, int next,
                                                    int begin, int end, uint32_t stage, unsigned* err) {
        const int lane = threadIdx.x % 32, g = lane / 4;
        const int mask = (1 << page_shift) - 1;
        int64_t at[2];  // rows from page 0's
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int token = next + 16 * i;
            int64_t from = i == 0 || page_shift > 4 ? page0 : page1;
            if (from < 0 || from >= pages) {
                if (token < end && token + 16 > begin) record_fault(err, kErrBitBadIndex);
                from = 0;
            }
            at[i] = from * page_rows + (token & mask);
        }
        auto wanted = [&](int token) { return token >= begin && token < end; };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t* src = codes + at[i / 2] * kRow + (i % 2) * (8 * kRow);
            const bool there = wanted(next + 8 * i + g);
            if constexpr (kLaneBytes == 32) {
                copy(stage + i * 32 * kLaneBytes + lane * 16, src, there);
                copy(stage + i * 32 * kLaneBytes + lane * 16 + 512, src + 16, there);
            } else {
                copy(stage + (i * 32 + lane) * kLaneBytes, src, there);
            }
        }
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(stage + 128 * kLaneBytes + lane * 4),
                     "l"(params + (lane < 16 ? at[0] : at[1])), "r"(wanted(next + lane) ? 4 : 0)
                     : "memory");
    }

    __device__ __forceinline__ void issue() {
        if (next < last) {
            const uint32_t stage = tc::smem_u32(mine) + put * kStageBytes;
            if (next >= begin && next + 32 <= end && p.cache.page_shift > 4 && (uint32_t)page[0] < (uint32_t)p.cache.pages)
                issue_whole(stage);
            else
                issue_parts(codes, params, p.cache.pages, p.cache.page_shift, page_rows, page[0], page[1], next, begin, end,
                            stage, p.err);
            next += WARPS * 32;
            look_up();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put + 1 == STAGES ? 0 : put + 1;
    }

    // The oldest step; the next one goes on its way.
    __device__ __forceinline__ void take(Keys<D, BITS>& k) {
        constexpr int kWords = Keys<D, BITS>::kWords;
        const int lane = threadIdx.x % 32, g = lane / 4;
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES > 1 ? STAGES - 2 : 0) : "memory");
        __syncwarp();  // the other lanes' scales; and all lanes are done with the step before
        if (STAGES > 1) issue();
        const uint8_t* stage = mine + get * kStageBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kLaneBytes == 32) {
                uint32_t a[4], b[4];
                lds<4>(stage + i * 32 * kLaneBytes + lane * 16, a);
                lds<4>(stage + i * 32 * kLaneBytes + lane * 16 + 512, b);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    k.w[i][j] = a[j];
                    k.w[i][4 + j] = b[j];
                }
            } else {
                lds<kWords>(stage + (i * 32 + lane) * kLaneBytes, k.w[i]);
            }
            k.param[i] = *reinterpret_cast<const uint32_t*>(stage + 128 * kLaneBytes + (g + 8 * i) * 4);
        }
        get = get + 1 == STAGES ? 0 : get + 1;
        if (STAGES == 1) {  // (what has been taken is in registers)
            __syncwarp();
            issue();
        }
    }
};

// 2^(a - m), 0 where a is -inf (and m too).
__device__ __forceinline__ float weight_of(float a, float m) { return exp2_approx(a - (m == -INFINITY ? 0.0f : m)); }

// (m, l) over two sets of tokens.
__device__ __forceinline__ void join_stats(float& m, float& l, float om, float ol) {
    const float to = fmaxf(m, om);
    l = l * weight_of(m, to) + ol * weight_of(om, to);
    m = to;
}

// Adds a step's logits to a lane's (m, l).  m is what l is relative to; it is raised where a
// logit exceeds it by more than the slack (rare).  It begins at kNothing, finite, so that
// what is not seen (-inf) has weight 0 beside it.
constexpr float kNothing = -3.402823466e38f;
constexpr float kSlack = 8.0f;
template <int D, int BITS, int HALVES>
__device__ __forceinline__ void add_logits(float (&m)[HALVES][2], float (&l)[HALVES][2], const float (&s)[2][HALVES][4],
                                           const Queries<D, BITS, HALVES>& q) {
    float top[HALVES][2];
    bool over = false;
#pragma unroll
    for (int x = 0; x < HALVES; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            top[x][y] = fmaxf(max3(s[0][x][y], s[0][x][2 + y], s[1][x][y]), s[1][x][2 + y]) * q.unit[x][y];
            over = over || top[x][y] > m[x][y] + kSlack;
        }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int x = 0; x < HALVES; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
                if (top[x][y] > m[x][y] + kSlack) {
                    l[x][y] *= exp2_approx(m[x][y] - top[x][y]);
                    m[x][y] = top[x][y];
                }
    }
#pragma unroll
    for (int x = 0; x < HALVES; ++x) {
        const uint64_t u = pair_f32(q.unit[x][0], q.unit[x][1]), to = pair_f32(-m[x][0], -m[x][1]);
        auto weights = [&](const float* v) {
            float a, b;
            split_f32(fma_f32x2(pair_f32(v[0], v[1]), u, to), a, b);
            return pair_f32(exp2_approx(a), exp2_approx(b));
        };
        const uint64_t sum = add_f32x2(add_f32x2(weights(s[0][x]), weights(s[0][x] + 2)),
                                       add_f32x2(weights(s[1][x]), weights(s[1][x] + 2)));
        split_f32(add_f32x2(pair_f32(l[x][0], l[x][1]), sum), l[x][0], l[x][1]);
    }
}

// The lanes' (m, l) of a warp, into part[row].
template <int HALVES>
__device__ __forceinline__ void warp_stats(float (&m)[HALVES][2], float (&l)[HALVES][2], float2* part) {
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
#pragma unroll
    for (int x = 0; x < HALVES; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
                join_stats(m[x][y], l[x][y], __shfl_xor_sync(0xffffffffu, m[x][y], d),
                           __shfl_xor_sync(0xffffffffu, l[x][y], d));
            if (g == 0) part[8 * x + 2 * t + y] = make_float2(m[x][y], l[x][y]);
        }
}

// Sums of four neighbours, tokens j .. j + 3 at place `to`, of which those of begin .. end - 1
// are written, and those before `older` added to what they had.
__device__ __forceinline__ void store_weights(const KvWeightsParams& p, int64_t to, int j, int begin, int end, int older,
                                              const float (&sum)[4]) {
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < older) w = *reinterpret_cast<const float4*>(p.previous + to);
    const float before[4] = {w.x, w.y, w.z, w.w};
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = (j + k < older ? before[k] : 0.0f) + sum[k];
    if (j >= begin && j + 4 <= end) {
        *reinterpret_cast<float4*>(p.weights + to) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (j + k >= begin && j + k < end) p.weights[to + k] = v[k];
    }
}

// All in one, while a cluster's shared memory holds the logits: a cluster takes one
// cache head of one sequence, each CTA a part of its tiles.  Keys are read once:
// logits stay in shared memory, the CTAs exchange each row's (m, l), and the
// weights are summed from there.
template <int D, int BITS, int HALVES>
__global__ void __launch_bounds__(kOneThreads, HALVES == 1 ? 4 : HALVES == 2 ? 2 : 1) kv_weigh_kernel(const KvWeightsParams p) {
    constexpr int ROWS = 8 * HALVES;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[kOneWarps][ROWS];      // a warp's maxima, then its sums
    __shared__ SharedQueries<D, BITS, ROWS> queries;
    __shared__ __align__(16) float2 mine[ROWS];  // this CTA's (m, l)
    __shared__ __align__(8) float factors[ROWS]; // of this CTA's weights: 2^(its m - m) / l
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int size = p.splits, rank = (int)tc::cluster_rank();
    const uint32_t item = blockIdx.x / (uint32_t)size;
    const uint32_t b = item / (uint32_t)p.a.cache.H;
    const int h = (int)(item - b * (uint32_t)p.a.cache.H);
    pdl_wait();
    const KvSeq seq = weights_sequence(p, b);
    if (seq.nq == 0) return;  // (the whole cluster)
    // what the rows see: tokens begin .. end - 1, and each of them all_lo .. all_hi
    const int base = seq.len - seq.nq, rows = min(ROWS, seq.nq * p.a.G);
    const int begin = p.a.window > 0 ? (int)min(max(base + 1 - p.a.window, (int64_t)0), (int64_t)seq.len) : 0, end = seq.len;
    const int all_lo = p.a.window > 0 ? (int)max(seq.len - p.a.window, (int64_t)0) : 0, all_hi = base;
    const int first_tile = begin / kOneTile, tiles = (end + kOneTile - 1) / kOneTile - first_tile;
    const int tile0 = first_tile + tiles * rank / size, tile1 = first_tile + tiles * (rank + 1) / size;
    const int32_t* table = p.a.table + b * p.a.table_width;
    // [pairs of rows][tokens]; 8 more tokens keep a warp's stores off each other's banks
    float2* logits = reinterpret_cast<float2*>(smem + KeyRing<D, BITS, kOneWarps, kOneStages>::kBytes);
    const int stride = p.chunk * kOneTile + 8, tokens = (tile1 - tile0) * kOneTile;
    // the products
    {
        float top[HALVES][2];
#pragma unroll
        for (int x = 0; x < HALVES; ++x) top[x][0] = top[x][1] = -INFINITY;
        KeyRing<D, BITS, kOneWarps, kOneStages> ring(p.a, table, smem, h, tile0, tile1, begin, end);
        queries.template make<kOneWarps>(p.a, p.scale, seq, h, rows);
        __syncthreads();
        Queries<D, BITS, HALVES> q;
        queries.load(q);
        int token = tile0 * kOneTile + warp * 32 + g;
        float2* to = logits + t * stride + warp * 32 + g;
        auto step = [&](auto edge) {
            Keys<D, BITS> now;
            ring.take(now);
            float s[2][HALVES][4];
            now.template logits<decltype(edge)::value>(q, p.scale.mantissa, token, s);
#pragma unroll
            for (int x = 0; x < HALVES; ++x) {
                if (8 * x + 2 * t < rows) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        to[4 * x * stride + 8 * k] = make_float2(s[k / 2][x][2 * (k % 2)], s[k / 2][x][2 * (k % 2) + 1]);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    top[x][y] = max3(top[x][y], s[0][x][y], s[0][x][2 + y]);
                    top[x][y] = max3(top[x][y], s[1][x][y], s[1][x][2 + y]);
                }
            }
        };
#pragma unroll 1
        for (int i = tile0; i < tile1; ++i, token += kOneTile, to += kOneTile) {
            const int first = i * kOneTile;
            if (first >= all_lo && first + kOneTile - 1 <= all_hi)
                step(std::false_type{});
            else
                step(std::true_type{});
        }
#pragma unroll
        for (int x = 0; x < HALVES; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) top[x][y] = fmaxf(top[x][y], __shfl_xor_sync(0xffffffffu, top[x][y], d));
                if (g == 0) part[warp][8 * x + 2 * t + y] = top[x][y];
            }
    }
    __syncthreads();
    // weights relative to this CTA's maxima, and their sums; a pair of rows at a time
    if (threadIdx.x < ROWS) {
        float m = part[0][threadIdx.x];
        for (int w = 1; w < kOneWarps; ++w) m = fmaxf(m, part[w][threadIdx.x]);
        m = threadIdx.x < rows ? m * queries.unit[threadIdx.x] : 0.0f;
        mine[threadIdx.x].x = m;
    }
    __syncthreads();
    for (int r = 0; 2 * r < rows; ++r) {
        const float u0 = queries.unit[2 * r], u1 = queries.unit[2 * r + 1];
        const float m0 = mine[2 * r].x == -INFINITY ? 0.0f : -mine[2 * r].x;
        const float m1 = mine[2 * r + 1].x == -INFINITY ? 0.0f : -mine[2 * r + 1].x;
        const uint64_t u = pair_f32(u0, u1), to = pair_f32(m0, m1);
        uint64_t l = pair_f32(0.0f, 0.0f);
        float4* a = reinterpret_cast<float4*>(logits + r * stride);  // two tokens at a time
#pragma unroll 4
        for (int i = threadIdx.x; i < tokens / 2; i += kOneThreads) {
            const float4 v = a[i];
            float4 e;
            split_f32(fma_f32x2(pair_f32(v.x, v.y), u, to), e.x, e.y);
            split_f32(fma_f32x2(pair_f32(v.z, v.w), u, to), e.z, e.w);
            e = make_float4(exp2_approx(e.x), exp2_approx(e.y), exp2_approx(e.z), exp2_approx(e.w));
            a[i] = e;
            l = add_f32x2(l, add_f32x2(pair_f32(e.x, e.y), pair_f32(e.z, e.w)));
        }
        float l0, l1;
        split_f32(l, l0, l1);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, d);
            l1 += __shfl_xor_sync(0xffffffffu, l1, d);
        }
        if (lane == 0) {
            part[warp][2 * r] = l0;
            part[warp][2 * r + 1] = l1;
        }
    }
    __syncthreads();
    if (threadIdx.x < rows) {
        float l = 0.0f;
        for (int w = 0; w < kOneWarps; ++w) l += part[w][threadIdx.x];
        mine[threadIdx.x].y = l;
    }
    tc::cluster_sync_all();
    if (threadIdx.x < ROWS) {
        float rm = -INFINITY, rl = 0.0f;
        if (threadIdx.x < rows)
            for (int c = 0; c < size; ++c) {
                float om, ol;
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                             : "=f"(om), "=f"(ol)
                             : "r"(tc::mapa(tc::smem_u32(&mine[threadIdx.x]), c))
                             : "memory");
                join_stats(rm, rl, om, ol);
            }
        factors[threadIdx.x] = rl > 0.0f ? weight_of(mine[threadIdx.x].x, rm) / rl : 0.0f;
    }
    __syncthreads();
    // (no CTA leaves while another reads its part)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    // four tokens a thread at a time, which lie in one page
    const int mask = (1 << p.a.cache.page_shift) - 1, older = p.previous != nullptr ? seq.len - seq.nq : 0;
    for (int i = threadIdx.x * 4; i < tokens; i += 4 * kOneThreads) {
        const int j = tile0 * kOneTile + i;
        if (j + 4 <= begin || j >= end) continue;
        const int64_t page = kv_page(p.a.cache, table, j >> p.a.cache.page_shift, p.a.err);
        if (page < 0) continue;
        const int64_t to = kv_weight(p.a.cache, page, h, j & mask);
        uint64_t sum[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = pair_f32(0.0f, 0.0f);
        for (int r = 0; 2 * r < rows; ++r) {
            const float4 a = *reinterpret_cast<const float4*>(logits + r * stride + i);
            const float4 c = *reinterpret_cast<const float4*>(logits + r * stride + i + 2);
            const uint64_t f = *reinterpret_cast<const uint64_t*>(factors + 2 * r);
            sum[0] = fma_f32x2(pair_f32(a.x, a.y), f, sum[0]);
            sum[1] = fma_f32x2(pair_f32(a.z, a.w), f, sum[1]);
            sum[2] = fma_f32x2(pair_f32(c.x, c.y), f, sum[2]);
            sum[3] = fma_f32x2(pair_f32(c.z, c.w), f, sum[3]);
        }
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float even, odd;
            split_f32(sum[k], even, odd);
            v[k] = even + odd;
        }
        store_weights(p, to, j, begin, end, older, v);
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The tokens that all of a block's rows see.
struct Edges {
    int lo, hi;
    __device__ __forceinline__ Edges(const KvAttnParams& p, const KvSeq& seq, int row0, int rows) {
        const int base = seq.len - seq.nq;
        hi = base + row0 / p.G;
        lo = p.window > 0 ? (int)max(base + (row0 + rows - 1) / p.G + 1 - p.window, (int64_t)0) : 0;
    }
    // Whether they are a warp's 32 from `token` on.
    __device__ __forceinline__ bool whole(int token) const { return token >= lo && token + 31 <= hi; }
};

// (m, l) over a part of the tokens, for a block of rows.
template <int D, int BITS, int HALVES>
__global__ void __launch_bounds__(kThreads) kv_stats_kernel(const KvWeightsParams p) {
    constexpr int ROWS = 8 * HALVES;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 part[kWarps][ROWS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4;
    // split fastest, then head, so that neighbours share rows and pages
    int64_t at = blockIdx.x;
    const int split = (int)(at % p.splits);
    at /= p.splits;
    const int h = (int)(at % p.a.cache.H);
    at /= p.a.cache.H;
    const int64_t blocks = (p.max_q * p.a.G + ROWS - 1) / ROWS;
    const int rb = (int)(at % blocks);
    const int64_t b = at / blocks;
    pdl_wait();
    const KvSeq seq = weights_sequence(p, b);
    if (rb >= kv_blocks<ROWS>(p.a, seq)) return;
    const KvSpan span = kv_span<ROWS, kTile>(p.a, seq, rb);
    const int row0 = rb * ROWS, rows = min(ROWS, seq.nq * p.a.G - row0);
    const int first = (int)((int64_t)span.tiles * split / p.splits), last = (int)((int64_t)span.tiles * (split + 1) / p.splits);
    float m[HALVES][2], l[HALVES][2];
#pragma unroll
    for (int x = 0; x < HALVES; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            m[x][y] = kNothing;
            l[x][y] = 0.0f;
        }
    if (first < last) {
        const int32_t* table = p.a.table + b * p.a.table_width;
        KeyRing<D, BITS, kWarps, kStages<D, BITS>> ring(p.a, table, smem, h, span.first + first, span.first + last, span.begin,
                                                          span.end);
        Queries<D, BITS, HALVES> q;
        q.load(p.a, p.scale, seq, h, row0, rows);
        int token = (span.first + first) * kTile + warp * 32 + g;
        const Edges edges(p.a, seq, row0, rows);
        auto step = [&](auto edge) {
            Keys<D, BITS> now;
            ring.take(now);
            float s[2][HALVES][4];
            now.template logits<decltype(edge)::value>(q, p.scale.mantissa, token, s);
            add_logits<D, BITS, HALVES>(m, l, s, q);
        };
        for (int i = first; i < last; ++i, token += kTile) {
            if (edges.whole(token - g))
                step(std::false_type{});
            else
                step(std::true_type{});
        }
#pragma unroll
        for (int x = 0; x < HALVES; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) m[x][y] = m[x][y] == kNothing ? -INFINITY : m[x][y];
    } else {
#pragma unroll
        for (int x = 0; x < HALVES; ++x) m[x][0] = m[x][1] = -INFINITY;
    }
    warp_stats<HALVES>(m, l, part[warp]);
    __syncthreads();
    if (threadIdx.x < rows) {
        float2 r = part[0][threadIdx.x];
        for (int w = 1; w < kWarps; ++w) join_stats(r.x, r.y, part[w][threadIdx.x].x, part[w][threadIdx.x].y);
        const int i = (row0 + threadIdx.x) / p.a.G;
        const int64_t row = (seq.q0 + i) * ((int64_t)p.a.G * p.a.cache.H) + h * p.a.G + row0 + threadIdx.x - i * p.a.G;
        p.stats[row * p.splits + split] = r;
    }
}

// The weights of a chunk of tiles, summed over all rows.
template <int D, int BITS, int HALVES>
__global__ void __launch_bounds__(kThreads) kv_sum_kernel(const KvWeightsParams p) {
    constexpr int ROWS = 8 * HALVES;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float sums[kChunk * kTile];
    __shared__ float2 stats[ROWS];  // (m, 1 / l)
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int64_t tiles_all = ((p.a.table_width << p.a.cache.page_shift) + kTile - 1) / kTile;
    const int64_t chunks = (tiles_all + p.chunk - 1) / p.chunk;
    int64_t at = blockIdx.x;
    const int tile0 = (int)(at % chunks) * p.chunk;
    at /= chunks;
    const int h = (int)(at % p.a.cache.H);
    const int64_t b = at / p.a.cache.H;
    pdl_wait();
    const KvSeq seq = weights_sequence(p, b);
    // Tokens that no row sees are left alone: their pages may be another sequence's by now.
    if (seq.nq == 0) return;
    const int begin = kv_span<ROWS, kTile>(p.a, seq, 0).begin;
    const int tiles = min(p.chunk, (seq.len + kTile - 1) / kTile - tile0);
    if (tiles <= 0 || (tile0 + tiles) * kTile <= begin) return;
    const int32_t* table = p.a.table + b * p.a.table_width;
    for (int i = threadIdx.x; i < tiles * kTile; i += kThreads) sums[i] = 0.0f;
    const int blocks = kv_blocks<ROWS>(p.a, seq);
    for (int rb = 0; rb < blocks; ++rb) {
        const KvSpan span = kv_span<ROWS, kTile>(p.a, seq, rb);
        const int first = max(span.first, tile0), last = min((span.end + kTile - 1) / kTile, tile0 + tiles);
        if (first >= last) continue;  // (the same for the whole block)
        const int row0 = rb * ROWS, rows = min(ROWS, seq.nq * p.a.G - row0);
        // keys, rows and their statistics wait together
        KeyRing<D, BITS, kWarps, kStages<D, BITS>> ring(p.a, table, smem, h, first, last, span.begin, span.end);
        Queries<D, BITS, HALVES> q;
        q.load(p.a, p.scale, seq, h, row0, rows);
        __syncthreads();
        {  // several lanes a row
            constexpr int kLanes = kThreads / ROWS;
            const int r = threadIdx.x / kLanes;
            float m = -INFINITY, l = 0.0f;
            if (r < rows) {
                const int i = (row0 + r) / p.a.G;
                const int64_t row = (seq.q0 + i) * ((int64_t)p.a.G * p.a.cache.H) + h * p.a.G + row0 + r - i * p.a.G;
                for (int s = threadIdx.x % kLanes; s < p.splits; s += kLanes) {
                    const float2 x = p.stats[row * p.splits + s];
                    join_stats(m, l, x.x, x.y);
                }
            }
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1)
                join_stats(m, l, __shfl_xor_sync(0xffffffffu, m, d), __shfl_xor_sync(0xffffffffu, l, d));
            if (threadIdx.x % kLanes == 0) stats[r] = make_float2(m == -INFINITY ? 0.0f : m, l > 0.0f ? 1.0f / l : 0.0f);
        }
        __syncthreads();
        uint64_t minus_m[HALVES], factor[HALVES];
#pragma unroll
        for (int x = 0; x < HALVES; ++x) {
            const float2 even = stats[8 * x + 2 * t], odd = stats[8 * x + 2 * t + 1];
            minus_m[x] = pair_f32(-even.x, -odd.x);
            factor[x] = pair_f32(even.y, odd.y);
        }
        int token = first * kTile + warp * 32 + g;
        const Edges edges(p.a, seq, row0, rows);
        float* to = sums + (first - tile0) * kTile + warp * 32 + g;
        auto step = [&](auto edge) {
            Keys<D, BITS> now;
            ring.take(now);
            float s[2][HALVES][4];
            now.template logits<decltype(edge)::value>(q, p.scale.mantissa, token, s);
            float sum[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint64_t both = pair_f32(0.0f, 0.0f);
#pragma unroll
                for (int x = 0; x < HALVES; ++x) {
                    const float* v = s[k / 2][x] + 2 * (k % 2);
                    float a, b;
                    split_f32(fma_f32x2(pair_f32(v[0], v[1]), pair_f32(q.unit[x][0], q.unit[x][1]), minus_m[x]), a, b);
                    both = fma_f32x2(pair_f32(exp2_approx(a), exp2_approx(b)), factor[x], both);
                }
                float a, b;
                split_f32(both, a, b);
                sum[k] = a + b;
            }
            // over the four lanes of a token: each ends with one of its four tokens
            const bool odd = t & 1, high = t & 2;
            float a = odd ? sum[0] : sum[1], b = odd ? sum[2] : sum[3];
            a = (odd ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, a, 1);
            b = (odd ? sum[3] : sum[2]) + __shfl_xor_sync(0xffffffffu, b, 1);
            const float c = __shfl_xor_sync(0xffffffffu, high ? a : b, 2);
            to[8 * t] += (high ? b : a) + c;
        };
        for (int i = first; i < last; ++i, token += kTile, to += kTile) {
            if (edges.whole(token - g))
                step(std::false_type{});
            else
                step(std::true_type{});
        }
    }
    __syncthreads();
    // four tokens a thread at a time, which lie in one page
    const int older = p.previous != nullptr ? seq.len - seq.nq : 0, mask = (1 << p.a.cache.page_shift) - 1;
#pragma unroll 2
    for (int i = threadIdx.x * 4; i < tiles * kTile; i += 4 * kThreads) {
        const int j = tile0 * kTile + i;
        if (j + 4 <= begin || j >= seq.len) continue;
        const int64_t page = kv_page(p.a.cache, table, j >> p.a.cache.page_shift, p.a.err);
        if (page < 0) continue;
        const float4 sum = *reinterpret_cast<const float4*>(sums + i);
        const float v[4] = {sum.x, sum.y, sum.z, sum.w};
        store_weights(p, kv_weight(p.a.cache, page, h, j & mask), j, begin, seq.len, older, v);
    }
}

struct WeightsPlan {
    int halves, splits, chunk;
    bool fused;  // one launch of clusters of `splits` CTAs, of `chunk` tiles at most each
    int64_t stats_blocks, sum_blocks;
    size_t smem;  // of the logits
};

// Shared memory of the logits up to which four blocks run on an SM, and two: with fewer the
// two kernels are quicker.
constexpr size_t kFewLogits = 36 * 1024;
constexpr size_t kMostLogits = 72 * 1024;

WeightsPlan weights_plan(int64_t B, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int sms) {
    WeightsPlan w = {};
    const int64_t rows = max_q * G;
    w.halves = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    const int64_t blocks = (rows + 8 * w.halves - 1) / (8 * w.halves), tiles = (max_kv + kTile - 1) / kTile;
    const int64_t base = std::max<int64_t>(B * H * blocks, 1);
    const int64_t one_tiles = (max_kv + kOneTile - 1) / kOneTile;
    // One launch: 96 sequences of 16384 tokens (4 bits, 8 x 128, four queries a head) 248 us
    // with 8 CTAs a cluster and 277 with 4; 48 of 32768, twice the logits a CTA, 288, and 342
    // by the two kernels for as many tokens.  With 16 rows two blocks run on an SM all the same: 64 of up to
    // 4096 in 73 us with 4 CTAs, 126 with 8; 16 of 4000 in 29, and 39 by the two kernels.  With 32 rows one does:
    // only where there is no more.  Beginning a block costs more than an SM gains by a fourth:
    // 24 of 4096 (8 rows, 8 bits) 46 us with 2 CTAs and 52 with 4, 16 of 1000 7.6 and 9.6.
    for (int64_t size = 1; size <= 8 && blocks == 1; size *= 2) {
        const int64_t chunk = (one_tiles + size - 1) / size;
        const size_t smem = (size_t)((rows + 1) / 2) * (size_t)(chunk * kOneTile + 8) * sizeof(float2);
        if (smem > (size < 8 && w.halves == 1 ? kFewLogits : kMostLogits)) continue;
        if (size < 8 && 2 * base * size < 3 * (int64_t)sms && size < one_tiles) continue;
        if (w.halves == 4 && base * size > 2 * sms) break;
        w.fused = true;
        w.splits = (int)size;
        w.chunk = (int)chunk;
        w.smem = smem;
        w.stats_blocks = w.sum_blocks = base * size;
        return w;
    }
    // (two chunks of 16 tokens over 8192, 64 rows a head: 20 and 29 us with three blocks an SM in
    // each kernel, 29 and 50 with eight; 16 of 16384 with 32 rows 73 + 95 and 89 + 105.  The
    // first kernel with up to 8 rows, five blocks of which run on an SM: 8 of 131072 tokens 100
    // us with eight blocks, 112 with three)
    const int64_t wanted = 3 * (int64_t)sms, wanted_stats = (w.halves == 1 ? 8 : 3) * (int64_t)sms;
    w.splits = (int)std::min<int64_t>(std::min<int64_t>(64, tiles), std::max<int64_t>(1, (wanted_stats + base - 1) / base));
    w.chunk = (int)std::min<int64_t>(kChunk, std::max<int64_t>(1, B * H * tiles / wanted));
    w.stats_blocks = B * H * blocks * w.splits;
    w.sum_blocks = B * H * ((tiles + w.chunk - 1) / w.chunk);
    return w;
}

template <int D, int BITS, int HALVES>
cudaError_t launch_form(const KvWeightsParams& p, const WeightsPlan& w, const LaunchEnv& env) {
    constexpr int kRing = KeyRing<D, BITS, kWarps, kStages<D, BITS>>::kBytes;
    if (w.fused) {
        constexpr int kOneRing = KeyRing<D, BITS, kOneWarps, kOneStages>::kBytes;
        const cudaError_t e = allow_smem<kv_weigh_kernel<D, BITS, HALVES>>(kOneRing + kMostLogits);
        if (e != cudaSuccess) return e;
        return launch_kernel(kv_weigh_kernel<D, BITS, HALVES>, dim3((unsigned)w.stats_blocks), dim3(kOneThreads),
                             kOneRing + w.smem, env.stream, dim3(w.splits, 1, 1), p);
    }
    cudaError_t e = allow_smem<kv_stats_kernel<D, BITS, HALVES>>(kRing);
    if (e == cudaSuccess) e = allow_smem<kv_sum_kernel<D, BITS, HALVES>>(kRing);
    if (e == cudaSuccess)
        e = launch_kernel(kv_stats_kernel<D, BITS, HALVES>, dim3((unsigned)w.stats_blocks), dim3(kThreads), kRing,
                          env.stream, kNoCluster, p);
    if (e != cudaSuccess) return e;
    return launch_kernel(kv_sum_kernel<D, BITS, HALVES>, dim3((unsigned)w.sum_blocks), dim3(kThreads), kRing, env.stream,
                         kNoCluster, p);
}

template <int D, int BITS>
cudaError_t launch_rows(const KvWeightsParams& p, const WeightsPlan& w, const LaunchEnv& env) {
    return w.halves == 1   ? launch_form<D, BITS, 1>(p, w, env)
           : w.halves == 2 ? launch_form<D, BITS, 2>(p, w, env)
                           : launch_form<D, BITS, 4>(p, w, env);
}

}  // namespace

size_t kv_weights_workspace(int64_t B, int64_t T_q, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int sms) {
    if (max_q * G > kKvWeightsFewRows) return kv_weights_many_workspace(B, T_q, G, H, max_kv, max_q, sms);
    const WeightsPlan w = weights_plan(B, G, H, max_kv, max_q, sms);
    return w.fused ? 0 : (size_t)(T_q * G * H) * (size_t)w.splits * sizeof(float2);
}

bool kv_weights_fits(int64_t B, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int sms) {
    if (max_q * G > kKvWeightsFewRows) return kv_weights_many_fits(B, G, H, max_kv, max_q, sms);
    const WeightsPlan w = weights_plan(B, G, H, max_kv, max_q, sms);
    return w.stats_blocks < kMaxRows && w.sum_blocks < kMaxRows;
}

cudaError_t launch_kv_weights(KvWeightsParams p, int64_t D, int64_t bits, void* workspace, const LaunchEnv& env) {
    if (p.max_q * p.a.G > kKvWeightsFewRows) return launch_kv_weights_many(p, D, bits, workspace, env);
    const WeightsPlan w =
        weights_plan(p.a.B, p.a.G, p.a.cache.H, p.a.table_width << p.a.cache.page_shift, p.max_q, env.sm_count);
    p.stats = static_cast<float2*>(workspace);
    p.splits = w.splits;
    p.chunk = w.chunk;
    // (1 <= mantissa < 2; a scale of 0: 0)
    p.scale.mantissa = 2.0f * std::frexp(std::fabs(p.a.scale_log2), &p.scale.exponent);
    --p.scale.exponent;
    if (D == 64) return bits == 4 ? launch_rows<64, 4>(p, w, env) : launch_rows<64, 8>(p, w, env);
    return bits == 4 ? launch_rows<128, 4>(p, w, env) : launch_rows<128, 8>(p, w, env);
}

}  // namespace i8ql
