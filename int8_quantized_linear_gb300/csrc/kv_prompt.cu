// Attention over the quantized key/value cache for many query rows (prompt
// chunks): the same result as kv_attention.cu on the tensor cores proper
// (tcgen05, accumulators in TMEM).
//
// A block (one per SM) holds 256 query rows of one cache head (query tokens x
// the head group's heads) as two M = 128 tiles, and walks the cache in tiles
// of 128 tokens:
//   S = Q K^T  (128 x 128, TMEM),  P = 2^(c S - m + 7) (fp16, back into S's
//   columns),  O += P V  (128 x D, TMEM; P is the A operand from TMEM)
// Bound by tensor throughput on paper (4 D flops a visible pair), in practice
// by instruction issue: unpacking a tile costs as many instructions as the
// softmax of 128 rows, which is why two M tiles share each unpacked tile.
//
// Roles: warps 0-3 and 4-7 the softmax of the two tiles (a thread a row: no
// shuffles), warps 8-11 unpack codes into the swizzled operand tiles, warp 12
// copies pages, warp 13 issues the MMAs.  While one tile's softmax runs, the
// tensor cores work on the other's products.  Four kinds of warp share one
// instruction cache, so the loops are kept rolled: unrolling the softmax over
// the row and the unpacking over the tile cost 20 % (650 against 541 us, when that
// was done, for two chunks of 2048 tokens over 8192, 32 query heads over 8 x 128, 4
// bits), inlining the waits as much again, and what is rare stands in functions.
//
// K and V become fp16 including scale and low value: fp16_rn(low + s code), one
// rounding of 2^-11 relative to the element (scale and low value have 8 bits), so
// the products need no factors per token.  Q and P as in kv_attention.cu.  Ranges:
// a row of Q is scaled to 2^8; a tile of K by the power of two that brings its
// largest element to 2^7, undone in c; V by one such power for all tiles so far, O
// being rescaled when it grows.  A token whose largest element is more than 2^12
// below that is held at an exponent of its own (least_exps), which S and P then make
// up for (uneven_tile), so that what fp16 keeps of a token's keys does not depend on
// its neighbours; of its values, with weights that reach 2^-14 at that distance, down
// to 2^-33 of the largest.  P's maximum m is only raised when a row exceeds it by 2^8
// (the sums are rescaled then), so P reaches at most 2^15 and keeps weights down to
// 2^-31 of the largest.  Value rows that are not finite count as 0 and turn the total
// of the rows that see them into no number (sees_not_finite): a product with the
// weight 0 would carry them to the other rows.
//
// Operand layout: K-major, 128-byte swizzle.  The order of the channels is
// free as long as Q and K agree, so key words are stored in the order in
// which they unpack; V is stored transposed (channels x tokens), eight tokens
// of a channel at a time, paired by byte permutes while unpacking.  Raw value
// rows are copied eight tokens at a time to a stride 16 bytes longer, which
// keeps the transposing reads off each other's banks.
//
// Measured: those two chunks now 490 us with the join (982 TFLOP/s, 51 % of a
// large bf16 product; the tensor pipe is busy 44 % of the time, the issue slots
// 53 %), 680 at 8 bits (707 TFLOP/s: one V stage, so that V's unpacking and P V
// take turns), 407 with 64 channels (590); one prompt of 8192 tokens 600 us (916
// TFLOP/s).  Parts of items cut between blocks go through memory: the join is 27 of
// those 490 with cold caches.

#include <cuda_runtime.h>

#include "kv_math.cuh"

namespace i8ql {
namespace {

constexpr int kTile = kKvPromptTile;  // cache tokens per tile
constexpr int kRows = kKvPromptRows;  // query rows per block: two M tiles
constexpr int kSoftmaxWarps = 8;
constexpr int kUnpackWarps = 4;
constexpr int kCopyWarp = kSoftmaxWarps + kUnpackWarps;
constexpr int kMmaWarp = kCopyWarp + 1;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kKStages = 2;      // unpacked K tiles
constexpr int kRawKeys = 2;      // raw K tiles (with the params of K and V)
// Tiles that beginning and ending an item counts (one prompt of 8192 tokens, whose
// items have 1 to 64 tiles: 789 us at 2, 586 at 4, 588 at 6, when it was chosen).
constexpr int kCost = 4;
constexpr int kInfo = 4;         // tiles whose exponents are kept
constexpr float kPShift = 7.0f;  // P = 2^(logit - m + kPShift)
constexpr float kSlack = 8.0f;   // a row's maximum may exceed m by this (log2)

template <int D, int BITS>
struct Cfg {
    static constexpr int kRowBytes = D * BITS / 8;
    static constexpr int kKTile = kTile * D * 2;  // an operand tile of K, and of V
    static constexpr int kVStages = BITS == 8 && D == 128 ? 1 : 2;
    static constexpr int kGroupStride = 8 * kRowBytes + 16;  // eight raw value rows
    static constexpr int kRawK = kTile * kRowBytes + 2 * kTile * 4;
    static constexpr int kRawV = kTile / 8 * kGroupStride;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kRows * D * 2;
    static constexpr int kOffV = kOffK + kKStages * kKTile;
    static constexpr int kOffRawK = kOffV + kVStages * kKTile;
    static constexpr int kOffRawV = kOffRawK + kRawKeys * kRawK;
    static constexpr int kSmem = kOffRawV + kRawV + 1024;  // (aligned to 1024 by hand)
};

// MMAs and commits of the lane with issue != 0.  The others run along: in a
// branch of one lane the descriptors could not stay in uniform registers.
template <int A_AT, int B_AT>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc,
                                       uint32_t accumulate, uint32_t issue) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 ta, tb;\n\t.reg .b64 da, db;\n\t"
        "add.u32 ta, %1, %7;\n\t"
        "add.u32 tb, %2, %8;\n\t"
        "mov.b64 da, {ta, %3};\n\t"
        "mov.b64 db, {tb, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(accumulate), "r"(issue), "n"(A_AT), "n"(B_AT)
        : "memory");
}

template <int A_AT, int B_AT>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t high, uint32_t idesc,
                                       uint32_t accumulate, uint32_t issue) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 ta, tb;\n\t.reg .b64 db;\n\t"
        "add.u32 ta, %1, %7;\n\t"
        "add.u32 tb, %2, %8;\n\t"
        "mov.b64 db, {tb, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b), "r"(high), "r"(idesc), "r"(accumulate), "r"(issue), "n"(A_AT), "n"(B_AT)
        : "memory");
}

__device__ __forceinline__ void commit_mma(uint64_t* bar, uint32_t issue) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar)),
        "r"(issue)
        : "memory");
}

#define I8QL_R8(r, i) "=r"((r)[i]), "=r"((r)[(i) + 1]), "=r"((r)[(i) + 2]), "=r"((r)[(i) + 3]), "=r"((r)[(i) + 4]), \
                      "=r"((r)[(i) + 5]), "=r"((r)[(i) + 6]), "=r"((r)[(i) + 7])
#define I8QL_W8(r, i) "r"((r)[i]), "r"((r)[(i) + 1]), "r"((r)[(i) + 2]), "r"((r)[(i) + 3]), "r"((r)[(i) + 4]), \
                      "r"((r)[(i) + 5]), "r"((r)[(i) + 6]), "r"((r)[(i) + 7])

// 32 columns of this warp's lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : I8QL_R8(r, 0), I8QL_R8(r, 8), I8QL_R8(r, 16), I8QL_R8(r, 24)
        : "r"(addr));
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        I8QL_W8(r, 0), I8QL_W8(r, 8), I8QL_W8(r, 16), I8QL_W8(r, 24)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            addr),
        I8QL_W8(r, 0), I8QL_W8(r, 8)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void unpack_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kUnpackWarps * 32) : "memory"); }

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair_u32(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_f32(float a, float b) {
    return pair_u32(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ void split_f32(uint64_t p, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Exponents of a tile, for the softmax.
struct TileInfo {
    int key_exp;  // K is held times 2^(134 - key_exp)
    int val_exp;  // V is held times 2^(134 - val_exp), from this tile on
};
// Added to val_exp where some tokens are so much smaller than others that they are
// held at exponents of their own (least_exps), keys or values.
constexpr int kUneven = 1 << 16;

// The least exponents a token's key and value row (their largest magnitudes, as
// bits) may be held at, the value's << 16: 12 above their own, so that elements stay
// clear of the subnormal numbers of fp16: they keep 11 bits down to 2^-9 of the
// largest, and a scale that is subnormal itself loses less than 2^-12 of the largest
// over all codes.  (Rows of zeros, and keys that are not finite, come out above any
// tile's exponent.)
__device__ __forceinline__ uint32_t least_exps(uint32_t bits_k, uint32_t bits_v) {
    return ((bits_k - 1) >> 23 | ((bits_v - 1) >> 23 << 16)) + (12u | 12u << 16);
}

// The maximum of a tile's S over the tokens the row sees.  EDGE: some row does not
// see some of them.
template <bool EDGE>
__device__ __forceinline__ float tile_maximum(uint32_t s_at, int token, int lo, int hi) {
    uint32_t x[32];
    float high[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int q = 0; q < kTile / 32; ++q) {
        tmem_ld32(s_at + q * 32, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            float y = __uint_as_float(x[j]), z = __uint_as_float(x[j + 1]);
            if (EDGE) {
                const int tok = token + q * 32 + j;
                y = tok <= hi && tok >= lo ? y : -INFINITY;
                z = tok + 1 <= hi && tok + 1 >= lo ? z : -INFINITY;
            }
            high[(j / 2) & 3] = max3(high[(j / 2) & 3], y, z);
        }
    }
    return max3(fmaxf(high[0], high[1]), high[2], high[3]);
}

// What a row's sums stand at.
struct RowSums {
    float unit;   // what a scaled logit counts (times 2^(key_exp - 134)), in log2 units
    float top;    // the maximum, in the same units
    float total;
    int val_exp;  // of O
};

// The tile's maximum `high` in the row's units, and whether it exceeds what the sums
// stand at by more than the slack (the first time: from -infinity).
__device__ __forceinline__ float in_units(const RowSums& row, float high, const TileInfo& info) {
    return high == -INFINITY ? -INFINITY : high * (row.unit * pow2(info.key_exp - 134));
}
__device__ __forceinline__ bool exceeds(const RowSums& row, float a) { return a > row.top + kSlack; }

// Whether some row of the warp does, or the exponent changes.
__device__ __forceinline__ bool sums_change(const RowSums& row, float high, const TileInfo& info) {
    return __any_sync(0xffffffffu, exceeds(row, in_units(row, high, info))) || info.val_exp != row.val_exp;
}

// Raises the maximum where it is exceeded, and brings O and the total to it and to the
// tile's exponent.
template <int D>
__device__ __forceinline__ void change_sums(RowSums& row, float high, const TileInfo& info, uint32_t o_at, bool first,
                                            float& shrunk) {
    const float a = in_units(row, high, info);
    const bool raise = exceeds(row, a);
    float f = 1.0f;
    if (raise) {
        const float shrink = shrink_reference(a);
        f = exp2_approx((row.top - a) * shrink);
        row.top = a;
        row.total *= f;
        if (shrink != 1.0f) {
            row.unit *= shrink;
            row.top *= shrink;
            shrunk *= shrink;
        }
    }
    if (!first) {
        f *= info.val_exp - row.val_exp > 126 ? 0.0f : pow2(row.val_exp - info.val_exp);
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
            uint32_t v[32];
            tmem_ld32(o_at + q * 32, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
            tmem_st32(o_at + q * 32, v);
        }
    }
    row.val_exp = info.val_exp;
}

// P over the columns of S; returns the sum of the row's weights.
template <bool EDGE>
__device__ __forceinline__ float tile_weights(const RowSums& row, int key_exp, uint32_t s_at, int token, int lo, int hi) {
    const float cst = row.unit * pow2(key_exp - 134);
    const uint64_t cst2 = pair_f32(cst, cst);
    const float shift = row.top == -INFINITY ? 0.0f : kPShift - row.top;
    const uint64_t shift2 = pair_f32(shift, shift);
    uint32_t x[32];
    uint64_t sum[2] = {0, 0};
#pragma unroll 1
    for (int q = 0; q < kTile / 32; ++q) {
        tmem_ld32(s_at + q * 32, x);
        tc::tmem_wait_ld();
        uint32_t h[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            float y, z;
            split_f32(fma_f32x2(pair_u32(x[j], x[j + 1]), cst2, shift2), y, z);
            y = exp2_approx(y);
            z = exp2_approx(z);
            if (EDGE) {
                const int tok = token + q * 32 + j;
                y = tok <= hi && tok >= lo ? y : 0.0f;
                z = tok + 1 <= hi && tok + 1 >= lo ? z : 0.0f;
            }
            sum[(j / 2) & 1] = add_f32x2(sum[(j / 2) & 1], pair_f32(y, z));
            h[j / 2] = pack_f16(y, z);
        }
        // (columns of S that have been read: chunk q of P lies in chunk q / 2)
        tmem_st16(s_at + q * 16, h);
    }
    float y, z;
    split_f32(add_f32x2(sum[0], sum[1]), y, z);
    return y + z;
}

// A tile some of whose tokens are held at exponents `down` below the tile's: the same,
// with S brought to the tile's before, and P (which the sum of the weights does not
// see) after.  (Rare: a function, so that the loop over the tiles stays small.)
template <int D>
__device__ __noinline__ RowSums uneven_tile(RowSums row, TileInfo info, const uint32_t* down, uint32_t s_at,
                                            uint32_t o_at, bool first, float* shrunk, int token, int lo, int hi) {
    info.val_exp -= kUneven;
#pragma unroll 1
    for (int q = 0; q < kTile / 32; ++q) {
        uint32_t x[32];
        tmem_ld32(s_at + q * 32, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int by = down[q * 32 + j] & 0xffff;
            x[j] = by > 126 ? 0u : __float_as_uint(__uint_as_float(x[j]) * pow2(-by));
        }
        tmem_st32(s_at + q * 32, x);
    }
    tmem_wait_st();
    const float high = tile_maximum<true>(s_at, token, lo, hi);
    if (sums_change(row, high, info)) change_sums<D>(row, high, info, o_at, first, *shrunk);
    row.total += tile_weights<true>(row, info.key_exp, s_at, token, lo, hi);
    tmem_wait_st();
#pragma unroll 1
    for (int q = 0; q < kTile / 64; ++q) {
        uint32_t x[32];
        tmem_ld32(s_at + q * 32, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int a = down[q * 64 + 2 * j] >> 16, b = down[q * 64 + 2 * j + 1] >> 16;
            x[j] = fma_f16x2(x[j], pack_f16(a > 24 ? 0.0f : pow2(-a), b > 24 ? 0.0f : pow2(-b)), 0u);
        }
        tmem_st32(s_at + q * 32, x);
    }
    return row;
}

// The bits of a row's largest magnitude (a row is low .. low + scale * kTop); not
// below infinity's when some element is not finite.
template <int BITS>
__device__ __forceinline__ uint32_t row_bits(uint32_t param) {
    constexpr float kTop = BITS == 4 ? 15.0f : 255.0f;
    const float lo = kv_low(param);
    return max(__float_as_uint(lo) & 0x7fffffffu, __float_as_uint(fmaf(kv_scale(param), kTop, lo)) & 0x7fffffffu);
}

// Whether the value rows of one of the sequence's tokens lo .. hi are not finite
// (rare: only asked once a block has met such a row).
template <int BITS>
__device__ __noinline__ bool sees_not_finite(const KvAttnParams& p, const KvCursor& c, int lo, int hi) {
    bool sees = false;
#pragma unroll 1
    for (int t = lo; t <= hi; ++t) {
        int64_t page = p.table[c.b * p.table_width + (t >> p.cache.page_shift)];
        if (page < 0 || page >= p.cache.pages) page = 0;  // (as copied)
        const int off = t & ((1 << p.cache.page_shift) - 1);
        sees = sees || row_bits<BITS>(p.cache.params[kv_row(p.cache, page, 1, c.h, off)]) >= 0x7f800000u;
    }
    return sees;
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(const KvAttnParams p) {
    using C = Cfg<D, BITS>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t raw_k_full[kRawKeys], raw_k_empty[kRawKeys], raw_v_full, raw_v_empty;
    __shared__ uint64_t k_full[kKStages], k_empty[kKStages], v_full[2], v_empty[2];
    __shared__ uint64_t q_full[2], s_full[2], p_full[2], o_full[2], info_full[kInfo], drained;
    __shared__ KvLocate locate;
    __shared__ KvCursor cursors[kSoftmaxWarps];  // (kept out of the registers of the softmax)
    __shared__ KvRange range;
    __shared__ TileInfo infos[kInfo];
    __shared__ uint32_t down[kInfo][kTile];  // how much a token's exponents are below the tile's: keys, and values << 16
    __shared__ float shrunk[kRows];  // by how much a row's unit and maximum have been shrunk
    __shared__ __align__(16) uint32_t exp_red[2][kUnpackWarps];  // largest exponents: keys, and values << 16
    static_assert(kUnpackWarps == 4);
    __shared__ uint32_t key_factor[kTile][2];                // scale and low value, each twice, as halves
    __shared__ __align__(16) uint16_t val_factor[2][kTile];  // scales, low values
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ int met_not_finite;  // some value row so far was not finite

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t smem_at = tc::smem_u32(smem);
    if (threadIdx.x == 0) {
        abort_flag = 0;
        met_not_finite = 0;
        for (int i = 0; i < kRawKeys; ++i) {
            tc::mbar_init(&raw_k_full[i], 1);
            tc::mbar_init(&raw_k_empty[i], kUnpackWarps);
        }
        tc::mbar_init(&raw_v_full, 1);
        tc::mbar_init(&raw_v_empty, kUnpackWarps);
        for (int i = 0; i < kKStages; ++i) {
            tc::mbar_init(&k_full[i], kUnpackWarps * 32);
            tc::mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&v_full[i], kUnpackWarps * 32);
            tc::mbar_init(&v_empty[i], 1);
            tc::mbar_init(&q_full[i], 128);
            tc::mbar_init(&s_full[i], 1);
            tc::mbar_init(&p_full[i], 128);
            tc::mbar_init(&o_full[i], 1);
        }
        for (int i = 0; i < kInfo; ++i) tc::mbar_init(&info_full[i], kUnpackWarps);
        tc::mbar_init(&drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == kMmaWarp) tc::tmem_alloc(&tmem_base, 512);
    tc::tc_fence_before();
    KvCursor start;
    const KvRange found = kv_locate<kRows, kTile, kCost, kThreads>(p, locate, start);  // (its barriers publish the above)
    tc::tc_fence_after();
    const uint32_t tmem = tmem_base;
    bool dead = false;
    // Waits of a whole warp; after one that gave up no work is done any more,
    // but every loop and barrier runs to its end.
    // (The test comes before the call: a barrier that is passed already, the
    // common case of the MMA warp, costs 40 cycles and not 170.)
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (dead || __all_sync(0xffffffffu, tc::mbar_test(tc::smem_u32(bar), parity))) return;
        dead = !tc::warp_wait(bar, parity, &abort_flag, p.err);
    };

    if (warp == kCopyWarp) {
        // ------------------------------------------------------------ copies
        KvCursor c = start;
        const int page_tokens = 1 << p.cache.page_shift;
        const int piece = min(page_tokens, kTile);
        const int kind = lane & 3;  // K codes, K params, V params, none
        const int at = (lane >> 2) * piece;
        const int at_v = lane * 8;  // V codes: eight tokens
        uint32_t kt = 0;            // tiles so far
        uint32_t keys_issued = 0, values_issued = 0;
        // An unpacking warp that gave up says so before it frees raw tiles that it
        // did not wait for, whose copies may still be on their way.
        auto wait_free = [&](uint64_t* bar, uint32_t parity) {
            wait(bar, parity);
            dead = dead || __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&abort_flag));
        };
        while (const int n = dead ? 0 : kv_take<kCost>(p, c, found.end)) {
            const int32_t* table = p.table + c.b * p.table_width;
            const int first = (c.span.first + c.tile) * kTile;
            auto needed = [&](int token, int tokens, int i) {
                return i < n && token < c.span.end && token + tokens > c.span.begin;
            };
            auto need_k = [&](int i) { return kind < 3 && at < kTile && needed(first + i * kTile + at, piece, i); };
            auto need_v = [&](int i) { return at_v < kTile && needed(first + i * kTile + at_v, 8, i); };
            auto page_of = [&](bool need, int token) { return need ? __ldg(table + (token >> p.cache.page_shift)) : 0; };
            auto checked = [&](int64_t page) {
                if (page >= 0 && page < p.cache.pages) return page;
                record_fault(p.err, kErrBitBadIndex);
                return (int64_t)0;
            };
            // pages are looked up a tile ahead
            int32_t next_k = page_of(need_k(0), first + at), next_v = page_of(need_v(0), first + at_v);
            for (int i = 0; i < n && !dead; ++i) {
                const int token = first + i * kTile;
                const bool nk = need_k(i), nv = need_v(i);
                const int64_t page_k = next_k, page_v = next_v;
                next_k = page_of(need_k(i + 1), token + kTile + at);
                next_v = page_of(need_v(i + 1), token + kTile + at_v);
                const uint32_t slot = kt % kRawKeys;
                const unsigned keys = __popc(__ballot_sync(0xffffffffu, nk && kind == 0));
                const unsigned groups = __popc(__ballot_sync(0xffffffffu, nv));
                wait_free(&raw_k_empty[slot], ((kt / kRawKeys) & 1) ^ 1);
                if (!dead) {
                    ++keys_issued;
                    if (lane == 0) tc::mbar_expect_tx(&raw_k_full[slot], keys * piece * (C::kRowBytes + 8));
                    __syncwarp();
                    if (nk) {
                        const int64_t row =
                            kv_row(p.cache, checked(page_k), kind == 2, c.h, (token + at) & (page_tokens - 1));
                        uint8_t* raw = smem + C::kOffRawK + slot * C::kRawK;
                        if (kind == 0)
                            bulk_load(raw + at * C::kRowBytes, p.cache.codes + row * C::kRowBytes,
                                      piece * C::kRowBytes, &raw_k_full[slot]);
                        else
                            bulk_load(raw + kTile * C::kRowBytes + (kind - 1) * kTile * 4 + at * 4,
                                      p.cache.params + row, piece * 4, &raw_k_full[slot]);
                    }
                }
                wait_free(&raw_v_empty, (kt & 1) ^ 1);
                if (!dead) {
                    ++values_issued;
                    if (lane == 0) tc::mbar_expect_tx(&raw_v_full, groups * 8 * C::kRowBytes);
                    __syncwarp();
                    if (nv) {
                        const int64_t row = kv_row(p.cache, checked(page_v), 1, c.h, (token + at_v) & (page_tokens - 1));
                        bulk_load(smem + C::kOffRawV + lane * C::kGroupStride, p.cache.codes + row * C::kRowBytes,
                                  8 * C::kRowBytes, &raw_v_full);
                    }
                    ++kt;
                }
            }
            if (!dead) kv_next_item<kRows, kTile, kCost>(p, c);
        }
        // the last copies land before the block's shared memory can go to
        // another (the unpacking warps may have given up on them)
        int none = 0;
        for (uint32_t k = keys_issued > kRawKeys ? keys_issued - kRawKeys : 0; k < keys_issued; ++k)
            tc::mbar_wait(&raw_k_full[k % kRawKeys], (k / kRawKeys) & 1, &none, p.err);
        if (values_issued > 0) tc::mbar_wait(&raw_v_full, (values_issued - 1) & 1, &none, p.err);
    } else if (warp >= kSoftmaxWarps && warp < kCopyWarp) {
        // ------------------------------------------------------------ unpacking
        KvCursor c = start;
        const int tid = threadIdx.x - kSoftmaxWarps * 32;  // 0 .. 127
        const int w4 = warp - kSoftmaxWarps;
        uint32_t kt = 0;
        constexpr int kLanesPerKey = C::kRowBytes / 16;
        constexpr int kChunks = BITS == 4 ? 4 : 2;  // operand chunks (8 channels) per 16 raw bytes
        constexpr int kValWords = D * BITS / 256;   // raw words of D / 8 channels
        constexpr int kPerWord = 32 / BITS;         // channels per word
        const int key_lane = tid % kLanesPerKey;
        const int val_group = tid & 15, val_part = tid >> 4;  // eight tokens, D / 8 channels
        while (const int n = kv_take<kCost>(p, c, found.end)) {
            uint32_t tile_exp = 8u << 16;  // of the tile's keys, and of the values so far << 16
            for (int i = 0; i < n; ++i, ++kt) {
                const int token = (c.span.first + c.tile + i) * kTile;
                const uint32_t slot = kt % kRawKeys, stage = kt % kKStages;
                const uint8_t* raw = smem + C::kOffRawK + slot * C::kRawK;
                wait(&raw_k_full[slot], (kt / kRawKeys) & 1);
                // one token's scales and low values; the tile's exponents
                uint32_t pk = 0, pv = 0;
                if (!dead && token + tid >= c.span.begin && token + tid < c.span.end) {
                    const uint32_t* params = reinterpret_cast<const uint32_t*>(raw + kTile * C::kRowBytes) + tid;
                    pk = params[0];
                    pv = params[kTile];
                }
                const uint32_t bits_k = row_bits<BITS>(pk);
                uint32_t bits_v = row_bits<BITS>(pv);
                if (bits_v >= 0x7f800000u) {
                    // not finite: it must not meet the weight 0 of a row that does not
                    // see it, so it counts as 0, and the rows that do see it look for it
                    bits_v = pv = 0;
                    met_not_finite = 1;
                }
                const uint32_t top_k = __reduce_max_sync(0xffffffffu, bits_k < 0x7f800000u ? bits_k : 0u);
                const uint32_t top_v = __reduce_max_sync(0xffffffffu, bits_v);
                const uint32_t least = least_exps(bits_k, bits_v);
                if (lane == 0) exp_red[kt & 1][w4] = top_k >> 23 | top_v >> 23 << 16;
                unpack_sync();
                const uint4 tops = *reinterpret_cast<const uint4*>(exp_red[kt & 1]);
                tile_exp = __vmaxu2(__vmaxu2(__vmaxu2(tops.x, tops.y), __vmaxu2(tops.z, tops.w)), (tile_exp & 0xffff0000u) | 8);
                const uint32_t exps = __vminu2(tile_exp, least), below = tile_exp - exps;
                const float fk = __uint_as_float((261u << 23) - (exps << 23));  // 2^(134 - exponent)
                const float fv = __uint_as_float((261u << 23) - (exps >> 16 << 23));
                const float ks = kv_scale(pk) * fk, kl = kv_low(pk) * fk;
                const float vs = kv_scale(pv) * fv, vl = kv_low(pv) * fv;
                key_factor[tid][0] = pack_f16(ks, ks);
                key_factor[tid][1] = pack_f16(kl, kl);
                const uint32_t v2 = pack_f16(vs, vl);
                val_factor[0][tid] = (uint16_t)v2;
                val_factor[1][tid] = (uint16_t)(v2 >> 16);
                down[kt % kInfo][tid] = below;
                if (tid == 0) {
                    infos[kt % kInfo].key_exp = tile_exp & 0xffff;
                    infos[kt % kInfo].val_exp = tile_exp >> 16;
                }
                unpack_sync();
                if (below) atomicOr(&infos[kt % kInfo].val_exp, kUneven);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&info_full[kt % kInfo]);
                // K: 16 raw bytes of a token at a time
                wait(&k_empty[stage], ((kt / kKStages) & 1) ^ 1);
                if (!dead) {
                    const uint32_t dst = smem_at + C::kOffK + stage * C::kKTile;
#pragma unroll 1
                    for (int r = 0; r < kLanesPerKey; ++r) {
                        const int tok = tid / kLanesPerKey + r * (kTile / kLanesPerKey);
                        uint32_t w[4];
                        lds<4>(raw + tok * C::kRowBytes + key_lane * 16, w);
                        const uint32_t s = key_factor[tok][0], o = key_factor[tok][1];
                        const int chunk0 = key_lane * kChunks;  // of the row's D / 8
                        const int block = chunk0 / 8, pos0 = chunk0 % 8;
                        const int flip = block & 1;  // lanes of the two blocks take their chunks in opposite order (banks)
                        const uint32_t row = dst + block * (kTile * 128) + tok * 128;
#pragma unroll
                        for (int j = 0; j < kChunks; ++j) {
                            uint32_t h[4];
                            if constexpr (BITS == 4) {
                                unpack_nibbles<false>(flip ? w[j ^ 1] : w[j], h);
                            } else {
                                const uint32_t a = flip ? w[2 * (j ^ 1)] : w[2 * j];
                                const uint32_t b = flip ? w[2 * (j ^ 1) + 1] : w[2 * j + 1];
                                h[0] = unpack_bytes<false>(a, 0x5150);
                                h[1] = unpack_bytes<false>(a, 0x5352);
                                h[2] = unpack_bytes<false>(b, 0x5150);
                                h[3] = unpack_bytes<false>(b, 0x5352);
                            }
                            sts16(row + (((pos0 + (j ^ flip)) ^ (tok & 7)) << 4), fma_f16x2(h[0], s, o),
                                  fma_f16x2(h[1], s, o), fma_f16x2(h[2], s, o), fma_f16x2(h[3], s, o));
                        }
                    }
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&k_full[stage]);
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&raw_k_empty[slot]);
                // V, transposed: eight tokens of D / 8 channels
                const uint32_t vstage = kt % C::kVStages;
                wait(&raw_v_full, kt & 1);
                wait(&v_empty[vstage], ((kt / C::kVStages) & 1) ^ 1);
                if (!dead) {
                    const uint8_t* src = smem + C::kOffRawV + val_group * C::kGroupStride + val_part * (kValWords * 4);
                    uint32_t s[4], o[4];
                    lds<4>(reinterpret_cast<const uint8_t*>(&val_factor[0][val_group * 8]), s);
                    lds<4>(reinterpret_cast<const uint8_t*>(&val_factor[1][val_group * 8]), o);
                    const uint32_t dst = smem_at + C::kOffV + vstage * C::kKTile + (val_group / 8) * (D * 128);
#pragma unroll 1
                    for (int k = 0; k < kValWords; ++k) {
                        uint32_t w[8], h[4][kPerWord];
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = *reinterpret_cast<const uint32_t*>(src + j * C::kRowBytes + k * 4);
#pragma unroll
                        for (int j = 0; j < 4; ++j) unpack_values<BITS, false>(w[2 * j], w[2 * j + 1], h[j]);
#pragma unroll
                        for (int e = 0; e < kPerWord; ++e) {
                            const int ch = val_part * (D / 8) + k * kPerWord + e;
                            sts16(dst + ch * 128 + (((val_group & 7) ^ (ch & 7)) << 4), fma_f16x2(h[0][e], s[0], o[0]),
                                  fma_f16x2(h[1][e], s[1], o[1]), fma_f16x2(h[2][e], s[2], o[2]),
                                  fma_f16x2(h[3][e], s[3], o[3]));
                        }
                    }
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&v_full[vstage]);
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&raw_v_empty);
            }
            kv_next_item<kRows, kTile, kCost>(p, c);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMAs
        KvCursor c = start;
        const uint32_t s_desc = tc::f16_idesc(kTile), o_desc = tc::f16_idesc(D);
        uint32_t kt = 0, items[2] = {0, 0}, steps[2] = {0, 0};
        // descriptors count in units of 16 bytes: 2 a step of 16 elements, and
        // the rest of a row's swizzle atoms behind the first 64 elements
        const uint32_t q_base = (uint32_t)tc::sw128_desc(smem_at + C::kOffQ);
        const uint32_t k_base = (uint32_t)tc::sw128_desc(smem_at + C::kOffK);
        const uint32_t v_base = (uint32_t)tc::sw128_desc(smem_at + C::kOffV);
        const uint32_t high = (uint32_t)(tc::sw128_desc(smem_at) >> 32);
        auto qk = [&](int m, uint32_t tile) {
            const uint32_t a = q_base + m * (128 * D * 2 / 16);
            const uint32_t b = k_base + (tile % kKStages) * (C::kKTile / 16);
            const uint32_t d = tmem + m * kTile, issue = !dead && lane == 0;
            __syncwarp();
            mma_ss<0, 0>(d, a, b, high, s_desc, 0, issue);
            mma_ss<2, 2>(d, a, b, high, s_desc, 1, issue);
            mma_ss<4, 4>(d, a, b, high, s_desc, 1, issue);
            mma_ss<6, 6>(d, a, b, high, s_desc, 1, issue);
            if constexpr (D == 128) {
                constexpr int kNext = 128 * 128 / 16;  // the second 64 channels: rows of 128 tokens or queries
                mma_ss<kNext, kNext>(d, a, b, high, s_desc, 1, issue);
                mma_ss<kNext + 2, kNext + 2>(d, a, b, high, s_desc, 1, issue);
                mma_ss<kNext + 4, kNext + 4>(d, a, b, high, s_desc, 1, issue);
                mma_ss<kNext + 6, kNext + 6>(d, a, b, high, s_desc, 1, issue);
            }
            commit_mma(&s_full[m], issue);
        };
        auto pv = [&](int m, uint32_t tile, bool first) {
            const uint32_t a = tmem + m * kTile;
            const uint32_t b = v_base + (tile % C::kVStages) * (C::kKTile / 16);
            const uint32_t d = tmem + 256 + m * D, issue = !dead && lane == 0;
            constexpr int kNext = D * 128 / 16;  // the second 64 tokens
            __syncwarp();
            mma_ts<0, 0>(d, a, b, high, o_desc, !first, issue);
            mma_ts<8, 2>(d, a, b, high, o_desc, 1, issue);
            mma_ts<16, 4>(d, a, b, high, o_desc, 1, issue);
            mma_ts<24, 6>(d, a, b, high, o_desc, 1, issue);
            mma_ts<32, kNext>(d, a, b, high, o_desc, 1, issue);
            mma_ts<40, kNext + 2>(d, a, b, high, o_desc, 1, issue);
            mma_ts<48, kNext + 4>(d, a, b, high, o_desc, 1, issue);
            mma_ts<56, kNext + 6>(d, a, b, high, o_desc, 1, issue);
        };
        auto commit = [&](uint64_t* bar) { commit_mma(bar, !dead && lane == 0); };
        while (const int n = kv_take<kCost>(p, c, found.end)) {
            const int rows = min(kRows, c.seq.nq * p.G - c.rb * kRows);
            const int tiles_m = rows > 128 ? 2 : 1;
            for (int m = 0; m < tiles_m; ++m) {
                wait(&q_full[m], items[m] & 1);
                ++items[m];
                if (m == 0) wait(&k_full[kt % kKStages], (kt / kKStages) & 1);
                tc::tc_fence_after();
                qk(m, kt);
            }
            commit(&k_empty[kt % kKStages]);
            for (int i = 0; i < n; ++i, ++kt) {
                // (neither waits for a product that is still to be issued)
                wait(&v_full[kt % C::kVStages], (kt / C::kVStages) & 1);
                if (i + 1 < n) wait(&k_full[(kt + 1) % kKStages], ((kt + 1) / kKStages) & 1);
                for (int m = 0; m < tiles_m; ++m) {
                    wait(&p_full[m], steps[m] & 1);
                    ++steps[m];
                    tc::tc_fence_after();
                    pv(m, kt, i == 0);
                    if (i + 1 < n) {
                        qk(m, kt + 1);
                    } else {
                        commit(&o_full[m]);
                    }
                }
                commit(&v_empty[kt % C::kVStages]);
                if (i + 1 < n) commit(&k_empty[(kt + 1) % kKStages]);
            }
            kv_next_item<kRows, kTile, kCost>(p, c);
        }
        // nothing may be in flight when the TMEM is given back
        if (lane == 0) tc::mma_commit(&drained);
        __syncwarp();
        int none = 0;
        tc::mbar_wait(&drained, 0, &none, p.err);
    } else {
        // ------------------------------------------------------------ softmax
        const int m = warp / 4;
        const int r = m * 128 + (warp % 4) * 32 + lane;  // row of the block
        const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t s_at = tmem + lanes + m * kTile, o_at = tmem + lanes + 256 + m * D;
        KvCursor& c = cursors[warp];
        if (lane == 0) c = start;
        if (threadIdx.x == 0) range = found;
        asm volatile("bar.sync 2, %0;" ::"n"(kSoftmaxWarps * 32) : "memory");
        uint32_t kt = 0, items = 0, steps = 0;
        bool split = false;
        // What a thread knows of its row of an item.
        struct Row {
            bool active, live;   // the item has this M tile; the row exists
            int hi, lo;          // the tokens it sees
            int all_hi, all_lo;  // tokens [all_lo, all_hi] are seen by every row of the M tile
            float unit;          // what a scaled logit counts (times 2^(key_exp - 134)), in log2 units
            int64_t out;         // where its output goes
        };
        // Takes up the cursor's item: the row of Q, scaled to 2^8 and permuted
        // as the keys unpack, goes into its operand tile (which the products
        // of the item before have left by the time its last S is there).
        auto take_up = [&](Row& row) {
            const int row0 = c.rb * kRows;
            const int rows = min(kRows, c.seq.nq * p.G - row0);
            row.active = m == 0 || rows > 128;
            if (!row.active) return;
            const int base = c.seq.len - c.seq.nq;
            row.live = r < rows;
            const int i = (row0 + (row.live ? r : 0)) / p.G;
            const int head = c.h * p.G + (row0 + (row.live ? r : 0)) - i * p.G;
            row.hi = row.live ? base + i : INT32_MAX;
            row.lo = row.live && p.window > 0 ? (int)max(base + i + 1 - p.window, (int64_t)0) : 0;
            row.all_hi = base + (row0 + m * 128) / p.G;
            const int last = row0 + min(rows, m * 128 + 128) - 1;
            row.all_lo = p.window > 0 ? (int)max(base + last / p.G + 1 - p.window, (int64_t)0) : 0;
            row.out = ((c.seq.q0 + i) * ((int64_t)p.cache.H * p.G) + head) * D;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (c.seq.q0 + i) * p.q_stride + (int64_t)head * D);
            uint32_t top = 0;
#pragma unroll 8
            for (int w = 0; w < D / 8; ++w) {
                const uint4 v = row.live ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
                const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a = words[j] & 0x7fff0000u, b = (words[j] << 16) & 0x7fff0000u;
                    top = max(top, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
                }
            }
            const int e = max((int)(top >> 23), 9) - 127;
            const float f = p.scale_log2 < 0.0f ? -pow2(8 - e) : pow2(8 - e);
            row.unit = pow2(e - 8) * fabsf(p.scale_log2);
            const uint32_t dst = smem_at + C::kOffQ + m * (128 * D * 2) + (r & 127) * 128;
#pragma unroll 4
            for (int w = 0; w < D / 8; ++w) {
                const uint4 v = row.live ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
                const float y[8] = {lo_bf16(v.x) * f, hi_bf16(v.x) * f, lo_bf16(v.y) * f, hi_bf16(v.y) * f,
                                    lo_bf16(v.z) * f, hi_bf16(v.z) * f, lo_bf16(v.w) * f, hi_bf16(v.w) * f};
                const uint32_t at = dst + (w / 8) * (128 * 128) + (((w & 7) ^ (r & 7)) << 4);
                if constexpr (BITS == 4)
                    sts16(at, pack_f16(y[0], y[4]), pack_f16(y[1], y[5]), pack_f16(y[2], y[6]), pack_f16(y[3], y[7]));
                else
                    sts16(at, pack_f16(y[0], y[1]), pack_f16(y[2], y[3]), pack_f16(y[4], y[5]), pack_f16(y[6], y[7]));
            }
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(&q_full[m]);
        };
        Row row = {};
        int n = kv_take<kCost>(p, c, range.end);
        if (n > 0) take_up(row);
        while (n > 0) {
            const bool begins = c.tile == 0, ends = c.tile + n == c.span.tiles;
            RowSums sums = {row.unit, -INFINITY, 0.0f, 8};
            if (row.active) {
                const int hi = row.hi, lo = row.lo;
                shrunk[r] = 1.0f;
                const int first = (c.span.first + c.tile) * kTile;
                for (int i = 0; i < n; ++i, ++steps) {
                    const int token = first + i * kTile;
                    const uint32_t k = kt + i;
                    // S first: an M tile that sat out an item may be two rounds of
                    // info_full behind, whose parity then passes at once; after this
                    // tile's S its exponents are there (they were written before K),
                    // and no later ones can be (those wait for this tile's P), so one
                    // test of the barrier passes, and acquires them
                    wait(&s_full[m], steps & 1);
                    const bool there = tc::mbar_test(tc::smem_u32(&info_full[k % kInfo]), (k / kInfo) & 1);
                    tc::tc_fence_after();
                    if (!dead && __all_sync(0xffffffffu, there)) {
                        const TileInfo info = infos[k % kInfo];
                        const bool edge = token + kTile - 1 > row.all_hi || token < row.all_lo;
                        const float high = edge ? tile_maximum<true>(s_at, token, lo, hi)
                                                : tile_maximum<false>(s_at, token, lo, hi);
                        if (sums_change(sums, high, info)) {
                            if (info.val_exp >= kUneven) {
                                sums = uneven_tile<D>(sums, info, down[k % kInfo], s_at, o_at, i == 0, &shrunk[r], token, lo,
                                                      hi);
                                tmem_wait_st();
                                tc::tc_fence_before();
                                tc::mbar_arrive(&p_full[m]);
                                continue;
                            }
                            change_sums<D>(sums, high, info, o_at, i == 0, shrunk[r]);
                        }
                        sums.total += edge ? tile_weights<true>(sums, info.key_exp, s_at, token, lo, hi)
                                           : tile_weights<false>(sums, info.key_exp, s_at, token, lo, hi);
                        tmem_wait_st();
                    }
                    tc::tc_fence_before();
                    tc::mbar_arrive(&p_full[m]);
                }
                // (set, if at all, before the exponents of the tile that were waited for)
                if (*reinterpret_cast<volatile int*>(&met_not_finite) && row.live &&
                    sees_not_finite<BITS>(p, c, max(lo, first), min(hi, first + n * kTile - 1)))
                    sums.total = NAN;
            }
            if (begins && !ends) {
                split = true;
                if (threadIdx.x == 0) {
                    KvSplitItem it;
                    it.q_row = c.seq.q0;
                    it.row0 = c.rb * kRows;
                    it.rows = min(kRows, c.seq.nq * p.G - it.row0);
                    it.h = c.h;
                    it.last_cta = kv_owner(range, c.at + kCost + c.span.tiles - 1, blockIdx.x);
                    it.pad = 0;
                    p.split[blockIdx.x] = it;
                }
            }
            // the next item's Q and its first products, before this one's results are written
            kt += n;
            __syncwarp();
            if (lane == 0) kv_next_item<kRows, kTile, kCost>(p, c);
            __syncwarp();
            Row next = {};
            n = kv_take<kCost>(p, c, range.end);
            if (n > 0) take_up(next);
            if (row.active) {
                wait(&o_full[m], items & 1);
                ++items;
                tc::tc_fence_after();
            }
            if (row.active && !dead) {
                const float back = pow2(sums.val_exp - 134);
                const float by = begins && ends ? (sums.total == 0.0f ? 0.0f : back / sums.total) : back;
                const int64_t slot = ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * kRows + r;
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t v[32];
                    __syncwarp();
                    tmem_ld32(o_at + q * 32, v);
                    tc::tmem_wait_ld();
                    float x[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = by == 0.0f ? 0.0f : __uint_as_float(v[j]) * by;
                    if (!row.live) {
                    } else if (begins && ends) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
                            *reinterpret_cast<uint4*>(p.out + row.out + q * 32 + j) =
                                make_uint4(pack_bf16(x[j], x[j + 1]), pack_bf16(x[j + 2], x[j + 3]),
                                           pack_bf16(x[j + 4], x[j + 5]), pack_bf16(x[j + 6], x[j + 7]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<float4*>(p.part_o + slot * D + q * 32 + j) =
                                make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                    }
                }
                if (row.live && !(begins && ends))
                    *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(sums.top / shrunk[r], sums.total);
            }
            row = next;
        }
        if (threadIdx.x == 0 && p.split != nullptr && !split) p.split[blockIdx.x].rows = 0;
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

template <int D, int BITS>
cudaError_t launch_form(const KvAttnParams& p, int64_t ctas, const LaunchEnv& env) {
    using C = Cfg<D, BITS>;
    static_assert(C::kSmem <= 227 * 1024 - 6144, "shared memory of a block");
    const cudaError_t e = allow_smem<kv_prompt_kernel<D, BITS>>(C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kv_prompt_kernel<D, BITS>, dim3((unsigned)ctas), dim3(kThreads), C::kSmem, env.stream,
                         kNoCluster, p);
}

}  // namespace

cudaError_t launch_kv_prompt(const KvAttnParams& p, int64_t D, int64_t bits, int64_t ctas, const LaunchEnv& env) {
    if (D == 64) return bits == 4 ? launch_form<64, 4>(p, ctas, env) : launch_form<64, 8>(p, ctas, env);
    return bits == 4 ? launch_form<128, 4>(p, ctas, env) : launch_form<128, 8>(p, ctas, env);
}

}  // namespace i8ql
