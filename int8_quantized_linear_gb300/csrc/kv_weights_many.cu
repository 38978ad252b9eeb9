// Attention weights summed per cached token, for many query rows (prompts): the
// same two passes as kv_weights.cu on the tensor cores proper (tcgen05,
// accumulators in TMEM).
//
// A block (one per SM) holds 256 query rows of one cache head (query tokens x the
// head group's heads) as two operand tiles of 128, and walks the cache in tiles of
// 128 tokens, which become fp16 operands once for both:
//   first pass:   S = Q K^T  (rows x tokens), a thread a row: its maximum and sum
//   second pass:  S^T = K Q^T  (tokens x rows), a thread a token: the sum of its weights
// so that neither needs a shuffle; the operand tiles are the same, only their roles
// in the product change.
//
// What a column of S needs of its own would come from shared memory, whose reads give
// each lane 4 bytes a cycle even where all read the same: a number per column costs
// as much as the exponential.  So scale and low value are inside the product, without
// rounding what they scale: with x = low + s c of 4-bit codes
//   x = s (c - 8) + o,   o = low + 8 s
// s (c - 8) has 8 + 3 bits, which fp16 holds exactly, and o meets only the sum of the
// row's q, so both go into 16 channels more, as sums of two fp16 numbers each (o_hi q_hi +
// o_hi q_lo + o_lo q_hi: 2^-22 of o sum q).  A byte is two such nibbles,
//   low + s c = 16 s (c_hi - 8) + s (c_lo - 8) + low + 136 s,
// products with the same q.  (With the scales outside the products instead, as two and
// three numbers a column, two chunks of 2048 tokens over 8192 took 970 us.)
// A tile is held times the power of two that brings its largest element to 2^7: tokens
// 2^21 below it lose bits.  A row of Q is scaled to 2^14 (first pass) or its 16 rows
// together are (second pass, where rows are columns: rows 2^14 below the largest of
// their 16 keep 2^-25 of it).  In the second pass a row's maximum and sum are
// one number, n_i = m_i + log2 l_i, rounded to 2^-24 of it, while no maximum of its half
// exceeds kNear.
//
// Large logits: a row's sum is relative to a reference r, an fp32 number near its maximum, and
// an exponent is taken in one step, c x - r with the product not rounded.  So both passes mean
// the same by it, but the largest exponent is not 0: it is what r was rounded by, which a sum
// has room for up to logits of 2^28.  Beyond, a row is far: r is the largest of its products
// q k themselves, which is taken off the others before the scale is multiplied in, so that the
// largest has the exponent 0, however large it is.  Tiles where logits could come near that
// (their exponents say so), and halves with large maxima in the second pass, go through
// functions of their own.  (The question costs the first pass up to 2 %.)
//
// The second pass leaves sums over up to 128-row halves of a group of row blocks per
// token in a workspace (a thread adds to its own place, in order), and a third kernel
// adds those up: no atomics, the same bits whatever the timing.
//
// Two chunks of 2048 tokens over 8192 (32 query heads, 8 cache heads, 128 channels, 4 bits):
// 311 and 374 us and 7 for the joining, 243 GFLOP a pass, 780 and 650 TFLOP/s.  Bound by
// the roles together: the products alone (nothing unpacked, no softmax) take 240 us a
// pass, the softmax alone 221 and 283.  Measured and dropped: 256 rows a product in the
// second pass (397 against 374 us), three stages with 8 warps unpacking every tile and
// one for the exponents (343 and 396).
//
// Roles: 16 softmax warps, a set of 8 for the even steps and one for the odd ones, each
// four warps for a half; 8 warps unpack codes into the swizzled operand tiles, four the
// even tiles and four the odd ones (128 channels of 8 bits: one tile fits, and four warps
// unpack them all); one copies pages, one issues the MMAs.  S is held twice per half (all
// 512 columns of TMEM): a set works on one step's while the other's products run.  Operand
// layout: K-major, 128-byte swizzle, channels in the order in which key words unpack.

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "kv_tc.cuh"
#include "kv_weights.cuh"

namespace i8ql {
namespace {

constexpr int kTile = kKvPromptTile;  // cache tokens per tile
constexpr int kRows = kKvPromptRows;  // query rows per block: two halves
constexpr int kSoftmaxWarps = 16;
constexpr int kUnpackWarps = 4;  // of a group; one works on the even tiles, one on the odd
constexpr int kCopyWarp = kSoftmaxWarps + 2 * kUnpackWarps;
constexpr int kMmaWarp = kCopyWarp + 1;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kInfo = 4;       // tiles whose exponents are kept
constexpr float kSlack = 8.0f; // a row's maximum may exceed what its sum is relative to by this (log2)

template <int D, int BITS>
struct Cfg {
    static constexpr int kRowBytes = D * BITS / 8;
    static constexpr int kNibbles = BITS / 4;
    // Unpacked tiles, and raw ones: even numbers, of which each unpacking group has its own
    // (a group that skipped rounds of a barrier could not tell them apart), or one, with one group.
    static constexpr int kStages = D == 128 && BITS == 8 ? 1 : 2;
    static constexpr int kRaw = D == 128 && BITS == 8 ? 2 : 4;
    static constexpr int kPart = kTile * D * 2;
    static constexpr int kKTile = kNibbles * kPart;
    // the 16 channels more: a swizzle atom's 64 channels hold those of four tiles, or of both halves of Q
    static constexpr int kMore = kTile * 128;
    static constexpr int kRawBytes = kTile * kRowBytes + kTile * 4;
    static constexpr int kOffQ = 0;  // [halves]
    static constexpr int kOffMoreQ = kOffQ + 2 * kPart;
    static constexpr int kOffK = kOffMoreQ + kMore;
    static constexpr int kOffMoreK = kOffK + kStages * kKTile;
    static constexpr int kOffRaw = kOffMoreK + kMore;
    // (at least what keeps a second block, which would wait for TMEM, off the SM)
    static constexpr int kSmem = std::max(kOffRaw + kRaw * kRawBytes + 1024, 116 * 1024);
};

// The work of a block: row blocks rb0 .. rb1 - 1 of a head of a sequence, over the
// tiles that it is given of those that they see.
struct Work {
    int64_t b;
    int h;
    int part;  // SUM: group of row blocks; else: which part of the tiles
    int chunk0, chunk1;  // SUM: tiles
    KvSeq seq;
    int rb0, rb1;
};

__device__ __forceinline__ KvSeq many_sequence(const KvWeightsParams& p, int64_t b) {
    KvSeq s = kv_sequence(p.a, b);
    if (s.nq > p.max_q) {
        record_fault(p.a.err, kErrBitBadIndex);
        s.nq = (int32_t)p.max_q;
    }
    return s;
}

template <bool SUM>
__device__ __forceinline__ Work find_work(const KvWeightsParams& p) {
    Work w;
    int64_t at = blockIdx.x;
    if constexpr (SUM) {
        const int chunk = (int)(at % p.chunks);
        at /= p.chunks;
        w.chunk0 = chunk * p.chunk;
    } else {
        w.part = (int)(at % p.splits);
        at /= p.splits;
    }
    w.h = (int)(at % p.a.cache.H);
    at /= p.a.cache.H;
    if constexpr (SUM) {
        // (late rows see most: first, of all sequences; 8192 tokens over themselves 474 us with
        // the early rows first, 420 so)
        w.part = p.groups - 1 - (int)(at / p.a.B);
        w.b = at % p.a.B;
        w.seq = many_sequence(p, w.b);
        const int blocks = kv_blocks<kRows>(p.a, w.seq);
        w.rb0 = (int)((int64_t)blocks * w.part / p.groups);
        w.rb1 = (int)((int64_t)blocks * (w.part + 1) / p.groups);
        w.chunk1 = min(w.chunk0 + p.chunk, (w.seq.len + kTile - 1) / kTile);
        if (w.chunk1 <= w.chunk0 || w.seq.nq == 0) w.rb0 = w.rb1 = w.chunk1 = 0;
    } else {
        // (late rows see most: first)
        const int64_t blocks_all = (p.max_q * p.a.G + kRows - 1) / kRows;
        w.b = at / blocks_all;
        w.seq = many_sequence(p, w.b);
        w.rb0 = (int)(blocks_all - 1 - at % blocks_all);
        w.rb1 = min(w.rb0 + 1, kv_blocks<kRows>(p.a, w.seq));
        w.chunk0 = w.chunk1 = 0;
    }
    return w;
}

// Row block rb's rows and tiles t0 .. t1 - 1 of the block's work.
struct Part {
    KvSpan span;
    int row0, rows;
    int t0, t1;
};

template <bool SUM>
__device__ __forceinline__ Part find_part(const KvWeightsParams& p, const Work& w, int rb) {
    Part r;
    r.span = kv_span<kRows, kTile>(p.a, w.seq, rb);
    r.row0 = rb * kRows;
    r.rows = min(kRows, w.seq.nq * p.a.G - r.row0);
    const int end = r.span.begin < r.span.end ? r.span.first + r.span.tiles : r.span.first;
    if constexpr (SUM) {
        r.t0 = max(r.span.first, w.chunk0);
        r.t1 = min(end, w.chunk1);
    } else {
        const int tiles = end - r.span.first;
        r.t0 = r.span.first + (int)((int64_t)tiles * w.part / p.splits);
        r.t1 = r.span.first + (int)((int64_t)tiles * (w.part + 1) / p.splits);
    }
    return r;
}

// A row's sum so far, relative to 2^ref; nothing yet: ref is -inf.  A negative sum: of a far
// row, whose ref is a product q k.
struct RowStats {
    float ref, sum;
};
constexpr float kNear = 4096.0f;
constexpr float kFar = 0x1p28f;
// Of a row's unit and a tile whose exponents add up to no more, what S counts is below 2^-6, and S
// is below 2^32 (128 channels of 2^15 x 2^8, and as much for the offsets): logits below 2^26.
constexpr int kFarExp = 127 + 127;
constexpr float kMostFloat = 3.402823466e38f;

// Products off by a power of two, 2^shift (|shift| <= 252), as they are, or the largest number.
struct Shift {
    float a, b;
    __device__ __forceinline__ explicit Shift(int shift) : a(pow2(shift >> 1)), b(pow2(shift - (shift >> 1))) {}
    __device__ __forceinline__ float operator()(uint32_t x) const {
        return fminf(fmaxf(__uint_as_float(x) * a * b, -kMostFloat), kMostFloat);
    }
};

// A reference is far scale + near.
__device__ __forceinline__ float far_part(const RowStats& r) { return r.sum < 0.0f ? r.ref : 0.0f; }
__device__ __forceinline__ float near_part(const RowStats& r) { return r.sum < 0.0f ? 0.0f : r.ref; }

// A row's sum over two sets of tokens.
__device__ __forceinline__ RowStats join_rows(const RowStats& a, const RowStats& b, float scale) {
    if (b.ref == -INFINITY) return a;
    if (a.ref == -INFINITY) return b;
    const float d = fmaf(far_part(b) - far_part(a), scale, near_part(b) - near_part(a));
    const RowStats high = d > 0.0f ? b : a, low = d > 0.0f ? a : b;
    return {high.ref, copysignf(fmaf(fabsf(low.sum), exp2_approx(-fabsf(d)), fabsf(high.sum)), high.sum)};
}

// Raises a row's reference to the maximum.
__device__ __forceinline__ void raise(RowStats& r, float to) {
    r.sum *= r.ref == -INFINITY ? 0.0f : exp2_approx(r.ref - to);
    r.ref = to;
}

// A tile of S of a row that sees all its tokens.  The exponents are relative to what the
// sum is: where one exceeds the slack (rare: the first time, and then as larger logits
// come), the reference is raised and all is done again.  Once: what a reference is rounded by
// would exceed the slack from 2^28 on, however often that is done.  (Asked once a tile: a vote
// after every 32 columns keeps the next ones from being loaded, 295 against 221 us for
// the softmax alone of two chunks of 2048 tokens over 8192.)
__device__ __forceinline__ void add_tokens(RowStats& r, uint32_t s_at, float unit) {
    const uint64_t u2 = pair_f32(unit, unit);
#pragma unroll 1
    for (bool first = true;; first = false) {
        const float ref = r.ref == -INFINITY ? 0.0f : -r.ref;
        const uint64_t ref2 = pair_f32(ref, ref);
        uint64_t sum[2] = {0, 0};
        float high[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
        for (int q = 0; q < kTile / 32; ++q) {
            uint32_t x[32];
            tmem_ld32(s_at + q * 32, x);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                float y, z;
                split_f32(fma_f32x2(pair_u32(x[j], x[j + 1]), u2, ref2), y, z);
                high[(j / 2) & 1] = max3(high[(j / 2) & 1], y, z);
                sum[(j / 2) & 1] = add_f32x2(sum[(j / 2) & 1], pair_f32(exp2_approx(y), exp2_approx(z)));
            }
        }
        const float top = fmaxf(high[0], high[1]);
        const bool again = first && (r.ref == -INFINITY || top > kSlack);
        if (!__any_sync(0xffffffffu, again)) {
            float a, b;
            split_f32(add_f32x2(sum[0], sum[1]), a, b);
            r.sum += a + b;
            return;
        }
        if (again) raise(r, top - ref);
    }
}

// A tile of a warp with far rows, or whose logits could make some: products off by 2^shift,
// of which the row sees lo .. hi.
__device__ __noinline__ RowStats add_far_tokens(RowStats r, uint32_t s_at, int shift, float scale, int token, int lo, int hi) {
    const Shift product(shift);
    float top = -INFINITY;
#pragma unroll 1
    for (int q = 0; q < kTile / 32; ++q) {
        uint32_t x[32];
        tmem_ld32(s_at + q * 32, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int tok = token + q * 32 + j;
            top = tok <= hi && tok >= lo ? fmaxf(top, product(x[j])) : top;
        }
    }
    float far = far_part(r), near = near_part(r), sum = fabsf(r.sum);
    if (top > -INFINITY && (r.ref == -INFINITY || fmaf(top - far, scale, -near) > 0.0f)) {
        const float logit = top * scale;
        const bool large = !(fabsf(logit) < kFar);
        const float to_far = large ? top : 0.0f, to_near = large ? 0.0f : logit;
        sum = r.ref == -INFINITY ? 0.0f : sum * exp2_approx(fmaf(far - to_far, scale, near - to_near));
        far = to_far;
        near = to_near;
    }
    __syncwarp();
#pragma unroll 1
    for (int q = 0; q < kTile / 32; ++q) {
        uint32_t x[32];
        tmem_ld32(s_at + q * 32, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int tok = token + q * 32 + j;
            sum += tok <= hi && tok >= lo ? exp2_approx(fmaf(product(x[j]) - far, scale, -near)) : 0.0f;
        }
    }
    return far != 0.0f ? RowStats{far, -sum} : RowStats{near, sum};
}

// A tile where some row does not see some token: this one sees lo .. hi.
__device__ __noinline__ RowStats add_some_tokens(RowStats r, uint32_t s_at, float unit, int token, int lo, int hi) {
#pragma unroll 1
    for (int q = 0; q < kTile / 32; ++q) {
        uint32_t x[32];
        tmem_ld32(s_at + q * 32, x);
        tc::tmem_wait_ld();
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int tok = token + q * 32 + j;
            x[j] = __float_as_uint(tok <= hi && tok >= lo ? __uint_as_float(x[j]) : -INFINITY);
            top = fmaxf(top, __uint_as_float(x[j]));
        }
        top = top > -INFINITY ? top * unit : top;
        if (top > r.ref + kSlack || (r.ref == -INFINITY && top > -INFINITY)) raise(r, top);
        const float ref = r.ref == -INFINITY ? 0.0f : -r.ref;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float v = __uint_as_float(x[j]);
            sum += v > -INFINITY ? exp2_approx(fmaf(v, unit, ref)) : 0.0f;
        }
        r.sum += sum;
    }
    return r;
}

// What the softmax needs of a half's rows: what a product counts (in log2 units, times
// the tile's), where rows are columns -n, and the last token that the row sees; for large
// logits what products are off by, as a power of two, and n in its parts.
constexpr int kGroup = 16;  // rows that share a unit where they are columns: those a warp takes up
struct RowFactors {
    float unit[kTile], minus_n[kTile];
    int hi[kTile], shift[kTile];
    float far[kTile], near[kTile], minus_log[kTile];
};

// The sum of 32 rows' weights of a token.
template <bool EDGE>
__device__ __forceinline__ void add_rows(uint64_t (&sum)[2], uint32_t s_at, const RowFactors& f, int c0, float unit, int token,
                                         int64_t window) {
    uint32_t x[32];
    tmem_ld32(s_at, x);
    tc::tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        const float u = f.unit[c0 + j / kGroup * kGroup] * unit;
        const uint64_t u2 = pair_f32(u, u);
        const ulonglong2 n = *reinterpret_cast<const ulonglong2*>(f.minus_n + c0 + j);
        float v[4];
        split_f32(fma_f32x2(pair_u32(x[j], x[j + 1]), u2, n.x), v[0], v[1]);
        split_f32(fma_f32x2(pair_u32(x[j + 2], x[j + 3]), u2, n.y), v[2], v[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = exp2_approx(v[k]);
            if (EDGE) {
                const int hi = f.hi[c0 + j + k];
                v[k] = token <= hi && (window == 0 || token > hi - window) ? v[k] : 0.0f;
            }
        }
        sum[0] = add_f32x2(sum[0], pair_f32(v[0], v[1]));
        sum[1] = add_f32x2(sum[1], pair_f32(v[2], v[3]));
    }
}

// The sum of all rows' weights of a token in a half with large maxima, its tile's products off
// by 2^shift.  (No weight exceeds 1: a product may come out above the largest of the
// first pass where its row has lost bits.)
__device__ __noinline__ float add_far_rows(uint32_t s_at, const RowFactors& f, int columns, int shift, float scale, int token,
                                           int64_t window) {
    float sum = 0.0f;
#pragma unroll 1
    for (int c0 = 0; c0 < columns * 32; c0 += 32) {
        uint32_t x[32];
        tmem_ld32(s_at + c0, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const Shift product(f.shift[c0 + j / kGroup * kGroup] + shift);
            const int hi = f.hi[c0 + j];
            const float v = fmaf(product(x[j]) - f.far[c0 + j], scale, -f.near[c0 + j]) + f.minus_log[c0 + j];
            sum += token <= hi && (window == 0 || token > hi - window) ? exp2_approx(fminf(v, 0.0f)) : 0.0f;
        }
    }
    return sum;
}

// fp16 parts of x: x = hi + lo but for 2^-22 of it.
__device__ __forceinline__ void split_f16(float x, uint32_t& hi, uint32_t& lo) {
    const __half h = __float2half_rn(x);
    hi = __half_as_ushort(h);
    lo = __half_as_ushort(__float2half_rn(x - __half2float(h)));
}

template <int D, int BITS, bool SUM>
__global__ void __launch_bounds__(kThreads, 1) kv_weights_many_kernel(const KvWeightsParams p) {
    using C = Cfg<D, BITS>;
    constexpr int kStages = C::kStages, kRaw = C::kRaw;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t raw_full[kRaw], raw_empty[kRaw], k_full[kStages], k_empty[kStages];
    __shared__ uint64_t q_full[2], s_full[2][2], s_empty[2][2], info_full[kInfo], drained;
    __shared__ __align__(16) uint32_t exp_red[2][kUnpackWarps];  // largest magnitudes, as bits
    __shared__ int tile_exp[kInfo];        // a tile is held times 2^(134 - tile_exp)
    __shared__ uint32_t factors[2][kTile];  // a token's scale, twice, as halves
    __shared__ __align__(16) RowFactors row_factors[2];
    __shared__ __align__(16) int large_rows[2][4];  // SUM: which warps' rows have large maxima among them
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t smem_at = tc::smem_u32(smem);
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < kRaw; ++i) {
            tc::mbar_init(&raw_full[i], 1);
            tc::mbar_init(&raw_empty[i], kUnpackWarps);
        }
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&k_full[i], kUnpackWarps * 32);
            tc::mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&q_full[i], 256);
            for (int j = 0; j < 2; ++j) {
                tc::mbar_init(&s_full[i][j], 1);
                tc::mbar_init(&s_empty[i][j], 128);
            }
        }
        for (int i = 0; i < kInfo; ++i) tc::mbar_init(&info_full[i], kUnpackWarps);
        tc::mbar_init(&drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    if (warp == kMmaWarp) tc::tmem_alloc(&tmem_base, 512);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_base;
    const Work work = find_work<SUM>(p);
    bool dead = false;
    // Waits of a whole warp; after one that gave up no work is done any more,
    // but every loop and barrier runs to its end.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (dead || __all_sync(0xffffffffu, tc::mbar_test(tc::smem_u32(bar), parity))) return;
        dead = !tc::warp_wait(bar, parity, &abort_flag, p.a.err);
    };

    if (warp == kCopyWarp) {
        // ------------------------------------------------------------ copies
        const int page_tokens = 1 << p.a.cache.page_shift;
        const int piece = min(page_tokens, kTile);
        const int is_param = lane & 1;
        const int at = (lane >> 1) * piece;
        const int32_t* table = p.a.table + work.b * p.a.table_width;
        uint32_t kt = 0;
        for (int rb = work.rb0; rb < work.rb1 && !dead; ++rb) {
            const Part r = find_part<SUM>(p, work, rb);
            auto needed = [&](int tile) {
                const int token = tile * kTile + at;
                return tile < r.t1 && at < kTile && token < r.span.end && token + piece > r.span.begin;
            };
            auto page_of = [&](int tile) {
                return needed(tile) ? __ldg(table + ((tile * kTile + at) >> p.a.cache.page_shift)) : 0;
            };
            int32_t ahead[2] = {page_of(r.t0), page_of(r.t0 + 1)};
            for (int tile = r.t0; tile < r.t1 && !dead; ++tile) {
                const bool need = needed(tile);
                int64_t page = ahead[0];
                ahead[0] = ahead[1];
                ahead[1] = page_of(tile + 2);
                const uint32_t slot = kt % kRaw;
                const unsigned pieces = __popc(__ballot_sync(0xffffffffu, need)) / 2;
                wait(&raw_empty[slot], ((kt / kRaw) & 1) ^ 1);
                // (an unpacking warp that gave up says so before it frees raw tiles that it
                // did not wait for, whose copies may still be on their way)
                dead = dead || __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&abort_flag));
                if (dead) break;
                if (lane == 0) tc::mbar_expect_tx(&raw_full[slot], pieces * piece * (C::kRowBytes + 4));
                __syncwarp();
                if (need) {
                    if (page < 0 || page >= p.a.cache.pages) {
                        record_fault(p.a.err, kErrBitBadIndex);
                        page = 0;
                    }
                    const int64_t row = kv_row(p.a.cache, page, 0, work.h, (tile * kTile + at) & (page_tokens - 1));
                    uint8_t* raw = smem + C::kOffRaw + slot * C::kRawBytes;
                    if (is_param)
                        bulk_load(raw + kTile * C::kRowBytes + at * 4, p.a.cache.params + row, piece * 4, &raw_full[slot]);
                    else
                        bulk_load(raw + at * C::kRowBytes, p.a.cache.codes + row * C::kRowBytes, piece * C::kRowBytes,
                                  &raw_full[slot]);
                }
                ++kt;
            }
        }
        // the last copies land before the block's shared memory can go to another
        int none = 0;
        for (uint32_t k = kt > kRaw ? kt - kRaw : 0; k < kt; ++k)
            tc::mbar_wait(&raw_full[k % kRaw], (k / kRaw) & 1, &none, p.a.err);
    } else if (warp >= kSoftmaxWarps && warp < kCopyWarp) {
        // ------------------------------------------------------------ unpacking
        const int tid = threadIdx.x & 127;
        const int w4 = warp % kUnpackWarps;
        const uint32_t group = (warp - kSoftmaxWarps) / kUnpackWarps;
        auto unpack_sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(group * 3 + 1), "n"(kUnpackWarps * 32) : "memory"); };
        uint32_t* const factor = factors[group];
        constexpr int kLanesPerKey = C::kRowBytes / 16;
        constexpr int kChunks = BITS == 4 ? 4 : 2;  // operand chunks (8 channels) per 16 raw bytes
        constexpr float kMiddle = BITS == 4 ? 8.0f : 136.0f;  // what the products leave of a code
        constexpr float kTop = BITS == 4 ? 8.0f : 128.0f;     // the largest of what they have, in scales
        const int key_lane = tid % kLanesPerKey;
        // of a tile's 16 channels more the second eight stay 0
        for (int i = (int)group; i < kStages; i += 2)
            sts16(smem_at + C::kOffMoreK + tid * 128 + (((2 * i + 1) ^ (tid & 7)) << 4), 0, 0, 0, 0);
        uint32_t kt = 0;
        for (int rb = work.rb0; rb < work.rb1; ++rb) {
            const Part r = find_part<SUM>(p, work, rb);
            for (int tile = r.t0; tile < r.t1; ++tile, ++kt) {
                if (group != (kStages == 1 ? 0 : kt % 2)) continue;
                const int token = tile * kTile;
                const uint32_t slot = kt % kRaw, stage = kt % kStages;
                const uint8_t* raw = smem + C::kOffRaw + slot * C::kRawBytes;
                wait(&raw_full[slot], (kt / kRaw) & 1);
                // the tile's exponent: of its largest scaled code, and of its largest offset
                uint32_t pk = 0;
                if (!dead && token + tid >= r.span.begin && token + tid < r.span.end)
                    pk = reinterpret_cast<const uint32_t*>(raw + kTile * C::kRowBytes)[tid];
                const float offset = fmaf(kv_scale(pk), kMiddle, kv_low(pk));
                const uint32_t bits = max(__float_as_uint(kv_scale(pk) * kTop) & 0x7fffffffu, __float_as_uint(offset) & 0x7fffffffu);
                const uint32_t top = __reduce_max_sync(0xffffffffu, bits < 0x7f800000u ? bits : 0u);
                if (lane == 0) exp_red[group][w4] = top;
                unpack_sync();  // (and the group's tile before is done with its factors)
                const uint4 tops = *reinterpret_cast<const uint4*>(exp_red[group]);
                const uint32_t e = max(max(max(tops.x, tops.y), max(tops.z, tops.w)) >> 23, 8u);
                const float f = __uint_as_float((261u - e) << 23);  // 2^(134 - e)
                factor[tid] = pack_f16(kv_scale(pk) * f, kv_scale(pk) * f);
                // this stage's last products are done: so is the softmax of four tiles ago
                wait(&k_empty[stage], ((kt / kStages) & 1) ^ 1);
                if (tid == 0) tile_exp[kt % kInfo] = (int)e;
                unpack_sync();
                if (lane == 0) tc::mbar_arrive(&info_full[kt % kInfo]);
                if (!dead) {
                    const uint32_t dst = smem_at + C::kOffK + stage * C::kKTile;
                    {
                        uint32_t o_hi, o_lo;
                        split_f16(offset * f * 128.0f, o_hi, o_lo);
                        sts16(smem_at + C::kOffMoreK + tid * 128 + (((2 * stage) ^ (tid & 7)) << 4), o_hi | o_hi << 16, o_lo, 0, 0);
                    }
#pragma unroll 1
                    for (int i = 0; i < kLanesPerKey; ++i) {
                        const int tok = tid / kLanesPerKey + i * (kTile / kLanesPerKey);
                        uint32_t w[4];
                        lds<4>(raw + tok * C::kRowBytes + key_lane * 16, w);
                        const uint32_t scale = factor[tok];
                        const int chunk0 = key_lane * kChunks;  // of the row's D / 8
                        const int block = chunk0 / 8, pos0 = chunk0 % 8;
                        const int flip = block & 1;  // lanes of the two blocks take their chunks in opposite order (banks)
                        const uint32_t row = dst + block * (kTile * 128) + tok * 128;
                        auto scaled = [&](uint32_t v) { return fma_f16x2(v, scale, 0x80008000u); };  // (exact; -0: a product)
#pragma unroll
                        for (int j = 0; j < kChunks; ++j) {
                            const uint32_t at = row + (((pos0 + (j ^ flip)) ^ (tok & 7)) << 4);
                            if constexpr (BITS == 4) {
                                uint32_t h[4];
                                unpack_nibbles<true>(flip ? w[j ^ 1] : w[j], h);
                                sts16(at, scaled(h[0]), scaled(h[1]), scaled(h[2]), scaled(h[3]));
                            } else {
                                // of 8 channels (0,2) (1,3) (4,6) (5,7): low nibbles, and 16 times the high ones
                                uint32_t lo[4], hi[4];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const uint32_t v = flip ? w[2 * (j ^ 1) + k] : w[2 * j + k], u = v >> 8;
                                    lo[2 * k] = sub_f16x2(and_or(v, 0x000f000fu, 0x64006400u), 0x64086408u);  // 1024 + c - 1032
                                    lo[2 * k + 1] = sub_f16x2(and_or(u, 0x000f000fu, 0x64006400u), 0x64086408u);
                                    hi[2 * k] = sub_f16x2(and_or(v, 0x00f000f0u, 0x64006400u), 0x64806480u);  // 1024 + 16 c - 1152
                                    hi[2 * k + 1] = sub_f16x2(and_or(u, 0x00f000f0u, 0x64006400u), 0x64806480u);
                                }
                                sts16(at, scaled(lo[0]), scaled(lo[1]), scaled(lo[2]), scaled(lo[3]));
                                sts16(at + C::kPart, scaled(hi[0]), scaled(hi[1]), scaled(hi[2]), scaled(hi[3]));
                            }
                        }
                    }
                    tc::fence_proxy_async_smem();
                }
                tc::mbar_arrive(&k_full[stage]);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&raw_empty[slot]);
            }
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMAs
        const uint32_t q_base = (uint32_t)tc::sw128_desc(smem_at + C::kOffQ);
        const uint32_t k_base = (uint32_t)tc::sw128_desc(smem_at + C::kOffK);
        const uint32_t more_q = (uint32_t)tc::sw128_desc(smem_at + C::kOffMoreQ);
        const uint32_t more_k = (uint32_t)tc::sw128_desc(smem_at + C::kOffMoreK);
        const uint32_t high = (uint32_t)(tc::sw128_desc(smem_at) >> 32), idesc = tc::f16_idesc(kTile);
        // All channels of a half and a stage's tile.
        auto product = [&](uint32_t d, uint32_t m, uint32_t stage, uint32_t issue) {
            const uint32_t q = q_base + m * (C::kPart / 16), k = k_base + stage * (C::kKTile / 16);
            const uint32_t a = SUM ? k : q, b = SUM ? q : k;
            constexpr int kNext = 128 * 128 / 16;  // the second 64 channels
            constexpr int kHigh = C::kPart / 16;   // the high nibbles, beside the same Q
            constexpr int A = SUM ? kHigh : 0, B = SUM ? 0 : kHigh;
            __syncwarp();
            mma_ss<0, 0>(d, a, b, high, idesc, 0, issue);
            mma_ss<2, 2>(d, a, b, high, idesc, 1, issue);
            mma_ss<4, 4>(d, a, b, high, idesc, 1, issue);
            mma_ss<6, 6>(d, a, b, high, idesc, 1, issue);
            if constexpr (D == 128) {
                mma_ss<kNext, kNext>(d, a, b, high, idesc, 1, issue);
                mma_ss<kNext + 2, kNext + 2>(d, a, b, high, idesc, 1, issue);
                mma_ss<kNext + 4, kNext + 4>(d, a, b, high, idesc, 1, issue);
                mma_ss<kNext + 6, kNext + 6>(d, a, b, high, idesc, 1, issue);
            }
            if constexpr (BITS == 8) {
                mma_ss<A, B>(d, a, b, high, idesc, 1, issue);
                mma_ss<A + 2, B + 2>(d, a, b, high, idesc, 1, issue);
                mma_ss<A + 4, B + 4>(d, a, b, high, idesc, 1, issue);
                mma_ss<A + 6, B + 6>(d, a, b, high, idesc, 1, issue);
                if constexpr (D == 128) {
                    mma_ss<A + kNext, B + kNext>(d, a, b, high, idesc, 1, issue);
                    mma_ss<A + kNext + 2, B + kNext + 2>(d, a, b, high, idesc, 1, issue);
                    mma_ss<A + kNext + 4, B + kNext + 4>(d, a, b, high, idesc, 1, issue);
                    mma_ss<A + kNext + 6, B + kNext + 6>(d, a, b, high, idesc, 1, issue);
                }
            }
            const uint32_t mq = more_q + 2 * m, mk = more_k + 2 * stage;
            mma_ss<0, 0>(d, SUM ? mk : mq, SUM ? mq : mk, high, idesc, 1, issue);
        };
        // (Every step of half 0 is a tile, and so is every one of half 1, which only the last
        // row block may leave out: the tile's number says all.)
        uint32_t kt = 0, item = 0;
        for (int rb = work.rb0; rb < work.rb1; ++rb) {
            const Part r = find_part<SUM>(p, work, rb);
            if (r.t0 >= r.t1) continue;
            const bool both = r.rows > 128;
            wait(&q_full[0], item & 1);
            if (both) wait(&q_full[1], item & 1);
            ++item;
            // A half that sits out is done with its last tiles (one of each set), whose
            // exponents the tiles to come would overwrite (one that takes part says so with its Q).
            for (uint32_t i = 1; !both && i <= min(kt, 2u); ++i) wait(&s_empty[1][(kt - i) & 1], ((kt - i) / 2) & 1);
            for (int tile = r.t0; tile < r.t1; ++tile, ++kt) {
                const uint32_t stage = kt % kStages, buf = kt % 2, round = (kt / 2) & 1;
                wait(&k_full[stage], (kt / kStages) & 1);
                const uint32_t d = tmem + buf * (2 * kTile);
                wait(&s_empty[0][buf], round ^ 1);
                tc::tc_fence_after();
                product(d, 0, stage, !dead && lane == 0);
                commit_mma(&s_full[0][buf], !dead && lane == 0);
                if (both) {
                    wait(&s_empty[1][buf], round ^ 1);
                    tc::tc_fence_after();
                    product(d + kTile, 1, stage, !dead && lane == 0);
                    commit_mma(&s_full[1][buf], !dead && lane == 0);
                }
                __syncwarp();
                commit_mma(&k_empty[stage], !dead && lane == 0);
            }
        }
        // nothing may be in flight when the TMEM is given back
        if (lane == 0) tc::mma_commit(&drained);
        __syncwarp();
        int none = 0;
        tc::mbar_wait(&drained, 0, &none, p.a.err);
    } else {
        // ------------------------------------------------------------ softmax
        const int set = warp / 8, m = (warp / 4) % 2;  // the steps and the half that the warp works on
        const int r_m = threadIdx.x & 127;             // row of the half
        const uint32_t s_at = tmem + ((uint32_t)((warp % 4) * 32) << 16) + (set * 2 + m) * kTile;
        auto half_sync = [&] { asm volatile("bar.sync %0, 256;" ::"r"(2 + m) : "memory"); };
        RowFactors& rf = row_factors[m];
        uint32_t kt = 0;
        float* part = nullptr;
        if constexpr (SUM) {
            const int64_t row = ((work.b * p.a.cache.H + work.h) * p.groups + work.part) * 2 + m;
            part = p.parts + row * p.part_stride + r_m;
            if (work.rb0 == work.rb1 && set == 0)  // fewer row blocks than groups
                for (int tile = work.chunk0; tile < work.chunk1; ++tile) part[(int64_t)tile * kTile] = 0.0f;
        }
        for (int rb = work.rb0; rb < work.rb1; ++rb) {
            const Part r = find_part<SUM>(p, work, rb);
            const bool active = r.t0 < r.t1 && r.rows > 128 * m;
            if constexpr (SUM) {
                // tiles that the first block does not see begin at 0
                if (rb == work.rb0 && set == 0)
                    for (int tile = work.chunk0; tile < work.chunk1; ++tile)
                        if (!active || tile < r.t0 || tile >= r.t1) part[(int64_t)tile * kTile] = 0.0f;
            }
            const int row_r = m * 128 + r_m;
            const bool live = row_r < r.rows;
            const int base = work.seq.len - work.seq.nq;
            const int i = (r.row0 + (live ? row_r : 0)) / p.a.G;
            const int head = work.h * p.a.G + (r.row0 + (live ? row_r : 0)) - i * p.a.G;
            const int64_t stat = ((work.seq.q0 + i) * ((int64_t)p.a.G * p.a.cache.H) + head) * p.splits;
            const int hi = base + i, lo = p.a.window > 0 ? (int)max(base + i + 1 - p.a.window, (int64_t)0) : 0;
            RowStats stats = {-INFINITY, 0.0f};
            if (active) {
                // The other set may still be at the row block before: its rows' factors, its
                // operand tile (every product of this half is done once its last two steps
                // have been waited for, one by each set) and its sums.
                half_sync();
                {
                    // Rows go into the operand tile, scaled to 2^14, permuted as the keys
                    // unpack: 16 rows a warp, a lane 8 channels of each of kMine of them.
                    constexpr int kLanes = D / 8, kSide = 32 / kLanes, kMine = 16 / kSide;
                    const int first = (set * 4 + warp % 4) * 16, w = lane % kLanes;
                    uint4 v[kMine];
                    uint32_t top[kMine];
#pragma unroll
                    for (int k = 0; k < kMine; ++k) {
                        const int row = r.row0 + m * 128 + first + k * kSide + lane / kLanes;
                        v[k] = make_uint4(0, 0, 0, 0);
                        if (row < r.row0 + r.rows) {
                            const int at = row / p.a.G;
                            v[k] = __ldg(reinterpret_cast<const uint4*>(p.a.q + (work.seq.q0 + at) * p.a.q_stride +
                                                                       (int64_t)(work.h * p.a.G + row - at * p.a.G) * D) + w);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kMine; ++k) {
                        const uint32_t words[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                        top[k] = 0;  // largest finite magnitude, as bits
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t a = words[j] & 0x7fff0000u, b = (words[j] << 16) & 0x7fff0000u;
                            top[k] = max(top[k], max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
                        }
                    }
                    if constexpr (SUM) {  // the group's
#pragma unroll
                        for (int k = 1; k < kMine; ++k) top[0] = max(top[0], top[k]);
                        top[0] = __reduce_max_sync(0xffffffffu, top[0]);
#pragma unroll
                        for (int k = 1; k < kMine; ++k) top[k] = top[0];
                    } else {
#pragma unroll
                        for (int d = 1; d < kLanes; d <<= 1)
#pragma unroll
                            for (int k = 0; k < kMine; ++k) top[k] = max(top[k], __shfl_xor_sync(0xffffffffu, top[k], d));
                    }
#pragma unroll
                    for (int k = 0; k < kMine; ++k) {
                        const int row = first + k * kSide + lane / kLanes;  // of the half
                        const int e = max((int)(top[k] >> 23), 15) - 127;
                        const float f = p.a.scale_log2 < 0.0f ? -pow2(14 - e) : pow2(14 - e);
                        const float y[8] = {lo_bf16(v[k].x) * f, hi_bf16(v[k].x) * f, lo_bf16(v[k].y) * f, hi_bf16(v[k].y) * f,
                                            lo_bf16(v[k].z) * f, hi_bf16(v[k].z) * f, lo_bf16(v[k].w) * f, hi_bf16(v[k].w) * f};
                        float q_sum = ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
#pragma unroll
                        for (int d = 1; d < kLanes; d <<= 1) q_sum += __shfl_xor_sync(0xffffffffu, q_sum, d);
                        const uint32_t at = smem_at + C::kOffQ + m * C::kPart + (w / 8) * (128 * 128) + row * 128 +
                                            (((w & 7) ^ (row & 7)) << 4);
                        if constexpr (BITS == 4)
                            sts16(at, pack_f16(y[0], y[4]), pack_f16(y[1], y[5]), pack_f16(y[2], y[6]), pack_f16(y[3], y[7]));
                        else
                            sts16(at, pack_f16(y[0], y[2]), pack_f16(y[1], y[3]), pack_f16(y[4], y[6]), pack_f16(y[5], y[7]));
                        if (w < 2) {  // of the channels more: the sum's parts, and zeros
                            uint32_t q_hi, q_lo;
                            split_f16(q_sum * 0.0078125f, q_hi, q_lo);
                            sts16(smem_at + C::kOffMoreQ + row * 128 + (((2 * m + w) ^ (row & 7)) << 4), w ? 0 : q_hi | q_lo << 16,
                                  w ? 0 : q_hi, 0, 0);
                        }
                        if (w == 0) {
                            rf.unit[row] = pow2(e - 14) * fabsf(p.a.scale_log2);
                            rf.shift[row] = e - 14;
                        }
                    }
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&q_full[m]);
                    if (SUM && set == 0) {
                        float top_m = -INFINITY, l = 0.0f;
                        bool far = false;
                        if (live) {
#pragma unroll 4
                            for (int s = 0; s < p.splits; ++s) {
                                const float2 x = p.stats[stat + s];
                                far = far || x.y < 0.0f;
                                const float to = fmaxf(top_m, x.x), shift = to == -INFINITY ? 0.0f : to;
                                l = l * exp2_approx(top_m - shift) + x.y * exp2_approx(x.x - shift);
                                top_m = to;
                            }
                        }
                        RowStats all = {top_m, l};
                        if (__any_sync(0xffffffffu, far)) {  // (rare)
                            all = {-INFINITY, 0.0f};
#pragma unroll 1
                            for (int s = 0; live && s < p.splits; ++s) {
                                const float2 x = p.stats[stat + s];
                                all = join_rows(all, RowStats{x.x, x.y}, fabsf(p.a.scale_log2));
                            }
                        }
                        const bool nothing = all.ref == -INFINITY;
                        const float near = nothing ? 0.0f : near_part(all);
                        const float minus_log = nothing ? -INFINITY : -log2f(fabsf(all.sum));
                        rf.minus_n[r_m] = minus_log - near;
                        rf.far[r_m] = far_part(all);
                        rf.near[r_m] = near;
                        rf.minus_log[r_m] = minus_log;
                        const bool large = all.sum < 0.0f || !(fabsf(near) < kNear);
                        const int some_large = __any_sync(0xffffffffu, large);
                        if (lane == 0) large_rows[m][warp % 4] = some_large;
                        rf.hi[r_m] = live ? hi : -1;
                    }
                }
                half_sync();
                const float own_unit = SUM ? 1.0f : rf.unit[r_m];
                // tiles of larger exponents take the functions for large logits: first pass, as the warp's
                // units are (from its first far row on all tiles); second, all where some maximum of the half is large
                int most_exp;
                if constexpr (SUM) {
                    const int4 some = *reinterpret_cast<const int4*>(large_rows[m]);
                    most_exp = (some.x | some.y | some.z | some.w) != 0 ? -1 : 255;
                } else {
                    most_exp = kFarExp - (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(own_unit)) >> 23);
                }
                // tokens [all_lo, all_hi] are seen by every row of the half
                const int all_hi = base + (r.row0 + m * 128) / p.a.G;
                const int last = r.row0 + min(r.rows, m * 128 + 128) - 1;
                const int all_lo = p.a.window > 0 ? (int)max(base + last / p.a.G + 1 - p.a.window, (int64_t)0) : 0;
                const int columns = (min(r.rows - m * 128, 128) + 31) / 32;
                const bool warp_live = SUM || (warp % 4) * 32 < r.rows - m * 128;
                for (int tile = r.t0 + (int)((kt & 1) ^ set); tile < r.t1; tile += 2) {
                    const uint32_t k = kt + (tile - r.t0);
                    const int token = tile * kTile;
                    float before = 0.0f;
                    if constexpr (SUM) {
                        if (rb > work.rb0) before = part[(int64_t)tile * kTile];
                    }
                    // S first: its exponent is there then, so one test of its barrier (whose
                    // earlier rounds this set has not waited for) passes, and acquires it
                    wait(&s_full[m][set], (k / 2) & 1);
                    const bool there = tc::mbar_test(tc::smem_u32(&info_full[k % kInfo]), (k / kInfo) & 1);
                    tc::tc_fence_after();
                    if (!dead && __all_sync(0xffffffffu, there) && warp_live) {
                        const bool edge = token + kTile - 1 > all_hi || token < all_lo;
                        const float unit = own_unit * pow2(tile_exp[k % kInfo] - 134);
                        if constexpr (SUM) {
                            float all;
                            if (__builtin_expect(most_exp < 0, 0)) {
                                all = add_far_rows(s_at, rf, columns, tile_exp[k % kInfo] - 134, fabsf(p.a.scale_log2),
                                                   token + r_m, p.a.window);
                            } else {
                                uint64_t sum[2] = {0, 0};
#pragma unroll 1
                                for (int q = 0; q < columns; ++q) {
                                    if (edge)
                                        add_rows<true>(sum, s_at + q * 32, rf, q * 32, unit, token + r_m, p.a.window);
                                    else
                                        add_rows<false>(sum, s_at + q * 32, rf, q * 32, unit, token + r_m, 0);
                                }
                                float a, b;
                                split_f32(add_f32x2(sum[0], sum[1]), a, b);
                                all = a + b;
                            }
                            part[(int64_t)tile * kTile] = before + all;
                        } else if (__builtin_expect(tile_exp[k % kInfo] > most_exp, 0)) {
                            stats = add_far_tokens(stats, s_at, rf.shift[r_m] + tile_exp[k % kInfo] - 134,
                                                   fabsf(p.a.scale_log2), token, edge ? lo : 0, edge ? hi : INT_MAX);
                            if (__any_sync(0xffffffffu, stats.sum < 0.0f)) most_exp = -1;
                        } else if (edge) {
                            stats = add_some_tokens(stats, s_at, unit, token, lo, hi);
                        } else {
                            add_tokens(stats, s_at, unit);
                        }
                    }
                    tc::tc_fence_before();
                    tc::mbar_arrive(&s_empty[m][set]);
                }
            }
            kt += max(r.t1 - r.t0, 0);
            if constexpr (!SUM) {
                // the two sets' sums of a row
                if (active) half_sync();
                if (set == 1) {
                    rf.unit[r_m] = stats.ref;
                    rf.minus_n[r_m] = stats.sum;
                }
                half_sync();
                if (set == 0 && live) {
                    stats = join_rows(stats, RowStats{rf.unit[r_m], rf.minus_n[r_m]}, fabsf(p.a.scale_log2));
                    p.stats[stat + work.part] = make_float2(stats.ref, stats.sum);
                }
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// weights = previous + the sums over the groups and halves.
__global__ void __launch_bounds__(256) kv_weights_join_kernel(const KvWeightsParams p) {
    const int64_t per = (p.part_stride + 255) / 256;
    const int64_t item = blockIdx.x / per;
    const int64_t j = (blockIdx.x - item * per) * 256 + threadIdx.x;
    const int64_t b = item / p.a.cache.H;
    const int h = (int)(item - b * p.a.cache.H);
    pdl_wait();
    const KvSeq seq = many_sequence(p, b);
    if (seq.nq == 0 || j >= seq.len || j < kv_span<kRows, kTile>(p.a, seq, 0).begin) return;
    const int64_t page = kv_page(p.a.cache, p.a.table + b * p.a.table_width, j >> p.a.cache.page_shift, p.a.err);
    if (page < 0) return;
    const int64_t to = kv_weight(p.a.cache, page, h, (int)j & ((1 << p.a.cache.page_shift) - 1));
    const float before = p.previous != nullptr && j < seq.len - seq.nq ? p.previous[to] : 0.0f;
    const float* part = p.parts + item * p.groups * 2 * p.part_stride + j;
    float sum = 0.0f;
#pragma unroll 8
    for (int g = 0; g < 2 * p.groups; ++g) sum += part[g * p.part_stride];
    p.weights[to] = before + sum;
}

struct ManyPlan {
    int splits, groups, chunk, chunks;
    int64_t part_stride, stats_blocks, sum_blocks, join_blocks;
    size_t stats_bytes, parts_bytes;
};

ManyPlan many_plan(int64_t B, int64_t T_q, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int sms) {
    ManyPlan w;
    const int64_t blocks = (max_q * G + kRows - 1) / kRows, tiles = (max_kv + kTile - 1) / kTile;
    const int64_t wanted = 3 * (int64_t)sms;
    auto parts_of = [&](int64_t base) {  // enough blocks, of four tiles at least
        return std::max<int64_t>(1, std::min((wanted + base - 1) / base, (tiles + 3) / 4));
    };
    w.splits = (int)std::min<int64_t>(64, parts_of(B * H * blocks));
    w.part_stride = tiles * kTile;
    // sums per group of row blocks: as many groups as row blocks while they stay small
    const int64_t most = std::max<int64_t>(1, ((int64_t)64 << 20) / (B * H * 2 * w.part_stride * 4));
    w.groups = (int)std::min(blocks, most);
    const int64_t chunks = parts_of(B * H * w.groups);
    w.chunk = (int)((tiles + chunks - 1) / chunks);
    w.chunks = (int)((tiles + w.chunk - 1) / w.chunk);
    w.stats_blocks = B * H * blocks * w.splits;
    w.sum_blocks = B * H * w.groups * w.chunks;
    w.join_blocks = B * H * ((w.part_stride + 255) / 256);
    w.stats_bytes = ((size_t)(T_q * G * H) * w.splits * sizeof(float2) + 255) / 256 * 256;
    w.parts_bytes = (size_t)(B * H * w.groups * 2) * (size_t)w.part_stride * sizeof(float);
    return w;
}

template <int D, int BITS>
cudaError_t launch_form(const KvWeightsParams& p, const ManyPlan& w, const LaunchEnv& env) {
    using C = Cfg<D, BITS>;
    static_assert(C::kSmem <= 227 * 1024 - 12288, "shared memory of a block");
    cudaError_t e = allow_smem<kv_weights_many_kernel<D, BITS, false>>(C::kSmem);
    if (e == cudaSuccess) e = allow_smem<kv_weights_many_kernel<D, BITS, true>>(C::kSmem);
    if (e == cudaSuccess)
        e = launch_kernel(kv_weights_many_kernel<D, BITS, false>, dim3((unsigned)w.stats_blocks), dim3(kThreads), C::kSmem,
                          env.stream, kNoCluster, p);
    if (e == cudaSuccess)
        e = launch_kernel(kv_weights_many_kernel<D, BITS, true>, dim3((unsigned)w.sum_blocks), dim3(kThreads), C::kSmem,
                          env.stream, kNoCluster, p);
    if (e != cudaSuccess) return e;
    return launch_kernel(kv_weights_join_kernel, dim3((unsigned)w.join_blocks), dim3(256), 0, env.stream, kNoCluster, p);
}

}  // namespace

size_t kv_weights_many_workspace(int64_t B, int64_t T_q, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int sms) {
    const ManyPlan w = many_plan(B, T_q, G, H, max_kv, max_q, sms);
    return w.stats_bytes + w.parts_bytes;
}

bool kv_weights_many_fits(int64_t B, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int sms) {
    const ManyPlan w = many_plan(B, 1, G, H, max_kv, max_q, sms);
    return w.stats_blocks < kMaxRows && w.sum_blocks < kMaxRows && w.join_blocks < kMaxRows;
}

cudaError_t launch_kv_weights_many(KvWeightsParams p, int64_t D, int64_t bits, void* workspace, const LaunchEnv& env) {
    const ManyPlan w =
        many_plan(p.a.B, p.a.T_q, p.a.G, p.a.cache.H, p.a.table_width << p.a.cache.page_shift, p.max_q, env.sm_count);
    p.stats = static_cast<float2*>(workspace);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.stats_bytes);
    p.splits = w.splits;
    p.groups = w.groups;
    p.chunk = w.chunk;
    p.chunks = w.chunks;
    p.part_stride = w.part_stride;
    if (D == 64) return bits == 4 ? launch_form<64, 4>(p, w, env) : launch_form<64, 8>(p, w, env);
    return bits == 4 ? launch_form<128, 4>(p, w, env) : launch_form<128, 8>(p, w, env);
}

}  // namespace i8ql
