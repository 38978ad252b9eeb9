// Attention weights summed per cached token, for many query rows (prompts): the
// same two passes as kv_weights.cu on the tensor cores proper (tcgen05,
// accumulators in TMEM).
//
// A block (one per SM) holds 256 query rows of one cache head (query tokens x the
// head group's heads) as two operand tiles of 128, and walks the cache in tiles of
// 128 tokens, whose codes become fp16 operands (as they lie: see kv_weights.cu) once for both:
//   first pass:   S = Q C^T  (rows x tokens), a thread a row: its maximum and sum
//   second pass:  S^T = C Q^T  (tokens x rows), a thread a token: the sum of its weights
// so that neither needs a shuffle; the operand tiles are the same, only their roles
// in the product change.  The scales stay outside the products, in fp32:
//   y = s_j S + low_j sum_d q_d,   a = unit_i y.
// In the second pass a row's maximum and sum are one number, n_i = m_i + log2 l_i,
// rounded to 2^-24 of it, as the logits themselves are.
//
// The second pass leaves sums over up to 128-row halves of a group of row blocks per
// token in a workspace (a thread adds to its own place, in order), and a third kernel
// adds those up: no atomics, the same bits whatever the timing.
//
// Roles: warps 0-3 and 4-7 the softmax of the two halves, warps 8-11 unpack codes
// into the swizzled operand tiles, warp 12 copies pages, warp 13 issues the MMAs.
// S is held twice per half (all 512 columns of TMEM), so products run ahead of the
// softmax.  Operand layout: K-major, 128-byte swizzle, channels in the order in which
// key words unpack.

#include <cuda_runtime.h>

#include <algorithm>

#include "kv_tc.cuh"
#include "kv_weights.cuh"

namespace i8ql {
namespace {

constexpr int kTile = kKvPromptTile;  // cache tokens per tile
constexpr int kRows = kKvPromptRows;  // query rows per block: two halves
constexpr int kSoftmaxWarps = 8;
constexpr int kUnpackWarps = 4;
constexpr int kCopyWarp = kSoftmaxWarps + kUnpackWarps;
constexpr int kMmaWarp = kCopyWarp + 1;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kStages = 2;     // unpacked tiles
constexpr int kRaw = 2;        // raw tiles
constexpr int kFactors = 4;    // tiles whose scales are kept
constexpr float kSlack = 8.0f; // a row's maximum may exceed what its sum is relative to by this (log2)

template <int D, int BITS>
struct Cfg {
    static constexpr int kRowBytes = D * BITS / 8;
    static constexpr int kKTile = kTile * D * 2;
    static constexpr int kRawBytes = kTile * kRowBytes + kTile * 4;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kRows * D * 2;
    static constexpr int kOffRaw = kOffK + kStages * kKTile;
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
        w.part = (int)(at % p.groups);
        at /= p.groups;
    } else {
        w.part = (int)(at % p.splits);
        at /= p.splits;
    }
    w.h = (int)(at % p.a.cache.H);
    at /= p.a.cache.H;
    if constexpr (SUM) {
        w.b = at;
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

// A row's sum so far, relative to 2^ref.
struct RowStats {
    float ref, sum;
};

// 32 columns of S of a row: tokens `token`.. with their scales and offsets.
template <bool EDGE>
__device__ __forceinline__ void add_tokens(RowStats& r, uint32_t s_at, const float* scale, const float* offset,
                                           float q_sum, float unit, int token, int lo, int hi) {
    uint32_t x[32];
    tmem_ld32(s_at, x);
    const uint64_t q2 = pair_f32(q_sum, q_sum);
    uint64_t y[16];
    float high[2] = {-INFINITY, -INFINITY};
    tc::tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(scale + j);
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(offset + j);
        const uint64_t zero = 0;
        uint64_t a = fma_f32x2(pair_u32(x[j], x[j + 1]), s.x, fma_f32x2(o.x, q2, zero));
        uint64_t b = fma_f32x2(pair_u32(x[j + 2], x[j + 3]), s.y, fma_f32x2(o.y, q2, zero));
        float v[4];
        split_f32(a, v[0], v[1]);
        split_f32(b, v[2], v[3]);
        if (EDGE) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = token + j + k <= hi && token + j + k >= lo ? v[k] : -INFINITY;
        }
        high[0] = max3(high[0], v[0], v[1]);
        high[1] = max3(high[1], v[2], v[3]);
        y[j / 2] = a;
        y[j / 2 + 1] = b;
    }
    const float top = fmaxf(high[0], high[1]) * unit;  // (unit >= 0; no number for nothing seen at unit 0)
    if (__any_sync(0xffffffffu, top > r.ref + kSlack)) {
        if (top > r.ref + kSlack) {
            r.sum *= exp2_approx(r.ref - top);
            r.ref = top;
        }
    }
    const float shift = r.ref == -INFINITY ? 0.0f : -r.ref;
    const uint64_t u2 = pair_f32(unit, unit), shift2 = pair_f32(shift, shift);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float a, b;
        split_f32(fma_f32x2(y[j], u2, shift2), a, b);
        a = exp2_approx(a);
        b = exp2_approx(b);
        if (EDGE) {
            const int tok = token + 2 * j;
            a = tok <= hi && tok >= lo ? a : 0.0f;
            b = tok + 1 <= hi && tok + 1 >= lo ? b : 0.0f;
        }
        sum[j & 1] = add_f32x2(sum[j & 1], pair_f32(a, b));
    }
    float a, b;
    split_f32(add_f32x2(sum[0], sum[1]), a, b);
    r.sum += a + b;
}

// What the columns of S^T need of their rows: unit, unit times the sum of the scaled
// row, and -n; the last token that the row sees.
struct RowFactors {
    float unit[kTile], sum[kTile], minus_n[kTile];
    int hi[kTile];
};

// The sum of 32 rows' weights of a token.
template <bool EDGE>
__device__ __forceinline__ void add_rows(uint64_t (&sum)[2], uint32_t s_at, const RowFactors& f, int c0, float scale,
                                         float offset, int token, int64_t window) {
    uint32_t x[32];
    tmem_ld32(s_at, x);
    const uint64_t s2 = pair_f32(scale, scale), o2 = pair_f32(offset, offset);
    tc::tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(f.unit + c0 + j);
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(f.sum + c0 + j);
        const ulonglong2 n = *reinterpret_cast<const ulonglong2*>(f.minus_n + c0 + j);
        const uint64_t zero = 0;
        float v[4];
        split_f32(fma_f32x2(pair_u32(x[j], x[j + 1]), fma_f32x2(u.x, s2, zero), fma_f32x2(q.x, o2, n.x)), v[0], v[1]);
        split_f32(fma_f32x2(pair_u32(x[j + 2], x[j + 3]), fma_f32x2(u.y, s2, zero), fma_f32x2(q.y, o2, n.y)), v[2], v[3]);
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

template <int D, int BITS, bool SUM>
__global__ void __launch_bounds__(kThreads, 1) kv_weights_many_kernel(const KvWeightsParams p) {
    using C = Cfg<D, BITS>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t raw_full[kRaw], raw_empty[kRaw], k_full[kStages], k_empty[kStages];
    __shared__ uint64_t q_full[2], s_full[2][2], s_empty[2][2], info_full[kFactors], drained;
    __shared__ __align__(16) float scales[kFactors][kTile], offsets[kFactors][kTile];
    __shared__ __align__(16) RowFactors row_factors[SUM ? 2 : 1];
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
            tc::mbar_init(&q_full[i], 128);
            for (int j = 0; j < 2; ++j) {
                tc::mbar_init(&s_full[i][j], 1);
                tc::mbar_init(&s_empty[i][j], 128);
            }
        }
        for (int i = 0; i < kFactors; ++i) tc::mbar_init(&info_full[i], kUnpackWarps * 32);
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
        const int tid = threadIdx.x - kSoftmaxWarps * 32;  // 0 .. 127
        constexpr int kLanesPerKey = C::kRowBytes / 16;
        constexpr int kChunks = BITS == 4 ? 4 : 2;  // operand chunks (8 channels) per 16 raw bytes
        const int key_lane = tid % kLanesPerKey;
        uint32_t kt = 0;
        for (int rb = work.rb0; rb < work.rb1; ++rb) {
            const Part r = find_part<SUM>(p, work, rb);
            for (int tile = r.t0; tile < r.t1; ++tile, ++kt) {
                const int token = tile * kTile;
                const uint32_t slot = kt % kRaw, stage = kt % kStages;
                const uint8_t* raw = smem + C::kOffRaw + slot * C::kRawBytes;
                wait(&raw_full[slot], (kt / kRaw) & 1);
                // this stage's last products are done: so is the softmax of four tiles ago
                wait(&k_empty[stage], ((kt / kStages) & 1) ^ 1);
                if (!dead) {
                    uint32_t pk = 0;
                    if (token + tid >= r.span.begin && token + tid < r.span.end)
                        pk = reinterpret_cast<const uint32_t*>(raw + kTile * C::kRowBytes)[tid];
                    scales[kt % kFactors][tid] = kv_scale(pk);
                    offsets[kt % kFactors][tid] = kv_low(pk);
                }
                tc::mbar_arrive(&info_full[kt % kFactors]);
                if (!dead) {
                    const uint32_t dst = smem_at + C::kOffK + stage * C::kKTile;
#pragma unroll 1
                    for (int i = 0; i < kLanesPerKey; ++i) {
                        const int tok = tid / kLanesPerKey + i * (kTile / kLanesPerKey);
                        uint32_t w[4];
                        lds<4>(raw + tok * C::kRowBytes + key_lane * 16, w);
                        const int chunk0 = key_lane * kChunks;  // of the row's D / 8
                        const int block = chunk0 / 8, pos0 = chunk0 % 8;
                        const int flip = block & 1;  // lanes of the two blocks take their chunks in opposite order (banks)
                        const uint32_t row = dst + block * (kTile * 128) + tok * 128;
#pragma unroll
                        for (int j = 0; j < kChunks; ++j) {
                            uint32_t h[4];
                            if constexpr (BITS == 4) {
                                kv_small_codes<4>(flip ? w[j ^ 1] : w[j], h);
                            } else {
                                uint32_t lo[2], hi[2];
                                kv_small_codes<8>(flip ? w[2 * (j ^ 1)] : w[2 * j], lo);
                                kv_small_codes<8>(flip ? w[2 * (j ^ 1) + 1] : w[2 * j + 1], hi);
                                h[0] = lo[0], h[1] = lo[1], h[2] = hi[0], h[3] = hi[1];
                            }
                            sts16(row + (((pos0 + (j ^ flip)) ^ (tok & 7)) << 4), h[0], h[1], h[2], h[3]);
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
        const uint32_t idesc = tc::f16_idesc(kTile);
        const uint32_t q_base = (uint32_t)tc::sw128_desc(smem_at + C::kOffQ);
        const uint32_t k_base = (uint32_t)tc::sw128_desc(smem_at + C::kOffK);
        const uint32_t high = (uint32_t)(tc::sw128_desc(smem_at) >> 32);
        uint32_t kt = 0, items[2] = {0, 0}, steps[2] = {0, 0};
        for (int rb = work.rb0; rb < work.rb1; ++rb) {
            const Part r = find_part<SUM>(p, work, rb);
            if (r.t0 >= r.t1) continue;
            const int halves = r.rows > 128 ? 2 : 1;
            for (int m = 0; m < halves; ++m) {
                wait(&q_full[m], items[m] & 1);
                ++items[m];
            }
            // A half that sits out is done with its last tile, whose scales the tiles to
            // come would overwrite (one that takes part says so with its row block's Q).
            if (halves == 1 && steps[1] > 0) wait(&s_empty[1][(steps[1] - 1) & 1], ((steps[1] - 1) / 2) & 1);
            for (int tile = r.t0; tile < r.t1; ++tile, ++kt) {
                wait(&k_full[kt % kStages], (kt / kStages) & 1);
                for (int m = 0; m < halves; ++m, __syncwarp()) {
                    const uint32_t buf = steps[m] & 1;
                    wait(&s_empty[m][buf], ((steps[m] / 2) & 1) ^ 1);
                    ++steps[m];
                    tc::tc_fence_after();
                    const uint32_t q = q_base + m * (128 * D * 2 / 16), k = k_base + (kt % kStages) * (C::kKTile / 16);
                    const uint32_t a = SUM ? k : q, b = SUM ? q : k;
                    const uint32_t d = tmem + (m * 2 + buf) * kTile, issue = !dead && lane == 0;
                    __syncwarp();
                    mma_ss<0, 0>(d, a, b, high, idesc, 0, issue);
                    mma_ss<2, 2>(d, a, b, high, idesc, 1, issue);
                    mma_ss<4, 4>(d, a, b, high, idesc, 1, issue);
                    mma_ss<6, 6>(d, a, b, high, idesc, 1, issue);
                    if constexpr (D == 128) {
                        constexpr int kNext = 128 * 128 / 16;  // the second 64 channels
                        mma_ss<kNext, kNext>(d, a, b, high, idesc, 1, issue);
                        mma_ss<kNext + 2, kNext + 2>(d, a, b, high, idesc, 1, issue);
                        mma_ss<kNext + 4, kNext + 4>(d, a, b, high, idesc, 1, issue);
                        mma_ss<kNext + 6, kNext + 6>(d, a, b, high, idesc, 1, issue);
                    }
                    commit_mma(&s_full[m][buf], issue);
                }
                commit_mma(&k_empty[kt % kStages], !dead && lane == 0);
            }
        }
        // nothing may be in flight when the TMEM is given back
        if (lane == 0) tc::mma_commit(&drained);
        __syncwarp();
        int none = 0;
        tc::mbar_wait(&drained, 0, &none, p.a.err);
    } else {
        // ------------------------------------------------------------ softmax
        const int m = warp / 4;
        const int r_m = threadIdx.x & 127;  // row of the half
        const uint32_t s_at = tmem + ((uint32_t)((warp % 4) * 32) << 16) + m * 2 * kTile;
        uint32_t kt = 0, steps = 0;
        float* part = nullptr;
        if constexpr (SUM) {
            const int64_t row = ((work.b * p.a.cache.H + work.h) * p.groups + work.part) * 2 + m;
            part = p.parts + row * p.part_stride + r_m;
            if (work.rb0 == work.rb1)  // fewer row blocks than groups
                for (int tile = work.chunk0; tile < work.chunk1; ++tile) part[(int64_t)tile * kTile] = 0.0f;
        }
        for (int rb = work.rb0; rb < work.rb1; ++rb) {
            const Part r = find_part<SUM>(p, work, rb);
            const bool active = r.t0 < r.t1 && r.rows > 128 * m;
            if constexpr (SUM) {
                // tiles that the first block does not see begin at 0
                if (rb == work.rb0)
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
                // the row goes into its operand tile, scaled to 2^14, permuted as the keys unpack
                const uint4* src = reinterpret_cast<const uint4*>(p.a.q + (work.seq.q0 + i) * p.a.q_stride + (int64_t)head * D);
                uint32_t top = 0;
#pragma unroll 8
                for (int w = 0; w < D / 8; ++w) {
                    const uint4 v = live ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
                    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t a = words[j] & 0x7fff0000u, b = (words[j] << 16) & 0x7fff0000u;
                        top = max(top, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
                    }
                }
                const int e = max((int)(top >> 23), 15) - 127;
                const float f = p.a.scale_log2 < 0.0f ? -pow2(14 - e) : pow2(14 - e);
                const float unit = pow2(e - 14) * (fabsf(p.a.scale_log2) * 0x1p24f);
                const uint32_t dst = smem_at + C::kOffQ + m * (128 * D * 2) + r_m * 128;
                float q_sum = 0.0f;
#pragma unroll 4
                for (int w = 0; w < D / 8; ++w) {
                    const uint4 v = live ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
                    const float y[8] = {lo_bf16(v.x) * f, hi_bf16(v.x) * f, lo_bf16(v.y) * f, hi_bf16(v.y) * f,
                                        lo_bf16(v.z) * f, hi_bf16(v.z) * f, lo_bf16(v.w) * f, hi_bf16(v.w) * f};
                    q_sum += ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
                    const uint32_t at = dst + (w / 8) * (128 * 128) + (((w & 7) ^ (r_m & 7)) << 4);
                    if constexpr (BITS == 4)
                        sts16(at, pack_f16(y[0], y[4]), pack_f16(y[1] * 0.0625f, y[5] * 0.0625f), pack_f16(y[2], y[6]),
                              pack_f16(y[3] * 0.0625f, y[7] * 0.0625f));
                    else
                        sts16(at, pack_f16(y[0], y[1]), pack_f16(y[2], y[3]), pack_f16(y[4], y[5]), pack_f16(y[6], y[7]));
                }
                q_sum *= 0x1p-24f;
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(&q_full[m]);
                if constexpr (SUM) {
                    float top_m = -INFINITY, l = 0.0f;
                    if (live) {
                        for (int s = 0; s < p.splits; ++s) top_m = fmaxf(top_m, p.stats[stat + s].x);
                        for (int s = 0; s < p.splits; ++s) {
                            const float2 x = p.stats[stat + s];
                            l = fmaf(x.y, exp2_approx(x.x - (top_m == -INFINITY ? 0.0f : top_m)), l);
                        }
                    }
                    RowFactors& rf = row_factors[m];
                    asm volatile("bar.sync %0, 128;" ::"r"(2 + m) : "memory");  // the last row block's are read
                    const bool some = l > 0.0f;
                    rf.unit[r_m] = some ? unit : 0.0f;
                    rf.sum[r_m] = some ? unit * q_sum : 0.0f;
                    rf.minus_n[r_m] = some ? -(top_m + log2f(l)) : -INFINITY;
                    rf.hi[r_m] = live ? hi : -1;
                    asm volatile("bar.sync %0, 128;" ::"r"(2 + m) : "memory");
                }
                // tokens [all_lo, all_hi] are seen by every row of the half
                const int all_hi = base + (r.row0 + m * 128) / p.a.G;
                const int last = r.row0 + min(r.rows, m * 128 + 128) - 1;
                const int all_lo = p.a.window > 0 ? (int)max(base + last / p.a.G + 1 - p.a.window, (int64_t)0) : 0;
                const int columns = (min(r.rows - m * 128, 128) + 31) / 32;
                const bool warp_live = SUM || (warp % 4) * 32 < r.rows - m * 128;
                for (int tile = r.t0; tile < r.t1; ++tile, ++steps) {
                    const uint32_t k = kt + (tile - r.t0), buf = steps & 1;
                    const int token = tile * kTile;
                    float before = 0.0f;
                    if constexpr (SUM) {
                        if (rb > work.rb0) before = part[(int64_t)tile * kTile];
                    }
                    // S first: its scales are there then, so one test of their barrier (whose
                    // earlier rounds a half that sat out a row block has not waited for)
                    // passes, and acquires them
                    wait(&s_full[m][buf], (steps / 2) & 1);
                    const bool there = tc::mbar_test(tc::smem_u32(&info_full[k % kFactors]), (k / kFactors) & 1);
                    tc::tc_fence_after();
                    if (!dead && __all_sync(0xffffffffu, there) && warp_live) {
                        const bool edge = token + kTile - 1 > all_hi || token < all_lo;
                        const uint32_t at = s_at + buf * kTile;
                        if constexpr (SUM) {
                            const float scale = scales[k % kFactors][r_m], offset = offsets[k % kFactors][r_m];
                            uint64_t sum[2] = {0, 0};
#pragma unroll 1
                            for (int q = 0; q < columns; ++q) {
                                if (edge)
                                    add_rows<true>(sum, at + q * 32, row_factors[m], q * 32, scale, offset, token + r_m, p.a.window);
                                else
                                    add_rows<false>(sum, at + q * 32, row_factors[m], q * 32, scale, offset, token + r_m, 0);
                            }
                            float a, b;
                            split_f32(add_f32x2(sum[0], sum[1]), a, b);
                            part[(int64_t)tile * kTile] = before + (a + b);
                        } else {
#pragma unroll 1
                            for (int q = 0; q < kTile / 32; ++q) {
                                const float* s = &scales[k % kFactors][q * 32];
                                const float* o = &offsets[k % kFactors][q * 32];
                                if (edge)
                                    add_tokens<true>(stats, at + q * 32, s, o, q_sum, unit, token + q * 32, lo, hi);
                                else
                                    add_tokens<false>(stats, at + q * 32, s, o, q_sum, unit, token + q * 32, lo, hi);
                            }
                        }
                    }
                    tc::tc_fence_before();
                    tc::mbar_arrive(&s_empty[m][buf]);
                }
            }
            kt += max(r.t1 - r.t0, 0);
            if constexpr (!SUM) {
                if (live && r.rows > 128 * m) p.stats[stat + work.part] = make_float2(stats.ref, stats.sum);
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
