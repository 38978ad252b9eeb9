// Attention weights summed per cached token: how much attention the query rows
// of a call give each token of the quantized cache, for eviction.
//
//   a_ij = c * sum_d q_id k_jd   (c = softmax scale * log2 e, j over the tokens that row i sees)
//   w_j  = previous_j + sum_i 2^(a_ij - m_i) / l_i,   m_i = max_j a_ij, l_i = sum_j 2^(a_ij - m_i)
// over the query rows of a cache head (its group's heads, all query tokens).
// As in the attention kernels k_jd = low_j + s_j code_jd, the products run on
// centred codes in fp16 (exact: q is scaled by a power of two per row, elements
// 2^32 below its largest round), and the scales are applied outside:
//   sum_d q_d k_jd = s_j sum_d q_d c_jd + (low_j + z s_j) sum_d q_d.
// Logits, maxima and sums are fp32.  Maximum and sum are kept apart (2^(a - m) / l, not
// 2^(a - m - log2 l)): beside a large m the logarithm would lose its bits.
//
// A weight needs its row's maximum and sum, which need all keys: two kernels
// that both go over the keys.  The first leaves each row's (m, l) over a part of
// the tokens, the second joins them and sums the weights of its tokens over all
// rows, in order; no atomics.  Tokens that no row sees keep what they have.
//
// The layout of the products is that of kv_attention.cu: 16 tokens are the M rows
// of an MMA (A: codes as they lie, a lane taking D / 4 neighbouring channels of
// a token), 8 query rows its columns.

#include <cuda_runtime.h>

#include <algorithm>

#include "kv_math.cuh"
#include "kv_weights.cuh"

namespace i8ql {
namespace {

constexpr int kTile = 128;   // tokens a block works on at a time
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 8;    // most tiles of a block of the second kernel

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

// A lane's share of 8 HALVES query rows.
template <int D, int BITS, int HALVES>
struct Queries {
    uint32_t f[D / 16][HALVES][2];  // B operand: rows g + 8 x, permuted as the keys' unpacking pairs channels
    // of rows 2t + y + 8 x, whose logits the lane holds:
    float sum[HALVES][2];          // the scaled row's sum
    float unit[HALVES][2];         // what a scaled logit counts, in log2 units
    int hi[HALVES][2], lo[HALVES][2];  // the tokens the row sees: lo .. hi (none: hi < lo)

    __device__ __forceinline__ void load(const KvAttnParams& p, const KvSeq& seq, int h, int row0, int rows) {
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
            const int e = max((int)(top >> 23), 9) - 127;
            const float by = p.scale_log2 < 0.0f ? -pow2(8 - e) : pow2(8 - e);
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
            total += __shfl_xor_sync(0xffffffffu, total, 1);
            total += __shfl_xor_sync(0xffffffffu, total, 2);
            const float u = pow2(e - 8) * fabsf(p.scale_log2);
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

// A warp's 32 tokens of a tile: token g + 8 i, a lane's quarter of each row.
template <int D, int BITS>
struct Keys {
    static constexpr int kWords = D * BITS / 128;
    uint32_t w[4][kWords];
    uint32_t param[4];

    // Pages of the tile's tokens; token 0's for those outside begin .. end (not read from).
    static __device__ __forceinline__ void pages(const KvAttnParams& p, const int32_t* table, int token, int begin,
                                                 int end, int (&page)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = token + 8 * i;
            page[i] = j >= begin && j < end ? __ldg(table + (j >> p.cache.page_shift)) : -1;
        }
    }

    __device__ __forceinline__ void load(const KvAttnParams& p, int h, int token, int begin, int end, const int (&page)[4]) {
        const int t = threadIdx.x % 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = token + 8 * i;
            param[i] = 0;
#pragma unroll
            for (int k = 0; k < kWords; ++k) w[i][k] = 0;
            if (j < begin || j >= end) continue;
            int64_t at = page[i];
            if (at < 0 || at >= p.cache.pages) {
                record_fault(p.err, kErrBitBadIndex);
                at = 0;
            }
            const int64_t row = kv_row(p.cache, at, 0, h, j & ((1 << p.cache.page_shift) - 1));
            lds<kWords>(p.cache.codes + row * (D * BITS / 8) + t * (kWords * 4), w[i]);
            param[i] = p.cache.params[row];
        }
    }

    // Logits in log2 units of tokens g + 16 i (+ 8) and rows 2t, 2t + 1 (+ 8 x); -inf where
    // a row does not see a token.
    template <int HALVES>
    __device__ __forceinline__ void logits(const Queries<D, BITS, HALVES>& q, int token, float (&s)[2][HALVES][4]) const {
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
                unpack_key<BITS, true>(w[2 * i][k], a);
                unpack_key<BITS, true>(w[2 * i + 1][k], b);
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
                const uint32_t pk = param[2 * i + z];
                const float scale = kv_scale(pk), off = fmaf(scale, kCentre<BITS>, kv_low(pk));
                const int j = token + 16 * i + 8 * z;
#pragma unroll
                for (int x = 0; x < HALVES; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float a = fmaf(scale, s[i][x][2 * z + y], off * q.sum[x][y]) * q.unit[x][y];
                        s[i][x][2 * z + y] = j >= q.lo[x][y] && j <= q.hi[x][y] ? a : -INFINITY;
                    }
            }
    }
};

// 2^(a - m), 0 where a is -inf (and m too).
__device__ __forceinline__ float weight_of(float a, float m) { return exp2_approx(a - (m == -INFINITY ? 0.0f : m)); }

// (m, l) over a part of the tokens, for a block of rows.
template <int D, int BITS, int HALVES>
__global__ void __launch_bounds__(kThreads) kv_stats_kernel(const KvWeightsParams p) {
    constexpr int ROWS = 8 * HALVES;
    __shared__ float2 part[kWarps][ROWS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
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
            m[x][y] = -INFINITY;
            l[x][y] = 0.0f;
        }
    if (first < last) {
        Queries<D, BITS, HALVES> q;
        q.load(p.a, seq, h, row0, rows);
        const int32_t* table = p.a.table + b * p.a.table_width;
        int token = (span.first + first) * kTile + warp * 32 + g;
        int page[4];
        Keys<D, BITS> keys;
        Keys<D, BITS>::pages(p.a, table, token, span.begin, span.end, page);
        keys.load(p.a, h, token, span.begin, span.end, page);
        Keys<D, BITS>::pages(p.a, table, token + kTile, span.begin, span.end, page);
        for (int i = first; i < last; ++i, token += kTile) {
            Keys<D, BITS> now = keys;
            if (i + 1 < last) keys.load(p.a, h, token + kTile, span.begin, span.end, page);
            if (i + 2 < last) Keys<D, BITS>::pages(p.a, table, token + 2 * kTile, span.begin, span.end, page);
            float s[2][HALVES][4];
            now.logits(q, token, s);
#pragma unroll
            for (int x = 0; x < HALVES; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float top = fmaxf(fmaxf(s[0][x][y], s[0][x][2 + y]), fmaxf(s[1][x][y], s[1][x][2 + y]));
                    const float to = fmaxf(m[x][y], top);
                    const float sum = (weight_of(s[0][x][y], to) + weight_of(s[0][x][2 + y], to)) +
                                      (weight_of(s[1][x][y], to) + weight_of(s[1][x][2 + y], to));
                    l[x][y] = fmaf(l[x][y], weight_of(m[x][y], to), sum);
                    m[x][y] = to;
                }
        }
    }
    auto join = [](float& m, float& l, float om, float ol) {
        const float to = fmaxf(m, om);
        l = l * weight_of(m, to) + ol * weight_of(om, to);
        m = to;
    };
#pragma unroll
    for (int x = 0; x < HALVES; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
                join(m[x][y], l[x][y], __shfl_xor_sync(0xffffffffu, m[x][y], d), __shfl_xor_sync(0xffffffffu, l[x][y], d));
            if (g == 0) part[warp][8 * x + 2 * t + y] = make_float2(m[x][y], l[x][y]);
        }
    __syncthreads();
    if (threadIdx.x < rows) {
        float2 r = part[0][threadIdx.x];
        for (int w = 1; w < kWarps; ++w) join(r.x, r.y, part[w][threadIdx.x].x, part[w][threadIdx.x].y);
        const int i = (row0 + threadIdx.x) / p.a.G;
        const int64_t row = (seq.q0 + i) * ((int64_t)p.a.G * p.a.cache.H) + h * p.a.G + row0 + threadIdx.x - i * p.a.G;
        p.stats[row * p.splits + split] = r;
    }
}

// The weights of a chunk of tiles, summed over all rows.
template <int D, int BITS, int HALVES>
__global__ void __launch_bounds__(kThreads) kv_sum_kernel(const KvWeightsParams p) {
    constexpr int ROWS = 8 * HALVES;
    __shared__ float sums[kChunk * kTile];
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
        __syncthreads();
        if (threadIdx.x < ROWS) {
            float m = -INFINITY, l = 0.0f;
            if (threadIdx.x < rows) {
                const int i = (row0 + threadIdx.x) / p.a.G;
                const int64_t row = (seq.q0 + i) * ((int64_t)p.a.G * p.a.cache.H) + h * p.a.G + row0 + threadIdx.x - i * p.a.G;
                const float2* part = p.stats + row * p.splits;
                for (int s = 0; s < p.splits; ++s) m = fmaxf(m, part[s].x);
                for (int s = 0; s < p.splits; ++s) l = fmaf(part[s].y, weight_of(part[s].x, m), l);
            }
            stats[threadIdx.x] = make_float2(m == -INFINITY ? 0.0f : m, l > 0.0f ? 1.0f / l : 0.0f);
        }
        __syncthreads();
        Queries<D, BITS, HALVES> q;
        q.load(p.a, seq, h, row0, rows);
        float2 st[HALVES][2];
#pragma unroll
        for (int x = 0; x < HALVES; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) st[x][y] = stats[8 * x + 2 * t + y];
        int token = first * kTile + warp * 32 + g;
        int page[4];
        Keys<D, BITS> keys;
        Keys<D, BITS>::pages(p.a, table, token, span.begin, span.end, page);
        keys.load(p.a, h, token, span.begin, span.end, page);
        Keys<D, BITS>::pages(p.a, table, token + kTile, span.begin, span.end, page);
        for (int i = first; i < last; ++i, token += kTile) {
            Keys<D, BITS> now = keys;
            if (i + 1 < last) keys.load(p.a, h, token + kTile, span.begin, span.end, page);
            if (i + 2 < last) Keys<D, BITS>::pages(p.a, table, token + 2 * kTile, span.begin, span.end, page);
            float s[2][HALVES][4];
            now.logits(q, token, s);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float sum = 0.0f;
#pragma unroll
                for (int x = 0; x < HALVES; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        sum = fmaf(exp2_approx(s[k / 2][x][2 * (k % 2) + y] - st[x][y].x), st[x][y].y, sum);
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (t == 0) sums[(i - tile0) * kTile + warp * 32 + g + 8 * k] += sum;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tiles * kTile; i += kThreads) {
        const int j = tile0 * kTile + i;
        if (j >= seq.len) break;
        if (j < begin) continue;
        const int64_t page = kv_page(p.a.cache, table, j >> p.a.cache.page_shift, p.a.err);
        if (page < 0) continue;
        const int64_t to = kv_weight(p.a.cache, page, h, j & ((1 << p.a.cache.page_shift) - 1));
        const float before = p.previous != nullptr && j < seq.len - seq.nq ? p.previous[to] : 0.0f;
        p.weights[to] = before + sums[i];
    }
}

struct WeightsPlan {
    int halves, splits, chunk;
    int64_t stats_blocks, sum_blocks;
};

WeightsPlan weights_plan(int64_t B, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int sms) {
    WeightsPlan w;
    const int64_t rows = max_q * G;
    w.halves = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    const int64_t blocks = (rows + 8 * w.halves - 1) / (8 * w.halves), tiles = (max_kv + kTile - 1) / kTile;
    const int64_t wanted = 8 * (int64_t)sms, base = std::max<int64_t>(B * H * blocks, 1);
    w.splits = (int)std::min<int64_t>(std::min<int64_t>(64, tiles), std::max<int64_t>(1, (wanted + base - 1) / base));
    w.chunk = (int)std::min<int64_t>(kChunk, std::max<int64_t>(1, B * H * tiles / wanted));
    w.stats_blocks = B * H * blocks * w.splits;
    w.sum_blocks = B * H * ((tiles + w.chunk - 1) / w.chunk);
    return w;
}

}  // namespace

size_t kv_weights_workspace(int64_t B, int64_t T_q, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int sms) {
    if (max_q * G > kKvWeightsFewRows) return kv_weights_many_workspace(B, T_q, G, H, max_kv, max_q, sms);
    return (size_t)(T_q * G * H) * (size_t)weights_plan(B, G, H, max_kv, max_q, sms).splits * sizeof(float2);
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
    auto run = [&](auto stats, auto sum) {
        const cudaError_t e = p.max_q == 0 ? cudaSuccess
                                           : launch_kernel(stats, dim3((unsigned)w.stats_blocks), dim3(kThreads), 0,
                                                           env.stream, kNoCluster, p);
        if (e != cudaSuccess) return e;
        return launch_kernel(sum, dim3((unsigned)w.sum_blocks), dim3(kThreads), 0, env.stream, kNoCluster, p);
    };
#define I8QL_WEIGHTS(D_, B_)                                                                 \
    (w.halves == 1   ? run(kv_stats_kernel<D_, B_, 1>, kv_sum_kernel<D_, B_, 1>)             \
     : w.halves == 2 ? run(kv_stats_kernel<D_, B_, 2>, kv_sum_kernel<D_, B_, 2>)             \
                     : run(kv_stats_kernel<D_, B_, 4>, kv_sum_kernel<D_, B_, 4>))
    if (D == 64) return bits == 4 ? I8QL_WEIGHTS(64, 4) : I8QL_WEIGHTS(64, 8);
    return bits == 4 ? I8QL_WEIGHTS(128, 4) : I8QL_WEIGHTS(128, 8);
#undef I8QL_WEIGHTS
}

}  // namespace i8ql
