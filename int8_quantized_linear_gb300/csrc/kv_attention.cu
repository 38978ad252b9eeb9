// Attention over the quantized key/value cache for few query rows (single
// tokens and short drafts): the codes are read once, in pages, and never
// written back wider.
//
//   a_j = c * sum_d q_d k_jd   (c = softmax scale * log2 e, j over the visible tokens)
//   o_d = sum_j w_j v_jd / sum_j w_j,   w_j = 2^(a_j - max a)
// with k_jd = low_j + s_j code_jd (and v the same), so that
//   sum_d q_d k_jd = s_j sum_d q_d (code_jd + z) + (low_j - z s_j) sum_d q_d
//   sum_j w_j v_jd = sum_j (w_j s_j) (code_jd + z) + sum_j w_j (low_j - z s_j)
// for any z: the products run on the codes themselves (small integers, exact
// in bf16) with the scales outside.  For keys z = 128 (4 bits: the biased
// nibble in the mantissa of 128, no subtraction) or -128 (8 bits: the signed
// byte); at most 8 MMA steps accumulate, so the shift costs no precision that
// the logits would show (about 1e-4 of their unit).  For values the sum runs
// over the whole context and z centres the codes (-8 or -128): left
// uncentred, sums far larger than the result would cancel.
//
// Precision: logits, maxima, totals and accumulators in fp32; w_j s_j is
// rounded to bf16 for the tensor cores (2^-9 relative and independent per
// token, the same as any bf16 attention), q and the codes not at all.
//
// Bound by the bytes of the cache: 136 bytes a token and head (4 bits, 128
// channels, K and V), against which a warp's unpacking is the next cost, so
// the layout of the MMA operands is chosen to unpack with the fewest
// instructions:
//  * the 16-row A operand is the head group's queries (8 or 16 rows; a
//    sequence with more rows takes several blocks), the tokens are N;
//  * the channel order of a sum over channels is free: a lane takes D / 4
//    neighbouring channels of a key row, and pairs code i with code i + 4 (4
//    bits) or i + 2 (8 bits), which one mask yields; q is permuted alike;
//  * the token order of a sum over tokens is free too: values are paired
//    across two rows by byte permutes, and P stays in the registers in which
//    Q K^T left it;
//  * lane g of a value operand holds D / 8 neighbouring channels, which are
//    then 2 D / 8 neighbouring output channels of a lane.
// A block is four such warps over 32 tokens of a 128-token tile each, with
// their own running maximum, and one warp that keeps 3 tiles of bulk copies
// in flight (about 50 KB a block, three blocks an SM).

#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "kv_schedule.cuh"
#include "quant_math.cuh"
#include "tc_common.cuh"

namespace i8ql {
namespace {

constexpr int kTile = 128;                   // tokens per pipeline stage
constexpr int kWarps = 4;                    // consumer warps
constexpr int kWarpTokens = kTile / kWarps;  // tokens of a stage per warp
constexpr int kThreads = kWarps * 32 + 32;
constexpr int kStages = 3;

template <int D, int BITS, int ROWS>
struct Cfg {
    static constexpr int kRowBytes = D * BITS / 8;
    static constexpr int kCodes = kTile * kRowBytes;
    static constexpr int kStageBytes = 2 * kCodes + 2 * kTile * 4;
    // a merge row: D floats, 4 more after every lane's share (no bank conflicts)
    static constexpr int kMergeRow = D + 16;
    static constexpr int kMergeBytes = 2 * ROWS * kMergeRow * 4;
    static constexpr int kSmem = kStages * kStageBytes + kMergeBytes;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Pairs of bf16 from a word of codes: 4 bits: nibbles (j, j + 4) as 128 +
// code; 8 bits: bytes (j, j + 2) as code - 128 (the low seven bits as 128 + u
// plus -128 or -256, all exact).
template <int BITS>
__device__ __forceinline__ void unpack_biased(uint32_t w, uint32_t (&pair)[16 / BITS]) {
    if constexpr (BITS == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) pair[j] = ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t u = w >> (8 * j);
            pair[j] = add_bf16x2((u & 0x007f007fu) | 0x43004300u, (u & 0x00800080u) ^ 0xc380c380u);
        }
    }
}

// What unpack_biased adds to a code, and the same for centred codes.
template <int BITS>
constexpr float kBiased = BITS == 4 ? 128.0f : -128.0f;
template <int BITS>
constexpr float kCentred = BITS == 4 ? -8.0f : -128.0f;

template <int BITS>
__device__ __forceinline__ void unpack_centred(uint32_t w, uint32_t (&pair)[16 / BITS]) {
    unpack_biased<BITS>(w, pair);
    if constexpr (BITS == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) pair[j] = sub_bf16x2(pair[j], 0x43084308u);  // 136
    }
}

// N words from shared memory (N = 1, 2 or a multiple of 4; aligned to min(N, 4) words).
template <int N>
__device__ __forceinline__ void lds(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
            w[i] = v.x;
            w[i + 1] = v.y;
            w[i + 2] = v.z;
            w[i + 3] = v.w;
        }
    }
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     tc::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

template <int D, int BITS, int HALVES>
__global__ void __launch_bounds__(kThreads, HALVES == 1 && BITS == 4 ? 3 : 2) kv_attention_kernel(const KvAttnParams p) {
    constexpr int ROWS = 8 * HALVES;
    using C = Cfg<D, BITS, ROWS>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ KvLocate locate;
    __shared__ float merge_ml[kWarps][ROWS][2];
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
    KvCursor c;
    const KvRange range = kv_locate<ROWS, kTile, kThreads>(p, locate, c);  // (its barriers also publish the mbarriers)
    int64_t left = range.end - range.begin;
    int stage = 0;
    uint32_t parity = 0;

    if (warp == kWarps) {
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
        while (left > 0 && ok) {
            const int n = (int)min(left, (int64_t)(c.span.tiles - c.tile));
            for (int i = 0; i < n && ok; ++i) {
                const int token = (c.span.first + c.tile + i) * kTile + at;
                const bool need = at < kTile && token < c.span.end && token + piece > c.span.begin;
                const uint8_t* src = nullptr;
                if (need) {
                    int64_t page = __ldg(p.table + c.b * p.table_width + (token >> p.cache.page_shift));
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
            left -= n;
            c.tile += n - 1;
            kv_next_item<ROWS, kTile>(p, c);
        }
        if (!ok) {
            // giving up: let the copies in flight land before the block's
            // shared memory can go to another
            int none = 0;
            for (int i = 0; i < min(issued, kStages); ++i) {
                if (--stage < 0) {
                    stage = kStages - 1;
                    parity ^= 1;
                }
                tc::mbar_wait(&full[stage], parity, &none, p.err);
            }
        }
        return;
    }

    // -------------------------------------------------------------- consumers
    constexpr int kKeyWords = D * BITS / 128;     // words of a key row per lane
    constexpr int kValWords = D * BITS / 256;     // words of a value row per lane
    constexpr int kOut = D / 8;                   // n-tiles of the output: channels per lane of a value row
    constexpr int kPairs = 16 / BITS;             // pairs per word
    constexpr int kSteps = D / 16;
    const int g = lane / 4, t = lane % 4;
    const int key_row = g ^ ((g >> 1) & 1);  // the token of column g: rows of both parities in every load (banks)
    const int tok0 = (2 * t) ^ (t & 1), tok1 = (2 * t + 1) ^ (t & 1);  // the tokens of columns 2t and 2t + 1
    float* merge = reinterpret_cast<float*>(smem + kStages * C::kStageBytes);

    int split_rows = 0;
    while (left > 0) {
        const int n = (int)min(left, (int64_t)(c.span.tiles - c.tile));
        const int row0 = c.rb * ROWS;
        const int rows = min(ROWS, c.seq.nq * p.G - row0);
        const int base = c.seq.len - c.seq.nq;
        // this lane's rows of Q (A operand), permuted as the keys' unpacking pairs channels
        uint32_t qf[kSteps][2 * HALVES];
        float q_sum[HALVES];
        int hi[HALVES], lo[HALVES];  // the tokens a row sees: lo .. hi
#pragma unroll
        for (int x = 0; x < HALVES; ++x) {
            const int r = g + 8 * x;
            const bool live = r < rows;
            const int i = (row0 + (live ? r : 0)) / p.G;
            const int head = c.h * p.G + (row0 + (live ? r : 0)) - i * p.G;
            hi[x] = live ? base + i : INT32_MAX;
            lo[x] = live && p.window > 0 ? (int)max(base + i + 1 - p.window, (int64_t)0) : 0;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (c.seq.q0 + i) * p.q_stride + (int64_t)head * D +
                                                              t * (D / 4));
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint4 v = live ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
                sum += ((lo_bf16(v.x) + hi_bf16(v.x)) + (lo_bf16(v.y) + hi_bf16(v.y))) +
                       ((lo_bf16(v.z) + hi_bf16(v.z)) + (lo_bf16(v.w) + hi_bf16(v.w)));
                uint32_t (&f0)[2 * HALVES] = qf[2 * w], (&f1)[2 * HALVES] = qf[2 * w + 1];
                if constexpr (BITS == 4) {  // 8 channels: (0,4) (1,5) | (2,6) (3,7)
                    f0[x] = __byte_perm(v.x, v.z, 0x5410);
                    f0[HALVES + x] = __byte_perm(v.x, v.z, 0x7632);
                    f1[x] = __byte_perm(v.y, v.w, 0x5410);
                    f1[HALVES + x] = __byte_perm(v.y, v.w, 0x7632);
                } else {  // twice 4 channels: (0,2) (1,3)
                    f0[x] = __byte_perm(v.x, v.y, 0x5410);
                    f0[HALVES + x] = __byte_perm(v.x, v.y, 0x7632);
                    f1[x] = __byte_perm(v.z, v.w, 0x5410);
                    f1[HALVES + x] = __byte_perm(v.z, v.w, 0x7632);
                }
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            q_sum[x] = sum * p.scale_log2;
        }
        // tokens [all_lo, all_hi] are seen by every row
        const int all_hi = base + row0 / p.G;
        const int all_lo = p.window > 0 ? (int)max(base + (row0 + rows - 1) / p.G + 1 - p.window, (int64_t)0) : 0;

        float o[kOut][4];
#pragma unroll
        for (int i = 0; i < kOut; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[HALVES], l[HALVES], z[HALVES];  // running maximum; this lane's share of the total and of sum w (low - z s)
#pragma unroll
        for (int x = 0; x < HALVES; ++x) {
            m[x] = -INFINITY;
            l[x] = z[x] = 0.0f;
        }

        for (int i = 0; i < n; ++i) {
            const bool ok = tc::warp_wait(&full[stage], parity, &abort_flag, p.err);
            const uint8_t* st = smem + stage * C::kStageBytes;
            const int token = (c.span.first + c.tile + i) * kTile + warp * kWarpTokens;
            if (ok) {
                // logits
                float s[4][4];
                const uint8_t* keys = st + (warp * kWarpTokens + key_row) * C::kRowBytes + t * (kKeyWords * 4);
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    uint32_t w[kKeyWords];
                    lds<kKeyWords>(keys + nt * 8 * C::kRowBytes, w);
                    s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
                    for (int k = 0; k < kKeyWords; ++k) {
                        uint32_t b[kPairs];
                        unpack_biased<BITS>(w[k], b);
#pragma unroll
                        for (int j = 0; j < kPairs; j += 2) {
                            const uint32_t (&a)[2 * HALVES] = qf[(k * kPairs + j) / 2];
                            if constexpr (HALVES == 1)
                                mma_bf16(s[nt], a[0], 0u, a[1], 0u, b[j], b[j + 1]);
                            else
                                mma_bf16(s[nt], a[0], a[1], a[2], a[3], b[j], b[j + 1]);
                        }
                    }
                }
                const uint32_t* kp = reinterpret_cast<const uint32_t*>(st + 2 * C::kCodes) + warp * kWarpTokens;
                float top[HALVES];
#pragma unroll
                for (int x = 0; x < HALVES; ++x) top[x] = -INFINITY;
                const bool edge = token + kWarpTokens - 1 > all_hi || token < all_lo;
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int tok = 8 * nt + (e ? tok1 : tok0);
                        const uint32_t param = kp[tok];
                        const float ks = kv_scale(param);
                        const float off = fmaf(ks, -kBiased<BITS>, kv_low(param));
                        const float kc = ks * p.scale_log2;
#pragma unroll
                        for (int x = 0; x < HALVES; ++x) {
                            float a = fmaf(s[nt][2 * x + e], kc, off * q_sum[x]);
                            if (edge && (token + tok > hi[x] || token + tok < lo[x])) a = -INFINITY;
                            s[nt][2 * x + e] = a;
                            top[x] = fmaxf(top[x], a);
                        }
                    }
                // softmax weights against the running maximum
                bool grew = false;
                float shift[HALVES];
#pragma unroll
                for (int x = 0; x < HALVES; ++x) {
                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
                    grew |= top[x] > m[x];
                }
                if (__any_sync(0xffffffffu, grew)) {
                    float f[HALVES];
#pragma unroll
                    for (int x = 0; x < HALVES; ++x) {
                        const float to = fmaxf(m[x], top[x]);
                        f[x] = to == -INFINITY ? 1.0f : exp2_approx(m[x] - to);
                        m[x] = to;
                        l[x] *= f[x];
                        z[x] *= f[x];
                    }
#pragma unroll
                    for (int j = 0; j < kOut; ++j)
#pragma unroll
                        for (int x = 0; x < HALVES; ++x) {
                            o[j][2 * x] *= f[x];
                            o[j][2 * x + 1] *= f[x];
                        }
                }
#pragma unroll
                for (int x = 0; x < HALVES; ++x) shift[x] = m[x] == -INFINITY ? 0.0f : m[x];
                const uint32_t* vp = kp + kTile;
                uint32_t pr[4][HALVES];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    float wgt[2][HALVES];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t param = vp[8 * nt + (e ? tok1 : tok0)];
                        const float vs = kv_scale(param);
                        const float off = fmaf(vs, -kCentred<BITS>, kv_low(param));
#pragma unroll
                        for (int x = 0; x < HALVES; ++x) {
                            const float a = s[nt][2 * x + e];
                            const float w = exp2_approx(a - shift[x]);
                            l[x] += w;
                            // a token a row does not see may hold anything: no product with it
                            const bool skip = edge && a == -INFINITY;
                            z[x] = skip ? z[x] : fmaf(w, off, z[x]);
                            wgt[e][x] = skip ? 0.0f : w * vs;
                        }
                    }
#pragma unroll
                    for (int x = 0; x < HALVES; ++x) pr[nt][x] = pack_bf16(wgt[0][x], wgt[1][x]);
                }
                // o += (w s) (codes of V)
                const uint8_t* vals = st + C::kCodes + warp * kWarpTokens * C::kRowBytes + g * (kValWords * 4);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t v[4][kValWords];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        lds<kValWords>(vals + (16 * half + 8 * (r >> 1) + ((r & 1) ? tok1 : tok0)) * C::kRowBytes, v[r]);
#pragma unroll
                    for (int k = 0; k < kValWords; ++k)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            uint32_t b0[kPairs], b1[kPairs];
                            unpack_centred<BITS>(__byte_perm(v[0][k], v[1][k], y ? 0x7632 : 0x5410), b0);
                            unpack_centred<BITS>(__byte_perm(v[2][k], v[3][k], y ? 0x7632 : 0x5410), b1);
#pragma unroll
                            for (int j = 0; j < kPairs; ++j) {
                                float (&acc)[4] = o[(2 * k + y) * kPairs + j];
                                const uint32_t (&a)[HALVES] = pr[2 * half], (&b)[HALVES] = pr[2 * half + 1];
                                if constexpr (HALVES == 1)
                                    mma_bf16(acc, a[0], 0u, b[0], 0u, b0[j], b1[j]);
                                else
                                    mma_bf16(acc, a[0], a[1], b[0], b[1], b0[j], b1[j]);
                            }
                        }
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[stage]);
            if (++stage == kStages) {
                stage = 0;
                parity ^= 1;
            }
        }

        // join the four warps: totals over the lanes of a row, then one common maximum
#pragma unroll
        for (int x = 0; x < HALVES; ++x) {
#pragma unroll
            for (int k = 1; k < 4; k <<= 1) {
                l[x] += __shfl_xor_sync(0xffffffffu, l[x], k);
                z[x] += __shfl_xor_sync(0xffffffffu, z[x], k);
            }
            if (t == 0) {
                merge_ml[warp][g + 8 * x][0] = m[x];
                merge_ml[warp][g + 8 * x][1] = l[x];
            }
        }
        consumer_sync();
#pragma unroll
        for (int x = 0; x < HALVES; ++x) {
            float top = merge_ml[0][g + 8 * x][0];
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, merge_ml[w][g + 8 * x][0]);
            const float f = m[x] == -INFINITY ? 0.0f : exp2_approx(m[x] - top);
#pragma unroll
            for (int j = 0; j < kOut; ++j) {
                o[j][2 * x] = f == 0.0f ? 0.0f : (o[j][2 * x] + z[x]) * f;
                o[j][2 * x + 1] = f == 0.0f ? 0.0f : (o[j][2 * x + 1] + z[x]) * f;
            }
        }
        // lane (g, t) holds channels 2t D/8 .. (2t + 2) D/8 of rows g and g + 8
        float* mine = merge + (warp & 1) * ROWS * C::kMergeRow + g * C::kMergeRow + t * (2 * kOut + 4);
        for (int turn = 0; turn < 2; ++turn) {
            if (warp / 2 == 1 - turn) {
#pragma unroll
                for (int x = 0; x < HALVES; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < kOut; j += 4) {
                            float4* dst = reinterpret_cast<float4*>(mine + 8 * x * C::kMergeRow + e * kOut + j);
                            float4 v = make_float4(o[j][2 * x + e], o[j + 1][2 * x + e], o[j + 2][2 * x + e],
                                                   o[j + 3][2 * x + e]);
                            if (turn == 1) {
                                const float4 u = *dst;
                                v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                            }
                            *dst = v;
                        }
            }
            consumer_sync();
        }
        const bool begins = c.tile == 0, ends = c.tile + n == c.span.tiles;
        const int tid = threadIdx.x;
        const bool store = *reinterpret_cast<volatile int*>(&abort_flag) == 0;
        if (store) {
            for (int k = tid; k < rows * (D / 8); k += kWarps * 32) {
                const int r = k / (D / 8), d = (k % (D / 8)) * 8;
                const float* src = merge + r * C::kMergeRow + d + 4 * (d / (2 * kOut));
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(src + j);
                    const float4 b = *reinterpret_cast<const float4*>(src + ROWS * C::kMergeRow + j);
                    v[j] = a.x + b.x;
                    v[j + 1] = a.y + b.y;
                    v[j + 2] = a.z + b.z;
                    v[j + 3] = a.w + b.w;
                }
                float top = merge_ml[0][r][0];
                for (int w = 1; w < kWarps; ++w) top = fmaxf(top, merge_ml[w][r][0]);
                float total = 0.0f;
                for (int w = 0; w < kWarps; ++w)
                    total += merge_ml[w][r][0] == -INFINITY ? 0.0f : merge_ml[w][r][1] * exp2_approx(merge_ml[w][r][0] - top);
                if (begins && ends) {
                    const int i = (row0 + r) / p.G;
                    const int head = c.h * p.G + row0 + r - i * p.G;
                    const float inv = top == -INFINITY ? 0.0f : 1.0f / total;
                    *reinterpret_cast<uint4*>(p.out + ((c.seq.q0 + i) * ((int64_t)p.cache.H * p.G) + head) * D + d) =
                        make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                                   pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
                } else {
                    const int64_t slot = ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * ROWS + r;
                    float4* dst = reinterpret_cast<float4*>(p.part_o + slot * D + d);
                    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                    if (d == 0) *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(top, total);
                }
            }
            if (begins && !ends) {
                split_rows = rows;
                if (tid == 0) {
                    KvSplitItem it;
                    it.q_row = c.seq.q0;
                    it.row0 = row0;
                    it.rows = rows;
                    it.h = c.h;
                    it.last_cta = kv_owner(range.total, range.ctas, range.end - left + c.span.tiles - 1);
                    it.pad = 0;
                    p.split[blockIdx.x] = it;
                }
            }
        }
        left -= n;
        if (left > 0) {
            c.tile += n - 1;
            kv_next_item<ROWS, kTile>(p, c);
            consumer_sync();  // the merge rows are free again
        }
    }
    if (threadIdx.x == 0 && p.split != nullptr && split_rows == 0) p.split[blockIdx.x].rows = 0;
}

// Joins the parts of an item cut between CTAs, in their order: a group of
// warps per row, the parts shared out among the group.
constexpr int kJoinWarps = 32;

template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32) kv_join_kernel(const KvAttnParams p) {
    constexpr int kPer = kJoinWarps / ROWS;  // warps per row
    constexpr int kVec = D / 32;             // channels per lane
    __shared__ float part[kJoinWarps][D];
    pdl_wait();
    const KvSplitItem it = p.split[blockIdx.x];
    if (it.rows == 0) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r = warp / kPer, sub = warp % kPer;
    const int first = blockIdx.x, count = it.last_cta - first + 1;
    // part k: the beginning (slot 1 of the first CTA), then slot 0 of the following ones
    auto slot = [&](int k) { return ((int64_t)(first + k) * 2 + (k == 0 ? 1 : 0)) * ROWS + r; };
    float top = -INFINITY, total = 0.0f, acc[kVec] = {};
    if (r < it.rows) {
        for (int k = lane; k < count; k += 32) top = fmaxf(top, p.part_ml[slot(k) * 2]);
#pragma unroll
        for (int m = 16; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        if (top != -INFINITY) {
            for (int k = lane; k < count; k += 32) {
                const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + slot(k) * 2);
                total += ml.y * exp2_approx(ml.x - top);
            }
#pragma unroll
            for (int m = 16; m; m >>= 1) total += __shfl_xor_sync(0xffffffffu, total, m);
#pragma unroll 4
            for (int k = sub; k < count; k += kPer) {
                const float f = exp2_approx(p.part_ml[slot(k) * 2] - top);
                const float* src = p.part_o + slot(k) * D + lane * kVec;
                if constexpr (kVec == 4) {
                    const float4 v = *reinterpret_cast<const float4*>(src);
                    acc[0] = fmaf(v.x, f, acc[0]);
                    acc[1] = fmaf(v.y, f, acc[1]);
                    acc[2] = fmaf(v.z, f, acc[2]);
                    acc[3] = fmaf(v.w, f, acc[3]);
                } else {
                    const float2 v = *reinterpret_cast<const float2*>(src);
                    acc[0] = fmaf(v.x, f, acc[0]);
                    acc[1] = fmaf(v.y, f, acc[1]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) part[warp][lane * kVec + i] = acc[i];
    __syncthreads();
    if (sub != 0 || r >= it.rows) return;
    const float inv = top == -INFINITY ? 0.0f : 1.0f / total;
    const int i = (it.row0 + r) / p.G;
    const int head = it.h * p.G + it.row0 + r - i * p.G;
    uint16_t* dst = p.out + ((it.q_row + i) * ((int64_t)p.cache.H * p.G) + head) * D + lane * kVec;
    float v[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        v[j] = acc[j];
        for (int w = 1; w < kPer; ++w) v[j] += part[warp + w][lane * kVec + j];
        v[j] *= inv;
    }
    if constexpr (kVec == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16(v[0], v[1]);
}

// How a call runs: rows per block and the number of CTAs.
struct Plan {
    int halves;
    int64_t ctas;
    bool split;  // an item may be cut between CTAs
};

Plan make_plan(int64_t B, int64_t T_q, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int64_t bits, int sms) {
    Plan pl;
    pl.halves = max_q * G <= 8 ? 1 : 2;
    const int64_t rows = 8 * pl.halves;
    const int64_t per_sm = pl.halves == 1 && bits == 4 ? 3 : 2;
    // no more CTAs than there can be tiles
    const int64_t item_tiles = std::max<int64_t>((max_kv + kTile - 1) / kTile, 1);
    const int64_t items = (T_q * G / rows + B) * H;
    pl.ctas = std::min<int64_t>(sms * per_sm, items > sms * per_sm ? sms * per_sm : items * item_tiles);
    pl.split = item_tiles > 1;
    return pl;
}

size_t part_bytes(int64_t ctas, int64_t rows, int64_t D) { return (size_t)(ctas * 2 * rows * (D + 2) * 4); }

template <int D, int BITS, int HALVES>
cudaError_t launch_form(const KvAttnParams& p, const Plan& pl, const LaunchEnv& env) {
    using C = Cfg<D, BITS, 8 * HALVES>;
    static std::once_flag once[64];
    static cudaError_t set[64];
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::call_once(once[dev & 63], [&] {
        set[dev & 63] = cudaFuncSetAttribute(kv_attention_kernel<D, BITS, HALVES>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (set[dev & 63] != cudaSuccess) return set[dev & 63];
    e = launch_kernel(kv_attention_kernel<D, BITS, HALVES>, dim3((unsigned)pl.ctas), dim3(kThreads), C::kSmem,
                      env.stream, kNoCluster, p);
    if (e != cudaSuccess || !pl.split) return e;
    return launch_kernel(kv_join_kernel<D, 8 * HALVES>, dim3((unsigned)pl.ctas), dim3(kJoinWarps * 32), 0, env.stream,
                         kNoCluster, p);
}

template <int D, int BITS>
cudaError_t launch_bits(const KvAttnParams& p, const Plan& pl, const LaunchEnv& env) {
    return pl.halves == 1 ? launch_form<D, BITS, 1>(p, pl, env) : launch_form<D, BITS, 2>(p, pl, env);
}

}  // namespace

size_t kv_attention_workspace(int64_t B, int64_t T_q, int64_t G, int64_t H, int64_t D, int64_t bits, int64_t max_kv,
                              int64_t max_q, int sms) {
    const Plan pl = make_plan(B, T_q, G, H, max_kv, max_q, bits, sms);
    if (!pl.split) return 0;
    return part_bytes(pl.ctas, 8 * pl.halves, D) + (size_t)pl.ctas * sizeof(KvSplitItem);
}

cudaError_t launch_kv_attention(KvAttnParams p, int64_t D, int64_t bits, int64_t max_q, void* workspace,
                                const LaunchEnv& env) {
    const Plan pl = make_plan(p.B, p.T_q, p.G, p.cache.H, p.table_width << p.cache.page_shift, max_q, bits,
                              env.sm_count);
    p.part_o = nullptr;
    p.part_ml = nullptr;
    p.split = nullptr;
    if (pl.split) {
        const int64_t slots = pl.ctas * 2 * 8 * pl.halves;
        p.part_o = static_cast<float*>(workspace);
        p.part_ml = p.part_o + slots * D;
        p.split = reinterpret_cast<KvSplitItem*>(p.part_ml + slots * 2);
    }
    if (D == 64) return bits == 4 ? launch_bits<64, 4>(p, pl, env) : launch_bits<64, 8>(p, pl, env);
    return bits == 4 ? launch_bits<128, 4>(p, pl, env) : launch_bits<128, 8>(p, pl, env);
}

}  // namespace i8ql
