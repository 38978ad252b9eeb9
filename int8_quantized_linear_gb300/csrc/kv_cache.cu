// Writing the quantized key/value cache, and reading it back.
//
//   store: per row x (one token of one head, D channels, bf16):
//     lo = min x, hi = max x, r = fl32(fl32(hi - lo) / L), L = 2^bits - 1,
//     s = the smallest bf16 >= r,
//     c[d] = rint(fl32(fl32(x[d] - lo) / s))  (ties to even; 0 when s = 0)
//   load: x[d] = bf16_rne(fl32(lo + s * c[d]))  (s * c is exact in fp32)
//
// lo is an input value, so it is exact in bf16.  The scale is held in 16 bits
// to keep a 4-bit row of 128 channels at 68 bytes; it is rounded up, not to
// nearest, so that the largest value stays inside the code range
// (hi - lo <= L s) and every value within half a step of lo + s c.  Rounding that to
// bf16 at most doubles it: x is a bf16 value too, no nearer than the nearest.
//
// Both are bound by bytes: a token of 8 heads x 128 channels is 4 KB of bf16
// and 1 KB of 4-bit rows.  A thread takes 16 channels of several rows, D / 16
// neighbouring lanes a row; minimum and maximum go through shuffles, so a row is
// read once and nothing is staged.  (16 channels, not 8:
// what a row costs beside its elements, addresses and scale, is then shared by half
// as many lanes.)  A thread's two rows are the key and the value of one token and head,
// loaded together and beside their slot, so that their place is worked out once:
// 127.6 us against 139.9 with two unrelated rows (131072 tokens of 8 heads x 128
// channels, 4 bits).  One row at a time, behind its slot, reached a third of the
// bandwidth.
//
// A third kernel turns queries and keys by their positions (rotary.cuh) on the
// way: the same store behind a key's rotation, and the queries written out.

#include <cuda_runtime.h>

#include <type_traits>

#include "kv_common.cuh"
#include "quant_math.cuh"
#include "rotary.cuh"

namespace i8ql {
namespace {

// Small blocks: 31.4 us for reading 32768 tokens of 8 heads x 128 channels back
// (4 bits), 33.4 with 256 threads.
constexpr int kKvThreads = 128;
constexpr int kKvChannels = 16;  // channels per thread
constexpr int kKvRows = 2;       // rows per thread: a token's key and value of a head
constexpr unsigned kKvOneWave = 1024;  // blocks that surely run at once
// Rotated store: query heads a group of lanes takes, and the threads an SM from which on it does
// (8192 tokens of 32 + 8 heads x 128 channels, 4 bits: 39.8, 34.5, 33.1 us with one, two and
// four; 64 tokens, where it would leave half of the GPU without work, one).
constexpr int kQueries = 4;
constexpr int kManyThreads = 16384;

struct KvMoveParams {
    KvCache cache;
    const int64_t* slots;
    uint32_t rows;  // T * H < 2^31
    uint32_t inv;   // floor(2^32 / H), or 2^32 - 1
    int64_t slot_limit;
    bool wide;  // load: keys and values lie on 32-byte boundaries
    unsigned* err;
};

// The token and head whose key and value a thread works on.
struct KvMoveRow {
    bool there;
    uint32_t t;  // token
    uint32_t h;  // head
};

template <int D>
__device__ __forceinline__ KvMoveRow move_row(const KvMoveParams& p) {
    constexpr int kGroups = kKvThreads / (D / kKvChannels);  // rows side by side in a block
    const uint32_t row = blockIdx.x * kGroups + threadIdx.x / (D / kKvChannels), heads = (uint32_t)p.cache.H;
    KvMoveRow r;
    r.there = row < p.rows;
    // row / heads: the estimate is at most one too small (row < 2^31)
    r.t = __umulhi(row, p.inv);
    r.h = row - r.t * heads;
    if (r.h >= heads) {
        ++r.t;
        r.h -= heads;
    }
    return r;
}

// Cache rows from a key to its value.
__device__ __forceinline__ int64_t value_rows(const KvCache& c) { return (int64_t)c.H << c.page_shift; }

// The key's row of the cache, or -1; the value's is value_rows on.
__device__ __forceinline__ int64_t cache_row(const KvMoveParams& p, const KvMoveRow& r, int64_t slot) {
    if (!r.there || slot < 0) return -1;
    if (slot >= p.slot_limit) {
        record_fault(p.err, kErrBitBadIndex);
        return -1;
    }
    const int64_t page = slot >> p.cache.page_shift;
    return kv_row(p.cache, page, 0, (int)r.h, (int)(slot - (page << p.cache.page_shift)));
}

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// fl32(x / L), x >= 0 (not a number and infinities as the division has them): as
// in kv_codes, with the correctly rounded reciprocal of L as a constant.
template <int L>
__device__ __forceinline__ float divided_by(float x) {
    if (!(x >= 0x1p-90f && x < 0x1p127f)) return __fdiv_rn(x, (float)L);
    constexpr float kInverse = (float)(1.0 / L);
    const float q = __fmul_rn(x, kInverse);
    return __fmaf_rn(__fmaf_rn(q, -(float)L, x), kInverse, q);
}

// The codes rint(fl32(t / s)) of t = x - lo, 0 <= t <= L s, in the low byte of
// each word.  bf16 values tie often (their differences are multiples of few
// units), so the quotient has to be the correctly rounded one: with r the
// correctly rounded reciprocal, q = fl(t r) is within an ulp, the remainder
// e = t - q s is exact, and fl(q + e r) is the correctly rounded quotient
// (Markstein's theorem, IBM J. Res. Dev. 34, 1990; the divisor's mantissa, 8
// bits, is not all ones).  s outside 2^-90 .. 2^90, where the remainder could
// leave the normal range, takes the division itself.  Adding 1.5 * 2^23 leaves
// the rounded integer, ties to even, in the low mantissa bits.  Two values per
// instruction, each with its own IEEE rounding.
__device__ __forceinline__ void kv_codes(const uint4& w, float lo, float s, uint32_t (&b)[8]) {
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    if (s >= 0x1p-90f && s <= 0x1p90f) {
        const float r = __frcp_rn(s);
        uint64_t lo2, r2, ns2, magic2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(lo2) : "f"(lo));
        asm("mov.b64 %0, {%1, %1};" : "=l"(r2) : "f"(r));
        asm("mov.b64 %0, {%1, %1};" : "=l"(ns2) : "f"(-s));
        asm("mov.b64 %0, {%1, %1};" : "=l"(magic2) : "f"(kRoundMagic));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n\t.reg .b64 t, q, e;\n\t"
                "mov.b64 t, {%2, %3};\n\t"
                "sub.rn.f32x2 t, t, %4;\n\t"
                "mul.rn.f32x2 q, t, %5;\n\t"
                "fma.rn.f32x2 e, q, %6, t;\n\t"
                "fma.rn.f32x2 q, e, %5, q;\n\t"
                "add.rn.f32x2 q, q, %7;\n\t"
                "mov.b64 {%0, %1}, q;\n\t}"
                : "=r"(b[2 * i]), "=r"(b[2 * i + 1])
                : "f"(lo_bf16(words[i])), "f"(hi_bf16(words[i])), "l"(lo2), "l"(r2), "l"(ns2), "l"(magic2));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[2 * i] = min(__float2uint_rn(__fdiv_rn(__fsub_rn(lo_bf16(words[i]), lo), s)), 255u);
            b[2 * i + 1] = min(__float2uint_rn(__fdiv_rn(__fsub_rn(hi_bf16(words[i]), lo), s)), 255u);
        }
    }
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// A row's (lo, -hi) as a pair, in every lane of the row: one minimum does both, over
// a thread's pairs, a pair's halves and the row's lanes (a row is a whole group of
// lanes; all lanes of the warp shuffle).
template <int LANES>
__device__ __forceinline__ uint32_t row_ends(const uint4& a, const uint4& b) {
    auto least4 = [](const uint4& x) { return min_bf16x2(min_bf16x2(x.x, x.y), min_bf16x2(x.z, x.w)); };
    auto most4 = [](const uint4& x) { return max_bf16x2(max_bf16x2(x.x, x.y), max_bf16x2(x.z, x.w)); };
    const uint32_t least = min_bf16x2(least4(a), least4(b));
    const uint32_t most = max_bf16x2(most4(a), most4(b)) ^ 0x80008000u;
    uint32_t ends = min_bf16x2(__byte_perm(least, most, 0x5410), __byte_perm(least, most, 0x7632));
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) ends = min_bf16x2(ends, __shfl_xor_sync(0xffffffffu, ends, m));
    return ends;
}

// The codes of 8 channels of a and 8 of b (4 bits: a word each; else two) of a row
// with these ends, and the row's (scale, low).
template <int BITS>
__device__ __forceinline__ uint32_t row_codes(const uint4& a, const uint4& b, uint32_t ends, uint32_t (&out)[4]) {
    const float lo = lo_bf16(ends), hi = -hi_bf16(ends);
    const float ratio = divided_by<(1 << BITS) - 1>(__fsub_rn(hi, lo));  // >= 0
    const uint32_t s_bits = (__float_as_uint(ratio) + 0xffffu) & 0xffff0000u;
    const float s = __uint_as_float(s_bits);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (s > 0.0f) kv_codes(j ? b : a, lo, s, c);
        if constexpr (BITS == 4) {
            // (only the low byte of each sum matters, and its halves do not meet)
            out[j] = low_bytes(c[0] + (c[1] << 4), c[2] + (c[3] << 4), c[4] + (c[5] << 4), c[6] + (c[7] << 4));
        } else {
            out[2 * j] = low_bytes(c[0], c[1], c[2], c[3]);
            out[2 * j + 1] = low_bytes(c[4], c[5], c[6], c[7]);
        }
    }
    return (s_bits >> 16) | (__float_as_uint(lo) & 0xffff0000u);
}

// 32768 tokens of 8 heads x 128 channels, 4 bits: 39.6 us, 4300 GB/s (63 % of a
// copy; 131072 tokens: 128 us, 5320 GB/s).  Bound by instruction issue: what the
// codes take an element, and what a row's scale takes.  10 blocks an SM: with the
// registers that the compiler takes unasked, fewer warps run, and it takes 2 us more.
template <int D, int BITS>
__global__ void __launch_bounds__(kKvThreads, 10) kv_store_kernel(const uint16_t* __restrict__ k,
                                                                  const uint16_t* __restrict__ v, int64_t k_stride,
                                                                  int64_t v_stride, KvMoveParams p) {
    constexpr int kLanes = D / kKvChannels;
    const int lane = threadIdx.x % kLanes;
    const KvMoveRow row = move_row<D>(p);
    pdl_wait();
    if (gridDim.x <= kKvOneWave) pdl_launch_dependents();
    uint4 w[kKvRows][2];
    int64_t slot = -1;
#pragma unroll
    for (int i = 0; i < kKvRows; ++i) {
        w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
        if (row.there) {
            const uint16_t* src = (i ? v + row.t * v_stride : k + row.t * k_stride) + (int64_t)row.h * D + lane * kKvChannels;
            w[i][0] = __ldg(reinterpret_cast<const uint4*>(src));
            w[i][1] = __ldg(reinterpret_cast<const uint4*>(src) + 1);
        }
    }
    if (row.there) slot = __ldg(p.slots + row.t);
    const int64_t key = cache_row(p, row, slot);
#pragma unroll
    for (int i = 0; i < kKvRows; ++i) {
        const uint32_t ends = row_ends<kLanes>(w[i][0], w[i][1]);
        if (key < 0) continue;
        const int64_t index = i ? key + value_rows(p.cache) : key;
        uint32_t out[4];  // the 16 codes: 4 bits in the first half
        const uint32_t param = row_codes<BITS>(w[i][0], w[i][1], ends, out);
        uint8_t* dst = p.cache.codes + index * (D * BITS / 8) + lane * (kKvChannels * BITS / 8);
        if constexpr (BITS == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
        else
            *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
        if (lane == 0) p.cache.params[index] = param;
    }
}

struct KvRotaryParams {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    uint16_t* q_out;
    int64_t q_out_stride;
    RotaryTable table;
    int q_heads;
    int q_units;  // groups of query heads of a token
    int units;    // of a token: those, then the cache's heads
    uint32_t rows;  // T x units
};

// A group of D / 16 lanes takes QUERIES query heads of a token, or the key and the value
// of a cache head.  Queries and keys are turned (rotary.cuh) before the key's ends are
// sought, and rounded to bf16 as if they had been written and read.  8192 tokens of 32 + 8 heads
// x 128 channels, 4 bits: 33.1 us for 179 MB, 5.4 TB/s: bound by bytes, and by the ramp at
// this size, as the store alone.
template <int D, int BITS, bool INTERLEAVED, int QUERIES>
__global__ void __launch_bounds__(kKvThreads) kv_store_rotary_kernel(const KvRotaryParams r, const KvMoveParams p) {
    constexpr int kLanes = D / kKvChannels, kMost = QUERIES > kKvRows ? QUERIES : kKvRows;
    const int lane = threadIdx.x % kLanes;
    const uint32_t row = blockIdx.x * (kKvThreads / kLanes) + threadIdx.x / kLanes;
    const bool there = row < r.rows;
    const uint32_t t = there ? row / (uint32_t)r.units : 0;
    const int unit = there ? (int)(row - t * (uint32_t)r.units) : 0;
    const int h = unit - r.q_units;  // < 0: queries
    const int q0 = unit * QUERIES;
    const RotaryChunks<4, INTERLEAVED> at(lane, D, r.table.rot);
    pdl_wait();
    uint32_t w[kMost][2][4] = {};
    int64_t slot = -1;
    auto load = [&](const uint16_t* src, uint32_t (&x)[2][4]) {
        const uint4 a = *(reinterpret_cast<const uint4*>(src) + at.a), b = *(reinterpret_cast<const uint4*>(src) + at.b);
        x[0][0] = a.x, x[0][1] = a.y, x[0][2] = a.z, x[0][3] = a.w;
        x[1][0] = b.x, x[1][1] = b.y, x[1][2] = b.z, x[1][3] = b.w;
    };
    auto word4 = [](const uint32_t (&x)[4]) { return make_uint4(x[0], x[1], x[2], x[3]); };
    RotaryAngles<4, INTERLEAVED> angle;
    bool turned = false;
    if (there) {
        if (h < 0) {
#pragma unroll
            for (int i = 0; i < QUERIES; ++i)
                if (q0 + i < r.q_heads) load(r.q + t * r.q_stride + (int64_t)(q0 + i) * D, w[i]);
        } else {
            load(r.k + t * r.k_stride + (int64_t)h * D, w[0]);
            load(r.v + t * r.v_stride + (int64_t)h * D, w[1]);
            slot = __ldg(p.slots + t);
        }
        const float* angles = rotary_row(r.table, t, p.err);
        turned = angles != nullptr && at.angle >= 0;
        if (turned) {
            angle.load(angles, r.table.rot, at, false);
            angle.turn(w[0][0], w[0][1], at.b_turned);
        }
    }
    if (__all_sync(0xffffffffu, !there || h < 0)) {  // nothing to quantize
        if (!there) return;
#pragma unroll
        for (int i = 0; i < QUERIES; ++i) {
            if (q0 + i >= r.q_heads) break;
            if (i > 0 && turned) angle.turn(w[i][0], w[i][1], at.b_turned);
            uint4* dst = reinterpret_cast<uint4*>(r.q_out + t * r.q_out_stride + (int64_t)(q0 + i) * D);
            dst[at.a] = word4(w[i][0]);
            dst[at.b] = word4(w[i][1]);
        }
        return;
    }
    if (there && h < 0) {
#pragma unroll 1
        for (int i = 0; i < QUERIES; ++i) {
            if (q0 + i >= r.q_heads) break;
            uint32_t x[2][4];
            load(r.q + t * r.q_stride + (int64_t)(q0 + i) * D, x);
            if (turned) angle.turn(x[0], x[1], at.b_turned);
            uint4* dst = reinterpret_cast<uint4*>(r.q_out + t * r.q_out_stride + (int64_t)(q0 + i) * D);
            dst[at.a] = word4(x[0]);
            dst[at.b] = word4(x[1]);
        }
    }
    KvMoveRow place = {there && h >= 0, t, (uint32_t)max(h, 0)};
    const int64_t key = cache_row(p, place, slot);
#pragma unroll
    for (int i = 0; i < kKvRows; ++i) {
        const uint4 a = word4(w[i][0]), b = word4(w[i][1]);
        const uint32_t ends = row_ends<kLanes>(a, b);
        if (key < 0) continue;
        const int64_t index = i ? key + value_rows(p.cache) : key;
        uint32_t out[4];
        const uint32_t param = row_codes<BITS>(a, b, ends, out);
        uint8_t* dst = p.cache.codes + index * (D * BITS / 8);
        if constexpr (BITS == 4) {
            reinterpret_cast<uint32_t*>(dst)[at.a] = out[0];
            reinterpret_cast<uint32_t*>(dst)[at.b] = out[1];
        } else {
            reinterpret_cast<uint2*>(dst)[at.a] = make_uint2(out[0], out[1]);
            reinterpret_cast<uint2*>(dst)[at.b] = make_uint2(out[2], out[3]);
        }
        if (lane == 0) p.cache.params[index] = param;
    }
}

// 32768 tokens of 8 heads x 128 channels, 4 bits: 31.4 us, 5420 GB/s (80 % of a
// copy); less at smaller sizes, where the chain of three loads (slot, codes,
// store) is not covered (16384 tokens: 19.1 us, 4450 GB/s).
template <int D, int BITS>
__global__ void __launch_bounds__(kKvThreads) kv_load_kernel(uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                             KvMoveParams p) {
    const int lane = threadIdx.x % (D / kKvChannels);
    const KvMoveRow row = move_row<D>(p);
    pdl_wait();
    if (gridDim.x <= kKvOneWave) pdl_launch_dependents();
    const int64_t key = cache_row(p, row, row.there ? __ldg(p.slots + row.t) : -1);
    if (!row.there) return;
    constexpr int kWords = kKvChannels * BITS / 32;
    uint32_t codes[kKvRows][kWords];
    uint32_t param[kKvRows];
#pragma unroll
    for (int i = 0; i < kKvRows; ++i) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) codes[i][j] = 0;
        param[i] = 0;  // stands for 0
        if (key >= 0) {
            const int64_t index = i ? key + value_rows(p.cache) : key;
            const uint8_t* src = p.cache.codes + index * (D * BITS / 8) + lane * (kWords * 4);
            if constexpr (BITS == 4) {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                codes[i][0] = v.x;
                codes[i][1] = v.y;
            } else {
                const uint4 v = *reinterpret_cast<const uint4*>(src);
                codes[i][0] = v.x;
                codes[i][1] = v.y;
                codes[i][2] = v.z;
                codes[i][3] = v.w;
            }
            param[i] = p.cache.params[index];
        }
    }
#pragma unroll
    for (int i = 0; i < kKvRows; ++i) {
        const float s = kv_scale(param[i]), lo = kv_low(param[i]);
        uint64_t s2, lo2, base2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
        asm("mov.b64 %0, {%1, %1};" : "=l"(lo2) : "f"(lo));
        asm("mov.b64 %0, {%1, %1};" : "=l"(base2) : "f"(8388608.0f));
        uint32_t out[kKvChannels / 2];
#pragma unroll
        for (int j = 0; j < kKvChannels / 2; ++j) {
            // a code in the mantissa of 2^23, less 2^23, is the code
            uint32_t a, b;
            if constexpr (BITS == 4) {
                const uint32_t word = codes[i][j / 4] >> (8 * (j % 4));
                a = (word & 15u) | 0x4b000000u;
                b = ((word >> 4) & 15u) | 0x4b000000u;
            } else {
                a = __byte_perm(codes[i][j / 2], 0x4b000000u, 0x7540 + 2 * (j % 2));
                b = __byte_perm(codes[i][j / 2], 0x4b000000u, 0x7541 + 2 * (j % 2));
            }
            asm("{\n\t.reg .b64 c;\n\t.reg .f32 x, y;\n\t"
                "mov.b64 c, {%1, %2};\n\t"
                "sub.rn.f32x2 c, c, %3;\n\t"
                "fma.rn.f32x2 c, c, %4, %5;\n\t"
                "mov.b64 {x, y}, c;\n\t"
                "cvt.rn.bf16x2.f32 %0, y, x;\n\t}"
                : "=r"(out[j])
                : "r"(a), "r"(b), "l"(base2), "l"(s2), "l"(lo2));
        }
        uint4* dst = reinterpret_cast<uint4*>((i ? v : k) + ((int64_t)row.t * p.cache.H + row.h) * D +
                                              lane * kKvChannels);
        // (two 16-byte stores each fill half of every sector: 35.5 against 33.4 us
        // for 32768 tokens of 8 heads x 128 channels, 4 bits)
        if (p.wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(out[0]), "r"(out[1]),
                         "r"(out[2]), "r"(out[3]), "r"(out[4]), "r"(out[5]), "r"(out[6]), "r"(out[7])
                         : "memory");
        } else {
            dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
            dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
        }
    }
}

KvMoveParams move_params(const KvCache& cache, const int64_t* slots, int64_t T, const LaunchEnv& env) {
    KvMoveParams p;
    p.cache = cache;
    p.slots = slots;
    p.rows = (uint32_t)(T * cache.H);
    p.inv = cache.H == 1 ? 0xffffffffu : (uint32_t)(((uint64_t)1 << 32) / (uint64_t)cache.H);
    p.slot_limit = cache.pages << cache.page_shift;
    p.wide = false;
    p.err = env.err;
    return p;
}

dim3 move_grid(uint32_t rows, int64_t D) {
    const int64_t per_block = kKvThreads / (D / kKvChannels);
    return dim3((unsigned)((rows + per_block - 1) / per_block));
}

}  // namespace

cudaError_t launch_kv_store(const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                            const int64_t* slots, const KvCache& cache, int64_t T, int64_t D, int64_t bits,
                            const LaunchEnv& env) {
    const KvMoveParams p = move_params(cache, slots, T, env);
    auto kernel = D == 64 ? (bits == 4 ? kv_store_kernel<64, 4> : kv_store_kernel<64, 8>)
                          : (bits == 4 ? kv_store_kernel<128, 4> : kv_store_kernel<128, 8>);
    return launch_kernel(kernel, move_grid(p.rows, D), dim3(kKvThreads), 0, env.stream, kNoCluster, k, v, k_stride,
                         v_stride, p);
}

cudaError_t launch_kv_load(const KvCache& cache, const int64_t* slots, uint16_t* k, uint16_t* v, int64_t T, int64_t D,
                           int64_t bits, const LaunchEnv& env) {
    KvMoveParams p = move_params(cache, slots, T, env);
    p.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31) == 0;
    auto kernel = D == 64 ? (bits == 4 ? kv_load_kernel<64, 4> : kv_load_kernel<64, 8>)
                          : (bits == 4 ? kv_load_kernel<128, 4> : kv_load_kernel<128, 8>);
    return launch_kernel(kernel, move_grid(p.rows, D), dim3(kKvThreads), 0, env.stream, kNoCluster, k, v, p);
}

cudaError_t launch_kv_store_rotary(const uint16_t* q, int64_t q_stride, uint16_t* q_out, int64_t q_out_stride,
                                   const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                                   const RotaryTable& table, bool interleaved, const int64_t* slots,
                                   const KvCache& cache, int64_t T, int64_t q_heads, int64_t D, int64_t bits,
                                   const LaunchEnv& env) {
    const KvMoveParams p = move_params(cache, slots, T, env);
    KvRotaryParams r = {q, k, v, q_stride, k_stride, v_stride, q_out, q_out_stride, table, (int)q_heads, 0, 0, 0};
    auto pick = [&](auto narrow4, auto narrow8, auto wide4, auto wide8) {
        return D == 64 ? (bits == 4 ? narrow4 : narrow8) : (bits == 4 ? wide4 : wide8);
    };
    auto launch = [&](auto queries) {
        constexpr int Q = decltype(queries)::value;
        r.q_units = ((int)q_heads + Q - 1) / Q;
        r.units = r.q_units + cache.H;
        r.rows = (uint32_t)(T * r.units);
        auto kernel = interleaved ? pick(kv_store_rotary_kernel<64, 4, true, Q>, kv_store_rotary_kernel<64, 8, true, Q>,
                                         kv_store_rotary_kernel<128, 4, true, Q>, kv_store_rotary_kernel<128, 8, true, Q>)
                                  : pick(kv_store_rotary_kernel<64, 4, false, Q>, kv_store_rotary_kernel<64, 8, false, Q>,
                                         kv_store_rotary_kernel<128, 4, false, Q>, kv_store_rotary_kernel<128, 8, false, Q>);
        return launch_kernel(kernel, move_grid(r.rows, D), dim3(kKvThreads), 0, env.stream, kNoCluster, r, p);
    };
    // several query heads a group of lanes, which share the angles, where enough groups are left
    if (T * (q_heads + cache.H) * (D / kKvChannels) >= (int64_t)kManyThreads * env.sm_count)
        return launch(std::integral_constant<int, kQueries>{});
    return launch(std::integral_constant<int, 1>{});
}

}  // namespace i8ql
