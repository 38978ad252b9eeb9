// Writing the quantized key/value cache, and reading it back.
//
//   store: per row x (one token of one head, D channels, bf16):
//     lo = min x, hi = max x, r = fl32(fl32(hi - lo) / L), L = 2^bits - 1,
//     s = the smallest bf16 >= r,
//     c[d] = rint(fl32(fl32(x[d] - lo) / s))  (ties to even; 0 when s = 0)
//   load: x[d] = bf16_rne(lo + s * c[d])  (s * c is exact in fp32)
//
// lo is an input value, so it is exact in bf16.  The scale is held in 16 bits
// to keep a 4-bit row of 128 channels at 68 bytes; it is rounded up, not to
// nearest, so that the largest value stays inside the code range
// (hi - lo <= L s) and every value within half a step of its code.
//
// Both are bound by bytes: a token of 8 heads x 128 channels is 4 KB of bf16
// and 1 KB of 4-bit rows.  A thread takes 8 channels (one 16-byte vector of
// bf16), D / 8 neighbouring lanes a row; minimum and maximum go through
// shuffles, so a row is read once and nothing is staged.

#include <cuda_runtime.h>

#include "kv_common.cuh"
#include "quant_math.cuh"

namespace i8ql {
namespace {

constexpr int kKvThreads = 256;

struct KvMoveParams {
    KvCache cache;
    const int64_t* slots;
    uint32_t rows;  // T * 2 * H
    int64_t slot_limit;
    unsigned* err;
};

// The row this thread works on; false when it has none.  *t is its token,
// *index its row of the cache (or -1: a token without a slot).
template <int D>
__device__ __forceinline__ bool locate_row(const KvMoveParams& p, uint32_t* t, int* kv, int* h, int64_t* index) {
    constexpr int kLanes = D / 8;
    const uint32_t row = blockIdx.x * (kKvThreads / kLanes) + threadIdx.x / kLanes;
    if (row >= p.rows) return false;
    const uint32_t two_h = 2u * (uint32_t)p.cache.H;
    *t = row / two_h;
    const uint32_t in_token = row - *t * two_h;
    *kv = in_token >= (uint32_t)p.cache.H;
    *h = (int)in_token - (*kv ? p.cache.H : 0);
    const int64_t slot = __ldg(p.slots + *t);
    *index = -1;
    if (slot >= p.slot_limit) {
        record_fault(p.err, kErrBitBadIndex);
    } else if (slot >= 0) {
        const int64_t page = slot >> p.cache.page_shift;
        *index = kv_row(p.cache, page, *kv, *h, (int)(slot - (page << p.cache.page_shift)));
    }
    return true;
}

// rint(fl32(t / s)) for 0 <= t <= L s: through the correctly rounded
// reciprocal r, whose product is within 255 * 3 * 2^-24 < 2^-14 of the
// quotient, and through the IEEE division where that lies next to a
// half-integer (or r overflowed, s being subnormal).
template <int BITS>
__device__ __forceinline__ uint32_t kv_code(float t, float s, float r) {
    constexpr float kNear = 6.103515625e-05f;  // 2^-14
    float u = __fmul_rn(t, r);
    const float d = __fsub_rn(u, rintf(u));
    if (!(fabsf(d) <= 0.5f - kNear)) u = __fdiv_rn(t, s);
    return min(__float2uint_rn(u), (1u << BITS) - 1u);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kKvThreads) kv_store_kernel(const uint16_t* __restrict__ k,
                                                              const uint16_t* __restrict__ v, int64_t k_stride,
                                                              int64_t v_stride, KvMoveParams p) {
    constexpr int kLanes = D / 8;
    pdl_wait();
    uint32_t t;
    int kv, h;
    int64_t index;
    // rows are whole lane groups, so a group leaves together and the shuffles
    // below only cross lanes of one row
    const bool live = locate_row<D>(p, &t, &kv, &h, &index) && index >= 0;
    const int lane = threadIdx.x % kLanes;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) {
        const uint16_t* src = (kv ? v + t * v_stride : k + t * k_stride) + (int64_t)h * D + lane * 8;
        w = __ldg(reinterpret_cast<const uint4*>(src));
    }
    const float x[8] = {lo_bf16(w.x), hi_bf16(w.x), lo_bf16(w.y), hi_bf16(w.y),
                        lo_bf16(w.z), hi_bf16(w.z), lo_bf16(w.w), hi_bf16(w.w)};
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    if (!live) return;
    constexpr float kLevels = (float)((1 << BITS) - 1);
    const float ratio = __fdiv_rn(__fsub_rn(hi, lo), kLevels);  // >= 0
    const uint32_t s_bits = (__float_as_uint(ratio) + 0xffffu) & 0xffff0000u;
    const float s = __uint_as_float(s_bits);
    const float r = __frcp_rn(s);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = s > 0.0f ? kv_code<BITS>(__fsub_rn(x[i], lo), s, r) : 0u;
    if constexpr (BITS == 4) {
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) word |= c[i] << (4 * i);
        reinterpret_cast<uint32_t*>(p.cache.codes + index * (D / 2))[lane] = word;
    } else {
        uint2 words;
        words.x = c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
        words.y = c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24);
        reinterpret_cast<uint2*>(p.cache.codes + index * D)[lane] = words;
    }
    if (lane == 0) p.cache.params[index] = (s_bits >> 16) | (__float_as_uint(lo) & 0xffff0000u);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kKvThreads) kv_load_kernel(uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                             KvMoveParams p) {
    constexpr int kLanes = D / 8;
    pdl_wait();
    uint32_t t;
    int kv, h;
    int64_t index;
    if (!locate_row<D>(p, &t, &kv, &h, &index)) return;
    const int lane = threadIdx.x % kLanes;
    uint32_t out[4] = {0, 0, 0, 0};
    if (index >= 0) {
        uint32_t c[8];
        if constexpr (BITS == 4) {
            const uint32_t word = reinterpret_cast<const uint32_t*>(p.cache.codes + index * (D / 2))[lane];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = (word >> (4 * i)) & 15u;
        } else {
            const uint2 words = reinterpret_cast<const uint2*>(p.cache.codes + index * D)[lane];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = ((i < 4 ? words.x : words.y) >> (8 * (i & 3))) & 255u;
        }
        const uint32_t param = p.cache.params[index];
        const float s = kv_scale(param), lo = kv_low(param);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float a = __fmaf_rn(s, __uint2float_rn(c[i]), lo), b = __fmaf_rn(s, __uint2float_rn(c[i + 1]), lo);
            out[i / 2] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(a)) |
                         ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(b)) << 16);
        }
    }
    uint16_t* dst = (kv ? v : k) + ((int64_t)t * p.cache.H + h) * D + lane * 8;
    *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
}

KvMoveParams move_params(const KvCache& cache, const int64_t* slots, int64_t T, const LaunchEnv& env) {
    KvMoveParams p;
    p.cache = cache;
    p.slots = slots;
    p.rows = (uint32_t)(T * 2 * cache.H);
    p.slot_limit = cache.pages << cache.page_shift;
    p.err = env.err;
    return p;
}

dim3 move_grid(uint32_t rows, int64_t D) {
    const int64_t per_block = kKvThreads / (D / 8);
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
    const KvMoveParams p = move_params(cache, slots, T, env);
    auto kernel = D == 64 ? (bits == 4 ? kv_load_kernel<64, 4> : kv_load_kernel<64, 8>)
                          : (bits == 4 ? kv_load_kernel<128, 4> : kv_load_kernel<128, 8>);
    return launch_kernel(kernel, move_grid(p.rows, D), dim3(kKvThreads), 0, env.stream, kNoCluster, k, v, p);
}

}  // namespace i8ql
