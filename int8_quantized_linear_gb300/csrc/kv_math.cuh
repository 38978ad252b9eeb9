// Arithmetic on cache rows shared by the two attention kernels: codes to fp16
// (exact), wide shared-memory loads, bulk copies of pages.
#pragma once

#include <atomic>

#include "kv_schedule.cuh"
#include "quant_math.cuh"
#include "tc_common.cuh"

namespace i8ql {
namespace {

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

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// What brings a softmax reference (log2 units) below 2^23; 1 where it is.  A weight's
// exponent is c a - m in one step, so it misses logit less reference by the rounding
// of m, which has to stay small: c and m are shrunk together.  Logits of that size are
// known to 2^-24 of their magnitude at best, which is more than shrinking blurs.
__device__ __forceinline__ float shrink_reference(float m) {
    const int e = (int)(__float_as_uint(m) >> 23 & 255) - 127;
    return e < 23 || e == 128 ? 1.0f : pow2(22 - e);
}

// What is subtracted from a centred code.
template <int BITS>
constexpr float kCentre = BITS == 4 ? 8.0f : 128.0f;

// (w & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}

// Small integers become fp16 as is widely done: put into the mantissa of 1024, whose
// last place counts 1, and less 1024.

// Eight nibbles as four pairs of fp16 (nibbles j and j + 4), CENTRED less 8: exact.
template <bool CENTRED>
__device__ __forceinline__ void unpack_nibbles(uint32_t w, uint32_t (&pair)[4]) {
    constexpr uint32_t kSub = CENTRED ? 0x64086408u : 0x64006400u;  // 1032 or 1024
    constexpr uint32_t kAdd = CENTRED ? 0xd480d480u : 0xd400d400u;  // -72 or -64
    const uint32_t u = w >> 8;
    pair[0] = sub_f16x2(and_or(w, 0x000f000fu, 0x64006400u), kSub);               // 1024 + c - ..
    pair[1] = fma_f16x2(and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, kAdd);  // (1024 + 16 c) / 16 - ..
    pair[2] = sub_f16x2(and_or(u, 0x000f000fu, 0x64006400u), kSub);
    pair[3] = fma_f16x2(and_or(u, 0x00f000f0u, 0x64006400u), 0x2c002c00u, kAdd);
}

// Two bytes as a pair of fp16, CENTRED less 128: exact.
template <bool CENTRED>
__device__ __forceinline__ uint32_t unpack_bytes(uint32_t w, uint32_t select) {
    return sub_f16x2(__byte_perm(w, 0x64646464u, select), CENTRED ? 0x64806480u : 0x64006400u);  // 1024 + c - ..
}

// A word of a key row as pairs along the channels: (j, j + 4) of 8 codes, or
// (2j, 2j + 1) of 4.
template <int BITS, bool CENTRED>
__device__ __forceinline__ void unpack_key(uint32_t w, uint32_t (&pair)[16 / BITS]) {
    if constexpr (BITS == 4) {
        unpack_nibbles<CENTRED>(w, pair);
    } else {
        pair[0] = unpack_bytes<CENTRED>(w, 0x5150);
        pair[1] = unpack_bytes<CENTRED>(w, 0x5352);
    }
}

// Words of two value rows as pairs along the tokens, one per channel.
template <int BITS, bool CENTRED>
__device__ __forceinline__ void unpack_values(uint32_t a, uint32_t b, uint32_t (&pair)[32 / BITS]) {
    if constexpr (BITS == 4) {
        uint32_t lo[4], hi[4];
        unpack_nibbles<CENTRED>(__byte_perm(a, b, 0x5410), lo);
        unpack_nibbles<CENTRED>(__byte_perm(a, b, 0x7632), hi);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            pair[j] = lo[j];
            pair[4 + j] = hi[j];
        }
    } else {
        const uint32_t lo = __byte_perm(a, b, 0x5140), hi = __byte_perm(a, b, 0x7362);  // a0 b0 a1 b1, a2 b2 a3 b3
        pair[0] = unpack_bytes<CENTRED>(lo, 0x5150);
        pair[1] = unpack_bytes<CENTRED>(lo, 0x5352);
        pair[2] = unpack_bytes<CENTRED>(hi, 0x5150);
        pair[3] = unpack_bytes<CENTRED>(hi, 0x5352);
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

// Lets KERNEL use `bytes` of dynamic shared memory on the current device (below
// 64, as launch_env checks); the runtime is told once per device.
template <auto KERNEL>
cudaError_t allow_smem(int bytes) {
    static std::atomic<bool> allowed[64];
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (allowed[dev & 63].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) allowed[dev & 63].store(true, std::memory_order_release);
    return e;
}

}  // namespace
}  // namespace i8ql
