// The quantized key/value cache: its layout, shared by the kernels that
// write it, read it back and attend over it.
//
// The cache is a pool of pages of P tokens (P a power of two, 16 .. 256):
//   codes  uint8 [pages, 2, H, P, D * bits / 8]   (K then V; 4-bit codes two
//          per byte, the even channel in the low nibble)
//   params bf16  [pages, 2, H, P, 2]              (scale, low)
// and a row (one token of one head) stands for x[d] = low + scale * code[d],
// codes 0 .. 2^bits - 1.  A page's rows of one head are contiguous, so the
// attention kernels fetch them as one bulk copy per array.
#pragma once

#include "common.cuh"

namespace i8ql {

constexpr int64_t kKvMinPage = I8QL_KV_MIN_PAGE;
constexpr int64_t kKvMaxPage = I8QL_KV_MAX_PAGE;

// A cache as the kernels see it.
struct KvCache {
    uint8_t* codes;
    uint32_t* params;  // (scale, low) as one word: the scale in the low half
    int64_t pages;
    int H;
    int page_shift;  // log2 P
};

namespace {

__device__ __forceinline__ float kv_scale(uint32_t param) { return __uint_as_float(param << 16); }
__device__ __forceinline__ float kv_low(uint32_t param) { return __uint_as_float(param & 0xffff0000u); }

// Index of a row: token `off` of page `page`, head h, K (0) or V (1).
__device__ __forceinline__ int64_t kv_row(const KvCache& c, int64_t page, int kv, int h, int off) {
    return (((page * 2 + kv) * c.H + h) << c.page_shift) + off;
}

}  // namespace
}  // namespace i8ql
