// Attention weights summed per cached token, and eviction by them: what their
// kernels share.
#pragma once

#include "kv_schedule.cuh"

namespace i8ql {

// |softmax scale * log2 e| = mantissa * 2^exponent.
struct KvScale {
    float mantissa;
    int exponent;
};

struct KvWeightsParams {
    KvAttnParams a;         // (out and the parts of its join unused)
    int64_t max_q;          // the most query tokens a sequence may have
    const float* previous;  // [pages][H][P]; null: nothing yet
    float* weights;         // the same layout; may be `previous`
    float2* stats;          // [T_q * Hq][splits]: a row's (maximum, sum) over a part of the tokens
    int splits;             // (one launch: CTAs of a cluster)
    int chunk;              // tiles of a block that sums (one launch: at most, of a CTA)
    KvScale scale;          // (few query rows)
    // many query rows only:
    int chunks;             // blocks of the tiles
    int groups;             // of row blocks that are summed together
    float* parts;           // [B][H][groups][2][part_stride]: sums over a group's rows, by halves of the row blocks
    int64_t part_stride;    // tokens of a table row, in whole tiles
};

// Query rows of a cache head up to which kv_weights.cu takes a call; the kernels for many of
// them (kv_weights_many.cu) fill operand tiles of 256 rows, whatever there is.  With 64 rows, 16
// sequences of up to 8191 tokens: 64 channels and 8 bits 110 us here and 211 there, 128
// channels and 4 bits 165 and 214.
constexpr int64_t kKvWeightsFewRows = 64;
size_t kv_weights_many_workspace(int64_t B, int64_t T_q, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int sms);
bool kv_weights_many_fits(int64_t B, int64_t G, int64_t H, int64_t max_kv, int64_t max_q, int sms);
cudaError_t launch_kv_weights_many(KvWeightsParams p, int64_t D, int64_t bits, void* workspace, const LaunchEnv& env);

struct KvEvictParams {
    KvCache cache;
    float* weights;  // [pages][H][P]
    const int32_t* table;
    int64_t table_width;
    const int32_t* kv_lens;
    const int32_t* new_table;  // `table` itself: in place
    int64_t new_width;
    int32_t* new_lens;  // [B]
    int32_t* kept;      // [B][H][budget]
    int64_t B;
    int budget, first, last;
    int row_bytes;  // of codes
    int cluster;    // CTAs that choose a sequence's head together
    bool cached;    // their shared memory holds the keys of as many tokens as the table has
    int chunks;     // blocks of rows of a sequence's head
    unsigned* err;
};

namespace {

// The codes of a key word as pairs of fp16 along the channels, (j, j + 4) of 8 or
// (2j, 2j + 1) of 4: 2^-24 times the code, as it lies (a subnormal number), and 2^-20
// times it in the odd pairs of 4-bit codes.
template <int BITS>
__device__ __forceinline__ void kv_small_codes(uint32_t w, uint32_t (&pair)[16 / BITS]) {
    if constexpr (BITS == 4) {
        const uint32_t u = w >> 8;
        pair[0] = w & 0x000f000fu;
        pair[1] = w & 0x00f000f0u;
        pair[2] = u & 0x000f000fu;
        pair[3] = u & 0x00f000f0u;
    } else {
        pair[0] = __byte_perm(w, 0, 0x4140);
        pair[1] = __byte_perm(w, 0, 0x4342);
    }
}

// A page of the table, or -1 where it is out of range (which is recorded).
__device__ __forceinline__ int64_t kv_page(const KvCache& c, const int32_t* table, int64_t i, unsigned* err) {
    const int64_t page = __ldg(table + i);
    if (page >= 0 && page < c.pages) return page;
    record_fault(err, kErrBitBadIndex);
    return -1;
}

// Index of a token's weight: token `off` of page `page`, head h.
__device__ __forceinline__ int64_t kv_weight(const KvCache& c, int64_t page, int h, int off) {
    return ((page * c.H + h) << c.page_shift) + off;
}

}  // namespace
}  // namespace i8ql
