// Eviction from the quantized key/value cache: of each sequence and cache head
// the tokens that got most attention stay, and move together.
//
// With n tokens and a budget of m < n, the first `first` and the last `last`
// tokens stay, and of those between the m - first - last with the largest
// weights, equal weights: the lower index first (not a number counts as the
// least).  What stays keeps its order: slot s of the new sequence is the s-th
// kept token.
//
// Choosing is a radix select: four passes over the weights' bits, 8 at a time
// from the top, each a histogram of the candidates that share the digits found
// so far; then one pass in order, in which running counts of the kept and of the
// ties give each kept token its slot.  Nothing depends on timing (the histogram's
// atomics only count).  Moving is bound by bytes: kept rows of codes, scales and
// weights, read and written once.

#include <cuda_runtime.h>

#include <algorithm>

#include "kv_weights.cuh"

namespace i8ql {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kMoveThreads = 128;

// Unsigned keys in the order of the weights: -0 and 0 alike, not a number least.
__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t b = __float_as_uint(w + 0.0f);
    if (w != w) return 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int evict_len(const KvEvictParams& p, int64_t b) {
    const int64_t most = min(p.table_width << p.cache.page_shift, (int64_t)INT32_MAX - 65536);
    const int64_t len = __ldg(p.kv_lens + b);
    if (len < 0 || len > most) record_fault(p.err, kErrBitBadIndex);
    return (int)min(max(len, (int64_t)0), most);
}

__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const KvEvictParams p) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t found_digit, found_left;
    __shared__ uint2 warp_sum[kSelectThreads / 32];
    const int64_t item = blockIdx.x;
    const int64_t b = item / p.cache.H;
    const int h = (int)(item - b * p.cache.H);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_wait();
    const int n = evict_len(p, b);
    const int kept_n = min(n, p.budget);
    int32_t* kept = p.kept + item * p.budget;
    if (h == 0 && threadIdx.x == 0) {
        if (((kept_n + (1 << p.cache.page_shift) - 1) >> p.cache.page_shift) > p.new_width)
            record_fault(p.err, kErrBitBadIndex);
        p.new_lens[b] = kept_n;
    }
    for (int s = kept_n + threadIdx.x; s < p.budget; s += kSelectThreads) kept[s] = -1;
    if (n <= p.budget) {
        for (int s = threadIdx.x; s < n; s += kSelectThreads) kept[s] = s;
        return;
    }
    const int32_t* table = p.table + b * p.table_width;
    const int mask = (1 << p.cache.page_shift) - 1;
    auto key_of = [&](int j) {
        const int64_t page = kv_page(p.cache, table, j >> p.cache.page_shift, p.err);
        return page < 0 ? 0 : weight_key(p.weights[kv_weight(p.cache, page, h, j & mask)]);
    };
    // the threshold, and how many of the tokens that have it stay
    const int lo = p.first, hi = n - p.last;
    uint32_t left = (uint32_t)(p.budget - p.first - p.last), value = 0, known = 0;
    if (left == 0) {
        value = 0xffffffffu;
    } else {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256) hist[threadIdx.x] = 0;
            __syncthreads();
            for (int j = lo + threadIdx.x; j < hi; j += kSelectThreads) {
                const uint32_t k = key_of(j);
                if ((k & known) == value) atomicAdd(&hist[k >> shift & 255], 1u);
            }
            __syncthreads();
            if (warp == 0) {
                // from the top digit down, 8 digits a lane
                uint32_t mine = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) mine += hist[255 - 8 * lane - i];
                uint32_t upto = mine;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const uint32_t o = __shfl_up_sync(0xffffffffu, upto, m);
                    if (lane >= m) upto += o;
                }
                uint32_t above = upto - mine;
                if (above < left && upto >= left) {
                    int d = 255 - 8 * lane;
                    while (above + hist[d] < left) above += hist[d--];
                    found_digit = (uint32_t)d;
                    found_left = left - above;
                }
            }
            __syncthreads();
            value |= found_digit << shift;
            known |= 255u << shift;
            left = found_left;
        }
    }
    // slots, in order
    uint32_t before = 0, ties_before = 0;  // kept without ties, and ties
    for (int j0 = 0; j0 < n; j0 += kSelectThreads) {
        const int j = j0 + threadIdx.x;
        bool sure = false, tie = false;
        if (j < n) {
            sure = j < lo || j >= hi;
            if (!sure) {
                const uint32_t k = key_of(j);
                sure = k > value;
                tie = k == value;
            }
        }
        const unsigned sures = __ballot_sync(0xffffffffu, sure), ties = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) warp_sum[warp] = make_uint2(__popc(sures), __popc(ties));
        __syncthreads();
        uint32_t s = before, t = ties_before, s_all = before, t_all = ties_before;
        for (int w = 0; w < kSelectThreads / 32; ++w) {
            const uint2 x = warp_sum[w];
            if (w < warp) {
                s += x.x;
                t += x.y;
            }
            s_all += x.x;
            t_all += x.y;
        }
        const unsigned less = (1u << lane) - 1u;
        s += __popc(sures & less);
        t += __popc(ties & less);
        if (sure || (tie && t < left)) kept[s + min(t, left)] = j;
        before = s_all;
        ties_before = t_all;
        __syncthreads();
    }
}

// The copies of one thread: 16 bytes of a kept token's key and value codes, and with
// the first lane of a row its scales and weight.
struct EvictRow {
    uint4 k, v;
    uint32_t pk, pv;
    float w;
    bool there;
    int64_t to, to_weight;

    __device__ __forceinline__ void load(const KvEvictParams& p, int64_t b, int h, int slot, int lane, int limit) {
        there = slot < limit;
        if (!there) return;
        const int mask = (1 << p.cache.page_shift) - 1;
        const int j = p.kept[(b * p.cache.H + h) * p.budget + slot];
        there = (uint32_t)j < (uint32_t)(p.table_width << p.cache.page_shift);  // (weights changed during the call)
        if (!there) return;
        const int64_t from_page = kv_page(p.cache, p.table + b * p.table_width, j >> p.cache.page_shift, p.err);
        const int64_t to_page = kv_page(p.cache, p.new_table + b * p.new_width, slot >> p.cache.page_shift, p.err);
        there = from_page >= 0 && to_page >= 0;
        if (!there) return;
        const int64_t from = kv_row(p.cache, from_page, 0, h, j & mask), values = (int64_t)p.cache.H << p.cache.page_shift;
        to = kv_row(p.cache, to_page, 0, h, slot & mask);
        to_weight = kv_weight(p.cache, to_page, h, slot & mask);
        k = *reinterpret_cast<const uint4*>(p.cache.codes + from * p.row_bytes + lane * 16);
        v = *reinterpret_cast<const uint4*>(p.cache.codes + (from + values) * p.row_bytes + lane * 16);
        if (lane == 0) {
            pk = p.cache.params[from];
            pv = p.cache.params[from + values];
            w = p.weights[kv_weight(p.cache, from_page, h, j & mask)];
        }
    }

    __device__ __forceinline__ void store(const KvEvictParams& p, int lane) const {
        if (!there) return;
        const int64_t values = (int64_t)p.cache.H << p.cache.page_shift;
        *reinterpret_cast<uint4*>(p.cache.codes + to * p.row_bytes + lane * 16) = k;
        *reinterpret_cast<uint4*>(p.cache.codes + (to + values) * p.row_bytes + lane * 16) = v;
        if (lane == 0) {
            p.cache.params[to] = pk;
            p.cache.params[to + values] = pv;
            p.weights[to_weight] = w;
        }
    }
};

// Slots of the new sequence that the move fills.
__device__ __forceinline__ int evict_slots(const KvEvictParams& p, int64_t b) {
    return (int)min((int64_t)min(evict_len(p, b), p.budget), p.new_width << p.cache.page_shift);
}

// To pages of their own: rows in any order.
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(const KvEvictParams p) {
    const int lanes = p.row_bytes / 16, side = kMoveThreads / lanes;
    const int64_t item = blockIdx.x / p.chunks;
    const int chunk = (int)(blockIdx.x - item * p.chunks);
    const int64_t b = item / p.cache.H;
    const int h = (int)(item - b * p.cache.H);
    const int lane = threadIdx.x % lanes;
    pdl_wait();
    EvictRow row;
    row.load(p, b, h, chunk * side + threadIdx.x / lanes, lane, evict_slots(p, b));
    row.store(p, lane);
}

// In place: a block takes all rows of a head, from the front.  A kept token's place is
// never before its slot, so a round's rows are read, then written, and no later round
// reads what they overwrote.
__global__ void __launch_bounds__(kSelectThreads) kv_compact_kernel(const KvEvictParams p) {
    const int lanes = p.row_bytes / 16, side = kSelectThreads / lanes;
    const int64_t b = blockIdx.x / p.cache.H;
    const int h = (int)(blockIdx.x - b * p.cache.H);
    const int lane = threadIdx.x % lanes;
    pdl_wait();
    const int n = evict_len(p, b);
    if (n <= p.budget) return;
    const int slots = evict_slots(p, b);
    for (int s0 = 0; s0 < slots; s0 += side) {
        EvictRow row;
        row.load(p, b, h, s0 + threadIdx.x / lanes, lane, slots);
        __syncthreads();
        row.store(p, lane);
    }
}

}  // namespace

bool kv_evict_fits(int64_t B, int64_t H, int64_t row_bytes, int64_t budget) {
    const int64_t side = kMoveThreads / (row_bytes / 16), chunks = (budget + side - 1) / side;
    return B == 0 || chunks < kMaxRows / B / H;
}

cudaError_t launch_kv_evict(KvEvictParams p, const LaunchEnv& env) {
    const int64_t items = p.B * p.cache.H;
    cudaError_t e = launch_kernel(kv_select_kernel, dim3((unsigned)items), dim3(kSelectThreads), 0, env.stream,
                                  kNoCluster, p);
    if (e != cudaSuccess) return e;
    if (p.new_table == p.table)
        return launch_kernel(kv_compact_kernel, dim3((unsigned)items), dim3(kSelectThreads), 0, env.stream, kNoCluster, p);
    const int side = kMoveThreads / (p.row_bytes / 16);
    p.chunks = (p.budget + side - 1) / side;
    return launch_kernel(kv_move_kernel, dim3((unsigned)(items * p.chunks)), dim3(kMoveThreads), 0, env.stream,
                         kNoCluster, p);
}

}  // namespace i8ql
