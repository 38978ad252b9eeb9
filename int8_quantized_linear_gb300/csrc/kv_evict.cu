// Eviction from the quantized key/value cache: of each sequence and cache head
// the tokens that got most attention stay, and move together.
//
// With n tokens and a budget of m < n, the first `first` and the last `last`
// tokens stay, and of those between the m - first - last with the largest
// weights, equal weights: the lower index first (not a number counts as the
// least).  What stays keeps its order: slot s of the new sequence is the s-th
// kept token.
//
// Choosing is a radix select: three passes over the weights' bits, 11, 11 and 10 from
// the top, each a histogram of the candidates that share the digits found so far;
// then one pass in order, in which running counts of the kept and of the ties give
// each kept token its slot.  A cluster of CTAs takes a sequence's head, each a run of
// its tokens, which it reads once, into shared memory; histograms and counts are added up
// through distributed shared memory.  Nothing depends on timing (the histogram's atomics
// only count).  32 sequences of up to 16384 tokens with 8 heads, cut to 2048: 28.0 us, bound by
// the instructions (issue slots 65 %) and the barriers between the passes; 70.7 with the
// weights read from memory in four passes of 8 bits.
//
// Moving is bound by bytes: kept rows of codes, scales and weights, read and written
// once: 128 channels of 4 bits, as above, 35.3 us.  A kept token's scales and weight are 4
// bytes each, in sectors of their own, so that 130 MB are read for the 73 that are needed,
// and 73 written: 5.7 TB/s.  (One, two or four rows a thread: 35 us each.)

#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kv_math.cuh"
#include "kv_weights.cuh"

namespace i8ql {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kMoveThreads = 128;
constexpr int kMoveRows = 2;

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

// Shared memory of the keys: 16384 a CTA let two of them run on an SM.  Longer runs (of
// more than 8 times as many tokens) are read from memory in every pass.
constexpr int kMostKeys = 16384;
constexpr int kBins = 2048;
constexpr int kSelectWarps = kSelectThreads / 32;

__device__ __forceinline__ uint32_t ld_cluster(const uint32_t* p, int rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tc::mapa(tc::smem_u32(p), rank)) : "memory");
    return v;
}

__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const KvEvictParams p) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ uint32_t hist[kBins];       // this CTA's
    __shared__ uint32_t warp_sum[kSelectWarps][2];
    __shared__ uint32_t counts[2];         // this CTA's kept without ties, and ties
    __shared__ uint32_t found_digit, found_left;
    const int size = p.cluster, rank = (int)tc::cluster_rank();
    const uint32_t item = blockIdx.x / (uint32_t)size;
    const uint32_t b = item / (uint32_t)p.cache.H;
    const int h = (int)(item - b * (uint32_t)p.cache.H);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_wait();
    const int n = evict_len(p, b);
    const int kept_n = min(n, p.budget);
    int32_t* kept = p.kept + (int64_t)item * p.budget;
    if (h == 0 && rank == 0 && threadIdx.x == 0) {
        if (((kept_n + (1 << p.cache.page_shift) - 1) >> p.cache.page_shift) > p.new_width)
            record_fault(p.err, kErrBitBadIndex);
        p.new_lens[b] = kept_n;
    }
    const int threads = size * kSelectThreads, thread = rank * kSelectThreads + threadIdx.x;
    for (int s = kept_n + thread; s < p.budget; s += threads) kept[s] = -1;
    if (n <= p.budget) {  // (the whole cluster)
        for (int s = thread; s < n; s += threads) kept[s] = s;
        return;
    }
    // This CTA's tokens j0 .. j1 - 1, and this warp's of them: whole groups of 128
    const int32_t* table = p.table + b * p.table_width;
    const int mask = (1 << p.cache.page_shift) - 1;
    const int run = ((n + size - 1) / size + 127) & ~127;
    const int j0 = (int)min((int64_t)run * rank, (int64_t)n), j1 = (int)min((int64_t)j0 + run, (int64_t)n);
    const int groups = (j1 - j0 + 127) / 128;
    const int g0 = groups * warp / kSelectWarps, g1 = groups * (warp + 1) / kSelectWarps;
    const bool cached = p.cached;
    // four neighbours, which lie in one page (what lies behind the end is not used)
    auto four = [&](int j) {
        uint4 k = make_uint4(0, 0, 0, 0);
        if (j < j1) {
            const int64_t page = kv_page(p.cache, table, j >> p.cache.page_shift, p.err);
            if (page >= 0) {
                const float4 w = *reinterpret_cast<const float4*>(p.weights + kv_weight(p.cache, page, h, j & mask));
                k = make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
            }
        }
        return k;
    };
    auto keys_of = [&](int g) {
        return cached ? *reinterpret_cast<const uint4*>(keys + g * 128 + lane * 4) : four(j0 + g * 128 + lane * 4);
    };
    if (cached) {
#pragma unroll 4
        for (int g = g0; g < g1; ++g) *reinterpret_cast<uint4*>(keys + g * 128 + lane * 4) = four(j0 + g * 128 + lane * 4);
        __syncwarp();
    }
    // the threshold, and how many of the tokens that have it stay
    const int lo = p.first, hi = n - p.last;
    uint32_t left = (uint32_t)(p.budget - p.first - p.last), value = 0, known = 0;
    if (left == 0) {
        value = 0xffffffffu;
    } else {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digits = pass == 2 ? 1023 : 2047;
            for (int i = threadIdx.x; i < kBins; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
            for (int g = g0; g < g1; ++g) {
                const uint4 k4 = keys_of(g);
                const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + g * 128 + lane * 4 + i;
                    const bool in = j >= lo && j < min(hi, j1) && (k[i] & known) == value;
                    // (the first lane's digit counts once for the warp: a histogram of few values,
                    // of zeros say, would serialise its atomics)
                    const unsigned live = __ballot_sync(0xffffffffu, in);
                    if (live == 0) continue;
                    const uint32_t d = k[i] >> shift & digits;
                    const int leader = __ffs(live) - 1;
                    const uint32_t first = __shfl_sync(0xffffffffu, d, leader);  // (all lanes take part)
                    const bool same = in && d == first;
                    const unsigned together = __ballot_sync(0xffffffffu, same);
                    if (in && (!same || lane == leader)) atomicAdd(&hist[d], same ? (uint32_t)__popc(together) : 1u);
                }
            }
            if (size > 1) tc::cluster_sync_all(); else __syncthreads();
            // two bins a thread, from the top digit down, of all CTAs
            const int d = kBins - 2 - 2 * (int)threadIdx.x;
            uint32_t upper = 0, lower = 0;
            if (size > 1) {
                for (int c = 0; c < size; ++c) {
                    upper += ld_cluster(&hist[d + 1], c);
                    lower += ld_cluster(&hist[d], c);
                }
            } else {
                upper = hist[d + 1];
                lower = hist[d];
            }
            uint32_t upto = upper + lower;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, upto, m);
                if (lane >= m) upto += o;
            }
            if (lane == 31) warp_sum[warp][0] = upto;
            __syncthreads();
            uint32_t above = warp_sum[lane][0];  // of warps before: by a sum over the lanes
            above = __reduce_add_sync(0xffffffffu, lane < warp ? above : 0u) + upto - upper - lower;
            if (above < left && above + upper + lower >= left) {
                const bool second = above + upper < left;
                found_digit = (uint32_t)(second ? d : d + 1);
                found_left = left - above - (second ? upper : 0u);
            }
            // (no CTA clears its bins while another reads them)
            if (size > 1) tc::cluster_sync_all(); else __syncthreads();
            value |= found_digit << shift;
            known |= digits << shift;
            left = found_left;
        }
    }
    // which of a lane's four tokens stay for sure, and which are ties, as bits
    auto marks = [&](int g, uint32_t& sures, uint32_t& ties) {
        const uint4 k4 = keys_of(g);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        sures = ties = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + g * 128 + lane * 4 + i;
            const bool middle = j >= lo && j < hi;
            if (j < j1 && (!middle || k[i] > value)) sures |= 1u << i;
            if (j < j1 && middle && k[i] == value) ties |= 1u << i;
        }
    };
    uint32_t sure_n = 0, tie_n = 0;
    for (int g = g0; g < g1; ++g) {
        uint32_t sures, ties;
        marks(g, sures, ties);
        const uint32_t all = __reduce_add_sync(0xffffffffu, (uint32_t)__popc(sures) | (uint32_t)__popc(ties) << 16);
        sure_n += all & 0xffff;
        tie_n += all >> 16;
    }
    if (lane == 0) {
        warp_sum[warp][0] = sure_n;
        warp_sum[warp][1] = tie_n;
    }
    __syncthreads();
    uint32_t sure_before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane][0] : 0u);
    uint32_t ties_before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane][1] : 0u);
    if (size > 1) {
        if (warp == kSelectWarps - 1 && lane == 0) {
            counts[0] = sure_before + sure_n;
            counts[1] = ties_before + tie_n;
        }
        tc::cluster_sync_all();
        for (int c = 0; c < rank; ++c) {
            sure_before += ld_cluster(&counts[0], c);
            ties_before += ld_cluster(&counts[1], c);
        }
        // (no CTA leaves while another reads its counts)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    for (int g = g0; g < g1; ++g) {
        uint32_t sures, ties;
        marks(g, sures, ties);
        const uint32_t mine = (uint32_t)__popc(sures) | (uint32_t)__popc(ties) << 16;
        uint32_t upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += o;
        }
        uint32_t s = sure_before + ((upto - mine) & 0xffff), t = ties_before + ((upto - mine) >> 16);
        const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
        sure_before += all & 0xffff;
        ties_before += all >> 16;
        // (weights that are read anew in each pass may have changed meanwhile: no slot past the row;
        // asked once a group, 0.6 us of 28.0; of each token 1.6)
        const uint32_t budget = (uint32_t)p.budget;
        auto place = [&](auto held) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool sure = sures >> i & 1, tie = ties >> i & 1;
                const uint32_t slot = s + min(t, left);
                if ((sure || (tie && t < left)) && (!decltype(held)::value || slot < budget))
                    kept[slot] = j0 + g * 128 + lane * 4 + i;
                s += sure;
                t += tie;
            }
        };
        if (sure_before + min(ties_before, left) <= budget)
            place(std::false_type{});
        else
            place(std::true_type{});
    }
    if (size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The copies of one thread: 16 bytes of a kept token's key and value codes, and with
// the first lane of a row its scales and weight.
struct EvictRow {
    uint4 k, v;
    uint32_t pk, pv;
    float w;
    bool there;
    int64_t from, to, from_weight, to_weight;

    __device__ __forceinline__ void find(const KvEvictParams& p, int64_t b, int h, int slot, int limit) {
        there = slot < limit;
        if (!there) return;
        const int mask = (1 << p.cache.page_shift) - 1;
        const int64_t to_page = kv_page(p.cache, p.new_table + b * p.new_width, slot >> p.cache.page_shift, p.err);
        const int j = p.kept[(b * p.cache.H + h) * p.budget + slot];
        there = (uint32_t)j < (uint32_t)(p.table_width << p.cache.page_shift);  // (weights changed during the call)
        if (!there) return;
        const int64_t from_page = kv_page(p.cache, p.table + b * p.table_width, j >> p.cache.page_shift, p.err);
        there = from_page >= 0 && to_page >= 0;
        if (!there) return;
        from = kv_row(p.cache, from_page, 0, h, j & mask);
        to = kv_row(p.cache, to_page, 0, h, slot & mask);
        from_weight = kv_weight(p.cache, from_page, h, j & mask);
        to_weight = kv_weight(p.cache, to_page, h, slot & mask);
    }

    __device__ __forceinline__ void load(const KvEvictParams& p, int lane) {
        if (!there) return;
        const int64_t values = (int64_t)p.cache.H << p.cache.page_shift;
        k = *reinterpret_cast<const uint4*>(p.cache.codes + from * p.row_bytes + lane * 16);
        v = *reinterpret_cast<const uint4*>(p.cache.codes + (from + values) * p.row_bytes + lane * 16);
        if (lane == 0) {
            pk = p.cache.params[from];
            pv = p.cache.params[from + values];
            w = p.weights[from_weight];
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

// To pages of their own: rows in any order, kMoveRows a thread, whose loads wait together.
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(const KvEvictParams p) {
    const int lanes = p.row_bytes / 16, side = kMoveThreads / lanes;
    const uint32_t item = blockIdx.x / (uint32_t)p.chunks;
    const int chunk = (int)(blockIdx.x - item * (uint32_t)p.chunks);
    const uint32_t b = item / (uint32_t)p.cache.H;
    const int h = (int)(item - b * (uint32_t)p.cache.H);
    const int lane = threadIdx.x % lanes;
    pdl_wait();
    const int slots = evict_slots(p, b), first = chunk * side * kMoveRows + threadIdx.x / lanes;
    EvictRow row[kMoveRows];
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) row[i].find(p, b, h, first + i * side, slots);
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) row[i].load(p, lane);
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) row[i].store(p, lane);
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
        row.find(p, b, h, s0 + threadIdx.x / lanes, slots);
        row.load(p, lane);
        __syncthreads();
        row.store(p, lane);
    }
}

}  // namespace

bool kv_evict_fits(int64_t B, int64_t H, int64_t row_bytes, int64_t budget) {
    const int64_t side = kMoveRows * kMoveThreads / (row_bytes / 16), chunks = (budget + side - 1) / side;
    return B == 0 || std::max<int64_t>(chunks, 8) < kMaxRows / B / H;
}

cudaError_t launch_kv_evict(KvEvictParams p, const LaunchEnv& env) {
    const int64_t items = p.B * p.cache.H, max_kv = p.table_width << p.cache.page_shift;
    // as many CTAs a sequence's head as keep the keys in shared memory, or as a GPU that
    // would be half empty has room for, while each has some thousand keys (a cluster's
    // barriers cost more than reading those)
    p.cluster = 1;
    while (p.cluster < 8 && (max_kv > (int64_t)kMostKeys * p.cluster ||
                             (2 * items * p.cluster <= env.sm_count && max_kv > 4096 * p.cluster)))
        p.cluster *= 2;
    const int64_t run = ((max_kv + p.cluster - 1) / p.cluster + 127) / 128 * 128;
    p.cached = run <= kMostKeys;
    const size_t smem = p.cached ? (size_t)run * 4 : 0;
    cudaError_t e = allow_smem<kv_select_kernel>(kMostKeys * 4);
    if (e != cudaSuccess) return e;
    e = launch_kernel(kv_select_kernel, dim3((unsigned)(items * p.cluster)), dim3(kSelectThreads), smem, env.stream,
                      dim3(p.cluster, 1, 1), p);
    if (e != cudaSuccess) return e;
    if (p.new_table == p.table)
        return launch_kernel(kv_compact_kernel, dim3((unsigned)items), dim3(kSelectThreads), 0, env.stream, kNoCluster, p);
    const int side = kMoveRows * kMoveThreads / (p.row_bytes / 16);
    p.chunks = (p.budget + side - 1) / side;
    return launch_kernel(kv_move_kernel, dim3((unsigned)(items * p.chunks)), dim3(kMoveThreads), 0, env.stream,
                         kNoCluster, p);
}

}  // namespace i8ql
