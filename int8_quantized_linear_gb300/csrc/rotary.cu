// Rotary positions: tables of angles, and rows turned by them (forward, and
// backward as their gradient is).
//
//   table: row r stands for position p (r, or positions[r]):
//     cos(p f_i) a, then sin(p f_i) a   (f_i radians a position, a the amplitude)
//   apply: rotary.cuh.  Bound by bytes: rows read and written once.
//
// The angle of a far position is many turns, of which only the fraction
// counts: fp32 would leave none of it (p f = 10^5 is known to 2^-8), fp64 is
// slow here.  A frequency is turned into fractions of a turn in fixed point once,
//   u = round(2^64 frac(f / 2 pi)),   frac(p f / 2 pi) = (p u mod 2^64) / 2^64,
// and the product wraps by itself: exact but for u's rounding (|p| 2^-65
// turns) and what 1 / 2 pi in two doubles leaves (f 2^-107).  The nearest quarter
// turn comes off as an integer; the rest, an eighth at most, becomes an angle of up to
// pi / 4 in fp32, whose sine and cosine are the first terms of their series (sine to the
// 9th power, 2^-29; cosine to the 10th, 2^-33).

#include <cuda_runtime.h>

#include <algorithm>

#include "rotary.cuh"

namespace i8ql {
namespace {

constexpr int kTableThreads = 256;
constexpr int kTableBlocks = 4;  // an SM

// A thread has one frequency, and rows apart.  131072 positions of 64 frequencies:
// 12.7 us, of 10 for the 67 MB that are written (issue slots 73 %: about 35 instructions an
// angle; 24.3 with a 64-bit product and calls of sine and cosine for each); by positions,
// which cannot be stepped, 17.8.
template <bool RANGE>
__global__ void __launch_bounds__(kTableThreads) rotary_table_kernel(const double* __restrict__ freqs,
                                                                     const int64_t* __restrict__ positions,
                                                                     float* __restrict__ table, int64_t P, int F,
                                                                     float amplitude) {
    const int side = kTableThreads / F;  // rows side by side
    const int i = threadIdx.x % F, r = threadIdx.x / F;
    pdl_wait();
    if (r >= side) return;
    // f / (2 pi), 1 / (2 pi) as the sum of two doubles
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double f = __ldg(freqs + i);
    const double hi = f * kHi, lo = fma(f, kHi, -hi) + f * kLo;
    // (exact for either sign: of what truncation leaves, the magnitude, below 2^64)
    const double part = hi - trunc(hi);
    const unsigned long long whole = (unsigned long long)rint(fabs(part) * 0x1p64);
    const unsigned long long u = (part < 0.0 ? 0ull - whole : whole) + (unsigned long long)llrint(lo * 0x1p64);
    // (positions in order: the next angle is a step further; no product)
    const uint32_t step = gridDim.x * side, first = blockIdx.x * side + r;
    uint64_t turn = (uint64_t)first * u;
    const uint64_t turn_step = (uint64_t)step * u;
    float* out = table + (int64_t)first * 2 * F + i;
    const int64_t out_step = (int64_t)step * 2 * F;
    const int count = first < P ? (int)((P - first + step - 1) / step) : 0;
    const int64_t* at = positions + first;
#pragma unroll 4
    for (int k = 0; k < count; ++k) {
        if constexpr (!RANGE) {
            turn = (uint64_t)__ldg(at) * u;
            at += step;
        }
        const uint32_t top = (uint32_t)(turn >> 32), q = (top + (1u << 29)) >> 30;  // nearest quarter
        const int32_t high = (int32_t)(top - (q << 30));
        // the rest in radians: its high word, and 23 bits of its low word in the mantissa of 1
        const float low = __uint_as_float((uint32_t)turn >> 9 | 0x3f800000u) - 1.0f;
        constexpr float kTurn = 6.283185307f * 0x1p-32f;
        const float x = fmaf((float)high, kTurn, low * kTurn), xx = x * x;
        const float s = x * fmaf(fmaf(fmaf(fmaf(xx, 1.0f / 362880.0f, -1.0f / 5040.0f), xx, 1.0f / 120.0f), xx, -1.0f / 6.0f),
                                 xx, 1.0f);
        const float c =
            fmaf(fmaf(fmaf(fmaf(fmaf(xx, -1.0f / 3628800.0f, 1.0f / 40320.0f), xx, -1.0f / 720.0f), xx, 1.0f / 24.0f), xx, -0.5f),
                 xx, 1.0f);
        const float a = q & 2 ? -amplitude : amplitude;
        out[0] = (q & 1 ? -s : c) * a;
        out[F] = (q & 1 ? c : s) * a;
        out += out_step;
        if constexpr (RANGE) turn += turn_step;
    }
}

struct RotaryApplyParams {
    const uint16_t* x;
    int64_t x_stride;
    uint16_t* out;
    int64_t out_stride;
    RotaryTable table;
    uint32_t rows;   // tokens x groups of heads
    int lanes;       // of a row
    int groups;      // of heads
    int heads;
    int D;
    bool backward;
    bool in_place;
    unsigned* err;
};

template <int W>
__device__ __forceinline__ void load_words(const uint16_t* p, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    }
}

template <int W>
__device__ __forceinline__ void store_words(uint16_t* p, const uint32_t (&w)[W]) {
    if constexpr (W == 4)
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

constexpr int kApplyThreads = 128;

// A thread takes two chunks of 2 W channels of HEADS heads of a token.
template <int W, bool INTERLEAVED, int HEADS>
__global__ void __launch_bounds__(kApplyThreads) rotary_apply_kernel(const RotaryApplyParams p) {
    const int side = kApplyThreads / p.lanes;
    const int r = threadIdx.x / p.lanes, lane = threadIdx.x - r * p.lanes;
    const int64_t row = (int64_t)blockIdx.x * side + r;
    pdl_wait();
    if (r >= side || row >= p.rows) return;
    const uint32_t t = (uint32_t)row / (uint32_t)p.groups;
    const int h0 = ((uint32_t)row - t * p.groups) * HEADS;
    const RotaryChunks<W, INTERLEAVED> at(lane, p.D, p.table.rot);
    const uint16_t* src = p.x + t * p.x_stride + (int64_t)h0 * p.D;
    uint16_t* dst = p.out + t * p.out_stride + (int64_t)h0 * p.D;
    uint32_t a[HEADS][W], b[HEADS][W];
    const bool moves = !p.in_place || at.angle >= 0;
    if (!moves) return;
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        if (h0 + h < p.heads) {
            load_words<W>(src + h * p.D + at.a * 2 * W, a[h]);
            if (at.b_there) load_words<W>(src + h * p.D + at.b * 2 * W, b[h]);
        }
    }
    const float* angles = rotary_row(p.table, t, p.err);
    const bool turned = angles != nullptr && at.angle >= 0;
    RotaryAngles<W, INTERLEAVED> angle;
    if (turned) angle.load(angles, p.table.rot, at, p.backward);
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        if (h0 + h >= p.heads) break;
        if (turned) angle.turn(a[h], b[h], at.b_turned);
        store_words<W>(dst + h * p.D + at.a * 2 * W, a[h]);
        if (at.b_there) store_words<W>(dst + h * p.D + at.b * 2 * W, b[h]);
    }
}

template <int W, bool INTERLEAVED>
cudaError_t launch_apply(RotaryApplyParams p, int64_t T, const LaunchEnv& env) {
    p.lanes = rotary_lanes(p.D, W);
    const int side = kApplyThreads / p.lanes;
    auto grid = [&](int heads) {
        p.groups = (p.heads + heads - 1) / heads;
        p.rows = (uint32_t)(T * p.groups);
        return dim3((unsigned)(((int64_t)p.rows + side - 1) / side));
    };
    // two heads a thread share the angles, where enough threads are left (8001 tokens of 32
    // heads x 96 channels, half of them turned: 18.5 us, 19.6 with one, 19.2 with four)
    const dim3 many = grid(2);
    if (many.x >= 4u * (unsigned)env.sm_count)
        return launch_kernel(rotary_apply_kernel<W, INTERLEAVED, 2>, many, dim3(kApplyThreads), 0, env.stream,
                             kNoCluster, p);
    const dim3 few = grid(1);
    return launch_kernel(rotary_apply_kernel<W, INTERLEAVED, 1>, few, dim3(kApplyThreads), 0, env.stream, kNoCluster, p);
}

}  // namespace

cudaError_t launch_rotary_table(const double* freqs, const int64_t* positions, float* table, int64_t P, int64_t F,
                                float amplitude, const LaunchEnv& env) {
    const int64_t rows = kTableThreads / F;
    const int64_t blocks = std::min<int64_t>((P + rows - 1) / rows, kTableBlocks * (int64_t)env.sm_count);
    return launch_kernel(positions ? rotary_table_kernel<false> : rotary_table_kernel<true>, dim3((unsigned)blocks),
                         dim3(kTableThreads), 0, env.stream, kNoCluster, freqs, positions, table, P, (int)F, amplitude);
}

cudaError_t launch_rotary_apply(const uint16_t* x, int64_t x_stride, const RotaryTable& table, uint16_t* out,
                                int64_t out_stride, int64_t T, int64_t heads, int64_t D, bool interleaved,
                                bool backward, const LaunchEnv& env) {
    RotaryApplyParams p = {};
    p.x = x;
    p.x_stride = x_stride;
    p.out = out;
    p.out_stride = out_stride;
    p.table = table;
    p.heads = (int)heads;
    p.D = (int)D;
    p.backward = backward;
    p.in_place = x == out;
    p.err = env.err;
    if (interleaved) return launch_apply<4, true>(p, T, env);
    return table.rot % 16 == 0 ? launch_apply<4, false>(p, T, env) : launch_apply<2, false>(p, T, env);
}

}  // namespace i8ql
