// Rotary positions: pairs of channels of a row turned by the angles of its
// token's position, as the kernels that rotate rows share it.
//
// A table row is rot / 2 cosines, then rot / 2 sines (fp32).  Of a row of D
// channels the first rot are turned: channel i with i + rot / 2, or with
// INTERLEAVED channel 2i with 2i + 1,
//   a' = bf16(fl32(fl32(a cos) - fl32(b sin)))
//   b' = bf16(fl32(fl32(b cos) + fl32(a sin)))
// every operation rounded by itself, so that all kernels (and a host that
// follows the formula) give the same bits.
#pragma once

#include "common.cuh"
#include "quant_math.cuh"

namespace i8ql {

struct RotaryTable {
    const float* rows;
    int64_t count;             // rows
    const int64_t* positions;  // null: token t takes row t
    int rot;                   // channels turned; a row's floats
};

namespace {

// The table row of token t, or null where its position is negative or past
// the table (which is recorded): such a row is not turned.
__device__ __forceinline__ const float* rotary_row(const RotaryTable& r, int64_t t, unsigned* err) {
    const int64_t at = r.positions ? __ldg(r.positions + t) : t;
    if (at < 0) return nullptr;
    if (at >= r.count) {
        record_fault(err, kErrBitBadIndex);
        return nullptr;
    }
    return r.rows + at * r.rot;
}

__device__ __forceinline__ uint32_t rotary_pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// (a, b) turned by (c, s); two pairs at a time, each operation with its own rounding.
__device__ __forceinline__ void rotary_turn2(float (&a)[2], float (&b)[2], const float (&c)[2], const float (&s)[2]) {
    float x[2], y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[i] = __fsub_rn(__fmul_rn(a[i], c[i]), __fmul_rn(b[i], s[i]));
        y[i] = __fadd_rn(__fmul_rn(b[i], c[i]), __fmul_rn(a[i], s[i]));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        a[i] = x[i];
        b[i] = y[i];
    }
}

// 2 W channels of a, paired with the same of b, in words of two channels.
template <int W>
__device__ __forceinline__ void rotary_halves(uint32_t (&a)[W], uint32_t (&b)[W], const float (&c)[2 * W],
                                              const float (&s)[2 * W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
        float x[2] = {lo_bf16(a[i]), hi_bf16(a[i])}, y[2] = {lo_bf16(b[i]), hi_bf16(b[i])};
        const float ci[2] = {c[2 * i], c[2 * i + 1]}, si[2] = {s[2 * i], s[2 * i + 1]};
        rotary_turn2(x, y, ci, si);
        a[i] = rotary_pack(x[0], x[1]);
        b[i] = rotary_pack(y[0], y[1]);
    }
}

// W words, each a pair of its own.
template <int W>
__device__ __forceinline__ void rotary_neighbours(uint32_t (&a)[W], const float* c, const float* s) {
#pragma unroll
    for (int i = 0; i < W; i += 2) {
        float x[2] = {lo_bf16(a[i]), lo_bf16(a[i + 1])}, y[2] = {hi_bf16(a[i]), hi_bf16(a[i + 1])};
        const float ci[2] = {c[i], c[i + 1]}, si[2] = {s[i], s[i + 1]};
        rotary_turn2(x, y, ci, si);
        a[i] = rotary_pack(x[0], y[0]);
        a[i + 1] = rotary_pack(x[1], y[1]);
    }
}

// Which two chunks of W words (2 W channels) of a row the lane'th lane takes:
// the two of a pair first, then those behind the turned channels in order; a
// row takes rotary_lanes lanes.
template <int W, bool INTERLEAVED>
struct RotaryChunks {
    int a, b;   // chunk numbers
    int angle;  // first angle of chunk a; -1: not turned
    // (interleaved) chunk b's first angle follows chunk a's, if it is turned at all
    bool b_there, b_turned;

    __device__ __forceinline__ RotaryChunks(int lane, int D, int rot) {
        const int chunks = D / (2 * W), turned = rot / (2 * W);
        if constexpr (INTERLEAVED) {
            a = 2 * lane;
            angle = a < turned ? a * W : -1;
            b = a + 1;
            b_turned = b < turned;
        } else {
            const bool pair = lane < turned / 2;
            a = pair ? lane : 2 * lane;
            angle = pair ? a * 2 * W : -1;
            b = pair ? lane + turned / 2 : a + 1;
            b_turned = pair;
        }
        b_there = b < chunks;
    }
};

__host__ __device__ constexpr int rotary_lanes(int64_t D, int words) { return (int)((D / (2 * words) + 1) / 2); }

// The angles a lane needs: of chunk a and b, 2 W cosines and sines in all.
template <int W, bool INTERLEAVED>
struct RotaryAngles {
    float c[2 * W], s[2 * W];

    __device__ __forceinline__ void load(const float* row, int rot, const RotaryChunks<W, INTERLEAVED>& at, bool backward) {
        // (interleaved: chunk b's angles are loaded with a's where both are turned)
        const int n = INTERLEAVED && !at.b_turned ? W : 2 * W;
#pragma unroll
        for (int i = 0; i < 2 * W; i += 4) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (i < n) {
                x = __ldg(reinterpret_cast<const float4*>(row + at.angle + i));
                y = __ldg(reinterpret_cast<const float4*>(row + rot / 2 + at.angle + i));
            }
            c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
            s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
        }
        if (backward) {
#pragma unroll
            for (int i = 0; i < 2 * W; ++i) s[i] = -s[i];
        }
    }

    __device__ __forceinline__ void turn(uint32_t (&a)[W], uint32_t (&b)[W], bool b_turned) const {
        if constexpr (INTERLEAVED) {
            rotary_neighbours<W>(a, c, s);
            if (b_turned) rotary_neighbours<W>(b, c + W, s + W);
        } else {
            rotary_halves<W>(a, b, c, s);
        }
    }
};

}  // namespace
}  // namespace i8ql
