// Row shapes of the layer-norm kernels: L lanes share a row and each holds NV
// vectors of 16 bytes, so a row is read once and stays in registers between
// its statistics and its result.
#pragma once

#include "mix.h"

namespace cnhwc {

// The shapes cover 64, 256, 1024 and (forward) 4096 vectors; longer rows take
// the looped kernels.  The least L that holds the row: a sum over 16 lanes is
// four in-register rotations, over 64 two exchanges more, beyond that it goes
// through LDS.
struct LnShape {
    int lanes;   // 16, 64, 256, 1024; 0: looped kernel
    int nv;      // 1..4
};

inline LnShape ln_shape(int64_t rows, int64_t c, int dtype, int max_vecs) {
    const int v = dtype == CNHWC_F32 ? 4 : 8;
    const int64_t vecs = (c + v - 1) / v;
    if (vecs > max_vecs) return {0, 0};
    int lanes = 16;
    while (vecs > int64_t(lanes) * 4) lanes *= 4;
    // few rows: spread each over more lanes while that gives them work and
    // CUs would stay idle (392 rows of 2048 bf16 forward: 64 lanes a row 5.5 us,
    // 256 lanes 4.1 us)
    while (lanes < 256 && vecs > lanes && rows * lanes < int64_t(kNumCUs) * 512) lanes *= 4;
    return {lanes, int((vecs + lanes - 1) / lanes)};
}

#ifdef __HIPCC__

// Sum over the L lanes of a row, in every lane.  Rows of more than a wave go
// through `red`, which alternates between two halves so that one barrier a
// sum is enough.
template <int L>
__device__ inline float row_sum(float v, float (*red)[16], int& phase) {
    if constexpr (L <= 64) {
        return lane_sum<L>(v);
    } else {
        v = lane_sum<64>(v);
        float* r = red[phase];
        phase ^= 1;
        if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = v;
        __syncthreads();
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < L / 64; ++w) s += r[w];
        return s;
    }
}

// Two sums at once.
template <int L>
__device__ inline void row_sum2(float& u, float& v, float2 (*red)[16], int& phase) {
    if constexpr (L <= 64) {
        u = lane_sum<L>(u);
        v = lane_sum<L>(v);
    } else {
        u = lane_sum<64>(u);
        v = lane_sum<64>(v);
        float2* r = red[phase];
        phase ^= 1;
        if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = float2{u, v};
        __syncthreads();
        u = v = 0.0f;
#pragma unroll
        for (int w = 0; w < L / 64; ++w) {
            u += r[w].x;
            v += r[w].y;
        }
    }
}

#endif

}  // namespace cnhwc
