// Gated feed-forward for few rows (decoding, small serving batches): every
// weight is read once, so the call is bound by streaming wg and wu.
//
// A block owns 16 hidden units.  Its waves split the reduction in chunks of 64
// channels; a lane reads 32 contiguous bytes of one weight row per chunk (a
// quarter of a 128-byte line, the wave reads whole lines) straight into the
// matrix instruction's operand registers: the two 32-deep products of a chunk
// take the lane's first and second 8 channels, an order of the reduction that
// x follows.  x comes from the L2.  The waves' sums are added through LDS in
// wave order.
#include "gated.h"

namespace cnhwc {
namespace {

template <typename T, int MT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void gated_rows_kernel(const GatedRowsArgs a) {
    __shared__ float sums[WAVES][2][MT][16][17];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int fr = lane & 15, grp = lane >> 4;
    const int64_t f0 = int64_t(blockIdx.x) * 16;
    // rows past the end read the last one: their results are not stored
    const int64_t fw = f0 + fr < a.f ? f0 + fr : a.f - 1;
    const char* gp = static_cast<const char*>(a.wg) + (fw * a.c + grp * 16) * 2;
    const char* up = static_cast<const char*>(a.wu) + (fw * a.c + grp * 16) * 2;
    const char* xp[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t r = t * 16 + fr;
        xp[t] = static_cast<const char*>(a.x) + ((r < a.rows ? r : a.rows - 1) * a.ldx + grp * 16) * 2;
    }
    f32x4 ag[MT], au[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) ag[t] = au[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto chunk = [&](int64_t k, auto whole) {
        constexpr bool W = decltype(whole)::value != 0;
        i32x4 g[2], u[2], x[MT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t o = (k + h * 8) * 2;
            const int left = W ? 8 : int(a.c - (k + grp * 16 + h * 8));
            if constexpr (W) {
                g[h] = load16<T>(gp + o);
                u[h] = load16<T>(up + o);
            } else {
                g[h] = load_n<T>(gp + o, left);
                u[h] = load_n<T>(up + o, left);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if constexpr (W) x[t][h] = load16<T>(xp[t] + o);
                else x[t][h] = load_n<T>(xp[t] + o, left);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                ag[t] = mfma16x16x32<T>(g[h], x[t][h], ag[t]);
                au[t] = mfma16x16x32<T>(u[h], x[t][h], au[t]);
            }
    };
    const int64_t whole = a.c / 64;
    int64_t q = wave;
#pragma unroll 4
    for (; q < whole; q += WAVES) chunk(q * 64, IC<1>{});
    if (q == whole && a.c % 64) chunk(q * 64, IC<0>{});

    // lane: hidden units 4*grp..+3 of row t*16 + fr
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sums[wave][0][t][fr][4 * grp + e] = ag[t][e];
            sums[wave][1][t][fr][4 * grp + e] = au[t][e];
        }
    __syncthreads();
    for (int i = tid; i < MT * 256; i += WAVES * 64) {
        const int t = i >> 8, r = (i >> 4) & 15, c = i & 15;
        const int64_t row = t * 16 + r, f = f0 + c;
        if (row < a.rows && f < a.f) {
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                g += sums[w][0][t][r][c];
                u += sums[w][1][t][r][c];
            }
            store1<T>(static_cast<char*>(a.y) + (row * a.ldy + f) * 2, act_value(a.act, g) * u);
        }
    }
}

template <typename T, int MT>
void launch(const GatedRowsArgs& a, hipStream_t st) {
    const int64_t blocks = (a.f + 15) / 16;
    // enough waves to keep the memory busy: 8 a CU where the reduction has
    // that many chunks
    const int64_t chunks = (a.c + 63) / 64;
    if (MT <= 2 && blocks * 4 < kNumCUs * 8 && chunks >= 16)
        gated_rows_kernel<T, MT, MT <= 2 ? 8 : 4><<<dim3((unsigned)blocks), MT <= 2 ? 512 : 256, 0, st>>>(a);
    else
        gated_rows_kernel<T, MT, 4><<<dim3((unsigned)blocks), 256, 0, st>>>(a);
}

template <typename T>
void launch_t(const GatedRowsArgs& a, hipStream_t st) {
    if (a.rows <= 16) launch<T, 1>(a, st);
    else if (a.rows <= 32) launch<T, 2>(a, st);
    else launch<T, 4>(a, st);
}

}  // namespace

int launch_gated_rows(int dtype, const GatedRowsArgs& a, hipStream_t st) {
    if (dtype == CNHWC_F16) launch_t<F16>(a, st);
    else launch_t<BF16>(a, st);
    return CNHWC_OK;
}

}  // namespace cnhwc
