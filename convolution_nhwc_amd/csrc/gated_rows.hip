// Gated feed-forward for few rows (decoding, small serving batches): every
// weight is read once, so the call is bound by streaming wg and wu.  The
// backward pass of few rows computes its dg and du here.
//
// A weight tile is the 16 rows of a matrix instruction: 8 hidden units' rows
// of wg and the same of wu, so that one instruction gives g and u of 8 units
// for 16 rows of x.  The waves of a block split the reduction in chunks of 64
// channels; a lane reads 16 contiguous bytes of one row per 32-deep product
// straight into the instruction's operand registers.  The waves' sums are
// added through LDS in wave order.
//
// gated_rows_kernel is one persistent block of 16 (or 8) waves a CU: a wave's share
// of x stays in its registers for all of the block's tiles, and the next
// tile's weights are on their way while the current one is added up.  With
// blocks of one tile instead, every tile read x again through the L2, which at
// 24 rows cost as much as the weights (2048 -> 5504 fp16: 16.8 us, of which 12.9
// without x).  Where a wave's share of x does not fit (gated_rows_wide_kernel:
// long rows) x is read per tile, which pays for up to 16 rows.
//
// One row, 2048 -> 8192 bf16: 12.0 us for 67 MB of weights, 5.6 TB/s.  24 rows,
// 2048 -> 5504 fp16: 10.9 us, 4.2 TB/s; at that size a launch's start is a
// quarter of the time.
#include "gated.h"

namespace cnhwc {
namespace {

// This lane's source in the weights: unit fr % 8 of the tile, wg for the first
// 8 lanes and wu for the others.  Units past the end read the last one: their
// results are not stored.
__device__ __attribute__((always_inline)) inline const char* weight_row(const GatedRowsArgs& a, int64_t tile, int fr) {
    const int64_t f = tile * 8 + (fr & 7);
    return static_cast<const char*>(fr < 8 ? a.wg : a.wu) + (f < a.f ? f : a.f - 1) * a.c * 2;
}
__device__ __attribute__((always_inline)) inline const char* x_row(const GatedRowsArgs& a, int64_t r) {
    return static_cast<const char*>(a.x) + (r < a.rows ? r : a.rows - 1) * a.ldx * 2;
}

// The two 32-deep operands of the chunk of 64 channels from k on; channels
// past c read as 0.
template <typename T>
__device__ __attribute__((always_inline)) inline void load_chunk(i32x4 (&r)[2], const char* row, int64_t k, int64_t c,
                                                                 int grp) {
    const char* p = row + (k + grp * 8) * 2;
    if (k + 64 <= c) {
        r[0] = load16<T>(p);
        r[1] = load16<T>(p + 64);
    } else {
        const int64_t left = c - k - grp * 8;
        r[0] = load_n<T>(p, int(left));
        r[1] = load_n<T>(p + 64, int(left - 32));
    }
}

// Adds the waves' sums of one tile and stores its results.
template <typename T, int MT, int WAVES, bool BWD>
__device__ __attribute__((always_inline)) inline void finish_tile(const GatedRowsArgs& a, const float (*sums)[MT][16][17],
                                                                  int64_t tile) {
    for (int i = threadIdx.x; i < MT * 128; i += WAVES * 64) {
        const int c = i & 7, r = (i >> 3) & 15, t = i >> 7;
        const int64_t row = t * 16 + r, f = tile * 8 + c;
        if (row < a.rows && (BWD || f < a.f)) {
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                g += sums[w][t][r][c];
                u += sums[w][t][r][c + 8];
            }
            if constexpr (BWD) {
                float dg = 0.0f, du = 0.0f;
                if (f < a.f) {
                    const float dy = elem<T>(load_n<T>(static_cast<const char*>(a.dy) + (row * a.lddy + f) * 2, 1), 0);
                    float v, d;
                    act_both(a.act, g, v, d);
                    dg = dy * u * d;
                    du = dy * v;
                }
                char* o = static_cast<char*>(a.dgu) + (row * 2 * a.fp + f) * 2;
                store1<T>(o, dg);
                store1<T>(o + a.fp * 2, du);
            } else {
                store1<T>(static_cast<char*>(a.y) + (row * a.ldy + f) * 2, act_value(a.act, g) * u);
            }
        }
    }
}

// MT: 16-row tiles of x; NC: chunks a wave.
template <typename T, int MT, int WAVES, int NC, bool BWD>
__global__ __launch_bounds__(WAVES * 64) void gated_rows_kernel(const GatedRowsArgs a) {
    __shared__ float sums[2][WAVES][MT][16][17];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, grp = lane >> 4;
    const int64_t tiles = (a.f + 7) / 8;
    i32x4 w[NC][2], next[NC][2], x[NC][MT][2];
    auto fetch = [&](int64_t tile) __attribute__((always_inline)) {
        const char* row = weight_row(a, tile < tiles ? tile : tiles - 1, fr);
#pragma unroll
        for (int i = 0; i < NC; ++i) load_chunk<T>(next[i], row, int64_t(wave + i * WAVES) * 64, a.c, grp);
    };
    fetch(blockIdx.x);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < NC; ++i)
            load_chunk<T>(x[i][t], x_row(a, t * 16 + fr), int64_t(wave + i * WAVES) * 64, a.c, grp);
    int buf = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) w[i][h] = next[i][h];
        if (tile + gridDim.x < tiles) fetch(tile + gridDim.x);
        __builtin_amdgcn_sched_barrier(0);   // the next tile's loads go out before this one's are waited for
        f32x4 acc[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[t] = mfma16x16x32<T>(w[i][h], x[i][t][h], acc[t]);
        // lane: units 4*grp..+3 of (g | u), row t*16 + fr
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[buf][wave][t][fr][4 * grp + e] = acc[t][e];
        // one barrier a tile: a wave writes this buffer again only after the
        // next tile's barrier, which it shares with those still reading here
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
        finish_tile<T, MT, WAVES, BWD>(a, sums[buf], tile);
        buf ^= 1;
    }
}

// One tile a block, x read with the weights, D chunks at a time.
template <typename T, int MT, int WAVES, int D, bool BWD>
__global__ __launch_bounds__(WAVES * 64) void gated_rows_wide_kernel(const GatedRowsArgs a) {
    __shared__ float sums[WAVES][MT][16][17];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, grp = lane >> 4;
    const char* row = weight_row(a, blockIdx.x, fr);
    const char* xp[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) xp[t] = x_row(a, t * 16 + fr);
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t chunks = (a.c + 63) / 64;
    for (int64_t q = wave; q < chunks; q += D * WAVES) {
        i32x4 w[D][2], x[D][MT][2];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            load_chunk<T>(w[d], row, (q + d * WAVES) * 64, a.c, grp);
#pragma unroll
            for (int t = 0; t < MT; ++t) load_chunk<T>(x[d][t], xp[t], (q + d * WAVES) * 64, a.c, grp);
        }
        __builtin_amdgcn_sched_barrier(0);   // every load is issued before the first product waits
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[t] = mfma16x16x32<T>(w[d][h], x[d][t][h], acc[t]);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[wave][t][fr][4 * grp + e] = acc[t][e];
    __syncthreads();
    finish_tile<T, MT, WAVES, BWD>(a, sums, blockIdx.x);
}

constexpr int waves_of(int mt) { return mt == 4 ? 8 : 16; }
constexpr int most_of(int mt, bool bwd) { return mt == 2 || (bwd && mt == 1) ? 2 : 4; }

template <typename T, int MT, int WAVES, int NC, bool BWD>
int launch_kept(const GatedRowsArgs& a, hipStream_t st) {
    const int64_t tiles = (a.f + 7) / 8;
    const dim3 grid((unsigned)(tiles < kNumCUs ? tiles : kNumCUs));
    gated_rows_kernel<T, MT, WAVES, NC, BWD><<<grid, WAVES * 64, 0, st>>>(a);
    return CNHWC_OK;
}

template <typename T, int MT, bool BWD>
int launch(const GatedRowsArgs& a, hipStream_t st) {
    // a wave has 128 registers in a block of 16 and 256 in one of 8; its chunks
    // of x take 8 * MT of them each, two tiles' weights 16 (four chunks of the
    // backward pass spill in a block of 16)
    constexpr int W = waves_of(MT), MOST = most_of(MT, BWD);
    const int64_t nc = ((a.c + 63) / 64 + W - 1) / W;
    if (nc == 1) return launch_kept<T, MT, W, 1, BWD>(a, st);
    if (nc == 2) return launch_kept<T, MT, W, 2, BWD>(a, st);
    if (nc <= MOST) return launch_kept<T, MT, W, MOST, BWD>(a, st);
    if constexpr (BWD && MT > 1) {
        return CNHWC_UNSUPPORTED;   // these go to the tiles: the weights' copy is made for them in any case
    } else {
        gated_rows_wide_kernel<T, MT, 8, MT == 1 ? 4 : MT == 2 ? 2 : 1, BWD>
            <<<dim3((unsigned)((a.f + 7) / 8)), 512, 0, st>>>(a);
        return CNHWC_OK;
    }
}

template <typename T, bool BWD>
int launch_t(const GatedRowsArgs& a, hipStream_t st) {
    if (a.rows <= 16) return launch<T, 1, BWD>(a, st);
    if (a.rows <= 32) return launch<T, 2, BWD>(a, st);
    return launch<T, 4, BWD>(a, st);
}

}  // namespace

bool gated_rows_kept(int64_t rows, int64_t c, bool bwd) {
    const int mt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    return (c + 63) / 64 <= int64_t(waves_of(mt)) * most_of(mt, bwd);
}

int launch_gated_rows(int dtype, const GatedRowsArgs& a, hipStream_t st) {
    if (dtype == CNHWC_F16) return a.dgu ? launch_t<F16, true>(a, st) : launch_t<F16, false>(a, st);
    return a.dgu ? launch_t<BF16, true>(a, st) : launch_t<BF16, false>(a, st);
}

}  // namespace cnhwc
