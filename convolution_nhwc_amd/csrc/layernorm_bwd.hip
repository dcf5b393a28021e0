// Layer norm over the channels of each row, backward.  With
// xhat = (x - mean) * rstd and g = dy * gamma,
//     dx = rstd * (g - sum(g)/c - xhat * sum(g * xhat)/c)
//     dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy
// One pass reads x and dy once: the lanes of a row keep it in registers
// between the two row sums and dx, and each lane owns the same columns of
// every row its block visits, so the column sums stay in fp32 registers until
// the block has done its rows.  A block then writes one partial row of each
// sum; a second launch adds the partial rows in a fixed order and rounds once.
// Bound by memory: 50176 rows of 384 bf16 take 24 us, 4.9 TB/s of x, dy and dx,
// and the second launch 4 us (an empty one 1.6).
#include "layernorm.h"

namespace cnhwc {
namespace {

template <typename T, typename P, int L, int NV, bool COLS>
__global__ __launch_bounds__(L > 256 ? L : 256) void ln_bwd_kernel(const LnArgs a) {
    constexpr int V = kVec<T>, ES = kElemBytes<T>, PS = kElemBytes<P>;
    constexpr int THREADS = L > 256 ? L : 256, RPB = THREADS / L, WAVES = THREADS / 64;
    constexpr bool JOIN = COLS && L <= 64;       // several waves hold the same columns
    __shared__ float2 red[2][16];
    __shared__ float join[JOIN ? WAVES * L * NV * V : 1];
    int phase = 0;
    const int li = threadIdx.x % L;
    float dg[COLS ? NV : 1][V], db[COLS ? NV : 1][V];
    if constexpr (COLS) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) dg[i][e] = db[i][e] = 0.0f;
    }
    float gamma[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) gamma[i][e] = 1.0f;
    if (a.gamma) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c0 = (i * L + li) * V;
#pragma unroll
            for (int h = 0; h < V; h += kVec<P>) {
                const i32x4 w = load_n<P>(static_cast<const char*>(a.gamma) + int64_t(c0 + h) * PS, a.c - c0 - h);
#pragma unroll
                for (int e = 0; e < kVec<P> && e < V; ++e) gamma[i][h + e] = elem<P>(w, e);
            }
        }
    }
    // a row's loads are issued before the row ahead of it is summed (but for
    // the widest rows, whose 1024 threads have 128 registers each)
    constexpr bool AHEAD = L < 1024;
    i32x4 nx[NV], ndy[NV];
    float nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](int64_t row) __attribute__((always_inline)) {
        const bool any = row < a.rows;
        const char* xp = static_cast<const char*>(a.x) + row * a.x_stride * ES;
        const char* dp = static_cast<const char*>(a.dy) + row * a.y_stride * ES;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c0 = (i * L + li) * V;
            nx[i] = load_n<T>(xp + int64_t(c0) * ES, any ? a.c - c0 : 0);
            ndy[i] = load_n<T>(dp + int64_t(c0) * ES, any ? a.c - c0 : 0);
        }
        if (any) {
            nmean = a.mean[row];
            nrstd = a.rstd[row];
        }
    };
    const int64_t first = int64_t(blockIdx.x) * RPB + threadIdx.x / L, stride = int64_t(gridDim.x) * RPB;
    if (AHEAD) fetch(first);
    for (int64_t row = first; row < a.rows; row += stride) {
        if (!AHEAD) fetch(row);
        i32x4 x[NV], dy[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = nx[i];
            dy[i] = ndy[i];
        }
        const float mean = nmean, rstd = nrstd;
        if (AHEAD) fetch(row + stride);
        float s1 = 0.0f, s2 = 0.0f;
        float g[NV][V];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // (columns past c hold dy = 0, which adds nothing to any sum while
            // mean * rstd is finite)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = elem<T>(dy[i], e), xh = (elem<T>(x[i], e) - mean) * rstd;
                g[i][e] = d * gamma[i][e];
                s1 += g[i][e];
                s2 += g[i][e] * xh;
                if constexpr (COLS) {
                    dg[i][e] += d * xh;
                    db[i][e] += d;
                }
            }
        }
        if (!(__builtin_fabsf(mean * rstd) < __builtin_inff())) {
            // x - mean may be small all the same: the row's own columns alone
            s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if ((i * L + li) * V + e < a.c) s2 += g[i][e] * ((elem<T>(x[i], e) - mean) * rstd);
        }
        row_sum2<L>(s1, s2, red, phase);
        const float m1 = s1 / a.cf, m2 = s2 / a.cf;
        if (a.y) {
            char* op = static_cast<char*>(a.y) + row * a.x_stride * ES;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c0 = (i * L + li) * V;
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (elem<T>(x[i], e) - mean) * rstd;
                    f[e] = rstd * (g[i][e] - m1 - xh * m2);
                }
                store_n<T>(op + int64_t(c0) * ES, pack_vec<T>(f), a.c - c0);
            }
        }
    }
    if constexpr (COLS) {
        float* part = a.part + int64_t(blockIdx.x) * 2 * a.c;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float(*acc)[V] = which == 0 ? dg : db;
            float* out = part + int64_t(which) * a.c;
            if constexpr (JOIN) {
                // rows of one wave first (L = 16), then the waves in order
                if constexpr (L == 16) {
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            acc[i][e] += __shfl_xor(acc[i][e], 16);
                            acc[i][e] += __shfl_xor(acc[i][e], 32);
                        }
                }
                const int wave = threadIdx.x >> 6;
                if (which) __syncthreads();
                if ((threadIdx.x & 63) < L) {
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int e = 0; e < V; ++e) join[wave * (L * NV * V) + (i * L + li) * V + e] = acc[i][e];
                }
                __syncthreads();
                for (int col = threadIdx.x; col < a.c; col += THREADS) {
                    float s = 0.0f;
#pragma unroll
                    for (int w = 0; w < WAVES; ++w) s += join[w * (L * NV * V) + col];
                    out[col] = s;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c0 = (i * L + li) * V;
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (c0 + e < a.c) out[c0 + e] = acc[i][e];
                }
            }
        }
    }
}

// Rows too long for registers: a block a row, two passes over it.
template <typename T, typename P>
__global__ __launch_bounds__(1024) void ln_bwd_long_kernel(const LnArgs a) {
    constexpr int V = kVec<T>, ES = kElemBytes<T>, PS = kElemBytes<P>;
    __shared__ float red[2][16];
    int phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* xp = static_cast<const char*>(a.x) + row * a.x_stride * ES;
        const char* dp = static_cast<const char*>(a.dy) + row * a.y_stride * ES;
        char* op = static_cast<char*>(a.y) + row * a.x_stride * ES;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c0 = int64_t(threadIdx.x) * V; c0 < a.c; c0 += 1024 * V) {
            const int left = int(a.c - c0);
            const i32x4 x = load_n<T>(xp + c0 * ES, left), dy = load_n<T>(dp + c0 * ES, left);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (e < left) {
                    const float g = elem<T>(dy, e) *
                                    (a.gamma ? load1<P>(static_cast<const char*>(a.gamma) + (c0 + e) * PS) : 1.0f);
                    s1 += g;
                    s2 += g * ((elem<T>(x, e) - mean) * rstd);
                }
            }
        }
        const float m1 = row_sum<1024>(s1, red, phase) / a.cf;
        const float m2 = row_sum<1024>(s2, red, phase) / a.cf;
        for (int64_t c0 = int64_t(threadIdx.x) * V; c0 < a.c; c0 += 1024 * V) {
            const int left = int(a.c - c0);
            const i32x4 x = load_n<T>(xp + c0 * ES, left), dy = load_n<T>(dp + c0 * ES, left);
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                f[e] = 0.0f;
                if (e < left) {
                    const float g = elem<T>(dy, e) *
                                    (a.gamma ? load1<P>(static_cast<const char*>(a.gamma) + (c0 + e) * PS) : 1.0f);
                    f[e] = rstd * (g - m1 - (elem<T>(x, e) - mean) * rstd * m2);
                }
            }
            store_n<T>(op + c0 * ES, pack_vec<T>(f), left);
        }
    }
}

// Column sums for such rows: a thread owns one vector of columns, a block
// (blockIdx.x, rows by blockIdx.y) writes one partial row.
template <typename T>
__global__ __launch_bounds__(256) void ln_bwd_cols_kernel(const LnArgs a) {
    constexpr int V = kVec<T>, ES = kElemBytes<T>;
    const int64_t c0 = (int64_t(blockIdx.x) * 256 + threadIdx.x) * V;
    if (c0 >= a.c) return;
    const int left = int(a.c - c0);
    float dg[V], db[V];
#pragma unroll
    for (int e = 0; e < V; ++e) dg[e] = db[e] = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const i32x4 x = load_n<T>(static_cast<const char*>(a.x) + (row * a.x_stride + c0) * ES, left);
        const i32x4 dy = load_n<T>(static_cast<const char*>(a.dy) + (row * a.y_stride + c0) * ES, left);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = elem<T>(dy, e);
            dg[e] += d * ((elem<T>(x, e) - mean) * rstd);
            db[e] += d;
        }
    }
    float* part = a.part + int64_t(blockIdx.y) * 2 * a.c;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (e < left) {
            part[c0 + e] = dg[e];
            part[a.c + c0 + e] = db[e];
        }
    }
}

// Sum of the partial rows, 16 columns by 64 slices of rows a block: each
// slice adds its rows in ascending order, then the slices are added pairwise
// in a fixed order.
template <typename P>
__global__ __launch_bounds__(1024) void ln_reduce_kernel(const float* part, int blocks, int64_t c, void* dgamma,
                                                         void* dbeta) {
    __shared__ float sums[64][17];
    const int lc = threadIdx.x & 15, sl = threadIdx.x >> 4;
    const int64_t col = int64_t(blockIdx.x) * 16 + lc;
    const int64_t c2 = 2 * c;
    float s = 0.0f;
    if (col < c2) {
#pragma unroll 8
        for (int b = sl; b < blocks; b += 64) s += part[int64_t(b) * c2 + col];
    }
    sums[sl][lc] = s;
    for (int h = 32; h > 0; h >>= 1) {
        __syncthreads();
        if (sl < h) sums[sl][lc] += sums[sl + h][lc];
    }
    if (sl == 0 && col < c2) {
        char* out = static_cast<char*>(col < c ? dgamma : dbeta);
        if (out) store1<P>(out + (col < c ? col : col - c) * kElemBytes<P>, sums[0][lc]);
    }
}

constexpr int kBwdMaxVecs = 2048;   // 1024 lanes hold two vectors each within 128 registers

template <typename T, typename P, int L, int NV>
void launch_shape(const LnArgs& a, int blocks, hipStream_t st) {
    constexpr int threads = L > 256 ? L : 256;
    if (a.part) ln_bwd_kernel<T, P, L, NV, true><<<dim3(blocks), threads, 0, st>>>(a);
    else ln_bwd_kernel<T, P, L, NV, false><<<dim3(blocks), threads, 0, st>>>(a);
}

template <typename T, typename P, int L>
void launch_lanes(const LnArgs& a, int nv, int blocks, hipStream_t st) {
    switch (nv) {
    case 1: launch_shape<T, P, L, 1>(a, blocks, st); break;
    case 2: launch_shape<T, P, L, 2>(a, blocks, st); break;
    case 3: launch_shape<T, P, L, 3>(a, blocks, st); break;
    default: launch_shape<T, P, L, 4>(a, blocks, st); break;
    }
}

template <typename T, typename P>
void launch(int dtype, const LnArgs& a, int blocks, hipStream_t st) {
    const LnShape s = ln_shape(a.rows, a.c, dtype, kBwdMaxVecs);
    switch (s.lanes) {
    case 16: launch_lanes<T, P, 16>(a, s.nv, blocks, st); break;
    case 64: launch_lanes<T, P, 64>(a, s.nv, blocks, st); break;
    case 256: launch_lanes<T, P, 256>(a, s.nv, blocks, st); break;
    case 1024:   // 1025..2048 vectors: two a lane
        launch_shape<T, P, 1024, 2>(a, blocks, st);
        break;
    default:
        if (a.y)
            ln_bwd_long_kernel<T, P><<<dim3((unsigned)(a.rows < 65536 ? a.rows : 65536)), 1024, 0, st>>>(a);
        if (a.part) {
            const int64_t cols = (int64_t(a.c) + 256 * kVec<T> - 1) / (256 * kVec<T>);
            ln_bwd_cols_kernel<T><<<dim3((unsigned)cols, (unsigned)blocks), 256, 0, st>>>(a);
        }
    }
}

}  // namespace

int layernorm_bwd_blocks(int dtype, int64_t rows, int64_t c) {
    if (rows <= 0) return 0;
    const LnShape s = ln_shape(rows, c, dtype, kBwdMaxVecs);
    if (s.lanes == 0) return int(rows < 64 ? rows : 64);
    const int rpb = s.lanes > 256 ? 1 : 256 / s.lanes;
    const int64_t steps = (rows + rpb - 1) / rpb;
    // a block's partial sums cost 16 bytes of traffic a column (written and
    // read), a row in 16 bits 6: at least eight row steps a block, once every
    // CU has four blocks (two where a row takes a whole one of 1024 threads)
    const int64_t full = int64_t(kNumCUs) * (s.lanes > 256 ? 2 : 4);
    int64_t b = (steps + 7) / 8;
    if (b < kNumCUs) b = steps < kNumCUs ? steps : kNumCUs;
    return int(b < full ? b : full);
}

int launch_layernorm_bwd(int dtype, int param_dtype, const LnArgs& a, int blocks, hipStream_t st) {
    const bool p32 = param_dtype == CNHWC_F32;
    if (dtype == CNHWC_F32) launch<F32, F32>(dtype, a, blocks, st);
    else if (dtype == CNHWC_F16) p32 ? launch<F16, F32>(dtype, a, blocks, st) : launch<F16, F16>(dtype, a, blocks, st);
    else p32 ? launch<BF16, F32>(dtype, a, blocks, st) : launch<BF16, BF16>(dtype, a, blocks, st);
    return CNHWC_OK;
}

int launch_layernorm_reduce(int param_dtype, const float* part, int blocks, int64_t c, void* dgamma, void* dbeta,
                            hipStream_t st) {
    const dim3 grid((unsigned)((2 * c + 15) / 16));
    if (param_dtype == CNHWC_F32) ln_reduce_kernel<F32><<<grid, 1024, 0, st>>>(part, blocks, c, dgamma, dbeta);
    else if (param_dtype == CNHWC_F16) ln_reduce_kernel<F16><<<grid, 1024, 0, st>>>(part, blocks, c, dgamma, dbeta);
    else ln_reduce_kernel<BF16><<<grid, 1024, 0, st>>>(part, blocks, c, dgamma, dbeta);
    return CNHWC_OK;
}

}  // namespace cnhwc
