// Layer norm over the channels of each row, forward:
//     y = (x - mean) * rstd * gamma + beta
// The row is read once into registers; the mean comes first and the variance
// from the deviations (not from E[x^2] - mean^2, which cancels), both in fp32.
// Bound by memory: 50176 rows of 384 fp16 take 16.1 us, 4.8 TB/s of x and y; a
// copy of 1 GiB reaches 5.1.
#include "layernorm.h"

namespace cnhwc {
namespace {

template <typename T, typename P, int L, int NV>
__global__ __launch_bounds__(L > 256 ? L : 256) void ln_fwd_kernel(const LnArgs a) {
    constexpr int V = kVec<T>, ES = kElemBytes<T>, PS = kElemBytes<P>;
    constexpr int RPB = L > 256 ? 1 : 256 / L;   // rows a block holds at a time
    __shared__ float red[2][16];
    int phase = 0;
    const int li = threadIdx.x % L;
    for (int64_t row = int64_t(blockIdx.x) * RPB + threadIdx.x / L; row < a.rows; row += int64_t(gridDim.x) * RPB) {
        const char* xp = static_cast<const char*>(a.x) + row * a.x_stride * ES;
        char* yp = static_cast<char*>(a.y) + row * a.y_stride * ES;
        i32x4 x[NV];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c0 = (i * L + li) * V;
            x[i] = load_n<T>(xp + int64_t(c0) * ES, a.c - c0);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) s += elem<T>(x[i], e);
        const float mean = row_sum<L>(s, red, phase) / a.cf;
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int left = a.c - (i * L + li) * V;
            if (left >= V) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = elem<T>(x[i], e) - mean;
                    q += d * d;
                }
            } else if (left > 0) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = elem<T>(x[i], e) - mean;
                    if (e < left) q += d * d;
                }
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<L>(q, red, phase) / a.cf + a.eps);
        if (li == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c0 = (i * L + li) * V, left = a.c - c0;
            if (left <= 0) continue;
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = (elem<T>(x[i], e) - mean) * rstd;
            if (a.gamma) {
#pragma unroll
                for (int h = 0; h < V; h += kVec<P>) {
                    const i32x4 g = load_n<P>(static_cast<const char*>(a.gamma) + int64_t(c0 + h) * PS, left - h);
#pragma unroll
                    for (int e = 0; e < kVec<P> && e < V; ++e) f[h + e] *= elem<P>(g, e);
                }
            }
            if (a.beta) {
#pragma unroll
                for (int h = 0; h < V; h += kVec<P>) {
                    const i32x4 b = load_n<P>(static_cast<const char*>(a.beta) + int64_t(c0 + h) * PS, left - h);
#pragma unroll
                    for (int e = 0; e < kVec<P> && e < V; ++e) f[h + e] += elem<P>(b, e);
                }
            }
            store_n<T>(yp + int64_t(c0) * ES, pack_vec<T>(f), left);
        }
    }
}

// Rows too long for registers: a block a row, three passes over it (the
// second and third out of the caches).
template <typename T, typename P>
__global__ __launch_bounds__(1024) void ln_fwd_long_kernel(const LnArgs a) {
    constexpr int V = kVec<T>, ES = kElemBytes<T>, PS = kElemBytes<P>;
    __shared__ float red[2][16];
    int phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* xp = static_cast<const char*>(a.x) + row * a.x_stride * ES;
        char* yp = static_cast<char*>(a.y) + row * a.y_stride * ES;
        float s = 0.0f;
        for (int64_t c0 = int64_t(threadIdx.x) * V; c0 < a.c; c0 += 1024 * V) {
            const i32x4 x = load_n<T>(xp + c0 * ES, int(a.c - c0));
#pragma unroll
            for (int e = 0; e < V; ++e) s += elem<T>(x, e);
        }
        const float mean = row_sum<1024>(s, red, phase) / a.cf;
        float q = 0.0f;
        for (int64_t c0 = int64_t(threadIdx.x) * V; c0 < a.c; c0 += 1024 * V) {
            const i32x4 x = load_n<T>(xp + c0 * ES, int(a.c - c0));
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = elem<T>(x, e) - mean;
                if (c0 + e < a.c) q += d * d;
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<1024>(q, red, phase) / a.cf + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        for (int64_t c0 = int64_t(threadIdx.x) * V; c0 < a.c; c0 += 1024 * V) {
            const int left = int(a.c - c0);
            const i32x4 x = load_n<T>(xp + c0 * ES, left);
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                f[e] = (elem<T>(x, e) - mean) * rstd;
                if (e < left) {
                    if (a.gamma) f[e] *= load1<P>(static_cast<const char*>(a.gamma) + (c0 + e) * PS);
                    if (a.beta) f[e] += load1<P>(static_cast<const char*>(a.beta) + (c0 + e) * PS);
                }
            }
            store_n<T>(yp + c0 * ES, pack_vec<T>(f), left);
        }
    }
}

template <typename T, typename P, int L, int NV>
void launch_shape(const LnArgs& a, hipStream_t st) {
    constexpr int RPB = L > 256 ? 1 : 256 / L;
    const int64_t want = (a.rows + RPB - 1) / RPB;
    const int64_t cap = int64_t(kNumCUs) * 32;
    ln_fwd_kernel<T, P, L, NV><<<dim3((unsigned)(want < cap ? want : cap)), L > 256 ? L : 256, 0, st>>>(a);
}

template <typename T, typename P, int L>
void launch_lanes(const LnArgs& a, int nv, hipStream_t st) {
    switch (nv) {
    case 1: launch_shape<T, P, L, 1>(a, st); break;
    case 2: launch_shape<T, P, L, 2>(a, st); break;
    case 3: launch_shape<T, P, L, 3>(a, st); break;
    default: launch_shape<T, P, L, 4>(a, st); break;
    }
}

template <typename T, typename P>
void launch(int dtype, const LnArgs& a, hipStream_t st) {
    const LnShape s = ln_shape(a.rows, a.c, dtype, 4096);
    switch (s.lanes) {
    case 16: launch_lanes<T, P, 16>(a, s.nv, st); break;
    case 64: launch_lanes<T, P, 64>(a, s.nv, st); break;
    case 256: launch_lanes<T, P, 256>(a, s.nv, st); break;
    case 1024: launch_lanes<T, P, 1024>(a, s.nv, st); break;
    default:
        ln_fwd_long_kernel<T, P><<<dim3((unsigned)(a.rows < 65536 ? a.rows : 65536)), 1024, 0, st>>>(a);
    }
}

}  // namespace

int launch_layernorm_fwd(int dtype, int param_dtype, const LnArgs& a, hipStream_t st) {
    const bool p32 = param_dtype == CNHWC_F32;
    if (dtype == CNHWC_F32) launch<F32, F32>(dtype, a, st);
    else if (dtype == CNHWC_F16) p32 ? launch<F16, F32>(dtype, a, st) : launch<F16, F16>(dtype, a, st);
    else p32 ? launch<BF16, F32>(dtype, a, st) : launch<BF16, BF16>(dtype, a, st);
    return CNHWC_OK;
}

}  // namespace cnhwc
