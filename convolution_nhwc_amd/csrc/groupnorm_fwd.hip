// Group norm over the pixels and the channels of a group, channels last, forward.
//
// The statistics of a group need all of its elements before the first result.
// Where one block's registers hold a sample's span of groups, it reads x once:
// mean, then the deviations from it, then the results, out of the same
// registers.  Otherwise a first launch leaves the mean and the sum of squared
// deviations of every block's part of a group, and a second one joins a
// sample's parts (a few values a group, every block for itself) and
// normalises; its reading of x comes out of the Infinity Cache where x fits it.
//
// Deviations are always taken from a mean, never as E[x^2] - mean^2 of fp32
// sums, which cancels; parts are joined by
//     M2 = M2a + M2b + (mean_b - mean_a)^2 n_a n_b / (n_a + n_b)
// (Chan, Golub and LeVeque), or in fp64.
//
// 16 x 56 x 56 x 384 fp16 in 32 groups with silu: 25 us, 3.4 TB/s of 86 MB moved (two
// launches 33).  The blocks fill the GPU once and so read, add up and write in
// step, where a copy does all three at once.  8 x 7 x 7 x 2048: 6 us, a launch and the
// latency of one pass.
#include "groupnorm.h"

namespace cnhwc {
namespace {

// z of the thread's channels: gamma rstd (x - mean) + beta.  (The difference comes
// first: gamma rstd x + (beta - gamma rstd mean), an instruction less, is wrong by
// the rounding of the first term where a group hardly spreads about its mean.)
template <typename T>
struct GnLine {
    float mean[kVec<T>], scale[kVec<T>], shift[kVec<T>];

    __device__ __attribute__((always_inline)) inline GnLine(const GnArgs& a, const GnParam<T>& gamma, const GnParam<T>& beta,
                                                            const float (&mu)[kVec<T>], const float (&rstd)[kVec<T>]) {
        gamma.get(a, 1.0f, scale);
        beta.get(a, 0.0f, shift);
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) {
            mean[e] = mu[e];
            scale[e] *= rstd[e];
        }
    }
    __device__ __attribute__((always_inline)) inline float z(float x, int e) const {
        return __builtin_fmaf(x - mean[e], scale[e], shift[e]);
    }
};

// ---- one launch ----

template <typename T, int NV, int SLOTS, bool WHOLE>
__global__ __launch_bounds__(gn_fwd_threads(NV)) void gn_fwd_kernel(const GnArgs a) {
    constexpr int V = kVec<T>, ES = kElemBytes<T>, TH = gn_fwd_threads(NV);
    __shared__ float arr[SLOTS * TH];
    __shared__ float means[SLOTS == 2 ? TH : TH * V];
    __shared__ float rstds[SLOTS == 2 ? TH : TH * V];
    const GnPlace<T> w(a, gn_block(blockIdx.x, gridDim.x), threadIdx.x);
    const int64_t step = int64_t(a.s.ty) * a.x_stride * ES;
    const int have = w.left > 0 ? fdiv(a.pixels - w.ty + a.s.ty - 1, a.s.d_ty) : 0;
    // (threads without elements: the span's first)
    const char* xp = static_cast<const char*>(a.x) +
                     ((w.sample * a.pixels + (have ? w.ty : 0)) * a.x_stride + (have ? w.c0 : w.c_lo)) * ES;
    const GnParam<T> gamma(a, a.gamma, w), beta(a, a.beta, w);
    i32x4 x[NV];
    gn_load<T, WHOLE>(x, xp, step, have, w.left);
    const GnSlots<T, SLOTS> slots(a, w);
    const float total = float(a.pixels) * float(a.each);
    const int64_t out = w.sample * a.groups + w.group0;
    // the mean: sums of each channel, then of the groups
    float v[V], s[SLOTS];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < have) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] += elem<T>(x[i], e);
        }
    slots.sum(s, v, w.dup);
    gn_forget(x);
    gn_group_sums<T, SLOTS>(a, w, s, arr, means, [&](int g, float t) __attribute__((always_inline)) {
        const float m = t / total;
        if (a.mean) a.mean[out + g] = m;
        return m;
    });
    float mean[V];
    slots.spread(mean, means, a, w);
    // the deviations
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < have) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = elem<T>(x[i], e) - mean[e];
                v[e] += d * d;
            }
        }
    if constexpr (!WHOLE) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = e < w.left ? v[e] : 0.0f;
    }
    slots.sum(s, v, w.dup);
    gn_forget(x);
    gn_group_sums<T, SLOTS>(a, w, s, arr, rstds, [&](int g, float t) __attribute__((always_inline)) {
        const float r = 1.0f / sqrtf(t / total + a.eps);
        if (a.rstd) a.rstd[out + g] = r;
        return r;
    });
    if (have == 0) return;
    float rstd[V];
    slots.spread(rstd, rstds, a, w);
    const GnLine<T> line(a, gamma, beta, mean, rstd);
    char* yp = static_cast<char*>(a.y) + ((w.sample * a.pixels + w.ty) * a.y_stride + w.c0) * ES;
    const int64_t ystep = int64_t(a.s.ty) * a.y_stride * ES;
    with_act(a.act, [&](auto ac) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < have) {
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    f[e] = gn_act<T, decltype(ac)::value>(line.z(elem<T>(x[i], e), e));
                gn_put<T, WHOLE>(yp + i * ystep, pack_vec<T>(f), w.left);
            }
    });
}

// ---- two launches ----

constexpr int kPix = 8;   // pixels in registers at a time

template <typename T, bool WHOLE>
__global__ __launch_bounds__(kGnThreads, 4) void gn_stats_kernel(const GnArgs a) {
    constexpr int V = kVec<T>, ES = kElemBytes<T>;
    __shared__ float2 part[kGnThreads * V];   // [pixel row][channel of the span]
    const GnPlace<T> w(a, blockIdx.x, threadIdx.x);
    const int len = w.p1 - w.p0, rows = a.s.ty;
    const int base = fdiv(len, a.s.d_ty), rem = len - base * rows;   // pixels of a row of threads: base, or one more
    if (w.left > 0) {
        float mean[V], m2[V], cnt = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) mean[e] = m2[e] = 0.0f;
        const char* xp = static_cast<const char*>(a.x) + ((w.sample * a.pixels + w.p0 + w.ty) * a.x_stride + w.c0) * ES;
        const int64_t step = int64_t(rows) * a.x_stride * ES;
        const int all = base + (w.ty < rem);
        for (int k = 0; k < all; k += kPix, xp += kPix * step) {
            i32x4 x[kPix];
            const int have = min(kPix, all - k);
#pragma unroll
            for (int i = 0; i < kPix; ++i) x[i] = gn_get<T, WHOLE>(xp + gn_pixel(i, have) * step, w.left);
            const float nb = float(have), inv = 1.0f / nb, tot = 1.0f / (cnt + nb);
            float q[V], s[V];
#pragma unroll
            for (int e = 0; e < V; ++e) s[e] = q[e] = 0.0f;
#pragma unroll
            for (int i = 0; i < kPix; ++i)
                if (i < have) {
#pragma unroll
                    for (int e = 0; e < V; ++e) s[e] += elem<T>(x[i], e);
                }
#pragma unroll
            for (int e = 0; e < V; ++e) s[e] *= inv;
#pragma unroll
            for (int i = 0; i < kPix; ++i)
                if (i < have) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float d = elem<T>(x[i], e) - s[e];
                        q[e] += d * d;
                    }
                }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = s[e] - mean[e];
                mean[e] += d * (nb * tot);
                m2[e] += q[e] + d * d * (cnt * nb * tot);
            }
            cnt += nb;
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e >= w.dup && e < w.left) part[w.ty * w.width + w.cs + e] = float2{mean[e], m2[e]};
    }
    __syncthreads();
    // the span's groups, some lanes each; sums of n mean, n mean^2 and M2 in fp64,
    // where the difference of the squares keeps what fp32 deviations have
    const int used = min(rows, len) * w.gw;
    const int lanes = gn_lanes(blockDim.x, w.groups, used);
    const int l = threadIdx.x & (lanes - 1);
    for (int g = threadIdx.x / lanes; g < w.groups; g += blockDim.x / lanes) {
        double s = 0.0, q = 0.0;
        for (int i = l; i < used; i += lanes) {
            const int y = a.s.pieces > 1 ? i / w.gw : fdiv(i, a.s.d_each);
            const float2 v = part[y * w.width + g * w.gw + (i - y * w.gw)];
            const double k = double(base + (y < rem)), m = double(v.x);
            s += k * m;
            q += k * m * m + double(v.y);
        }
        s = gn_lane_sum(s, lanes);
        q = gn_lane_sum(q, lanes);
        if (l == 0) {
            const double mu = s / (double(len) * double(w.gw));
            a.part[((w.sample * a.s.chunks + w.chunk) * a.groups + w.group0 + g) * a.s.pieces + w.piece] =
                float2{float(mu), float(q - s * mu)};
        }
    }
}

template <typename T, bool WHOLE>
__global__ __launch_bounds__(kGnThreads, 3) void gn_apply_kernel(const GnArgs a) {
    constexpr int V = kVec<T>, ES = kElemBytes<T>;
    __shared__ float2 stat[kGnThreads * V];   // (at most a group a channel)
    const GnPlace<T> w(a, blockIdx.x, threadIdx.x);
    const int len = w.p1 - w.p0, rows = a.s.ty;
    const int base = fdiv(len, a.s.d_ty), all = w.left > 0 ? base + (w.ty < len - base * rows) : 0;
    // (threads without elements: the block's first)
    const char* xp = static_cast<const char*>(a.x) +
                     ((w.sample * a.pixels + w.p0 + (all ? w.ty : 0)) * a.x_stride + (all ? w.c0 : w.c_lo)) * ES;
    const int64_t step = int64_t(rows) * a.x_stride * ES;
    const GnParam<T> gamma(a, a.gamma, w), beta(a, a.beta, w);
    // the first vectors are on their way while the parts are joined
    i32x4 x[kPix];
#pragma unroll
    for (int i = 0; i < kPix; ++i) x[i] = gn_get<T, WHOLE>(xp + gn_pixel(i, all) * step, w.left);
    {
        const int parts = a.s.chunks * a.s.pieces;
        const int lanes = gn_lanes(blockDim.x, w.groups, parts);
        const int l = threadIdx.x & (lanes - 1);
        for (int g = threadIdx.x / lanes; g < w.groups; g += blockDim.x / lanes) {
            const float2* p = a.part + (w.sample * a.s.chunks * a.groups + w.group0 + g) * a.s.pieces;
            double s = 0.0, q = 0.0;
            for (int i0 = l; i0 < parts; i0 += 8 * lanes) {
                float2 v[8];
                double k[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int i = i0 + u * lanes;
                    v[u] = float2{0.0f, 0.0f};
                    k[u] = 0.0;
                    if (i < parts) {
                        const int ch = fdiv(i, a.s.d_pieces), pc = i - ch * a.s.pieces;
                        v[u] = p[int64_t(ch) * a.groups * a.s.pieces + pc];
                        k[u] = double(min(a.s.chunk, a.pixels - ch * a.s.chunk)) *
                               double(a.s.pieces > 1 ? min(a.s.span, a.each - pc * a.s.span) : a.each);
                    }
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const double m = double(v[u].x);
                    s += k[u] * m;
                    q += k[u] * m * m + double(v[u].y);
                }
            }
            s = gn_lane_sum(s, lanes);
            q = gn_lane_sum(q, lanes);
            if (l == 0) {
                const double total = double(a.pixels) * a.each, mu = s / total;
                const float2 r = {float(mu), 1.0f / sqrtf(relu_f(float((q - s * mu) / total)) + a.eps)};
                stat[g] = r;
                if (w.chunk == 0 && w.piece == 0) {
                    const int64_t o = w.sample * a.groups + w.group0 + g;
                    if (a.mean) a.mean[o] = r.x;
                    if (a.rstd) a.rstd[o] = r.y;
                }
            }
        }
    }
    __syncthreads();
    if (all == 0) return;
    float mean[V], rstd[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float2 r = stat[w.group_of(a, e)];
        mean[e] = r.x;
        rstd[e] = r.y;
    }
    const GnLine<T> line(a, gamma, beta, mean, rstd);
    char* yp = static_cast<char*>(a.y) + ((w.sample * a.pixels + w.p0 + w.ty) * a.y_stride + w.c0) * ES;
    const int64_t ystep = int64_t(rows) * a.y_stride * ES;
    with_act(a.act, [&](auto ac) __attribute__((always_inline)) {
        for (int k = 0;;) {
#pragma unroll
            for (int i = 0; i < kPix; ++i)
                if (k + i < all) {
                    float f[V];
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        f[e] = gn_act<T, decltype(ac)::value>(line.z(elem<T>(x[i], e), e));
                    gn_store<T>(yp + i * ystep, pack_vec<T>(f), w.left);
                }
            k += kPix;
            if (k >= all) break;
            xp += kPix * step;
            yp += kPix * ystep;
#pragma unroll
            for (int i = 0; i < kPix; ++i) x[i] = gn_get<T, WHOLE>(xp + gn_pixel(i, all - k) * step, w.left);
        }
    });
}

template <typename T, int NV>
void launch_nv(const GnArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)(a.n * a.s.spans));
    // (a span of groups of at least a vector is one too: only narrower groups' may not be whole)
    if constexpr (!gn_plain_only(NV)) {
        if (a.each < kVec<T>) {
            if (a.s.whole) return gn_fwd_kernel<T, NV, kVec<T>, true><<<grid, a.s.threads, 0, st>>>(a);
            return gn_fwd_kernel<T, NV, kVec<T>, false><<<grid, a.s.threads, 0, st>>>(a);
        }
    }
    gn_fwd_kernel<T, NV, 2, true><<<grid, a.s.threads, 0, st>>>(a);
}

template <typename T>
void launch(const GnArgs& a, hipStream_t st) {
    switch (a.s.nv) {
    case 1: return launch_nv<T, 1>(a, st);
    case 2: return launch_nv<T, 2>(a, st);
    case 4: return launch_nv<T, 4>(a, st);
    case 8: return launch_nv<T, 8>(a, st);
    case 12: return launch_nv<T, 12>(a, st);
    case 32: return launch_nv<T, 32>(a, st);
    }
    const dim3 grid((unsigned)(a.n * a.s.spans * a.s.chunks));
    if (a.s.whole) {
        gn_stats_kernel<T, true><<<grid, a.s.threads, 0, st>>>(a);
        gn_apply_kernel<T, true><<<grid, a.s.threads, 0, st>>>(a);
    } else {
        gn_stats_kernel<T, false><<<grid, a.s.threads, 0, st>>>(a);
        gn_apply_kernel<T, false><<<grid, a.s.threads, 0, st>>>(a);
    }
}

}  // namespace

int launch_groupnorm_fwd(int dtype, const GnArgs& a, hipStream_t st) {
    if (dtype == CNHWC_F32) launch<F32>(a, st);
    else if (dtype == CNHWC_F16) launch<F16>(a, st);
    else launch<BF16>(a, st);
    return CNHWC_OK;
}

}  // namespace cnhwc
