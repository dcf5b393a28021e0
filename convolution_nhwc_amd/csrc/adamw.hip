// One AdamW step over many tensors of any length and type:
//     m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//     p -= lr (decay p + (m / c1) / (sqrt(v / c2) + eps)),  copy = p in 16 bits
// A launch takes up to 52 tensors, whose pointers travel in its arguments; a
// block finds its tensor by the block numbers they start at and updates 1024 or 2048
// elements of it, a wave 256 at a time (four a lane).  Bound by memory: 28
// bytes an element with fp32 moments, 16-bit gradients and a 16-bit copy, 16
// with 8-bit moments.  50.4 million elements: 262 us, 5.4 TB/s, and 157 to 162, 5.1 TB/s
// with the vector units 93 % busy.  Tensors of a small model, 52 a launch (2.6
// million elements): 15 us, three quarters of it latencies (the arguments', the loads',
// the fp64 chain's).
//
// 8-bit moments: a wave's 256 elements share a scale, the largest |m| (v), and a
// code has 3 mantissa bits under 4 (m, signed) or 5 (v) exponent bits, so that
// the second moments keep 2^32 of range and the step its proportions.  Half a
// step of such a code is up to 6 %, more than beta2 = 0.999 moves a moment in
// 60 steps; so a value goes to one of its two neighbours by a drawn number,
// and the moments are right on average.  The border that the drawn number sets
// between two codes,
//     (code + (r + 1/2) / 65536) in the code's own exponent, times the scale,
// is a product of 20 and 24 bits and exact in fp64; with m and v computed in
// fp64 too, in a given order, the codes follow from the definition to the bit.
// (fp64 runs at the rate of fp32 on this GPU.)
#include "adamw.h"
#include "philox.h"

namespace cnhwc {
namespace {

template <int N, int A>
struct __attribute__((packed, aligned(A))) Raw {
    uint32_t w[N];
};

// Four elements as they lie in memory: 16 bytes of fp32, 8 of 16-bit types.  FULL:
// all four are there; otherwise `left` of them.  (Checked at every access, ends
// cost a third of the kernel.)
template <bool FULL>
__device__ __attribute__((always_inline)) inline i32x4 load4(const void* base, int64_t i, bool f32, int left) {
    i32x4 r = {0, 0, 0, 0};
    if (f32) {
        const char* p = static_cast<const char*>(base) + i * 4;
        if (FULL || left >= 4) {
            const Raw<4, 4> v = *reinterpret_cast<const Raw<4, 4>*>(p);
            r = i32x4{int(v.w[0]), int(v.w[1]), int(v.w[2]), int(v.w[3])};
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < left) r[e] = reinterpret_cast<const int*>(p)[e];
        }
    } else {
        const char* p = static_cast<const char*>(base) + i * 2;
        if (FULL || left >= 4) {
            const Raw<2, 2> v = *reinterpret_cast<const Raw<2, 2>*>(p);
            r[0] = int(v.w[0]);
            r[1] = int(v.w[1]);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < left) r[e >> 1] |= int(uint32_t(reinterpret_cast<const unsigned short*>(p)[e]) << (16 * (e & 1)));
        }
    }
    return r;
}
__device__ __attribute__((always_inline)) inline void unpack4(float* f, const i32x4& r, int type) {
    if (type == CNHWC_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = elem<F32>(r, e);
    } else if (type == CNHWC_BF16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = elem<BF16>(r, e);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = elem<F16>(r, e);
    }
}
template <bool FULL>
__device__ __attribute__((always_inline)) inline void store4(void* base, int64_t i, const float* f, int type, int left) {
    if (type == CNHWC_F32) {
        char* p = static_cast<char*>(base) + i * 4;
        if (FULL || left >= 4) {
            Raw<4, 4> v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v.w[e] = __builtin_bit_cast(uint32_t, f[e]);
            *reinterpret_cast<Raw<4, 4>*>(p) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < left) reinterpret_cast<float*>(p)[e] = f[e];
        }
    } else {
        char* p = static_cast<char*>(base) + i * 2;
        const bool bf = type == CNHWC_BF16;
        const Raw<2, 2> v = {{bf ? pack2<BF16>(f[0], f[1]) : pack2<F16>(f[0], f[1]),
                              bf ? pack2<BF16>(f[2], f[3]) : pack2<F16>(f[2], f[3])}};
        if (FULL || left >= 4) {
            *reinterpret_cast<Raw<2, 2>*>(p) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < left)
                    reinterpret_cast<unsigned short*>(p)[e] = (unsigned short)(v.w[e >> 1] >> (16 * (e & 1)));
        }
    }
}
// Four codes.
template <bool FULL>
__device__ __attribute__((always_inline)) inline uint32_t load_codes(const void* base, int64_t i, int left) {
    const unsigned char* p = static_cast<const unsigned char*>(base) + i;
    if (FULL || left >= 4) return reinterpret_cast<const Raw<1, 1>*>(p)->w[0];
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < left) r |= uint32_t(p[e]) << (8 * e);
    return r;
}
template <bool FULL>
__device__ __attribute__((always_inline)) inline void store_codes(void* base, int64_t i, uint32_t c, int left) {
    unsigned char* p = static_cast<unsigned char*>(base) + i;
    if (FULL || left >= 4) {
        reinterpret_cast<Raw<1, 1>*>(p)->w[0] = c;
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < left) p[e] = (unsigned char)(c >> (8 * e));
}

// A code's value without its scale: exponent field and fraction are those of an
// fp32 number whose least normal exponent is moved to the code's (bits: 4 for
// m, 5 for v): its bits here, times kUp.
template <int BITS>
constexpr float kUp = BITS == 4 ? 0x1p112f : 0x1p96f;
__device__ __attribute__((always_inline)) inline float m_bits(uint32_t codes, int e) {   // with its sign
    const uint32_t c = codes >> (8 * e);
    return __builtin_bit_cast(float, (c << 20 & 0x07f00000u) | (c << 24 & 0x80000000u));
}
__device__ __attribute__((always_inline)) inline float v_bits(uint32_t codes, int e) {
    return __builtin_bit_cast(float, (codes >> (8 * e) & 255u) << 20);
}

// A scale, in the forms that encode needs.
template <int BITS>
struct Scale {
    double up;            // scale * kUp
    float near, inv;      // scale * near has a reciprocal, inv
    __device__ __attribute__((always_inline)) inline explicit Scale(float s) {
        up = double(s) * double(kUp<BITS>);
        near = s < 0x1p-60f ? 0x1p64f : s > 0x1p60f ? 0x1p-64f : 1.0f;
        inv = __builtin_amdgcn_rcpf(s * near);
    }
    // The code of 0 <= a (at most about the scale; af: in fp32).  The quotient only
    // picks a neighbour, the exact border decides: taken one too low next to a
    // code's own value, the border of the code below still leads up to it.
    __device__ __attribute__((always_inline)) inline uint32_t encode(double a, float af, uint32_t r16) const {
        constexpr uint32_t top = BITS == 4 ? 15u << 3 : 31u << 3;
        const float t = fminf(af * near * inv, 1.0f) * (1.0f / kUp<BITS>);
        const uint32_t c = __builtin_bit_cast(uint32_t, t) >> 20;
        const float border = __builtin_bit_cast(float, (c << 20) | (r16 << 4) | 8u);
        const uint32_t n = a > double(border) * up ? c + 1 : c;
        return n < top ? n : top;
    }
};

// The largest of a wave, as unsigned words (of non-negative floats in order,
// infinity and NaN above all others): along each 16 lanes, then from row to row.
template <int CTRL, int ROWS>
__device__ __attribute__((always_inline)) inline uint32_t dpp_max(uint32_t v) {
    const uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xf, false));
    return o > v ? o : v;
}
__device__ __attribute__((always_inline)) inline uint32_t wave_max(uint32_t v) {
    v = dpp_max<0x111, 0xf>(v);   // from the lanes 1, 2, 4 and 8 before
    v = dpp_max<0x112, 0xf>(v);
    v = dpp_max<0x114, 0xf>(v);
    v = dpp_max<0x118, 0xf>(v);
    v = dpp_max<0x142, 0xa>(v);   // the last lane of a row to the next one
    v = dpp_max<0x143, 0xc>(v);   // of the lower half to the upper
    return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

// beta x + (1 - beta) y, rounded operation by operation.  The definition says so:
// (9 x + y) / 10 of short x and y often lies midway between two fp32 numbers,
// and a fused operation turned the scale of one block in a hundred there.
__device__ __attribute__((always_inline)) inline double moved(double beta, double x, double y) {
#pragma clang fp contract(off)
    return beta * x + (1.0 - beta) * y;
}

struct Scalars {
    float lr, inv_c1, rsqrt_c2, gscale;
    int64_t step;
};
__device__ __attribute__((always_inline)) inline Scalars scalars(const AdamArgs& a) {
    Scalars s = {a.lr, a.inv_c1, a.rsqrt_c2, 1.0f, a.step};
    if (a.grad_scale) s.gscale = *a.grad_scale;
    if (a.device_lr) s.lr *= *a.device_lr;
    if (a.device_step) {
        s.step += *a.device_step;
        s.inv_c1 = float(1.0 / (1.0 - adam_power(a.beta1, s.step)));
        s.rsqrt_c2 = float(1.0 / sqrt(1.0 - adam_power(a.beta2, s.step)));
    }
    return s;
}

__device__ __attribute__((always_inline)) inline float updated(float p, float m, float v, const Scalars& s, float eps,
                                                               float decay) {
    // the hardware's square root and reciprocal (1 ulp), subnormals scaled
    const bool tiny = v < 0x1p-96f;
    const float root = __builtin_amdgcn_sqrtf(tiny ? v * 0x1p64f : v) * (tiny ? s.rsqrt_c2 * 0x1p-32f : s.rsqrt_c2);
    const float d = root + eps;
    float u = m * s.inv_c1 * __builtin_amdgcn_rcpf(d);
    if (__builtin_expect(!(d > 0x1p-120f && d < 0x1p120f), 0)) u = m * s.inv_c1 / d;
    return p - s.lr * (decay * p + u);
}

// The N blocks of 256 elements of this wave from element i0 on (of the lane), the
// next kAdamWaves * 256 further: loads, then step by step.
template <int BITS, int N, bool FULL>
__device__ __attribute__((always_inline)) inline void adamw_blocks(const AdamArgs& a, const AdamItem& it, int64_t i0) {
    const int lane = threadIdx.x & 63;
    const bool p32 = it.p_type == CNHWC_F32, g32 = it.g_type == CNHWC_F32;
    auto at = [&](int u) __attribute__((always_inline)) -> int64_t { return i0 + u * (kAdamWaves * kAdamBlock); };
    auto left = [&](int u) __attribute__((always_inline)) -> int {
        if (FULL) return 4;
        const int64_t l = it.n - at(u);
        return l < 4 ? (l > 0 ? int(l) : 0) : 4;
    };
    i32x4 p[N], g[N], m[N], v[N];   // (8 bits: codes in word 0, the scale in word 1)
    if constexpr (BITS == 32) {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            m[u] = load4<FULL>(it.m, at(u), true, left(u));
            v[u] = load4<FULL>(it.v, at(u), true, left(u));
        }
    } else {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            m[u] = v[u] = i32x4{0, 0, 0, 0};
            m[u][0] = int(load_codes<FULL>(it.m, at(u), left(u)));
            v[u][0] = int(load_codes<FULL>(it.v, at(u), left(u)));
            if (FULL || left(u) > 0) {
                m[u][1] = __builtin_bit_cast(int, it.ms[at(u) / kAdamBlock]);
                v[u][1] = __builtin_bit_cast(int, it.vs[at(u) / kAdamBlock]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) g[u] = load4<FULL>(it.g, at(u), g32, left(u));
#pragma unroll
    for (int u = 0; u < N; ++u) p[u] = load4<FULL>(it.p, at(u), p32, left(u));
    const Scalars s = scalars(a);
    const float decay = it.decay;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        float pf[4], gf[4];
        unpack4(pf, p[u], it.p_type);
        unpack4(gf, g[u], it.g_type);
#pragma unroll
        for (int e = 0; e < 4; ++e) gf[e] *= s.gscale;
        if constexpr (BITS == 32) {
            const float b1 = float(a.beta1), b2 = float(a.beta2), a1 = float(1.0 - a.beta1), a2 = float(1.0 - a.beta2);
            float mf[4], vf[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mf[e] = b1 * elem<F32>(m[u], e) + a1 * gf[e];
                vf[e] = b2 * elem<F32>(v[u], e) + a2 * gf[e] * gf[e];
                pf[e] = updated(pf[e], mf[e], vf[e], s, a.eps, decay);
            }
            store4<FULL>(it.m, at(u), mf, CNHWC_F32, left(u));
            store4<FULL>(it.v, at(u), vf, CNHWC_F32, left(u));
        } else {
            const int mw = m[u][1], vw = v[u][1];
            const double ms = double(__builtin_bit_cast(float, mw)) * double(kUp<4>), vs = double(__builtin_bit_cast(float, vw)) * double(kUp<5>);
            double md[4], vd[4];
            float mf[4], vf[4];
            uint32_t mmax = 0, vmax = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const double gd = gf[e];
                md[e] = moved(a.beta1, double(m_bits(uint32_t(m[u][0]), e)) * ms, gd);
                vd[e] = moved(a.beta2, double(v_bits(uint32_t(v[u][0]), e)) * vs, gd * gd);
                mf[e] = float(md[e]);
                vf[e] = float(vd[e]);
                pf[e] = updated(pf[e], mf[e], vf[e], s, a.eps, decay);
                const uint32_t mb = __builtin_bit_cast(uint32_t, mf[e]) & 0x7fffffffu, vb = __builtin_bit_cast(uint32_t, vf[e]) & 0x7fffffffu;
                // (elements that are not there are 0: zero codes, gradients)
                mmax = mb > mmax ? mb : mmax;
                vmax = vb > vmax ? vb : vmax;
            }
            mmax = wave_max(mmax);
            vmax = wave_max(vmax);
            const Philox4 w = philox(uint64_t(at(u) >> 2) | uint64_t(uint32_t(it.tensor)) << 32, uint64_t(s.step), a.seed);
            const float nms = __builtin_bit_cast(float, mmax < 0x7f800000u ? mmax : 0x7fc00000u);
            const float nvs = __builtin_bit_cast(float, vmax < 0x7f800000u ? vmax : 0x7fc00000u);
            const Scale<4> sm(nms);
            const Scale<5> sv(nvs);
            uint32_t mcodes = 0, vcodes = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t cm = sm.encode(fabs(md[e]), fabsf(mf[e]), w.w[e] & 0xffffu);
                uint32_t cv = sv.encode(vd[e], vf[e], w.w[e] >> 16);
                if (vd[e] > 0.0 && cv == 0) cv = 1;
                mcodes |= (cm | (md[e] < 0.0 && cm ? 128u : 0u)) << (8 * e);
                vcodes |= cv << (8 * e);
            }
            if (mmax == 0 || mmax >= 0x7f800000u) mcodes = 0;
            if (vmax == 0 || vmax >= 0x7f800000u) vcodes = 0;
            store_codes<FULL>(it.m, at(u), mcodes, left(u));
            store_codes<FULL>(it.v, at(u), vcodes, left(u));
            if (lane == 0) {
                it.ms[at(u) / kAdamBlock] = nms;
                it.vs[at(u) / kAdamBlock] = nvs;
            }
        }
        store4<FULL>(it.p, at(u), pf, it.p_type, left(u));
        if (it.copy) store4<FULL>(it.copy, at(u), pf, it.copy_type, left(u));
    }
}

template <int BITS, int DEEP>   // 32 or 8; 1 or 2
__global__ __launch_bounds__(kAdamWaves * 64) void adamw_kernel(const AdamArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The last tensor that starts at or before this block: the lanes look at all of
    // them at once (the arguments are far away: one after the other, the six
    // readings of a search took longer than a small tensor's step).
    const uint32_t mine = lane < kAdamItems ? a.first[lane] : ~0u;
    const int k = __builtin_popcountll(__ballot(mine <= blockIdx.x)) - 1;
    const uint32_t first = uint32_t(__builtin_amdgcn_readlane(int(mine), k));
    const AdamItem& it = a.item[k];
    const int64_t w0 = int64_t(blockIdx.x - first) * adam_chunk(DEEP) + wave * kAdamBlock;   // the wave's first element
    constexpr int64_t kStride = kAdamWaves * kAdamBlock;
    if (w0 + (DEEP - 1) * kStride + kAdamBlock <= it.n) {
        adamw_blocks<BITS, DEEP, true>(a, it, w0 + lane * 4);
    } else {
#pragma unroll 1
        for (int64_t w = w0; w < it.n && w < w0 + DEEP * kStride; w += kStride) adamw_blocks<BITS, 1, false>(a, it, w + lane * 4);
    }
}

// Results leave with the streaming policy: whole lines, written once.
template <bool FULL>
__device__ __attribute__((always_inline)) inline void moments4(int64_t i, int left, uint32_t mc, uint32_t vc, float sm, float sv, float* mv,
                                                               float* vv) {
    float fm[4], fv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        fm[e] = m_bits(mc, e) * kUp<4> * sm;
        fv[e] = v_bits(vc, e) * kUp<5> * sv;
    }
    if constexpr (FULL) {
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
        __builtin_nontemporal_store(f32x4_any{fm[0], fm[1], fm[2], fm[3]}, reinterpret_cast<f32x4_any*>(mv + i));
        __builtin_nontemporal_store(f32x4_any{fv[0], fv[1], fv[2], fv[3]}, reinterpret_cast<f32x4_any*>(vv + i));
    } else {
        store4<false>(mv, i, fm, CNHWC_F32, left);
        store4<false>(vv, i, fv, CNHWC_F32, left);
    }
}
constexpr int kMomentsDeep = 4;
__global__ __launch_bounds__(256) void adamw_moments_kernel(int64_t n, const void* m, const void* v, const float* ms,
                                                            const float* vs, float* mv, float* vv) {
    const int64_t i0 = (int64_t(blockIdx.x) * (256 * kMomentsDeep) + threadIdx.x) * 4;
    if ((int64_t(blockIdx.x) + 1) * (256 * kMomentsDeep) * 4 <= n) {
        uint32_t mc[kMomentsDeep], vc[kMomentsDeep];
        float sm[kMomentsDeep], sv[kMomentsDeep];
#pragma unroll
        for (int u = 0; u < kMomentsDeep; ++u) {
            const int64_t i = i0 + u * 1024;
            mc[u] = load_codes<true>(m, i, 4);
            vc[u] = load_codes<true>(v, i, 4);
            sm[u] = ms[i / kAdamBlock];
            sv[u] = vs[i / kAdamBlock];
        }
#pragma unroll
        for (int u = 0; u < kMomentsDeep; ++u) moments4<true>(i0 + u * 1024, 4, mc[u], vc[u], sm[u], sv[u], mv, vv);
    } else {
        for (int64_t i = i0; i < n && i < i0 + kMomentsDeep * 1024; i += 1024) {
            const int left = n - i < 4 ? int(n - i) : 4;
            moments4<false>(i, left, load_codes<false>(m, i, left), load_codes<false>(v, i, left), ms[i / kAdamBlock], vs[i / kAdamBlock], mv,
                            vv);
        }
    }
}

}  // namespace

int launch_adamw(int bits, int deep, const AdamArgs& a, unsigned blocks, hipStream_t st) {
    if (bits == 32) {
        if (deep == 1) adamw_kernel<32, 1><<<blocks, kAdamWaves * 64, 0, st>>>(a);
        else adamw_kernel<32, 2><<<blocks, kAdamWaves * 64, 0, st>>>(a);
    } else {
        if (deep == 1) adamw_kernel<8, 1><<<blocks, kAdamWaves * 64, 0, st>>>(a);
        else adamw_kernel<8, 2><<<blocks, kAdamWaves * 64, 0, st>>>(a);
    }
    return CNHWC_OK;
}

int launch_adamw_moments(int64_t n, const void* m, const void* v, const float* ms, const float* vs, float* mv,
                         float* vv, hipStream_t st) {
    const int64_t blocks = (n + 256 * kMomentsDeep * 4 - 1) / (256 * kMomentsDeep * 4);   // (n < 2^35: at most 2^23)
    adamw_moments_kernel<<<unsigned(blocks), 256, 0, st>>>(n, m, v, ms, vs, mv, vv);
    return CNHWC_OK;
}

}  // namespace cnhwc
