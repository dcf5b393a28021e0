// Internals of the group norm (groupnorm_fwd.hip, groupnorm_bwd.hip,
// groupnorm_host.cpp).
//
// A block takes a span of channels over a chunk of a sample's pixels.  A span
// is some whole groups, or, of a group that is wider than a block, one of its
// pieces; its channels lie over the threads in 16-byte vectors, and the threads
// that are left take further pixels.  Where a span is not whole vectors, the last one
// starts early and shares its first channels with the one before, which alone
// adds them up; both write them, with the same values.  (Cut short instead, it is
// loaded and stored element by element: 38 x 1377 pixels of 240 bf16 channels in 16
// groups backward 82 us, now 43; 15 x 408 of 736 in 32 groups 37 and 17.)  Where a sample's whole span fits the
// registers of one block (resident), one launch reads x once; otherwise chunks
// of pixels leave their sums in the workspace and a second launch reads x again.
#pragma once

#include "act.h"
#include "mix.h"

namespace cnhwc {

constexpr int kGnThreads = 512;   // most threads of a block of the two-launch kernels

// Vectors a thread of a resident kernel holds, and the most threads of its block:
// a wave has 128 registers in a block of 1024 threads and 256 in one of 512, and
// up to 50 (forward) or 83 hold other than x (and dy).  (Forward, 20 in half the threads
// would hold less than 12.)
// Spans that are narrower than a vector, or whose groups are, come in fewer variants.
constexpr int kGnFwd[] = {1, 2, 4, 8, 12, 32}, kGnBwd[] = {1, 2, 4, 8, 12, 16, 20};
constexpr bool gn_plain_only(int nv) { return nv != 4 && nv != 12; }
constexpr int gn_fwd_threads(int nv) { return nv <= 12 ? 1024 : 512; }
constexpr int kGnBwdThreads = 512;

// How the channels and pixels of a problem are dealt to blocks.
struct GnShape {
    int nv;          // resident: vectors (pixels) of a thread, one of kGnFwd or kGnBwd; 0: two launches
    int whole;       // every span is at least a vector wide
    int span;        // channels of a span (the last one may be narrower)
    int spans;       // spans of a sample
    int per;         // groups of a span (1 where groups are cut into pieces)
    int pieces;      // spans a group is cut into
    int vecs;        // 16-byte vectors of a span's row
    int ty;          // pixels that a block's threads take at a time
    int threads;
    int chunk;       // pixels of a block (the last chunk of a sample may be shorter)
    int chunks;
    FastDiv d_spans, d_vecs, d_chunks, d_each, d_pieces, d_ty;
};

struct GnArgs {
    const void* x;
    const void* dy;        // backward
    const void* gamma;     // NULL: 1
    const void* beta;      // NULL: 0
    void* y;               // forward: y; backward: dx (NULL: not computed)
    float* mean;           // [n][groups]
    float* rstd;
    float2* part;          // two launches, [n][chunks][groups * pieces]: forward mean and sum of squared deviations of
                           // a block's elements, backward sum(g) and sum(g xhat)
    float* cols;           // backward: [n * chunks][2][c] column sums of dz xhat and dz (NULL: not asked for)
    int64_t n, x_stride, y_stride;
    int pixels, c, groups, each;   // each: channels of a group
    int act, p32;                  // p32: gamma and beta are fp32
    float eps;
    GnShape s;
};

GnShape gn_shape(int dtype, int64_t n, int64_t pixels, int64_t c, int64_t groups, bool bwd);

int launch_groupnorm_fwd(int dtype, const GnArgs& a, hipStream_t st);
int launch_groupnorm_bwd(int dtype, const GnArgs& a, hipStream_t st);

#ifdef __HIPCC__

// exp2(x c), c = hi + lo: the product's rounding is made good, which the
// hardware's exponential would scale by x.  (Neither an infinite product, d inf or
// NaN, nor an infinite result, from t = 128 on, has anything to make good: inf
// times a negative d is -inf, and inf - inf NaN.)
__device__ __attribute__((always_inline)) inline float exp2_of(float x, float hi, float lo) {
    const float t = x * hi, e = __builtin_amdgcn_exp2f(t);
    const float d = __builtin_fmaf(x, lo, __builtin_fmaf(x, hi, -t));
    return t > -1e4f && t < 128.0f ? __builtin_fmaf(e, d * 0.69314718056f, e) : e;
}
constexpr float kLog2e = 1.44269504f, kLog2eLo = 1.92596299e-8f;   // their sum is log2(e) to 48 bits
__device__ __attribute__((always_inline)) inline float exp_of(float x) { return exp2_of(x, kLog2e, kLog2eLo); }

// Phi(-|g|) = e q as normal_tail has it, for fp32 results: eight terms of the same
// form (least e with an error of Phi below e of its value and 0.03 e of 1, by
// linear programming over |g| <= 13.5: 1.3e-7), and e = exp(-g^2 / 2) with the
// square's rounding made good.
__device__ __attribute__((always_inline)) inline float normal_tail_f32(float g, float& e) {
    const float h = g * g;
    e = exp2_of(h, -0.5f * kLog2e, -0.5f * kLog2eLo);
    if (h < 1e4f) e = __builtin_fmaf(e, -0.5f * __builtin_fmaf(g, g, -h), e);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, __builtin_fabsf(g), 1.0f));
    float q = __builtin_fmaf(0.03638098f, t, -0.16006877f);
    q = __builtin_fmaf(q, t, 0.21113554f);
    q = __builtin_fmaf(q, t, -0.05792161f);
    q = __builtin_fmaf(q, t, 0.13070858f);
    q = __builtin_fmaf(q, t, 0.09929341f);
    q = __builtin_fmaf(q, t, 0.12084834f);
    q = __builtin_fmaf(q, t, 0.11962346f);
    return q * t;
}

// act(z) and act'(z) as the element type needs them.  The 16-bit types take the
// hardware's exponential and gelu's six-term tail, whose errors vanish under
// their rounding; fp32 results the forms above (the library's functions took
// three times the instructions: 5 x 1189 pixels of 1517 channels with gelu
// backward 107 us, two thirds of it arithmetic).
template <typename T, int ACT>
__device__ __attribute__((always_inline)) inline float gn_act(float z) {
    if constexpr (ACT == CNHWC_ACT_NONE) {
        return z;
    } else if constexpr (!std::is_same<T, F32>::value) {
        return act_value(ACT, z);
    } else if constexpr (ACT == CNHWC_ACT_GELU) {
        float e;
        const float q = normal_tail_f32(z, e);
        return __builtin_fmaf(-__builtin_fabsf(mul_0(z, e)), q, relu_f(z));
    } else if constexpr (ACT == CNHWC_ACT_RELU) {
        return relu_f(z);
    } else {
        const float s = __builtin_amdgcn_rcpf(1.0f + exp_of(-z));
        return ACT == CNHWC_ACT_SILU ? z * s : s;
    }
}
template <typename T, int ACT>
__device__ __attribute__((always_inline)) inline float gn_slope(float z) {
    if constexpr (ACT == CNHWC_ACT_NONE) {
        return 1.0f;
    } else if constexpr (!std::is_same<T, F32>::value) {
        float v, d;
        act_both(ACT, z, v, d);
        return d;
    } else if constexpr (ACT == CNHWC_ACT_GELU) {
        float e;
        const float q = normal_tail_f32(z, e) * e;
        return __builtin_fmaf(mul_0(z, e), 0.39894228040143268f, z >= 0.0f ? 1.0f - q : q);
    } else if constexpr (ACT == CNHWC_ACT_RELU) {
        return z > 0.0f ? 1.0f : 0.0f;
    } else {
        const float e = exp_of(-__builtin_fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e);
        if constexpr (ACT == CNHWC_ACT_SIGMOID) return e * r * r;
        // s (1 + z (1 - s)), 1 - s without the difference
        const float s = z >= 0.0f ? r : e * r;
        return s * __builtin_fmaf(z, z >= 0.0f ? e * r : r, 1.0f);
    }
}

// A vector of results of the two-launch kernels leaves with the streaming policy:
// kept, the last lines would still be written back at the end of the kernel.  (The
// resident kernels' spans are cut out of lines that several blocks write, which
// meet in the L2: 16 x 3136 pixels of 384 fp16 channels with the policy 57 us,
// without 25.)
typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <typename T>
__device__ __attribute__((always_inline)) inline void gn_store(char* p, i32x4 r, int n) {
    if (n >= kVec<T>) __builtin_nontemporal_store(i32x4_any(r), reinterpret_cast<i32x4_any*>(p));
    else store_n<T>(p, r, n);
}

// The vectors of a thread's pixels, `have` of them from p on.  Whole ones are loaded
// without a branch, the last again in the place of those that are not there: a
// load behind a branch makes the compiler wait for all that are in flight, where
// the first ones could be worked on.
template <typename T, bool WHOLE, int NV>
__device__ __attribute__((always_inline)) inline void gn_load(i32x4 (&x)[NV], const char* p, int64_t step, int have, int left) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if constexpr (WHOLE) {
            x[i] = load16<T>(p);
            p += i + 1 < have ? step : 0;
        } else {
            x[i] = load_n<T>(p + i * step, i < have ? left : 0);
        }
    }
}
// The same for a few pixels at a time: which one the i-th load takes, of those left.
__device__ __attribute__((always_inline)) inline int gn_pixel(int i, int left) { return min(i, max(left, 1) - 1); }
template <typename T, bool WHOLE>
__device__ __attribute__((always_inline)) inline i32x4 gn_get(const char* p, int left) {
    if constexpr (WHOLE) return load16<T>(p);
    else return load_n<T>(p, left);
}
// A whole vector, or the only one of a span that is narrower.
template <typename T, bool WHOLE>
__device__ __attribute__((always_inline)) inline void gn_put(char* p, const i32x4& r, int left) {
    if constexpr (WHOLE) store16<T>(p, r);
    else store_n<T>(p, r, left);
}

// Keeps what is computed from the vectors so far from being kept in registers for
// the next pass over them: unpacked, they take twice the room.
template <int N>
__device__ __attribute__((always_inline)) inline void gn_forget(i32x4 (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(x[i]));
}

// f(IC<act>): the activation as a constant, chosen once a block
template <typename F>
__device__ __attribute__((always_inline)) inline void with_act(int act, F&& f) {
    switch (act) {
    case CNHWC_ACT_SILU: f(IC<CNHWC_ACT_SILU>{}); break;
    case CNHWC_ACT_GELU: f(IC<CNHWC_ACT_GELU>{}); break;
    case CNHWC_ACT_RELU: f(IC<CNHWC_ACT_RELU>{}); break;
    case CNHWC_ACT_SIGMOID: f(IC<CNHWC_ACT_SIGMOID>{}); break;
    default: f(IC<CNHWC_ACT_NONE>{});
    }
}

// Consecutive numbers for the blocks of an XCD (blocks go round the 8 in turn):
// the spans of a sample lie side by side in memory, and their lines meet in
// that XCD's L2.
__device__ inline int gn_block(int b, int blocks) {
    const int x = b & 7, base = blocks >> 3, rem = blocks & 7;
    return x * base + (x < rem ? x : rem) + (b >> 3);
}

// Where a block's and a thread's elements are.
template <typename T>
struct GnPlace {
    int span, piece, group0, groups;   // of the block: its span, piece of a group, first group, number of groups
    int c_lo, width, gw;               // first channel, channels, channels of a group (in the block)
    int p0, p1;                        // pixels
    int chunk;
    int64_t sample;
    // of the thread: vector, pixel; its first channel, also within the span; channels of the
    // vector that exist, and those of them that the vector before has too
    int tx, ty, c0, cs, left, dup;

    __device__ __attribute__((always_inline)) inline GnPlace(const GnArgs& a, int block, int tid) {
        const int rest = fdiv(block, a.s.d_chunks);
        chunk = block - rest * a.s.chunks;
        sample = fdiv(rest, a.s.d_spans);
        span = rest - int(sample) * a.s.spans;
        piece = 0;
        if (a.s.pieces > 1) {
            group0 = fdiv(span, a.s.d_pieces);
            piece = span - group0 * a.s.pieces;
            groups = 1;
            c_lo = group0 * a.each + piece * a.s.span;
            gw = width = min(a.s.span, a.each - piece * a.s.span);
        } else {
            group0 = span * a.s.per;
            groups = min(a.s.per, a.groups - group0);
            c_lo = group0 * a.each;
            gw = a.each;
            width = groups * a.each;
        }
        p0 = chunk * a.s.chunk;
        p1 = min(p0 + a.s.chunk, a.pixels);
        ty = fdiv(tid, a.s.d_vecs);
        tx = tid - ty * a.s.vecs;
        cs = start(tx, width);
        c0 = c_lo + cs;
        left = ty < a.s.ty && tx * kVec<T> < width ? min(kVec<T>, width - cs) : 0;
        dup = tx * kVec<T> - cs;
    }
    // the channel of the span that a vector starts at
    static __device__ __attribute__((always_inline)) inline int start(int vec, int width) { return max(0, min(vec * kVec<T>, width - kVec<T>)); }
    // the block's group that the thread's element e belongs to (elements that are not there: the last)
    __device__ __attribute__((always_inline)) inline int group_of(const GnArgs& a, int e) const {
        return a.s.pieces > 1 ? 0 : min(fdiv(cs + e, a.s.d_each), groups - 1);
    }
};

// Lanes that share one of `items` (a power of two, at most 64).
__device__ inline int gn_lanes(int threads, int items, int most) {
    int l = 1;
    while (l < 64 && l < most && 2 * l * items <= threads) l *= 2;
    return l;
}
template <typename V>
__device__ inline V gn_lane_sum(V v, int lanes) {
    for (int h = 1; h < lanes; h *= 2) v += __shfl_xor(v, h);
    return v;
}

// A per-channel vector's values at the thread's channels (def where there is none).
// Loads return in order: what the first pass needs is asked for before x is.
template <typename T>
struct GnParam {
    i32x4 raw[kVec<T> / 4];
    bool there;

    __device__ __attribute__((always_inline)) inline GnParam(const GnArgs& a, const void* p, const GnPlace<T>& w) : there(p != nullptr) {
#pragma unroll
        for (int h = 0; h < kVec<T> / 4; ++h) raw[h] = i32x4{0, 0, 0, 0};
        if (!p) return;
        if (a.p32) {
#pragma unroll
            for (int h = 0; h < kVec<T> / 4; ++h)
                raw[h] = load_n<F32>(static_cast<const char*>(p) + int64_t(w.c0 + 4 * h) * 4, w.left - 4 * h);
        } else if constexpr (!std::is_same<T, F32>::value) {
            raw[0] = load_n<T>(static_cast<const char*>(p) + int64_t(w.c0) * 2, w.left);
        }
    }
    __device__ __attribute__((always_inline)) inline void get(const GnArgs& a, float def, float (&v)[kVec<T>]) const {
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) {
            v[e] = elem<F32>(raw[e >> 2], e & 3);
            if constexpr (!std::is_same<T, F32>::value) v[e] = a.p32 ? v[e] : elem<T>(raw[0], e);
            v[e] = there ? v[e] : def;
        }
    }
};

// The groups that a thread's vector touches.  Groups of at least a vector touch it
// in two parts (SLOTS 2: the elements before `cut`, and from there on), narrower
// ones in any (a slot an element).
template <typename T, int SLOTS>
struct GnSlots {
    int first, second, cut;

    __device__ __attribute__((always_inline)) inline GnSlots(const GnArgs& a, const GnPlace<T>& w) {
        if constexpr (SLOTS == 2) {
            first = min(fdiv(w.cs, a.s.d_each), w.groups - 1);
            second = min(first + 1, w.groups - 1);
            cut = (first + 1) * a.each - w.cs;
        }
    }
    // per-channel values added up by slot, those of the vector before left out
    __device__ __attribute__((always_inline)) inline void sum(float (&s)[SLOTS], const float (&v)[kVec<T>], int dup) const {
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) s[k] = 0.0f;
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) {
            const float u = e >= dup ? v[e] : 0.0f;
            if constexpr (SLOTS == 2) {
                s[0] += e < cut ? u : 0.0f;
                s[1] += e < cut ? 0.0f : u;
            } else {
                s[e] = u;
            }
        }
    }
    // a value of each group at the thread's channels
    __device__ __attribute__((always_inline)) inline void spread(float (&v)[kVec<T>], const float* of, const GnArgs& a, const GnPlace<T>& w) const {
        if constexpr (SLOTS == 2) {
            const float lo = of[first], hi = of[second];
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) v[e] = e < cut ? lo : hi;
        } else {
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) v[e] = of[w.group_of(a, e)];
        }
    }
};

// out[group] = f(group, sum over the block of the group's slots); one lane calls f.
// arr: SLOTS * threads values of scratch.  Ends with a barrier.
template <typename T, int SLOTS, typename F>
__device__ __attribute__((always_inline)) inline void gn_group_sums(const GnArgs& a, const GnPlace<T>& w, const float (&s)[SLOTS], float* arr,
                                                                    float* out, F&& f) {
    constexpr int V = kVec<T>;
    const int threads = blockDim.x, ty = a.s.ty, vecs = a.s.vecs;
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) arr[k * threads + threadIdx.x] = s[k];
    __syncthreads();
    const int lanes = gn_lanes(threads, w.groups, 64);
    const int l = threadIdx.x & (lanes - 1);
    for (int g = threadIdx.x / lanes; g < w.groups; g += threads / lanes) {
        const int c0 = g * w.gw, c1 = c0 + w.gw;
        float t = 0.0f;
        if constexpr (SLOTS == 2) {
            // lanes over the group's vectors first, then over pixel rows
            const int v0 = c0 / V, n = (c1 + V - 1) / V - v0;
            int lv = 1;
            while (lv < n && lv < lanes) lv *= 2;
            const int ly = lanes / lv, y0 = l / lv;
            for (int v = l & (lv - 1); v < n; v += lv) {
                const float* p = arr + (GnPlace<T>::start(v0 + v, w.width) < c0 ? threads : 0) + v0 + v;
#pragma unroll 4
                for (int y = y0; y < ty; y += ly) t += p[y * vecs];
            }
        } else {
            for (int c = c0; c < c1; ++c) {
                const float* p = arr + (c - GnPlace<T>::start(c / V, w.width)) * threads + c / V;
#pragma unroll 4
                for (int y = l; y < ty; y += lanes) t += p[y * vecs];
            }
        }
        t = gn_lane_sum(t, lanes);
        if (l == 0) out[g] = f(g, t);
    }
    __syncthreads();
}

#endif

}  // namespace cnhwc
