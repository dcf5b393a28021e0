// Shared by the channel-mixing kernels (layer norm, gated feed-forward,
// dropout): the fp32 element tag, 16-byte row accesses at any element
// alignment, lane reductions, and the launchers' argument blocks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device.h"
#include "internal.h"

namespace cnhwc {

struct F32 {
    static constexpr bool is_bf16 = false;
};

// ---- argument blocks and launchers ------------------------------------------

struct LnArgs {
    const void* x;
    const void* dy;        // backward
    const void* gamma;     // NULL: 1
    const void* beta;      // NULL: 0
    void* y;               // forward: y; backward: dx (NULL: not computed)
    float* mean;           // written by the forward pass (may be NULL), read by the backward pass
    float* rstd;
    float* part;           // backward: [blocks][2][c] fp32 partial column sums (NULL: none)
    int64_t rows, x_stride, y_stride;
    int c;
    float eps, cf;         // cf: c as a float (sums are divided by it)
};

int launch_layernorm_fwd(int dtype, int param_dtype, const LnArgs& a, hipStream_t st);
// Blocks of the backward pass, i.e. partial rows of LnArgs::part.
int layernorm_bwd_blocks(int dtype, int64_t rows, int64_t c);
int launch_layernorm_bwd(int dtype, int param_dtype, const LnArgs& a, int blocks, hipStream_t st);
// dgamma / dbeta (either may be NULL) = sums over the partial rows, in order.
int launch_layernorm_reduce(int param_dtype, const float* part, int blocks, int64_t c, void* dgamma,
                            void* dbeta, hipStream_t st);

struct DropArgs {
    const void* x;
    const void* residual;           // NULL: 0
    void* y;
    const uint64_t* device_offset;  // NULL: none
    int64_t n;                      // rows * c
    int64_t x_stride, res_stride, y_stride;
    int64_t c;
    uint64_t seed, offset, threshold;   // keep where word >= threshold (up to 2^32)
    float scale;
    bool flat;                      // every stride equals c
};

int launch_dropout(int dtype, const DropArgs& a, hipStream_t st);

#ifdef __HIPCC__

// ---- rows in vectors of 16 bytes ----------------------------------------------

template <typename T>
constexpr int kVec = std::is_same<T, F32>::value ? 4 : 8;
template <typename T>
constexpr int kElemBytes = std::is_same<T, F32>::value ? 4 : 2;

// The global memory path takes 16-byte accesses at any element-aligned
// address, so rows of odd width are read and written as wide as aligned ones.
template <int A>
struct __attribute__((packed, aligned(A))) Words {
    uint32_t w[4];
};

template <typename T>
__device__ inline i32x4 load16(const void* p) {
    const Words<kElemBytes<T>> v = *static_cast<const Words<kElemBytes<T>>*>(p);
    return i32x4{int(v.w[0]), int(v.w[1]), int(v.w[2]), int(v.w[3])};
}
template <typename T>
__device__ inline void store16(void* p, i32x4 r) {
    Words<kElemBytes<T>> v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = uint32_t(r[i]);
    *static_cast<Words<kElemBytes<T>>*>(p) = v;
}

template <typename T>
__device__ inline float load1(const void* p) {
    if constexpr (std::is_same<T, F32>::value) return *static_cast<const float*>(p);
    else return to_f32<T>(*static_cast<const unsigned short*>(p));
}
template <typename T>
__device__ inline void store1(void* p, float v) {
    if constexpr (std::is_same<T, F32>::value) *static_cast<float*>(p) = v;
    else *static_cast<unsigned short*>(p) = pack1<T>(v);
}

// Element e of a 16-byte vector.
template <typename T>
__device__ inline float elem(const i32x4& r, int e) {
    if constexpr (std::is_same<T, F32>::value) {
        // by value: a bit cast of the subscript itself reads element 0
        const int v = r[e];
        return __builtin_bit_cast(float, v);
    }
    else return to_f32<T>((unsigned short)(uint32_t(r[e >> 1]) >> (16 * (e & 1))));
}
template <typename T>
__device__ inline i32x4 pack_vec(const float* f) {
    i32x4 r;
    if constexpr (std::is_same<T, F32>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = __builtin_bit_cast(int, f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = int(pack2<T>(f[2 * i], f[2 * i + 1]));
    }
    return r;
}

// The vector at p whose first n elements exist (n <= 0: none); the others read as 0.
template <typename T>
__device__ inline i32x4 load_n(const char* p, int n) {
    i32x4 r = {0, 0, 0, 0};
    if (n >= kVec<T>) {
        r = load16<T>(p);
    } else if (n > 0) {
#pragma unroll
        for (int e = 0; e < kVec<T> - 1; ++e) {
            if (e < n) {
                if constexpr (std::is_same<T, F32>::value)
                    r[e] = reinterpret_cast<const int*>(p)[e];
                else
                    r[e >> 1] |= int(uint32_t(reinterpret_cast<const unsigned short*>(p)[e]) << (16 * (e & 1)));
            }
        }
    }
    return r;
}
template <typename T>
__device__ inline void store_n(char* p, i32x4 r, int n) {
    if (n >= kVec<T>) {
        store16<T>(p, r);
    } else if (n > 0) {
#pragma unroll
        for (int e = 0; e < kVec<T> - 1; ++e) {
            if (e < n) {
                if constexpr (std::is_same<T, F32>::value)
                    reinterpret_cast<int*>(p)[e] = r[e];
                else
                    reinterpret_cast<unsigned short*>(p)[e] = (unsigned short)(uint32_t(r[e >> 1]) >> (16 * (e & 1)));
            }
        }
    }
}

// ---- sums over lanes ------------------------------------------------------------

template <int CTRL>
__device__ inline float dpp_add(float v) {
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true);
    return v + __builtin_bit_cast(float, o);
}

// Sum over each aligned group of L lanes (16 or 64), in every lane: row
// rotations by 8, 4, 2, 1 within 16 lanes, then exchanges over rows.
template <int L>
__device__ inline float lane_sum(float v) {
    static_assert(L == 16 || L == 64, "lanes");
    v = dpp_add<0x128>(v);
    v = dpp_add<0x124>(v);
    v = dpp_add<0x122>(v);
    v = dpp_add<0x121>(v);
    if constexpr (L == 64) {
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
    }
    return v;
}

#endif  // __HIPCC__

}  // namespace cnhwc
