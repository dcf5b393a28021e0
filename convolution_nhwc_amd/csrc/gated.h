// Internals of the gated feed-forward block (gated_gemm.hip, gated_rows.hip,
// mix_host.cpp).
#pragma once

#include "mix.h"

namespace cnhwc {

// The four products of the two passes on the tiled kernel:
//   PROJ  [g | u] = x [wg ; wu]^T       both operands k-contiguous, g and u of one
//                                       element in the same lane
//   DX    dx = [dg | du] [wg ; wu]      right operand rows are the reduction
//   DW    [dwg ; dwu] = [dg | du]^T x   both operands' rows are the reduction
enum GatedProduct { kProj = 0, kDx = 1, kDw = 2 };

// What a kernel does with its sums: round them (PROJ: y = act(g) u), form dg
// and du (PROJ), or store them as partial sums of a split reduction.
enum GatedEnd { kEndFwd = 0, kEndBwd = 1, kEndPart = 2 };

struct GatedArgs {
    // operands, rows of ld elements (a multiple of 8), 16-byte aligned
    const void* a;          // PROJ: x   DX, DW: dg | du [rows][2 fp]
    const void* b0;         // PROJ, DX: wg   DW: x
    const void* b1;         // PROJ, DX: wu   DW: unused
    int64_t lda, ldb;
    int64_t m;              // output rows: PROJ, DX: rows   DW: 2 fp
    int64_t n;              // output columns: PROJ: f (of g and of u)   DX, DW: c
    int64_t k;              // reduction length: PROJ: c   DX: fp (of each half)   DW: rows
    int64_t nb;             // DX, DW: columns of the right operand's rows (a multiple of 8, >= n)
    int segs;               // DX: 2 (dg with wg, du with wu), else 1
    int steps_seg;          // 64-deep steps of one segment
    int splits;             // reduction splits
    int act, end;           // PROJ
    int wide;               // results (and dy) move in whole aligned 16-byte vectors
    int64_t f, fp;          // hidden width, and rounded up to a multiple of 8
    // results
    void* y;                // PROJ forward: y   DX: dx
    int64_t ldy;
    const void* dy;         // PROJ backward
    int64_t lddy;
    void* dgu;              // PROJ backward: dg | du [rows][2 fp]
    void* dwg;              // DW [f][c]
    void* dwu;
    float* part;            // splits > 1: [splits][m][part_ld] fp32
    int64_t part_ld;        // PROJ: 2 fp   DX, DW: n rounded up to a multiple of 4
    int tiles_m, tiles_n;
};

// The tile shapes: 256 x 256 with one block of 8 waves a CU, 128 x 128 with
// two blocks of 4 waves a CU.
constexpr int kGatedBig = 256, kGatedSmall = 128;

int launch_gated_product(int dtype, GatedProduct prod, int tile, const GatedArgs& a, hipStream_t st);
// dx and the weights' gradients on small tiles in one launch, a block a tile
// (at most two blocks a CU, what its LDS takes), and the join of both where both
// are split.
int launch_gated_pair(int dtype, const GatedArgs& dx, const GatedArgs& dw, hipStream_t st);
int launch_gated_pair_reduce(int dtype, const GatedArgs& dx, const GatedArgs& dw, hipStream_t st);
// Folds the partial sums of a split product into its result.
int launch_gated_reduce(int dtype, GatedProduct prod, const GatedArgs& a, hipStream_t st);
// Copies of up to three operands, one launch: dst [rows][ldd] = src [rows][cols]
// (row stride ld), columns cols..ldd-1 zero.
struct GatedPack {
    const void* src;
    void* dst;
    int64_t ld, rows;
};
int launch_gated_pack(const GatedPack* p, int n, int64_t cols, int64_t ldd, hipStream_t st);
// dst[0..n) = 0 (16-bit elements)
int launch_gated_zero(void* dst, int64_t n, hipStream_t st);

// Few rows: the weights are streamed once, any strides and alignment.  With
// dgu: dg | du (row stride 2 fp, columns f..fp-1 zero) in the place of y.
constexpr int kGatedFewRows = 64;
struct GatedRowsArgs {
    const void* x;
    const void* wg;
    const void* wu;
    void* y;
    int64_t rows, c, f, ldx, ldy;
    int act;
    const void* dy;
    void* dgu;
    int64_t lddy, fp;
};
// (CNHWC_UNSUPPORTED: more than 16 rows of dg and du whose x does not stay in
// registers)
int launch_gated_rows(int dtype, const GatedRowsArgs& a, hipStream_t st);
// whether x stays in registers
bool gated_rows_kept(int64_t rows, int64_t c, bool bwd);

#ifdef __HIPCC__

// exp and the reciprocal below are the hardware's (1 ulp): their error is far
// under the rounding of the 16-bit result.
__device__ inline float sigmoid_f(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// max(g, 0), NaN where g is one: a single instruction (compared and selected,
// a lane's 64 spilled their masks).
__device__ inline float relu_f(float g) { return __builtin_elementwise_maximum(g, 0.0f); }

// The normal distribution function of -|g|, and times sqrt(2 pi) its density.
// Phi(-a) = exp(-a^2 / 2) t P(t) with t = 1 / (1 + 0.3 a), where erfcx's slow
// fall is nearly a polynomial in t.  P has six terms, fitted by linear
// programming to the least e with an error below e relative to Phi and below
// 0.03 e of 1, up to a = 13.5: 1.02e-5 of the value and 3.1e-7 (in fp32
// arithmetic 1.5e-5, where a^2 / 2 rounds, and 4.4e-7; half a step of an fp16
// result is 2.4e-4 of it at least).  The relative bound is what the results
// of negative g show: they are the tail itself.  Five terms reach 8.2e-5 and
// 2.5e-6, seven 2.1e-6 and 6e-8 for one instruction more; the library's erff
// takes about four times the instructions, and 64 of them a lane cost a third
// of a 384-channel tile.
//
// Returned as q and e = exp(-a^2 / 2), with Phi(-a) = e q.
__device__ inline float normal_tail(float g, float& e) {
    e = __builtin_amdgcn_exp2f(g * g * (-0.5f * 1.44269504088896341f));
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, __builtin_fabsf(g), 1.0f));
    float q = __builtin_fmaf(-0.07963219f, t, 0.22314219f);
    q = __builtin_fmaf(q, t, -0.02441341f);
    q = __builtin_fmaf(q, t, 0.1478436f);
    q = __builtin_fmaf(q, t, 0.11291612f);
    q = __builtin_fmaf(q, t, 0.12014362f);
    return q * t;
}
// a * b, and 0 where one of them is 0 whatever the other: gelu's products with
// its tail and density, which have fallen to 0 long before g is infinite (inf *
// 0 is NaN, where gelu's value and slope have limits).  v_mul_legacy_f32, which
// the compiler has as an intrinsic without a builtin's name.
__device__ float mul_0(float a, float b) __asm("llvm.amdgcn.fmul.legacy");

// act(g)
__device__ inline float act_value(int act, float g) {
    switch (act) {
    case CNHWC_ACT_SILU: return g * sigmoid_f(g);
    case CNHWC_ACT_GELU: {
        // g Phi(g) = max(g, 0) - |g| Phi(-|g|)
        float e;
        const float q = normal_tail(g, e);
        return __builtin_fmaf(-__builtin_fabsf(mul_0(g, e)), q, relu_f(g));
    }
    case CNHWC_ACT_RELU: return relu_f(g);
    default: return sigmoid_f(g);
    }
}

// act(g) and act'(g)
__device__ inline void act_both(int act, float g, float& v, float& d) {
    switch (act) {
    case CNHWC_ACT_SILU: {
        const float s = sigmoid_f(g);
        v = g * s;
        d = s * (1.0f + g * (1.0f - s));
        break;
    }
    case CNHWC_ACT_GELU: {
        float e;
        const float q = normal_tail(g, e) * e;
        const float c = g >= 0.0f ? 1.0f - q : q;
        v = mul_0(g, c);
        d = __builtin_fmaf(mul_0(g, e), 0.39894228040143268f, c);
        break;
    }
    case CNHWC_ACT_RELU:
        v = relu_f(g);
        d = g > 0.0f ? 1.0f : 0.0f;
        break;
    default: {
        // s (1 - s) by exp(-|g|): the difference loses its bits where s nears 1
        // (half a percent of the slope at g = 12, all of it past 17)
        const float e = __expf(-__builtin_fabsf(g)), r = __builtin_amdgcn_rcpf(1.0f + e);
        const float q = e * r;
        v = g >= 0.0f ? r : q;
        d = q * r;
    }
    }
}

#endif

}  // namespace cnhwc
