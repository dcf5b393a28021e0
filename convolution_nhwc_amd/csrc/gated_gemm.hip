// The matrix products of the gated feed-forward block on MFMA.
//
// One kernel serves the three products of gated.h.  A block computes tiles of
// 2*HM rows by 2*HN columns (HM = HN = 128 with 8 waves, 64 with 4); each
// operand's 64-deep slice of the tile is two half tiles in LDS, and a wave
// owns the same quarter of every half, so its result is four quadrants
// (row half, column half).  In PROJ the column halves are the same hidden
// units of wg and of wu: g and u of an element meet in one lane's registers
// and the activation and product (or, backward, dg and du) follow without
// another pass over memory.
//
// A step of the reduction runs in two phases, one row half each:
//     phase   reads into registers                         multiplies row half
//       0     row half 0, column half 1                            0
//       1     row half 1, column half 0 of the next step           1
// so the two phases read the same amount, every half tile is read once, and
// its LDS is free one phase later, where the asynchronous loads of the step
// after next (row half 1: of the next) refill it.  With two stages a load has
// two phases to land; every phase's wait allows the eight younger loads.  The
// 8-wave block runs its two halves of waves (one wave of each on every SIMD)
// half a phase apart, with a barrier on each side of the multiplications:
// while one wave of a SIMD multiplies, the other reads and issues loads.  The
// 4-wave block needs one barrier a phase and overlaps with the second block of
// its CU instead.
//
// Blocks are persistent: the loads run on into a block's next tile while the
// current one is rounded and stored, so a tile's first operands are there when
// its turn comes, and its stores drain under the next tile's products.
//
// A half tile whose rows are contiguous in the reduction (x, wg, wu in PROJ;
// dg | du in DX) lies in LDS as rows of 64 elements, read with 16-byte reads;
// one whose rows are the reduction (wg, wu in DX; both operands of DW) as 64
// rows of HM or HN elements, read with the transposing read.  16- or 32-byte
// units are exchanged by an exclusive-or with row bits so that the lanes of a
// read spread over all banks (no conflicts counted); the exchange is done by
// the load's source address.
//
// Addresses: a tile's operands are buffer views on 64-bit bases, so neither
// tensor size nor row count is limited by 32-bit offsets; rows past an
// operand's end read as zero by the view's length, columns past the
// reduction's end by an out-of-range offset.
//
// Measured, bf16 normal operands: 16384 x 2048 -> 8192 forward 764 to 790 us by
// card, 1.39 to 1.44 PFLOP/s with the activation in it (the library's product of
// 8192^3 runs at 1.37 to 1.39); its backward pass of 8192 rows 1259 us, 1.31 (in
// a trace of ten passes projections 1.12, dx 1.44, weights 1.33, while the clock
// falls).  The forward and dx are bound by
// power: the matrix cores are busy 73 % of the cycles and the clock falls to
// 1.7-1.95 GHz under them (products alone, without a load, reach 2.0 PFLOP/s).
// With a short reduction the activation counts: 50176 x 384 -> 1024 fp16 gelu 97 to
// 105 us by card, 0.75 to 0.81 PFLOP/s, of a tile's 16 us 7 for its six steps and
// most of the others for 64 activations a lane and their stores, which no
// products hide.
#include "gated.h"

namespace cnhwc {
namespace {

constexpr int kBK = 64;   // reduction depth of a step

// ---- LDS reads and loads -----------------------------------------------------------
//
// What one phase moves: a row half into a (Q 16-row tiles by two 32-deep
// products, from offset OA) and a column half into b (two tiles, from offset
// OB), by the layouts of the two operands; then, while those reads run, the
// loads of two half tiles are issued.  Each function is one asm block that ends
// with its wait, so no register of it is live while a read is in flight; the
// loads write LDS only.  (Issued before the reads, the loads held them up: a
// CU takes one KiB in 16 cycles, four waves' loads of a phase in 260.)
//
// Rows contiguous in the reduction: p[0] / p[1] address the first and second
// product, tiles follow 2048 bytes apart in a and 512 in b (whose tiles
// interleave by 4 rows).  Rows that are the reduction (transposing reads, 4
// consecutive k a read): p[tile], HB bytes to k + 4, KB to the second product.

// This wave's two loads of a half tile: view, per-lane offsets, offset of the
// step.  They go to an LDS address `to` (of the stage) plus an immediate (of the
// half), the second one KiB on.
struct Load {
    i32x4 r;
    uint32_t v[2];
    uint32_t s;
};

#define CNHWC_RD(d, a, o) "ds_read_b128 %" #d ", %" #a " offset:%" #o "\n\t"
#define CNHWC_TR(d, a, o) "ds_read_b64_tr_b16 %" #d ", %" #a " offset:%" #o "\n\t"
#define CNHWC_LD(r, v0, v1, so, to, o)                                                       \
    "s_add_u32 m0, %" #to ", %" #o "\n\ts_nop 0\n\tbuffer_load_dwordx4 %" #v0 ", %" #r ", %" #so \
    " offen lds\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %" #v1          \
    ", %" #r ", %" #so " offen lds\n\t"

__device__ __attribute__((always_inline)) inline i32x4 join(i32x2 a, i32x2 b) { return i32x4{a[0], a[1], b[0], b[1]}; }

// b alone
template <int OB>
__device__ __attribute__((always_inline)) inline void read_rows(i32x4 (&b)[2][2], const uint32_t (&pb)[2]) {
    asm volatile(CNHWC_RD(0, 4, 6) CNHWC_RD(1, 5, 6) CNHWC_RD(2, 4, 7) CNHWC_RD(3, 5, 7) "s_waitcnt lgkmcnt(0)"
                 : "=&v"(b[0][0]), "=&v"(b[0][1]), "=&v"(b[1][0]), "=&v"(b[1][1])
                 : "v"(pb[0]), "v"(pb[1]), "i"(OB), "i"(OB + 512)
                 : "memory");
}
template <int OB, int HB, int KB>
__device__ __attribute__((always_inline)) inline void read_cols(i32x4 (&b)[2][2], const uint32_t (&pb)[2]) {
    i32x2 t[8];
    asm volatile(CNHWC_TR(0, 8, 10) CNHWC_TR(1, 8, 11) CNHWC_TR(2, 8, 12) CNHWC_TR(3, 8, 13) CNHWC_TR(4, 9, 10)
                     CNHWC_TR(5, 9, 11) CNHWC_TR(6, 9, 12) CNHWC_TR(7, 9, 13) "s_waitcnt lgkmcnt(0)"
                 : "=&v"(t[0]), "=&v"(t[1]), "=&v"(t[2]), "=&v"(t[3]), "=&v"(t[4]), "=&v"(t[5]), "=&v"(t[6]),
                   "=&v"(t[7])
                 : "v"(pb[0]), "v"(pb[1]), "i"(OB), "i"(OB + HB), "i"(OB + KB), "i"(OB + KB + HB)
                 : "memory");
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) b[j][k] = join(t[4 * j + 2 * k], t[4 * j + 2 * k + 1]);
}
// a and b, and the loads
template <int OA, int OB, int T0, int T1>
__device__ __attribute__((always_inline)) inline void read_rows_rows(i32x4 (&a)[4][2], i32x4 (&b)[2][2], const uint32_t (&pa)[2],
                                                                 const uint32_t (&pb)[2], const Load& d0, uint32_t to0, const Load& d1, uint32_t to1) {
    asm volatile(
        CNHWC_RD(0, 14, 30) CNHWC_RD(1, 15, 30) CNHWC_RD(2, 14, 31) CNHWC_RD(3, 15, 31) CNHWC_RD(4, 12, 26)
        CNHWC_RD(5, 13, 26) CNHWC_RD(6, 12, 27) CNHWC_RD(7, 13, 27) CNHWC_RD(8, 12, 28) CNHWC_RD(9, 13, 28)
        CNHWC_RD(10, 12, 29) CNHWC_RD(11, 13, 29) CNHWC_LD(16, 17, 18, 19, 20, 32) CNHWC_LD(21, 22, 23, 24, 25, 33)
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(b[0][0]), "=&v"(b[0][1]), "=&v"(b[1][0]), "=&v"(b[1][1]), "=&v"(a[0][0]), "=&v"(a[0][1]),
          "=&v"(a[1][0]), "=&v"(a[1][1]), "=&v"(a[2][0]), "=&v"(a[2][1]), "=&v"(a[3][0]), "=&v"(a[3][1])
        : "v"(pa[0]), "v"(pa[1]), "v"(pb[0]), "v"(pb[1]), "s"(d0.r), "v"(d0.v[0]), "v"(d0.v[1]), "s"(d0.s),
          "s"(to0), "s"(d1.r), "v"(d1.v[0]), "v"(d1.v[1]), "s"(d1.s), "s"(to1), "i"(OA), "i"(OA + 2048),
          "i"(OA + 4096), "i"(OA + 6144), "i"(OB), "i"(OB + 512),
          "i"(T0), "i"(T1)
        : "memory", "m0", "scc");
}
template <int OA, int OB, int T0, int T1, int HB, int KB>
__device__ __attribute__((always_inline)) inline void read_rows_cols(i32x4 (&a)[4][2], i32x4 (&b)[2][2], const uint32_t (&pa)[2],
                                                                 const uint32_t (&pb)[2], const Load& d0, uint32_t to0, const Load& d1, uint32_t to1) {
    i32x2 t[8];
    asm volatile(
        CNHWC_TR(0, 18, 34) CNHWC_TR(1, 18, 35) CNHWC_TR(2, 18, 36) CNHWC_TR(3, 18, 37) CNHWC_TR(4, 19, 34)
        CNHWC_TR(5, 19, 35) CNHWC_TR(6, 19, 36) CNHWC_TR(7, 19, 37) CNHWC_RD(8, 16, 30) CNHWC_RD(9, 17, 30)
        CNHWC_RD(10, 16, 31) CNHWC_RD(11, 17, 31) CNHWC_RD(12, 16, 32) CNHWC_RD(13, 17, 32)
        CNHWC_RD(14, 16, 33) CNHWC_RD(15, 17, 33) CNHWC_LD(20, 21, 22, 23, 24, 38) CNHWC_LD(25, 26, 27, 28, 29, 39)
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(t[0]), "=&v"(t[1]), "=&v"(t[2]), "=&v"(t[3]), "=&v"(t[4]), "=&v"(t[5]), "=&v"(t[6]), "=&v"(t[7]),
          "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[1][0]), "=&v"(a[1][1]), "=&v"(a[2][0]), "=&v"(a[2][1]),
          "=&v"(a[3][0]), "=&v"(a[3][1])
        : "v"(pa[0]), "v"(pa[1]), "v"(pb[0]), "v"(pb[1]), "s"(d0.r), "v"(d0.v[0]), "v"(d0.v[1]), "s"(d0.s),
          "s"(to0), "s"(d1.r), "v"(d1.v[0]), "v"(d1.v[1]), "s"(d1.s), "s"(to1), "i"(OA), "i"(OA + 2048),
          "i"(OA + 4096), "i"(OA + 6144), "i"(OB), "i"(OB + HB), "i"(OB + KB), "i"(OB + KB + HB),
          "i"(T0), "i"(T1)
        : "memory", "m0", "scc");
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) b[j][k] = join(t[4 * j + 2 * k], t[4 * j + 2 * k + 1]);
}
template <int OA, int OB, int T0, int T1, int HB, int KB>
__device__ __attribute__((always_inline)) inline void read_cols_cols(i32x4 (&a)[4][2], i32x4 (&b)[2][2], const uint32_t (&pa)[4],
                                                                 const uint32_t (&pb)[2], const Load& d0, uint32_t to0, const Load& d1, uint32_t to1) {
    i32x2 t[24];
    asm volatile(
        CNHWC_TR(0, 28, 44) CNHWC_TR(1, 28, 45) CNHWC_TR(2, 28, 46) CNHWC_TR(3, 28, 47) CNHWC_TR(4, 29, 44)
        CNHWC_TR(5, 29, 45) CNHWC_TR(6, 29, 46) CNHWC_TR(7, 29, 47) CNHWC_TR(8, 24, 40) CNHWC_TR(9, 24, 41)
        CNHWC_TR(10, 24, 42) CNHWC_TR(11, 24, 43) CNHWC_TR(12, 25, 40) CNHWC_TR(13, 25, 41)
        CNHWC_TR(14, 25, 42) CNHWC_TR(15, 25, 43) CNHWC_TR(16, 26, 40) CNHWC_TR(17, 26, 41)
        CNHWC_TR(18, 26, 42) CNHWC_TR(19, 26, 43) CNHWC_TR(20, 27, 40) CNHWC_TR(21, 27, 41)
        CNHWC_TR(22, 27, 42) CNHWC_TR(23, 27, 43) CNHWC_LD(30, 31, 32, 33, 34, 48) CNHWC_LD(35, 36, 37, 38, 39, 49)
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(t[0]), "=&v"(t[1]), "=&v"(t[2]), "=&v"(t[3]), "=&v"(t[4]), "=&v"(t[5]), "=&v"(t[6]), "=&v"(t[7]),
          "=&v"(t[8]), "=&v"(t[9]), "=&v"(t[10]), "=&v"(t[11]), "=&v"(t[12]), "=&v"(t[13]), "=&v"(t[14]),
          "=&v"(t[15]), "=&v"(t[16]), "=&v"(t[17]), "=&v"(t[18]), "=&v"(t[19]), "=&v"(t[20]), "=&v"(t[21]),
          "=&v"(t[22]), "=&v"(t[23])
        : "v"(pa[0]), "v"(pa[1]), "v"(pa[2]), "v"(pa[3]), "v"(pb[0]), "v"(pb[1]), "s"(d0.r), "v"(d0.v[0]),
          "v"(d0.v[1]), "s"(d0.s), "s"(to0), "s"(d1.r), "v"(d1.v[0]), "v"(d1.v[1]), "s"(d1.s), "s"(to1),
          "i"(OA), "i"(OA + HB), "i"(OA + KB), "i"(OA + KB + HB), "i"(OB), "i"(OB + HB), "i"(OB + KB), "i"(OB + KB
          + HB),
          "i"(T0), "i"(T1)
        : "memory", "m0", "scc");
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) b[j][k] = join(t[4 * j + 2 * k], t[4 * j + 2 * k + 1]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) a[i][k] = join(t[8 + 4 * i + 2 * k], t[9 + 4 * i + 2 * k]);
}
template <int OA, int OB, int T0, int T1>
__device__ __attribute__((always_inline)) inline void read_rows_rows(i32x4 (&a)[2][2], i32x4 (&b)[2][2], const uint32_t (&pa)[2],
                                                                 const uint32_t (&pb)[2], const Load& d0, uint32_t to0, const Load& d1, uint32_t to1) {
    asm volatile(
        CNHWC_RD(0, 10, 24) CNHWC_RD(1, 11, 24) CNHWC_RD(2, 10, 25) CNHWC_RD(3, 11, 25) CNHWC_RD(4, 8, 22)
        CNHWC_RD(5, 9, 22) CNHWC_RD(6, 8, 23) CNHWC_RD(7, 9, 23) CNHWC_LD(12, 13, 14, 15, 16, 26)
        CNHWC_LD(17, 18, 19, 20, 21, 27) "s_waitcnt lgkmcnt(0)"
        : "=&v"(b[0][0]), "=&v"(b[0][1]), "=&v"(b[1][0]), "=&v"(b[1][1]), "=&v"(a[0][0]), "=&v"(a[0][1]),
          "=&v"(a[1][0]), "=&v"(a[1][1])
        : "v"(pa[0]), "v"(pa[1]), "v"(pb[0]), "v"(pb[1]), "s"(d0.r), "v"(d0.v[0]), "v"(d0.v[1]), "s"(d0.s),
          "s"(to0), "s"(d1.r), "v"(d1.v[0]), "v"(d1.v[1]), "s"(d1.s), "s"(to1), "i"(OA), "i"(OA + 2048),
          "i"(OB), "i"(OB + 512),
          "i"(T0), "i"(T1)
        : "memory", "m0", "scc");
}
template <int OA, int OB, int T0, int T1, int HB, int KB>
__device__ __attribute__((always_inline)) inline void read_rows_cols(i32x4 (&a)[2][2], i32x4 (&b)[2][2], const uint32_t (&pa)[2],
                                                                 const uint32_t (&pb)[2], const Load& d0, uint32_t to0, const Load& d1, uint32_t to1) {
    i32x2 t[8];
    asm volatile(
        CNHWC_TR(0, 14, 28) CNHWC_TR(1, 14, 29) CNHWC_TR(2, 14, 30) CNHWC_TR(3, 14, 31) CNHWC_TR(4, 15, 28)
        CNHWC_TR(5, 15, 29) CNHWC_TR(6, 15, 30) CNHWC_TR(7, 15, 31) CNHWC_RD(8, 12, 26) CNHWC_RD(9, 13, 26)
        CNHWC_RD(10, 12, 27) CNHWC_RD(11, 13, 27) CNHWC_LD(16, 17, 18, 19, 20, 32) CNHWC_LD(21, 22, 23, 24, 25, 33)
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(t[0]), "=&v"(t[1]), "=&v"(t[2]), "=&v"(t[3]), "=&v"(t[4]), "=&v"(t[5]), "=&v"(t[6]), "=&v"(t[7]),
          "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[1][0]), "=&v"(a[1][1])
        : "v"(pa[0]), "v"(pa[1]), "v"(pb[0]), "v"(pb[1]), "s"(d0.r), "v"(d0.v[0]), "v"(d0.v[1]), "s"(d0.s),
          "s"(to0), "s"(d1.r), "v"(d1.v[0]), "v"(d1.v[1]), "s"(d1.s), "s"(to1), "i"(OA), "i"(OA + 2048),
          "i"(OB), "i"(OB + HB), "i"(OB + KB), "i"(OB + KB + HB),
          "i"(T0), "i"(T1)
        : "memory", "m0", "scc");
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) b[j][k] = join(t[4 * j + 2 * k], t[4 * j + 2 * k + 1]);
}
template <int OA, int OB, int T0, int T1, int HB, int KB>
__device__ __attribute__((always_inline)) inline void read_cols_cols(i32x4 (&a)[2][2], i32x4 (&b)[2][2], const uint32_t (&pa)[2],
                                                                 const uint32_t (&pb)[2], const Load& d0, uint32_t to0, const Load& d1, uint32_t to1) {
    i32x2 t[16];
    asm volatile(
        CNHWC_TR(0, 18, 34) CNHWC_TR(1, 18, 35) CNHWC_TR(2, 18, 36) CNHWC_TR(3, 18, 37) CNHWC_TR(4, 19, 34)
        CNHWC_TR(5, 19, 35) CNHWC_TR(6, 19, 36) CNHWC_TR(7, 19, 37) CNHWC_TR(8, 16, 30) CNHWC_TR(9, 16, 31)
        CNHWC_TR(10, 16, 32) CNHWC_TR(11, 16, 33) CNHWC_TR(12, 17, 30) CNHWC_TR(13, 17, 31)
        CNHWC_TR(14, 17, 32) CNHWC_TR(15, 17, 33) CNHWC_LD(20, 21, 22, 23, 24, 38) CNHWC_LD(25, 26, 27, 28, 29, 39)
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(t[0]), "=&v"(t[1]), "=&v"(t[2]), "=&v"(t[3]), "=&v"(t[4]), "=&v"(t[5]), "=&v"(t[6]), "=&v"(t[7]),
          "=&v"(t[8]), "=&v"(t[9]), "=&v"(t[10]), "=&v"(t[11]), "=&v"(t[12]), "=&v"(t[13]), "=&v"(t[14]),
          "=&v"(t[15])
        : "v"(pa[0]), "v"(pa[1]), "v"(pb[0]), "v"(pb[1]), "s"(d0.r), "v"(d0.v[0]), "v"(d0.v[1]), "s"(d0.s),
          "s"(to0), "s"(d1.r), "v"(d1.v[0]), "v"(d1.v[1]), "s"(d1.s), "s"(to1), "i"(OA), "i"(OA + HB), "i"(OA
          + KB), "i"(OA + KB + HB), "i"(OB), "i"(OB + HB), "i"(OB + KB), "i"(OB + KB + HB),
          "i"(T0), "i"(T1)
        : "memory", "m0", "scc");
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) b[j][k] = join(t[4 * j + 2 * k], t[4 * j + 2 * k + 1]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) a[i][k] = join(t[8 + 4 * i + 2 * k], t[9 + 4 * i + 2 * k]);
}
#undef CNHWC_RD
#undef CNHWC_TR
#undef CNHWC_LD

// ---- one operand of the tile --------------------------------------------------------

// Where this lane's loads of its wave's two 1 KiB regions of a half tile come
// from.  ROWS: the operand's rows are contiguous in the reduction.  PERM: its
// rows are read in the order that gives a lane 8 consecutive ones over two
// 16-row tiles (the result's columns).  HALF: rows (ROWS) or columns of a half.
template <bool ROWS, bool PERM, int HALF>
struct Operand {
    uint32_t voff[2];   // byte offset in the first half; the second is `half` on
    uint32_t half;
    int lane_k[2];      // ROWS: its k within a step

    __device__ __attribute__((always_inline)) Operand(int wave, int lane, int64_t ld) {
        half = uint32_t(ROWS ? HALF * ld * 2 : HALF * 2);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int region = wave * 2 + q;
            if constexpr (ROWS) {
                const int row = region * 8 + (lane >> 3);
                const int unit = (lane & 7) ^ (PERM ? ((row & 3) | ((row >> 1) & 4)) : (row & 7));
                voff[q] = uint32_t(row * ld * 2 + unit * 16);
                lane_k[q] = unit * 8;
            } else {
                constexpr int U = HALF / 8;   // 16-byte units of a row
                const int k = region * (64 / U) + lane / U, pos = lane % U;
                voff[q] = uint32_t(k * ld * 2 + ((((pos >> 1) ^ swz(k)) << 5) | ((pos & 1) << 4)));
                lane_k[q] = 0;
            }
        }
    }
    // which 32-byte unit of a row of HALF elements moves where
    __device__ static int swz(int k) {
        if constexpr (HALF == 128) return (k & 3) | ((k >> 1) & 4);
        else return ((k >> 1) & 1) | ((k >> 2) & 2);
    }
};

// A kernel's ARG-th argument block read again from where it was passed: what
// only a tile's start and end need is not held in scalar registers over its
// steps (nor anything computed from it before the loop).
typedef const __attribute__((address_space(4))) GatedArgs ArgsMem;
template <int ARG>
__device__ __attribute__((always_inline)) inline ArgsMem& args_again() {
    auto p = (ArgsMem*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p[ARG];
}

struct Tile {
    int64_t m0, n0;
    int split, s_lo, steps;
};

// The v-th tile of the launch: consecutive tiles on one XCD (blocks go round
// the 8 XCDs in turn), in groups of 8 tile rows so that the tiles at work on
// an XCD share operands in its L2.
template <int TILE, int NT, int ARG>
__device__ __attribute__((always_inline)) inline Tile tile_of(int v) {
    ArgsMem& a = args_again<ARG>();
    const int tiles = a.tiles_m * a.tiles_n, total = tiles * a.splits;
    const int x = v & 7, base = total >> 3, rem = total & 7;
    const int id = x * base + (x < rem ? x : rem) + (v >> 3);
    Tile t;
    t.split = id / tiles;
    const int r0 = id - t.split * tiles;
    const int per = 8 * a.tiles_n, grp = r0 / per, r = r0 - grp * per;
    const int rows = a.tiles_m - grp * 8 < 8 ? a.tiles_m - grp * 8 : 8;
    const int tn = r / rows, tm = grp * 8 + (r - tn * rows);
    t.m0 = int64_t(tm) * TILE;
    t.n0 = int64_t(tn) * NT;
    const int all = a.segs * a.steps_seg;
    // (at most 2^25 steps and 64 splits)
    t.s_lo = int(uint32_t(all) * uint32_t(t.split) / uint32_t(a.splits));
    t.steps = int(uint32_t(all) * uint32_t(t.split + 1) / uint32_t(a.splits)) - t.s_lo;
    return t;
}

// A value that is the same in every lane, which the compiler does not always see.
__device__ __attribute__((always_inline)) inline uint32_t uniform(uint32_t v) {
    return uint32_t(__builtin_amdgcn_readfirstlane(int(v)));
}
// A view's words for the loads written in asm.
__device__ __attribute__((always_inline)) inline i32x4 words_of(const char* p, uint32_t n) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    return i32x4{int(uniform(uint32_t(u))), int(uniform(uint32_t(u >> 32) & 0xffffu)), int(uniform(n)), int(kRsrcWord3)};
}

__device__ __attribute__((always_inline)) inline __amdgpu_buffer_rsrc_t view(const char* p, int64_t n) {
    return make_rsrc(p, n > 0 ? (n < 0x7fffffff ? uint32_t(n) : 0x7fffffffu) : 0u);
}

// dg and du stay in the caches: the next two products read them.  (The other
// results leave with the streaming policy: kept, they crowd the operands out of
// the L2; 16384 x 2048 -> 8192 forward 783 us instead of 764 on one card, 50176 x
// 384 -> 1024 gelu 113 instead of 109.)
//
// They are rounded to the operands' 16 bits, as the matrix instructions take
// them: the gradients' relative error is 2.35e-3 in bf16 and 2.9e-4 in fp16,
// where dg and du in fp32 leave the rounding of the result alone, 1.66e-3 and
// 2.1e-4.  As two 16-bit terms each they would double both products, 60 % of the
// backward pass.  The bits of a call are the same every time.
__device__ __attribute__((always_inline)) inline void store16_at(i32x4 v, __amdgpu_buffer_rsrc_t r, uint32_t off) {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 0);
}

constexpr int kTileThreads(int tile) { return tile == kGatedBig ? 512 : 256; }
constexpr int kTileLds(int tile) { return 8 * (tile / 2) * 128; }

// Tiles first, first + stride, ... of one product.  END: what follows the
// products (a GatedEnd); ACT only where PROD is kProj; ARG: which argument block
// of the kernel.
template <typename T, int PROD, int TILE, int END, int ACT, int ARG>
__device__ __attribute__((always_inline)) inline void gated_product(const GatedArgs& a, unsigned char* lds,
                                                                    const int first, const int stride) {
    constexpr bool AROWS = PROD != kDw, BROWS = PROD == kProj;
    constexpr int WN = TILE / 64;                     // waves: 2 over rows, WN over columns
    constexpr int HALF = TILE / 2;                    // rows / columns of a half tile
    constexpr int NT = PROD == kProj ? HALF : TILE;   // result columns of a tile
    constexpr int QM = HALF / 32;                     // 16-row tiles of a quadrant; 2 tiles of columns
    constexpr bool PP = TILE == kGatedBig;            // two wave groups half a phase apart
    constexpr int HBYTES = HALF * 128;                // a half tile in LDS
    constexpr int BBASE = 4 * HBYTES;                 // A: [half][stage], then B
    // stores of a tile's results per wave, all of them issued whatever the
    // tile's edges (the offsets past them are out of range): the waits of the
    // next tile's first step count over them
    constexpr int STORES = END == kEndPart ? 0 : PROD == kProj ? 2 * QM * (END == kEndBwd ? 2 : 1) : 4 * QM;
    static_assert(8 * HBYTES == kTileLds(TILE), "half tiles");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int total = a.tiles_m * a.tiles_n * a.splits;

    // ---- load cursor ----
    // Row operands: a view of the tile's rows, the reduction by the loads'
    // scalar offset.  Reduction operands: a view of a step's 64 rows that moves
    // on with the cursor, shorter at the end of the operand.
    const Operand<AROWS, false, HALF> A(wave, lane, a.lda);
    const Operand<BROWS, PROD == kProj, HALF> B(wave, lane, a.ldb);
    const char *pa_src = nullptr, *pb_src = nullptr, *pu_src = nullptr;   // view bases (pu_src: PROJ, wu)
    uint32_t na = 0, nb = 0;       // their lengths
    uint32_t na_end = 0, nb_end = 0;   // lengths in a segment's last step (reduction operands)
    uint32_t so = 0;               // bytes into the rows (row operands)
    uint32_t so_step = kBK * 2;    // 0 once no tile is left: an offset past an empty view would pass its check
    const int k_end = int(a.k - int64_t(a.steps_seg - 1) * kBK);   // depth of a segment's last step
    int cv = first;                // tile
    int seg = 0, sk = 0;           // segment and step within it
    int todo = 0;                  // steps left of the tile; 0: no tile left, the views are empty
    // the cursor onto the first step of tile cv.  (One closure whose two ways
    // end in the same assignments: stores to different variables at the ends
    // of two branches are merged into one through a pointer, and with it the
    // cursor leaves the registers.)
    auto aim = [&]() __attribute__((always_inline)) {
        int t_todo = 0x7fffffff, t_sk = 0, t_seg = 0;
        uint32_t t_so = 0, t_step = 0, t_na = 0, t_nb = 0, t_na_end = 0, t_nb_end = 0;
        const char *t_pa = nullptr, *t_pb = nullptr, *t_pu = nullptr;
        if (cv < total) {
            ArgsMem& a = args_again<ARG>();
            const Tile t = tile_of<TILE, NT, ARG>(cv);
            t_todo = t.steps;
            t_sk = t.s_lo;
            if (PROD == kDx && t_sk >= a.steps_seg) {
                t_seg = 1;
                t_sk -= a.steps_seg;
            }
            const int64_t kk = int64_t(t_sk) * kBK;
            const int64_t ktail = (PROD == kDx ? a.f : a.k) - int64_t(a.steps_seg - 1) * kBK;   // rows of the last step
            t_so = uint32_t(kk * 2);
            t_step = kBK * 2;
            const char* ap = static_cast<const char*>(a.a);
            if constexpr (AROWS) {
                const int64_t rows = a.m - t.m0 < TILE ? a.m - t.m0 : TILE;
                t_pa = ap + (t.m0 * a.lda + (PROD == kDx ? t_seg * a.fp : 0)) * 2;
                // (in DX the last row of dg ends where its du begins: the mask
                // of the reduction's end keeps every lane inside)
                t_na = uint32_t(((rows - 1) * a.lda + a.k) * 2);
            } else {
                t_pa = ap + (kk * a.lda + t.m0) * 2;
                t_na = uint32_t(kBK * a.lda * 2);
                t_na_end = uint32_t((ktail * a.lda - t.m0) * 2);
            }
            if constexpr (BROWS) {
                const int64_t rows = a.n - t.n0 < HALF ? a.n - t.n0 : HALF;
                t_pb = static_cast<const char*>(a.b0) + t.n0 * a.ldb * 2;
                t_pu = static_cast<const char*>(a.b1) + t.n0 * a.ldb * 2;
                t_nb = uint32_t(((rows - 1) * a.ldb + a.k) * 2);
            } else {
                t_pb = static_cast<const char*>(PROD == kDx && t_seg ? a.b1 : a.b0) + (kk * a.ldb + t.n0) * 2;
                t_nb = uint32_t(kBK * a.ldb * 2);
                t_nb_end = uint32_t(((ktail - 1) * a.ldb + a.nb - t.n0) * 2);
            }
        }
        todo = t_todo;
        sk = t_sk;
        seg = t_seg;
        so = t_so;
        so_step = t_step;
        na = t_na;
        nb = t_nb;
        na_end = t_na_end;
        nb_end = t_nb_end;
        pa_src = t_pa;
        pb_src = t_pb;
        pu_src = t_pu;
    };
    Load la0, la1, lb0, lb1;       // of the cursor's step; la1: of the step before
    // one of the cursor's loads from its state
    using LA0 = IC<0>;
    using LA1 = IC<1>;
    using LB0 = IC<2>;
    using LB1 = IC<3>;
    auto set = [&](auto wc) __attribute__((always_inline)) {
        constexpr int W = decltype(wc)::value, h = W & 1;
        const bool last = sk == a.steps_seg - 1;
        const int kl = last ? k_end : kBK;
        Load l;
        if constexpr (W < 2) {
            uint32_t len = na;
            if constexpr (!AROWS) len = last ? na_end + 0u : na + 0u;   // (values, not a choice of variables)
            l.r = words_of(pa_src, len);
            l.s = AROWS ? uniform(so) : 0u;
#pragma unroll
            for (int q = 0; q < 2; ++q) l.v[q] = !AROWS || A.lane_k[q] < kl ? A.voff[q] + h * A.half : kOob;
        } else {
            const char* src = pb_src;
            if constexpr (BROWS && h == 1) src = pu_src;
            uint32_t len = nb;
            if constexpr (!BROWS) len = last ? nb_end + 0u : nb + 0u;
            l.r = words_of(src, len);
            l.s = BROWS ? uniform(so) : 0u;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                l.v[q] = !BROWS || B.lane_k[q] < kl ? B.voff[q] + (BROWS ? 0 : h * B.half) : kOob;
        }
        if constexpr (W == 0) la0 = l;
        else if constexpr (W == 1) la1 = l;
        else if constexpr (W == 2) lb0 = l;
        else lb1 = l;
    };
    // past the end of a tile or of a segment
    auto turn = [&]() __attribute__((always_inline)) {
        if (todo == 0) {
            cv += stride;
            aim();
        } else if (PROD == kDx && seg == 0 && sk == a.steps_seg) {
            ArgsMem& a = args_again<ARG>();
            seg = 1;   // on to du and wu
            sk = 0;
            so = 0;
            pa_src += a.fp * 2;
            pb_src = static_cast<const char*>(a.b1) +
                        (pb_src - static_cast<const char*>(a.b0) - int64_t(a.steps_seg) * kBK * a.ldb * 2);
        }
    };
    // The cursor moves on by `run` steps at a time: between, the loads differ
    // from step to step by an offset alone (hop), a few scalar instructions
    // between the products.  Everything else -- another tile or segment, the
    // mask or the view of a segment's last step, the step after either, where
    // la1 follows -- is worked out from the cursor (move).  Worked out every
    // step, it cost 0.13 us of a step of 1.15.
    const bool tail = !AROWS || !BROWS || k_end != kBK;   // a segment's last step is special
    int run = 1, until = 1;
    auto hop = [&]() __attribute__((always_inline)) {
        if constexpr (AROWS) {
            la1.s = la0.s;
            la0.s += so_step;
        } else {
            la1.r[0] = la0.r[0];
            la1.r[1] = la0.r[1];
            const uint64_t q = (uint64_t(uint32_t(la0.r[0])) | uint64_t(uint32_t(la0.r[1])) << 32) + kBK * a.lda * 2;
            la0.r[0] = int(uint32_t(q));
            la0.r[1] = int(uint32_t(q >> 32));
        }
        if constexpr (BROWS) {
            lb0.s = lb1.s = la0.s;
        } else {
            const uint64_t q = (uint64_t(uint32_t(lb0.r[0])) | uint64_t(uint32_t(lb0.r[1])) << 32) + kBK * a.ldb * 2;
            lb0.r[0] = lb1.r[0] = int(uint32_t(q));
            lb0.r[1] = lb1.r[1] = int(uint32_t(q >> 32));
        }
        --until;
    };
    auto set_all = [&]() __attribute__((always_inline)) {
        set(LA0{});
        set(LB0{});
        set(LB1{});
    };
    auto move = [&]() __attribute__((always_inline)) {
        todo -= run;
        sk += run;
        so += (run - 1) * so_step;
        if (!AROWS) pa_src += (run - 1) * (kBK * a.lda * 2);
        if (!BROWS) pb_src += (run - 1) * (kBK * a.ldb * 2);
        --sk;                      // la1: the step the cursor leaves
        set(LA1{});
        ++sk;
        so += so_step;
        if (!AROWS) pa_src += kBK * a.lda * 2;
        if (!BROWS) pb_src += kBK * a.ldb * 2;
        const bool turned = todo == 0 || (PROD == kDx && seg == 0 && sk == a.steps_seg);
        if (turned) turn();
        set_all();
        run = 1;
        if (!turned) {
            const int last = a.steps_seg - (tail ? 1 : 0) - sk;   // steps to the special one, or past the end
            run = todo < last ? todo : last;
            if (run < 1) run = 1;
        }
        until = run;
    };

    // ---- fragment addresses, in the stage of the current step ----
    const int fr = lane & 15, grp = lane >> 4;
    const uint32_t lds0 = lds_addr(lds);
    constexpr int HB = 4 * HALF * 2, KB = 32 * HALF * 2;
    uint32_t pa[AROWS ? 2 : QM], pb[2];
    if constexpr (AROWS) {
        const uint32_t row = lds0 + uint32_t(wm * QM * 16 + fr) * 128;
        pa[0] = row + ((grp ^ (fr & 7)) << 4);
        pa[1] = row + (((grp + 4) ^ (fr & 7)) << 4);
    } else {
        const int k = grp * 8 + (fr >> 2);
#pragma unroll
        for (int i = 0; i < QM; ++i)
            pa[i] = lds0 + k * (HALF * 2) + (((wm * QM + i) ^ Operand<false, false, HALF>::swz(k)) << 5) + 8 * (fr & 3);
    }
    if constexpr (BROWS) {
        const uint32_t row = lds0 + BBASE + uint32_t(wn * 32 + 8 * (fr >> 2) + (fr & 3)) * 128;
        pb[0] = row + ((grp ^ (fr & 7)) << 4);
        pb[1] = row + (((grp + 4) ^ (fr & 7)) << 4);
    } else {
        const int k = grp * 8 + (fr >> 2);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            pb[j] = lds0 + BBASE + k * (HALF * 2) + (((wn * 2 + j) ^ Operand<false, false, HALF>::swz(k)) << 5) +
                    8 * (fr & 3);
    }

    i32x4 fa[QM][2], fb0[2][2], fb1[2][2], fbn[2][2];   // fbn: column half 0 of the next step
    f32x4 acc[2][2][QM][2];
    // products of row half X with column half Y; FIRST: the tile's first, onto 0
    auto products = [&](auto xc, auto yc, auto fc) __attribute__((always_inline)) {
        constexpr int X = decltype(xc)::value, Y = decltype(yc)::value;
        constexpr bool FIRST = decltype(fc)::value != 0;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int i = 0; i < QM; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[X][Y][i][j] = mfma16x16x32<T>(Y ? fb1[j][ks] : fb0[j][ks], fa[i][ks],
                                                      FIRST && ks == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[X][Y][i][j]);
        }
    };
    auto begin = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        if (PP) __builtin_amdgcn_s_setprio(1);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto end = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        if (PP) {
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int delta = HBYTES;            // from the current step's stage to the other
    uint32_t to = lds0 + wave * 2048;   // this wave's loads into the current step's stage
    bool drained = true;           // no result stores behind the loads in flight
    auto step = [&](auto fc) __attribute__((always_inline)) {
        constexpr bool FIRST = decltype(fc)::value != 0;
        auto wait = [&]() __attribute__((always_inline)) {
            if (FIRST && STORES > 0 && !drained) wait_vm<8 + STORES>();
            else wait_vm<8>();
        };
        // phase 0; loads row half 1 of the next step, column half 0 of the one after
        constexpr int A1 = 2 * HBYTES, B0 = BBASE, B1 = BBASE + 2 * HBYTES;
        const uint32_t other = to + delta;
        if constexpr (BROWS) read_rows_rows<0, 2 * HBYTES, A1, B0>(fa, fb1, pa, pb, la1, other, lb0, to);
        else if constexpr (AROWS) read_rows_cols<0, 2 * HBYTES, A1, B0, HB, KB>(fa, fb1, pa, pb, la1, other, lb0, to);
        else read_cols_cols<0, 2 * HBYTES, A1, B0, HB, KB>(fa, fb1, pa, pb, la1, other, lb0, to);
        wait();
        begin();
        products(IC<0>{}, IC<0>{}, fc);
        products(IC<0>{}, IC<1>{}, fc);
        end();
        // phase 1; loads row half 0 and column half 1 of the step after next
        {
            const uint32_t pn[2] = {pb[0] + delta, pb[1] + delta};
            if constexpr (BROWS) read_rows_rows<2 * HBYTES, 0, 0, B1>(fa, fbn, pa, pn, la0, to, lb1, to);
            else if constexpr (AROWS) read_rows_cols<2 * HBYTES, 0, 0, B1, HB, KB>(fa, fbn, pa, pn, la0, to, lb1, to);
            else read_cols_cols<2 * HBYTES, 0, 0, B1, HB, KB>(fa, fbn, pa, pn, la0, to, lb1, to);
        }
        wait();
        begin();
        products(IC<1>{}, IC<0>{}, fc);
        products(IC<1>{}, IC<1>{}, fc);
        // between them: the cursor's next loads and the other stage's addresses
        hop();
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) fb0[j][ks] = fbn[j][ks];
#pragma unroll
        for (int i = 0; i < (AROWS ? 2 : QM); ++i) pa[i] += delta;
        pb[0] += delta;
        pb[1] += delta;
        to = other;
        delta = -delta;
#pragma unroll
        for (int i = 0; i < 4 * QM; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, QM == 4 ? 2 : 1, 0);   // products
            __builtin_amdgcn_sched_group_barrier(0x004, 2, 0);                 // scalar
            __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);                 // vector
        }
        if (until == 0) move();
        end();
    };

    // ---- results of a tile ----
    // (the views' bases and lengths cover the rows of this tile; an offset of
    // kOob is dropped)
    auto results = [&](const Tile& t) __attribute__((always_inline)) {
        ArgsMem& a = args_again<ARG>();
        // the lane, made anew: neither it nor what follows from it is worth
        // registers over the steps
        int zero = 0;
        asm volatile("" : "+v"(zero));
        const int lane = int(__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, uint32_t(zero))));
        const int fr = lane & 15, grp = lane >> 4;
        const int mrow = wm * QM * 16 + fr;           // + half * HALF + 16 * i
        const int64_t mleft = a.m - t.m0;
        bool wide = a.wide != 0;   // whole 16-byte vectors, all inside or all outside the result
        if constexpr (END == kEndPart) {
            constexpr int64_t HSTEP = PROD == kProj ? 0 : HALF;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int i = 0; i < QM; ++i) {
                    const int64_t ml = x * HALF + mrow + 16 * i;
                    if (ml >= mleft) continue;
                    float* p = a.part + (int64_t(t.split) * a.m + t.m0 + ml) * a.part_ld;
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            // PROJ: 8 hidden units a lane over its two tiles
                            const int64_t n = t.n0 + y * HSTEP + wn * 32 +
                                              (PROD == kProj ? 8 * grp + 4 * j : 16 * j + 4 * grp);
                            if (n < (PROD == kProj ? a.fp : a.n))
                                *reinterpret_cast<f32x4*>(p + (PROD == kProj ? y * a.fp : 0) + n) = acc[x][y][i][j];
                        }
                }
        } else if constexpr (PROD == kProj) {
            const int fl = wn * 32 + 8 * grp;         // 8 hidden units a lane
            const int64_t f = t.n0 + fl;
            const int cnt = int(a.f - f < 8 ? a.f - f : 8);   // that exist
            const int rows = int(mleft < TILE ? mleft : TILE);
            // y, or dy: 16-byte vectors by view and offset, or elements by pointer
            const char* base = static_cast<const char*>(END == kEndFwd ? a.y : a.dy);
            const int64_t ld = END == kEndFwd ? a.ldy : a.lddy;
            base += (t.m0 * ld + t.n0) * 2;
            const __amdgpu_buffer_rsrc_t rb = view(base, ((mleft - 1) * ld + a.f - t.n0) * 2);
            const uint32_t step = uint32_t(ld * 32);          // 16 rows
            const uint32_t off = cnt == 8 ? uint32_t((mrow * ld + fl) * 2) : kOob;
            auto at = [&](int x, int i) __attribute__((always_inline)) -> uint32_t {
                return mrow + x * HALF + 16 * i < rows && cnt == 8 ? off + uint32_t(x * (HALF / 16) + i) * step : kOob;
            };
            auto ptr = [&](int x, int i) __attribute__((always_inline)) -> char* {
                return const_cast<char*>(base) + ((mrow + x * HALF + 16 * i) * ld + fl) * 2;
            };
            auto left = [&](int x, int i) __attribute__((always_inline)) -> int {
                return mrow + x * HALF + 16 * i < rows ? cnt : 0;
            };
            if constexpr (END == kEndFwd) {
                auto value = [&](int x, int i) __attribute__((always_inline)) -> i32x4 {
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[e] = act_value(ACT, acc[x][0][i][e >> 2][e & 3]) * acc[x][1][i][e >> 2][e & 3];
                    return pack_vec<T>(o);
                };
                if (wide) {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int i = 0; i < QM; ++i) buf_store16(value(x, i), rb, at(x, i));
                } else {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int i = 0; i < QM; ++i) store_n<T>(ptr(x, i), value(x, i), left(x, i));
                }
            } else {
                const char* gp = static_cast<const char*>(a.dgu) + (t.m0 * 2 * a.fp + t.n0) * 2;
                const __amdgpu_buffer_rsrc_t rg = view(gp, (mleft * 2 * a.fp - t.n0) * 2);
                const uint32_t gstep = uint32_t(a.fp * 64);
                const uint32_t goff = uint32_t((mrow * 2 * a.fp + fl) * 2);
                i32x4 dyv[2][QM];
                if (wide) {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int i = 0; i < QM; ++i) dyv[x][i] = buf_load16(rb, at(x, i));
                } else {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int i = 0; i < QM; ++i) dyv[x][i] = load_n<T>(ptr(x, i), left(x, i));
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < QM; ++i) {
                        float dg[8], du[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float v, d;
                            act_both(ACT, acc[x][0][i][e >> 2][e & 3], v, d);
                            const float t1 = elem<T>(dyv[x][i], e);
                            dg[e] = t1 * acc[x][1][i][e >> 2][e & 3] * d;
                            du[e] = t1 * v;
                        }
                        i32x4 pg = pack_vec<T>(dg), pu = pack_vec<T>(du);
                        if (cnt < 8) {
                            // the columns f..fp-1 are operands of dx: exactly 0
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                const int mask = 2 * w + 1 < cnt ? -1 : 2 * w < cnt ? 0xffff : 0;
                                pg[w] &= mask;
                                pu[w] &= mask;
                            }
                        }
                        const uint32_t o = f < a.fp && mrow + x * HALF + 16 * i < rows
                                               ? goff + uint32_t(x * (HALF / 16) + i) * gstep : kOob;
                        store16_at(pg, rg, o);
                        store16_at(pu, rg, o == kOob ? kOob : o + uint32_t(a.fp * 2));
                    }
            }
        } else {
            // rows of dx, or of dwg and then dwu; a tile of DW that holds the
            // last rows of dwg and the first of dwu stores in two passes
            const bool up = PROD == kDw && t.m0 >= a.fp;
            const bool both = PROD == kDw && !up && t.m0 + TILE > a.fp;
            const int64_t r0 = up ? t.m0 - a.fp : t.m0;
            const int64_t ld = PROD == kDw ? a.n : a.ldy;
            int64_t rows = PROD == kDw ? a.f - r0 : mleft;
            char* op = static_cast<char*>(PROD == kDx ? a.y : up ? a.dwu : a.dwg) + (r0 * ld + t.n0) * 2;
            int first = 0;                        // the tile's row that is the pass's row 0
            for (;;) {
                const __amdgpu_buffer_rsrc_t ro = view(op, ((rows - 1) * ld + a.n - t.n0) * 2);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < QM; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            // lanes of odd 16-lane rows take the second tile: 8 consecutive columns each
                            const f32x4 v0 = acc[x][y][i][0], v1 = acc[x][y][i][1];
                            const auto lo = __builtin_amdgcn_permlane16_swap(pack2<T>(v0[0], v0[1]),
                                                                             pack2<T>(v1[0], v1[1]), false, false);
                            const auto hi = __builtin_amdgcn_permlane16_swap(pack2<T>(v0[2], v0[3]),
                                                                             pack2<T>(v1[2], v1[3]), false, false);
                            const i32x4 v = {int(lo[0]), int(hi[0]), int(lo[1]), int(hi[1])};
                            const int ml = x * HALF + mrow + 16 * i - first;
                            const int c = y * HALF + wn * 32 + 16 * (grp & 1) + 8 * (grp >> 1);
                            const bool in = ml >= 0 && ml < rows && t.n0 + c < a.n;
                            if (wide) buf_store16(v, ro, in ? uint32_t((ml * ld + c) * 2) : kOob);
                            else if (in) store_n<T>(op + (ml * ld + c) * 2, v, int(a.n - t.n0 - c < 8 ? a.n - t.n0 - c : 8));
                        }
                if (PROD != kDw || !both || first) break;
                first = int(a.fp - t.m0);
                rows = a.f;
                op = static_cast<char*>(a.dwu) + t.n0 * 2;
            }
            if (both) wide = false;               // (more stores than the next step's wait counts)
        }
        drained = !wide || STORES == 0;
        if (drained) wait_vm<0>();
    };

    // ---- the block's tiles ----
    Tile cur = tile_of<TILE, NT, ARG>(first);
    aim();
    // steps 0 and 1 but for row half 1 of step 1, which phase 0 loads
    auto load = [&](const Load& l, int at) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t r = make_rsrc(
            reinterpret_cast<const void*>(uint64_t(uint32_t(l.r[0])) | uint64_t(uint32_t(l.r[1])) << 32), uint32_t(l.r[2]));
#pragma unroll
        for (int q = 0; q < 2; ++q) dma16(r, lds + at + wave * 2048 + q * 1024, l.v[q], l.s);
    };
    set_all();
#pragma unroll
    for (int stg = 0; stg < 2; ++stg) {
        load(lb0, BBASE + stg * HBYTES);
        load(la0, stg * HBYTES);
        load(lb1, BBASE + (2 + stg) * HBYTES);
        run = 1;                   // here the cursor moves by single steps
        move();
        if (stg == 0) load(la1, 2 * HBYTES);
    }
    wait_vm<8>();
    __builtin_amdgcn_s_barrier();
    if constexpr (BROWS) read_rows<0>(fb0, pb);
    else read_cols<0, HB, KB>(fb0, pb);
    __builtin_amdgcn_s_barrier();
    if (PP && wm == 1) __builtin_amdgcn_s_barrier();
    for (int v = first;;) {
        step(IC<1>{});
        for (int s = 1; s < cur.steps; ++s) step(IC<0>{});
        results(cur);
        v += stride;
        if (v >= total) break;
        cur = tile_of<TILE, NT, ARG>(v);
    }
    if (PP && wm == 0) __builtin_amdgcn_s_barrier();
    wait_vm<0>();   // the loads past the last step still write LDS
}

template <typename T, int PROD, int TILE, int END, int ACT>
__global__ __launch_bounds__(kTileThreads(TILE), 2) void gated_gemm_kernel(const GatedArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[kTileLds(TILE)];
    gated_product<T, PROD, TILE, END, ACT, 0>(a, lds, int(blockIdx.x), int(gridDim.x));
}

// dx and the weights' gradients in one launch, where neither fills the GPU:
// blocks below `split` take tiles of dx, the others of dwg and dwu, one tile
// each.
struct GatedPair {
    GatedArgs p[2];
    int split;
};
template <typename T, int END0, int END1>
__global__ __launch_bounds__(kTileThreads(kGatedSmall), 2) void gated_pair_kernel(const GatedPair a) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[kTileLds(kGatedSmall)];
    const int b = blockIdx.x;
    if (b < a.split) {
        if (b >= a.p[0].tiles_m * a.p[0].tiles_n * a.p[0].splits) return;
        gated_product<T, kDx, kGatedSmall, END0, 0, 0>(a.p[0], lds, b, a.split);
    } else {
        gated_product<T, kDw, kGatedSmall, END1, 0, 1>(a.p[1], lds, b - a.split, int(gridDim.x) - a.split);
    }
}

// ---- joining a split reduction: splits are added in ascending order -------------

template <typename T>
__global__ __launch_bounds__(256) void gated_join_proj_kernel(const GatedArgs a) {
    const int64_t vecs = a.fp / 8, n = a.m * vecs;
    for (int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x; v < n; v += int64_t(gridDim.x) * 256) {
        const int64_t m = n <= 0xffffffffll ? int64_t(uint32_t(v) / uint32_t(vecs)) : v / vecs, f = (v - m * vecs) * 8;
        float g[8], u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = u[e] = 0.0f;
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) {
            const float* p = a.part + (int64_t(s) * a.m + m) * a.part_ld + f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 pg = *reinterpret_cast<const f32x4*>(p + 4 * h);
                const f32x4 pu = *reinterpret_cast<const f32x4*>(p + a.fp + 4 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    g[4 * h + e] += pg[e];
                    u[4 * h + e] += pu[e];
                }
            }
        }
        const int left = int(a.f - f < 8 ? a.f - f : 8);
        if (a.end == kEndFwd) {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = act_value(a.act, g[e]) * u[e];
            store_n<T>(static_cast<char*>(a.y) + (m * a.ldy + f) * 2, pack_vec<T>(g), left);
        } else {
            const i32x4 dyv = load_n<T>(static_cast<const char*>(a.dy) + (m * a.lddy + f) * 2, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float val, d;
                act_both(a.act, g[e], val, d);
                const float t = elem<T>(dyv, e);
                g[e] = e < left ? t * u[e] * d : 0.0f;
                u[e] = e < left ? t * val : 0.0f;
            }
            char* p = static_cast<char*>(a.dgu) + (m * 2 * a.fp + f) * 2;
            *reinterpret_cast<i32x4*>(p) = pack_vec<T>(g);
            *reinterpret_cast<i32x4*>(p + a.fp * 2) = pack_vec<T>(u);
        }
    }
}

template <typename T, bool DW>
__device__ __attribute__((always_inline)) inline void join_splits(const GatedArgs& a) {
    const int64_t vecs = a.part_ld / 4, n = a.m * vecs;
    for (int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x; v < n; v += int64_t(gridDim.x) * 256) {
        const int64_t m = n <= 0xffffffffll ? int64_t(uint32_t(v) / uint32_t(vecs)) : v / vecs, c = (v - m * vecs) * 4;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int q = 0; q < a.splits; ++q)
            s += *reinterpret_cast<const f32x4*>(a.part + (int64_t(q) * a.m + m) * a.part_ld + c);
        char* row;
        if constexpr (DW) {
            const bool up = m >= a.fp;
            const int64_t f = up ? m - a.fp : m;
            if (f >= a.f) continue;
            row = static_cast<char*>(up ? a.dwu : a.dwg) + f * a.n * 2;
        } else {
            row = static_cast<char*>(a.y) + m * a.ldy * 2;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < a.n) store1<T>(row + (c + e) * 2, s[e]);
    }
}

template <typename T, bool DW>
__global__ __launch_bounds__(256) void gated_join_kernel(const GatedArgs a) {
    join_splits<T, DW>(a);
}
template <typename T>
__global__ __launch_bounds__(256) void gated_join_pair_kernel(const GatedPair a) {
    if (blockIdx.y == 0) join_splits<T, false>(a.p[0]);
    else join_splits<T, true>(a.p[1]);
}

// Rows copied to a wider, 16-byte-aligned stride with zeros behind them; one
// operand per blockIdx.y.
struct PackArgs {
    GatedPack p[3];
};
__global__ __launch_bounds__(256) void gated_pack_kernel(const PackArgs a, int64_t cols, int64_t ldd) {
    const GatedPack p = blockIdx.y == 0 ? a.p[0] : blockIdx.y == 1 ? a.p[1] : a.p[2];
    const unsigned short* src = static_cast<const unsigned short*>(p.src);
    unsigned short* dst = static_cast<unsigned short*>(p.dst);
    const int64_t vecs = ldd / 8, n = p.rows * vecs;
    for (int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x; v < n; v += int64_t(gridDim.x) * 256) {
        const int64_t r = n <= 0xffffffffll ? int64_t(uint32_t(v) / uint32_t(vecs)) : v / vecs;
        const int64_t c = (v - r * vecs) * 8;
        const int left = int(cols - c < 8 ? cols - c : 8);
        *reinterpret_cast<i32x4*>(dst + r * ldd + c) = load_n<F16>(reinterpret_cast<const char*>(src + r * p.ld + c), left);
    }
}

__global__ __launch_bounds__(256) void gated_zero_kernel(unsigned short* dst, int64_t n) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) dst[i] = 0;
}

unsigned blocks_for(int64_t n) {
    const int64_t b = (n + 255) / 256, cap = int64_t(kNumCUs) * 16;
    return unsigned(b < cap ? b : cap);
}

template <typename T, int PROD, int END, int ACT>
int launch_tile(int tile, const GatedArgs& a, hipStream_t st) {
    const int64_t tiles = int64_t(a.tiles_m) * a.tiles_n * a.splits;
    // (block indices run past the last tile by at most one grid)
    if (tiles < 1 || tiles > 0x7fffffff - 4 * kNumCUs) return CNHWC_UNSUPPORTED;
    const int64_t slots = tile == kGatedBig ? kNumCUs : 2 * kNumCUs;
    const int64_t blocks = tiles < slots ? tiles : slots;
    if (tile == kGatedBig)
        gated_gemm_kernel<T, PROD, kGatedBig, END, ACT><<<dim3((unsigned)blocks), 512, 0, st>>>(a);
    else
        gated_gemm_kernel<T, PROD, kGatedSmall, END, ACT><<<dim3((unsigned)blocks), 256, 0, st>>>(a);
    return CNHWC_OK;
}

template <typename T, int END>
int launch_proj(int tile, const GatedArgs& a, hipStream_t st) {
    switch (a.act) {
    case CNHWC_ACT_SILU: return launch_tile<T, kProj, END, CNHWC_ACT_SILU>(tile, a, st);
    case CNHWC_ACT_GELU: return launch_tile<T, kProj, END, CNHWC_ACT_GELU>(tile, a, st);
    case CNHWC_ACT_RELU: return launch_tile<T, kProj, END, CNHWC_ACT_RELU>(tile, a, st);
    default: return launch_tile<T, kProj, END, CNHWC_ACT_SIGMOID>(tile, a, st);
    }
}

template <typename T>
int launch_prod(GatedProduct prod, int tile, const GatedArgs& a, hipStream_t st) {
    const bool part = a.splits > 1;
    switch (prod) {
    case kProj:
        if (part) return launch_tile<T, kProj, kEndPart, 0>(tile, a, st);
        return a.end == kEndFwd ? launch_proj<T, kEndFwd>(tile, a, st) : launch_proj<T, kEndBwd>(tile, a, st);
    case kDx:
        return part ? launch_tile<T, kDx, kEndPart, 0>(tile, a, st) : launch_tile<T, kDx, kEndFwd, 0>(tile, a, st);
    default:
        return part ? launch_tile<T, kDw, kEndPart, 0>(tile, a, st) : launch_tile<T, kDw, kEndFwd, 0>(tile, a, st);
    }
}

template <typename T>
void join(GatedProduct prod, const GatedArgs& a, hipStream_t st) {
    if (prod == kProj) gated_join_proj_kernel<T><<<blocks_for(a.m * (a.fp / 8)), 256, 0, st>>>(a);
    else if (prod == kDx) gated_join_kernel<T, false><<<blocks_for(a.m * (a.part_ld / 4)), 256, 0, st>>>(a);
    else gated_join_kernel<T, true><<<blocks_for(a.m * (a.part_ld / 4)), 256, 0, st>>>(a);
}

template <typename T>
void launch_pair(const GatedPair& g, int blocks, hipStream_t st) {
    const bool p0 = g.p[0].splits > 1, p1 = g.p[1].splits > 1;
    if (p0 && p1) gated_pair_kernel<T, kEndPart, kEndPart><<<blocks, 256, 0, st>>>(g);
    else if (p0) gated_pair_kernel<T, kEndPart, kEndFwd><<<blocks, 256, 0, st>>>(g);
    else if (p1) gated_pair_kernel<T, kEndFwd, kEndPart><<<blocks, 256, 0, st>>>(g);
    else gated_pair_kernel<T, kEndFwd, kEndFwd><<<blocks, 256, 0, st>>>(g);
}

}  // namespace

int launch_gated_product(int dtype, GatedProduct prod, int tile, const GatedArgs& a, hipStream_t st) {
    return dtype == CNHWC_F16 ? launch_prod<F16>(prod, tile, a, st) : launch_prod<BF16>(prod, tile, a, st);
}

int launch_gated_reduce(int dtype, GatedProduct prod, const GatedArgs& a, hipStream_t st) {
    if (dtype == CNHWC_F16) join<F16>(prod, a, st);
    else join<BF16>(prod, a, st);
    return CNHWC_OK;
}

int launch_gated_pair(int dtype, const GatedArgs& dx, const GatedArgs& dw, hipStream_t st) {
    GatedPair g;
    g.p[0] = dx;
    g.p[1] = dw;
    const int64_t n0 = int64_t(dx.tiles_m) * dx.tiles_n * dx.splits, n1 = int64_t(dw.tiles_m) * dw.tiles_n * dw.splits;
    g.split = int((n0 + 7) / 8 * 8);   // a multiple of the XCDs, whose tiles stay together
    if (g.split + n1 > 2 * kNumCUs) return CNHWC_UNSUPPORTED;
    const int blocks = g.split + int(n1);
    if (dtype == CNHWC_F16) launch_pair<F16>(g, blocks, st);
    else launch_pair<BF16>(g, blocks, st);
    return CNHWC_OK;
}

int launch_gated_pair_reduce(int dtype, const GatedArgs& dx, const GatedArgs& dw, hipStream_t st) {
    GatedPair g;
    g.p[0] = dx;
    g.p[1] = dw;
    g.split = 0;
    const int64_t v0 = dx.m * (dx.part_ld / 4), v1 = dw.m * (dw.part_ld / 4);
    const dim3 grid(blocks_for(v0 > v1 ? v0 : v1), 2);
    if (dtype == CNHWC_F16) gated_join_pair_kernel<F16><<<grid, 256, 0, st>>>(g);
    else gated_join_pair_kernel<BF16><<<grid, 256, 0, st>>>(g);
    return CNHWC_OK;
}

int launch_gated_pack(const GatedPack* p, int n, int64_t cols, int64_t ldd, hipStream_t st) {
    PackArgs a = {};
    int64_t most = 0;
    for (int i = 0; i < n; ++i) {
        a.p[i] = p[i];
        most = p[i].rows > most ? p[i].rows : most;
    }
    gated_pack_kernel<<<dim3(blocks_for(most * (ldd / 8)), n), 256, 0, st>>>(a, cols, ldd);
    return CNHWC_OK;
}

int launch_gated_zero(void* dst, int64_t n, hipStream_t st) {
    gated_zero_kernel<<<blocks_for(n), 256, 0, st>>>(static_cast<unsigned short*>(dst), n);
    return CNHWC_OK;
}

}  // namespace cnhwc
