// The matrix products of the gated feed-forward block on MFMA.
//
// One kernel serves the three products of gated.h.  A block computes a tile
// of 2*HM rows by 2*HN columns (HM = HN = 128 with 8 waves, 64 with 4); each
// operand's 64-deep slice of the tile is two half tiles in LDS, and a wave
// owns the same quarter of every half, so its result is four quadrants
// (row half, column half).  In PROJ the column halves are the same hidden
// units of wg and of wu: g and u of an element meet in one lane's registers
// and the activation and product (or, backward, dg and du) follow without
// another pass over memory.
//
// A step of the reduction runs in four phases, one quadrant each:
//     phase   reads into registers   multiplies
//       0     row half 0             (0, 0)
//       1     column half 1          (0, 1)
//       2     row half 1             (1, 1)
//       3     column half 0 of the   (1, 0)
//             next step
// so every half tile is read once and its LDS is free one phase later, where
// the asynchronous loads of the step after next refill it: with two stages a
// load has seven phases to land, and every phase's wait allows the same
// twelve younger loads in flight.  The 8-wave block runs its two halves of
// waves (one wave of each on every SIMD) half a phase apart, with a barrier on
// each side of the multiplications: while one wave of a SIMD multiplies, the
// other reads and issues loads.  The 4-wave block needs one barrier a phase
// and overlaps with the second block of its CU instead.
//
// A half tile whose rows are contiguous in the reduction (x, wg, wu in PROJ;
// dg | du in DX) lies in LDS as rows of 64 elements, read with 16-byte reads;
// one whose rows are the reduction (wg, wu in DX; both operands of DW) as 64
// rows of HM or HN elements, read with the transposing read.  16- or 32-byte
// units are exchanged by an exclusive-or with row bits so that the lanes of a
// read spread over all banks; the exchange is done by the load's source
// address.
//
// Addresses: each half tile's source is a buffer view rebuilt every step from
// a 64-bit base, so neither tensor size nor row count is limited by 32-bit
// offsets; rows past an operand's end read as zero by the view's length,
// columns past the reduction's end by an out-of-range offset.
#include "gated.h"

namespace cnhwc {
namespace {

constexpr int kBK = 64;   // reduction depth of a step

// Reads of one quadrant operand: NT 16-row tiles by two 32-deep products, all
// landed when the block ends (one asm block with its wait, so no register of
// it is live while a read is in flight).  p0 / p1: this lane's address for the
// first and second product; OFF: byte offset; TS: bytes from tile to tile.
template <int NT, int OFF, int TS>
__device__ __attribute__((always_inline)) inline void read_rows(i32x4 (&r)[NT][2], uint32_t p0, uint32_t p1) {
    if constexpr (NT == 4)
        asm volatile(
            "ds_read_b128 %0, %8 offset:%10\n\t"
            "ds_read_b128 %1, %9 offset:%10\n\t"
            "ds_read_b128 %2, %8 offset:%11\n\t"
            "ds_read_b128 %3, %9 offset:%11\n\t"
            "ds_read_b128 %4, %8 offset:%12\n\t"
            "ds_read_b128 %5, %9 offset:%12\n\t"
            "ds_read_b128 %6, %8 offset:%13\n\t"
            "ds_read_b128 %7, %9 offset:%13\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[1][0]), "=&v"(r[1][1]), "=&v"(r[2][0]), "=&v"(r[2][1]),
              "=&v"(r[3][0]), "=&v"(r[3][1])
            : "v"(p0), "v"(p1), "i"(OFF), "i"(OFF + TS), "i"(OFF + 2 * TS), "i"(OFF + 3 * TS)
            : "memory");
    else
        asm volatile(
            "ds_read_b128 %0, %4 offset:%6\n\t"
            "ds_read_b128 %1, %5 offset:%6\n\t"
            "ds_read_b128 %2, %4 offset:%7\n\t"
            "ds_read_b128 %3, %5 offset:%7\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[1][0]), "=&v"(r[1][1])
            : "v"(p0), "v"(p1), "i"(OFF), "i"(OFF + TS)
            : "memory");
}

// The same with the transposing read, two tiles at a time: a lane gets 4
// consecutive k of its column per read, KB bytes apart for the second product
// and HB bytes for k + 4.
template <int OFF, int KB, int HB>
__device__ __attribute__((always_inline)) inline void read_cols2(i32x4 (&r0)[2], i32x4 (&r1)[2], uint32_t p0,
                                                                 uint32_t p1) {
    i32x2 a, b, c, d, e, f, g, h;
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8 offset:%10\n\t"
        "ds_read_b64_tr_b16 %1, %8 offset:%11\n\t"
        "ds_read_b64_tr_b16 %2, %8 offset:%12\n\t"
        "ds_read_b64_tr_b16 %3, %8 offset:%13\n\t"
        "ds_read_b64_tr_b16 %4, %9 offset:%10\n\t"
        "ds_read_b64_tr_b16 %5, %9 offset:%11\n\t"
        "ds_read_b64_tr_b16 %6, %9 offset:%12\n\t"
        "ds_read_b64_tr_b16 %7, %9 offset:%13\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d), "=&v"(e), "=&v"(f), "=&v"(g), "=&v"(h)
        : "v"(p0), "v"(p1), "i"(OFF), "i"(OFF + HB), "i"(OFF + KB), "i"(OFF + KB + HB)
        : "memory");
    r0[0] = i32x4{a[0], a[1], b[0], b[1]};
    r0[1] = i32x4{c[0], c[1], d[0], d[1]};
    r1[0] = i32x4{e[0], e[1], f[0], f[1]};
    r1[1] = i32x4{g[0], g[1], h[0], h[1]};
}

// One operand of the tile: where its half tiles come from.  ROWS: contiguous
// in the reduction.  PERM: its rows are read in the order that gives a lane 8
// consecutive ones over two tiles (the result's columns).
template <bool ROWS, bool PERM, int HALF>
struct Operand {
    const char* base[2];   // half 0 / 1 at the current step
    const char* end[2];
    int64_t step;          // bytes from step to step
    uint32_t voff[2];      // this lane's offset in its wave's two 1 KiB regions
    int kc;                // ROWS: this lane's k within the step

    __device__ __attribute__((always_inline)) void lanes(int wave, int lane, int64_t ld) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int region = wave * 2 + q;
            if constexpr (ROWS) {
                const int row = region * 8 + (lane >> 3);
                const int swz = PERM ? ((row & 3) | ((row >> 1) & 4)) : (row & 7);
                voff[q] = uint32_t(row * ld * 2 + (((lane & 7) ^ swz) << 4));
            } else {
                constexpr int CH = HALF / 8;   // 16-byte units of a row
                const int k = region * (64 / CH) + lane / CH, pos = lane % CH;
                voff[q] = uint32_t(k * ld * 2 + ((((pos >> 1) ^ kswz(k)) << 5) | ((pos & 1) << 4)));
            }
        }
        kc = 0;
    }
    // exchange of 32-byte units in a row of HALF elements
    __device__ static int kswz(int k) {
        if constexpr (HALF == 128) return (k & 3) | ((k >> 1) & 4);
        else return ((k >> 1) & 1) | ((k >> 2) & 2);
    }
    // this lane's k within a step for region q
    __device__ __attribute__((always_inline)) static int lane_k(int wave, int lane, int q) {
        const int row = (wave * 2 + q) * 8 + (lane >> 3);
        const int swz = PERM ? ((row & 3) | ((row >> 1) & 4)) : (row & 7);
        return ((lane & 7) ^ swz) * 8;
    }
};

// END: what follows the products (a GatedEnd); ACT only where PROD is kProj.
template <typename T, int PROD, int TILE, int END, int ACT>
__global__ __launch_bounds__(TILE == kGatedBig ? 512 : 256, 2) void gated_gemm_kernel(const GatedArgs a) {
    constexpr bool AROWS = PROD != kDw, BROWS = PROD == kProj;
    constexpr int WN = TILE / 64, WAVES = 2 * WN;     // waves: 2 over rows, WN over columns
    constexpr int HALF = TILE / 2;                    // rows / columns of a half tile
    constexpr int QM = HALF / 32;                     // 16-row tiles of a quadrant; 2 tiles of columns
    constexpr bool PP = TILE == kGatedBig;            // two wave groups half a phase apart
    constexpr int HBYTES = HALF * 128;                // a half tile in LDS
    constexpr int BBASE = 4 * HBYTES;                 // A: [half][stage], then B
    __shared__ __attribute__((aligned(1024))) unsigned char lds[8 * HBYTES];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    // ---- block -> tile: consecutive tiles on one XCD (blocks go round the 8
    // XCDs in turn), in groups of 8 tile rows so that the tiles at work on an
    // XCD share operands in its L2
    const int tiles = a.tiles_m * a.tiles_n;
    const int total = tiles * a.splits;
    int id = blockIdx.x;
    {
        const int x = id & 7, q = id >> 3, base = total >> 3, rem = total & 7;
        id = x * base + (x < rem ? x : rem) + q;
    }
    const int split = id / tiles;
    int tm, tn;
    {
        const int t = id - split * tiles;
        const int per = 8 * a.tiles_n, grp = t / per, r = t - grp * per;
        const int rows = a.tiles_m - grp * 8 < 8 ? a.tiles_m - grp * 8 : 8;
        tn = r / rows;
        tm = grp * 8 + (r - tn * rows);
    }
    const int64_t m0 = int64_t(tm) * TILE;
    const int64_t n0 = int64_t(tn) * (PROD == kProj ? HALF : TILE);
    const int all_steps = a.segs * a.steps_seg;
    const int s_lo = int(int64_t(all_steps) * split / a.splits);
    const int s_hi = int(int64_t(all_steps) * (split + 1) / a.splits);
    const int steps = s_hi - s_lo;

    // ---- operand sources ----
    Operand<AROWS, false, HALF> A;
    Operand<BROWS, PROD == kProj, HALF> B;
    A.lanes(wave, lane, a.lda);
    B.lanes(wave, lane, a.ldb);
    int seg = 0, sk = s_lo;        // segment and step within it of the next loads
    int left = steps;              // steps still to load
    if (PROD == kDx && s_lo >= a.steps_seg) { seg = 1; sk = s_lo - a.steps_seg; }
    const char* ap = static_cast<const char*>(a.a);
    auto set_sources = [&]() __attribute__((always_inline)) {
        const int64_t kk = int64_t(sk) * kBK;
        if constexpr (AROWS) {
            const char* e = ap + ((a.m - 1) * a.lda + (PROD == kDx ? 2 * a.fp : a.k)) * 2;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                A.base[h] = ap + ((m0 + h * HALF) * a.lda + (PROD == kDx ? seg * a.fp : 0) + kk) * 2;
                A.end[h] = e;
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                A.base[h] = ap + (kk * a.lda + m0 + h * HALF) * 2;
                A.end[h] = ap + a.k * a.lda * 2;
            }
        }
        if constexpr (PROD == kProj) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const char* w = static_cast<const char*>(h ? a.b1 : a.b0);
                B.base[h] = w + (n0 * a.ldb + kk) * 2;
                B.end[h] = w + ((a.n - 1) * a.ldb + a.k) * 2;
            }
        } else {
            const char* w = static_cast<const char*>(PROD == kDx && seg ? a.b1 : a.b0);
            // rows of the right operand that exist
            const int64_t rows = PROD == kDx ? a.f : a.k;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                B.base[h] = w + (kk * a.ldb + n0 + h * HALF) * 2;
                B.end[h] = w + ((rows - 1) * a.ldb + a.nb) * 2;
            }
        }
    };
    set_sources();
    auto advance = [&]() __attribute__((always_inline)) {
        --left;
        ++sk;
        if (PROD == kDx && sk == a.steps_seg && seg == 0) {
            seg = 1;
            sk = 0;
        }
        set_sources();
    };
    // the two loads of this wave for one half tile of the cursor's step
    int akc[2], bkc[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        akc[q] = Operand<AROWS, false, HALF>::lane_k(wave, lane, q);
        bkc[q] = Operand<BROWS, PROD == kProj, HALF>::lane_k(wave, lane, q);
    }
    auto view = [&](const char* base, const char* end) __attribute__((always_inline)) {
        const int64_t n = left > 0 ? end - base : 0;
        return make_rsrc(base, n > 0 ? (n < 0x7fffffff ? uint32_t(n) : 0x7fffffffu) : 0u);
    };
    auto load_a = [&](auto hc, auto stg) __attribute__((always_inline)) {
        constexpr int H = decltype(hc)::value, STG = decltype(stg)::value;
        const __amdgpu_buffer_rsrc_t r = view(A.base[H], A.end[H]);
        const int64_t kleft = a.k - int64_t(sk) * kBK;
        const int kl = kleft < kBK ? int(kleft) : kBK;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t vo = !AROWS || akc[q] < kl ? A.voff[q] : kOob;
            dma16(r, lds + (H * 2 + STG) * HBYTES + (wave * 2 + q) * 1024, vo, 0);
        }
    };
    auto load_b = [&](auto hc, auto stg) __attribute__((always_inline)) {
        constexpr int H = decltype(hc)::value, STG = decltype(stg)::value;
        const __amdgpu_buffer_rsrc_t r = view(B.base[H], B.end[H]);
        const int64_t kleft = a.k - int64_t(sk) * kBK;
        const int kl = kleft < kBK ? int(kleft) : kBK;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t vo = !BROWS || bkc[q] < kl ? B.voff[q] : kOob;
            dma16(r, lds + BBASE + (H * 2 + STG) * HBYTES + (wave * 2 + q) * 1024, vo, 0);
        }
    };

    // ---- fragment addresses ----
    const int fr = lane & 15, grp = lane >> 4;
    const uint32_t lds0 = lds_addr(lds);
    uint32_t pa[4], pb[2];
    if constexpr (AROWS) {
        const uint32_t row = uint32_t(wm * QM * 16 + fr) * 128;
        pa[0] = lds0 + row + ((grp ^ (fr & 7)) << 4);
        pa[1] = lds0 + row + (((grp + 4) ^ (fr & 7)) << 4);
        pa[2] = pa[3] = 0;
    } else {
        const int k = grp * 8 + (fr >> 2);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pa[i] = i < QM ? lds0 + k * (HALF * 2) + (((wm * QM + i) ^ Operand<false, false, HALF>::kswz(k)) << 5) +
                                 8 * (fr & 3)
                           : 0;
    }
    if constexpr (BROWS) {
        const uint32_t row = uint32_t(wn * 32 + 8 * (fr >> 2) + (fr & 3)) * 128;
        pb[0] = lds0 + BBASE + row + ((grp ^ (fr & 7)) << 4);
        pb[1] = lds0 + BBASE + row + (((grp + 4) ^ (fr & 7)) << 4);
    } else {
        const int k = grp * 8 + (fr >> 2);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            pb[j] = lds0 + BBASE + k * (HALF * 2) + (((wn * 2 + j) ^ Operand<false, false, HALF>::kswz(k)) << 5) +
                    8 * (fr & 3);
    }

    i32x4 fa[QM][2], fb0[2][2], fb1[2][2];
    f32x4 acc[2][2][QM][2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int i = 0; i < QM; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[x][y][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto read_a = [&](auto hc, auto stg) __attribute__((always_inline)) {
        constexpr int OFF = (decltype(hc)::value * 2 + decltype(stg)::value) * HBYTES;
        if constexpr (AROWS) {
            read_rows<QM, OFF, 2048>(fa, pa[0], pa[1]);
        } else {
            read_cols2<OFF, 32 * HALF * 2, 4 * HALF * 2>(fa[0], fa[1], pa[0], pa[1]);
            if constexpr (QM == 4)
                read_cols2<OFF, 32 * HALF * 2, 4 * HALF * 2>(fa[2], fa[3], pa[2], pa[3]);
        }
    };
    auto read_b = [&](i32x4 (&f)[2][2], auto hc, auto stg) __attribute__((always_inline)) {
        constexpr int OFF = (decltype(hc)::value * 2 + decltype(stg)::value) * HBYTES;
        if constexpr (BROWS) read_rows<2, OFF, 512>(f, pb[0], pb[1]);
        else read_cols2<OFF, 32 * HALF * 2, 4 * HALF * 2>(f[0], f[1], pb[0], pb[1]);
    };
    auto multiply = [&](auto xc, auto yc) __attribute__((always_inline)) {
        constexpr int X = decltype(xc)::value, Y = decltype(yc)::value;
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        if (PP) __builtin_amdgcn_s_setprio(1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int i = 0; i < QM; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[X][Y][i][j] = mfma16x16x32<T>(Y ? fb1[j][ks] : fb0[j][ks], fa[i][ks], acc[X][Y][i][j]);
        __builtin_amdgcn_sched_barrier(0);
        if (PP) {
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using H0 = IC<0>;
    using H1 = IC<1>;
    auto step = [&](auto stg) __attribute__((always_inline)) {
        using S = decltype(stg);
        using N = IC<1 - S::value>;
        load_b(H0{}, S{});
        read_a(H0{}, S{});
        wait_vm<12>();
        multiply(H0{}, H0{});
        load_a(H0{}, S{});
        read_b(fb1, H1{}, S{});
        wait_vm<12>();
        multiply(H0{}, H1{});
        load_b(H1{}, S{});
        read_a(H1{}, S{});
        wait_vm<12>();
        multiply(H1{}, H1{});
        load_a(H1{}, S{});
        advance();
        // fb0 of this step is still to be multiplied: the next step's goes
        // to a copy that takes its place afterwards
        i32x4 next[2][2];
        read_b(next, H0{}, N{});
        wait_vm<12>();
        multiply(H1{}, H0{});
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) fb0[j][ks] = next[j][ks];
    };

    // ---- prologue: two steps of loads, the first column half ----
    load_b(H0{}, IC<0>{});
    load_a(H0{}, IC<0>{});
    load_b(H1{}, IC<0>{});
    load_a(H1{}, IC<0>{});
    advance();
    load_b(H0{}, IC<1>{});
    load_a(H0{}, IC<1>{});
    load_b(H1{}, IC<1>{});
    load_a(H1{}, IC<1>{});
    advance();
    wait_vm<12>();
    __builtin_amdgcn_s_barrier();
    read_b(fb0, H0{}, IC<0>{});
    __builtin_amdgcn_s_barrier();
    if (PP && wm == 1) __builtin_amdgcn_s_barrier();
    for (int s = 0; s < steps; s += 2) {
        step(IC<0>{});
        if (s + 1 < steps) step(IC<1>{});
    }
    if (PP && wm == 0) __builtin_amdgcn_s_barrier();
    wait_vm<0>();   // the loads past the last step still write LDS

    // ---- results ----
    if constexpr (PROD == kProj) {
        const int64_t f = n0 + wn * 32 + 8 * grp;   // 8 hidden units per lane
        if (f >= a.fp) return;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < QM; ++i) {
                const int64_t m = m0 + x * HALF + (wm * QM + i) * 16 + fr;
                if (m >= a.m) continue;
                if constexpr (END == kEndPart) {
                    float* p = a.part + (int64_t(split) * a.m + m) * a.part_ld + f;
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            *reinterpret_cast<f32x4*>(p + y * a.fp + 4 * j) = acc[x][y][i][j];
                } else if constexpr (END == kEndFwd) {
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[e] = act_value(ACT, acc[x][0][i][e >> 2][e & 3]) * acc[x][1][i][e >> 2][e & 3];
                    store_n<T>(static_cast<char*>(a.y) + (m * a.ldy + f) * 2, pack_vec<T>(o), int(a.f - f < 8 ? a.f - f : 8));
                } else {
                    const int left = int(a.f - f < 8 ? a.f - f : 8);
                    const i32x4 dyv = load_n<T>(static_cast<const char*>(a.dy) + (m * a.lddy + f) * 2, left);
                    float dg[8], du[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float v, d;
                        act_both(ACT, acc[x][0][i][e >> 2][e & 3], v, d);
                        const float t = elem<T>(dyv, e);
                        // the columns f..fp-1 are operands of dx: exactly 0
                        dg[e] = e < left ? t * acc[x][1][i][e >> 2][e & 3] * d : 0.0f;
                        du[e] = e < left ? t * v : 0.0f;
                    }
                    char* p = static_cast<char*>(a.dgu) + (m * 2 * a.fp + f) * 2;
                    *reinterpret_cast<i32x4*>(p) = pack_vec<T>(dg);
                    *reinterpret_cast<i32x4*>(p + a.fp * 2) = pack_vec<T>(du);
                }
            }
    } else {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < QM; ++i) {
                const int64_t m = m0 + x * HALF + (wm * QM + i) * 16 + fr;
                if (m >= a.m) continue;
                char* row = nullptr;
                if constexpr (END != kEndPart) {
                    if constexpr (PROD == kDx) {
                        row = static_cast<char*>(a.y) + m * a.ldy * 2;
                    } else {
                        const bool up = m >= a.fp;
                        const int64_t f = up ? m - a.fp : m;
                        if (f >= a.f) continue;
                        row = static_cast<char*>(up ? a.dwu : a.dwg) + f * a.n * 2;
                    }
                }
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int64_t n = n0 + y * HALF + wn * 32 + j * 16 + 4 * grp;
                        const f32x4 v = acc[x][y][i][j];
                        if (n >= a.n) continue;
                        if constexpr (END == kEndPart) {
                            *reinterpret_cast<f32x4*>(a.part + (int64_t(split) * a.m + m) * a.part_ld + n) = v;
                        } else if (n + 4 <= a.n) {
                            struct __attribute__((packed, aligned(2))) W2 { uint32_t w[2]; };
                            *reinterpret_cast<W2*>(row + n * 2) = W2{{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])}};
                        } else {
#pragma unroll
                            for (int e = 0; e < 3; ++e)
                                if (n + e < a.n) store1<T>(row + (n + e) * 2, v[e]);
                        }
                    }
            }
    }
}

// ---- joining a split reduction: splits are added in ascending order -------------

template <typename T>
__global__ __launch_bounds__(256) void gated_join_proj_kernel(const GatedArgs a) {
    const int64_t vecs = a.fp / 8, n = a.m * vecs;
    for (int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x; v < n; v += int64_t(gridDim.x) * 256) {
        const int64_t m = v / vecs, f = (v - m * vecs) * 8;
        float g[8], u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = u[e] = 0.0f;
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
__global__ __launch_bounds__(256) void gated_join_kernel(const GatedArgs a) {
    const int64_t vecs = a.part_ld / 4, n = a.m * vecs;
    for (int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x; v < n; v += int64_t(gridDim.x) * 256) {
        const int64_t m = v / vecs, c = (v - m * vecs) * 4;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
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

// Rows copied to a wider, 16-byte-aligned stride with zeros behind them.
__global__ __launch_bounds__(256) void gated_pack_kernel(const unsigned short* src, int64_t lds, int64_t rows,
                                                         int64_t cols, unsigned short* dst, int64_t ldd) {
    const int64_t vecs = ldd / 8, n = rows * vecs;
    for (int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x; v < n; v += int64_t(gridDim.x) * 256) {
        const int64_t r = v / vecs, c = (v - r * vecs) * 8;
        const int left = int(cols - c < 8 ? cols - c : 8);
        const i32x4 x = load_n<F16>(reinterpret_cast<const char*>(src + r * lds + c), left);
        *reinterpret_cast<i32x4*>(dst + r * ldd + c) = x;
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
    const int64_t blocks = int64_t(a.tiles_m) * a.tiles_n * a.splits;
    if (blocks < 1 || blocks > 0x7fffffff) return CNHWC_UNSUPPORTED;
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

}  // namespace

int launch_gated_product(int dtype, GatedProduct prod, int tile, const GatedArgs& a, hipStream_t st) {
    return dtype == CNHWC_F16 ? launch_prod<F16>(prod, tile, a, st) : launch_prod<BF16>(prod, tile, a, st);
}

int launch_gated_reduce(int dtype, GatedProduct prod, const GatedArgs& a, hipStream_t st) {
    if (dtype == CNHWC_F16) join<F16>(prod, a, st);
    else join<BF16>(prod, a, st);
    return CNHWC_OK;
}

int launch_gated_pack(const void* src, int64_t lds, int64_t rows, int64_t cols, void* dst, int64_t ldd,
                      hipStream_t st) {
    gated_pack_kernel<<<blocks_for(rows * (ldd / 8)), 256, 0, st>>>(static_cast<const unsigned short*>(src), lds, rows,
                                                                    cols, static_cast<unsigned short*>(dst), ldd);
    return CNHWC_OK;
}

int launch_gated_zero(void* dst, int64_t n, hipStream_t st) {
    gated_zero_kernel<<<blocks_for(n), 256, 0, st>>>(static_cast<unsigned short*>(dst), n);
    return CNHWC_OK;
}

}  // namespace cnhwc
