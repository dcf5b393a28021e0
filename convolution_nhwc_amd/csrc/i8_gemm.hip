// Products in 8-bit integers on MFMA, y = act(x w^T sx sw + bias) + residual.
//
// The loop is that of the 16-bit products' projections, byte for byte: a block
// computes tiles of 2 * HALF rows by 2 * HALF columns (256 x 256 with 8 waves,
// 128 x 128 with 4), a step is 128 bytes of every row, each operand's slice two
// half tiles in LDS, and a wave owns the same quarter of every half.  A 16 x 16
// instruction is 64 products deep where the 16-bit one is 32, in the same
// cycles and from the same 16 bytes a lane, so the rhythm of reads, loads and
// products carries over:
//     phase   reads into registers                         multiplies row half
//       0     row half 0, column half 1                            0
//       1     row half 1, column half 0 of the next step           1
// Every half tile is read once, and its LDS is free one phase later, where the
// asynchronous loads of the step after next refill it; each phase waits for all
// but the eight youngest loads.  The 8-wave block runs its two halves of waves
// half a phase apart; the 4-wave block overlaps with the second block of its CU.
//
// Blocks are persistent: the loads run on into a block's next tile while the
// current one is scaled, rounded and stored.
//
// Integer sums are exact in any order, so split reductions give the same bits as
// whole ones.
//
// 16384 x 8192 -> 8192 on large tiles: 2.87 POP/s (a library's 8192^3: 2.1 to 2.4).  At 2048
// channels a tile's results count: 16384 x 2048 -> 8192 takes 260 us, 320 with gelu (matrix
// cores 42 % busy): 256 x 256 activations that no product hides.  50176 x 1024 -> 384 with
// a residual on small tiles 43 us, 3.7 TB/s.
#include "i8.h"
#include "tile_core.h"

namespace cnhwc {
namespace {

typedef const __attribute__((address_space(4))) I8GemmArgs ArgsMem;
// The arguments read again from where they were passed: what only a tile's
// start and end need is not held in scalar registers over its steps.
__device__ __attribute__((always_inline)) inline ArgsMem& args_again() {
    auto p = (ArgsMem*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *p;
}

struct Tile {
    int64_t m0, n0;
    int split, s_lo, steps;
};

// The v-th tile of the launch: consecutive tiles on one XCD, in groups of 8 tile
// rows so that the tiles at work on an XCD share operands in its L2.
template <int TILE>
__device__ __attribute__((always_inline)) inline Tile tile_of(int v) {
    ArgsMem& a = args_again();
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
    t.n0 = int64_t(tn) * TILE;
    t.s_lo = int(uint32_t(a.steps) * uint32_t(t.split) / uint32_t(a.splits));
    t.steps = int(uint32_t(a.steps) * uint32_t(t.split + 1) / uint32_t(a.splits)) - t.s_lo;
    return t;
}

constexpr int kTileThreads(int tile) { return tile == kI8Big ? 512 : 256; }
constexpr int kTileLds(int tile) { return 8 * (tile / 2) * 128; }

// Eight consecutive values of a row from their sums; ACT kActAny: the activation
// is `act`.
constexpr int kActAny = 100;
template <int ACT, bool BF16OUT>
__device__ __attribute__((always_inline)) inline i32x4 finish8(const i32x4& s0, const i32x4& s1, float sx, const float (&sw)[8],
                                                               const float (&bias)[8], bool res, const i32x4& r, int act = 0) {
    using T = std::conditional_t<BF16OUT, BF16, F16>;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int s = e < 4 ? s0[e & 3] : s1[e & 3];
        f[e] = i8_act(ACT == kActAny ? act : ACT, float(s) * sx * sw[e] + bias[e]);
    }
    if (res) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += elem<T>(r, e);
    }
    return pack_vec<T>(f);
}
__device__ __attribute__((always_inline)) inline void load8(float (&v)[8], const float* p, int n, bool there) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = there && e < n ? p[e] : 0.0f;
}

// The scales and the bias of a tile lie in LDS behind the operands, loaded with
// its first step: asked for at its end, they and the residual would wait for the
// stores before them (loads and stores complete in order).  Both are asm, for the
// compiler waits for every load in flight before an LDS read that it sees.
__device__ __attribute__((always_inline)) inline void load_words(const i32x4& r, uint32_t voff, uint32_t to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %1, %0, 0 offen lds" : : "s"(r), "v"(voff), "s"(to) : "memory", "m0");
}
__device__ __attribute__((always_inline)) inline void read_words8(float (&v)[8], uint32_t at) {
    i32x4 a, b;
    asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:16\n\ts_waitcnt lgkmcnt(0)" : "=&v"(a), "=&v"(b) : "v"(at) : "memory");
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = elem<F32>(a, e);
        v[4 + e] = elem<F32>(b, e);
    }
}
// words at `at` and every 64 bytes on
template <int N>
__device__ __attribute__((always_inline)) inline void read_words_by16(float (&v)[N], uint32_t at) {
    static_assert(N == 2 || N == 4, "rows");
    if constexpr (N == 4)
        asm volatile("ds_read_b32 %0, %4\n\tds_read_b32 %1, %4 offset:64\n\tds_read_b32 %2, %4 offset:128\n\tds_read_b32 %3, %4 offset:192\n\t"
                     "s_waitcnt lgkmcnt(0)" : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]) : "v"(at) : "memory");
    else
        asm volatile("ds_read_b32 %0, %2\n\tds_read_b32 %1, %2 offset:64\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v[0]), "=&v"(v[1]) : "v"(at) : "memory");
}

template <int TILE, bool PART, bool BF16OUT>
__global__ __launch_bounds__(kTileThreads(TILE), 2) void i8_gemm_kernel(const I8GemmArgs a) {
    constexpr int WN = TILE / 64;                     // waves: 2 over rows, WN over columns
    constexpr int HALF = TILE / 2;                    // rows / columns of a half tile
    constexpr int QM = HALF / 32;                     // 16-row tiles of a quadrant; 2 tiles of columns
    constexpr bool PP = TILE == kI8Big;               // two wave groups half a phase apart
    constexpr int HBYTES = HALF * 128;                // a half tile in LDS
    constexpr int BBASE = 4 * HBYTES;                 // A: [half][stage], then B
    // stores of a tile's results per wave, all of them issued whatever the
    // tile's edges: the waits of the next tile's first step count over them
    constexpr int STORES = PART ? 0 : 4 * QM;
    constexpr int VBASE = kTileLds(TILE);             // scales of rows, of columns, bias; twice
    constexpr int VBYTES = PART ? 0 : 3 * TILE * 4;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[VBASE + 2 * VBYTES];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int first = int(blockIdx.x), stride = int(gridDim.x);
    const int total = a.tiles_m * a.tiles_n * a.splits;

    // ---- load cursor: views of the tile's rows, the reduction by the loads' scalar offset ----
    const Operand<true, false, HALF> A(wave, lane, a.lda);
    const Operand<true, true, HALF> B(wave, lane, a.ldb);
    const char *pa_src = nullptr, *pb_src = nullptr, *pu_src = nullptr;   // view bases; pu: the second column half
    uint32_t na = 0, nb = 0, nu = 0;   // their lengths
    uint32_t so = 0;                   // bytes into the rows
    uint32_t so_step = kBK * 2;        // 0 once no tile is left: an offset past an empty view would pass its check
    const int k_end = int(a.k - int64_t(a.steps - 1) * kBK);   // depth of the last step
    int cv = first, sk = 0;            // tile, and step within the reduction
    int todo = 0;                      // steps left of the tile
    auto aim = [&]() __attribute__((always_inline)) {
        int t_todo = 0x7fffffff, t_sk = 0;
        uint32_t t_so = 0, t_step = 0, t_na = 0, t_nb = 0, t_nu = 0;
        const char *t_pa = nullptr, *t_pb = nullptr, *t_pu = nullptr;
        if (cv < total) {
            ArgsMem& a = args_again();
            const Tile t = tile_of<TILE>(cv);
            t_todo = t.steps;
            t_sk = t.s_lo;
            t_so = uint32_t(t_sk) * (kBK * 2);
            t_step = kBK * 2;
            const int64_t rows = a.m - t.m0 < TILE ? a.m - t.m0 : TILE;
            t_pa = static_cast<const char*>(a.a) + t.m0 * a.lda * 2;
            t_na = uint32_t(((rows - 1) * a.lda + a.k) * 2);
            const int64_t left = a.n - t.n0;
            t_pb = static_cast<const char*>(a.b) + t.n0 * a.ldb * 2;
            t_nb = uint32_t(((left < HALF ? left : HALF) - 1) * a.ldb * 2 + a.bk);
            // (a second half without columns reads the first one's again: a view
            // shorter than its scalar offset would pass every check)
            t_pu = left > HALF ? t_pb + HALF * a.ldb * 2 : t_pb;
            t_nu = left > HALF ? uint32_t(((left < TILE ? left : TILE) - HALF - 1) * a.ldb * 2 + a.bk) : t_nb;
        }
        todo = t_todo;
        sk = t_sk;
        so = t_so;
        so_step = t_step;
        na = t_na;
        nb = t_nb;
        nu = t_nu;
        pa_src = t_pa;
        pb_src = t_pb;
        pu_src = t_pu;
    };
    Load la0, la1, lb0, lb1;           // of the cursor's step; la1: of the step before
    auto set_a = [&](Load& l, int h) __attribute__((always_inline)) {
        const int kl = sk == a.steps - 1 ? k_end : kBK;
        l.r = words_of(pa_src, na);
        l.s = uniform(so);
#pragma unroll
        for (int q = 0; q < 2; ++q) l.v[q] = A.lane_k[q] < kl ? A.voff[q] + h * A.half : kOob;
    };
    auto set_b = [&](Load& l, const char* src, uint32_t n) __attribute__((always_inline)) {
        const int kl = sk == a.steps - 1 ? k_end : kBK;
        l.r = words_of(src, n);
        l.s = uniform(so);
#pragma unroll
        for (int q = 0; q < 2; ++q) l.v[q] = B.lane_k[q] < kl ? B.voff[q] : kOob;
    };
    auto set_all = [&]() __attribute__((always_inline)) {
        set_a(la0, 0);
        set_b(lb0, pb_src, nb);
        set_b(lb1, pu_src, nu);
    };
    // The cursor moves on by `run` steps at a time: between, the loads differ by
    // an offset alone (hop); another tile or the mask of the last step is worked
    // out from the cursor (move).
    const bool tail = k_end != kBK;
    int run = 1, until = 1;
    auto hop = [&]() __attribute__((always_inline)) {
        la1.s = la0.s;
        la0.s += so_step;
        lb0.s = lb1.s = la0.s;
        --until;
    };
    auto move = [&]() __attribute__((always_inline)) {
        todo -= run;
        sk += run;
        so += (run - 1) * so_step;
        --sk;                          // la1: the step the cursor leaves
        set_a(la1, 1);
        ++sk;
        so += so_step;
        const bool turned = todo == 0;
        if (turned) {
            cv += stride;
            aim();
        }
        set_all();
        run = 1;
        if (!turned) {
            const int last = a.steps - (tail ? 1 : 0) - sk;   // steps to the special one, or past the end
            run = todo < last ? todo : last;
            if (run < 1) run = 1;
        }
        until = run;
    };

    // ---- fragment addresses, in the stage of the current step ----
    const int fr = lane & 15, grp = lane >> 4;
    const uint32_t lds0 = lds_addr(lds);
    uint32_t pa[2], pb[2];
    {
        const uint32_t row = lds0 + uint32_t(wm * QM * 16 + fr) * 128;
        pa[0] = row + ((grp ^ (fr & 7)) << 4);
        pa[1] = row + (((grp + 4) ^ (fr & 7)) << 4);
        const uint32_t col = lds0 + BBASE + uint32_t(wn * 32 + 8 * (fr >> 2) + (fr & 3)) * 128;
        pb[0] = col + ((grp ^ (fr & 7)) << 4);
        pb[1] = col + (((grp + 4) ^ (fr & 7)) << 4);
    }

    i32x4 fa[QM][2], fb0[2][2], fb1[2][2], fbn[2][2];   // fbn: column half 0 of the next step
    i32x4 acc[2][2][QM][2];
    auto products = [&](auto xc, auto yc, auto fc) __attribute__((always_inline)) {
        constexpr int X = decltype(xc)::value, Y = decltype(yc)::value;
        constexpr bool FIRST = decltype(fc)::value != 0;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int i = 0; i < QM; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[X][Y][i][j] = mfma16x16x64(Y ? fb1[j][ks] : fb0[j][ks], fa[i][ks],
                                                   FIRST && ks == 0 ? i32x4{0, 0, 0, 0} : acc[X][Y][i][j]);
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
    int delta = HBYTES;                // from the current step's stage to the other
    uint32_t to = lds0 + wave * 2048;  // this wave's loads into the current step's stage
    bool drained = true;               // no result stores behind the loads in flight
    bool only = false;                 // the tile's first step is its last: its scales have to be there after it
    auto step = [&](auto fc) __attribute__((always_inline)) {
        constexpr bool FIRST = decltype(fc)::value != 0;
        auto wait = [&](bool strict) __attribute__((always_inline)) {
            if (FIRST && STORES > 0 && !drained && !strict) wait_vm<8 + STORES>();
            else wait_vm<8>();
        };
        // phase 0; loads row half 1 of the next step, column half 0 of the one after
        constexpr int A1 = 2 * HBYTES, B0 = BBASE, B1 = BBASE + 2 * HBYTES;
        const uint32_t other = to + delta;
        read_rows_rows<0, 2 * HBYTES, A1, B0>(fa, fb1, pa, pb, la1, other, lb0, to);
        wait(false);
        begin();
        products(IC<0>{}, IC<0>{}, fc);
        products(IC<0>{}, IC<1>{}, fc);
        end();
        // phase 1; loads row half 0 and column half 1 of the step after next
        {
            const uint32_t pn[2] = {pb[0] + delta, pb[1] + delta};
            read_rows_rows<2 * HBYTES, 0, 0, B1>(fa, fbn, pa, pn, la0, to, lb1, to);
        }
        wait(FIRST && only);
        begin();
        products(IC<1>{}, IC<0>{}, fc);
        products(IC<1>{}, IC<1>{}, fc);
        // between them: the cursor's next loads and the other stage's addresses
        hop();
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) fb0[j][ks] = fbn[j][ks];
        pa[0] += delta;
        pa[1] += delta;
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

    // the lane, made anew: neither it nor what follows from it is worth registers over
    // the steps
    auto lane_again = [&]() __attribute__((always_inline)) -> int {
        int zero = 0;
        asm volatile("" : "+v"(zero));
        return int(__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, uint32_t(zero))));
    };

    // the scales and bias of tile t into the half of their LDS that `odd` tells: a wave
    // loads 64 words of each of up to two vectors (behind the operands' ends: zeros)
    int odd = 0;
    auto vectors = [&](const Tile& t) __attribute__((always_inline)) {
        if constexpr (!PART) {
            ArgsMem& a = args_again();
            constexpr int W = TILE / 64;   // waves that cover a vector; a block has twice as many
            static_assert(kTileThreads(TILE) / 64 == 2 * W, "waves");
            const uint32_t to = lds0 + VBASE + odd * VBYTES;
            const int q = wave % W;
            const uint32_t voff = uint32_t(q * 64 + lane_again()) * 4;
            const int64_t mleft = a.m - t.m0 < TILE ? a.m - t.m0 : TILE, nleft = a.n - t.n0 < TILE ? a.n - t.n0 : TILE;
            if (wave < W) {
                load_words(words_of(reinterpret_cast<const char*>(a.end.sx + t.m0), uint32_t(mleft * 4)), voff, uniform(to + q * 256));
                const bool there = a.end.bias != nullptr;
                load_words(words_of(there ? reinterpret_cast<const char*>(a.end.bias + t.n0) : nullptr, there ? uint32_t(nleft * 4) : 0u), voff,
                           uniform(to + 2 * TILE * 4 + q * 256));
            } else {
                load_words(words_of(reinterpret_cast<const char*>(a.end.sw + t.n0), uint32_t(nleft * 4)), voff, uniform(to + TILE * 4 + q * 256));
            }
        }
    };

    // ---- results of a tile: lane has row mrow (+ x HALF + 16 i), 8 columns from fl (+ y HALF) ----
    auto results = [&](const Tile& t) __attribute__((always_inline)) {
        ArgsMem& a = args_again();
        const int lane = lane_again();
        const int fr = lane & 15, grp = lane >> 4;
        const int mrow = wm * QM * 16 + fr, fl = wn * 32 + 8 * grp;
        const int64_t mleft = a.m - t.m0;
        if constexpr (PART) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int i = 0; i < QM; ++i) {
                    const int64_t ml = x * HALF + mrow + 16 * i;
                    if (ml >= mleft) continue;
                    int* p = a.part + (int64_t(t.split) * a.m + t.m0 + ml) * a.part_ld;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int64_t n = t.n0 + y * HALF + fl;
                        if (n < a.n) {
                            *reinterpret_cast<i32x4*>(p + n) = acc[x][y][i][0];
                            *reinterpret_cast<i32x4*>(p + n + 4) = acc[x][y][i][1];
                        }
                    }
                }
            drained = true;
            wait_vm<0>();
        } else {
            const I8End o = {a.end.sx, a.end.sw, a.end.bias, a.end.residual, a.end.y, a.end.ldr, a.end.ldy, a.end.act, a.end.bf16};
            const int wide = a.wide;
            const bool res = o.residual != nullptr;
            const int rows = int(mleft < TILE ? mleft : TILE);
            char* base = static_cast<char*>(o.y) + (t.m0 * o.ldy + t.n0) * 2;
            const char* rbase = static_cast<const char*>(o.residual) + (t.m0 * o.ldr + t.n0) * 2;
            const __amdgpu_buffer_rsrc_t ry = view(base, ((mleft - 1) * o.ldy + a.n - t.n0) * 2);
            const __amdgpu_buffer_rsrc_t rr = view(rbase, res ? ((mleft - 1) * o.ldr + a.n - t.n0) * 2 : 0);
            const uint32_t vec = lds0 + VBASE + odd * VBYTES;
            // whole vectors: offsets in the views, whose ends drop what is outside
            const uint32_t ystep = uint32_t(o.ldy * 32), rstep = uint32_t(o.ldr * 32);   // 16 rows
            const uint32_t yoff = uint32_t((mrow * o.ldy + fl) * 2), roff = uint32_t((mrow * o.ldr + fl) * 2);
            const int nleft = int(a.n - t.n0 < TILE ? a.n - t.n0 : TILE);
            auto at = [&](uint32_t off, uint32_t step, int x, int y, int i) __attribute__((always_inline)) -> uint32_t {
                return mrow + x * HALF + 16 * i < rows && y * HALF + fl < nleft ? off + uint32_t(x * (HALF / 16) + i) * step + y * HALF * 2 : kOob;
            };
            // any others: pointers, and the values of a vector that exist
            auto ptr = [&](const char* p, int64_t ld, int x, int y, int i) __attribute__((always_inline)) {
                return const_cast<char*>(p) + ((mrow + x * HALF + 16 * i) * ld + y * HALF + fl) * 2;
            };
            auto left = [&](int x, int y, int i) __attribute__((always_inline)) -> int {
                const int n = nleft - (y * HALF + fl);
                return mrow + x * HALF + 16 * i < rows && n > 0 ? (n < 8 ? n : 8) : 0;
            };
            // The four quadrants one after the other; on the small tile, which has the
            // registers, all residuals are on their way first: asked for later, they
            // wait for the stores before them.
            constexpr int kAhead = QM == 4 ? 0 : 4;
            auto all = [&](auto ac, auto wc) __attribute__((always_inline)) {
                constexpr int ACT = decltype(ac)::value;
                constexpr int WIDE = decltype(wc)::value;
                i32x4 r[4][QM];
                auto fetch = [&](auto qc) __attribute__((always_inline)) {
                    constexpr int Q = decltype(qc)::value, y = Q >> 1, x = Q & 1;
                    if constexpr (Q < 4) {
#pragma unroll
                        for (int i = 0; i < QM; ++i) {
                            r[Q][i] = i32x4{0, 0, 0, 0};
                            if (res) {
                                if (WIDE) r[Q][i] = buf_load16(rr, at(roff, rstep, x, y, i));
                                else r[Q][i] = load_n<F16>(ptr(rbase, o.ldr, x, y, i), left(x, y, i));
                            }
                        }
                    }
                };
                sfor<kAhead>([&](auto qc) __attribute__((always_inline)) { fetch(qc); });
                sfor<2>([&](auto yc) __attribute__((always_inline)) {
                    constexpr int y = decltype(yc)::value;
                    float sw[8], bias[8];
                    read_words8(sw, vec + TILE * 4 + uint32_t(y * HALF + fl) * 4);
                    read_words8(bias, vec + 2 * TILE * 4 + uint32_t(y * HALF + fl) * 4);
                    sfor<2>([&](auto xc) __attribute__((always_inline)) {
                        constexpr int x = decltype(xc)::value, Q = 2 * y + x;
                        fetch(IC<Q + kAhead>{});
                        float sx[QM];
                        read_words_by16(sx, vec + uint32_t(mrow + x * HALF) * 4);
#pragma unroll
                        for (int i = 0; i < QM; ++i) {
                            const i32x4 v = finish8<ACT, BF16OUT>(acc[x][y][i][0], acc[x][y][i][1], sx[i], sw, bias, res, r[Q][i], o.act);
                            if (WIDE == 1) buf_store16(v, ry, at(yoff, ystep, x, y, i));
                            else if (WIDE == 2) __builtin_amdgcn_raw_buffer_store_b128(v, ry, at(yoff, ystep, x, y, i), 0, 0);
                            else store_n<F16>(ptr(base, o.ldy, x, y, i), v, left(x, y, i));
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    });
                });
            };
            auto by_act = [&](auto wc) __attribute__((always_inline)) {
                switch (o.act) {
                case CNHWC_ACT_SILU: all(IC<CNHWC_ACT_SILU>{}, wc); break;
                case CNHWC_ACT_GELU: all(IC<CNHWC_ACT_GELU>{}, wc); break;
                case CNHWC_ACT_RELU: all(IC<CNHWC_ACT_RELU>{}, wc); break;
                case CNHWC_ACT_SIGMOID: all(IC<CNHWC_ACT_SIGMOID>{}, wc); break;
                default: all(IC<CNHWC_ACT_NONE>{}, wc);
                }
            };
            // (rows or alignment of odd sizes: the activation is chosen at each value)
            if (!wide) all(IC<kActAny>{}, IC<0>{});
            else if (wide == 1) by_act(IC<1>{});
            else by_act(IC<2>{});
            drained = !wide;
            if (drained) wait_vm<0>();
        }
    };

    // ---- the block's tiles ----
    Tile cur = tile_of<TILE>(first);
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
        run = 1;                       // here the cursor moves by single steps
        move();
        if (stg == 0) load(la1, 2 * HBYTES);
    }
    wait_vm<8>();
    __builtin_amdgcn_s_barrier();
    read_rows<0>(fb0, pb);
    __builtin_amdgcn_s_barrier();
    if (PP && wm == 1) __builtin_amdgcn_s_barrier();
    for (int v = first;;) {
        vectors(cur);
        only = cur.steps == 1;
        step(IC<1>{});
        for (int s = 1; s < cur.steps; ++s) step(IC<0>{});
        results(cur);
        odd ^= 1;
        v += stride;
        if (v >= total) break;
        cur = tile_of<TILE>(v);
    }
    if (PP && wm == 0) __builtin_amdgcn_s_barrier();
    wait_vm<0>();   // the loads past the last step still write LDS
}

// The sums of all splits, and what becomes of them.
template <bool BF16OUT>
__global__ __launch_bounds__(256) void i8_join_kernel(const I8GemmArgs a) {
    const int64_t vecs = (a.n + 7) / 8, total = a.m * vecs;
    for (int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x; v < total; v += int64_t(gridDim.x) * 256) {
        const int64_t m = total <= 0xffffffffll ? int64_t(uint32_t(v) / uint32_t(vecs)) : v / vecs, n = (v - m * vecs) * 8;
        i32x4 s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
#pragma unroll 4
        for (int q = 0; q < a.splits; ++q) {
            const int* p = a.part + (int64_t(q) * a.m + m) * a.part_ld + n;
            s0 += *reinterpret_cast<const i32x4*>(p);
            s1 += *reinterpret_cast<const i32x4*>(p + 4);
        }
        const int cnt = int(a.n - n < 8 ? a.n - n : 8);
        float sw[8], bias[8];
        load8(sw, a.end.sw + n, cnt, true);
        load8(bias, a.end.bias + n, cnt, a.end.bias != nullptr);
        const bool res = a.end.residual != nullptr;
        i32x4 r = {0, 0, 0, 0};
        if (res) r = load_n<F16>(static_cast<const char*>(a.end.residual) + (m * a.end.ldr + n) * 2, cnt);
        const float sx = a.end.sx[m];
        i32x4 o;
        switch (a.end.act) {
        case CNHWC_ACT_SILU: o = finish8<CNHWC_ACT_SILU, BF16OUT>(s0, s1, sx, sw, bias, res, r); break;
        case CNHWC_ACT_GELU: o = finish8<CNHWC_ACT_GELU, BF16OUT>(s0, s1, sx, sw, bias, res, r); break;
        case CNHWC_ACT_RELU: o = finish8<CNHWC_ACT_RELU, BF16OUT>(s0, s1, sx, sw, bias, res, r); break;
        case CNHWC_ACT_SIGMOID: o = finish8<CNHWC_ACT_SIGMOID, BF16OUT>(s0, s1, sx, sw, bias, res, r); break;
        default: o = finish8<CNHWC_ACT_NONE, BF16OUT>(s0, s1, sx, sw, bias, res, r);
        }
        store_n<F16>(static_cast<char*>(a.end.y) + (m * a.end.ldy + n) * 2, o, cnt);
    }
}

template <int TILE>
int launch_tile(const I8GemmArgs& a, hipStream_t st) {
    const int64_t tiles = int64_t(a.tiles_m) * a.tiles_n * a.splits;
    // (block indices run past the last tile by at most one grid)
    if (tiles < 1 || tiles > 0x7fffffff - 4 * kNumCUs) return CNHWC_UNSUPPORTED;
    const int64_t slots = TILE == kI8Big ? kNumCUs : 2 * kNumCUs;
    const dim3 blocks((unsigned)(tiles < slots ? tiles : slots));
    if (a.splits > 1) i8_gemm_kernel<TILE, true, false><<<blocks, kTileThreads(TILE), 0, st>>>(a);
    else if (a.end.bf16) i8_gemm_kernel<TILE, false, true><<<blocks, kTileThreads(TILE), 0, st>>>(a);
    else i8_gemm_kernel<TILE, false, false><<<blocks, kTileThreads(TILE), 0, st>>>(a);
    return CNHWC_OK;
}

}  // namespace

int launch_i8_gemm(int tile, const I8GemmArgs& a, hipStream_t st) {
    return tile == kI8Big ? launch_tile<kI8Big>(a, st) : launch_tile<kI8Small>(a, st);
}

int launch_i8_join(const I8GemmArgs& a, hipStream_t st) {
    const int64_t want = (a.m * ((a.n + 7) / 8) + 255) / 256, cap = int64_t(kNumCUs) * 16;
    const dim3 blocks((unsigned)(want < cap ? want : cap));
    if (a.end.bf16) i8_join_kernel<true><<<blocks, 256, 0, st>>>(a);
    else i8_join_kernel<false><<<blocks, 256, 0, st>>>(a);
    return CNHWC_OK;
}

}  // namespace cnhwc
