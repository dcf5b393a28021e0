// C ABI of the channel-mixing operators: argument checks, workspace sizes, the
// choice of kernels and the launches.  No device code lives here.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <exception>
#include <string>

#include "gated.h"
#include "layernorm.h"

namespace cnhwc {
namespace {

constexpr int64_t kMaxI32 = 0x7fffffff;
constexpr int64_t kMaxRowBytes = int64_t(1) << 61;

int fail(int status, const std::string& why) { return set_error(status, why); }
int ok() { return set_error(CNHWC_OK, ""); }
int bad(const std::string& why) { return set_error(CNHWC_INVALID_ARG, why); }

// No exception may cross the C boundary (a reason string can fail to allocate).
template <typename F>
int guarded(F&& f) {
    try {
        return f();
    } catch (const std::exception&) {
        return CNHWC_INVALID_ARG;
    }
}

int elem_bytes(int dtype) { return dtype == CNHWC_F32 ? 4 : 2; }

std::string num(int64_t v) { return std::to_string(v); }

int check_rows(int64_t rows) {
    if (rows < 0) return bad("rows must be >= 0 (got " + num(rows) + ")");
    return CNHWC_OK;
}

// A row stride: 0 (dense) or at least the row's width; writes the effective one.
int check_stride(int64_t stride, int64_t width, int64_t rows, int es, const char* what, int64_t* out) {
    if (stride != 0 && stride < width)
        return bad(std::string(what) + " must be 0 or >= " + num(width) + " (got " + num(stride) + ")");
    *out = stride ? stride : width;
    if (rows > 0 && *out > kMaxRowBytes / es / rows)
        return bad(std::string(what) + " * rows exceeds the address range");
    return CNHWC_OK;
}

struct View {
    const char* name;
    const void* p;
    int64_t bytes;    // first to last byte
    int align;
};

View rows_view(const char* name, const void* p, int64_t rows, int64_t stride, int64_t width, int es) {
    return {name, p, rows > 0 ? ((rows - 1) * stride + width) * es : 0, es};
}

int check_view(const View& v) {
    if (v.bytes == 0) return CNHWC_OK;   // nothing of it is read or written
    if (!v.p) return bad(std::string(v.name) + " is NULL");
    if (reinterpret_cast<uintptr_t>(v.p) % unsigned(v.align) != 0)
        return fail(CNHWC_MISALIGNED, std::string(v.name) + " is not " + num(v.align) + "-byte aligned");
    return CNHWC_OK;
}

bool overlap(const View& a, const View& b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + uintptr_t(b.bytes) && y < x + uintptr_t(a.bytes);
}

// Every view valid; no written one overlapping any other.
int check_views(const View* in, int nin, const View* out, int nout) {
    for (int i = 0; i < nin; ++i)
        if (int st = check_view(in[i])) return st;
    for (int i = 0; i < nout; ++i)
        if (int st = check_view(out[i])) return st;
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlap(out[i], in[j])) return bad(std::string(out[i].name) + " overlaps " + in[j].name);
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return bad(std::string(out[i].name) + " overlaps " + out[j].name);
    }
    return CNHWC_OK;
}

int launched(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return fail(CNHWC_HIP_ERROR, std::string("launch of ") + what + " failed: " + hipGetErrorString(e));
    return CNHWC_OK;
}

// ---- layer norm -----------------------------------------------------------------

struct Ln {
    int64_t rows, c, xs, ys;
    float eps;
    int dtype, param;
};

int validate(const cnhwc_layernorm_problem* q, Ln* o) {
    if (!q) return bad("problem descriptor is NULL");
    if (q->reserved != 0) return bad("reserved field must be 0");
    if (int st = check_rows(q->rows)) return st;
    if (q->c < 1 || q->c > kMaxI32) return bad("c must be in [1, 2^31) (got " + num(q->c) + ")");
    if (!(q->eps >= 0.0f) || !std::isfinite(q->eps)) return bad("eps must be finite and >= 0");
    if (q->dtype != CNHWC_F16 && q->dtype != CNHWC_BF16 && q->dtype != CNHWC_F32)
        return bad("dtype must be CNHWC_F16, CNHWC_BF16 or CNHWC_F32 (got " + num(q->dtype) + ")");
    if (q->param_dtype != q->dtype && q->param_dtype != CNHWC_F32)
        return bad("param_dtype must be dtype or CNHWC_F32 (got " + num(q->param_dtype) + ")");
    *o = {q->rows, q->c, 0, 0, q->eps, q->dtype, q->param_dtype};
    const int es = elem_bytes(q->dtype);
    if (int st = check_stride(q->x_stride, q->c, q->rows, es, "x_stride", &o->xs)) return st;
    return check_stride(q->y_stride, q->c, q->rows, es, "y_stride", &o->ys);
}

LnArgs ln_args(const Ln& p) {
    LnArgs a;
    std::memset(&a, 0, sizeof a);
    a.rows = p.rows;
    a.x_stride = p.xs;
    a.y_stride = p.ys;
    a.c = int(p.c);
    a.eps = p.eps;
    a.cf = float(p.c);
    return a;
}

int64_t ln_part_bytes(const Ln& p) { return int64_t(layernorm_bwd_blocks(p.dtype, p.rows, p.c)) * 2 * p.c * 4; }

// ---- gated feed-forward ------------------------------------------------------------

struct Gated {
    int64_t rows, c, f, xs, ys;
    int act, dtype;
};

constexpr int64_t kGatedMaxDim = int64_t(1) << 20;

int validate(const cnhwc_gated_problem* q, Gated* o) {
    if (!q) return bad("problem descriptor is NULL");
    if (q->reserved != 0) return bad("reserved field must be 0");
    if (int st = check_rows(q->rows)) return st;
    if (q->rows > kMaxI32) return bad("rows must be < 2^31");
    if (q->c < 1 || q->c > kGatedMaxDim) return bad("c must be in [1, 2^20] (got " + num(q->c) + ")");
    if (q->f < 1 || q->f > kGatedMaxDim) return bad("f must be in [1, 2^20] (got " + num(q->f) + ")");
    if (q->act < CNHWC_ACT_SILU || q->act > CNHWC_ACT_SIGMOID)
        return bad("act must be a CNHWC_ACT_* (got " + num(q->act) + ")");
    if (q->dtype != CNHWC_F16 && q->dtype != CNHWC_BF16)
        return bad("dtype must be CNHWC_F16 or CNHWC_BF16 (got " + num(q->dtype) + ")");
    *o = {q->rows, q->c, q->f, 0, 0, q->act, q->dtype};
    if (int st = check_stride(q->x_stride, q->c, q->rows, 2, "x_stride", &o->xs)) return st;
    if (int st = check_stride(q->y_stride, q->f, q->rows, 2, "y_stride", &o->ys)) return st;
    if (o->xs > 2 * kGatedMaxDim) return bad("x_stride must be <= 2^21");
    if (o->ys > 2 * kGatedMaxDim) return bad("y_stride must be <= 2^21");
    return CNHWC_OK;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tile and the number of reduction splits of one product.  head > 0: the
// first `head` rows run on the large tile in whole rounds of the GPU, the others
// in a second launch on the small one.
struct Shape {
    int tile, splits;
    int64_t tiles_m, tiles_n;
    int64_t head;
};

// Estimated microseconds of each choice, the least one wins.  The rates are
// measured (bf16 normal operands, one product at a time): a 64-deep step of the
// 256 x 256 tile takes 1.45 us (1.55 where an operand is read transposed), of
// two 128 x 128 tiles sharing a CU 0.95 us (1.0), of one alone 0.7 us; a tile's
// start and results cost `fixed` on top (the backward projections read dy and
// write twice the forward's; the large tiles of the weights' gradients all store
// at once, 73 x 3456 -> 5880 in three rounds of two steps 38 us, in five of
// small tiles 30); partial sums move at 6 TB/s, mostly within the
// caches, and the joining launch costs 5 us.  So small tiles win where large
// ones leave CUs idle or the reduction is short, and a reduction is split into
// as many parts as fill the CUs.  For example 50176 x 384 -> 1024: dx on small
// tiles 90 us, on large ones 100; dwg and dwu in 10 splits of the small tile 99 us
// with their join, unsplit 446.
double tile_cost(GatedProduct prod, int end, int tile, int64_t m, int64_t n, int64_t steps, int64_t s) {
    const bool big = tile == kGatedBig, dual = prod == kProj;
    const int64_t tm = ceil_div(m, tile), tn = ceil_div(n, dual ? tile / 2 : tile);
    const double step = big ? (dual ? 1.45 : 1.55) : (dual ? 0.95 : 1.0), step_alone = big ? step : 0.7;
    const double fixed = dual ? (end == kEndBwd ? (big ? 8.0 : 4.5) : (big ? 4.0 : 2.5)) :
                         (big ? (prod == kDw && s == 1 ? 9.0 : 5.0) : 3.5);
    const int64_t slots = big ? kNumCUs : 2 * kNumCUs;
    const int64_t tiles = tm * tn * s, deep = ceil_div(steps, s), rest = tiles % slots;
    double cost = double(tiles / slots) * (double(deep) * step + fixed);
    if (rest) cost += double(deep) * (rest <= kNumCUs ? step_alone : step) + fixed;
    if (s > 1) cost += 5.0 + double(m) * double(dual ? 2 * n : n) * double(s) * 8 / 6.0e6;
    return cost;
}

Shape choose_shape(GatedProduct prod, int end, int64_t m, int64_t n, int64_t steps, double* cost_out = nullptr) {
    const cnhwc_override& ov = current_override();
    const bool dual = prod == kProj;
    auto cost_of = [&](int tile, int64_t rows, int64_t s) { return tile_cost(prod, end, tile, rows, n, steps, s); };
    Shape best = {0, 0, 0, 0, 0};
    double best_cost = 0;
    auto offer = [&](int tile, int64_t s, int64_t head, double cost) {
        if (best.tile != 0 && cost >= best_cost) return;
        best = {tile, int(s), ceil_div(m, tile), ceil_div(n, dual ? tile / 2 : tile), head};
        best_cost = cost;
    };
    const bool forced_tile = ov.tune == kGatedBig || ov.tune == kGatedSmall;
    for (int tile : {kGatedBig, kGatedSmall}) {
        if (forced_tile && ov.tune != tile) continue;
        const int64_t forced = std::min<int64_t>(std::min(ov.split_c, 64), steps);
        const int64_t lo = forced > 0 ? forced : 1, hi = forced > 0 ? forced : 64;
        for (int64_t s = lo; s <= hi && (s == lo || steps / s >= 4); ++s) offer(tile, s, 0, cost_of(tile, m, s));
    }
    if (prod != kDw && !forced_tile && ov.split_c <= 0) {
        // whole rounds of large tiles, the rest on small ones (3 us: one more
        // launch); 50176 x 384 -> 1024 is 6 1/8 rounds
        const int64_t tn = ceil_div(n, dual ? kGatedBig / 2 : kGatedBig);
        const int64_t head = ceil_div(m, kGatedBig) * tn / kNumCUs * kNumCUs / tn * kGatedBig;
        if (head > 0 && head < m)
            offer(kGatedBig, 1, head, cost_of(kGatedBig, head, 1) + 3.0 + cost_of(kGatedSmall, m - head, 1));
    }
    if (cost_out) *cost_out = best_cost;
    return best;
}

// dx and the weights' gradients in one launch of small tiles, a block a tile:
// the splits of both, if that is estimated faster than one after the other
// (which costs a launch more, 4 us, and a second join).  3137 x 385 -> 1027: 57 us
// for the whole backward pass, 69 one after the other.
bool choose_pair(int64_t rows, int64_t c, int64_t fp, double apart, Shape* dx, Shape* dw) {
    const cnhwc_override& ov = current_override();
    if (ov.tune != 0 || ov.split_c != 0) return false;
    const int64_t steps_x = 2 * ceil_div(fp, 64), steps_w = ceil_div(rows, 64);
    const int64_t tn = ceil_div(c, kGatedSmall), mx = ceil_div(rows, kGatedSmall), mw = ceil_div(2 * fp, kGatedSmall);
    if (mx * tn + mw * tn > 2 * kNumCUs) return false;
    double best = apart + 4.0;
    bool found = false;
    for (int64_t sx = 1; sx <= 32 && (sx == 1 || steps_x / sx >= 4); ++sx)
        for (int64_t sw = 1; sw <= 32 && (sw == 1 || steps_w / sw >= 4); ++sw) {
            const int64_t tiles = up(mx * tn * sx, 8) + mw * tn * sw;
            if (tiles > 2 * kNumCUs) break;
            const double step = tiles <= kNumCUs ? 0.7 : 1.0;
            double cost = double(std::max(ceil_div(steps_x, sx), ceil_div(steps_w, sw))) * step + 3.5;
            if (sx > 1 || sw > 1) cost += 5.0;
            if (sx > 1) cost += double(rows) * double(c) * double(sx) * 8 / 6.0e6;
            if (sw > 1) cost += double(2 * fp) * double(c) * double(sw) * 8 / 6.0e6;
            if (cost < best) {
                best = cost;
                found = true;
                *dx = {kGatedSmall, int(sx), mx, tn, 0};
                *dw = {kGatedSmall, int(sw), mw, tn, 0};
            }
        }
    return found;
}

int64_t part_bytes(const Shape& s, int64_t m, int64_t ld) { return s.splits > 1 ? s.splits * m * ld * 4 : 0; }

// Everything one pass needs, with the workspace laid out.
struct GatedPlan {
    bool few_rows = false;            // the projections on the few-rows kernel
    bool pack_x = false, pack_w = false;
    int64_t cp, fp;                   // c, f rounded up to multiples of 8
    Shape proj{}, dx{}, dw{};
    bool pair = false;                // dx and dw in one launch (where both are asked for)
    Shape pair_dx{}, pair_dw{};
    int64_t off_x = 0, off_wg = 0, off_wu = 0, off_dgu = 0, off_part = 0, bytes = 0;
};

GatedPlan plan_gated(const Gated& p, int op, bool x_off, bool w_off) {
    GatedPlan g;
    g.cp = up(p.c, 8);
    g.fp = up(p.f, 8);
    if (p.rows == 0) return g;
    // x also where a row gap would put columns past c next to a row's end:
    // those are masked, so only the 16-byte alignment of every row counts
    g.pack_x = x_off || p.xs % 8 != 0 || p.c % 8 != 0;
    g.pack_w = w_off || p.c % 8 != 0;
    // The few-row kernel while x stays in registers (64 x 2048 -> 8192 21.6 us,
    // on tiles 23.1), up to one 16-row tile of x (16 x 4096 -> 8192 25.2 us, on
    // tiles 29.1; 32 rows 45, on tiles 30) or where the tiles would need a copy of
    // the weights first (64 x 2500 -> 1000 12.5 us, on tiles 24.8), which the
    // backward pass makes in any case.  (By c alone, not by the pointers: the
    // workspace for any pointers has to do for aligned ones.)
    const bool bwd = op != CNHWC_OP_FWD;
    g.few_rows = p.rows <= kGatedFewRows && (p.rows <= 16 || gated_rows_kept(p.rows, p.c, bwd) || (!bwd && p.c % 8 != 0));
    if (g.few_rows && !bwd) {
        g.pack_x = g.pack_w = false;
        return g;
    }
    auto take = [&](int64_t n) {
        const int64_t at = g.bytes;
        g.bytes = up(at + n, 256);
        return at;
    };
    if (g.pack_x) g.off_x = take(p.rows * g.cp * 2);
    if (g.pack_w) {
        g.off_wg = take(p.f * g.cp * 2);
        g.off_wu = take(p.f * g.cp * 2);
    }
    const int64_t csteps = ceil_div(g.cp, 64);
    int64_t part = 0;
    if (!g.few_rows) {
        g.proj = choose_shape(kProj, op == CNHWC_OP_FWD ? kEndFwd : kEndBwd, p.rows, p.f, csteps);
        part = part_bytes(g.proj, p.rows, 2 * g.fp);
    }
    if (op != CNHWC_OP_FWD) {
        g.off_dgu = take(p.rows * 2 * g.fp * 2);
        double cx = 0, cw = 0;
        g.dx = choose_shape(kDx, kEndFwd, p.rows, p.c, 2 * ceil_div(g.fp, 64), &cx);
        g.dw = choose_shape(kDw, kEndFwd, 2 * g.fp, p.c, ceil_div(p.rows, 64), &cw);
        g.pair = choose_pair(p.rows, p.c, g.fp, cx + cw, &g.pair_dx, &g.pair_dw);
        const int64_t ld = up(p.c, 4);
        part = std::max(part, std::max(part_bytes(g.dx, p.rows, ld), part_bytes(g.dw, 2 * g.fp, ld)));
        if (g.pair)
            part = std::max(part, up(part_bytes(g.pair_dx, p.rows, ld), 256) + part_bytes(g.pair_dw, 2 * g.fp, ld));
    }
    if (part) g.off_part = take(part);
    return g;
}

bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

const char* dt_name(int dtype) { return dtype == CNHWC_F16 ? "f16" : "bf16"; }

std::string shape_name(const char* what, int dtype, const Shape& s) {
    std::string n = std::string("gated_") + what + "_" + dt_name(dtype) + "_t" + num(s.tile);
    if (s.head) n += "+t" + num(kGatedSmall);
    if (s.splits > 1) n += "_split" + num(s.splits) + "+join";
    return n;
}

// One product on the tiled kernel, and the join of its splits.
int run_product(int dtype, GatedProduct prod, const Shape& s, GatedArgs a, char* ws, int64_t off_part,
                hipStream_t st) {
    if (s.tiles_m * s.tiles_n > kMaxI32 / s.splits)
        return fail(CNHWC_UNSUPPORTED, "the problem needs more than 2^31 tiles");
    a.splits = s.splits;
    a.part = s.splits > 1 ? reinterpret_cast<float*>(ws + off_part) : nullptr;
    auto run = [&](int tile) -> int {
        a.tiles_m = int(ceil_div(a.m, tile));
        a.tiles_n = int(ceil_div(a.n, prod == kProj ? tile / 2 : tile));
        const int rc = launch_gated_product(dtype, prod, tile, a, st);
        if (rc) return fail(rc, "launcher of the gated product refused it");
        return launched("gated_gemm");
    };
    const int64_t m = a.m;
    if (s.head) a.m = s.head;
    int rc = run(s.tile);
    if (rc) return rc;
    if (s.head) {
        // the rows behind
        a.m = m - s.head;
        a.a = static_cast<const char*>(a.a) + s.head * a.lda * 2;
        if (a.y) a.y = static_cast<char*>(a.y) + s.head * a.ldy * 2;
        if (a.dy) a.dy = static_cast<const char*>(a.dy) + s.head * a.lddy * 2;
        if (a.dgu) a.dgu = static_cast<char*>(a.dgu) + s.head * 2 * a.fp * 2;
        return run(kGatedSmall);
    }
    if (s.splits > 1) {
        launch_gated_reduce(dtype, prod, a, st);
        if ((rc = launched("gated_join"))) return rc;
    }
    return CNHWC_OK;
}

int run_gated(const cnhwc_gated_problem* prob, int op, const void* dy, const void* x, const void* wg, const void* wu,
              void* y, void* dx, void* dwg, void* dwu, void* ws, size_t ws_bytes, void* stream) {
    Gated p;
    int rc = validate(prob, &p);
    if (rc) return rc;
    const bool bwd = op != CNHWC_OP_FWD;
    if (bwd) {
        if ((dwg == nullptr) != (dwu == nullptr)) return bad("dwg and dwu must both be given or both be NULL");
        if (!dx && !dwg) return bad("dx, dwg and dwu are all NULL");
    }
    View in[4], out[4];
    int nin = 0, nout = 0;
    in[nin++] = rows_view("x", x, p.rows, p.xs, p.c, 2);
    in[nin++] = rows_view("wg", wg, p.f, p.c, p.c, 2);
    in[nin++] = rows_view("wu", wu, p.f, p.c, p.c, 2);
    if (bwd) in[nin++] = rows_view("dy", dy, p.rows, p.ys, p.f, 2);
    if (!bwd) out[nout++] = rows_view("y", y, p.rows, p.ys, p.f, 2);
    if (dx) out[nout++] = rows_view("dx", dx, p.rows, p.xs, p.c, 2);
    if (dwg) {
        out[nout++] = rows_view("dwg", dwg, p.f, p.c, p.c, 2);
        out[nout++] = rows_view("dwu", dwu, p.f, p.c, p.c, 2);
    }
    if ((rc = check_views(in, nin, out, nout))) return rc;
    const GatedPlan g = plan_gated(p, op, off16(x), off16(wg) || off16(wu));
    if (g.bytes > 0) {
        const View wv = {"workspace", ws, g.bytes, 16};
        if ((rc = check_view(wv))) return rc;
        if (int64_t(ws_bytes) < g.bytes)
            return fail(CNHWC_WORKSPACE_TOO_SMALL,
                        "workspace needs " + num(g.bytes) + " bytes, got " + std::to_string(ws_bytes));
        for (int i = 0; i < nin; ++i)
            if (overlap(wv, in[i])) return bad(std::string("workspace overlaps ") + in[i].name);
        for (int i = 0; i < nout; ++i)
            if (overlap(wv, out[i])) return bad(std::string("workspace overlaps ") + out[i].name);
    }
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();   // a stale error from earlier work must not be blamed on this call
    if (p.rows == 0) {
        if (dwg) {
            launch_gated_zero(dwg, p.f * p.c, st);   // sums over no rows
            if ((rc = launched("gated_zero"))) return rc;
            launch_gated_zero(dwu, p.f * p.c, st);
            if ((rc = launched("gated_zero"))) return rc;
        }
        return ok();
    }
    if (g.few_rows) {
        GatedRowsArgs a = {x, wg, wu, y, p.rows, p.c, p.f, p.xs, p.ys, p.act, dy,
                           bwd ? static_cast<char*>(ws) + g.off_dgu : nullptr, p.ys, g.fp};
        if ((rc = launch_gated_rows(p.dtype, a, st))) return fail(rc, "launcher of the few-row product refused it");
        if ((rc = launched("gated_rows"))) return rc;
        if (!bwd) return ok();
    }
    char* w = static_cast<char*>(ws);
    const void *xo = x, *go = wg, *uo = wu;
    int64_t ldx = p.xs;
    GatedPack pack[3];
    int packs = 0;
    if (g.pack_x) {
        pack[packs++] = {x, w + g.off_x, p.xs, p.rows};
        xo = w + g.off_x;
        ldx = g.cp;
    }
    if (g.pack_w) {
        pack[packs++] = {wg, w + g.off_wg, p.c, p.f};
        pack[packs++] = {wu, w + g.off_wu, p.c, p.f};
        go = w + g.off_wg;
        uo = w + g.off_wu;
    }
    if (packs) {
        launch_gated_pack(pack, packs, p.c, g.cp, st);
        if ((rc = launched("gated_pack"))) return rc;
    }
    GatedArgs a;
    std::memset(&a, 0, sizeof a);
    a.a = xo;
    a.b0 = go;
    a.b1 = uo;
    a.lda = ldx;
    a.ldb = g.cp;
    a.m = p.rows;
    a.n = p.f;
    a.k = g.cp;
    a.segs = 1;
    a.steps_seg = int(ceil_div(g.cp, 64));
    a.act = p.act;
    a.end = bwd ? kEndBwd : kEndFwd;
    a.f = p.f;
    a.fp = g.fp;
    a.y = y;
    a.ldy = p.ys;
    a.dy = dy;
    a.lddy = p.ys;
    a.dgu = bwd ? w + g.off_dgu : nullptr;
    a.part_ld = 2 * g.fp;
    a.wide = p.f % 8 == 0 && p.ys % 8 == 0 && !off16(bwd ? dy : y);
    if (!g.few_rows && (rc = run_product(p.dtype, kProj, g.proj, a, w, g.off_part, st))) return rc;
    GatedArgs ax = a, aw = a;
    ax.a = aw.a = w + g.off_dgu;
    ax.lda = aw.lda = 2 * g.fp;
    ax.n = aw.n = p.c;
    ax.nb = aw.nb = g.cp;
    ax.part_ld = aw.part_ld = up(p.c, 4);
    // dx = [dg | du] [wg ; wu]
    ax.k = g.fp;
    ax.segs = 2;
    ax.steps_seg = int(ceil_div(g.fp, 64));
    ax.y = dx;
    ax.ldy = p.xs;
    ax.wide = p.c % 8 == 0 && p.xs % 8 == 0 && !off16(dx);
    // [dwg ; dwu] = [dg | du]^T x
    aw.b0 = xo;
    aw.b1 = nullptr;
    aw.ldb = ldx;
    aw.m = 2 * g.fp;
    aw.k = p.rows;
    aw.steps_seg = int(ceil_div(p.rows, 64));
    aw.y = nullptr;
    aw.dwg = dwg;
    aw.dwu = dwu;
    aw.wide = p.c % 8 == 0 && !off16(dwg) && !off16(dwu);
    if (dx && dwg && g.pair) {
        auto set = [](GatedArgs& v, const Shape& s, float* part) {
            v.tiles_m = int(s.tiles_m);
            v.tiles_n = int(s.tiles_n);
            v.splits = s.splits;
            v.part = s.splits > 1 ? part : nullptr;
        };
        char* part = w + g.off_part;
        set(ax, g.pair_dx, reinterpret_cast<float*>(part));
        set(aw, g.pair_dw,
            reinterpret_cast<float*>(part + up(part_bytes(g.pair_dx, p.rows, ax.part_ld), 256)));
        if ((rc = launch_gated_pair(p.dtype, ax, aw, st))) return fail(rc, "launcher of the gated gradients refused them");
        if ((rc = launched("gated_pair"))) return rc;
        const bool sx = ax.splits > 1, sw = aw.splits > 1;
        if (sx && sw) launch_gated_pair_reduce(p.dtype, ax, aw, st);
        else if (sx) launch_gated_reduce(p.dtype, kDx, ax, st);
        else if (sw) launch_gated_reduce(p.dtype, kDw, aw, st);
        if ((sx || sw) && (rc = launched("gated_join"))) return rc;
        return ok();
    }
    if (dx && (rc = run_product(p.dtype, kDx, g.dx, ax, w, g.off_part, st))) return rc;
    if (dwg && (rc = run_product(p.dtype, kDw, g.dw, aw, w, g.off_part, st))) return rc;
    return ok();
}

}  // namespace
}  // namespace cnhwc

using namespace cnhwc;

extern "C" {

int cnhwc_layernorm_fwd(const cnhwc_layernorm_problem* prob, const void* x, const void* gamma, const void* beta,
                        void* y, float* mean, float* rstd, void* hip_stream) {
    return guarded([&]() -> int {
        Ln p;
        int rc = validate(prob, &p);
        if (rc) return rc;
        const int es = elem_bytes(p.dtype), ps = elem_bytes(p.param);
        View in[3] = {rows_view("x", x, p.rows, p.xs, p.c, es)}, out[3];
        int nin = 1, nout = 0;
        if (gamma) in[nin++] = {"gamma", gamma, p.c * ps, ps};
        if (beta) in[nin++] = {"beta", beta, p.c * ps, ps};
        out[nout++] = rows_view("y", y, p.rows, p.ys, p.c, es);
        if (mean) out[nout++] = {"mean", mean, p.rows * 4, 4};
        if (rstd) out[nout++] = {"rstd", rstd, p.rows * 4, 4};
        if ((rc = check_views(in, nin, out, nout))) return rc;
        if (p.rows == 0) return ok();
        LnArgs a = ln_args(p);
        a.x = x;
        a.gamma = gamma;
        a.beta = beta;
        a.y = y;
        a.mean = mean;
        a.rstd = rstd;
        (void)hipGetLastError();
        launch_layernorm_fwd(p.dtype, p.param, a, reinterpret_cast<hipStream_t>(hip_stream));
        if ((rc = launched("layernorm_fwd"))) return rc;
        return ok();
    });
}

int cnhwc_layernorm_workspace_size(const cnhwc_layernorm_problem* prob, size_t* bytes) {
    return guarded([&]() -> int {
        Ln p;
        if (int rc = validate(prob, &p)) return rc;
        if (bytes) *bytes = size_t(ln_part_bytes(p));
        return ok();
    });
}

int cnhwc_layernorm_bwd(const cnhwc_layernorm_problem* prob, const void* dy, const void* x, const void* gamma,
                        const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta, void* ws,
                        size_t ws_bytes, void* hip_stream) {
    return guarded([&]() -> int {
        Ln p;
        int rc = validate(prob, &p);
        if (rc) return rc;
        if (!dx && !dgamma && !dbeta) return bad("dx, dgamma and dbeta are all NULL");
        const int es = elem_bytes(p.dtype), ps = elem_bytes(p.param);
        View in[5] = {rows_view("dy", dy, p.rows, p.ys, p.c, es), rows_view("x", x, p.rows, p.xs, p.c, es),
                      {"mean", mean, p.rows * 4, 4}, {"rstd", rstd, p.rows * 4, 4}};
        View out[4];
        int nin = 4, nout = 0;
        if (gamma) in[nin++] = {"gamma", gamma, p.c * ps, ps};
        if (dx) out[nout++] = rows_view("dx", dx, p.rows, p.xs, p.c, es);
        if (dgamma) out[nout++] = {"dgamma", dgamma, p.c * ps, ps};
        if (dbeta) out[nout++] = {"dbeta", dbeta, p.c * ps, ps};
        const bool cols = dgamma || dbeta;
        const int64_t need = cols ? ln_part_bytes(p) : 0;
        if (need > 0) out[nout++] = {"workspace", ws, need, 16};
        if ((rc = check_views(in, nin, out, nout))) return rc;
        if (int64_t(ws_bytes) < need)
            return fail(CNHWC_WORKSPACE_TOO_SMALL,
                        "workspace needs " + num(need) + " bytes, got " + std::to_string(ws_bytes));
        hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
        (void)hipGetLastError();
        const int blocks = layernorm_bwd_blocks(p.dtype, p.rows, p.c);
        if (p.rows > 0) {
            LnArgs a = ln_args(p);
            a.x = x;
            a.dy = dy;
            a.gamma = gamma;
            a.mean = const_cast<float*>(mean);
            a.rstd = const_cast<float*>(rstd);
            a.y = dx;
            a.part = cols ? static_cast<float*>(ws) : nullptr;
            launch_layernorm_bwd(p.dtype, p.param, a, blocks, st);
            if ((rc = launched("layernorm_bwd"))) return rc;
        }
        if (cols) {
            launch_layernorm_reduce(p.param, static_cast<const float*>(ws), blocks, p.c, dgamma, dbeta, st);
            if ((rc = launched("layernorm_reduce"))) return rc;
        }
        return ok();
    });
}

int cnhwc_gated_workspace_size(const cnhwc_gated_problem* prob, int op, int unaligned, size_t* bytes) {
    return guarded([&]() -> int {
        Gated p;
        if (int rc = validate(prob, &p)) return rc;
        if (op != CNHWC_OP_FWD && op != CNHWC_OP_DGRAD)
            return bad("op must be CNHWC_OP_FWD (1) or CNHWC_OP_DGRAD (2, the whole backward pass)");
        if (bytes) *bytes = size_t(plan_gated(p, op, unaligned != 0, unaligned != 0).bytes);
        return ok();
    });
}

int cnhwc_gated_plan(const cnhwc_gated_problem* prob, int op, char* name, size_t cap) {
    return guarded([&]() -> int {
        Gated p;
        if (int rc = validate(prob, &p)) return rc;
        if (op != CNHWC_OP_FWD && op != CNHWC_OP_DGRAD)
            return bad("op must be CNHWC_OP_FWD (1) or CNHWC_OP_DGRAD (2, the whole backward pass)");
        const GatedPlan g = plan_gated(p, op, false, false);
        std::string s;
        if (p.rows == 0) s = "none";
        else {
            if (g.pack_x || g.pack_w) s = "pack ";
            s += g.few_rows ? std::string("gated_rows_") + dt_name(p.dtype) : shape_name("proj", p.dtype, g.proj);
            if (op != CNHWC_OP_FWD) {
                const char* pair = g.pair ? "pair:" : "";
                s += std::string(" ") + pair + shape_name("dx", p.dtype, g.pair ? g.pair_dx : g.dx);
                s += std::string(" ") + pair + shape_name("dw", p.dtype, g.pair ? g.pair_dw : g.dw);
            }
        }
        if (name && cap > 0) {
            std::strncpy(name, s.c_str(), cap - 1);
            name[cap - 1] = '\0';
        }
        return ok();
    });
}

int cnhwc_gated_fwd(const cnhwc_gated_problem* prob, const void* x, const void* wg, const void* wu, void* y, void* ws,
                    size_t ws_bytes, void* hip_stream) {
    return guarded([&]() -> int {
        return run_gated(prob, CNHWC_OP_FWD, nullptr, x, wg, wu, y, nullptr, nullptr, nullptr, ws, ws_bytes,
                         hip_stream);
    });
}

int cnhwc_gated_bwd(const cnhwc_gated_problem* prob, const void* dy, const void* x, const void* wg, const void* wu,
                    void* dx, void* dwg, void* dwu, void* ws, size_t ws_bytes, void* hip_stream) {
    return guarded([&]() -> int {
        return run_gated(prob, CNHWC_OP_DGRAD, dy, x, wg, wu, nullptr, dx, dwg, dwu, ws, ws_bytes, hip_stream);
    });
}

int cnhwc_dropout(const cnhwc_dropout_problem* prob, const void* x, const void* residual, void* y,
                  const uint64_t* device_offset, void* hip_stream) {
    return guarded([&]() -> int {
        if (!prob) return bad("problem descriptor is NULL");
        const cnhwc_dropout_problem& q = *prob;
        if (q.reserved != 0) return bad("reserved field must be 0");
        int rc = check_rows(q.rows);
        if (rc) return rc;
        if (q.c < 1 || q.c > kMaxI32) return bad("c must be in [1, 2^31) (got " + num(q.c) + ")");
        if (!(q.p >= 0.0 && q.p <= 1.0)) return bad("p must be in [0, 1]");
        if (q.dtype != CNHWC_F16 && q.dtype != CNHWC_BF16 && q.dtype != CNHWC_F32)
            return bad("dtype must be CNHWC_F16, CNHWC_BF16 or CNHWC_F32 (got " + num(q.dtype) + ")");
        const int es = elem_bytes(q.dtype);
        DropArgs a;
        std::memset(&a, 0, sizeof a);
        if ((rc = check_stride(q.x_stride, q.c, q.rows, es, "x_stride", &a.x_stride))) return rc;
        if ((rc = check_stride(q.residual_stride, q.c, q.rows, es, "residual_stride", &a.res_stride))) return rc;
        if ((rc = check_stride(q.y_stride, q.c, q.rows, es, "y_stride", &a.y_stride))) return rc;
        View in[3] = {rows_view("x", x, q.rows, a.x_stride, q.c, es)};
        int nin = 1;
        if (residual) in[nin++] = rows_view("residual", residual, q.rows, a.res_stride, q.c, es);
        const View yv = rows_view("y", y, q.rows, a.y_stride, q.c, es);
        if (device_offset) in[nin++] = {"device_offset", device_offset, 8, 8};
        for (int i = 0; i < nin; ++i)
            if ((rc = check_view(in[i]))) return rc;
        if ((rc = check_view(yv))) return rc;
        for (int i = 0; i < nin; ++i) {
            // in place: each element is read by the thread that writes it
            const bool same = (i == 0 && y == x && a.y_stride == a.x_stride) ||
                              (i == 1 && residual && y == residual && a.y_stride == a.res_stride);
            if (!same && overlap(yv, in[i])) return bad(std::string("y overlaps ") + in[i].name);
        }
        if (q.rows == 0) return ok();
        a.x = x;
        a.residual = residual;
        a.y = y;
        a.device_offset = device_offset;
        a.n = q.rows * q.c;
        a.c = q.c;
        a.seed = q.seed;
        a.offset = q.offset;
        a.threshold = uint64_t(std::nearbyint(q.p * 4294967296.0));
        a.scale = q.p < 1.0 ? float(1.0 / (1.0 - q.p)) : 0.0f;
        a.flat = a.x_stride == q.c && a.y_stride == q.c && (!residual || a.res_stride == q.c);
        (void)hipGetLastError();
        launch_dropout(q.dtype, a, reinterpret_cast<hipStream_t>(hip_stream));
        if ((rc = launched("dropout"))) return rc;
        return ok();
    });
}

}  // extern "C"
