// C ABI of the group norm: argument checks, workspace sizes, the split into
// blocks and the launches.  No device code lives here.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <iterator>
#include <string>

#include "groupnorm.h"
#include "host_checks.h"

namespace cnhwc {

// The span of groups that one block can hold for a sample: as narrow as its rows
// stay at least 64 bytes and nearly whole vectors, for the most blocks.  False where
// no span fits.
static bool gn_resident(GnShape& s, int64_t v, int64_t n, int64_t pixels, int64_t each, int64_t groups, bool bwd) {
    const int* const nvs = bwd ? kGnBwd : kGnFwd;
    const int variants = bwd ? std::size(kGnBwd) : std::size(kGnFwd);
    auto most = [&](int nv) -> int64_t { return bwd ? kGnBwdThreads : gn_fwd_threads(nv); };
    int64_t best = -1;
    for (int64_t per = 1; per <= groups; ++per) {
        const int64_t vecs = ceil_div(per * each, v), spans = ceil_div(groups, per);
        if (vecs > 1024) break;
        // (also the last span, which may not be full)
        const bool whole = (groups - (spans - 1) * per) * each >= v;
        const bool narrow = vecs < 4 && per < groups, plain = whole && (bwd || each >= v);
        if (!whole && narrow) continue;
        // lanes' work that is done twice, and idle ones of a last span that is not full, in percent; rows of
        // under 48 bytes count as half idle, of under 64 as a tenth
        const int64_t score = (spans * vecs * v - groups * each) * 100 / (groups * each) + (narrow ? vecs < 3 ? 50 : 10 : 0);
        if (best >= 0 && score >= best) continue;
        // few blocks: the most threads; many: four vectors a thread, so that a CU has several at work
        int nv = 0;
        for (int i = 0; i < variants; ++i) {
            if (!plain && gn_plain_only(nvs[i])) continue;
            const int64_t ty = ceil_div(pixels, nvs[i]);
            if (ty * vecs > most(nvs[i])) continue;
            nv = nvs[i];
            if (nv >= 4 || n * spans < 2 * kNumCUs) break;
        }
        if (nv == 0) continue;
        best = score;
        s.nv = nv;
        s.whole = whole;
        s.per = int(per);
        s.vecs = int(vecs);
        s.ty = int(ceil_div(pixels, nv));
        if (best < 8) break;
    }
    if (best < 0) return false;
    // Estimated microseconds of both ways.  Resident blocks load, reduce and store in
    // step: a round of them costs its latency and by what a CU's waves hold (the
    // backward pass is bound by its arithmetic); two launches cost by the bytes
    // they read twice.  Measured with 32 groups and silu, resident and in two
    // launches: forward 16 images of 56 x 56 x 384 25.6 and 33 us, x 512 30 and 36, 64
    // of 14 x 14 x 1024 18 and 20; backward 45 and 58; two images of 56 x 56 x 384 35
    // and 19, 64 of 28 x 28 x 256 44 and 34.
    const int64_t blocks = n * ceil_div(groups, s.per), waves = ceil_div(int64_t(s.ty) * s.vecs, 64);
    const int64_t room = bwd ? 512 / (88 + 8 * s.nv) * 4 : std::min(512 / (56 + 4 * s.nv), 8) * 4;
    const int64_t per_cu = std::min(std::max<int64_t>(1, room / waves), ceil_div(blocks, kNumCUs));
    const double rounds = std::max(1.0, double(blocks) / double(kNumCUs * per_cu)), held = double(s.nv) * double(per_cu * waves);
    const double one = rounds * (bwd ? 7.0 + 0.24 * held : 4.0 + 0.11 * held);
    const double megabytes = double(n) * double(pixels) * double(groups * each) * (16.0 / double(v)) / 1e6;
    return one < (bwd ? 11.0 + 1.1 * megabytes : 10.0 + 0.6 * megabytes);
}

GnShape gn_shape(int dtype, int64_t n, int64_t pixels, int64_t c, int64_t groups, bool bwd) {
    const int64_t v = dtype == CNHWC_F32 ? 4 : 8, each = c / groups, widest = kGnThreads * v;
    GnShape s;
    std::memset(&s, 0, sizeof s);
    s.pieces = 1;
    GnShape one = s;
    if (current_override().tune != 1 && gn_resident(one, v, n, pixels, each, groups, bwd)) {
        s = one;
        s.span = int(s.per * each);
        s.spans = int(ceil_div(groups, s.per));
        s.chunk = int(pixels);
        s.chunks = 1;
    } else {
        s.pieces = int(ceil_div(each, widest));
        s.per = s.pieces > 1 ? 1 : int(std::min(groups, widest / each));
        // narrower spans while there are few blocks and a span's row stays 128 bytes
        if (s.pieces == 1) {
            auto blocks = [&](int64_t per) {
                const int64_t vecs = ceil_div(per * each, v), ty = std::max<int64_t>(1, kGnThreads / vecs);
                return n * ceil_div(groups, per) * ceil_div(pixels, ty * 8);
            };
            while (s.per > 1 && blocks(s.per) < 2 * kNumCUs && (s.per + 1) / 2 * each * (16 / v) >= 128)
                s.per = (s.per + 1) / 2;
        }
        s.span = int(s.pieces > 1 ? up(ceil_div(each, s.pieces), v) : s.per * each);
        s.pieces = s.pieces > 1 ? int(ceil_div(each, s.span)) : 1;
        s.spans = int(s.pieces > 1 ? groups * s.pieces : ceil_div(groups, s.per));
        s.vecs = int(ceil_div(s.span, v));
        s.whole = (s.pieces > 1 ? each - (s.pieces - 1) * int64_t(s.span) : (groups - (s.spans - 1) * int64_t(s.per)) * each) >= v;
        // pixels at a time: the count that leaves the fewest threads of the block's waves idle
        s.ty = 1;
        double best = 0;
        for (int64_t ty = 1; ty * s.vecs <= kGnThreads && ty <= std::max<int64_t>(pixels, 1); ++ty) {
            const int64_t t = ty * s.vecs;
            const double used = double(t) / double(up(t, 64)) * std::min(1.0, double(t) / (kGnThreads / 2));
            if (used >= best) {
                best = used;
                s.ty = int(ty);
            }
        }
        // Chunks: blocks in whole rounds of the GPU (12 waves a CU), a block's start and
        // its sums counted as six pixels a thread; at most 256 chunks, whose parts
        // every block of the second launch joins.
        const int64_t waves = ceil_div(int64_t(s.ty) * s.vecs, 64), slots = kNumCUs * (12 / waves);
        const int64_t steps = ceil_div(pixels, s.ty);
        int64_t chunks = 1;
        double least = 0;
        for (int64_t deep = 4; deep <= std::max<int64_t>(steps, 4); deep += 1 + deep / 16) {
            const int64_t k = ceil_div(steps, deep);
            if (k > 256) continue;
            const double cost = double(ceil_div(n * s.spans * k, slots)) * double(deep + 6);
            if (least == 0 || cost < least) {
                least = cost;
                chunks = k;
            }
        }
        s.chunk = int(up(ceil_div(pixels, chunks), s.ty));
        s.chunks = int(ceil_div(pixels, s.chunk));
    }
    s.threads = int(up(int64_t(s.ty) * s.vecs, 64));
    s.d_spans = make_fastdiv(uint32_t(s.spans));
    s.d_vecs = make_fastdiv(uint32_t(s.vecs));
    s.d_chunks = make_fastdiv(uint32_t(s.chunks));
    s.d_each = make_fastdiv(uint32_t(each));
    s.d_pieces = make_fastdiv(uint32_t(s.pieces));
    s.d_ty = make_fastdiv(uint32_t(s.ty));
    return s;
}

namespace {

struct Gn {
    int64_t n, pixels, c, rows, xs, ys;
    float eps;
    int groups, act, dtype, param;
};

int validate(const cnhwc_groupnorm_problem* q, Gn* o) {
    if (!q) return bad("problem descriptor is NULL");
    if (q->reserved != 0) return bad("reserved field must be 0");
    if (q->n < 0) return bad("n must be >= 0 (got " + num(q->n) + ")");
    if (q->pixels < 1) return bad("pixels must be >= 1 (got " + num(q->pixels) + ")");
    if (q->n > kMaxI32 / q->pixels) return bad("n * pixels must be < 2^31");
    if (q->pixels > kMaxI32 / 2) return bad("pixels must be < 2^30");
    if (q->c < 1 || q->c > int64_t(1) << 20) return bad("c must be in [1, 2^20] (got " + num(q->c) + ")");
    if (q->groups < 1 || q->c % q->groups != 0)
        return bad("groups must divide c (got " + num(q->groups) + " groups of " + num(q->c) + " channels)");
    if (!(q->eps >= 0.0f) || !std::isfinite(q->eps)) return bad("eps must be finite and >= 0");
    if (q->act != CNHWC_ACT_NONE && (q->act < CNHWC_ACT_SILU || q->act > CNHWC_ACT_SIGMOID))
        return bad("act must be CNHWC_ACT_NONE or a CNHWC_ACT_* (got " + num(q->act) + ")");
    if (q->dtype != CNHWC_F16 && q->dtype != CNHWC_BF16 && q->dtype != CNHWC_F32)
        return bad("dtype must be CNHWC_F16, CNHWC_BF16 or CNHWC_F32 (got " + num(q->dtype) + ")");
    if (q->param_dtype != q->dtype && q->param_dtype != CNHWC_F32)
        return bad("param_dtype must be dtype or CNHWC_F32 (got " + num(q->param_dtype) + ")");
    *o = {q->n, q->pixels, q->c, q->n * q->pixels, 0, 0, q->eps, q->groups, q->act, q->dtype, q->param_dtype};
    const int es = elem_bytes(q->dtype);
    if (int st = check_stride(q->x_stride, q->c, o->rows, es, "x_stride", &o->xs)) return st;
    return check_stride(q->y_stride, q->c, o->rows, es, "y_stride", &o->ys);
}

struct GnPlan {
    GnShape s;
    int64_t part_sample, cols, bytes;   // bytes of a sample's parts; where the column sums start
};

int plan(const Gn& p, bool bwd, GnPlan* g) {
    std::memset(g, 0, sizeof *g);
    if (p.n == 0) return CNHWC_OK;
    g->s = gn_shape(p.dtype, p.n, p.pixels, p.c, p.groups, bwd);
    const int64_t blocks = p.n * g->s.chunks;
    if (blocks > kMaxI32 / g->s.spans) return fail(CNHWC_UNSUPPORTED, "the problem needs more than 2^31 blocks");
    g->part_sample = g->s.nv ? 0 : g->s.chunks * p.groups * g->s.pieces * int64_t(8);
    g->bytes = g->cols = up(p.n * g->part_sample, 256);
    if (bwd) g->bytes += blocks * 2 * p.c * 4;
    return CNHWC_OK;
}

// launch(first sample, samples): in as many launches as it takes, for one has less than 2^32
// threads.
template <typename F>
int by_samples(const Gn& p, const GnPlan& g, const char* what, F&& launch) {
    const int64_t most = std::max<int64_t>(1, ((int64_t(1) << 32) - 1) / (int64_t(g.s.spans) * g.s.chunks * g.s.threads));
    for (int64_t n0 = 0; n0 < p.n; n0 += most) {
        launch(n0, std::min(most, p.n - n0));
        if (int rc = launched(what)) return rc;
    }
    return CNHWC_OK;
}
template <typename T>
T* moved(T* p, int64_t bytes) {
    return p ? reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + uintptr_t(bytes)) : nullptr;
}

GnArgs gn_args(const Gn& p, const GnPlan& g) {
    GnArgs a;
    std::memset(&a, 0, sizeof a);
    a.n = p.n;
    a.x_stride = p.xs;
    a.y_stride = p.ys;
    a.pixels = int(p.pixels);
    a.c = int(p.c);
    a.groups = p.groups;
    a.each = int(p.c / p.groups);
    a.act = p.act;
    a.p32 = p.param == CNHWC_F32;
    a.eps = p.eps;
    a.s = g.s;
    return a;
}

}  // namespace
}  // namespace cnhwc

using namespace cnhwc;

extern "C" {

int cnhwc_groupnorm_workspace_size(const cnhwc_groupnorm_problem* prob, int op, size_t* bytes) {
    return guarded([&]() -> int {
        Gn p;
        int rc = validate(prob, &p);
        if (rc) return rc;
        if (op != CNHWC_OP_FWD && op != CNHWC_OP_DGRAD) return bad("op must be CNHWC_OP_FWD or CNHWC_OP_DGRAD");
        if (!bytes) return bad("bytes is NULL");
        GnPlan g;
        if ((rc = plan(p, op != CNHWC_OP_FWD, &g))) return rc;
        *bytes = size_t(g.bytes);
        return ok();
    });
}

int cnhwc_groupnorm_fwd(const cnhwc_groupnorm_problem* prob, const void* x, const void* gamma, const void* beta,
                        void* y, float* mean, float* rstd, void* ws, size_t ws_bytes, void* hip_stream) {
    return guarded([&]() -> int {
        Gn p;
        int rc = validate(prob, &p);
        if (rc) return rc;
        const int es = elem_bytes(p.dtype), ps = elem_bytes(p.param);
        View in[3] = {rows_view("x", x, p.rows, p.xs, p.c, es)}, out[3];
        int nin = 1, nout = 0;
        if (gamma) in[nin++] = {"gamma", gamma, p.c * ps, ps};
        if (beta) in[nin++] = {"beta", beta, p.c * ps, ps};
        out[nout++] = rows_view("y", y, p.rows, p.ys, p.c, es);
        if (mean) out[nout++] = {"mean", mean, p.n * p.groups * 4, 4};
        if (rstd) out[nout++] = {"rstd", rstd, p.n * p.groups * 4, 4};
        if ((rc = check_views(in, nin, out, nout))) return rc;
        GnPlan g;
        if ((rc = plan(p, false, &g))) return rc;
        if ((rc = check_ws(ws, ws_bytes, g.bytes, in, nin, out, nout))) return rc;
        if (p.n == 0) return ok();
        GnArgs a = gn_args(p, g);
        a.x = x;
        a.gamma = gamma;
        a.beta = beta;
        a.y = y;
        a.mean = mean;
        a.rstd = rstd;
        a.part = static_cast<float2*>(ws);
        (void)hipGetLastError();
        rc = by_samples(p, g, "groupnorm_fwd", [&](int64_t n0, int64_t n) {
            GnArgs b = a;
            b.n = n;
            b.x = moved(a.x, n0 * p.pixels * p.xs * es);
            b.y = moved(a.y, n0 * p.pixels * p.ys * es);
            b.mean = moved(a.mean, n0 * p.groups * 4);
            b.rstd = moved(a.rstd, n0 * p.groups * 4);
            b.part = moved(a.part, n0 * g.part_sample);
            launch_groupnorm_fwd(p.dtype, b, reinterpret_cast<hipStream_t>(hip_stream));
        });
        return rc ? rc : ok();
    });
}

int cnhwc_groupnorm_bwd(const cnhwc_groupnorm_problem* prob, const void* dy, const void* x, const void* gamma,
                        const void* beta, const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta,
                        void* ws, size_t ws_bytes, void* hip_stream) {
    return guarded([&]() -> int {
        Gn p;
        int rc = validate(prob, &p);
        if (rc) return rc;
        if (!dx && !dgamma && !dbeta) return bad("dx, dgamma and dbeta are all NULL");
        const int es = elem_bytes(p.dtype), ps = elem_bytes(p.param);
        View in[6], out[3];
        int nin = 0, nout = 0;
        in[nin++] = rows_view("dy", dy, p.rows, p.ys, p.c, es);
        in[nin++] = rows_view("x", x, p.rows, p.xs, p.c, es);
        in[nin++] = {"mean", mean, p.n * p.groups * 4, 4};
        in[nin++] = {"rstd", rstd, p.n * p.groups * 4, 4};
        if (gamma) in[nin++] = {"gamma", gamma, p.c * ps, ps};
        if (beta) in[nin++] = {"beta", beta, p.c * ps, ps};
        if (dx) out[nout++] = rows_view("dx", dx, p.rows, p.xs, p.c, es);
        if (dgamma) out[nout++] = {"dgamma", dgamma, p.c * ps, ps};
        if (dbeta) out[nout++] = {"dbeta", dbeta, p.c * ps, ps};
        if ((rc = check_views(in, nin, out, nout))) return rc;
        GnPlan g;
        if ((rc = plan(p, true, &g))) return rc;
        if ((rc = check_ws(ws, ws_bytes, g.bytes, in, nin, out, nout))) return rc;
        hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
        (void)hipGetLastError();
        GnArgs a = gn_args(p, g);
        const bool weights = dgamma || dbeta;
        if (p.n > 0) {
            a.x = x;
            a.dy = dy;
            a.gamma = gamma;
            a.beta = beta;
            a.y = dx;
            a.mean = const_cast<float*>(mean);
            a.rstd = const_cast<float*>(rstd);
            a.part = dx ? static_cast<float2*>(ws) : nullptr;
            a.cols = weights ? reinterpret_cast<float*>(static_cast<char*>(ws) + g.cols) : nullptr;
            rc = by_samples(p, g, "groupnorm_bwd", [&](int64_t n0, int64_t n) {
                GnArgs b = a;
                b.n = n;
                b.x = moved(a.x, n0 * p.pixels * p.xs * es);
                b.dy = moved(a.dy, n0 * p.pixels * p.ys * es);
                b.y = moved(a.y, n0 * p.pixels * p.xs * es);
                b.mean = moved(a.mean, n0 * p.groups * 4);
                b.rstd = moved(a.rstd, n0 * p.groups * 4);
                b.part = moved(a.part, n0 * g.part_sample);
                b.cols = moved(a.cols, n0 * g.s.chunks * 2 * p.c * 4);
                launch_groupnorm_bwd(p.dtype, b, st);
            });
            if (rc) return rc;
        }
        if (weights) {
            // (over no rows the sums are 0)
            launch_layernorm_reduce(p.param, a.cols, int(p.n * g.s.chunks), p.c, dgamma, dbeta, st);
            if ((rc = launched("groupnorm_reduce"))) return rc;
        }
        return ok();
    });
}

}  // extern "C"
