// C ABI of the AdamW step: argument checks and the launches.  No device code
// lives here.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>
#include <vector>

#include "adamw.h"
#include "host_checks.h"

namespace cnhwc {
namespace {

bool is_type(int t) { return t == CNHWC_F16 || t == CNHWC_BF16 || t == CNHWC_F32; }

struct Span {
    uintptr_t lo, hi;   // addresses [lo, hi)
    uint32_t id;        // tensor * 8 + role; the gradient's role, and the scalars, are read only
};
constexpr const char* kRole[] = {"p", "m", "v", "m_scale", "v_scale", "copy", "gradient", "a device scalar"};
constexpr uint32_t kReadOnly = 6;

std::string name_of(uint32_t id) {
    const uint32_t role = id % 8;
    return role == 7 ? kRole[7] : std::string(kRole[role]) + " of tensor " + num(id / 8);
}

// No written span may overlap any other.  Programs list their buffers in
// order, role by role: spans arrive as a few ascending runs, which are joined.
int check_apart(std::vector<Span>& s, std::vector<size_t>& runs) {
    auto before = [](const Span& a, const Span& b) { return a.lo < b.lo; };
    runs.push_back(s.size());
    for (size_t i = 0; i + 1 < runs.size(); ++i)
        if (!std::is_sorted(s.begin() + long(runs[i]), s.begin() + long(runs[i + 1]), before))
            std::sort(s.begin() + long(runs[i]), s.begin() + long(runs[i + 1]), before);
    for (size_t i = 2; i < runs.size(); ++i)
        std::inplace_merge(s.begin(), s.begin() + long(runs[i - 1]), s.begin() + long(runs[i]), before);
    // ascending starts: a span that overlaps an earlier one starts under the
    // greatest end so far; of the read spans only a written one matters, and
    // the other way round
    const Span *far_w = nullptr, *far_r = nullptr;
    for (const Span& v : s) {
        const bool written = v.id % 8 < kReadOnly;
        const Span* hit = far_w && v.lo < far_w->hi ? far_w : written && far_r && v.lo < far_r->hi ? far_r : nullptr;
        if (hit) return bad(name_of(written ? v.id : hit->id) + " overlaps " + name_of(written ? hit->id : v.id));
        const Span*& far = written ? far_w : far_r;
        if (!far || v.hi > far->hi) far = &v;
    }
    return CNHWC_OK;
}

int run(const cnhwc_adamw_problem* prob, const cnhwc_adamw_tensor* tensors, const float* grad_scale,
        const float* device_lr, const int64_t* device_step, hipStream_t st) {
    if (!prob) return bad("problem descriptor is NULL");
    const cnhwc_adamw_problem& q = *prob;
    if (q.reserved[0] != 0 || q.reserved[1] != 0) return bad("reserved fields must be 0");
    if (q.count < 0 || q.count > 65535) return bad("count must be in [0, 65535] (got " + num(q.count) + ")");
    if (!(q.lr >= 0.0) || !std::isfinite(q.lr)) return bad("lr must be finite and >= 0");
    if (!(q.beta1 >= 0.0 && q.beta1 < 1.0)) return bad("beta1 must be in [0, 1)");
    if (!(q.beta2 >= 0.0 && q.beta2 < 1.0)) return bad("beta2 must be in [0, 1)");
    if (!(q.eps >= 0.0) || !std::isfinite(q.eps)) return bad("eps must be finite and >= 0");
    if (q.step < (device_step ? 0 : 1)) return bad("step must be >= 1 (got " + num(q.step) + ")");
    if (q.state_bits != 8 && q.state_bits != 32) return bad("state_bits must be 8 or 32 (got " + num(q.state_bits) + ")");
    if (q.count > 0 && !tensors) return bad("tensors is NULL");
    const bool small = q.state_bits == 8;
    std::vector<Span> spans;
    std::vector<size_t> runs;
    spans.reserve(size_t(q.count) * 7 + 3);
    int rc;
    auto add = [&](const void* p, int64_t bytes, int align, uint32_t id) -> int {
        if (bytes == 0) return CNHWC_OK;
        if (!p) return bad(name_of(id) + " is NULL");
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (lo % unsigned(align) != 0)
            return fail(CNHWC_MISALIGNED, name_of(id) + " is not " + num(align) + "-byte aligned");
        spans.push_back({lo, lo + uintptr_t(bytes), id});
        return CNHWC_OK;
    };
    for (int i = 0; i < q.count; ++i) {
        const cnhwc_adamw_tensor& t = tensors[i];
        auto which = [&] { return " of tensor " + num(i); };
        if (t.reserved != 0) return bad("reserved field" + which() + " must be 0");
        if (t.n < 0 || t.n >= int64_t(1) << 34) return bad("n" + which() + " must be in [0, 2^34) (got " + num(t.n) + ")");
        if (!std::isfinite(t.weight_decay)) return bad("weight_decay" + which() + " must be finite");
        if (!is_type(t.p_dtype)) return bad("p_dtype" + which() + " must be CNHWC_F16, CNHWC_BF16 or CNHWC_F32");
        if (!is_type(t.g_dtype)) return bad("g_dtype" + which() + " must be CNHWC_F16, CNHWC_BF16 or CNHWC_F32");
        if (t.copy && !is_type(t.copy_dtype)) return bad("copy_dtype" + which() + " must be CNHWC_F16, CNHWC_BF16 or CNHWC_F32");
    }
    for (uint32_t role = 0; role < 7; ++role) {
        runs.push_back(spans.size());
        if ((role == 3 || role == 4) && !small) continue;
        for (int i = 0; i < q.count; ++i) {
            const cnhwc_adamw_tensor& t = tensors[i];
            const uint32_t id = uint32_t(i) * 8 + role;
            const int64_t scales = ceil_div(t.n, kAdamBlock) * 4;
            const int sb = small ? 1 : 4;
            switch (role) {
            case 0: rc = add(t.p, t.n * elem_bytes(t.p_dtype), elem_bytes(t.p_dtype), id); break;
            case 1: rc = add(t.m, t.n * sb, sb, id); break;
            case 2: rc = add(t.v, t.n * sb, sb, id); break;
            case 3: rc = add(t.m_scale, scales, 4, id); break;
            case 4: rc = add(t.v_scale, scales, 4, id); break;
            case 5: rc = t.copy ? add(t.copy, t.n * elem_bytes(t.copy_dtype), elem_bytes(t.copy_dtype), id) : CNHWC_OK; break;
            default: rc = add(t.g, t.n * elem_bytes(t.g_dtype), elem_bytes(t.g_dtype), id);
            }
            if (rc) return rc;
        }
    }
    runs.push_back(spans.size());
    if (grad_scale && (rc = add(grad_scale, 4, 4, 7))) return rc;
    if (device_lr && (rc = add(device_lr, 4, 4, 7))) return rc;
    if (device_step && (rc = add(device_step, 8, 8, 7))) return rc;
    if ((rc = check_apart(spans, runs))) return rc;

    AdamArgs a;
    std::memset(&a, 0, sizeof a);
    a.eps = float(q.eps);
    a.lr = float(q.lr);
    a.beta1 = q.beta1;
    a.beta2 = q.beta2;
    a.step = q.step;
    a.seed = q.seed;
    a.grad_scale = grad_scale;
    a.device_lr = device_lr;
    a.device_step = device_step;
    if (!device_step) {
        a.inv_c1 = float(1.0 / (1.0 - adam_power(q.beta1, q.step)));
        a.rsqrt_c2 = float(1.0 / std::sqrt(1.0 - adam_power(q.beta2, q.step)));
    }
    (void)hipGetLastError();
    constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;   // a launch has less than 2^32 threads
    int64_t pairs = 0;   // the launch's blocks at two scale blocks a wave
    int count = 0;
    auto flush = [&]() -> int {
        if (count == 0) return CNHWC_OK;
        // One scale block a wave while that fills the GPU a few times at most, for the
        // latency (2.6 million elements in 52 tensors, 8 bits: 14.9 us, with two 16.2; 50 million
        // 174 and 169).
        const int deep = pairs <= 8 * kNumCUs ? 1 : 2;
        uint32_t blocks = 0;
        for (int i = 0; i < kAdamItems; ++i) {
            a.first[i] = i < count ? blocks : ~0u;
            if (i < count) blocks += uint32_t(ceil_div(a.item[i].n, adam_chunk(deep)));
        }
        launch_adamw(q.state_bits, deep, a, blocks, st);
        count = 0;
        pairs = 0;
        return launched("adamw");
    };
    for (int i = 0; i < q.count; ++i) {
        const cnhwc_adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        const int64_t need = ceil_div(t.n, adam_chunk(2));   // at most 2^23
        if (pairs + need > kMaxBlocks && (rc = flush())) return rc;
        a.item[count++] = {t.p, t.g, t.m, t.v, t.m_scale, t.v_scale, t.copy, t.n, float(t.weight_decay), uint16_t(i),
                           uint8_t(t.p_dtype), uint8_t(t.g_dtype), uint8_t(t.copy ? t.copy_dtype : 0)};
        pairs += need;
        if (count == kAdamItems && (rc = flush())) return rc;
    }
    if ((rc = flush())) return rc;
    return ok();
}

}  // namespace
}  // namespace cnhwc

using namespace cnhwc;

extern "C" {

int cnhwc_adamw(const cnhwc_adamw_problem* prob, const cnhwc_adamw_tensor* tensors, const float* grad_scale,
                const float* device_lr, const int64_t* device_step, void* hip_stream) {
    return guarded([&]() -> int {
        return run(prob, tensors, grad_scale, device_lr, device_step, reinterpret_cast<hipStream_t>(hip_stream));
    });
}

int cnhwc_adamw_moments(int64_t n, const void* m, const void* v, const float* m_scale, const float* v_scale,
                        float* m_values, float* v_values, void* hip_stream) {
    return guarded([&]() -> int {
        // (one launch, which has less than 2^32 threads: 16 elements each)
        if (n < 0 || n >= int64_t(1) << 35) return bad("n must be in [0, 2^35) (got " + num(n) + ")");
        const int64_t scales = ceil_div(n, kAdamBlock) * 4;
        const View in[4] = {{"m", m, n, 1}, {"v", v, n, 1}, {"m_scale", m_scale, scales, 4}, {"v_scale", v_scale, scales, 4}};
        const View out[2] = {{"m_values", m_values, n * 4, 4}, {"v_values", v_values, n * 4, 4}};
        if (int rc = check_views(in, 4, out, 2)) return rc;
        if (n == 0) return ok();
        (void)hipGetLastError();
        launch_adamw_moments(n, m, v, m_scale, v_scale, m_values, v_values, reinterpret_cast<hipStream_t>(hip_stream));
        if (int rc = launched("adamw_moments")) return rc;
        return ok();
    });
}

}  // extern "C"
