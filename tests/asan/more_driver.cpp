// Host-side checks of position rotation, the norms per head and the AdamW step
// under AddressSanitizer and UBSan.
//
// Test infrastructure: built by tests/test_more_asan_host.py with the operators'
// sources, sanitizers on their host side. Everything called here returns before
// any kernel is launched or device touched: the workspace sizes over many
// descriptions, the layout of the tensors' table, and the argument checks. A
// sanitizer report aborts the run with a non-zero status.
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "matopt_adamw.h"

static char g_text[512];
namespace matopt {
opt_status fail(opt_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_text, sizeof g_text, fmt, ap);
    va_end(ap);
    return st;
}
}  // namespace matopt

namespace {

int failures = 0;

void expect(bool ok, const char* what) {
    if (!ok) {
        std::fprintf(stderr, "FAILED: %s (%s)\n", what, g_text);
        ++failures;
    }
}

const uintptr_t kBase = uintptr_t(1) << 40;
template <class T = void>
T* at(uintptr_t off) { return (T*)(kBase + off); }

void heads() {
    std::mt19937_64 r(3);
    for (int n = 0; n < 20000; ++n) {
        opt_heads_desc d{};
        d.dtype = r() % 3;
        d.heads = 1 + r() % 200, d.kv_heads = r() % 200, d.head_dim = 1 + r() % 512;
        d.batch = (int64_t)std::exp2((r() % 2200) / 100.0) - 1, d.tokens = (int64_t)std::exp2((r() % 2200) / 100.0) - 1;
        uint64_t need = 1;
        const bool fits = d.batch * d.tokens <= INT32_MAX;
        expect(opt_qk_norm_workspace_size(&d, &need) == (fits ? OPT_OK : OPT_EUNSUPPORTED), "heads size");
        if (fits) expect(need % 256 == 0 && (need > 0) == (d.batch * d.tokens > 0), "heads size is whole");
    }
    opt_heads_desc d{};
    d.dtype = OPT_F32, d.heads = 4, d.kv_heads = 2, d.head_dim = 64, d.batch = INT64_MAX, d.tokens = INT64_MAX;
    uint64_t need = 0;
    expect(opt_qk_norm_workspace_size(&d, &need) == OPT_EUNSUPPORTED, "heads sizes whose product overflows");
    d.batch = 3, d.tokens = 5;
    opt_rotary rope{};
    rope.turns = at<uint64_t>(0), rope.rot = 64, rope.scale = 1.f;
    const int64_t most = INT64_MAX / 8;
    const opt_attention_tensor ok = {at(0), 5 * 256, 256, 64}, far = {at(0), most, most, most}, bad = {at(0), 64, 64, 64};
    expect(opt_rotary_apply(&d, &rope, 0, &far, &ok, &bad, &ok, nullptr) == OPT_EINVAL, "rows that overlap");
    expect(opt_rotary_apply(&d, &rope, 0, &far, &ok, &far, &ok, nullptr) == OPT_EINVAL, "equal huge strides overlap");
    rope.rot = 66;
    expect(opt_rotary_apply(&d, &rope, 1, &ok, &ok, &ok, &ok, nullptr) == OPT_EINVAL, "rot past head_dim");
    rope.rot = 64, rope.scale = NAN;
    expect(opt_rotary_apply(&d, &rope, 1, &ok, &ok, &ok, &ok, nullptr) == OPT_EINVAL, "scale");
    d.batch = 0;
    rope.scale = 1.f;
    expect(opt_rotary_apply(&d, &rope, 1, nullptr, nullptr, nullptr, nullptr, nullptr) == OPT_OK, "no tokens");
    expect(opt_qk_norm_forward(&d, nullptr, nullptr, nullptr, nullptr, nullptr, 0.f, nullptr, nullptr, nullptr, nullptr,
                               nullptr) == OPT_OK, "norm of no tokens");
}

opt_adamw_desc tensor(uintptr_t base, int64_t n, int bits) {
    opt_adamw_desc x{};
    x.n = n, x.state_bits = bits, x.lr_scale = 1.f;
    x.W = at<float>(base), x.G = at(base + (1u << 20)), x.m = at(base + (2u << 20)), x.v = at(base + (3u << 20));
    if (bits == 8) x.m_scale = at<float>(base + (4u << 20)), x.v_scale = at<float>(base + (5u << 20));
    return x;
}

void adamw() {
    std::mt19937_64 r(9);
    const opt_adamw_hparams hp = {1e-3, 0.9, 0.999, 1e-8};
    opt_adamw_t g = nullptr;
    for (int n = 0; n < 300; ++n) {
        std::vector<opt_adamw_desc> d(1 + r() % 300);
        for (auto& x : d) {
            x = tensor(0, (int64_t)std::exp2((r() % 2500) / 100.0) - 1, r() % 2 ? 32 : 8);
            x.G_dtype = r() % 3;
        }
        uint64_t need = 0, less = 0;
        expect(opt_adamw_workspace_size(d.data(), (int32_t)d.size(), &need) == OPT_OK && need % 256 == 0, "adamw size");
        expect(opt_adamw_workspace_size(d.data(), 1, &less) == OPT_OK && less <= need, "adamw size grows");
        // 200 000 elements at most apart: these overlap unless there is one
        const opt_status st = opt_adamw_create(d.data(), (int32_t)d.size(), &hp, at(uintptr_t(1) << 36), 0, nullptr, &g);
        expect((st == OPT_EINVAL || st == OPT_ENOWS) && !g, "overlaps or no workspace");
    }
    std::vector<opt_adamw_desc> d;
    for (int i = 0; i < 2000; ++i) d.push_back(tensor((uintptr_t)i << 23, 1 + i * 13, i % 2 ? 32 : 8));
    uint64_t need = 0;
    expect(opt_adamw_workspace_size(d.data(), 2000, &need) == OPT_OK, "2000 tensors");
    expect(opt_adamw_create(d.data(), 2000, &hp, at(uintptr_t(1) << 36), need - 1, nullptr, &g) == OPT_ENOWS && !g, "ENOWS");
    expect(opt_adamw_create(d.data(), 2000, &hp, at((uintptr_t)7 << 23), need, nullptr, &g) == OPT_EINVAL && !g, "workspace on a tensor");
    d[1234].v = d[77].m_scale;
    expect(opt_adamw_create(d.data(), 2000, &hp, at(uintptr_t(1) << 36), need, nullptr, &g) == OPT_EINVAL && !g, "overlap among 2000");
    expect(opt_adamw_workspace_size(d.data(), 0, &need) == OPT_EINVAL, "no tensors");
    expect(opt_adamw_workspace_size(d.data(), INT32_MAX, &need) == OPT_EINVAL, "too many tensors");
    d[0].n = INT64_MAX;
    expect(opt_adamw_workspace_size(d.data(), 1, &need) == OPT_EUNSUPPORTED, "too many elements");
    opt_adamw_destroy(nullptr);
}

}  // namespace

int main() {
    heads();
    adamw();
    std::printf("host checks: %d failures\n", failures);
    return failures ? 1 : 0;
}
