// Host-side checks of the training-pass operators' C ABI under
// AddressSanitizer and UBSan.
//
// Test infrastructure: built by tests/test_train_asan_host.py with the
// operators' sources, sanitizers on their host side. Everything called here
// returns before any kernel is launched: the workspace sizes over many
// descriptions, and the argument checks. A sanitizer report aborts the run
// with a non-zero status.
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>

#include "matopt_train.h"

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
void* at(uintptr_t off) { return (void*)(kBase + off); }

void attention_sizes() {
    std::mt19937_64 r(5);
    for (int n = 0; n < 20000; ++n) {
        opt_attention_desc a{};
        a.dtype = r() % 2 ? OPT_BF16 : OPT_F16;
        a.kv_heads = 1 + r() % 16;
        a.heads = a.kv_heads * (1 + r() % 8);
        a.head_dim = 8 * (1 + r() % 16);
        a.batch = r() % 200;
        a.q_len = (int32_t)std::exp2((r() % 1700) / 100.0) - 1;
        a.k_len = (int32_t)std::exp2((r() % 1700) / 100.0) - 1;
        a.causal = r() % 2;
        a.window = a.causal && r() % 3 == 0 ? 1 + r() % 4000 : 0;
        a.scale = 0.1f;
        if (r() % 2) {
            a.q_start = a.k_start = (const int32_t*)at(0);
            a.q_tokens = (int64_t)a.q_len * (r() % 20);
            a.k_tokens = (int64_t)a.k_len * (r() % 20);
        }
        uint64_t f = 1, b = 1;
        expect(opt_attention_workspace_size(&a, 0, &f) == OPT_OK, "attention size");
        expect(opt_attention_workspace_size(&a, 1, &b) == OPT_OK, "attention backward size");
        const uint64_t rows = a.q_start ? (uint64_t)a.q_tokens : (uint64_t)a.batch * a.q_len;
        expect(f % 256 == 0 && b % 256 == 0 && b >= rows * a.heads * 4, "attention size is whole");
    }
}

void attention_errors() {
    opt_attention_desc a{};
    a.dtype = OPT_BF16, a.batch = 2, a.heads = 4, a.kv_heads = 2, a.head_dim = 64, a.q_len = a.k_len = 100;
    a.scale = 0.125f;
    const opt_attention_tensor t = {at(0), 25600, 256, 64};
    uint64_t need = 0;
    expect(opt_attention_workspace_size(&a, 1, &need) == OPT_OK, "size");
    expect(opt_attention_backward(&a, &t, &t, &t, &t, &t, (float*)at(0), &t, &t, &t, at(0), need - 1, nullptr) == OPT_ENOWS, "ENOWS");
    expect(opt_attention_backward(&a, &t, &t, &t, &t, &t, (float*)at(0), &t, &t, nullptr, at(0), need, nullptr) == OPT_EINVAL, "null dv");
    expect(opt_attention_forward(&a, &t, &t, &t, &t, nullptr, nullptr, 0, nullptr) == OPT_EINVAL, "null lse");
    opt_attention_desc b = a;
    b.batch = INT32_MAX, b.heads = INT32_MAX, b.kv_heads = 1, b.q_len = 1 << 30;
    expect(opt_attention_workspace_size(&b, 1, &need) == OPT_EUNSUPPORTED, "too many blocks");
    b = a;
    b.q_start = b.k_start = (const int32_t*)at(0);
    b.q_tokens = INT64_MAX;
    expect(opt_attention_workspace_size(&b, 1, &need) == OPT_EUNSUPPORTED, "too many tokens");
    b = a;
    b.batch = 0;
    expect(opt_attention_forward(&b, &t, &t, &t, &t, nullptr, nullptr, 0, nullptr) == OPT_OK, "no sequences");
    b = a;
    b.q_len = 0;
    expect(opt_attention_forward(&b, &t, &t, &t, &t, nullptr, nullptr, 0, nullptr) == OPT_OK, "no queries");
}

void norm_and_dropout() {
    const opt_rng rng = {1, 2, nullptr};
    uint64_t need = 0;
    for (int64_t cols = 1; cols <= OPT_MAX_DIM; cols += 1 + cols / 7)
        for (int64_t rows : {int64_t(0), int64_t(1), int64_t(5), int64_t(4099), int64_t(1) << 20, (int64_t(1) << 31) - 1})
            expect(opt_layer_norm_workspace_size(rows, cols, &need) == OPT_OK && need <= (uint64_t(1) << 29), "norm size");
    expect(opt_layer_norm_workspace_size(4, OPT_MAX_DIM + 1, &need) == OPT_EUNSUPPORTED, "norm cols");
    expect(opt_layer_norm_workspace_size(4, 16, &need) == OPT_OK, "norm size 4 x 16");
    expect(opt_layer_norm_forward(0, 16, OPT_F32, nullptr, 0, OPT_F32, nullptr, 0, nullptr, nullptr, 1e-5f, 0.f, nullptr,
                                  nullptr, 0, nullptr, 0, nullptr, nullptr, nullptr) == OPT_OK, "norm of no rows");
    expect(opt_layer_norm_backward(4, 16, OPT_F32, at(0), 16, OPT_F32, at(0), 16, nullptr, 0, (float*)at(0), (float*)at(0),
                                   (float*)at(0), 0.5f, &rng, at(0), 16, nullptr, 0, (float*)at(0), nullptr, at(0), need - 1,
                                   nullptr) == OPT_ENOWS, "norm ENOWS");
    expect(opt_dropout(0, 5, OPT_F32, nullptr, 0, nullptr, 0, nullptr, 0, 0.5f, &rng, nullptr) == OPT_OK, "dropout of no rows");
    expect(opt_dropout(5, 5, OPT_F32, at(0), 5, nullptr, 0, at(0), 5, 0.999999f, &rng, nullptr) == OPT_EUNSUPPORTED, "p near 1");
    expect(opt_dropout(5, 5, OPT_F32, at(0), 5, nullptr, 0, at(0), 5, INFINITY, &rng, nullptr) == OPT_EINVAL, "p infinite");
    expect(opt_dropout(5, 5, OPT_F32, at(0), INT64_MAX, nullptr, 0, at(0), 5, 0.5f, &rng, nullptr) == OPT_EUNSUPPORTED, "stride");
}

void policy() {
    opt_policy_desc a{};
    a.dtype = OPT_BF16, a.rows = INT32_MAX, a.vocab = 7, a.ld = 7, a.logit_scale = 1.f, a.clip_low = a.clip_high = 0.2f;
    uint64_t need = 0;
    expect(opt_policy_loss_workspace_size(&a, &need) == OPT_OK && need >= (uint64_t)INT32_MAX * 4, "policy size");
    const opt_policy_rows rows = {at(0), (float*)at(0), nullptr, (float*)at(0), (float*)at(0)};
    expect(opt_policy_loss_step(&a, at(0), &rows, 1.f, (float*)at(0), nullptr, at(0), 7, at(0), need - 1, nullptr) == OPT_ENOWS, "policy ENOWS");
    a.kl_coef = 0.1f;
    expect(opt_policy_loss_step(&a, at(0), &rows, 1.f, (float*)at(0), nullptr, at(0), 7, at(0), need, nullptr) == OPT_EINVAL, "no ref_logp");
    a.rows = 0;
    expect(opt_policy_loss_backward(&a, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr) == OPT_OK, "no rows");
}

}  // namespace

int main() {
    attention_sizes();
    attention_errors();
    norm_and_dropout();
    policy();
    std::printf("host checks: %d failures\n", failures);
    return failures ? 1 : 0;
}
