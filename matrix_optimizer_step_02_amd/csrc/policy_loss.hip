// Clipped policy loss with a KL term on logits (HBM-bandwidth bound).
//
//   z = scale x,  lse = log sum_j exp(z_j),  logp = z_t - lse
//   r = exp(logp - old),  d = ref - logp
//   term  = max(-A r, -A clip(r)) + kl (exp(d) - d - 1)
//   slope = w ((-A r where that is the larger or equal) + kl (1 - exp(d)))
//   dx_j  = grad scale slope ([j = t] - exp(z_j - lse))
//
// One workgroup per row, of 256 or 1024 threads, or one wavefront for up to
// 2048 logits. The row is read once: each thread keeps its groups of eight
// logits in registers as they are stored (up to 80 registers of 1024
// threads: 163840 16-bit or 81920 32-bit logits, more than half of a CU's
// register file), takes the maximum, the sum of exponentials and the gradient
// from there, so a pass moves one read and one write of the logits: 4096 rows
// of 131072 16-bit logits take 405 to 435 us, 4.9 to 5.3 TB/s. Longer rows keep
// a running maximum and sum and read the row a second time, mostly from the
// last-level cache (2048 rows of 131072 32-bit logits: 511 us; 150000 16-bit
// logits 349 us that way, 270 from registers). The exponentials are taken in
// base 2, with log2(e) folded into the scale.
//
// Logits enter as differences from the row's maximum M, taken before anything
// is rounded at M's magnitude: with s = sum_j exp(z_j - M),
//   logp = (z_t - M) - log s,  p_j = exp(z_j - M) / s,  1 - p_t = -expm1(logp)
// so that an offset common to the row's logits costs nothing (a rounded
// M + log s put 7e-5 into logp at an offset of 1000). Logits in registers take
// one fused operation for it, x c - fl(M c), whose common shift M c - fl(M c)
// is known to the bit and leaves log s again; (x - M) c is an operation more
// (4096 x 131072: 500 against 486 us). Longer rows take that, and rows whose
// shift would grow large (|M c| from 2^20, as where all logits are the type's
// lowest value) are rewritten as x - M.
//
// The loss is the sum of the rows' terms, which a second kernel (past 16384
// rows a third) adds in 64 bits in a fixed order.
#include "train.h"

namespace matopt {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct PolicyArgs {
    const void *logits, *target;
    const float *old_logp, *ref_logp, *advantage, *weight;
    float *logp, *lse, *rest, *slope, *term;   // NULL where the call does not return them; rest: of lse's rounding
    void* dlogits;                      // NULL: forward only
    int64_t ld, ldd;
    int32_t vocab, target_i64;
    uint32_t rows, first;               // first: row of the launch's first workgroup
    float scale, lo, hi, kl, grad;
};

// Eight logits as stored.
template <class T>
struct Raw8 {
    static constexpr int W = sizeof(T) * 2;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p) {
        const auto* q = (const __attribute__((address_space(1))) u32x4u*)p;
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const u32x4u r = q[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[4 * i + e] = r[e];
        }
    }
    __device__ __forceinline__ void set(int e, T x) {
        if constexpr (sizeof(T) == 4) {
            w[e] = __builtin_bit_cast(uint32_t, x);
        } else {
            const uint32_t b = __builtin_bit_cast(uint16_t, x);
            w[e >> 1] = e & 1 ? (w[e >> 1] & 0xffffu) | b << 16 : (w[e >> 1] & 0xffff0000u) | b;
        }
    }
    // the first n elements, -inf (which adds nothing to a sum of exponentials) past them
    __device__ __forceinline__ void load_n(const T* p, int n) {
        if (n >= 8) return load(p);
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) set(e, e < n ? gptr(p)[e] : (T)-INFINITY);
    }
    // Makes the registers look rewritten, so that the compiler converts them
    // again in the next phase rather than keep the converted values, twice
    // the registers, across phases (88 spilled at 131072 16-bit logits).
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int i = 0; i < W; ++i) asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, w[e]);
        else return (float)__builtin_bit_cast(T, (uint16_t)(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]));
    }
};

constexpr int row_threads(int nt) { return nt < 256 ? 256 : nt; }   // of a workgroup

// A value that all of a wavefront's threads have: in a scalar register.
__device__ __forceinline__ float uniform(float x) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// Over the NT threads of a row: a wavefront, or the whole workgroup.
template <int NT, bool MAX>
__device__ __forceinline__ float row_reduce(float x, float* part) {
    x = MAX ? wave_max(x) : wave_sum(x);
    if constexpr (NT == 64) return uniform(x);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    float s = part[0];
#pragma unroll
    for (int k = 1; k < NT / 64; ++k) s = MAX ? fmaxf(s, part[k]) : s + part[k];
    return uniform(s);
}

__device__ __forceinline__ int64_t target_of(const PolicyArgs& a, uint32_t row) {
    return a.target_i64 ? gptr((const int64_t*)a.target)[row] : gptr((const int32_t*)a.target)[row];
}

// a + b rounded, and the error of that rounding (Knuth).
__device__ __forceinline__ float two_sum(float a, float b, float& rest) {
#pragma clang fp contract(off) reassociate(off)
    const float s = a + b, t = s - a;
    rest = (a - (s - t)) + (b - t);
    return s;
}

// What a row's log probability makes of the loss: its term and slope. max and
// >= would lose a NaN of any of the row's inputs; the unclipped term holds
// them all but ref's. An advantage of 0 makes that term 0 also where the ratio
// passes the range of fp32.
__device__ __forceinline__ void row_loss(const PolicyArgs& a, uint32_t row, float w, float logp, float& term,
                                         float& slope) {
    const float adv = gptr(a.advantage)[row];
    const float r = expf(logp - gptr(a.old_logp)[row]);
    const float clipped = fminf(fmaxf(r, a.lo), a.hi);
    const float free = adv == 0.f && r == INFINITY ? 0.f : -adv * r, bound = -adv * clipped;
    term = fmaxf(free, bound);
    slope = free >= bound ? free : 0.f;
    if (a.kl != 0.f) {
        const float d = gptr(a.ref_logp)[row] - logp, e = expm1f(d);
        term += a.kl * (e - d);
        slope -= a.kl * e;
    }
    if (free != free) term = slope = free;
    term *= w;
    slope *= w;
}

// NV: groups of eight a thread keeps; 0: the row is read twice.
template <class T, int NT, int NV>
__global__ __launch_bounds__(row_threads(NT)) void policy_row_kernel(PolicyArgs a) {
    __shared__ float part[2][NT / 64];
    constexpr int R = row_threads(NT) / NT;
    uint32_t row = a.first + blockIdx.x;
    int tid = threadIdx.x;
    if constexpr (R > 1) {
        row = a.first + blockIdx.x * R + __builtin_amdgcn_readfirstlane(threadIdx.x / NT), tid %= NT;
        if (row >= a.rows) return;
    }
    const int V = a.vocab, G = (V + 7) >> 3;
    const T* x = (const T*)a.logits + (int64_t)row * a.ld;
    T* dx = a.dlogits ? (T*)a.dlogits + (int64_t)row * a.ldd : nullptr;
    const float w = gptr(a.weight)[row];
    if (w == 0.f) {
        if (dx) {
            const float z[8] = {};
            for (int g = tid; g < G; g += NT) store_n(dx + 8 * (int64_t)g, V - 8 * g, z);
        }
        if (tid == 0) {
            gptr(a.term)[row] = 0.f;
            if (a.logp) gptr(a.logp)[row] = 0.f;
            if (a.lse) gptr(a.lse)[row] = 0.f;
            if (a.rest) gptr(a.rest)[row] = 0.f;
            if (a.slope) gptr(a.slope)[row] = 0.f;
        }
        return;
    }
    const float c = a.scale * kLog2e;
    const int64_t t = target_of(a, row);
    const bool valid = t >= 0 && t < V;
    const float xt = valid ? (float)gptr(x)[t] : NAN;   // before any store: dlogits may be logits

    Raw8<T> keep[NV > 0 ? NV : 1];
    float m = -INFINITY, s = 0.f;   // the maximum, and the sum of exp2((x - m) c + shift)
    float mc = 0.f, shift = 0.f;
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int g = tid + i * NT;
            keep[i].load_n(x + 8 * (int64_t)(g < G ? g : 0), g < G ? V - 8 * g : 0);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, keep[i].get(e));
        m = row_reduce<NT, true>(m, part[0]);
        mc = uniform(m * c);
        shift = fmaf(m, c, -mc);
        if (!(fabsf(mc) < 0x1p20f)) {   // the same for all threads of the row
            // The differences in place of the logits, rounded to their type:
            // exact within a factor of two of m, and past that below -2^19 / c
            // and without a part in any sum.
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                keep[i].again();
                Raw8<T> r;
#pragma unroll
                for (int j = 0; j < Raw8<T>::W; ++j) r.w[j] = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) r.set(e, from_f32<T>(keep[i].get(e) - m));
                r.again();
                keep[i] = r;
            }
            mc = shift = 0.f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            keep[i].again();
#pragma unroll
            for (int e = 0; e < 8; ++e) s += __builtin_amdgcn_exp2f(fmaf(keep[i].get(e), c, -mc));
        }
        s = row_reduce<NT, false>(s, part[1]);
    } else {
        constexpr int U = 4;
        for (int g0 = tid; g0 < G; g0 += U * NT) {
            Raw8<T> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int g = g0 + u * NT;
                r[u].load_n(x + 8 * (int64_t)(g < G ? g : 0), g < G ? V - 8 * g : 0);
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, r[u].get(e));
            if (top == -INFINITY) {   // nothing yet but -inf, or a NaN, which must reach the sum
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < 8; ++e) s += r[u].get(e) != r[u].get(e) ? NAN : 0.f;
                continue;
            }
            s *= __builtin_amdgcn_exp2f((m - top) * c);
            m = top;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += __builtin_amdgcn_exp2f((r[u].get(e) - m) * c);
        }
        const float all = row_reduce<NT, true>(m, part[0]);
        if (m != -INFINITY) s *= __builtin_amdgcn_exp2f((m - all) * c);
        m = all;
        s = row_reduce<NT, false>(s, part[1]);
    }
    const float ls = (log2f(s) - shift) * kLn2;
    float logp = fmaf(xt - m, a.scale, -ls);
    if (logp > 0.f) logp = 0.f;   // the sum's rounding, where the target holds nearly all of it
    float term, slope;
    row_loss(a, row, w, logp, term, slope);
    if (tid == 0) {
        gptr(a.term)[row] = term;
        if (a.logp) gptr(a.logp)[row] = logp;
        if (a.lse) {
            // scale m + ls as the nearest fp32 value, and what that leaves out
            const float z = a.scale * m, small = fmaf(a.scale, m, -z) + ls;
            float rest;
            const float lse = two_sum(z, small, rest);
            gptr(a.lse)[row] = lse;
            if (a.rest) gptr(a.rest)[row] = rest;
        }
        if (a.slope) gptr(a.slope)[row] = slope;
    }
    if (!dx) return;
    const float k = a.grad * a.scale * slope, ks = uniform(k / s);
    auto write = [&](int g, const Raw8<T>& r) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            o[e] = -ks * __builtin_amdgcn_exp2f(NV > 0 ? fmaf(r.get(e), c, -mc) : (r.get(e) - m) * c);
        store_n(dx + 8 * (int64_t)g, V - 8 * g, o);
    };
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            keep[i].again();
            if (tid + i * NT < G) write(tid + i * NT, keep[i]);
        }
    } else {
        for (int g = tid; g < G; g += NT) {
            Raw8<T> r;
            r.load_n(x + 8 * (int64_t)g, V - 8 * g);
            write(g, r);
        }
    }
    // the target's entry, by the thread that wrote its group
    if (valid && (int)(t >> 3) % NT == tid) gptr(dx)[t] = from_f32<T>(k * -expm1f(logp));
}

// dlogits from the saved log-sum and slope: z_j - lse is one rounding of the
// exact difference, of its own magnitude, and takes what lse's rounding left
// out (rest) from there. kBackPer groups of a row per
// thread, NT threads of a workgroup on one row: a wavefront up to 2048 logits
// (65536 rows of 1000 16-bit logits 30 us, of 2000 77; with 256 threads a row
// 65 and 109).
constexpr int kBackThreads = 256, kBackPer = 4;
template <class T, int NT>
__global__ __launch_bounds__(kBackThreads) void policy_backward_kernel(PolicyArgs a, const float* grad) {
    const uint32_t row = a.first + blockIdx.x * (kBackThreads / NT) + __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
    if (row >= a.rows) return;
    const int V = a.vocab, G = (V + 7) >> 3, g0 = blockIdx.y * (NT * kBackPer) + threadIdx.x % NT;
    const T* x = (const T*)a.logits + (int64_t)row * a.ld;
    T* dx = (T*)a.dlogits + (int64_t)row * a.ldd;
    const float slope = gptr(a.slope)[row];
    const float k = slope == 0.f ? 0.f : (grad ? *gptr(grad) : 1.f) * a.scale * slope;
    const float lse = gptr(a.lse)[row], rest = a.rest ? gptr(a.rest)[row] : 0.f;
    const int64_t t = target_of(a, row);
    Raw8<T> r[kBackPer];
#pragma unroll
    for (int i = 0; i < kBackPer; ++i) {
        const int g = g0 + i * NT;
        if (k != 0.f) r[i].load_n(x + 8 * (int64_t)(g < G ? g : 0), g < G ? V - 8 * g : 0);
    }
#pragma unroll
    for (int i = 0; i < kBackPer; ++i) {
        const int g = g0 + i * NT;
        if (g >= G) continue;
        float o[8] = {}, logp = 0.f;
        if (k != 0.f) {   // a row without slope is not read: it may hold anything
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = fmaf(r[i].get(e), a.scale, -lse) - rest;
                if (8 * (int64_t)g + e == t) logp = z;
                o[e] = -k * __builtin_amdgcn_exp2f(z * kLog2e);
            }
        }
        store_n(dx + 8 * (int64_t)g, V - 8 * g, o);
        if (k != 0.f && t >> 3 == g && t < V) gptr(dx)[t] = from_f32<T>(k * -expm1f(logp));
    }
}

// Sums of `per` values each, a workgroup per sum.
constexpr int kLossThreads = 1024;
template <class I, class O>
__global__ __launch_bounds__(kLossThreads) void policy_sum_kernel(int64_t n, int64_t per, const I* in, O* out) {
    __shared__ double part[kLossThreads / 64];
    const int64_t from = blockIdx.x * per, to = from + per < n ? from + per : n;
    double s = 0.0;
    for (int64_t r = from + threadIdx.x; r < to; r += kLossThreads) s += gptr(in)[r];
#pragma unroll
    for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x) return;
    s = part[0];
    for (int k = 1; k < kLossThreads / 64; ++k) s += part[k];
    gptr(out)[blockIdx.x] = (O)s;
}

// One workgroup adds 4096 terms in 3 us, 16384 in 5.5 and 65536 in 18, at its
// own pace and not memory's: past 16384 they are added in parts first, and
// then the parts (5.7 and 9.4 us; 10^6 terms 10 in place of 270).
constexpr int64_t kLossPart = 4096;
int64_t loss_parts(int64_t rows) { return rows <= 4 * kLossPart ? 0 : (rows + kLossPart - 1) / kLossPart; }
uint64_t align256(uint64_t n) { return (n + 255) / 256 * 256; }

void launch_sum(int64_t rows, const float* term, float* loss, hipStream_t s) {
    const int64_t parts = loss_parts(rows);
    if (parts == 0) {
        policy_sum_kernel<<<1, kLossThreads, 0, s>>>(rows, rows, term, loss);
        return;
    }
    double* part = (double*)((char*)term + align256((uint64_t)rows * 4));
    policy_sum_kernel<<<dim3((uint32_t)parts), kLossThreads, 0, s>>>(rows, kLossPart, term, part);
    policy_sum_kernel<<<1, kLossThreads, 0, s>>>(parts, parts, (const double*)part, loss);
}

// Small vocabularies take a wavefront a row, four rows a workgroup, without
// barriers: 65536 rows of 1000 16-bit logits 48 us, of 2000 103, against 122
// and 169 with 256 threads a row, where starting the workgroups is the bound
// (64 rows of 2000: 4.8 against 4.2). Then small workgroups, so that several
// rows share a CU; past what 1024 threads hold in 80 registers the row is
// streamed.
template <class T, int NT, int NV>
void launch_rows(PolicyArgs a, int64_t rows, hipStream_t s) {
    constexpr int64_t N = row_threads(NT), R = N / NT, most = most_blocks(N);
    a.rows = (uint32_t)rows;
    for (int64_t r = 0; r < rows; r += most * R) {
        const int64_t blocks = (rows - r + R - 1) / R;
        a.first = (uint32_t)r;
        policy_row_kernel<T, NT, NV><<<dim3((uint32_t)(blocks < most ? blocks : most)), N, 0, s>>>(a);
    }
}
template <class T>
void launch_rows(const PolicyArgs& a, int64_t rows, hipStream_t s) {
    const int64_t v = a.vocab;
    constexpr int K = 4 / sizeof(T);   // logits per register
    if (v <= 8 * 64 * 2) launch_rows<T, 64, 2>(a, rows, s);
    else if (v <= 8 * 64 * 4) launch_rows<T, 64, 4>(a, rows, s);
    else if (v <= 8 * 256 * 2) launch_rows<T, 256, 2>(a, rows, s);
    else if (v <= 8 * 256 * 4) launch_rows<T, 256, 4>(a, rows, s);
    else if (v <= 8 * 1024 * 2) launch_rows<T, 1024, 2>(a, rows, s);
    else if (v <= 8 * 1024 * 4) launch_rows<T, 1024, 4>(a, rows, s);
    else if (v <= 8 * 1024 * 8) launch_rows<T, 1024, 8>(a, rows, s);
    else if (v <= 8 * 1024 * 8 * K) launch_rows<T, 1024, 8 * K>(a, rows, s);
    else if (v <= 8 * 1024 * 10 * K) launch_rows<T, 1024, 10 * K>(a, rows, s);
    else launch_rows<T, 1024, 0>(a, rows, s);
}

template <class T, int NT>
void launch_backward(PolicyArgs a, int64_t rows, int64_t chunks, const float* grad, hipStream_t s) {
    constexpr int64_t R = kBackThreads / NT;
    const int64_t most = most_blocks(kBackThreads) / chunks;
    a.rows = (uint32_t)rows;
    for (int64_t r = 0; r < rows; r += most * R) {
        const int64_t blocks = (rows - r + R - 1) / R;
        a.first = (uint32_t)r;
        const dim3 grid((uint32_t)(blocks < most ? blocks : most), (uint32_t)chunks);
        policy_backward_kernel<T, NT><<<grid, kBackThreads, 0, s>>>(a, grad);
    }
}
template <class T>
void launch_backward(const PolicyArgs& a, int64_t rows, int64_t chunks, const float* grad, hipStream_t s) {
    if (a.vocab <= 8 * 64 * kBackPer) launch_backward<T, 64>(a, rows, 1, grad, s);
    else launch_backward<T, kBackThreads>(a, rows, chunks, grad, s);
}

opt_status check_policy(const opt_policy_desc* a) {
    if (!a) return fail(OPT_EINVAL, "desc is NULL");
    if (!train_dtype(a->dtype)) return fail(OPT_EUNSUPPORTED, "dtype must be OPT_F32, OPT_BF16 or OPT_F16");
    if (a->rows < 0 || a->vocab < 1) return fail(OPT_EINVAL, "rows must be >= 0 and vocab >= 1");
    if (a->rows > INT32_MAX || a->vocab > INT32_MAX - 65536) return fail(OPT_EUNSUPPORTED, "rows or vocab too large");
    if (a->ld < a->vocab) return fail(OPT_EINVAL, "ld < vocab");
    if (!(a->logit_scale > 0.f) || !(a->logit_scale < INFINITY)) return fail(OPT_EINVAL, "logit_scale must be positive and finite");
    if (!(a->clip_low >= 0.f && a->clip_low <= 1.f) || !(a->clip_high >= 0.f))
        return fail(OPT_EINVAL, "clip_low must be in [0, 1] and clip_high >= 0");
    if (!(a->kl_coef >= 0.f)) return fail(OPT_EINVAL, "kl_coef must be >= 0");
    if (!train_aligned(a->lse_rest, 4)) return fail(OPT_EINVAL, "lse_rest is not aligned to its element size");
    return OPT_OK;
}

opt_status check_vector(const void* p, uintptr_t align, const char* name) {
    if (!p) return fail(OPT_EINVAL, "%s is NULL", name);
    if (!train_aligned(p, align)) return fail(OPT_EINVAL, "%s is not aligned to its element size", name);
    return OPT_OK;
}

opt_status check_rows(const opt_policy_desc* a, const opt_policy_rows* in) {
    if (!in) return fail(OPT_EINVAL, "rows' inputs are NULL");
    if (opt_status st = check_vector(in->target, a->target_i64 ? 8 : 4, "target")) return st;
    if (opt_status st = check_vector(in->old_logp, 4, "old_logp")) return st;
    if (opt_status st = check_vector(in->advantage, 4, "advantage")) return st;
    if (opt_status st = check_vector(in->weight, 4, "weight")) return st;
    if (a->kl_coef != 0.f)
        if (opt_status st = check_vector(in->ref_logp, 4, "ref_logp")) return st;
    return OPT_OK;
}

opt_status check_dlogits(const opt_policy_desc* a, const void* logits, const void* dlogits, int64_t ldd) {
    if (opt_status st = check_vector(dlogits, train_bytes(a->dtype), "dlogits")) return st;
    if (ldd < a->vocab) return fail(OPT_EINVAL, "ldd < vocab");
    if (dlogits == logits && ldd != a->ld) return fail(OPT_EINVAL, "dlogits in place of logits needs ldd == ld");
    return OPT_OK;
}

PolicyArgs policy_args(const opt_policy_desc* a, const void* logits, const opt_policy_rows* in) {
    PolicyArgs p = {};
    p.logits = logits;
    if (in) {
        p.target = in->target, p.old_logp = in->old_logp, p.ref_logp = in->ref_logp;
        p.advantage = in->advantage, p.weight = in->weight;
    }
    p.rest = a->lse_rest;
    p.ld = a->ld, p.vocab = (int32_t)a->vocab, p.target_i64 = a->target_i64;
    p.scale = a->logit_scale, p.lo = 1.f - a->clip_low, p.hi = 1.f + a->clip_high, p.kl = a->kl_coef, p.grad = 1.f;
    return p;
}

uint64_t policy_bytes(const opt_policy_desc* a) {
    return align256((uint64_t)a->rows * 4) + align256((uint64_t)loss_parts(a->rows) * 8);
}

opt_status run_rows(const opt_policy_desc* a, PolicyArgs p, float* loss, void* ws, uint64_t ws_bytes, void* stream) {
    if (opt_status st = check_vector(loss, 4, "loss")) return st;
    if (ws_bytes < policy_bytes(a)) return fail(OPT_ENOWS, "workspace too small");
    if (a->rows && (!ws || !train_aligned(ws, 256))) return fail(OPT_EINVAL, "workspace is NULL or not 256-byte aligned");
    if (opt_status st = train_pending()) return st;
    p.term = (float*)ws;
    const hipStream_t s = (hipStream_t)stream;
    if (a->rows) {
        if (a->dtype == OPT_F32) launch_rows<float>(p, a->rows, s);
        else if (a->dtype == OPT_BF16) launch_rows<__bf16>(p, a->rows, s);
        else launch_rows<_Float16>(p, a->rows, s);
    }
    launch_sum(a->rows, p.term, loss, s);
    return train_launched("policy loss");
}

}  // namespace
}  // namespace matopt

using namespace matopt;

extern "C" {

opt_status opt_policy_loss_workspace_size(const opt_policy_desc* a, uint64_t* bytes) {
    if (!bytes) return fail(OPT_EINVAL, "bytes is NULL");
    if (opt_status st = check_policy(a)) return st;
    *bytes = policy_bytes(a);
    return OPT_OK;
}

opt_status opt_policy_loss_forward(const opt_policy_desc* a, const void* logits, const opt_policy_rows* in,
                                   float* loss, float* logp, float* lse, float* slope, void* workspace,
                                   uint64_t workspace_bytes, void* stream) {
    if (opt_status st = check_policy(a)) return st;
    PolicyArgs p = policy_args(a, logits, in);
    if (a->rows) {
        if (opt_status st = check_vector(logits, train_bytes(a->dtype), "logits")) return st;
        if (opt_status st = check_rows(a, in)) return st;
        if (opt_status st = check_vector(logp, 4, "logp")) return st;
        if (opt_status st = check_vector(lse, 4, "lse")) return st;
        if (opt_status st = check_vector(slope, 4, "slope")) return st;
        p.logp = logp, p.lse = lse, p.slope = slope;
    }
    return run_rows(a, p, loss, workspace, workspace_bytes, stream);
}

opt_status opt_policy_loss_step(const opt_policy_desc* a, const void* logits, const opt_policy_rows* in, float grad,
                                float* loss, float* logp, void* dlogits, int64_t ldd, void* workspace,
                                uint64_t workspace_bytes, void* stream) {
    if (opt_status st = check_policy(a)) return st;
    PolicyArgs p = policy_args(a, logits, in);
    if (a->rows) {
        if (opt_status st = check_vector(logits, train_bytes(a->dtype), "logits")) return st;
        if (opt_status st = check_rows(a, in)) return st;
        if (opt_status st = check_dlogits(a, logits, dlogits, ldd)) return st;
        if (!train_aligned(logp, 4)) return fail(OPT_EINVAL, "logp is not aligned to its element size");
        p.logp = logp, p.dlogits = dlogits, p.ldd = ldd, p.grad = grad;
    }
    return run_rows(a, p, loss, workspace, workspace_bytes, stream);
}

opt_status opt_policy_loss_backward(const opt_policy_desc* a, const void* logits, const void* target,
                                    const float* lse, const float* slope, const float* grad, void* dlogits,
                                    int64_t ldd, void* stream) {
    if (opt_status st = check_policy(a)) return st;
    if (a->rows == 0) return OPT_OK;
    if (opt_status st = check_vector(logits, train_bytes(a->dtype), "logits")) return st;
    if (opt_status st = check_vector(target, a->target_i64 ? 8 : 4, "target")) return st;
    if (opt_status st = check_vector(lse, 4, "lse")) return st;
    if (opt_status st = check_vector(slope, 4, "slope")) return st;
    if (opt_status st = check_dlogits(a, logits, dlogits, ldd)) return st;
    if (!train_aligned(grad, 4)) return fail(OPT_EINVAL, "grad is not aligned to its element size");
    const int64_t chunks = ((a->vocab + 7) / 8 + kBackThreads * kBackPer - 1) / (kBackThreads * kBackPer);
    if (chunks > 65535) return fail(OPT_EUNSUPPORTED, "vocab too large");
    if (opt_status st = train_pending()) return st;
    PolicyArgs p = policy_args(a, logits, nullptr);
    p.target = target, p.lse = (float*)lse, p.slope = (float*)slope, p.dlogits = dlogits, p.ldd = ldd;
    const hipStream_t s = (hipStream_t)stream;
    if (a->dtype == OPT_F32) launch_backward<float>(p, a->rows, chunks, grad, s);
    else if (a->dtype == OPT_BF16) launch_backward<__bf16>(p, a->rows, chunks, grad, s);
    else launch_backward<_Float16>(p, a->rows, chunks, grad, s);
    return train_launched("policy loss backward");
}

}  // extern "C"
