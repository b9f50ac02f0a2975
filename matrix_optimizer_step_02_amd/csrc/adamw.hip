// The AdamW step over many tensors at once, and the norm of all gradients
// (HBM-bandwidth bound; for small tensors the launch).
//
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,  g = scale G
//   W <- W - lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + decay W)
//
// One launch walks all tensors of one kind (size of state, type of gradient): a
// workgroup takes one chunk of 4096 elements, found in a table that create()
// uploads, so that a hundred norm weights cost one launch and an embedding fills
// the GPU. Everything of an element is read once and written once, eight elements
// a thread at a time, all loads of a thread in flight together: gradients are
// widened behind them (within a branch on their type each would wait for its
// own: 134 M elements, norm and step, 762 us, 754 so).
//
// States of 8 bits: 32 lanes hold a block of 256 elements, whose largest
// magnitude they find by exchanges; the scale is a power of two, so that scaling
// is exact and a code depends on the value and its random bits alone.
#include <algorithm>
#include <cmath>
#include <exception>
#include <vector>

#include "matopt_adamw.h"
#include "train.h"

namespace matopt {
namespace {

constexpr int kThreads = 256, kSets = 2;                  // groups of eight elements a thread
constexpr int64_t kChunk = kThreads * kSets * 8;
constexpr int kNormBlocks = 1024, kKinds = 6;              // workgroups of a launch; 32 and 8 bits, three types
constexpr int64_t kMostElements = int64_t(1) << 35;       // a group's number fits 32 bits of the counter
constexpr int kMostTensors = 1 << 20;

struct Seg {
    float* W;
    const void* G;
    void *m, *v;
    float *ms, *vs;
    void* copy;
    int64_t n;
    float lr_scale, decay;
    int32_t copy_dtype;   // -1 for none
    uint32_t index;
};
struct Chunk {
    uint32_t seg, at;   // the tensor and which of its chunks
};

struct StepArgs {
    const Seg* segs;
    const Chunk* chunks;
    const float* grad_scale;
    const int64_t* device_step;
    float b1, ob1, b2, ob2, eps, lr, c1, c2;   // c1 = 1 / (1 - b1^t), c2 = 1 / sqrt(1 - b2^t)
    double log_b1, log_b2;
    Drop rng;
};

// The first n of eight gradients as stored; the others are zeros.
template <class T>
using Eight = T __attribute__((ext_vector_type(8)));
template <class T>
__device__ __forceinline__ Eight<T> load_g(const Seg& s, int64_t i, int n) {
    typedef T at1 __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    const T* p = (const T*)s.G + i;
    Eight<T> x = {};
    if (n >= 8) {
        x = *(const __attribute__((address_space(1))) at1*)p;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) x[e] = gptr(p)[e];
    }
    return x;
}
__device__ __forceinline__ void store_copy(const Seg& s, int64_t i, int n, const float (&f)[8]) {
    if (s.copy_dtype == OPT_BF16) store_n((__bf16*)s.copy + i, n, f);
    else if (s.copy_dtype == OPT_F16) store_n((_Float16*)s.copy + i, n, f);
}

__device__ __forceinline__ int left8(int64_t n, int64_t i) { return n - i < 8 ? (n - i < 0 ? 0 : (int)(n - i)) : 8; }

// The bias corrections at the step that device memory holds.
__device__ __forceinline__ void corrections(const StepArgs& a, float& c1, float& c2) {
    c1 = a.c1, c2 = a.c2;
    if (a.device_step) {
        const int64_t at = *gptr(a.device_step);
        const double t = at < 1 ? 1.0 : (double)at;
        c1 = (float)(-1.0 / expm1(t * a.log_b1));
        c2 = (float)(1.0 / sqrt(-expm1(t * a.log_b2)));
    }
}

// Each product and sum is rounded (no fused multiply-add): a state of 8 bits is
// a function of these values to the bit.
__device__ __forceinline__ void moments(const StepArgs& a, float g, float& m, float& v) {
#pragma clang fp contract(off)
    m = m * a.b1 + g * a.ob1;
    v = v * a.b2 + g * g * a.ob2;
}
__device__ __forceinline__ float weight(const StepArgs& a, float lr, float decay, float c1, float c2, float w, float m, float v) {
    return w - lr * (m * c1 / (sqrtf(v) * c2 + a.eps) + decay * w);
}

template <class T>
__global__ __launch_bounds__(kThreads) void adamw_kernel(StepArgs a) {
    const Chunk ch = a.chunks[blockIdx.x];
    const Seg s = a.segs[ch.seg];
    float scale = 1.f, c1, c2;
    if (a.grad_scale) scale = *gptr(a.grad_scale);
    if (scale != scale) return;
    corrections(a, c1, c2);
    const float lr = a.lr * s.lr_scale;
    Eight<T> g[kSets];
    float w[kSets][8], m[kSets][8], v[kSets][8];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
        const int64_t i = ch.at * kChunk + 8 * (k * kThreads + threadIdx.x);
        const int n = left8(s.n, i);
        g[k] = load_g<T>(s, i, n);
        load_n((const float*)s.m + i, n, m[k]);
        load_n((const float*)s.v + i, n, v[k]);
        load_n(s.W + i, n, w[k]);
    }
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
        const int64_t i = ch.at * kChunk + 8 * (k * kThreads + threadIdx.x);
        const int n = left8(s.n, i);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            moments(a, (float)g[k][e] * scale, m[k][e], v[k][e]);
            w[k][e] = weight(a, lr, s.decay, c1, c2, w[k][e], m[k][e], v[k][e]);
        }
        store_n((float*)s.m + i, n, m[k]);
        store_n((float*)s.v + i, n, v[k]);
        store_n(s.W + i, n, w[k]);
        store_copy(s, i, n, w[k]);
    }
}

// ------------------------------------------------------------ 8-bit states ----

typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u32x2u load_bytes(const void* p, int n) {
    const auto* q = (const __attribute__((address_space(1))) uint8_t*)p;
    if (n >= 8) return *(const __attribute__((address_space(1))) u32x2u*)q;
    u32x2u x = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) x[e >> 2] |= (uint32_t)q[e] << (8 * (e & 3));
    return x;
}
__device__ __forceinline__ void store_bytes(void* p, int n, u32x2u x) {
    auto* q = (__attribute__((address_space(1))) uint8_t*)p;
    if (n >= 8) {
        *(__attribute__((address_space(1))) u32x2u*)q = x;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) q[e] = (uint8_t)(x[e >> 2] >> (8 * (e & 3)));
}

template <bool E5M2>
__device__ __forceinline__ void decode(u32x2u x, float scale, float (&f)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        f32x2 lo, hi;
        if constexpr (E5M2) {
            lo = __builtin_amdgcn_cvt_pk_f32_bf8(x[k], false);
            hi = __builtin_amdgcn_cvt_pk_f32_bf8(x[k], true);
        } else {
            lo = __builtin_amdgcn_cvt_pk_f32_fp8(x[k], false);
            hi = __builtin_amdgcn_cvt_pk_f32_fp8(x[k], true);
        }
        f[4 * k] = lo[0] * scale, f[4 * k + 1] = lo[1] * scale, f[4 * k + 2] = hi[0] * scale, f[4 * k + 3] = hi[1] * scale;
    }
}

// Exponent of a block's scale from its largest finite magnitude, over its 32
// lanes of eight values.
template <int TOP>
__device__ __forceinline__ int block_exponent(const float (&f)[8]) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = fabsf(f[e]);
        top = fmaxf(top, x < INFINITY ? x : 0.f);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor(top, k));
    const int e = (int)(__float_as_uint(top) >> 23) - 127 - TOP;
    return e < -120 ? -120 : e > 120 ? 120 : e;
}
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Magnitude y = |x| / scale to a code with DIGITS mantissa bits, r 16 random
// bits. From 2^(1 - BIAS) on the bits below the code's are y's low 23 - DIGITS:
// r is added at their top and they are cut off, which carries into the exponent.
// Below, a step is 2^(1 - BIAS - DIGITS) and the code their number. KEEP: what is
// above 0 stays so. A v that is lost while its m is not (2^-16 of the block's largest
// m, where v's smallest code is 2^-31 to 2^-30 of the largest v) would have the next
// steps divide that m by next to nothing: gradients spread over 2^14 and more of a
// block made steps of 1000 times the rate.
template <int DIGITS, int BIAS, bool KEEP>
__device__ __forceinline__ uint32_t encode(float x, float inverse, uint32_t r) {
    const float y = fabsf(x) * inverse;
    const uint32_t normal = ((__float_as_uint(y) + (r << (7 - DIGITS))) >> (23 - DIGITS)) - ((127 - BIAS) << DIGITS);
    const uint32_t small = ((uint32_t)(y * (float)(uint64_t(1) << (BIAS - 1 + DIGITS + 16))) + r) >> 16;
    uint32_t code = y < 1.f / (1 << (BIAS - 1)) ? small : normal;
    if (KEEP && x > 0.f && code == 0) code = 1;
    if (!(fabsf(x) < INFINITY)) code = 0x7f;
    return code | (x < 0.f ? 0x80u : 0u);
}

template <class T>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(StepArgs a) {
    const Chunk ch = a.chunks[blockIdx.x];
    const Seg s = a.segs[ch.seg];
    float scale = 1.f, c1, c2;
    if (a.grad_scale) scale = *gptr(a.grad_scale);
    if (scale != scale) return;
    corrections(a, c1, c2);
    const float lr = a.lr * s.lr_scale;
    const uint64_t offset = drop_offset(a.rng);
    Eight<T> g[kSets];
    float w[kSets][8], ms[kSets], vs[kSets];
    u32x2u mc[kSets], vc[kSets];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
        const int64_t i = ch.at * kChunk + 8 * (k * kThreads + threadIdx.x);
        const int n = left8(s.n, i);
        g[k] = load_g<T>(s, i, n);
        load_n(s.W + i, n, w[k]);
        mc[k] = load_bytes((const char*)s.m + i, n);
        vc[k] = load_bytes((const char*)s.v + i, n);
        ms[k] = n ? gptr(s.ms)[i / OPT_ADAMW_BLOCK] : 0.f;
        vs[k] = n ? gptr(s.vs)[i / OPT_ADAMW_BLOCK] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
        const int64_t i = ch.at * kChunk + 8 * (k * kThreads + threadIdx.x);
        const int n = left8(s.n, i);
        float m[8], v[8];
        decode<false>(mc[k], ms[k], m);
        decode<true>(vc[k], vs[k], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            moments(a, (float)g[k][e] * scale, m[e], v[e]);
            if (e >= n) m[e] = v[e] = 0.f;
            w[k][e] = weight(a, lr, s.decay, c1, c2, w[k][e], m[e], v[e]);
        }
        store_n(s.W + i, n, w[k]);
        store_copy(s, i, n, w[k]);
        uint32_t bits[4];
        philox((uint32_t)(i >> 3), s.index, offset, a.rng.seed, bits);
        const int me = block_exponent<7>(m), ve = block_exponent<14>(v);
        const float mi = power(-me), vi = power(-ve);
        u32x2u mo = {0, 0}, vo = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t r = e & 1 ? bits[e >> 1] >> 16 : bits[e >> 1] & 0xffffu;
            mo[e >> 2] |= encode<3, 7, false>(m[e], mi, (r >> 8) | (r & 255u) << 8) << (8 * (e & 3));
            vo[e >> 2] |= encode<2, 15, true>(v[e], vi, r) << (8 * (e & 3));
        }
        store_bytes((char*)s.m + i, n, mo);
        store_bytes((char*)s.v + i, n, vo);
        if (n && (threadIdx.x & 31) == 0) {
            gptr(s.ms)[i / OPT_ADAMW_BLOCK] = power(me);
            gptr(s.vs)[i / OPT_ADAMW_BLOCK] = power(ve);
        }
    }
}

// ----------------------------------------------------------- gradient norm ----

__device__ __forceinline__ double block_sum(double x, double* sh, int waves) {
#pragma unroll
    for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    double s = 0.0;
    for (int k = 0; k < waves; ++k) s += sh[k];
    return s;
}

// Squares are exact in 64 bits, and their sums there lose nothing that a norm
// in 32 bits would show, whatever the number of elements.
// After a step it runs at 3.3 TB/s of its own reads (268 MB: 80 us) beside the
// step's last writes, which leave the caches meanwhile; twice the workgroups or
// twice the loads in flight took 85 us.
template <class T>
__global__ __launch_bounds__(kThreads) void adamw_norm_kernel(const Seg* segs, const Chunk* chunks, uint32_t count, double* part) {
    __shared__ double sh[kThreads / 64];
    double sum = 0.0;
    for (uint32_t c = blockIdx.x; c < count; c += gridDim.x) {
        const Chunk ch = chunks[c];
        const Seg s = segs[ch.seg];
        Eight<T> g[kSets];
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
            const int64_t i = ch.at * kChunk + 8 * (k * kThreads + threadIdx.x);
            g[k] = load_g<T>(s, i, left8(s.n, i));
        }
#pragma unroll
        for (int k = 0; k < kSets; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fma((double)(float)g[k][e], (double)(float)g[k][e], sum);
    }
    sum = block_sum(sum, sh, kThreads / 64);
    if (threadIdx.x == 0) gptr(part)[blockIdx.x] = sum;
}

constexpr int kClipThreads = 1024;
__global__ __launch_bounds__(kClipThreads) void adamw_clip_kernel(const double* part, uint32_t parts, float max_norm, float* norm, float* scale) {
    __shared__ double sh[kClipThreads / 64];
    double mine = 0.0;
    for (uint32_t k = threadIdx.x; k < parts; k += kClipThreads) mine += gptr(part)[k];
    const double sum = block_sum(mine, sh, kClipThreads / 64);
    if (threadIdx.x) return;
    const double x = sqrt(sum);
    *gptr(norm) = (float)x;
    *gptr(scale) = x < INFINITY ? (float)fmin(1.0, (double)max_norm / (x + 1e-6)) : NAN;
}

// -------------------------------------------------------------------- host ----

struct Span {
    uintptr_t lo, hi;
    int tensor;
    const char* what;
    bool written;
};

uint64_t up256(uint64_t n) { return (n + 255) / 256 * 256; }

opt_status check_hparams(const opt_adamw_hparams* hp) {
    if (!hp) return fail(OPT_EINVAL, "hp is NULL");
    if (!(hp->lr >= 0) || !(hp->lr < INFINITY)) return fail(OPT_EINVAL, "lr must be >= 0 and finite");
    if (!(hp->beta1 >= 0 && hp->beta1 < 1 && hp->beta2 >= 0 && hp->beta2 < 1))
        return fail(OPT_EINVAL, "beta1 and beta2 must be in [0, 1)");
    if ((float)hp->beta1 >= 1.f || (float)hp->beta2 >= 1.f) return fail(OPT_EUNSUPPORTED, "beta1 or beta2 rounds to 1 in fp32");
    if (!((float)hp->eps > 0.f) || !((float)hp->eps < INFINITY)) return fail(OPT_EINVAL, "eps must be positive and finite in fp32");
    return OPT_OK;
}

opt_status check_sizes(const opt_adamw_desc* d, int32_t count) {
    if (!d) return fail(OPT_EINVAL, "descs is NULL");
    if (count < 1 || count > kMostTensors) return fail(OPT_EINVAL, "count must be in [1, %d]", kMostTensors);
    uint64_t chunks = 0;
    for (int i = 0; i < count; ++i) {
        const opt_adamw_desc& x = d[i];
        if (x.n < 0) return fail(OPT_EINVAL, "tensor %d: n must be >= 0", i);
        if (x.n > kMostElements) return fail(OPT_EUNSUPPORTED, "tensor %d: more than 2^35 elements", i);
        if (x.state_bits != 32 && x.state_bits != 8) return fail(OPT_EUNSUPPORTED, "tensor %d: state_bits must be 32 or 8", i);
        if (!train_dtype(x.G_dtype)) return fail(OPT_EUNSUPPORTED, "tensor %d: G_dtype must be OPT_F32, OPT_BF16 or OPT_F16", i);
        if (x.W16 && x.W16_dtype != OPT_BF16 && x.W16_dtype != OPT_F16)
            return fail(OPT_EUNSUPPORTED, "tensor %d: W16_dtype must be OPT_BF16 or OPT_F16", i);
        if (!(x.lr_scale >= 0.f && x.lr_scale < INFINITY && x.weight_decay >= 0.f && x.weight_decay < INFINITY))
            return fail(OPT_EINVAL, "tensor %d: lr_scale and weight_decay must be >= 0 and finite", i);
        chunks += (uint64_t)((x.n + kChunk - 1) / kChunk);
    }
    if (chunks > (uint64_t)most_blocks(kThreads)) return fail(OPT_EUNSUPPORTED, "too many elements in one group");
    return OPT_OK;
}

opt_status check_pointers(const opt_adamw_desc* d, int32_t count, std::vector<Span>& spans) {
    for (int i = 0; i < count; ++i) {
        const opt_adamw_desc& x = d[i];
        const bool narrow = x.state_bits == 8;
        if (!narrow && (x.m_scale || x.v_scale))
            return fail(OPT_EINVAL, "tensor %d: m_scale and v_scale go with states of 8 bits", i);
        if (x.n == 0) continue;
        const uint64_t n = (uint64_t)x.n, blocks = (n + OPT_ADAMW_BLOCK - 1) / OPT_ADAMW_BLOCK, state = narrow ? 1 : 4;
        const struct { const void* p; uint64_t each, n; const char* what; bool written, needed; } ts[] = {
            {x.W, 4, n, "W", true, true}, {x.G, (uint64_t)train_bytes(x.G_dtype), n, "G", false, true},
            {x.m, state, n, "m", true, true}, {x.v, state, n, "v", true, true},
            {x.m_scale, 4, blocks, "m_scale", true, narrow}, {x.v_scale, 4, blocks, "v_scale", true, narrow},
            {x.W16, 2, n, "W16", true, false}};
        for (const auto& t : ts) {
            if (!t.p && t.needed) return fail(OPT_EINVAL, "tensor %d: %s is NULL", i, t.what);
            if (!t.p) continue;
            if (!train_aligned(t.p, t.each)) return fail(OPT_EINVAL, "tensor %d: %s is not aligned to its element", i, t.what);
            spans.push_back({(uintptr_t)t.p, (uintptr_t)t.p + t.each * t.n, i, t.what, t.written});
        }
    }
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
    // the furthest end so far of what is written, and of gradients
    const Span *out = nullptr, *in = nullptr;
    for (const Span& s : spans) {
        const Span* hit = out && out->hi > s.lo ? out : s.written && in && in->hi > s.lo ? in : nullptr;
        if (hit) return fail(OPT_EINVAL, "tensors overlap: %s of tensor %d and %s of tensor %d", hit->what, hit->tensor, s.what, s.tensor);
        const Span*& last = s.written ? out : in;
        if (!last || s.hi > last->hi) last = &s;
    }
    return OPT_OK;
}

struct Layout {
    uint64_t segs, chunks, part, bytes;
    uint32_t count[kKinds], total;   // chunks of each kind, in the table's order
};
int kind_of(const opt_adamw_desc& x) { return (x.state_bits == 8 ? 3 : 0) + x.G_dtype; }
static_assert(OPT_F32 == 0 && OPT_BF16 == 1 && OPT_F16 == 2, "kind_of counts types");
Layout layout_of(const opt_adamw_desc* d, int32_t count) {
    Layout l = {};
    for (int i = 0; i < count; ++i) l.count[kind_of(d[i])] += (uint32_t)((d[i].n + kChunk - 1) / kChunk);
    for (const uint32_t n : l.count) l.total += n;
    l.chunks = up256(sizeof(Seg) * (uint64_t)count);
    l.part = l.chunks + up256(sizeof(Chunk) * (uint64_t)l.total);
    l.bytes = l.part + up256(sizeof(double) * kNormBlocks * kKinds);
    return l;
}

opt_status hip_fail(hipError_t e, const char* what) { return fail(OPT_EHIP, "%s: %s", what, hipGetErrorString(e)); }

}  // namespace
}  // namespace matopt

struct opt_adamw_s {
    opt_adamw_hparams hp;
    matopt::Layout at;
    char* ws;
    int device;
    int64_t t;
};

namespace matopt {
namespace {

opt_status check_group(opt_adamw_t g) {
    if (!g) return fail(OPT_EINVAL, "group is NULL");
    int cur = -1;
    const hipError_t e = hipGetDevice(&cur);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    if (cur != g->device) return fail(OPT_ESTATE, "group was created on device %d, current device is %d", g->device, cur);
    return train_pending();
}

opt_status create(const opt_adamw_desc* d, int32_t count, const opt_adamw_hparams* hp, void* ws, uint64_t bytes, void* stream, opt_adamw_t* out) {
    std::vector<Span> spans;
    if (opt_status st = check_pointers(d, count, spans)) return st;
    const Layout l = layout_of(d, count);
    if (bytes < l.bytes)
        return fail(OPT_ENOWS, "workspace of %llu bytes, %llu needed", (unsigned long long)bytes, (unsigned long long)l.bytes);
    if (!ws || !train_aligned(ws, 256)) return fail(OPT_EINVAL, "workspace is NULL or not 256-byte aligned");
    for (const Span& s : spans)
        if (s.lo < (uintptr_t)ws + l.bytes && (uintptr_t)ws < s.hi)
            return fail(OPT_EINVAL, "tensor %d: %s overlaps the workspace", s.tensor, s.what);
    if (stream) {
        hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
        const hipError_t e = hipStreamIsCapturing((hipStream_t)stream, &capture);
        if (e != hipSuccess) return hip_fail(e, "hipStreamIsCapturing");
        if (capture != hipStreamCaptureStatusNone) return fail(OPT_ESTATE, "a group is not created while its stream is captured");
    }
    std::vector<char> image(l.part, 0);
    Seg* segs = (Seg*)image.data();
    Chunk* chunks = (Chunk*)(image.data() + l.chunks);
    uint32_t at[kKinds] = {};
    for (int k = 1; k < kKinds; ++k) at[k] = at[k - 1] + l.count[k - 1];
    for (int i = 0; i < count; ++i) {
        const opt_adamw_desc& x = d[i];
        segs[i] = {x.W, x.G, x.m, x.v, x.m_scale, x.v_scale, x.W16, x.n, x.lr_scale, x.weight_decay,
                   x.W16 ? x.W16_dtype : -1, (uint32_t)i};
        for (int64_t c = 0; c * kChunk < x.n; ++c) chunks[at[kind_of(x)]++] = {(uint32_t)i, (uint32_t)c};
    }
    opt_adamw_s g = {*hp, l, (char*)ws, -1, 0};
    if (opt_status st = train_pending()) return st;
    hipError_t e = hipGetDevice(&g.device);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    e = hipMemcpyAsync(ws, image.data(), image.size(), hipMemcpyHostToDevice, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "hipMemcpyAsync(table)");
    e = hipStreamSynchronize((hipStream_t)stream);   // a step may run on another stream
    if (e != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
    *out = new opt_adamw_s(g);
    return OPT_OK;
}

}  // namespace
}  // namespace matopt

using namespace matopt;

extern "C" {

opt_status opt_adamw_workspace_size(const opt_adamw_desc* descs, int32_t count, uint64_t* bytes) {
    if (!bytes) return fail(OPT_EINVAL, "bytes is NULL");
    if (opt_status st = check_sizes(descs, count)) return st;
    *bytes = layout_of(descs, count).bytes;
    return OPT_OK;
}

opt_status opt_adamw_create(const opt_adamw_desc* descs, int32_t count, const opt_adamw_hparams* hp, void* workspace,
                            uint64_t workspace_bytes, void* stream, opt_adamw_t* out) {
    if (!out) return fail(OPT_EINVAL, "out is NULL");
    *out = nullptr;
    if (opt_status st = check_sizes(descs, count)) return st;
    if (opt_status st = check_hparams(hp)) return st;
    try {
        return create(descs, count, hp, workspace, workspace_bytes, stream, out);
    } catch (const std::exception& e) {
        return fail(OPT_ESTATE, "out of host memory: %s", e.what());
    }
}

opt_status opt_adamw_grad_norm(opt_adamw_t g, float max_norm, float* norm, float* scale, void* stream) {
    if (!(max_norm > 0.f)) return fail(OPT_EINVAL, "max_norm must be positive");
    for (const float* p : {norm, scale})
        if (!p || !train_aligned(p, 4)) return fail(OPT_EINVAL, "norm or scale is NULL or not aligned to 4 bytes");
    if (opt_status st = check_group(g)) return st;
    double* part = (double*)(g->ws + g->at.part);
    const Chunk* chunks = (const Chunk*)(g->ws + g->at.chunks);
    uint32_t parts = 0;
    for (int k = 0; k < kKinds; ++k) {
        const uint32_t count = g->at.count[k], blocks = count < kNormBlocks ? count : kNormBlocks;
        if (count == 0) continue;
        auto* kernel = k % 3 == OPT_F32 ? adamw_norm_kernel<float> : k % 3 == OPT_BF16 ? adamw_norm_kernel<__bf16> : adamw_norm_kernel<_Float16>;
        kernel<<<blocks, kThreads, 0, (hipStream_t)stream>>>((const Seg*)g->ws, chunks, count, part + parts);
        chunks += count, parts += blocks;
    }
    adamw_clip_kernel<<<1, kClipThreads, 0, (hipStream_t)stream>>>(part, parts, max_norm, norm, scale);
    return train_launched("gradient norm");
}

opt_status opt_adamw_step(opt_adamw_t g, const float* grad_scale, const opt_rng* rng, const int64_t* device_step, void* stream) {
    if (!train_aligned(grad_scale, 4)) return fail(OPT_EINVAL, "grad_scale is not aligned to 4 bytes");
    if (!train_aligned(device_step, 8)) return fail(OPT_EINVAL, "device_step is not aligned to 8 bytes");
    if (opt_status st = check_group(g)) return st;
    if (g->at.count[3] + g->at.count[4] + g->at.count[5] && !rng) return fail(OPT_EINVAL, "states of 8 bits need an rng");
    g->t += 1;
    const opt_adamw_hparams& hp = g->hp;
    StepArgs a = {};
    a.segs = (const Seg*)g->ws;
    a.chunks = (const Chunk*)(g->ws + g->at.chunks);
    a.grad_scale = grad_scale, a.device_step = device_step;
    a.b1 = (float)hp.beta1, a.ob1 = (float)(1 - hp.beta1), a.b2 = (float)hp.beta2, a.ob2 = (float)(1 - hp.beta2);
    a.eps = (float)hp.eps, a.lr = (float)hp.lr;
    a.log_b1 = std::log(hp.beta1), a.log_b2 = std::log(hp.beta2);
    a.c1 = (float)(-1 / std::expm1((double)g->t * a.log_b1));
    a.c2 = (float)(1 / std::sqrt(-std::expm1((double)g->t * a.log_b2)));
    a.rng = make_drop(0.f, rng);
    void (*const kernels[kKinds])(StepArgs) = {adamw_kernel<float>,  adamw_kernel<__bf16>,  adamw_kernel<_Float16>,
                                               adamw8_kernel<float>, adamw8_kernel<__bf16>, adamw8_kernel<_Float16>};
    for (int k = 0; k < kKinds; ++k) {
        const uint32_t count = g->at.count[k];
        if (count) kernels[k]<<<count, kThreads, 0, (hipStream_t)stream>>>(a);
        a.chunks += count;
    }
    return train_launched("AdamW step");
}

opt_status opt_adamw_get_step(opt_adamw_t g, int64_t* t) {
    if (!g || !t) return fail(OPT_EINVAL, "group or t is NULL");
    *t = g->t;
    return OPT_OK;
}

opt_status opt_adamw_set_step(opt_adamw_t g, int64_t t) {
    if (!g) return fail(OPT_EINVAL, "group is NULL");
    if (t < 0) return fail(OPT_EINVAL, "t must be >= 0");
    g->t = t;
    return OPT_OK;
}

opt_status opt_adamw_set_lr(opt_adamw_t g, double lr) {
    if (!g) return fail(OPT_EINVAL, "group is NULL");
    if (!(lr >= 0) || !(lr < INFINITY)) return fail(OPT_EINVAL, "lr must be >= 0 and finite");
    g->hp.lr = lr;
    return OPT_OK;
}

void opt_adamw_destroy(opt_adamw_t g) { delete g; }

}  // extern "C"
