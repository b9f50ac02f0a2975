// What the training-pass operators share: storage types, vector accesses of
// any alignment, the counter-based generator and workgroup sums.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmem.h"
#include "matopt_train.h"

namespace matopt {

opt_status fail(opt_status st, const char* fmt, ...);

inline opt_status train_launched(const char* what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? OPT_OK : fail(OPT_EHIP, "%s launch: %s", what, hipGetErrorString(e));
}

inline opt_status train_pending() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? OPT_OK : fail(OPT_EHIP, "pending HIP error: %s", hipGetErrorString(e));
}

// Workgroups of `threads` in one launch: its threads are counted in 32 bits.
constexpr int64_t most_blocks(int threads) { return (int64_t(1) << 31) / threads; }

inline bool train_dtype(int32_t d) { return d == OPT_F32 || d == OPT_BF16 || d == OPT_F16; }
inline int64_t train_bytes(int32_t d) { return d == OPT_F32 ? 4 : 2; }
inline bool train_aligned(const void* p, uintptr_t a) { return (uintptr_t)p % a == 0; }

// --------------------------------------------------------- storage types ----

template <class T>
__device__ __forceinline__ float to_f32(T x) { return (float)x; }

// Round to nearest even (the conversion instructions' mode).
template <class T>
__device__ __forceinline__ T from_f32(float x) { return (T)x; }

// Eight consecutive elements. The alignment is one element's: the hardware
// loads and stores 16 bytes at any address of a global buffer, so a row that
// starts at an odd column costs no other code path.
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        const auto* q = (const __attribute__((address_space(1))) f32x4u*)p;
        const f32x4u a = q[0], b = q[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = a[e], f[e + 4] = b[e];
    } else {
        typedef T t8 __attribute__((ext_vector_type(8)));
        const u32x4u r = *(const __attribute__((address_space(1))) u32x4u*)p;
        const t8 a = __builtin_bit_cast(t8, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (float)a[e];
    }
}

template <class T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        auto* q = (__attribute__((address_space(1))) f32x4u*)p;
        f32x4u a, b;
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = f[e], b[e] = f[e + 4];
        q[0] = a;
        q[1] = b;
    } else {
        typedef T t8 __attribute__((ext_vector_type(8)));
        t8 a;
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = (T)f[e];
        *(__attribute__((address_space(1))) u32x4u*)p = __builtin_bit_cast(u32x4u, a);
    }
}

// The first n (0 .. 8) of eight elements; the others read as `fill`.
template <class T>
__device__ __forceinline__ void load_n(const T* p, int n, float (&f)[8], float fill = 0.f) {
    if (n >= 8) {
        load8(p, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = e < n ? (float)gptr(p)[e] : fill;
    }
}

template <class T>
__device__ __forceinline__ void store_n(T* p, int n, const float (&f)[8]) {
    if (n >= 8) {
        store8(p, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) gptr(p)[e] = (T)f[e];
    }
}

// ------------------------------------------------------------- generator ----

// What a kernel needs of opt_rng and p: keep where bits >= drop, times scale.
struct Drop {
    uint64_t seed, offset;
    const uint64_t* device_offset;
    uint32_t drop;
    float scale;
};

inline Drop make_drop(float p, const opt_rng* rng) {
    Drop d = {};
    d.drop = (uint32_t)(65536.0 * (double)p + 0.5);
    d.scale = (float)(65536.0 / (65536.0 - (double)d.drop));
    if (rng) d.seed = rng->seed, d.offset = rng->offset, d.device_offset = rng->device_offset;
    return d;
}

inline opt_status check_drop(float p, const opt_rng* rng) {
    if (!(p >= 0.f && p < 1.f)) return fail(OPT_EINVAL, "p must be in [0, 1)");
    if (p > 0.f && !rng) return fail(OPT_EINVAL, "rng is NULL and p > 0");
    if (65536.0 * (double)p + 0.5 >= 65536.0) return fail(OPT_EUNSUPPORTED, "p rounds to 1 in steps of 2^-16");
    return OPT_OK;
}

// Philox4x32-10: four 32-bit words per 128-bit counter and 64-bit key. A
// round is two 32 x 32 -> 64 bit products; for eight elements of 16 bits each
// that is 2.5 products an element, where 32 bits each would take 5: at HBM
// speed the products, which run at a quarter of the vector rate, are what a
// dropout kernel has to hide.
__device__ __forceinline__ void philox(uint32_t c0, uint32_t c1, uint64_t offset, uint64_t seed, uint32_t (&out)[4]) {
    uint32_t x0 = c0, x1 = c1, x2 = (uint32_t)offset, x3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
        x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
        x1 = (uint32_t)b;
        x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
        x3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    out[0] = x0, out[1] = x1, out[2] = x2, out[3] = x3;
}

__device__ __forceinline__ uint64_t drop_offset(const Drop& d) {
    return d.offset + (d.device_offset ? *gptr(d.device_offset) : 0);
}

// Elements 8 g .. 8 g + 7 of row r through dropout, in place. The product is
// kept apart from any later sum (no fused multiply-add): the operators define
// it as rounded to fp32.
__device__ __forceinline__ void drop8(const Drop& d, uint64_t offset, uint32_t g, uint32_t r, float (&f)[8]) {
#pragma clang fp contract(off)
    uint32_t w[4];
    philox(g, r, offset, d.seed, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t bits = e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu;
        f[e] = bits >= d.drop ? f[e] * d.scale : 0.f;
    }
}

// ------------------------------------------------------- workgroup sums ----

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
    return x;
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int m = 32; m; m >>= 1) x = fmaxf(x, __shfl_xor(x, m));
    return x;
}

}  // namespace matopt
