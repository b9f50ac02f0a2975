// Dropout and layer norm (HBM-bandwidth bound).
//
// dropout:     y = residual + keep scale x
// layer norm:  h = residual + keep scale x;  y = (h - mean) rstd w + b
//   backward:  z = dy w;  g = rstd (z - mean(z) - xh mean(z xh)) + dh
//              dx = keep scale g;  dres = g;  dw = sum dy xh;  db = sum dy
//
// Every tensor is read once and written once. A row of the norm lives in the
// registers of 16, 32 or 64 threads (up to 512 columns) or of a workgroup of
// 128 to 1024 threads, eight columns a thread (sixteen past 8192 columns: more a
// thread leaves the backward pass short of registers), so mean and variance
// are two passes over registers: the variance is the sum of squares about the
// mean, with no cancellation. The weight's and bias's gradients are column
// sums: a thread keeps its columns over all rows of its workgroup, each
// workgroup writes one partial row, and a second kernel adds the partial rows
// in a fixed order.
#include "train.h"

namespace matopt {
namespace {

// --------------------------------------------------------------- dropout ----

constexpr int kDropThreads = 256;
constexpr int kDropPer = 4;   // groups of eight elements per thread: four independent loads in flight

// i / d for i < 2^32 by one 64-bit product: m = floor(2^(32+s) / d) + 1 with
// s = ceil(log2 d) is exact over that range (d - 2^(32+s) mod d <= 2^s).
struct FastDiv {
    uint64_t m;
    uint32_t d, s;
};
FastDiv fast_div(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    const unsigned __int128 one = 1;
    return {(uint64_t)((one << (32 + s)) / d + 1), d, s};
}
__device__ __forceinline__ uint32_t div_by(uint32_t i, FastDiv f) {
    // m has up to 33 bits: its top bit's product is i itself
    const uint64_t lo = (uint64_t)i * (uint32_t)f.m;
    const uint64_t hi = (lo >> 32) + ((f.m >> 32) ? (uint64_t)i * (uint32_t)(f.m >> 32) : 0);
    return (uint32_t)(hi >> f.s);
}

template <class T, bool RES>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(uint32_t rows, int64_t cols, FastDiv groups,
                                                               const T* x, int64_t ldx, const T* res, int64_t ldr,
                                                               T* y, int64_t ldy, Drop d, uint32_t first_row) {
    const uint64_t total = (uint64_t)rows * groups.d;
    const uint64_t base = (uint64_t)blockIdx.x * (kDropThreads * kDropPer) + threadIdx.x;
    const uint64_t offset = drop_offset(d);
    float f[kDropPer][8], q[kDropPer][8];
    uint32_t row[kDropPer], g[kDropPer];
    int n[kDropPer];
#pragma unroll
    for (int i = 0; i < kDropPer; ++i) {
        const uint64_t at = base + (uint64_t)i * kDropThreads;
        n[i] = 0;
        if (at >= total) continue;
        row[i] = div_by((uint32_t)at, groups);
        g[i] = (uint32_t)at - row[i] * groups.d;
        const int64_t left = cols - 8 * (int64_t)g[i];
        n[i] = left < 8 ? (int)left : 8;
        load_n(x + (int64_t)row[i] * ldx + 8 * (int64_t)g[i], n[i], f[i]);
        if constexpr (RES) load_n(res + (int64_t)row[i] * ldr + 8 * (int64_t)g[i], n[i], q[i]);
    }
#pragma unroll
    for (int i = 0; i < kDropPer; ++i) {
        if (n[i] == 0) continue;
        if (d.drop) drop8(d, offset, g[i], row[i] + first_row, f[i]);
        if constexpr (RES) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[i][e] = q[i][e] + f[i][e];
        }
        store_n(y + (int64_t)row[i] * ldy + 8 * (int64_t)g[i], n[i], f[i]);
    }
}

template <class T>
void dropout_launch(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* res, int64_t ldr, void* y,
                    int64_t ldy, const Drop& d, hipStream_t s) {
    // Launches of at most 2^31 groups, so that positions fit 32 bits; a row of
    // more groups than that (cols < 2^34) is a launch of its own.
    const int64_t groups = (cols + 7) / 8;
    const int64_t most = (int64_t(1) << 31) / groups;
    const int64_t step = most < 1 ? 1 : most;
    const FastDiv f = fast_div((uint32_t)groups);
    for (int64_t r = 0; r < rows; r += step) {
        const int64_t n = rows - r < step ? rows - r : step;
        const int64_t blocks = (n * groups + kDropThreads * kDropPer - 1) / (kDropThreads * kDropPer);
        const T* xp = (const T*)x + r * ldx;
        const T* rp = res ? (const T*)res + r * ldr : nullptr;
        T* yp = (T*)y + r * ldy;
        if (res)
            dropout_kernel<T, true><<<dim3((uint32_t)blocks), kDropThreads, 0, s>>>((uint32_t)n, cols, f, xp, ldx, rp,
                                                                                   ldr, yp, ldy, d, (uint32_t)r);
        else
            dropout_kernel<T, false><<<dim3((uint32_t)blocks), kDropThreads, 0, s>>>((uint32_t)n, cols, f, xp, ldx,
                                                                                    rp, ldr, yp, ldy, d, (uint32_t)r);
    }
}

// ------------------------------------------------------------ layer norm ----

constexpr int norm_threads(int tpr) { return tpr <= 64 ? 256 : tpr; }   // of a workgroup

// Sum of one value per thread over the TPR threads of a row: a part of a
// wavefront, or the whole workgroup. The callers rotate `slot`, so one barrier
// per sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float (*part)[16], int slot) {
#pragma unroll
    for (int m = (TPR < 64 ? TPR : 64) / 2; m; m >>= 1) x += __shfl_xor(x, m);
    if constexpr (TPR <= 64) return x;
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < TPR / 64; ++k) s += part[slot][k];
    return s;
}

// Columns of this thread's group i: eight, none, or with EIGHTS unset (cols
// not a multiple of 8) some. With EIGHTS a group costs one mask, else eight.
template <int TPR, bool EIGHTS>
__device__ __forceinline__ int group_cols(int cols, int t, int i) {
    const int left = cols - 8 * (t + i * TPR);
    if constexpr (EIGHTS) return left > 0 ? 8 : 0;
    return left < 0 ? 0 : left < 8 ? left : 8;
}
template <bool EIGHTS, class T>
__device__ __forceinline__ void load_g(const T* p, int n, float (&f)[8]) {
    if constexpr (!EIGHTS) return load_n(p, n, f);
    if (n) {
        load8(p, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
    }
}
template <bool EIGHTS, class T>
__device__ __forceinline__ void store_g(T* p, int n, const float (&f)[8]) {
    if constexpr (!EIGHTS) return store_n(p, n, f);
    if (n) store8(p, f);
}

// H: h's and the residual's type. VPT: groups of eight columns per thread.
template <class T, class H, int TPR, int VPT, bool EIGHTS>
__global__ __launch_bounds__(norm_threads(TPR)) void norm_forward_kernel(
    uint32_t rows, int cols, const T* x, int64_t ldx, const H* res, int64_t ldr, const float* w, const float* b,
    float eps, Drop d, T* y, int64_t ldy, H* h, int64_t ldh, float* mean_out, float* rstd_out, uint32_t first) {
    __shared__ float part[2][16];
    const int t = threadIdx.x % TPR;
    const uint32_t row = first + blockIdx.x * (norm_threads(TPR) / TPR) + threadIdx.x / TPR;
    if (row >= rows) return;   // all threads of a row; where it takes the workgroup, none is past the rows
    float f[VPT][8];
    int n[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (t + i * TPR);
        n[i] = group_cols<TPR, EIGHTS>(cols, t, i);
        load_g<EIGHTS>(x + (int64_t)row * ldx + c, n[i], f[i]);
    }
    if (h) {   // a residual or dropout: h is a tensor of its own
        const uint64_t offset = drop_offset(d);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (n[i] == 0) continue;
            const int c = 8 * (t + i * TPR);
            float q[8];
            if (res) load_g<EIGHTS>(res + (int64_t)row * ldr + c, n[i], q);
            if (d.drop) drop8(d, offset, (uint32_t)(c >> 3), row, f[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (res) f[i][e] = q[e] + f[i][e];
                f[i][e] = to_f32(from_f32<H>(f[i][e]));   // the norm is of what is stored
                if (e >= n[i]) f[i][e] = 0.f;
            }
            store_g<EIGHTS>(h + (int64_t)row * ldh + c, n[i], f[i]);
        }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += f[i][e];
    const float mean = row_sum<TPR>(s, part, 0) / (float)cols;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[i][e] = e < n[i] ? f[i][e] - mean : 0.f;
            s += f[i][e] * f[i][e];
        }
    const float rstd = 1.f / sqrtf(row_sum<TPR>(s, part, 1) / (float)cols + eps);
    if (t == 0) {
        gptr(mean_out)[row] = mean;
        gptr(rstd_out)[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (n[i] == 0) continue;
        const int c = 8 * (t + i * TPR);
        float wv[8], bv[8];
        load_g<EIGHTS>(w + c, n[i], wv);
        if (b) load_g<EIGHTS>(b + c, n[i], bv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[i][e] = f[i][e] * rstd * wv[e];
            if (b) f[i][e] += bv[e];
        }
        store_g<EIGHTS>(y + (int64_t)row * ldy + c, n[i], f[i]);
    }
}

// Rows blockIdx.x * R + k, then gridDim.x * R further, with R rows at a time. part_w and part_b hold one row of `cols`
// column sums per workgroup.
template <class T, class H, int TPR, int VPT, bool EIGHTS>
__global__ __launch_bounds__(norm_threads(TPR), 4) void norm_backward_kernel(
    uint32_t rows, int cols, const T* dy, int64_t lddy, const H* h, int64_t ldh, const H* dh, int64_t lddh,
    const float* w, const float* mean_in, const float* rstd_in, Drop d, T* dx, int64_t lddx, H* dres, int64_t lddres,
    float* part_w, float* part_b) {
    constexpr int R = norm_threads(TPR) / TPR;
    __shared__ float part[4][16];
    __shared__ float cross[R > 1 ? norm_threads(TPR) * 8 : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    int n[VPT];
    // The weight stays in registers over the rows, but for the widest rows,
    // where 128 registers a thread have no room for it and each row reads it
    // again (from L2).
    constexpr bool KEEP_W = VPT == 1;
    float dw[VPT][8] = {}, db[VPT][8] = {}, wv[KEEP_W ? VPT : 1][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (t + i * TPR);
        n[i] = group_cols<TPR, EIGHTS>(cols, t, i);
        if constexpr (KEEP_W) load_g<EIGHTS>(w + c, n[i], wv[i]);
    }
    const uint64_t offset = drop_offset(d);
    const float inv = 1.f / (float)cols;
    int slot = 0;
    for (uint32_t row = blockIdx.x * R + sub; row < rows; row += gridDim.x * R) {
        const float mean = gptr(mean_in)[row], rstd = gptr(rstd_in)[row];
        float z[VPT][8], xh[VPT][8];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (t + i * TPR);
            load_g<EIGHTS>(dy + (int64_t)row * lddy + c, n[i], z[i]);
            load_g<EIGHTS>(h + (int64_t)row * ldh + c, n[i], xh[i]);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if constexpr (!KEEP_W) load_g<EIGHTS>(w + 8 * (t + i * TPR), n[i], wv[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[i][e] = e < n[i] ? (xh[i][e] - mean) * rstd : 0.f;
                dw[i][e] += z[i][e] * xh[i][e];
                db[i][e] += z[i][e];
                z[i][e] *= wv[KEEP_W ? i : 0][e];
                s1 += z[i][e];
                s2 += z[i][e] * xh[i][e];
            }
        }
        s1 = row_sum<TPR>(s1, part, slot) * inv;
        s2 = row_sum<TPR>(s2, part, slot + 1) * inv;
        slot ^= 2;   // the next row's sums go to the other pair: a slower wavefront may still read this one
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if constexpr (VPT > 1) __builtin_amdgcn_sched_barrier(0);   // one group's values at a time
            if (n[i] == 0) continue;
            const int c = 8 * (t + i * TPR);
            float g[8], q[8];
            if (dh) load_g<EIGHTS>(dh + (int64_t)row * lddh + c, n[i], q);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] = rstd * (z[i][e] - s1 - xh[i][e] * s2);
                if (dh) g[e] += q[e];
            }
            if (dres) store_g<EIGHTS>(dres + (int64_t)row * lddres + c, n[i], g);
            if (dx) {
                if (d.drop) drop8(d, offset, (uint32_t)(c >> 3), row, g);
                store_g<EIGHTS>(dx + (int64_t)row * lddx + c, n[i], g);
            }
        }
    }
    // one partial row per workgroup: the sums of its R rows' threads meet in
    // LDS and are added in order
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (t + i * TPR);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float(&v)[8] = k ? db[i] : dw[i];
            float* out = (k ? part_b : part_w) + (int64_t)blockIdx.x * cols + c;
            if constexpr (R > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 8; ++e) cross[e * norm_threads(TPR) + threadIdx.x] = v[e];
                __syncthreads();
                if (sub != 0) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int j = 1; j < R; ++j) v[e] += cross[e * norm_threads(TPR) + j * TPR + t];
            }
            store_g<EIGHTS>(out, n[i], v);
        }
    }
}

// Column sums of the partial rows: 32 columns per workgroup (a 128-byte line),
// 32 slices of the rows, eight loads of a slice in flight, added in slice
// order. For 1024 rows of 2048 columns 4.5 us; 16 columns 6.8, 8 columns 12.5;
// one load in flight and 16 slices 20.
constexpr int kSumCols = 32, kSumSlices = 32;
__global__ __launch_bounds__(kSumCols* kSumSlices) void norm_sum_kernel(int parts, int cols, const float* part_w,
                                                                        const float* part_b, float* dw, float* db) {
    __shared__ float sh[kSumSlices][kSumCols];
    const float* src = blockIdx.y ? part_b : part_w;
    float* dst = blockIdx.y ? db : dw;
    const int lane = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
    const int c = blockIdx.x * kSumCols + lane;
    float s = 0.f;
    if (c < cols)
        for (int r0 = slice; r0 < parts; r0 += 8 * kSumSlices) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = r0 + k * kSumSlices;
                v[k] = r < parts ? gptr(src)[(int64_t)r * cols + c] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
    sh[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < kSumSlices; ++k) s += sh[k][lane];
        gptr(dst)[c] = s;
    }
}

// Workgroups of the backward pass, and partial rows: what the GPU holds at
// once at 128 registers a thread (1024 threads a CU), so that all run through
// their rows together; past 1024 of them each has four rows at least, so that
// the partial rows stay a small part of what is moved (4099 rows of 1000:
// 2048 workgroups 15 + 7 us, 1024 15 + 4; 32000 rows of 777: 89 and 130).
int norm_blocks(int64_t rows, int64_t cols) {
    const int per = cols <= 128 ? 16 : cols <= 256 ? 8 : cols <= 512 ? 4 : 1;
    int threads = 256;
    if (cols > 512) threads = cols <= 1024 ? 128 : cols <= 2048 ? 256 : cols <= 4096 ? 512 : 1024;
    const int64_t most = 256 * 1024 / threads;
    int64_t b = (rows + per - 1) / per;
    if (b > 1024) b = b / 4 > 1024 ? b / 4 : 1024;
    return (int)(b < most ? b : most);
}

struct NormFwd {
    uint32_t rows;
    int cols;
    const void *x, *res;
    const float *w, *b;
    void *y, *h;
    int64_t ldx, ldr, ldy, ldh;
    float eps;
    float *mean, *rstd;
    Drop d;
};
struct NormBwd {
    uint32_t rows;
    int cols, blocks;
    const void *dy, *h, *dh;
    const float *w, *mean, *rstd;
    void *dx, *dres;
    int64_t lddy, ldh, lddh, lddx, lddres;
    float *part_w, *part_b;
    Drop d;
};

template <class T, class H, int TPR, int VPT, bool EIGHTS>
void run(const NormFwd& a, hipStream_t s) {
    constexpr int64_t R = norm_threads(TPR) / TPR, most = most_blocks(norm_threads(TPR));
    for (int64_t first = 0; first < a.rows; first += most * R) {
        const int64_t blocks = (a.rows - first + R - 1) / R;
        norm_forward_kernel<T, H, TPR, VPT, EIGHTS>
            <<<dim3((uint32_t)(blocks < most ? blocks : most)), norm_threads(TPR), 0, s>>>(
                a.rows, a.cols, (const T*)a.x, a.ldx, (const H*)a.res, a.ldr, a.w, a.b, a.eps, a.d, (T*)a.y, a.ldy,
                (H*)a.h, a.ldh, a.mean, a.rstd, (uint32_t)first);
    }
}
template <class T, class H, int TPR, int VPT, bool EIGHTS>
void run(const NormBwd& a, hipStream_t s) {
    norm_backward_kernel<T, H, TPR, VPT, EIGHTS><<<dim3(a.blocks), norm_threads(TPR), 0, s>>>(
        a.rows, a.cols, (const T*)a.dy, a.lddy, (const H*)a.h, a.ldh, (const H*)a.dh, a.lddh, a.w, a.mean, a.rstd,
        a.d, (T*)a.dx, a.lddx, (H*)a.dres, a.lddres, a.part_w, a.part_b);
}

template <class T, class H, bool EIGHTS, class A>
void by_width(const A& a, hipStream_t s) {
    if (a.cols <= 128) run<T, H, 16, 1, EIGHTS>(a, s);
    else if (a.cols <= 256) run<T, H, 32, 1, EIGHTS>(a, s);
    else if (a.cols <= 512) run<T, H, 64, 1, EIGHTS>(a, s);
    else if (a.cols <= 1024) run<T, H, 128, 1, EIGHTS>(a, s);
    else if (a.cols <= 2048) run<T, H, 256, 1, EIGHTS>(a, s);
    else if (a.cols <= 4096) run<T, H, 512, 1, EIGHTS>(a, s);
    else if (a.cols <= 8192) run<T, H, 1024, 1, EIGHTS>(a, s);
    else run<T, H, 1024, 2, EIGHTS>(a, s);
}
template <class T, class H, class A>
void by_width(const A& a, hipStream_t s) {
    a.cols % 8 ? by_width<T, H, false>(a, s) : by_width<T, H, true>(a, s);
}

template <class A>
void by_type(int32_t dtype, int32_t h_dtype, const A& a, hipStream_t s) {
    if (dtype == OPT_F32) by_width<float, float>(a, s);
    else if (dtype == OPT_BF16) h_dtype == OPT_F32 ? by_width<__bf16, float>(a, s) : by_width<__bf16, __bf16>(a, s);
    else h_dtype == OPT_F32 ? by_width<_Float16, float>(a, s) : by_width<_Float16, _Float16>(a, s);
}

struct Operand {
    const void* p;
    int64_t ld;
    int32_t dtype;
    const char* name;
};

opt_status check_operand(const Operand& o, int64_t rows, int64_t cols) {
    if (!o.p) return fail(OPT_EINVAL, "%s is NULL", o.name);
    if (o.ld < cols) return fail(OPT_EINVAL, "row stride of %s is below cols", o.name);
    if (rows > 1 && o.ld > (int64_t(1) << 40)) return fail(OPT_EUNSUPPORTED, "row stride of %s is too large", o.name);
    if (!train_aligned(o.p, train_bytes(o.dtype))) return fail(OPT_EINVAL, "%s is not aligned to its element size", o.name);
    return OPT_OK;
}

opt_status check_norm(int64_t rows, int64_t cols, int32_t dtype, int32_t h_dtype, float p, const opt_rng* rng) {
    if (rows < 0 || cols < 1) return fail(OPT_EINVAL, "rows must be >= 0 and cols >= 1");
    if (cols > OPT_MAX_DIM) return fail(OPT_EUNSUPPORTED, "cols must be <= %d", OPT_MAX_DIM);
    if (rows >= int64_t(1) << 31) return fail(OPT_EUNSUPPORTED, "rows must be < 2^31");
    if (!train_dtype(dtype)) return fail(OPT_EUNSUPPORTED, "dtype must be OPT_F32, OPT_BF16 or OPT_F16");
    if (h_dtype != dtype && h_dtype != OPT_F32) return fail(OPT_EUNSUPPORTED, "h_dtype must be dtype or OPT_F32");
    return check_drop(p, rng);
}

}  // namespace
}  // namespace matopt

using namespace matopt;

extern "C" {

opt_status opt_dropout(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t ldx, const void* residual,
                       int64_t ldr, void* y, int64_t ldy, float p, const opt_rng* rng, void* stream) {
    if (rows < 0 || cols < 0) return fail(OPT_EINVAL, "negative dimension");
    if (rows >= int64_t(1) << 32 || cols >= int64_t(1) << 34) return fail(OPT_EUNSUPPORTED, "dimension too large");
    if (!train_dtype(dtype)) return fail(OPT_EUNSUPPORTED, "dtype must be OPT_F32, OPT_BF16 or OPT_F16");
    if (opt_status st = check_drop(p, rng)) return st;
    if (rows == 0 || cols == 0) return OPT_OK;
    if (opt_status st = check_operand({x, ldx, dtype, "x"}, rows, cols)) return st;
    if (opt_status st = check_operand({y, ldy, dtype, "y"}, rows, cols)) return st;
    if (residual)
        if (opt_status st = check_operand({residual, ldr, dtype, "residual"}, rows, cols)) return st;
    if (opt_status st = train_pending()) return st;
    const Drop d = make_drop(p, rng);
    const hipStream_t s = (hipStream_t)stream;
    if (dtype == OPT_F32) dropout_launch<float>(rows, cols, x, ldx, residual, ldr, y, ldy, d, s);
    else if (dtype == OPT_BF16) dropout_launch<__bf16>(rows, cols, x, ldx, residual, ldr, y, ldy, d, s);
    else dropout_launch<_Float16>(rows, cols, x, ldx, residual, ldr, y, ldy, d, s);
    return train_launched("dropout");
}

opt_status opt_layer_norm_forward(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t ldx,
                                  int32_t h_dtype, const void* residual, int64_t ldr, const float* weight,
                                  const float* bias, float eps, float p, const opt_rng* rng, void* y, int64_t ldy,
                                  void* h, int64_t ldh, float* mean, float* rstd, void* stream) {
    if (opt_status st = check_norm(rows, cols, dtype, h_dtype, p, rng)) return st;
    if (!(eps >= 0.f)) return fail(OPT_EINVAL, "eps must be >= 0");
    const bool own_h = residual || p > 0.f;
    if (own_h && !h) return fail(OPT_EINVAL, "h is NULL with a residual or dropout");
    if (!own_h && h) return fail(OPT_EINVAL, "h must be NULL without a residual and dropout: it is x");
    if (rows == 0) return OPT_OK;
    if (opt_status st = check_operand({x, ldx, dtype, "x"}, rows, cols)) return st;
    if (opt_status st = check_operand({y, ldy, dtype, "y"}, rows, cols)) return st;
    if (residual)
        if (opt_status st = check_operand({residual, ldr, h_dtype, "residual"}, rows, cols)) return st;
    if (h)
        if (opt_status st = check_operand({h, ldh, h_dtype, "h"}, rows, cols)) return st;
    if (!weight || !mean || !rstd) return fail(OPT_EINVAL, "weight, mean or rstd is NULL");
    if (!train_aligned(weight, 4) || !train_aligned(bias, 4) || !train_aligned(mean, 4) || !train_aligned(rstd, 4))
        return fail(OPT_EINVAL, "an fp32 vector is not aligned to 4 bytes");
    if (opt_status st = train_pending()) return st;
    NormFwd a = {(uint32_t)rows, (int)cols, x, residual, weight, bias, y, h, ldx, ldr, ldy, ldh, eps, mean, rstd,
                 make_drop(p, rng)};
    by_type(dtype, own_h ? h_dtype : dtype, a, (hipStream_t)stream);
    return train_launched("layer norm");
}

opt_status opt_layer_norm_workspace_size(int64_t rows, int64_t cols, uint64_t* bytes) {
    if (!bytes) return fail(OPT_EINVAL, "bytes is NULL");
    if (opt_status st = check_norm(rows, cols, OPT_F32, OPT_F32, 0.f, nullptr)) return st;
    *bytes = (uint64_t)norm_blocks(rows, cols) * (uint64_t)cols * 8;
    return OPT_OK;
}

opt_status opt_layer_norm_backward(int64_t rows, int64_t cols, int32_t dtype, const void* dy, int64_t lddy,
                                   int32_t h_dtype, const void* h, int64_t ldh, const void* dh, int64_t lddh,
                                   const float* weight, const float* mean, const float* rstd, float p,
                                   const opt_rng* rng, void* dx, int64_t lddx, void* dres, int64_t lddres,
                                   float* dweight, float* dbias, void* workspace, uint64_t workspace_bytes,
                                   void* stream) {
    if (opt_status st = check_norm(rows, cols, dtype, h_dtype, p, rng)) return st;
    if (!dweight) return fail(OPT_EINVAL, "dweight is NULL");
    if (!train_aligned(dweight, 4) || !train_aligned(dbias, 4))
        return fail(OPT_EINVAL, "an fp32 vector is not aligned to 4 bytes");
    if (rows > 0) {
        if (opt_status st = check_operand({dy, lddy, dtype, "dy"}, rows, cols)) return st;
        if (opt_status st = check_operand({h, ldh, h_dtype, "h"}, rows, cols)) return st;
        if (opt_status st = check_operand({dx, lddx, dtype, "dx"}, rows, cols)) return st;
        if (dh)
            if (opt_status st = check_operand({dh, lddh, h_dtype, "dh"}, rows, cols)) return st;
        if (dres)
            if (opt_status st = check_operand({dres, lddres, h_dtype, "dres"}, rows, cols)) return st;
        if (!weight || !mean || !rstd) return fail(OPT_EINVAL, "weight, mean or rstd is NULL");
        if (!train_aligned(weight, 4) || !train_aligned(mean, 4) || !train_aligned(rstd, 4))
            return fail(OPT_EINVAL, "an fp32 vector is not aligned to 4 bytes");
        if (!workspace || !train_aligned(workspace, 256)) return fail(OPT_EINVAL, "workspace is NULL or not 256-byte aligned");
    }
    const int blocks = norm_blocks(rows, cols);
    if (workspace_bytes < (uint64_t)blocks * (uint64_t)cols * 8) return fail(OPT_ENOWS, "workspace too small");
    if (opt_status st = train_pending()) return st;
    const hipStream_t s = (hipStream_t)stream;
    float* part_w = (float*)workspace;
    float* part_b = part_w + (int64_t)blocks * cols;
    if (rows > 0) {
        NormBwd a = {(uint32_t)rows, (int)cols, blocks, dy, h, dh, weight, mean, rstd, dx, dres,
                     lddy, ldh, lddh, lddx, lddres, part_w, part_b, make_drop(p, rng)};
        by_type(dtype, h_dtype, a, s);
    }
    // no rows: no partial rows, the sums are zeros
    norm_sum_kernel<<<dim3((uint32_t)((cols + kSumCols - 1) / kSumCols), dbias ? 2 : 1), kSumCols * kSumSlices, 0, s>>>(
        blocks, (int)cols, part_w, part_b, dweight, dbias);
    return train_launched("layer norm backward");
}

}  // extern "C"
