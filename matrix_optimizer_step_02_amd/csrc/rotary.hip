// Position rotation of queries and keys, and their norms per head with the
// rotation in the same pass (HBM-bandwidth bound).
//
//   rotation:  (a, b) -> s (a cos - b sin, b cos + a sin), angle p f_i of pair i at position p
//   norm:      y = R(x rstd w),  rstd = 1 / sqrt(mean(x^2) + eps)
//   backward:  g = R^T dy,  z = g w,  xh = x rstd,  dx = rstd (z - xh mean(z xh)),  dw = sum g xh
//
// Every tensor is read once and written once. A head's row lies in L lanes of
// a wavefront (a power of two), sixteen elements each: two groups of eight
// that hold the partners of their pairs, so that the rotation needs no other
// lane and the norm one sum over the L lanes. A lane keeps the cosines and
// sines of its eight pairs over the heads of a token.
//
// Angles. What turns is the fraction of a turn, so the frequencies come as
// F_i = round(2^64 f_i / (2 pi)) and p F_i mod 2^64, an integer product, is the
// angle reduced to one turn with an error of |p| 2^-65 turns: a position of
// 2^31 is as exact as position 1, where p f_i in fp32 would be off by 2^31 2^-24
// = 128 radians. The top 32 bits go into polynomials on an eighth of a turn to
// each side (the Taylor series, cut below 2^-29).
#include "train.h"

#include <utility>

namespace matopt {
namespace {

constexpr int kThreads = 256;

struct Heads {
    char* p;
    int64_t batch, token, head;   // strides in elements
};

struct Rope {
    const uint64_t* turns;
    const void* pos;   // NULL: first + index along the tokens
    int64_t first, pos_batch, pos_token;
    float scale;
    int32_t pos64, rot, pairs, inverse;
};

// One of the two tensors of a call. in: x; dy: the gradient of y (backward);
// out: y or dx; rstd: (token, head).
struct Side {
    Heads in, dy, out;
    const float* w;
    float *rstd, *part;
    int32_t heads, parts, blocks;   // parts of `per` heads; backward: workgroups
};

struct Args {
    Side q, k;
    Rope r;
    uint32_t tokens, total, first;   // per sequence; in all, or up to this launch's end; this launch's first
    int32_t dim, per, shift;         // heads to a thread's turn, log2 of L
    float eps;
};

// ------------------------------------------------------------------ angles ----

// sin and cos of `top` 2^-32 turns. Within 2^-29 of a turn to the nearest
// quarter, x = 2 pi r 2^-32 in [-pi / 4, pi / 4]; the terms left out are below
// 2e-9 (sine) and 2e-10 (cosine), and both are within 2 2^-24 of the exact ones.
__device__ __forceinline__ void turn(uint32_t top, float& sn, float& cs) {
    const uint32_t quarter = (top + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(top - (quarter << 30)) * 1.46291807926715968105e-9f;   // 2 pi 2^-32
    const float z = x * x;
    float s = fmaf(z, 1.f / 362880, -1.f / 5040);
    s = fmaf(z, s, 1.f / 120);
    s = fmaf(z, s, -1.f / 6);
    s = fmaf(z * s, x, x);
    float c = fmaf(z, -1.f / 3628800, 1.f / 40320);
    c = fmaf(z, c, -1.f / 720);
    c = fmaf(z, c, 1.f / 24);
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.f);
    const bool odd = quarter & 1;
    const float a = odd ? c : s, b = odd ? s : c;
    sn = quarter & 2 ? -a : a;
    cs = (quarter + 1) & 2 ? -b : b;
}

// A lane's sixteen elements: n_a from a, n_b from b, and its first pair.
struct Unit {
    int a, b, na, nb, f, nf;   // nf = 0: not rotated
};
__device__ __forceinline__ int upto8(int n) { return n < 0 ? 0 : n < 8 ? n : 8; }
__device__ __forceinline__ Unit unit_of(int u, int dim, int rot, bool pairs) {
    Unit x = {};
    const int half = rot / 2, turned = pairs ? (rot + 15) / 16 : (half + 7) / 8;
    if (u < turned) {
        x.f = 8 * u;
        x.nf = upto8(half - x.f);
        if (pairs) {
            x.a = 16 * u, x.b = x.a + 8;
            x.na = upto8(rot - x.a), x.nb = upto8(rot - x.b);
        } else {
            x.a = 8 * u, x.b = half + x.a;
            x.na = x.nb = x.nf;
        }
    } else {
        x.a = rot + 16 * (u - turned), x.b = x.a + 8;
        x.na = upto8(dim - x.a), x.nb = upto8(dim - x.b);
    }
    return x;
}

__device__ __forceinline__ void angles(const Rope& r, const Unit& x, uint32_t b, uint32_t t, float (&c)[8], float (&s)[8]) {
    if (x.nf == 0) return;
    int64_t p = r.first + t;
    if (r.pos) {
        const int64_t at = b * r.pos_batch + t * r.pos_token;
        p = r.pos64 ? gptr((const int64_t*)r.pos)[at] : (int64_t)gptr((const int32_t*)r.pos)[at];
    }
    if (r.inverse) p = (int64_t)(0 - (uint64_t)p);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint64_t f = e < x.nf ? gptr(r.turns)[x.f + e] : 0;
        turn((uint32_t)((uint64_t)p * f >> 32), s[e], c[e]);
        s[e] *= r.scale;
        c[e] *= r.scale;
    }
}

__device__ __forceinline__ void rotate(bool pairs, const Unit& x, const float (&c)[8], const float (&s)[8], float (&a)[8], float (&b)[8]) {
    if (x.nf == 0) return;
    if (pairs) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y = a[2 * e], z = a[2 * e + 1];
            a[2 * e] = y * c[e] - z * s[e];
            a[2 * e + 1] = z * c[e] + y * s[e];
            y = b[2 * e], z = b[2 * e + 1];
            b[2 * e] = y * c[e + 4] - z * s[e + 4];
            b[2 * e + 1] = z * c[e + 4] + y * s[e + 4];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float y = a[e], z = b[e];
            a[e] = y * c[e] - z * s[e];
            b[e] = z * c[e] + y * s[e];
        }
    }
}

// Groups of a row, whole ones or none (EIGHTS) or any number of elements, as
// stored: loads in flight take half the registers in 16 bits.
template <class T>
using Eight = T __attribute__((ext_vector_type(8)));
template <bool EIGHTS, class T>
__device__ __forceinline__ Eight<T> get(const T* p, int n) {
    typedef T at1 __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    Eight<T> f = {};
    if (EIGHTS ? n != 0 : n >= 8) {
        f = *(const __attribute__((address_space(1))) at1*)p;
    } else if constexpr (!EIGHTS) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) f[e] = gptr(p)[e];
    }
    return f;
}
template <class T>
__device__ __forceinline__ void widen(const Eight<T>& x, float (&f)[8], float mul = 1.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)x[e] * mul;
}
template <bool EIGHTS, class T>
__device__ __forceinline__ void put(T* p, int n, const float (&f)[8]) {
    if constexpr (!EIGHTS) return store_n(p, n, f);
    if (n) store8(p, f);
}

template <class T>
__device__ __forceinline__ T* row_of(const Heads& t, uint32_t b, uint32_t s, int h) {
    return (T*)t.p + (int64_t)b * t.batch + (int64_t)s * t.token + (int64_t)h * t.head;
}

// Sum over the 2^shift lanes of a row.
__device__ __forceinline__ float lanes_sum(float x, int shift) {
    for (int m = (1 << shift) >> 1; m; m >>= 1) x += __shfl_xor(x, m);
    return x;
}

// ----------------------------------------------------------------- forward ----

// A thread's turn is one token and `per` heads of q or of k, HB at a time.
constexpr int kHeadsAhead = 4;   // heads whose loads are in flight together
template <class T, bool EIGHTS, bool NORM>
__global__ __launch_bounds__(kThreads) void heads_forward_kernel(Args a) {
    constexpr int HB = kHeadsAhead;
    const int u = threadIdx.x & ((1 << a.shift) - 1);
    const uint32_t item = blockIdx.x * (kThreads >> a.shift) + (threadIdx.x >> a.shift);
    const uint32_t parts = a.q.parts + a.k.parts, row = a.first + item / parts;
    if (row >= a.total) return;
    int part = item % parts;
    const bool is_k = part >= a.q.parts;
    const Side& x = is_k ? a.k : a.q;
    if (is_k) part -= a.q.parts;
    const uint32_t b = row / a.tokens, t = row - b * a.tokens;
    const Unit n = unit_of(u, a.dim, a.r.rot, a.r.pairs);
    float c[8], s[8];
    Eight<float> wa, wb;
    const int end = min((part + 1) * a.per, x.heads);
    for (int h0 = part * a.per; h0 < end; h0 += HB) {
        Eight<T> ra[HB], rb[HB];
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            if (h0 + i >= end) continue;
            const T* p = row_of<T>(x.in, b, t, h0 + i);
            ra[i] = get<EIGHTS>(p + n.a, n.na);
            rb[i] = get<EIGHTS>(p + n.b, n.nb);
        }
        if (h0 == part * a.per) {
            if constexpr (NORM) {
                wa = get<EIGHTS>(x.w + n.a, n.na);
                wb = get<EIGHTS>(x.w + n.b, n.nb);
            }
            angles(a.r, n, b, t, c, s);
        }
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            if (h0 + i >= end) continue;
            float fa[8], fb[8];
            widen<T>(ra[i], fa);
            widen<T>(rb[i], fb);
            if constexpr (NORM) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += fa[e] * fa[e] + fb[e] * fb[e];
                const float rstd = 1.f / sqrtf(lanes_sum(sum, a.shift) / (float)a.dim + a.eps);
                if (u == 0) gptr(x.rstd)[(int64_t)row * x.heads + h0 + i] = rstd;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    fa[e] = fa[e] * rstd * wa[e];
                    fb[e] = fb[e] * rstd * wb[e];
                }
            }
            rotate(a.r.pairs, n, c, s, fa, fb);
            T* p = row_of<T>(x.out, b, t, h0 + i);
            put<EIGHTS>(p + n.a, n.na, fa);
            put<EIGHTS>(p + n.b, n.nb, fb);
        }
    }
}

// ---------------------------------------------------------------- backward ----

// Workgroups [0, q.blocks) take q, the others k. Each keeps its lanes' weight
// gradients over all its turns and leaves one row of them.
template <class T, bool EIGHTS>
__global__ __launch_bounds__(kThreads, 3) void heads_backward_kernel(Args a) {
    constexpr int HB = sizeof(T) == 4 ? 1 : 2;
    __shared__ float cross[16][kThreads + 1];
    const int u = threadIdx.x & ((1 << a.shift) - 1), slots = kThreads >> a.shift;
    const bool is_k = (int)blockIdx.x >= a.q.blocks;
    const Side& x = is_k ? a.k : a.q;
    const uint32_t block = blockIdx.x - (is_k ? a.q.blocks : 0);
    const Unit n = unit_of(u, a.dim, a.r.rot, a.r.pairs);
    const float inv = 1.f / (float)a.dim;
    float da[8] = {}, db[8] = {};
    const Eight<float> wa = get<EIGHTS>(x.w + n.a, n.na), wb = get<EIGHTS>(x.w + n.b, n.nb);
    const uint64_t items = (uint64_t)a.total * x.parts;
    for (uint64_t item = (uint64_t)block * slots + (threadIdx.x >> a.shift); item < items; item += (uint64_t)x.blocks * slots) {
        const uint32_t row = x.parts == 1 ? (uint32_t)item : (uint32_t)(item / (uint32_t)x.parts);
        const int part = (int)(item - (uint64_t)row * x.parts);
        const uint32_t b = row / a.tokens, t = row - b * a.tokens;
        float c[8], s[8];
        const int end = min((part + 1) * a.per, x.heads);
        for (int h0 = part * a.per; h0 < end; h0 += HB) {
            Eight<T> rxa[HB], rxb[HB], rga[HB], rgb[HB];
            float rstd[HB];
#pragma unroll
            for (int i = 0; i < HB; ++i) {
                if (h0 + i >= end) continue;
                const T* p = row_of<T>(x.in, b, t, h0 + i);
                const T* g = row_of<T>(x.dy, b, t, h0 + i);
                rxa[i] = get<EIGHTS>(p + n.a, n.na);
                rxb[i] = get<EIGHTS>(p + n.b, n.nb);
                rga[i] = get<EIGHTS>(g + n.a, n.na);
                rgb[i] = get<EIGHTS>(g + n.b, n.nb);
                rstd[i] = gptr(x.rstd)[(int64_t)row * x.heads + h0 + i];
            }
            if (h0 == part * a.per) angles(a.r, n, b, t, c, s);
#pragma unroll
            for (int i = 0; i < HB; ++i) {
                if (h0 + i >= end) continue;
                float xa[8], xb[8], ga[8], gb[8], sum = 0.f;
                widen<T>(rga[i], ga);
                widen<T>(rgb[i], gb);
                rotate(a.r.pairs, n, c, s, ga, gb);
                widen<T>(rxa[i], xa, rstd[i]);
                widen<T>(rxb[i], xb, rstd[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    da[e] += ga[e] * xa[e];
                    db[e] += gb[e] * xb[e];
                    ga[e] *= wa[e];
                    gb[e] *= wb[e];
                    sum += ga[e] * xa[e] + gb[e] * xb[e];
                }
                sum = lanes_sum(sum, a.shift) * inv;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ga[e] = (ga[e] - xa[e] * sum) * rstd[i];
                    gb[e] = (gb[e] - xb[e] * sum) * rstd[i];
                }
                T* p = row_of<T>(x.out, b, t, h0 + i);
                put<EIGHTS>(p + n.a, n.na, ga);
                put<EIGHTS>(p + n.b, n.nb, gb);
            }
        }
    }
    // the slots' sums meet in LDS and are added in order
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cross[e][threadIdx.x] = da[e];
        cross[e + 8][threadIdx.x] = db[e];
    }
    __syncthreads();
    for (int v = threadIdx.x; v < 16 << a.shift; v += kThreads) {
        const int e = v >> a.shift, at = v & ((1 << a.shift) - 1);
        float sum = 0.f;
        for (int j = 0; j < slots; ++j) sum += cross[e][(j << a.shift) + at];
        const Unit m = unit_of(at, a.dim, a.r.rot, a.r.pairs);
        const int col = e < 8 ? m.a + e : m.b + e - 8, left = e < 8 ? m.na - e : m.nb - (e - 8);
        if (left > 0) gptr(x.part)[(int64_t)block * a.dim + col] = sum;
    }
}

// Column sums of the partial rows: 16 columns a workgroup, 64 slices of the
// rows, added in slice order. blockIdx.y: q or k.
constexpr int kSumCols = 16, kSumSlices = 64;
__global__ __launch_bounds__(kSumCols* kSumSlices) void heads_sum_kernel(int dim, int rows_q, int rows_k, const float* part_q,
                                                                         const float* part_k, float* dwq, float* dwk) {
    __shared__ float sh[kSumSlices][kSumCols];
    const int rows = blockIdx.y ? rows_k : rows_q;
    const float* src = blockIdx.y ? part_k : part_q;
    float* dst = blockIdx.y ? dwk : dwq;
    const int lane = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols, c = blockIdx.x * kSumCols + lane;
    float s = 0.f;
    if (c < dim)
        for (int r0 = slice; r0 < rows; r0 += 8 * kSumSlices) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = r0 + k * kSumSlices;
                v[k] = r < rows ? gptr(src)[(int64_t)r * dim + c] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
    sh[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && c < dim) {
#pragma unroll
        for (int k = 1; k < kSumSlices; ++k) s += sh[k][lane];
        gptr(dst)[c] = s;
    }
}

// -------------------------------------------------------------------- host ----

constexpr int kMaxHeadDim = 512;
constexpr int kBackwardBlocks = 768;   // what the GPU holds at once at three wavefronts a SIMD

int units_of(int dim, int rot, bool pairs) {
    const int turned = pairs ? (rot + 15) / 16 : (rot / 2 + 7) / 8;
    return turned + (dim - rot + 15) / 16;
}
bool whole_groups(int dim, int rot, bool pairs) {
    return (dim - rot) % 8 == 0 && (pairs ? rot : rot / 2) % 8 == 0;
}

opt_status check_heads(const opt_heads_desc* d) {
    if (!d) return fail(OPT_EINVAL, "desc is NULL");
    if (!train_dtype(d->dtype)) return fail(OPT_EUNSUPPORTED, "dtype must be OPT_F32, OPT_BF16 or OPT_F16");
    if (d->batch < 0 || d->tokens < 0) return fail(OPT_EINVAL, "negative batch or tokens");
    if (d->heads < 1 || d->kv_heads < 0) return fail(OPT_EINVAL, "heads must be >= 1 and kv_heads >= 0");
    if (d->heads > 65536 || d->kv_heads > 65536) return fail(OPT_EUNSUPPORTED, "more than 65536 heads");
    if (d->head_dim < 1) return fail(OPT_EINVAL, "head_dim must be >= 1");
    if (d->head_dim > kMaxHeadDim) return fail(OPT_EUNSUPPORTED, "head_dim must be <= %d", kMaxHeadDim);
    if (d->batch > INT32_MAX || d->tokens > INT32_MAX || d->batch * d->tokens > INT32_MAX)
        return fail(OPT_EUNSUPPORTED, "batch * tokens must be < 2^31");
    return OPT_OK;
}

opt_status check_rope(const opt_heads_desc* d, const opt_rotary* r, bool inverse, Rope& x) {
    x = {};
    if (!r) return OPT_OK;
    if (r->rot < 2 || r->rot % 2 || r->rot > d->head_dim)
        return fail(OPT_EINVAL, "rot must be even and in [2, head_dim]");
    if (r->layout != OPT_ROTARY_HALF && r->layout != OPT_ROTARY_PAIRS)
        return fail(OPT_EINVAL, "layout must be OPT_ROTARY_HALF or OPT_ROTARY_PAIRS");
    if (!(r->scale > 0.f) || !(r->scale < INFINITY)) return fail(OPT_EINVAL, "scale must be positive and finite");
    if (!r->turns || !train_aligned(r->turns, 8)) return fail(OPT_EINVAL, "turns is NULL or not aligned to 8 bytes");
    if (!train_aligned(r->positions, r->positions_i64 ? 8 : 4)) return fail(OPT_EINVAL, "positions is not aligned to its element");
    if (r->position_batch_stride < 0 || r->position_token_stride < 0) return fail(OPT_EINVAL, "negative stride of positions");
    x.turns = r->turns, x.pos = r->positions, x.first = r->first;
    x.pos_batch = r->position_batch_stride, x.pos_token = r->position_token_stride;
    x.scale = r->scale, x.pos64 = r->positions_i64 != 0, x.rot = r->rot, x.pairs = r->layout == OPT_ROTARY_PAIRS;
    x.inverse = inverse;
    return OPT_OK;
}

opt_status check_tensor(const opt_heads_desc* d, const opt_attention_tensor* t, const char* name, int heads, bool output, Heads& x) {
    if (!t) return fail(OPT_EINVAL, "%s is NULL", name);
    if (!t->data) return fail(OPT_EINVAL, "%s has no data", name);
    if (!train_aligned(t->data, train_bytes(d->dtype))) return fail(OPT_EINVAL, "%s is not aligned to its element", name);
    if (t->batch_stride < 0 || t->token_stride < 0 || t->head_stride < 0) return fail(OPT_EINVAL, "negative stride of %s", name);
    if (output) {   // axes by stride: each has to step over what lies within it
        struct { int64_t n, stride; } x[3] = {{d->batch, t->batch_stride}, {d->tokens, t->token_stride}, {heads, t->head_stride}};
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2 - i; ++j)
                if (x[j].stride > x[j + 1].stride) std::swap(x[j], x[j + 1]);
        __int128 size = d->head_dim;
        for (const auto& y : x) {
            if (y.n <= 1) continue;
            if (y.stride < size) return fail(OPT_EINVAL, "rows of %s overlap", name);
            size += (__int128)y.stride * (y.n - 1);
        }
    }
    x = {(char*)t->data, t->batch_stride, t->token_stride, t->head_stride};
    return OPT_OK;
}

opt_status check_vector(const float* p, const char* name) {
    if (!p || !train_aligned(p, 4)) return fail(OPT_EINVAL, "%s is NULL or not aligned to 4 bytes", name);
    return OPT_OK;
}

void set_rows(const opt_heads_desc* d, Args& a) {
    a.tokens = (uint32_t)d->tokens, a.total = (uint32_t)(d->batch * d->tokens), a.dim = d->head_dim;
    a.q.heads = d->heads, a.k.heads = d->kv_heads;
    const int units = units_of(a.dim, a.r.rot, a.r.pairs);
    a.shift = 0;
    while ((1 << a.shift) < units) ++a.shift;
}

// Heads to a thread's turn: all that share a token's angles, but fewer where
// the launch would leave CUs without work.
void set_per(Args& a, int64_t want, int step) {
    const int most = a.q.heads > a.k.heads ? a.q.heads : a.k.heads;
    const auto parts = [&](int heads, int per) { return (heads + per - 1) / per; };
    a.per = most;
    while (a.per > step && ((int64_t)a.total * (parts(a.q.heads, a.per) + parts(a.k.heads, a.per)) << a.shift) < want)
        a.per = (a.per / 2 + step - 1) / step * step;
    while (a.per > 1 && ((int64_t)a.total * (parts(a.q.heads, a.per) + parts(a.k.heads, a.per)) << a.shift) < want / 8) a.per = (a.per + 1) / 2;
    a.q.parts = parts(a.q.heads, a.per), a.k.parts = parts(a.k.heads, a.per);
}

template <class T, bool NORM>
void forward(Args a, hipStream_t s) {
    set_per(a, 1 << 19, kHeadsAhead);
    const int64_t parts = a.q.parts + a.k.parts, slots = kThreads >> a.shift;
    int64_t step = most_blocks(kThreads) * slots / parts;   // tokens of one launch
    const int64_t total = a.total;
    for (int64_t first = 0; first < total; first += step) {
        const int64_t n = total - first < step ? total - first : step;
        a.first = (uint32_t)first, a.total = (uint32_t)(first + n);   // none of the next launch's: out may be in
        const dim3 g((uint32_t)((n * parts + slots - 1) / slots));
        if (whole_groups(a.dim, a.r.rot, a.r.pairs)) heads_forward_kernel<T, true, NORM><<<g, kThreads, 0, s>>>(a);
        else heads_forward_kernel<T, false, NORM><<<g, kThreads, 0, s>>>(a);
    }
}
template <bool NORM>
void forward(int32_t dtype, const Args& a, hipStream_t s) {
    if (dtype == OPT_F32) forward<float, NORM>(a, s);
    else if (dtype == OPT_BF16) forward<__bf16, NORM>(a, s);
    else forward<_Float16, NORM>(a, s);
}

// Workgroups of the backward pass for each tensor, in proportion to its heads.
void set_blocks(Args& a) {
    set_per(a, 1 << 18, 2);
    const int64_t slots = kThreads >> a.shift, heads = a.q.heads + a.k.heads;
    for (Side* x : {&a.q, &a.k}) {
        const int64_t need = ((int64_t)a.total * x->parts + slots - 1) / slots;
        int64_t share = kBackwardBlocks * (int64_t)x->heads / heads;
        if (share < 1) share = 1;
        x->blocks = (int)(x->heads == 0 ? 0 : need < share ? need : share);
    }
}
template <class T>
void backward(const Args& a, hipStream_t s) {
    const dim3 g((uint32_t)(a.q.blocks + a.k.blocks));
    if (whole_groups(a.dim, a.r.rot, a.r.pairs)) heads_backward_kernel<T, true><<<g, kThreads, 0, s>>>(a);
    else heads_backward_kernel<T, false><<<g, kThreads, 0, s>>>(a);
}

}  // namespace
}  // namespace matopt

using namespace matopt;

extern "C" {

opt_status opt_rotary_apply(const opt_heads_desc* d, const opt_rotary* r, int32_t inverse, const opt_attention_tensor* q,
                            const opt_attention_tensor* k, const opt_attention_tensor* yq, const opt_attention_tensor* yk,
                            void* stream) {
    if (opt_status st = check_heads(d)) return st;
    if (!r) return fail(OPT_EINVAL, "rotary is NULL");
    Args a = {};
    if (opt_status st = check_rope(d, r, inverse != 0, a.r)) return st;
    if (d->batch == 0 || d->tokens == 0) return OPT_OK;
    if (opt_status st = check_tensor(d, q, "q", d->heads, false, a.q.in)) return st;
    if (opt_status st = check_tensor(d, yq, "yq", d->heads, true, a.q.out)) return st;
    if (d->kv_heads) {
        if (opt_status st = check_tensor(d, k, "k", d->kv_heads, false, a.k.in)) return st;
        if (opt_status st = check_tensor(d, yk, "yk", d->kv_heads, true, a.k.out)) return st;
    }
    if (opt_status st = train_pending()) return st;
    set_rows(d, a);
    forward<false>(d->dtype, a, (hipStream_t)stream);
    return train_launched("rotary");
}

opt_status opt_qk_norm_forward(const opt_heads_desc* d, const opt_rotary* r, const opt_attention_tensor* q,
                               const opt_attention_tensor* k, const float* q_weight, const float* k_weight, float eps,
                               const opt_attention_tensor* yq, const opt_attention_tensor* yk, float* q_rstd, float* k_rstd,
                               void* stream) {
    if (opt_status st = check_heads(d)) return st;
    Args a = {};
    if (opt_status st = check_rope(d, r, false, a.r)) return st;
    if (!(eps >= 0.f) || !(eps < INFINITY)) return fail(OPT_EINVAL, "eps must be >= 0 and finite");
    if (d->batch == 0 || d->tokens == 0) return OPT_OK;
    if (opt_status st = check_tensor(d, q, "q", d->heads, false, a.q.in)) return st;
    if (opt_status st = check_tensor(d, yq, "yq", d->heads, true, a.q.out)) return st;
    if (opt_status st = check_vector(q_weight, "q_weight")) return st;
    if (opt_status st = check_vector(q_rstd, "q_rstd")) return st;
    if (d->kv_heads) {
        if (opt_status st = check_tensor(d, k, "k", d->kv_heads, false, a.k.in)) return st;
        if (opt_status st = check_tensor(d, yk, "yk", d->kv_heads, true, a.k.out)) return st;
        if (opt_status st = check_vector(k_weight, "k_weight")) return st;
        if (opt_status st = check_vector(k_rstd, "k_rstd")) return st;
    }
    if (opt_status st = train_pending()) return st;
    a.q.w = q_weight, a.k.w = k_weight, a.q.rstd = q_rstd, a.k.rstd = k_rstd, a.eps = eps;
    set_rows(d, a);
    forward<true>(d->dtype, a, (hipStream_t)stream);
    return train_launched("qk norm");
}

opt_status opt_qk_norm_workspace_size(const opt_heads_desc* d, uint64_t* bytes) {
    if (!bytes) return fail(OPT_EINVAL, "bytes is NULL");
    if (opt_status st = check_heads(d)) return st;
    *bytes = 0;
    if (d->batch * d->tokens) *bytes = ((uint64_t)(kBackwardBlocks + 2) * d->head_dim * 4 + 255) / 256 * 256;
    return OPT_OK;
}

opt_status opt_qk_norm_backward(const opt_heads_desc* d, const opt_rotary* r, const opt_attention_tensor* dyq,
                                const opt_attention_tensor* dyk, const opt_attention_tensor* q, const opt_attention_tensor* k,
                                const float* q_weight, const float* k_weight, const float* q_rstd, const float* k_rstd,
                                const opt_attention_tensor* dq, const opt_attention_tensor* dk, float* dq_weight,
                                float* dk_weight, void* workspace, uint64_t workspace_bytes, void* stream) {
    uint64_t need = 0;
    if (opt_status st = opt_qk_norm_workspace_size(d, &need)) return st;
    Args a = {};
    if (opt_status st = check_rope(d, r, true, a.r)) return st;
    if (opt_status st = check_vector(dq_weight, "dq_weight")) return st;
    if (d->kv_heads)
        if (opt_status st = check_vector(dk_weight, "dk_weight")) return st;
    if (need) {
        if (opt_status st = check_tensor(d, dyq, "dyq", d->heads, false, a.q.dy)) return st;
        if (opt_status st = check_tensor(d, q, "q", d->heads, false, a.q.in)) return st;
        if (opt_status st = check_tensor(d, dq, "dq", d->heads, true, a.q.out)) return st;
        if (opt_status st = check_vector(q_weight, "q_weight")) return st;
        if (opt_status st = check_vector(q_rstd, "q_rstd")) return st;
        if (d->kv_heads) {
            if (opt_status st = check_tensor(d, dyk, "dyk", d->kv_heads, false, a.k.dy)) return st;
            if (opt_status st = check_tensor(d, k, "k", d->kv_heads, false, a.k.in)) return st;
            if (opt_status st = check_tensor(d, dk, "dk", d->kv_heads, true, a.k.out)) return st;
            if (opt_status st = check_vector(k_weight, "k_weight")) return st;
            if (opt_status st = check_vector(k_rstd, "k_rstd")) return st;
        }
        if (workspace_bytes < need)
            return fail(OPT_ENOWS, "workspace of %llu bytes, %llu needed", (unsigned long long)workspace_bytes,
                        (unsigned long long)need);
        if (!workspace || !train_aligned(workspace, 256)) return fail(OPT_EINVAL, "workspace is NULL or not 256-byte aligned");
    }
    if (opt_status st = train_pending()) return st;
    hipStream_t s = (hipStream_t)stream;
    a.q.w = q_weight, a.k.w = k_weight, a.q.rstd = (float*)q_rstd, a.k.rstd = (float*)k_rstd;
    if (need) {
        set_rows(d, a);
        set_blocks(a);
        a.q.part = (float*)workspace;
        a.k.part = a.q.part + (int64_t)a.q.blocks * a.dim;
        if (d->dtype == OPT_F32) backward<float>(a, s);
        else if (d->dtype == OPT_BF16) backward<__bf16>(a, s);
        else backward<_Float16>(a, s);
    }
    const dim3 g((uint32_t)((d->head_dim + kSumCols - 1) / kSumCols), d->kv_heads ? 2 : 1);
    heads_sum_kernel<<<g, kSumCols * kSumSlices, 0, s>>>(d->head_dim, a.q.blocks, a.k.blocks, a.q.part, a.k.part, dq_weight,
                                                         dk_weight);
    return train_launched("qk norm backward");
}

}  // extern "C"
