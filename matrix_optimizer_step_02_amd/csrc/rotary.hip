// Position rotation of queries and keys, and their norms per head with the
// rotation in the same pass (HBM-bandwidth bound).
//
//   rotation:  (a, b) -> s (a cos - b sin, b cos + a sin), angle p f_i of pair i at position p
//   norm:      y = R(x rstd w),  rstd = 1 / sqrt(mean(x^2) + eps)
//   backward:  g = R^T dy,  z = g w,  xh = x rstd,  dx = rstd (z - xh mean(z xh)),  dw = sum g xh
//
// Every tensor is read once and written once. A head's row lies in L lanes of
// a wavefront (a power of two), two groups of G elements each that hold the
// partners of their pairs, so that the rotation needs no other lane and the norm
// one sum over the L lanes. A lane keeps the cosines and sines of its pairs over
// the heads of a token. G is 4, or less where the turned part and the rest are not
// made of whole groups of 4: a group is one load or store then too. (16384 tokens, 16
// / 8 heads of 128 in bf16, forward and backward: rotation 79 us, norm 100; groups
// of 8 83 and 102.)
//
// Angles. What turns is the fraction of a turn, so the frequencies come as
// F_i = round(2^64 f_i / (2 pi)) and p F_i mod 2^64, an integer product, is the
// angle reduced to one turn with an error of |p| 2^-65 turns: a position of
// 2^31 is as exact as position 1, where p f_i in fp32 would be off by 2^31 2^-24
// = 128 radians. The top 32 bits go into polynomials on an eighth of a turn to
// each side (the Taylor series, cut below 2^-29).
#include "places.h"
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
    int32_t dim, per, shift, group;  // heads to a thread's turn, log2 of L, group_of
    float eps;
};

// ------------------------------------------------------------------ angles ----

// sin and cos of `top` 2^-32 turns. r = top less the nearest quarter lies within 2^29,
// an eighth of a turn, and x = 2 pi r 2^-32 in [-pi / 4, pi / 4]; the terms left out are below
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

// A lane's two groups of G elements: n_a of them from a, n_b from b, and its first
// pair of n_f (0: not turned).
struct Unit {
    int a, b, na, nb, f, nf;
};
template <int G>
__device__ __forceinline__ int upto(int n) { return n < 0 ? 0 : n < G ? n : G; }
template <int G>
__device__ __forceinline__ Unit unit_of(int u, int dim, int rot, bool pairs) {
    Unit x = {};
    const int half = rot / 2, turned = pairs ? (rot + 2 * G - 1) / (2 * G) : (half + G - 1) / G;
    if (u < turned) {
        x.f = G * u;
        x.nf = upto<G>(half - x.f);
        if (pairs) {
            x.a = 2 * G * u, x.b = x.a + G;
            x.na = upto<G>(rot - x.a), x.nb = upto<G>(rot - x.b);
        } else {
            x.a = G * u, x.b = half + x.a;
            x.na = x.nb = x.nf;
        }
    } else {
        x.a = rot + 2 * G * (u - turned), x.b = x.a + G;
        x.na = upto<G>(dim - x.a), x.nb = upto<G>(dim - x.b);
    }
    return x;
}

template <int G>
__device__ __forceinline__ void angles(const Rope& r, const Unit& x, uint32_t b, uint32_t t, float (&c)[G], float (&s)[G]) {
    if (x.nf == 0) return;
    int64_t p = r.first + t;
    if (r.pos) {
        const int64_t at = b * r.pos_batch + t * r.pos_token;
        p = r.pos64 ? gptr((const int64_t*)r.pos)[at] : (int64_t)gptr((const int32_t*)r.pos)[at];
    }
    if (r.inverse) p = (int64_t)(0 - (uint64_t)p);
#pragma unroll
    for (int e = 0; e < G; ++e) {
        const uint64_t f = e < x.nf ? gptr(r.turns)[x.f + e] : 0;
        turn((uint32_t)((uint64_t)p * f >> 32), s[e], c[e]);
        s[e] *= r.scale;
        c[e] *= r.scale;
    }
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float y = a, z = b;
    a = y * c - z * s;
    b = z * c + y * s;
}
template <int G>
__device__ __forceinline__ void rotate(bool pairs, const Unit& x, const float (&c)[G], const float (&s)[G], float (&a)[G], float (&b)[G]) {
    if (x.nf == 0) return;
    if (pairs) {
        if constexpr (G == 1) {   // the pair is the lane's two elements
            turn_pair(a[0], b[0], c[0], s[0]);
        } else {
#pragma unroll
            for (int e = 0; e < G / 2; ++e) {
                turn_pair(a[2 * e], a[2 * e + 1], c[e], s[e]);
                turn_pair(b[2 * e], b[2 * e + 1], c[e + G / 2], s[e + G / 2]);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < G; ++e) turn_pair(a[e], b[e], c[e], s[e]);
    }
}

// Groups of a row, whole ones or none (WHOLE) or any number of elements, as
// stored: loads in flight take half the registers in 16 bits.
template <class T, int G>
struct Group {
    T v __attribute__((ext_vector_type(G)));
};
template <bool WHOLE, int G, class T>
__device__ __forceinline__ Group<T, G> get(const T* p, int n) {
    typedef T vec __attribute__((ext_vector_type(G), aligned(sizeof(T))));
    Group<T, G> f = {};
    if (WHOLE ? n != 0 : n >= G) {
        if constexpr (G == 1) {
            f.v[0] = *gptr(p);
        } else {
            f.v = *(const __attribute__((address_space(1))) vec*)p;
        }
    } else if constexpr (!WHOLE) {
#pragma unroll
        for (int e = 0; e < G; ++e)
            if (e < n) f.v[e] = gptr(p)[e];
    }
    return f;
}
template <class T, int G>
__device__ __forceinline__ void widen(const Group<T, G>& x, float (&f)[G], float mul = 1.f) {
#pragma unroll
    for (int e = 0; e < G; ++e) f[e] = (float)x.v[e] * mul;
}
template <bool WHOLE, int G, class T>
__device__ __forceinline__ void put(T* p, int n, const float (&f)[G]) {
    typedef T vec __attribute__((ext_vector_type(G), aligned(sizeof(T))));
    if (WHOLE ? n != 0 : n >= G) {
        if constexpr (G == 1) {
            *gptr(p) = (T)f[0];
        } else {
            vec x;
#pragma unroll
            for (int e = 0; e < G; ++e) x[e] = (T)f[e];
            *(__attribute__((address_space(1))) vec*)p = x;
        }
    } else if constexpr (!WHOLE) {
#pragma unroll
        for (int e = 0; e < G; ++e)
            if (e < n) gptr(p)[e] = (T)f[e];
    }
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
// heads whose loads are in flight together: 79 us as above, four 96, eight 99
constexpr int kHeadsAhead = 2;
template <class T, int G, bool WHOLE, bool NORM>
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
    const Unit n = unit_of<G>(u, a.dim, a.r.rot, a.r.pairs);
    float c[G], s[G];
    Group<float, G> wa, wb;
    const int end = min((part + 1) * a.per, x.heads);
    for (int h0 = part * a.per; h0 < end; h0 += HB) {
        Group<T, G> ra[HB], rb[HB];
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            if (h0 + i >= end) continue;
            const T* p = row_of<T>(x.in, b, t, h0 + i);
            ra[i] = get<WHOLE, G>(p + n.a, n.na);
            rb[i] = get<WHOLE, G>(p + n.b, n.nb);
        }
        if (h0 == part * a.per) {
            if constexpr (NORM) {
                wa = get<WHOLE, G>(x.w + n.a, n.na);
                wb = get<WHOLE, G>(x.w + n.b, n.nb);
            }
            angles(a.r, n, b, t, c, s);
        }
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            if (h0 + i >= end) continue;
            float fa[G], fb[G];
            widen<T, G>(ra[i], fa);
            widen<T, G>(rb[i], fb);
            if constexpr (NORM) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < G; ++e) sum += fa[e] * fa[e] + fb[e] * fb[e];
                const float rstd = 1.f / sqrtf(lanes_sum(sum, a.shift) / (float)a.dim + a.eps);
                if (u == 0) gptr(x.rstd)[(int64_t)row * x.heads + h0 + i] = rstd;
#pragma unroll
                for (int e = 0; e < G; ++e) {
                    fa[e] = fa[e] * rstd * wa.v[e];
                    fb[e] = fb[e] * rstd * wb.v[e];
                }
            }
            rotate(a.r.pairs, n, c, s, fa, fb);
            T* p = row_of<T>(x.out, b, t, h0 + i);
            put<WHOLE, G>(p + n.a, n.na, fa);
            put<WHOLE, G>(p + n.b, n.nb, fb);
        }
    }
}

// ---------------------------------------------------------------- backward ----

// Workgroups [0, q.blocks) take q, the others k. Each keeps its lanes' weight
// gradients over all its turns and leaves one row of them.
template <class T, int G, bool WHOLE>
__global__ __launch_bounds__(kThreads, 4) void heads_backward_kernel(Args a) {
    constexpr int HB = sizeof(T) == 4 ? 1 : 2;
    __shared__ float cross[2 * G][kThreads + 1];
    const int u = threadIdx.x & ((1 << a.shift) - 1), slots = kThreads >> a.shift;
    const bool is_k = (int)blockIdx.x >= a.q.blocks;
    const Side& x = is_k ? a.k : a.q;
    const uint32_t block = blockIdx.x - (is_k ? a.q.blocks : 0);
    const Unit n = unit_of<G>(u, a.dim, a.r.rot, a.r.pairs);
    const float inv = 1.f / (float)a.dim;
    float da[G] = {}, db[G] = {};
    const Group<float, G> wa = get<WHOLE, G>(x.w + n.a, n.na), wb = get<WHOLE, G>(x.w + n.b, n.nb);
    const uint64_t items = (uint64_t)a.total * x.parts;
    for (uint64_t item = (uint64_t)block * slots + (threadIdx.x >> a.shift); item < items; item += (uint64_t)x.blocks * slots) {
        const uint32_t row = x.parts == 1 ? (uint32_t)item : (uint32_t)(item / (uint32_t)x.parts);
        const int part = (int)(item - (uint64_t)row * x.parts);
        const uint32_t b = row / a.tokens, t = row - b * a.tokens;
        float c[G], s[G];
        const int end = min((part + 1) * a.per, x.heads);
        for (int h0 = part * a.per; h0 < end; h0 += HB) {
            Group<T, G> rxa[HB], rxb[HB], rga[HB], rgb[HB];
            float rstd[HB];
#pragma unroll
            for (int i = 0; i < HB; ++i) {
                if (h0 + i >= end) continue;
                const T* p = row_of<T>(x.in, b, t, h0 + i);
                const T* g = row_of<T>(x.dy, b, t, h0 + i);
                rxa[i] = get<WHOLE, G>(p + n.a, n.na);
                rxb[i] = get<WHOLE, G>(p + n.b, n.nb);
                rga[i] = get<WHOLE, G>(g + n.a, n.na);
                rgb[i] = get<WHOLE, G>(g + n.b, n.nb);
                rstd[i] = gptr(x.rstd)[(int64_t)row * x.heads + h0 + i];
            }
            if (h0 == part * a.per) angles(a.r, n, b, t, c, s);
#pragma unroll
            for (int i = 0; i < HB; ++i) {
                if (h0 + i >= end) continue;
                float xa[G], xb[G], ga[G], gb[G], sum = 0.f;
                widen<T, G>(rga[i], ga);
                widen<T, G>(rgb[i], gb);
                rotate(a.r.pairs, n, c, s, ga, gb);
                widen<T, G>(rxa[i], xa, rstd[i]);
                widen<T, G>(rxb[i], xb, rstd[i]);
#pragma unroll
                for (int e = 0; e < G; ++e) {
                    da[e] += ga[e] * xa[e];
                    db[e] += gb[e] * xb[e];
                    ga[e] *= wa.v[e];
                    gb[e] *= wb.v[e];
                    sum += ga[e] * xa[e] + gb[e] * xb[e];
                }
                sum = lanes_sum(sum, a.shift) * inv;
#pragma unroll
                for (int e = 0; e < G; ++e) {
                    ga[e] = (ga[e] - xa[e] * sum) * rstd[i];
                    gb[e] = (gb[e] - xb[e] * sum) * rstd[i];
                }
                T* p = row_of<T>(x.out, b, t, h0 + i);
                put<WHOLE, G>(p + n.a, n.na, ga);
                put<WHOLE, G>(p + n.b, n.nb, gb);
            }
        }
    }
    // the slots' sums meet in LDS and are added in order
#pragma unroll
    for (int e = 0; e < G; ++e) {
        cross[e][threadIdx.x] = da[e];
        cross[e + G][threadIdx.x] = db[e];
    }
    __syncthreads();
    for (int v = threadIdx.x; v < 2 * G << a.shift; v += kThreads) {
        const int e = v >> a.shift, at = v & ((1 << a.shift) - 1);
        float sum = 0.f;
        for (int j = 0; j < slots; ++j) sum += cross[e][(j << a.shift) + at];
        const Unit m = unit_of<G>(at, a.dim, a.r.rot, a.r.pairs);
        const int col = e < G ? m.a + e : m.b + e - G, left = e < G ? m.na - e : m.nb - (e - G);
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
constexpr int kBackwardBlocks = 1024;   // what the GPU holds at once at four wavefronts a SIMD

int units_of(int dim, int rot, bool pairs, int g) {
    const int turned = pairs ? (rot + 2 * g - 1) / (2 * g) : (rot / 2 + g - 1) / g;
    return turned + (dim - rot + 2 * g - 1) / (2 * g);
}
// The largest group of which both parts are whole ones, if a wavefront holds the
// row in them; else 0: groups of eight, looked at element by element.
int group_of(int dim, int rot, bool pairs) {
    for (int g : {4, 2, 1})
        if ((dim - rot) % g == 0 && (pairs ? rot : rot / 2) % g == 0) return units_of(dim, rot, pairs, g) <= 64 ? g : 0;
    return 0;
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

Place place_of(const opt_heads_desc* d, int heads, const Heads& t) {
    return {(int64_t)((uintptr_t)t.p / train_bytes(d->dtype)), {{d->batch, t.batch}, {d->tokens, t.token}, {heads, t.head}}, d->head_dim};
}
// A result and what is read by threads that may not have read it yet when it is
// written: other memory, or (OWN: what the same thread reads) the same place, every
// element written where it was read.
template <bool OWN>
opt_status check_place(const opt_heads_desc* d, int y_heads, const Heads& y, const char* y_name, int x_heads, const Heads& x, const char* x_name) {
    if (OWN && y.p == x.p) {
        const bool same = (d->batch == 1 || y.batch == x.batch) && (d->tokens == 1 || y.token == x.token) && (x_heads == 1 || y.head == x.head);
        return same ? OPT_OK : fail(OPT_EINVAL, "%s is %s with other strides", y_name, x_name);
    }
    if (!shares(place_of(d, y_heads, y), place_of(d, x_heads, x))) return OPT_OK;
    return fail(OPT_EINVAL, OWN ? "%s overlaps %s other than in its place" : "%s overlaps %s", y_name, x_name);
}
opt_status check_places(const opt_heads_desc* d, const Args& a) {
    const int h = d->heads, kv = d->kv_heads;
    if (opt_status st = check_place<true>(d, h, a.q.out, "yq", h, a.q.in, "q")) return st;
    if (kv == 0) return OPT_OK;
    if (opt_status st = check_place<true>(d, kv, a.k.out, "yk", kv, a.k.in, "k")) return st;
    if (opt_status st = check_place<false>(d, h, a.q.out, "yq", kv, a.k.in, "k")) return st;
    if (opt_status st = check_place<false>(d, kv, a.k.out, "yk", h, a.q.in, "q")) return st;
    return check_place<false>(d, h, a.q.out, "yq", kv, a.k.out, "yk");
}
opt_status check_gradient_places(const opt_heads_desc* d, const Args& a) {
    const int h = d->heads, kv = d->kv_heads;
    if (opt_status st = check_place<true>(d, h, a.q.out, "dq", h, a.q.in, "q")) return st;
    if (opt_status st = check_place<true>(d, h, a.q.out, "dq", h, a.q.dy, "dyq")) return st;
    if (kv == 0) return OPT_OK;
    if (opt_status st = check_place<true>(d, kv, a.k.out, "dk", kv, a.k.in, "k")) return st;
    if (opt_status st = check_place<true>(d, kv, a.k.out, "dk", kv, a.k.dy, "dyk")) return st;
    for (const auto& x : {std::make_pair(&a.k.in, "k"), std::make_pair(&a.k.dy, "dyk")})
        if (opt_status st = check_place<false>(d, h, a.q.out, "dq", kv, *x.first, x.second)) return st;
    for (const auto& x : {std::make_pair(&a.q.in, "q"), std::make_pair(&a.q.dy, "dyq")})
        if (opt_status st = check_place<false>(d, kv, a.k.out, "dk", h, *x.first, x.second)) return st;
    return check_place<false>(d, h, a.q.out, "dq", kv, a.k.out, "dk");
}

opt_status check_vector(const float* p, const char* name) {
    if (!p || !train_aligned(p, 4)) return fail(OPT_EINVAL, "%s is NULL or not aligned to 4 bytes", name);
    return OPT_OK;
}

void set_rows(const opt_heads_desc* d, Args& a) {
    a.tokens = (uint32_t)d->tokens, a.total = (uint32_t)(d->batch * d->tokens), a.dim = d->head_dim;
    a.q.heads = d->heads, a.k.heads = d->kv_heads;
    a.group = group_of(a.dim, a.r.rot, a.r.pairs);
    const int units = units_of(a.dim, a.r.rot, a.r.pairs, a.group ? a.group : 8);
    a.shift = 0;
    while ((1 << a.shift) < units) ++a.shift;
}

// Heads to a thread's turn: `most`, which share a token's angles (forward, as
// above: rotation 79 us with four, 81 with eight, 90 with all; norm, both
// directions, backward with four 100, with eight 99, with all 113), but fewer where
// the launch would leave CUs without work.
void set_per(Args& a, int most) {
    const auto parts = [&](int heads) { return (heads + a.per - 1) / a.per; };
    for (a.per = most; a.per > 1; a.per /= 2)
        if (((int64_t)a.total * (parts(a.q.heads) + parts(a.k.heads)) << a.shift) >= 1 << 16) break;
    a.q.parts = parts(a.q.heads), a.k.parts = parts(a.k.heads);
}

template <class T, bool NORM>
void forward(Args a, hipStream_t s) {
    set_per(a, 4);
    const int64_t parts = a.q.parts + a.k.parts, slots = kThreads >> a.shift;
    int64_t step = most_blocks(kThreads) * slots / parts;   // tokens of one launch
    const int64_t total = a.total;
    for (int64_t first = 0; first < total; first += step) {
        const int64_t n = total - first < step ? total - first : step;
        a.first = (uint32_t)first, a.total = (uint32_t)(first + n);   // none of the next launch's: out may be in
        const dim3 g((uint32_t)((n * parts + slots - 1) / slots));
        switch (a.group) {
            case 4: heads_forward_kernel<T, 4, true, NORM><<<g, kThreads, 0, s>>>(a); break;
            case 2: heads_forward_kernel<T, 2, true, NORM><<<g, kThreads, 0, s>>>(a); break;
            case 1: heads_forward_kernel<T, 1, true, NORM><<<g, kThreads, 0, s>>>(a); break;
            default: heads_forward_kernel<T, 8, false, NORM><<<g, kThreads, 0, s>>>(a);
        }
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
    set_per(a, 8);
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
    switch (a.group) {
        case 4: heads_backward_kernel<T, 4, true><<<g, kThreads, 0, s>>>(a); break;
        case 2: heads_backward_kernel<T, 2, true><<<g, kThreads, 0, s>>>(a); break;
        case 1: heads_backward_kernel<T, 1, true><<<g, kThreads, 0, s>>>(a); break;
        default: heads_backward_kernel<T, 8, false><<<g, kThreads, 0, s>>>(a);
    }
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
    if (opt_status st = check_places(d, a)) return st;
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
    if (opt_status st = check_places(d, a)) return st;
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
        if (opt_status st = check_gradient_places(d, a)) return st;
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
