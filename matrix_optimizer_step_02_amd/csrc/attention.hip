// Attention, forward and backward, on 16-bit matrix instructions.
//
//   S = scale Q K^T,  L_i = log sum_j exp(S_ij),  P = exp(S - L),  O = P V
//   D_i = sum_d dO_id O_id,  dP = dO V^T,  dS = P (dP - D)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
//
// One pass over the keys with a running maximum and sum (forward); the
// backward pass recomputes P from the saved L and holds nothing of size
// n_q x n_k. dQ is summed over keys by one kernel and dK, dV over queries (and
// the heads of a group) by another, each in its own registers: S and dP are
// formed twice (7 products instead of 5), and in return no atomics, no fp32
// copy of dQ in memory, and equal inputs give equal bits.
//
// Operand layout. v_mfma_f32_32x32x16 takes eight consecutive k values of one
// row per lane and leaves, in lane l and register r, column l % 32 and row
// 8 (r / 4) + 4 (l / 32) + r % 4. The forward and dQ kernels form S^T = K Q^T,
// so a lane owns one query: maximum, sum, L and D are one value per lane, and
// the 8 registers of 16 keys are, rounded to 16 bits, already the B operand
// of the next product (O^T = V^T P^T, dQ^T = K^T dS^T) if its A operand lists
// the keys in the same order: 4 (l / 32) + {0 .. 3} and 8 more. That A
// operand is the transpose of what LDS holds, and ds_read_b64_tr_b16 delivers
// it: 16 lanes read four rows of 16 columns and lane i gets column i of the
// four rows, just the group of four keys the order asks for. The dK/dV kernel
// is the same with keys and queries exchanged (a lane owns one key).
//
// LDS. Tiles of 64 rows are copied by global_load_lds, 16 bytes a lane, into
// rows of 256 bytes (128 for head_dim <= 64). The 16-byte group q of row r
// sits in slot q ^ swz(r); with swz taking the low two row bits as the high
// slot bits, both the reads of 16 rows at one group (A operands) and of four
// rows at four groups (transposed) touch every bank once.
//
// Precision. The matrix instructions take 16-bit operands, so P and dS are
// rounded once each where they enter one (half a step of the tensors' type);
// S, dP, L, D and every sum are fp32, and D is of the rounded O, which is what
// the caller holds. Holding P or dS as two 16-bit parts would double the
// products that take it.
//
// What bounds it. The matrix units are busy 47 to 58 % of the time at the
// clock measured (8192 x 8192, 16 heads of 128). The copies of the next tile
// are issued before the products of this one, but the compiler, which cannot
// tell the two tiles' LDS apart, waits for them before the first transposed
// read: in the dQ kernel after 16 of 48 products, with two sets of wavefronts
// also in the forward kernel, after 16 of 32 (not with one set). In the dK/dV
// kernel the wait stands before the first product: the loads of L and D, which
// follow the copies, complete in order behind them.
#include "train.h"

namespace matopt {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Read by every load that falls outside a sequence or past head_dim.
__device__ __attribute__((aligned(64))) uint32_t g_attn_zero[16];

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTile = 64;       // rows of an LDS tile
// A running maximum is raised only where it would grow by more than this
// (in powers of two): P stays below 2^8, far from any overflow, its relative
// rounding is unchanged, and the accumulators are rescaled in the first tile
// and rarely after it.
constexpr float kGrow = 8.f;
constexpr float kLowest = -1e30f;   // a maximum before any key: finite, so that exp2(-inf - m) = 0

struct Tensor {
    char* p;
    int64_t batch, token, head;   // strides in bytes
};

struct AttnArgs {
    Tensor q, k, v, o, dout, dq, dk, dv;
    float *lse, *delta;
    float *part, *part_v, *part_m, *part_l;   // partial results of splits (workspace)
    const int32_t *q_start, *k_start, *q_lens, *k_lens;
    int64_t q_tokens, k_tokens;   // rows of lse and delta; packed: the token axes
    int32_t batch, heads, kv_heads, head_dim, q_len, k_len, causal, window, splits, kv_splits;
    uint32_t first;   // of the workgroups, this launch's first
    int32_t listed;   // packed: row blocks are found by their place in a list (find_listed)
    float scale;
};

template <class T>
struct Frag;
template <>
struct Frag<__bf16> {
    typedef __bf16 type __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x16 mma(type a, type b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Frag<_Float16> {
    typedef _Float16 type __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x16 mma(type a, type b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

typedef __attribute__((address_space(3))) char* lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Geometry of one LDS tile of kTile rows. DB: 32-column blocks of head_dim.
template <int DB>
struct Geo {
    static constexpr int RB = DB > 2 ? 256 : 128;   // bytes per row
    static constexpr int SLOTS = RB / 16;
    static constexpr int BYTES = kTile * RB;
    static constexpr int CHUNKS = BYTES / 1024;     // 1 KiB per wavefront and copy instruction
    static __device__ __forceinline__ int swz(int row) {
        return DB > 2 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
    }
    // swz(row + i rows of a chunk) ^ swz(row), for a row in the first chunk of a wavefront
    static __device__ __forceinline__ constexpr int chunk_swz(int i) { return DB > 2 ? i & 3 : (2 * i) & 3; }
};

// Where one sequence's rows are.
struct Seq {
    int nq, nk, q_rows, k_rows;   // lengths, and the rows whose results are stored
    int64_t q0, k0;               // first row in the token axis (packed), or 0
    int64_t l0;                   // first row in lse and delta
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// First row and length of packed sequence b: offsets that do not ascend, or
// leave the token axis, cannot make an access leave it.
__device__ __forceinline__ int64_t packed(const int32_t* start, int64_t tokens, int most, int b, int& n) {
    const int64_t from = min(max((int64_t)gptr(start)[b], (int64_t)0), tokens);
    const int64_t to = min(max((int64_t)gptr(start)[b + 1], from), tokens);
    n = (int)min(to - from, (int64_t)most);
    return from;
}

__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b) {
    Seq s;
    if (a.q_start) {
        s.q0 = s.l0 = packed(a.q_start, a.q_tokens, a.q_len, b, s.nq);
        s.k0 = packed(a.k_start, a.k_tokens, a.k_len, b, s.nk);
        s.q_rows = s.nq;
        s.k_rows = s.nk;
    } else {
        s.nq = a.q_lens ? clampi(gptr(a.q_lens)[b], 0, a.q_len) : a.q_len;
        s.nk = a.k_lens ? clampi(gptr(a.k_lens)[b], 0, a.k_len) : a.k_len;
        s.q_rows = a.q_len;
        s.k_rows = a.k_len;
        s.q0 = s.k0 = 0;
        s.l0 = (int64_t)b * a.q_len;
    }
    return s;
}

__device__ __forceinline__ char* rows_of(const Tensor& t, int b, int64_t row0, int h) {
    return t.p + (int64_t)b * t.batch + row0 * t.token + (int64_t)h * t.head;
}

// Copies 64-row tiles of one tensor into LDS. Chunk i of a wavefront is 1024
// bytes of rows; its lanes' rows and groups follow from chunk 0's (rows 1024 /
// RB further, the swizzle's low slot bits counting chunks), so two registers
// hold what the eight addresses of a tile need. PIN computes them anew for
// each tile (a kernel short of registers; the others run 5 % faster with
// them kept).
template <int DB, int W, bool PIN = false>
struct Copy {
    using G = Geo<DB>;
    static constexpr int PER_WAVE = G::CHUNKS / W;   // of W wavefronts
    int row0, group0;   // of chunk 0
    int64_t token;

    __device__ __forceinline__ void init(int64_t token_stride) {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % W;
        token = token_stride;
        row0 = wave * PER_WAVE * (1024 / G::RB) + lane / G::SLOTS;
        group0 = (lane % G::SLOTS) ^ G::swz(row0);
    }
    // rows first .. first + 63 of a sequence of n rows
    __device__ __forceinline__ void tile(char* lds, const char* base, int first, int n, int head_dim) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % W;
        const char* origin = base + (int64_t)first * token;
        int r0 = row0, g0 = group0;
        if constexpr (PIN) asm volatile("" : "+v"(r0), "+v"(g0));
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i) {
            const int row = r0 + i * (1024 / G::RB), group = g0 ^ G::chunk_swz(i);
            const uint32_t off = (uint32_t)row * (uint32_t)token + 16 * group;
            const bool in = row < n - first && 8 * group < head_dim;
            const void* src = in ? (const void*)(origin + off) : (const void*)g_attn_zero;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(lds + (wave * PER_WAVE + i) * 1024),
                                             16, 0, 0);
        }
    }
};

// Barrier after which every wavefront sees the tiles that all of them copied.
// The copies are vector-memory operations, which a workgroup fence does not
// wait for, so each wavefront waits for its own (and for its LDS reads of the
// tile that the next copy overwrites) before it arrives.
__device__ __forceinline__ void tile_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A lane's LDS addresses of a tile. The swizzle is an exclusive or and tiles
// are aligned to 1024 bytes, so one register per kind of read holds them all:
// k step s flips bits 5 .. 7 of a row's address, the 32-column block d bits 6
// and 7 of a transposed read's, its second half bit 5. `at` (a multiple of
// 1024) reaches the tile of another tensor by the instruction's offset.
template <class T, int DB>
struct Lane {
    using G = Geo<DB>;
    using F = typename Frag<T>::type;
    uint32_t row0;   // A operand, k step 0: row l % 32, group l / 32
    uint32_t col0;   // transposed, block 0: row 4 (l / 32) + l % 16 / 4

    __device__ __forceinline__ void init() {
        const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
        row0 = l32 * G::RB + ((h ^ G::swz(l32)) << 4);
        const int row = 4 * h + ((lane & 15) >> 2);
        const int group = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
        col0 = row * G::RB + ((group ^ G::swz(row)) << 4) + 8 * (lane & 1);
    }
    // The same within the tile at `tile`.
    __device__ __forceinline__ Lane in(const char* tile) const {
        const uint32_t t = (uint32_t)(uintptr_t)(lds_char)tile;
        return {row0 + t, col0 + t};
    }
    // Keeps what is derived from the two registers from being computed ahead
    // and held over the code between (16 registers).
    __device__ __forceinline__ void pin() { asm volatile("" : "+v"(row0), "+v"(col0)); }
    // rows 32 blk .. of the tile, k step s
    __device__ __forceinline__ F rows(int at, int blk, int s) const {
        typedef __attribute__((address_space(3))) const F* ptr;
        return *(ptr)(lds_char)(uintptr_t)((row0 ^ (uint32_t)(s << 5)) + at + blk * 32 * G::RB);
    }
    // columns 32 d .. as rows of A, tile rows 16 st .. 16 st + 15 as k, in the accumulators' order
    __device__ __forceinline__ F cols(int at, int st, int d) const {
        typedef __attribute__((address_space(3))) s16x4* ptr;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (ptr)(lds_char)(uintptr_t)((col0 ^ (uint32_t)(d << 6)) + at + st * 16 * G::RB));
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (ptr)(lds_char)(uintptr_t)((col0 ^ (uint32_t)(d << 6 | 32)) + at + (16 * st + 8) * G::RB));
        return __builtin_bit_cast(F, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// B operand fragments of 32 rows in registers: row l % 32 (of n), k 16 s + 8 (l / 32) ..
// What is outside is read from the zeros, so that all loads go out at once.
template <class T, int DB>
__device__ __forceinline__ void load_rows(typename Frag<T>::type (&f)[2 * DB], const char* base, int64_t token, int row,
                                          int n, int head_dim) {
    const int h = (threadIdx.x & 63) >> 5;
    const char* p = base + (int64_t)row * token;
    const char* zero = (const char*)g_attn_zero;
#pragma unroll
    for (int s = 0; s < 2 * DB; ++s) {
        const int c = 16 * s + 8 * h;
        const char* q = row < n && c < head_dim ? p + 2 * c : zero;
        f[s] = __builtin_bit_cast(typename Frag<T>::type, *gptr((const u32x4*)q));
    }
}

// Sum or maximum over the two half-waves (lanes l and l + 32).
__device__ __forceinline__ float other_half(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float((threadIdx.x & 63) < 32 ? r[1] : r[0]);
}

// Registers 8 k .. 8 k + 7 of an accumulator, rounded to 16 bits: P or dS as
// an operand.
template <class T>
__device__ __forceinline__ typename Frag<T>::type pack8(const f32x16& x, int k) {
    typename Frag<T>::type f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (T)x[8 * k + e];
    return f;
}

// A 32-row block of an output whose transpose is in accumulators: lane's row,
// columns 32 d + 8 g + 4 h .. + 3 in registers 4 g ..
template <class T, int DB>
__device__ __forceinline__ void store_t(const f32x16 (&acc)[DB], float mul, char* row, int head_dim) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            if (32 * d + 8 * g >= head_dim) continue;
            typedef T t4 __attribute__((ext_vector_type(4)));
            t4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (T)(acc[d][4 * g + e] * mul);
            *gptr((u32x2*)(row + 2 * (32 * d + 8 * g + 4 * h))) = __builtin_bit_cast(u32x2, v);
        }
}

// Workgroup id -> (row block, head-and-batch index). Ids go to the XCDs in
// turn, so id % 8 keeps a key head, with the `group` heads that share it, on
// one XCD, whose L2 then serves its keys to all their row blocks; the heads of
// one sequence spread over the XCDs, since sequences may differ in length.
// Blocks run longest work first: `reverse` where that is the last one (a
// causal sequence's last queries see the most keys).
__device__ __forceinline__ void locate(int id, int blocks, int pairs, int group, bool reverse, int& blk, int& pair) {
    if (pairs % 8 == 0) {
        if (pairs / group % 8) group = 1;
        const int per = pairs / 8, r = id / 8, c = r % per;
        pair = (c / group * 8 + id % 8) * group + c % group;
        blk = r / per;
    } else {
        pair = id % pairs;
        blk = id / pairs;
    }
    if (reverse) blk = blocks - 1 - blk;
}

// Keys [lo, hi) that query i of a sequence sees.
struct Sight {
    int nk, off, window, causal;
    __device__ __forceinline__ int hi(int i) const { return causal ? clampi(i + off + 1, 0, nk) : nk; }
    __device__ __forceinline__ int lo(int i) const { return window ? max(i + off - window + 1, 0) : 0; }
};

// Workgroups come in three shapes: four wavefronts (128 rows), eight (256
// rows) that share the same tiles, or two sets of four (128 rows) with LDS
// tiles of their own, which take the tiles in turn and join their sums through
// LDS. Registers leave room for two wavefronts a SIMD (three for dK and dV at
// head_dim <= 64): two workgroups a CU of the first shape, one of the others.
// Where the launch has fewer workgroups than the GPU has CUs (few queries on a
// long context), the tiles are also split over workgroups, which leave fp32
// partial sums in the workspace for a second kernel to join: 509 queries on
// 8192 keys, 16 / 8 heads of 128, take 49 + 5 us in place of 215. The host
// chooses (shape_of, splits_of).

// Row blocks of packed sequences, as a list without the blocks that a shorter
// sequence lacks (a launch that covers the longest one for each sequence would
// be mostly of those: 4 to 12 % of the time at 13 sequences of 8192 tokens).
// Finds entry `at` of the list of all (sequence, level) with level below the
// sequence's number of blocks, highest level first, so that the longest
// sequences' far blocks come first: a bisection over the levels in each
// wavefront, a sequence per lane. false: past the list's end.
constexpr int kListed = 256;   // sequences at most: four turns of 64 per step
__device__ __forceinline__ bool find_listed(const int32_t* start, int64_t tokens, int most, int batch, int rows, int at,
                                            int& seq, int& level, int& levels) {
    const int lane = threadIdx.x & 63;
    int n[kListed / 64];
#pragma unroll
    for (int c = 0; c < kListed / 64; ++c) {
        const int b = 64 * c + lane;
        int len = 0;
        if (b < batch) packed(start, tokens, most, b, len);
        n[c] = (len + rows - 1) / rows;
    }
    const auto above = [&](int x) {   // entries of levels x and higher
        int s = 0;
#pragma unroll
        for (int c = 0; c < kListed / 64; ++c) s += max(n[c] - x, 0);
#pragma unroll
        for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m);
        return __builtin_amdgcn_readfirstlane(s);
    };
    if (at >= above(0)) return false;
    int lo = 0, hi = (most + rows - 1) / rows;   // above(lo) > at >= above(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (above(mid) > at) lo = mid;
        else hi = mid;
    }
    level = lo;
    int left = at - above(lo + 1);   // which of the sequences that have this level
#pragma unroll
    for (int c = 0; c < kListed / 64; ++c) {
        uint64_t has = __ballot(n[c] > lo);
        const int k = __popcll(has);
        if (left >= 0 && left < k) {
            for (; left; --left) has &= has - 1;
            const int l = __ffsll((unsigned long long)has) - 1;
            seq = 64 * c + l;
            levels = __builtin_amdgcn_readlane(n[c], l);
            left = -1;
        } else if (left >= 0) {
            left -= k;
        }
    }
    return true;
}

struct Block {
    int b, hq, hk, i0, split;
};
// false: no rows here.
__device__ __forceinline__ bool block_of(const AttnArgs& a, int blocks, int rows, Block& x) {
    const int group = a.heads / a.kv_heads;
    const int pairs = a.listed ? a.heads : a.batch * a.heads, per = blocks * pairs;   // workgroups of one split
    const int at = a.first + blockIdx.x;
    x.split = at / per;
    int blk, pair;
    locate(at - x.split * per, blocks, pairs, group, a.causal && !a.listed, blk, pair);
    x.b = pair / a.heads, x.hq = pair % a.heads, x.hk = x.hq / group;
    if (a.listed) {
        int levels;
        if (!find_listed(a.q_start, a.q_tokens, a.q_len, a.batch, rows, blk, x.b, blk, levels)) return false;
    }
    x.i0 = blk * rows;
    return true;
}

// Key tiles [first, end) of this workgroup's queries and split.
__device__ __forceinline__ void tile_range(const AttnArgs& a, const Sight& see, int i0, int rows, int nq, int split, int& first, int& end) {
    first = end = 0;
    if (i0 >= nq) return;
    first = see.lo(i0) / kTile;
    end = (see.hi(min(i0 + rows, nq) - 1) + kTile - 1) / kTile;
    if (a.splits > 1) {
        const int each = (max(end - first, 0) + a.splits - 1) / a.splits;
        first += split * each;
        end = min(end, first + each);
    }
}

// Row of the partial results: (split, head, row of lse).
__device__ __forceinline__ int64_t part_row(const AttnArgs& a, int split, int hq, int64_t row) {
    return ((int64_t)split * a.heads + hq) * a.q_tokens + row;
}

// Lane's columns of a transposed accumulator as fp32 partial results.
template <int DB>
__device__ __forceinline__ void store_part(const f32x16 (&acc)[DB], float* row) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[d][4 * g + e];
            *gptr((f32x4*)(row + 32 * d + 8 * g + 4 * h)) = v;
        }
}

// A row that sees nothing holds sums of 0 times what it does not see, which
// are NaN where that is not finite.
template <int DB>
__device__ __forceinline__ void clear(f32x16 (&acc)[DB]) {
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
}

// Hands accumulators (and two more values) from set 1 to set 0 through the
// LDS of the tiles, which every wavefront has left: 64 (16 DB + 2) floats of
// each wavefront.
template <int DB>
__device__ __forceinline__ void give(char* smem, int wave, const f32x16 (&acc)[DB], float x, float y) {
    const int lane = threadIdx.x & 63;
    float* to = (float*)smem + wave * (DB * 1024 + 128);
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[d][4 * g + e];
            *(f32x4*)(to + (d * 4 + g) * 256 + lane * 4) = v;
        }
    to[DB * 1024 + lane] = x;
    to[DB * 1024 + 64 + lane] = y;
}
template <int DB>
__device__ __forceinline__ void take(const char* smem, int wave, float mine, float theirs, f32x16 (&acc)[DB]) {
    const int lane = threadIdx.x & 63;
    const float* from = (const float*)smem + wave * (DB * 1024 + 128);
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 v = *(const f32x4*)(from + (d * 4 + g) * 256 + lane * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[d][4 * g + e] = acc[d][4 * g + e] * mine + v[e] * theirs;
        }
}

// --------------------------------------------------------------- forward ----

template <class T, int DB, int W, int SETS>
__global__ __launch_bounds__(SETS * 64 * W, 2) void attn_forward_kernel(AttnArgs a, int blocks) {
    using G = Geo<DB>;
    using FT = Frag<T>;
    using F = typename FT::type;
    __shared__ __attribute__((aligned(1024))) char smem[SETS * 4 * G::BYTES];
    Block wg;
    if (!block_of(a, blocks, 32 * W, wg)) return;
    const int b = wg.b, hq = wg.hq, hk = wg.hk, i0 = wg.i0;
    const Seq sq = sequence(a, b);
    if (i0 >= sq.q_rows) return;
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
    const int wave8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = wave8 % W;
    const int set = SETS > 1 ? wave8 / W : 0;
    const int w0 = i0 + 32 * wave, i = w0 + l32;   // the wavefront's first query, the lane's query
    const Sight see = {sq.nk, sq.nk - sq.nq, a.window, a.causal};

    Lane<T, DB> ln;
    ln.init();
    F qf[2 * DB];
    load_rows<T, DB>(qf, rows_of(a.q, b, sq.q0, hq), a.q.token, i, sq.nq, a.head_dim);
    Copy<DB, W> ck, cv;
    ck.init(a.k.token);
    cv.init(a.v.token);
    const char* kb = rows_of(a.k, b, sq.k0, hk);
    const char* vb = rows_of(a.v, b, sq.k0, hk);

    f32x16 o[DB] = {};
    float m = kLowest, l = 0.f;
    const float c = a.scale * kLog2e;
    int first_t, end_t;
    tile_range(a, see, i0, 32 * W, sq.nq, wg.split, first_t, end_t);
    // keys that any query of this wavefront sees, and the lane's
    const int wlast = min(w0 + 32, sq.nq) - 1;
    const int whi = w0 < sq.nq ? see.hi(wlast) : 0, wlo = see.lo(w0);
    const int hi = i < sq.nq ? see.hi(i) : 0, lo = see.lo(i);
    // tiles from full_lo up to full_hi need no mask
    const int full_hi = see.hi(w0) / kTile, full_lo = (see.lo(max(wlast, w0)) + kTile - 1) / kTile;

    // turn r of a set is tile first_t + SETS r + set, in buffers r & 1
    auto kt = [&](int r) { return smem + (4 * set + (r & 1)) * G::BYTES; };
    auto fill = [&](int r) {
        const int t = first_t + SETS * r + set;
        if (t >= end_t) return;
        ck.tile(kt(r), kb, t * kTile, sq.nk, a.head_dim);
        cv.tile(kt(r) + 2 * G::BYTES, vb, t * kTile, sq.nk, a.head_dim);
    };
    const int turns = (end_t - first_t + SETS - 1) / SETS;
    fill(0);
    for (int r = 0; r < turns; ++r) {
        tile_barrier();
        fill(r + 1);
        const int t = first_t + SETS * r + set;
        if (t >= end_t || t * kTile >= whi || (t + 1) * kTile <= wlo) continue;
        const Lane<T, DB> at = ln.in(kt(r));
        constexpr int K = 0, V = 2 * G::BYTES;
        f32x16 s[2] = {};
#pragma unroll
        for (int ks = 0; ks < 2 * DB; ++ks)
#pragma unroll
            for (int n = 0; n < 2; ++n) s[n] = FT::mma(at.rows(K, n, ks), qf[ks], s[n]);
        if (t >= full_hi || t < full_lo || w0 + 32 > sq.nq) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = t * kTile + 32 * n + 8 * (e >> 2) + 4 * h + (e & 3);
                    if (j >= hi || j < lo) s[n][e] = -INFINITY;
                }
        }
        float mx = s[0][0];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[n][e]);
        if (__any(mx * c > m + kGrow)) {
            mx = fmaxf(mx, other_half(mx));
            const float mn = fmaxf(m, mx * c);
            const float k = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= k;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= k;
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[n][e] = __builtin_amdgcn_exp2f(fmaf(s[n][e], c, -m));
                l += s[n][e];
            }
#pragma unroll
        for (int st = 0; st < 4; ++st) {
            const F p = pack8<T>(s[st >> 1], st & 1);
#pragma unroll
            for (int d = 0; d < DB; ++d) o[d] = FT::mma(at.cols(V, st, d), p, o[d]);
        }
    }
    l += other_half(l);
    if constexpr (SETS > 1) {
        tile_barrier();
        if (set == 1) give<DB>(smem, wave, o, m, l);
        __syncthreads();
        if (set == 1) return;
        const float* from = (const float*)smem + wave * (DB * 1024 + 128) + DB * 1024 + lane;
        const float m1 = from[0], l1 = from[64], mn = fmaxf(m, m1);
        const float k0 = __builtin_amdgcn_exp2f(m - mn), k1 = __builtin_amdgcn_exp2f(m1 - mn);
        take<DB>(smem, wave, k0, k1, o);
        l = l * k0 + l1 * k1;
        m = mn;
    }
    if (l == 0.f) clear(o);
    if (i >= sq.q_rows) return;
    if (a.splits > 1) {
        const int64_t row = part_row(a, wg.split, hq, sq.l0 + i);
        store_part<DB>(o, a.part + row * (32 * DB));
        if (h == 0) {
            gptr(a.part_m)[row] = m;
            gptr(a.part_l)[row] = l;
        }
        return;
    }
    store_t<T, DB>(o, l == 0.f ? 0.f : 1.f / l, rows_of(a.o, b, sq.q0, hq) + (int64_t)i * a.o.token, a.head_dim);
    if (h == 0) gptr(a.lse)[(int64_t)hq * a.q_tokens + sq.l0 + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Joins the key splits of one row: out and lse (ML), or the sum of partial
// gradients times scale. Eight columns a thread, 16 threads a row.
constexpr int kJoinThreads = 256, kJoinRows = kJoinThreads / 16;
template <class T, bool ML>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a, int width, int blocks) {
    const int b = blockIdx.x / blocks / a.heads, hq = blockIdx.x / blocks % a.heads;
    const Seq sq = sequence(a, b);
    const int i = blockIdx.x % blocks * kJoinRows + threadIdx.x / 16, col = threadIdx.x % 16 * 8;
    if (i >= sq.q_rows || col >= a.head_dim) return;
    float m = kLowest, l = 0.f, x[8] = {};
    if constexpr (ML)
        for (int s = 0; s < a.splits; ++s) m = fmaxf(m, gptr(a.part_m)[part_row(a, s, hq, sq.l0 + i)]);
    for (int s = 0; s < a.splits; ++s) {
        const int64_t row = part_row(a, s, hq, sq.l0 + i);
        float v[8], k = 1.f;
        if constexpr (ML) {
            k = __builtin_amdgcn_exp2f(gptr(a.part_m)[row] - m);
            l += gptr(a.part_l)[row] * k;
        }
        load8(a.part + row * width + col, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(v[e], k, x[e]);
    }
    const float mul = ML ? (l == 0.f ? 0.f : 1.f / l) : a.scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= mul;
    const Tensor& t = ML ? a.o : a.dq;
    store8((T*)(rows_of(t, b, sq.q0, hq) + (int64_t)i * t.token) + col, x);
    if (ML && col == 0)
        gptr(a.lse)[(int64_t)hq * a.q_tokens + sq.l0 + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// -------------------------------------------------------------- backward ----

// dQ, and D for the other kernel. A lane owns one query, as in the forward pass.
template <class T, int DB, int W, int SETS>
__global__ __launch_bounds__(SETS * 64 * W, 2) void attn_dq_kernel(AttnArgs a, int blocks) {
    using G = Geo<DB>;
    using FT = Frag<T>;
    using F = typename FT::type;
    __shared__ __attribute__((aligned(1024))) char smem[SETS * 4 * G::BYTES];
    Block wg;
    if (!block_of(a, blocks, 32 * W, wg)) return;
    const int b = wg.b, hq = wg.hq, hk = wg.hk, i0 = wg.i0;
    const Seq sq = sequence(a, b);
    if (i0 >= sq.q_rows) return;
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
    const int wave8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = wave8 % W;
    const int set = SETS > 1 ? wave8 / W : 0;
    const int w0 = i0 + 32 * wave, i = w0 + l32;
    const Sight see = {sq.nk, sq.nk - sq.nq, a.window, a.causal};

    Lane<T, DB> ln;
    ln.init();
    F qf[2 * DB], gf[2 * DB];
    float D = 0.f;
    {
        F of[2 * DB];
        load_rows<T, DB>(of, rows_of(a.o, b, sq.q0, hq), a.o.token, i, sq.nq, a.head_dim);
        load_rows<T, DB>(gf, rows_of(a.dout, b, sq.q0, hq), a.dout.token, i, sq.nq, a.head_dim);
        load_rows<T, DB>(qf, rows_of(a.q, b, sq.q0, hq), a.q.token, i, sq.nq, a.head_dim);
        // D is the diagonal of O dO^T, by the products that form dP = V dO^T:
        // where a row sees one key, O is that key's V to the bit, dP - D is
        // zero, and so are its gradients
        f32x16 x = {};
#pragma unroll
        for (int s = 0; s < 2 * DB; ++s) x = FT::mma(of[s], gf[s], x);
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (8 * (r >> 2) + 4 * h + (r & 3) == l32) D = x[r];
        const float y = other_half(D);
        D = ((l32 >> 2) & 1) == h ? D : y;   // the half that holds it
    }
    const int64_t at_row = (int64_t)hq * a.q_tokens + sq.l0 + i;
    // a row that sees no key has L = -inf: with +inf in its place P is 0
    float L2 = INFINITY;
    if (i < sq.nq) {
        L2 = gptr(a.lse)[at_row] * kLog2e;
        if (L2 == -INFINITY) L2 = INFINITY;
        if (h == 0 && set == 0 && wg.split == 0) gptr(a.delta)[at_row] = D;
    }
    Copy<DB, W> ck, cv;
    ck.init(a.k.token);
    cv.init(a.v.token);
    const char* kb = rows_of(a.k, b, sq.k0, hk);
    const char* vb = rows_of(a.v, b, sq.k0, hk);
    f32x16 dq[DB] = {};
    const float c = a.scale * kLog2e;
    int first_t, end_t;
    tile_range(a, see, i0, 32 * W, sq.nq, wg.split, first_t, end_t);
    const int wlast = min(w0 + 32, sq.nq) - 1;
    const int whi = w0 < sq.nq ? see.hi(wlast) : 0, wlo = see.lo(w0);
    const int hi = i < sq.nq ? see.hi(i) : 0, lo = see.lo(i);
    const int full_hi = see.hi(w0) / kTile, full_lo = (see.lo(max(wlast, w0)) + kTile - 1) / kTile;

    auto kt = [&](int r) { return smem + (4 * set + (r & 1)) * G::BYTES; };
    auto fill = [&](int r) {
        const int t = first_t + SETS * r + set;
        if (t >= end_t) return;
        ck.tile(kt(r), kb, t * kTile, sq.nk, a.head_dim);
        cv.tile(kt(r) + 2 * G::BYTES, vb, t * kTile, sq.nk, a.head_dim);
    };
    const int turns = (end_t - first_t + SETS - 1) / SETS;
    fill(0);
    for (int r = 0; r < turns; ++r) {
        tile_barrier();
        fill(r + 1);
        const int t = first_t + SETS * r + set;
        if (t >= end_t || t * kTile >= whi || (t + 1) * kTile <= wlo) continue;
        const Lane<T, DB> at = ln.in(kt(r));
        constexpr int K = 0, V = 2 * G::BYTES;
        const bool edge = t >= full_hi || t < full_lo;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            f32x16 s = {}, dp = {};
#pragma unroll
            for (int ks = 0; ks < 2 * DB; ++ks) {
                s = FT::mma(at.rows(K, n, ks), qf[ks], s);
                dp = FT::mma(at.rows(V, n, ks), gf[ks], dp);
            }
            if (edge) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = t * kTile + 32 * n + 8 * (e >> 2) + 4 * h + (e & 3);
                    if (j >= hi || j < lo) s[e] = -INFINITY;
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, -L2)) * (dp[e] - D);
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const F p = pack8<T>(s, st);
#pragma unroll
                for (int d = 0; d < DB; ++d) dq[d] = FT::mma(at.cols(K, 2 * n + st, d), p, dq[d]);
            }
        }
    }
    if constexpr (SETS > 1) {
        tile_barrier();
        if (set == 1) give<DB>(smem, wave, dq, 0.f, 0.f);
        __syncthreads();
        if (set == 1) return;
        take<DB>(smem, wave, 1.f, 1.f, dq);
    }
    if (hi <= lo) clear(dq);
    if (i >= sq.q_rows) return;
    if (a.splits > 1)
        store_part<DB>(dq, a.part + part_row(a, wg.split, hq, sq.l0 + i) * (32 * DB));
    else
        store_t<T, DB>(dq, a.scale, rows_of(a.dq, b, sq.q0, hq) + (int64_t)i * a.dq.token, a.head_dim);
}

// The dK/dV kernel holds P times 2^kLift<T>. float16 has steps of 2^-24 below
// 2^-14, which a P of 1 / n is at n keys seen alike: 1.3 % off, all to one
// side, at 10^6, and 0 from 2^25. Lifted by 2^14 it is a normal number down to
// 2^-28 (sequences have at most 2^29 tokens), and P = 1, with room for the
// rounding of large scores, stays below float16's largest, 2^16. dP - D is
// lowered by as much in the operation that forms it, and dV where it is stored.
template <class T>
constexpr int kLift = __is_same(T, _Float16) ? 14 : 0;
template <class T>
constexpr float kLower = 1.f / (1 << kLift<T>);

// dK and dV of 32 W keys, summed over the queries that see them and over the
// heads of the group; the steps are (head, query tile). A lane owns one key.
// The keys' accumulators (128 registers at head_dim 128) and operands (64)
// leave little of the 256 registers that two wavefronts a SIMD have, so the
// addresses are computed where they are used; past head_dim 96 some are
// spilled all the same (12 bytes a lane with two sets, 20 with one) and read
// back in each step. At head_dim <= 64 a workgroup of
// four is held to 168 registers, three wavefronts a SIMD: 68 us against 78 (6 x
// 1000 tokens, 16 heads of 64).
template <class T, int DB, int W, int SETS>
__global__ __launch_bounds__(SETS * 64 * W, DB <= 2 && SETS * W == 4 ? 3 : 2) void attn_dkv_kernel(AttnArgs a, int blocks) {
    using G = Geo<DB>;
    using FT = Frag<T>;
    using F = typename FT::type;
    __shared__ __attribute__((aligned(1024))) char smem[SETS * 4 * G::BYTES];
    __shared__ __attribute__((aligned(16))) float stat[SETS][2][2][kTile];   // [set][buffer][L, D]
    int blk, pair;
    const int pairs = a.listed ? a.kv_heads : a.batch * a.kv_heads, per = blocks * pairs, wg = a.first + blockIdx.x, split = wg / per;
    locate(wg - split * per, blocks, pairs, 1, false, blk, pair);
    const int hk = pair % a.kv_heads, group = a.heads / a.kv_heads;
    int b = pair / a.kv_heads;
    if (a.listed) {
        int level, levels;
        if (!find_listed(a.k_start, a.k_tokens, a.k_len, a.batch, 32 * W, blk, b, level, levels)) return;
        blk = a.causal ? levels - 1 - level : level;   // the first keys of a causal sequence have the most queries
    }
    const Seq sq = sequence(a, b);
    const int j0 = blk * 32 * W;
    if (j0 >= sq.k_rows) return;
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
    const int wave8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = wave8 % W, set = SETS > 1 ? wave8 / W : 0;
    const int w0 = j0 + 32 * wave, j = w0 + l32;   // the wavefront's first key, the lane's key
    const int off = sq.nk - sq.nq;

    Lane<T, DB> ln;
    ln.init();
    F kf[2 * DB], vf[2 * DB];
    load_rows<T, DB>(kf, rows_of(a.k, b, sq.k0, hk), a.k.token, j, sq.nk, a.head_dim);
    load_rows<T, DB>(vf, rows_of(a.v, b, sq.k0, hk), a.v.token, j, sq.nk, a.head_dim);
    Copy<DB, W, true> cq, cg;
    cq.init(a.q.token);
    cg.init(a.dout.token);
    f32x16 dk[DB] = {}, dv[DB] = {};
    const float c = a.scale * kLog2e;

    // queries [lo, hi) that see key j: j <= i + off, and j > i + off - window
    auto qlo = [&](int key) { return a.causal ? clampi(key - off, 0, sq.nq) : 0; };
    auto qhi = [&](int key) { return a.window ? clampi(key - off + a.window, 0, sq.nq) : sq.nq; };
    const int jl = min(j0 + 32 * W, sq.nk) - 1, wl = min(w0 + 32, sq.nk) - 1;
    const bool any = j0 < sq.nk;
    const int first_t = any ? qlo(j0) / kTile : 0;
    const int end_t = any ? (qhi(jl) + kTile - 1) / kTile : 0;
    const int tiles = max(end_t - first_t, 0);
    const int wlo = qlo(w0), whi = w0 < sq.nk ? qhi(wl) : 0;
    const int lo = qlo(j), hi = j < sq.nk ? qhi(j) : 0;
    const int full_lo = (qlo(max(wl, w0)) + kTile - 1) / kTile, full_hi = qhi(w0) / kTile;

    // buffers of turn r
    auto qt = [&](int r) { return smem + (4 * set + (r & 1)) * G::BYTES; };
    auto gt = [&](int r) { return smem + (4 * set + 2 + (r & 1)) * G::BYTES; };
    // step n: query tile n % tiles of the group's head n / tiles; this split's
    // steps are [from, to), and turn r of a set is step from + SETS r + set
    const int steps = tiles * group, each = (steps + a.kv_splits - 1) / a.kv_splits;
    const int from = split * each, to = min(steps, from + each), turns = (to - from + SETS - 1) / SETS;
    auto fill = [&](int r) {
        const int n = from + SETS * r + set;
        if (n >= to) return;
        const int hq = hk * group + n / tiles, first = (first_t + n % tiles) * kTile;
        cq.tile(qt(r), rows_of(a.q, b, sq.q0, hq), first, sq.nq, a.head_dim);
        cg.tile(gt(r), rows_of(a.dout, b, sq.q0, hq), first, sq.nq, a.head_dim);
        if (wave == 0) {
            const int i = first + lane;
            const int64_t at = (int64_t)hq * a.q_tokens + sq.l0 + i;
            float L = INFINITY, D = 0.f;
            if (i < sq.nq) {
                L = gptr(a.lse)[at] * kLog2e;
                L = L == -INFINITY ? INFINITY : L - kLift<T>;
                D = gptr(a.delta)[at] * kLower<T>;
            }
            stat[set][r & 1][0][lane] = L;
            stat[set][r & 1][1][lane] = D;
        }
    };
    fill(0);
    for (int r = 0; r < turns; ++r) {
        tile_barrier();
        fill(r + 1);
        const int n = from + SETS * r + set;
        if (n >= to) continue;
        const int t = first_t + n % tiles;
        if (t * kTile >= whi || (t + 1) * kTile <= wlo) continue;
        Lane<T, DB> at = ln.in(qt(r));
        constexpr int Q = 0, O = 2 * G::BYTES;
        const bool edge = t < full_lo || t >= full_hi || w0 + 32 > sq.nk;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            at.pin();
            if constexpr (DB > 2) __builtin_amdgcn_sched_barrier(0);
            f32x16 s = {}, dp = {};
#pragma unroll
            for (int ks = 0; ks < 2 * DB; ++ks) {
                s = FT::mma(at.rows(Q, u, ks), kf[ks], s);
                dp = FT::mma(at.rows(O, u, ks), vf[ks], dp);
            }
            if (edge) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int i = t * kTile + 32 * u + 8 * (e >> 2) + 4 * h + (e & 3);
                    if (i >= hi || i < lo) s[e] = -INFINITY;
                }
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 L = *(const f32x4*)&stat[set][r & 1][0][32 * u + 8 * g + 4 * h];
                const f32x4 D = *(const f32x4*)&stat[set][r & 1][1][32 * u + 8 * g + 4 * h];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[4 * g + e] = __builtin_amdgcn_exp2f(fmaf(s[4 * g + e], c, -L[e]));
                    dp[4 * g + e] = s[4 * g + e] * fmaf(dp[4 * g + e], kLower<T>, -D[e]);
                }
            }
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const F p = pack8<T>(s, st), ds = pack8<T>(dp, st);
                if constexpr (DB > 2) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    dv[d] = FT::mma(at.cols(O, 2 * u + st, d), p, dv[d]);
                    dk[d] = FT::mma(at.cols(Q, 2 * u + st, d), ds, dk[d]);
                }
            }
        }
    }
    if constexpr (SETS > 1) {
        // set 1's dK and set 0's dV cross over through LDS, and each set stores the sum it then has
        static_assert(2 * W * DB * 16 * 256 <= sizeof smem, "the accumulators do not fit the tiles' LDS");
        tile_barrier();
        float* mine = (float*)smem + (set * W + wave) * DB * 1024 + lane * 4;
        float* theirs = (float*)smem + ((1 - set) * W + wave) * DB * 1024 + lane * 4;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = set ? dk[d][4 * g + e] : dv[d][4 * g + e];
                *(f32x4*)(mine + (d * 4 + g) * 256) = x;
            }
        __syncthreads();
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 x = *(const f32x4*)(theirs + (d * 4 + g) * 256);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (set) dv[d][4 * g + e] += x[e];
                    else dk[d][4 * g + e] += x[e];
            }
    }
    if (hi <= lo) clear(dk), clear(dv);
    if (j >= sq.k_rows) return;
    if (a.kv_splits > 1) {
        const int64_t row = (((int64_t)split * a.kv_heads + hk) * a.k_tokens + (a.q_start ? sq.k0 : (int64_t)b * a.k_len) + j) * (32 * DB);
        if (SETS == 1 || set == 0) store_part<DB>(dk, a.part + row);
        if (SETS == 1 || set == 1) store_part<DB>(dv, a.part_v + row);
        return;
    }
    if (SETS == 1 || set == 0)
        store_t<T, DB>(dk, a.scale, rows_of(a.dk, b, sq.k0, hk) + (int64_t)j * a.dk.token, a.head_dim);
    if (SETS == 1 || set == 1)
        store_t<T, DB>(dv, kLower<T>, rows_of(a.dv, b, sq.k0, hk) + (int64_t)j * a.dv.token, a.head_dim);
}

// Adds the splits of dK and dV: eight columns a thread, 16 threads a row.
template <class T>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kv_kernel(AttnArgs a, int width, int blocks) {
    const int b = blockIdx.x / blocks / a.kv_heads, hk = blockIdx.x / blocks % a.kv_heads;
    const Seq sq = sequence(a, b);
    const int j = blockIdx.x % blocks * kJoinRows + threadIdx.x / 16, col = threadIdx.x % 16 * 8;
    if (j >= sq.k_rows || col >= a.head_dim) return;
    const bool v_part = blockIdx.y;
    const float* part = v_part ? a.part_v : a.part;
    const int64_t row = (a.q_start ? sq.k0 : (int64_t)b * a.k_len) + j;
    float x[8] = {};
    for (int s = 0; s < a.kv_splits; ++s) {
        float v[8];
        load8(part + (((int64_t)s * a.kv_heads + hk) * a.k_tokens + row) * width + col, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += v[e];
    }
    const float mul = v_part ? kLower<T> : a.scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= mul;
    const Tensor& t = v_part ? a.dv : a.dk;
    store8((T*)(rows_of(t, b, sq.k0, hk) + (int64_t)j * t.token) + col, x);
}

// Packed token axes: writes the rows that no sequence covers, which lie before
// the first one, between two, after the last and past q_len or k_len of a
// longer one, as zeros (lse: -inf); the products that take these tensors read
// whole token axes. Workgroups of gap x (the one before sequence x), most of
// which are empty: 1 to 2 us of a call over 13 sequences in 8192 tokens.
constexpr int kGapThreads = 256;
__global__ __launch_bounds__(kGapThreads) void attn_uncovered_kernel(AttnArgs a, int backward) {
    const bool keys = blockIdx.z;
    const int32_t* start = keys ? a.k_start : a.q_start;
    const int64_t tokens = keys ? a.k_tokens : a.q_tokens;
    const int most = keys ? a.k_len : a.q_len, groups = a.head_dim / 8;
    const int64_t each = (int64_t)(keys ? a.kv_heads : a.heads) * groups;
    const Tensor t = keys ? a.dk : backward ? a.dq : a.o;
    const u32x4 zero = {};
    for (int64_t gap = blockIdx.x; gap <= a.batch; gap += gridDim.x) {
        int n;
        int64_t from = 0, to = tokens;
        if (gap > 0) {
            from = packed(start, tokens, most, (int)gap - 1, n);
            from += n;
        }
        if (gap < a.batch) to = packed(start, tokens, most, (int)gap, n);
        for (int64_t i = (int64_t)blockIdx.y * kGapThreads + threadIdx.x; i < (to - from) * each; i += (int64_t)gridDim.y * kGapThreads) {
            const int64_t row = from + i / each;
            const int h = (int)(i % each / groups), c = (int)(i % each % groups);
            *gptr((u32x4*)(rows_of(t, 0, row, h) + 16 * c)) = zero;
            if (keys) *gptr((u32x4*)(rows_of(a.dv, 0, row, h) + 16 * c)) = zero;
            if (!backward && c == 0) gptr(a.lse)[(int64_t)h * a.q_tokens + row] = -INFINITY;
        }
    }
}

// ------------------------------------------------------------------ host ----

opt_status check_attention(const opt_attention_desc* a) {
    if (!a) return fail(OPT_EINVAL, "desc is NULL");
    if (a->dtype != OPT_BF16 && a->dtype != OPT_F16) return fail(OPT_EUNSUPPORTED, "dtype must be OPT_BF16 or OPT_F16");
    if (a->batch < 0 || a->q_len < 0 || a->k_len < 0) return fail(OPT_EINVAL, "negative batch or length");
    if (a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads)
        return fail(OPT_EINVAL, "heads must be a positive multiple of kv_heads");
    if (a->head_dim < 8 || a->head_dim % 8) return fail(OPT_EINVAL, "head_dim must be a positive multiple of 8");
    if (a->head_dim > 128) return fail(OPT_EUNSUPPORTED, "head_dim must be <= 128");
    // the sums of a length, an offset between lengths and a window fit in 32 bits
    if (a->q_len > (1 << 29) || a->k_len > (1 << 29)) return fail(OPT_EUNSUPPORTED, "sequence too long");
    if (a->window < 0) return fail(OPT_EINVAL, "window must be >= 0");
    if (a->window > 0 && !a->causal) return fail(OPT_EUNSUPPORTED, "a window needs causal");
    if (!(a->scale > 0.f) || !(a->scale < INFINITY)) return fail(OPT_EINVAL, "scale must be positive and finite");
    if ((a->q_start != nullptr) != (a->k_start != nullptr)) return fail(OPT_EINVAL, "q_start and k_start come together");
    if (a->q_start && (a->q_lens || a->k_lens)) return fail(OPT_EINVAL, "lengths and packed offsets exclude each other");
    for (const int32_t* p : {a->q_start, a->k_start, a->q_lens, a->k_lens})
        if (!train_aligned(p, 4)) return fail(OPT_EINVAL, "an offset or length array is not aligned to 4 bytes");
    if (a->q_start && (a->q_tokens < 0 || a->k_tokens < 0)) return fail(OPT_EINVAL, "negative q_tokens or k_tokens");
    if (a->q_start && (a->q_tokens > int64_t(1) << 40 || a->k_tokens > int64_t(1) << 40))
        return fail(OPT_EUNSUPPORTED, "too many packed tokens");
    // workgroups of all launches are counted in 31 bits
    const double longest = a->q_len > a->k_len ? a->q_len : a->k_len;
    if ((longest / kJoinRows + 1) * a->batch * a->heads > INT32_MAX)
        return fail(OPT_EUNSUPPORTED, "too many row blocks");
    return OPT_OK;
}

opt_status tensor(const opt_attention_desc* a, const opt_attention_tensor* t, const char* name, bool empty, Tensor& out) {
    if (!t) return fail(OPT_EINVAL, "%s is NULL", name);
    if (empty) return OPT_OK;
    if (!t->data) return fail(OPT_EINVAL, "%s has no data", name);
    if (!train_aligned(t->data, 16)) return fail(OPT_EINVAL, "%s is not 16-byte aligned", name);
    if (t->batch_stride < 0 || t->token_stride < 0 || t->head_stride < 0) return fail(OPT_EINVAL, "negative stride of %s", name);
    if (t->batch_stride % 8 || t->token_stride % 8 || t->head_stride % 8)
        return fail(OPT_EINVAL, "strides of %s must be multiples of 8", name);
    if (t->token_stride > (1 << 24)) return fail(OPT_EUNSUPPORTED, "token stride of %s is above 2^24", name);
    out = {(char*)t->data, t->batch_stride * 2, t->token_stride * 2, t->head_stride * 2};
    return OPT_OK;
}

// Rows of an output's token axis.
int64_t out_tokens(const opt_attention_desc* a, bool keys) {
    return a->q_start ? (keys ? a->k_tokens : a->q_tokens) : (keys ? a->k_len : a->q_len);
}

// An output's rows must not share memory: with more than one of each, no stride may be 0.
opt_status output(const opt_attention_desc* a, const opt_attention_tensor* t, const char* name, bool empty, int heads,
                  int64_t tokens, Tensor& out) {
    if (opt_status st = tensor(a, t, name, empty, out)) return st;
    if (empty) return OPT_OK;
    if ((!a->q_start && a->batch > 1 && t->batch_stride == 0) || (tokens > 1 && t->token_stride < a->head_dim) ||
        (heads > 1 && t->head_stride < a->head_dim))
        return fail(OPT_EINVAL, "rows of %s overlap", name);
    return OPT_OK;
}

AttnArgs attn_args(const opt_attention_desc* a) {
    AttnArgs x = {};
    x.q_start = a->q_start, x.k_start = a->k_start, x.q_lens = a->q_lens, x.k_lens = a->k_lens;
    x.q_tokens = a->q_start ? a->q_tokens : (int64_t)a->batch * a->q_len;
    x.k_tokens = a->q_start ? a->k_tokens : (int64_t)a->batch * a->k_len;
    x.batch = a->batch, x.heads = a->heads, x.kv_heads = a->kv_heads, x.head_dim = a->head_dim;
    x.q_len = a->q_start && a->q_tokens < a->q_len ? (int32_t)a->q_tokens : a->q_len;   // no sequence is longer than all
    x.k_len = a->q_start && a->k_tokens < a->k_len ? (int32_t)a->k_tokens : a->k_len;
    x.causal = a->causal != 0, x.scale = a->scale;
    x.window = a->window < x.k_len ? a->window : 0;   // as long as the keys: it hides none
    return x;
}

int64_t row_blocks(int len, int rows) { return (len + rows - 1) / rows; }

// Blocks of 128 rows with work to do. Packed sequences: the launch covers the
// longest for each, the blocks past a shorter one's end leave at once.
int64_t busy_blocks(const AttnArgs& x, bool keys) {
    const int64_t n = row_blocks(keys ? x.k_len : x.q_len, 128) * x.batch;
    const int64_t packed = (keys ? x.k_tokens : x.q_tokens) / 128 + x.batch;
    return (x.q_start && packed < n ? packed : n) * (keys ? x.kv_heads : x.heads);
}
// Tiles of 64 keys a block of queries steps through (or of queries a block of
// keys, over the heads of its group).
int64_t block_steps(const AttnArgs& x, bool keys) {
    const int len = keys ? x.q_len : x.k_len;
    const int64_t n = x.window && x.window + 128 < len ? x.window + 128 : len;
    return (n + kTile - 1) / kTile * (keys ? x.heads / x.kv_heads : 1);
}

// Parts to split a block's steps into, over workgroups: enough for one on each
// CU, but at least eight steps each, so that the partial sums stay below what
// is read. Twice as many for the keys of a causal sequence, whose blocks are
// uneven, if 32 steps are left to each (dK and dV of 4096 tokens, 16 / 8 heads
// of 128: 232 us without, 181 with; 4 x 1024: 69 and 87). For its queries
// twice as many gained nothing (46 against 42 us, 2048 tokens).
int splits_of(const AttnArgs& x, bool keys) {
    const int64_t wgs = busy_blocks(x, keys), steps = block_steps(x, keys);
    if (wgs == 0) return 1;
    int64_t s = 256 / wgs;
    if (s > steps / 8) s = steps / 8;
    if (s < 1) s = 1;
    if (keys && x.causal && wgs * s <= 256 && steps >= 64 * s) s *= 2;
    return (int)(s > 32 ? 32 : s);
}

enum Kind { FORWARD, DQ, DKV };

// Wavefronts and sets of a workgroup. `wgs`: workgroups of 128 rows with work.
//  - Up to one a CU: two sets. Also while there are few and uneven ones, the
//    longest of which would run on alone: causal, below 1024, of 32 steps at
//    least. Forward, us, two sets against one: 76 / 104 (3500 tokens, 16 heads
//    of 128), 83 / 101 (4096), but 37 / 33 (4 x 1024), 327 / 287 (4 x 4096).
//    dK and dV with dQ: 946 / 1182 (8192 tokens, 8 key heads), but 440 / 428
//    (2 x 4096, 16 of 96). The forward pass of packed sequences, which are
//    uneven among themselves, up to 2048 where two such workgroups fit a CU:
//    77 / 105 (8192 tokens, the longest sequence 4194, 16 heads of 64).
//  - Plenty: eight wavefronts share each tile. Half the copies into LDS, which
//    cost power, and the clock follows the power drawn: 277 us against 298 of
//    four (forward, 8192 tokens), 521 / 534 (not causal); few ones are left
//    with a part-filled last round: 51 / 46 (6 x 1000, 16 heads of 64). Not
//    for the keys at head_dim <= 64, where three workgroups of four fit a CU:
//    1072 / 1026.
//  - Else one set of four.
enum Shape { W4S2, W4S1, W8S1 };
Shape shape_of(const AttnArgs& x, Kind kind) {
    const bool keys = kind == DKV, narrow = x.head_dim <= 64;
    const int splits = keys ? x.kv_splits : x.splits;
    const int64_t wgs = busy_blocks(x, keys) * splits, steps = block_steps(x, keys) / splits;
    const int64_t few = x.q_start && narrow && kind == FORWARD ? 2048 : 1024;
    if (wgs <= 256 || (x.causal && wgs < few && steps >= 32)) return W4S2;
    return wgs >= 1024 && !(keys && narrow) ? W8S1 : W4S1;
}

template <class T, int DB, int W, int SETS>
void launch_shape(Kind kind, AttnArgs x, hipStream_t s) {
    const bool keys = kind == DKV;
    int64_t blocks = row_blocks(keys ? x.k_len : x.q_len, 32 * W), sequences = x.batch;
    // the list where it is shorter than a block of every sequence for each of the longest one's
    const int64_t list = (keys ? x.k_tokens : x.q_tokens) / (32 * W) + x.batch;
    x.listed = x.q_start && x.batch <= kListed && list < blocks * sequences;
    if (x.listed) blocks = list, sequences = 1;
    const int64_t grid = blocks * sequences * (keys ? (int64_t)x.kv_heads * x.kv_splits : (int64_t)x.heads * x.splits);
    constexpr int64_t most = most_blocks(SETS * 64 * W);
    for (int64_t first = 0; first < grid; first += most) {
        const dim3 g((uint32_t)(grid - first < most ? grid - first : most)), n(SETS * 64 * W);
        x.first = (uint32_t)first;
        if (kind == FORWARD) attn_forward_kernel<T, DB, W, SETS><<<g, n, 0, s>>>(x, (int)blocks);
        else if (kind == DQ) attn_dq_kernel<T, DB, W, SETS><<<g, n, 0, s>>>(x, (int)blocks);
        else attn_dkv_kernel<T, DB, W, SETS><<<g, n, 0, s>>>(x, (int)blocks);
    }
}

template <class T, int DB>
void launch(Kind kind, const AttnArgs& x, hipStream_t s) {
    if ((kind == DKV ? x.k_len : x.q_len) == 0 || x.batch == 0) return;
    switch (shape_of(x, kind)) {
        case W4S2: launch_shape<T, DB, 4, 2>(kind, x, s); break;
        case W4S1: launch_shape<T, DB, 4, 1>(kind, x, s); break;
        case W8S1: launch_shape<T, DB, 8, 1>(kind, x, s); break;
    }
    if (kind == DKV ? x.kv_splits > 1 : x.splits > 1) {
        const int jb = (int)row_blocks(kind == DKV ? x.k_len : x.q_len, kJoinRows);
        const int64_t n = (int64_t)jb * x.batch * (kind == DKV ? x.kv_heads : x.heads);
        const dim3 j((uint32_t)n, kind == DKV ? 2 : 1);
        if (kind == FORWARD) attn_join_kernel<T, true><<<j, kJoinThreads, 0, s>>>(x, 32 * DB, jb);
        else if (kind == DQ) attn_join_kernel<T, false><<<j, kJoinThreads, 0, s>>>(x, 32 * DB, jb);
        else attn_join_kv_kernel<T><<<j, kJoinThreads, 0, s>>>(x, 32 * DB, jb);
    }
}
template <class T>
void launch(Kind kind, const AttnArgs& x, hipStream_t s) {
    if (x.head_dim <= 32) launch<T, 1>(kind, x, s);
    else if (x.head_dim <= 64) launch<T, 2>(kind, x, s);
    else if (x.head_dim <= 96) launch<T, 3>(kind, x, s);
    else launch<T, 4>(kind, x, s);
}
void launch(Kind kind, int32_t dtype, const AttnArgs& x, hipStream_t s) {
    dtype == OPT_BF16 ? launch<__bf16>(kind, x, s) : launch<_Float16>(kind, x, s);
}

void launch_uncovered(bool backward, const AttnArgs& x, hipStream_t s) {
    if (!x.q_start) return;
    const int64_t gaps = (int64_t)x.batch + 1, slices = 1024 / gaps;
    const dim3 g((uint32_t)(gaps < 65536 ? gaps : 65536), (uint32_t)(slices < 1 ? 1 : slices > 64 ? 64 : slices), backward ? 2 : 1);
    attn_uncovered_kernel<<<g, kGapThreads, 0, s>>>(x, backward);
}

// The workspace: D (backward), then the splits' partial results. dQ's are
// joined before dK's and dV's are written, in the same place.
struct Space {
    uint64_t delta, part, part_v, part_m, part_l, bytes;
    int splits, kv_splits;
};
Space space_of(const AttnArgs& x, bool backward) {
    const auto up = [](uint64_t n) { return (n + 255) / 256 * 256; };
    const uint64_t rows = (uint64_t)x.q_tokens * (uint64_t)x.heads, width = (uint64_t)(x.head_dim + 31) / 32 * 32;
    const uint64_t k_rows = (uint64_t)x.k_tokens * (uint64_t)x.kv_heads;
    Space s = {};
    s.splits = rows ? splits_of(x, false) : 1;
    s.kv_splits = backward && k_rows ? splits_of(x, true) : 1;
    if (backward) s.bytes += up(rows * 4);
    s.part = s.bytes;
    const uint64_t q_part = s.splits > 1 ? up(s.splits * rows * width * 4) : 0;
    if (backward) {
        const uint64_t k_part = s.kv_splits > 1 ? up(s.kv_splits * k_rows * width * 4) : 0;
        s.part_v = s.part + k_part;
        s.bytes += q_part > 2 * k_part ? q_part : 2 * k_part;
    } else if (s.splits > 1) {
        s.bytes += q_part;
        s.part_m = s.bytes, s.bytes += up(s.splits * rows * 4);
        s.part_l = s.bytes, s.bytes += up(s.splits * rows * 4);
    }
    return s;
}
void use_space(AttnArgs& x, const Space& s, void* ws) {
    char* p = (char*)ws;
    x.splits = s.splits, x.kv_splits = s.kv_splits;
    x.delta = (float*)(p + s.delta);
    x.part = (float*)(p + s.part), x.part_v = (float*)(p + s.part_v);
    x.part_m = (float*)(p + s.part_m), x.part_l = (float*)(p + s.part_l);
}

opt_status check_workspace(const void* ws, uint64_t bytes, uint64_t need) {
    if (bytes < need) return fail(OPT_ENOWS, "workspace of %llu bytes, %llu needed", (unsigned long long)bytes,
                                  (unsigned long long)need);
    if (need && (!ws || !train_aligned(ws, 256))) return fail(OPT_EINVAL, "workspace is NULL or not 256-byte aligned");
    return OPT_OK;
}

}  // namespace
}  // namespace matopt

using namespace matopt;

extern "C" {

opt_status opt_attention_workspace_size(const opt_attention_desc* a, int32_t backward, uint64_t* bytes) {
    if (!bytes) return fail(OPT_EINVAL, "bytes is NULL");
    if (opt_status st = check_attention(a)) return st;
    *bytes = space_of(attn_args(a), backward != 0).bytes;
    return OPT_OK;
}

opt_status opt_attention_forward(const opt_attention_desc* a, const opt_attention_tensor* q,
                                 const opt_attention_tensor* k, const opt_attention_tensor* v,
                                 const opt_attention_tensor* out, float* lse, void* workspace,
                                 uint64_t workspace_bytes, void* stream) {
    if (opt_status st = check_attention(a)) return st;
    AttnArgs x = attn_args(a);
    // nothing to read, and nothing to write (packed tokens are written without sequences too)
    const bool no_q = x.q_tokens == 0 || a->q_len == 0 || a->batch == 0, no_k = x.k_tokens == 0 || a->k_len == 0;
    const bool no_out = x.q_tokens == 0;
    if (opt_status st = tensor(a, q, "q", no_q, x.q)) return st;
    if (opt_status st = tensor(a, k, "k", no_k || no_q, x.k)) return st;
    if (opt_status st = tensor(a, v, "v", no_k || no_q, x.v)) return st;
    if (opt_status st = output(a, out, "out", no_out, a->heads, out_tokens(a, false), x.o)) return st;
    if (!no_out && (!lse || !train_aligned(lse, 4))) return fail(OPT_EINVAL, "lse is NULL or not aligned to 4 bytes");
    const Space space = space_of(x, false);
    if (opt_status st = check_workspace(workspace, workspace_bytes, space.bytes)) return st;
    if (no_out) return OPT_OK;
    if (opt_status st = train_pending()) return st;
    x.lse = lse;
    use_space(x, space, workspace);
    launch(FORWARD, a->dtype, x, (hipStream_t)stream);
    launch_uncovered(false, x, (hipStream_t)stream);
    return train_launched("attention");
}

opt_status opt_attention_backward(const opt_attention_desc* a, const opt_attention_tensor* dout,
                                  const opt_attention_tensor* q, const opt_attention_tensor* k,
                                  const opt_attention_tensor* v, const opt_attention_tensor* out, const float* lse,
                                  const opt_attention_tensor* dq, const opt_attention_tensor* dk,
                                  const opt_attention_tensor* dv, void* workspace, uint64_t workspace_bytes,
                                  void* stream) {
    if (opt_status st = check_attention(a)) return st;
    AttnArgs x = attn_args(a);
    const bool no_q = x.q_tokens == 0 || a->q_len == 0 || a->batch == 0;
    const bool no_k = x.k_tokens == 0 || a->k_len == 0 || a->batch == 0;
    const bool no_dq = x.q_tokens == 0, no_dk = x.k_tokens == 0;   // nothing to write
    if (opt_status st = tensor(a, dout, "dout", no_q, x.dout)) return st;
    if (opt_status st = tensor(a, q, "q", no_q, x.q)) return st;
    if (opt_status st = tensor(a, k, "k", no_k, x.k)) return st;
    if (opt_status st = tensor(a, v, "v", no_k, x.v)) return st;
    if (opt_status st = tensor(a, out, "out", no_q, x.o)) return st;
    if (!no_q && (!lse || !train_aligned(lse, 4))) return fail(OPT_EINVAL, "lse is NULL or not aligned to 4 bytes");
    if (opt_status st = output(a, dq, "dq", no_dq, a->heads, out_tokens(a, false), x.dq)) return st;
    if (opt_status st = output(a, dk, "dk", no_dk, a->kv_heads, out_tokens(a, true), x.dk)) return st;
    if (opt_status st = output(a, dv, "dv", no_dk, a->kv_heads, out_tokens(a, true), x.dv)) return st;
    const Space space = space_of(x, true);
    if (opt_status st = check_workspace(workspace, workspace_bytes, space.bytes)) return st;
    if (no_dq && no_dk) return OPT_OK;
    if (opt_status st = train_pending()) return st;
    x.lse = (float*)lse;
    use_space(x, space, workspace);
    if (!no_q) launch(DQ, a->dtype, x, (hipStream_t)stream);
    if (!no_k) launch(DKV, a->dtype, x, (hipStream_t)stream);
    launch_uncovered(true, x, (hipStream_t)stream);
    return train_launched("attention backward");
}

}  // extern "C"
