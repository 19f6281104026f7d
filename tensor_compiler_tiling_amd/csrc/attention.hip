// Attention of new tokens over the key-value cache.
//
//   z_j = scale * q . k_j,  y = sum_j exp(z_j) v_j / sum_j exp(z_j)
//
// over the places j that the token sees.  One pass over the keys with the
// running maximum m of z and the running sum: what has been summed is scaled
// by exp(m_old - m_new) where m grows (Milakov and Gimelshein, "Online normalizer
// calculation for softmax", 2018), here only by kLag at least.  All of it in units of
// log2, with exp2.
//
// The heads of a group share their keys, so the rows of a product are (token,
// head of the group) pairs, token by token, and a tile of rows reads a page
// once for all of them.  Both products are computed transposed:
//   Z^T [keys x rows] = K Q^T,   Y^T [dim x rows] = V^T P^T
// An instruction's result then has one row of q a lane, whose maximum, sum and
// scaling are the lane's own, and holds neighbouring keys in a lane's
// registers, in the order in which the second product takes them as its right
// operand: the weights P never leave their registers.  The left operand of the
// second product, V^T, comes from LDS by the transposing read.
//
// Roundings: products of 16-bit values summed in fp32; maximum, weights and sums
// fp32; P goes into the second product rounded to the type of q (by up to 2^-8 or 2^-11
// of a weight, at random, as the result's own rounding), the sum of the weights
// is made from the unrounded ones.  8-bit rows widen to 16 bits with their
// scale, exactly in bf16.  For fp16, whose range is short, they widen to half
// their value (448 * 2^8 would pass 65504; what falls below 2^-24 so is less than
// fp16's own smallest step), and P is held times 2^7: with m lagging by up to
// 2^8, below, its range is 2^-31 to 2^15 of the largest weight.
#include "kv_device.hpp"

#include <type_traits>

namespace ct {

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef unsigned int uint2v __attribute__((ext_vector_type(2)));

enum { DT_E4M3 = 3 };

constexpr float kLag = 8.0f;  // log2 by which weights may pass 1 before what is summed is scaled

// log2 of what P is held times
template <int DT> constexpr float p_shift() { return DT == DT_F16 ? 7.0f : 0.0f; }

template <int DT>
__device__ __forceinline__ floatx16 mma32(uint4v a, uint4v b, floatx16 c) {
    if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(halfx8, a), __builtin_bit_cast(halfx8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <int DT>
__device__ __forceinline__ floatx4 mma16(uint4v a, uint4v b, floatx4 c) {
    if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, a), __builtin_bit_cast(halfx8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <int DT>
__device__ __forceinline__ unsigned pack2(float a, float b) {
    if constexpr (DT == DT_F16)
        return __builtin_bit_cast(unsigned, halfx2{(_Float16)a, (_Float16)b});
    else
        return __builtin_bit_cast(unsigned, bf16x2{(__bf16)a, (__bf16)b});
}

// Four 8-bit codes times a power of two, as two dwords of the 16-bit type.
template <int DT>
__device__ __forceinline__ uint2v widen4(unsigned codes, float scale) {
    if constexpr (DT == DT_F16)
        return {__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, false)),
                __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, true))};
    else
        return {__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, false)),
                __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, true))};
}

// 8 values of a 16-byte piece of 16 codes.
template <int DT>
__device__ __forceinline__ uint4v widen8(uint4v piece, int half, float scale) {
    const uint2v a = widen4<DT>(piece[2 * half], scale), b = widen4<DT>(piece[2 * half + 1], scale);
    return uint4v{a[0], a[1], b[0], b[1]};
}

// Half the scale for fp16 (above); the other half is in the score's factor
// and in the last step.
template <int DT, bool Q8>
__device__ __forceinline__ float used_scale(float s) { return DT == DT_F16 ? 0.5f * s : s; }

// Four keys of a column: lane i of 16 names row i / 4 of 4, columns 4 (i % 4) to
// + 3 of 16, and gets column i.
__device__ __forceinline__ uint2v read_transposed(const uint16_t* p) {
    typedef __attribute__((address_space(3))) shortx4 lds_short4;
    return __builtin_bit_cast(uint2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)p));
}

// Keeps the compiler from moving a wave's accesses of LDS past each other; the
// hardware runs them in order.
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local"); }

// A value that the compiler takes for new here: it is made at this place, and what
// a rare path makes of it is not made ahead of the loop, where it would be kept in
// registers.
template <typename T>
__device__ __forceinline__ T in_place(T v) {
    asm volatile("" : "+v"(v));
    return v;
}

// What sums at maximum m are scaled by for a greater one; 0 past 2^-126.
__device__ __forceinline__ float fall_to(float m, float next) { return m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - next); }

// A sum of a wave or part at the common maximum: what is infinite stays so (in 8 bits
// nothing is).
__device__ __forceinline__ float fallen(float o, float fall) {
    return fall == 0.0f && !__builtin_isfinite(o) ? o : o * fall;
}

// The greater of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float max_of_halves(float v) {
    typedef unsigned int pair __attribute__((ext_vector_type(2)));
    const pair r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Ends a turn of the tile kernel: what was written to LDS is there, and no access
// of it crosses (loads of global memory may be on their way).
__device__ __forceinline__ void end_turn() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A value that all lanes share, as a scalar.  What is the wave's own (its index,
// its keys, its loop's ends) goes through this, so that the branches on it are
// scalar too.  With conditions as masks, where registers were short, the compiler
// (ROCm 7.2) copied values away before it had put the mask back: waves that had
// skipped a branch lost them.
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int wave_of() { return scalar((int)threadIdx.x >> 6); }

__device__ __forceinline__ uint4v load16(const char* p) {
    uint4v v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// Values that are not finite become 0; what is returned is not 0 if there was any.
// 16-bit caches by arithmetic on both halves of a dword: adding one in the exponent's
// last place carries into the sign's exactly where all of the exponent is ones.
// Compares have a lane mask a value alive, for which the row forms' scalars did not
// suffice (128 wide 140 spilled, 4 so; one token of 1200 12.3 -> 11.1 us, windows 28.4 ->
// 24.5).  Between the widening of 8-bit rows compares are the faster (trees 32 x 64
// 155 us and 163, 16 x 8 tokens over 4096 58.3 and 59.7) and spill nothing in the loop.
template <int DT, bool Q8>
__device__ __forceinline__ unsigned clear_not_finite(uint4v& v) {
    constexpr unsigned E = DT == DT_F16 ? 0x7c00u : 0x7f80u, ONE = DT == DT_F16 ? 0x04000400u : 0x00800080u;
    unsigned bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (Q8) {
            if ((v[i] & E) == E) v[i] &= 0xffff0000u, bad = 1;
            if (((v[i] >> 16) & E) == E) v[i] &= 0xffffu, bad = 1;
        } else {
            const unsigned hit = ((v[i] & (E << 16 | E)) + ONE) & 0x80008000u;
            v[i] &= ~((hit - (hit >> 15)) | hit);
            bad |= hit;
        }
    }
    return bad;
}

// ------------------------------------------------------------ what is seen --
// A tile of rows of one kv head: its sequence and first row.
struct Tile {
    int seq, r0;       // seq < 0: none
    int first, count;  // the sequence's new tokens
    int len, ctx;      // keys that the pages hold, and the place of the first new token
};

// The tile-th tile of `rows` rows, counted over the sequences.  With starts,
// every wave counts the sequences' tiles by itself, 64 at a time.
__device__ __forceinline__ Tile find_tile(const AttendParams& p, int tile, int rows) {
    Tile t{-1, 0, 0, 0, 0, 0};
    if (!p.b.starts) {
        const int per = (p.b.even * p.group + rows - 1) / rows;
        t.seq = tile / per;
        if (t.seq >= p.b.sequences) t.seq = -1;
        t.r0 = (tile - t.seq * per) * rows;
    } else {
        const int lane = threadIdx.x & 63;
        int before = 0;
        for (int s0 = 0; s0 < p.b.sequences; s0 += 64) {
            const int seq = s0 + lane;
            int n = 0;
            if (seq < p.b.sequences) n = (span_of(p.b, seq).count * p.group + rows - 1) / rows;
            int upto = n;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int u = __shfl_up(upto, o);
                if (lane >= o) upto += u;
            }
            const unsigned long long hit = __ballot(before + upto > tile);
            if (hit) {
                const int at = __builtin_ctzll(hit);
                t.seq = s0 + at;
                t.r0 = (tile - before - __shfl(upto - n, at)) * rows;
                break;
            }
            before += __shfl(upto, 63);
        }
    }
    t.seq = scalar(t.seq);
    t.r0 = scalar(t.r0);
    if (t.seq < 0) return t;
    const Span sp = span_of(p.b, t.seq);
    t.first = scalar(sp.first);
    t.count = scalar(sp.count);
    const int len = scalar(length_of(p.b, t.seq)), most = p.b.width * p.c.page;
    t.ctx = len - t.count;
    t.len = len < most ? len : most;
    return t;
}

// The key tiles (of KT keys) that rows [r0, r0 + rows) of a tile can see: those
// of the sinks, [0, sinks), then [from, from + rest).
struct Keys {
    int sinks, from, rest;
    __device__ __forceinline__ int total() const { return sinks + rest; }
    __device__ __forceinline__ int at(int i) const { return i < sinks ? i : from + i - sinks; }
};

template <int KT>
__device__ __forceinline__ Keys keys_of(const AttendParams& p, const Tile& t, int r0, int rows) {
    const int last = t.count * p.group - 1;
    const int i0 = r0 / p.group, i1 = (r0 + rows - 1 < last ? r0 + rows - 1 : last) / p.group;
    // the places of the rows' tokens: a node of a tree may lie anywhere behind the context
    const int lowest = p.tree ? t.ctx - 1 : t.ctx + i0, highest = p.tree ? t.len - 1 : t.ctx + i1;
    const int lo = clampi(lowest - p.window + 1, 0, t.len), hi = clampi(highest + 1, 0, t.len);
    const int cover = (hi + KT - 1) / KT, first = ((p.sinks < lo ? p.sinks : lo) + KT - 1) / KT;
    const int sinks = scalar(first < cover ? first : cover), from = scalar(lo / KT > sinks ? lo / KT : sinks);
    return {sinks, from, scalar(cover > from ? cover - from : 0)};
}

// Bits [a, b) of 64.
__device__ __forceinline__ unsigned long long bits_between(int a, int b) {
    a = clampi(a, 0, 64);
    b = clampi(b, 0, 64);
    if (b <= a) return 0;
    return (~0ull >> (64 - (b - a))) << a;
}

// What a row sees.
struct Row {
    int token, head;  // of the call's tokens and of q's heads; token < 0: no row
    int pos;
    int nodes;        // of a tree: how many drafted nodes it sees
};

__device__ __forceinline__ unsigned long long tree_word(const AttendParams& p, const Tile& t, int token, int word) {
    const int left = t.count - word * 64;  // nodes beyond the sequence's are none
    if (word < 0 || word >= p.words || left <= 0) return 0;
    const unsigned long long w = (unsigned long long)p.tree[(long long)token * p.words + word];
    return left >= 64 ? w : w & (~0ull >> (64 - left));
}

__device__ __forceinline__ Row row_of(const AttendParams& p, const Tile& t, int head0, int r) {
    Row row{-1, 0, -1, 0};
    if (r >= t.count * p.group) return row;
    const int i = r / p.group;
    row.token = t.first + i;
    row.head = head0 + r - i * p.group;
    row.pos = t.ctx + i;
    if (p.tree) {
        const int words = (t.count + 63) / 64;
        for (int w = 0; w < words; ++w) row.nodes += __builtin_popcountll(tree_word(p, t, row.token, w));
        row.pos = t.ctx + row.nodes - 1;
    }
    return row;
}

// Keys k0 to k0 + 63 that a row sees, as bits.
__device__ __forceinline__ unsigned long long seen(const AttendParams& p, const Tile& t, const Row& row, int k0) {
    if (row.token < 0) return 0;
    // places before the row's own, in its window or among the sinks
    const int end = (p.tree ? t.ctx - 1 : row.pos) + 1 - k0, all = t.len - k0;
    unsigned long long m = bits_between(row.pos - p.window + 1 - k0, end) | bits_between(0, end < p.sinks - k0 ? end : p.sinks - k0);
    if (p.tree && k0 + 64 > t.ctx) {
        const int j0 = k0 - t.ctx;  // the first key as a node; negative where the tile begins in the context
        const int word = j0 >= 0 ? j0 >> 6 : -((63 - j0) >> 6), sh = j0 - word * 64;
        unsigned long long n = tree_word(p, t, row.token, word) >> sh;
        if (sh) n |= tree_word(p, t, row.token, word + 1) << (64 - sh);
        if (row.nodes > p.window) {
            // the nodes that it sees lie at ctx, ctx + 1, ...: drop those outside of the window, but for sinks
            int rank = 0;
            for (int w = 0; w <= word; ++w) {
                const unsigned long long u = tree_word(p, t, row.token, w);
                rank += __builtin_popcountll(w < word ? u : sh ? u & (~0ull >> (64 - sh)) : 0);
            }
            unsigned long long left = n;
            const int keep = p.sinks - t.ctx, drop = row.nodes - p.window;
            for (; left && rank < drop; ++rank, left &= left - 1)
                if (rank >= keep) n &= ~(left & -left);
        }
        m |= n;
    }
    return m & bits_between(0, all);
}

// Does a row see any of keys [a, b)?
__device__ __forceinline__ bool sees_any(const AttendParams& p, const Tile& t, const Row& row, int a, int b) {
    if (a < 0) a = 0;
    if (b > t.len) b = t.len;
    const int end = (p.tree ? t.ctx - 1 : row.pos) + 1, low = row.pos - p.window + 1, last = b < end ? b : end;
    bool any = (a > low ? a : low) < last || a < (last < p.sinks ? last : p.sinks);
    if (p.tree)
        for (int k = a > t.ctx ? a : t.ctx; k < b; k += 64) any |= (seen(p, t, row, k) & bits_between(0, b - k)) != 0;
    return row.token >= 0 && any;
}

// The maximum of a row in stages [from, to) that has found none: -infinity where it
// sees nothing there, else the least number.  All its scores are then -infinity (or
// NaN, as its sums are), and unless other parts have a greater maximum, its result is
// 0 / 0 and not that of a row that sees nothing: NaN, also where V is infinite, so
// without other parts its weights' sum l is NaN.
template <int KT>
__device__ __forceinline__ void least_maximum(const AttendParams& p, const Tile& t, const Row& row, const Keys& keys, int from, int to,
                                              float& m, float& l) {
    bool any = false;
    if (from < keys.sinks) any |= sees_any(p, t, row, from * KT, (to < keys.sinks ? to : keys.sinks) * KT);
    if (to > keys.sinks) any |= sees_any(p, t, row, keys.at(from > keys.sinks ? from : keys.sinks) * KT, (keys.at(to - 1) + 1) * KT);
    any = any && m == -INFINITY;
    l = any && p.parts <= 1 ? __builtin_nanf("") : l;
    m = any ? -0x1.fffffep127f : m;
}

// Does every row among tokens [i0, i1] see all of keys [k0, k0 + KT)?
template <int KT>
__device__ __forceinline__ bool all_seen(const AttendParams& p, const Tile& t, int i0, int i1, int k0) {
    const int lowest = p.tree ? t.ctx - 1 : t.ctx + i0, highest = p.tree ? t.ctx + t.count - 1 : t.ctx + i1;
    if (k0 + KT > t.len || k0 + KT > lowest + 1) return false;
    return k0 > highest - p.window || k0 + KT <= p.sinks;
}

// A weight of 0 does not clear what is not finite.  Where some row of a stage does
// not see all of its keys, V therefore goes into the product without such values,
// and the rows that see one get it by this: a key's value in the cache, and of
// it what is not finite (0 for the others).  In 8 bits that is NaN, and what its scale
// takes past the range of the type.
template <int DT, bool Q8>
struct CacheRow {
    const char* v;
    float scale;
    int dim;
    __device__ __forceinline__ CacheRow(const AttendParams& p, const Tile& t, int head, int key) : dim(p.c.dim) {
        const Place at = place_of(p.c, key);
        int page = page_of(p.b, t.seq, at.index);
        if ((unsigned)page >= (unsigned)p.c.pages) page = 0;
        v = p.c.v + page * p.c.ld_page + at.in * p.c.ld_token + head * p.c.ld_head;
        // waited for here: on its way past a row that does not see the key, it would have the
        // loop over the keys begin with a wait for all loads
        if constexpr (Q8)
            scale = in_place(used_scale<DT, Q8>(p.c.vs[page * p.c.lds_page + at.in * p.c.lds_token + head * p.c.lds_head]));
    }
    __device__ __forceinline__ float not_finite(int d) const {
        d = d < dim ? d : dim - 1;  // what lies beyond is not stored
        if constexpr (Q8) {
            const float f = __builtin_amdgcn_cvt_f32_fp8((uint8_t)v[d], 0) * scale;
            return fabsf(f) <= (DT == DT_F16 ? 65504.0f : 0x1.fep127f) ? 0.0f : f * INFINITY;
        }
        const float f = Elem<DT>::to_f32(reinterpret_cast<const typename Elem<DT>::T*>(v)[d]);
        return __builtin_isfinite(f) ? 0.0f : f;
    }
};

// Which of keys k0 to k0 + KT - 1 have values that are infinite (or not finite), as
// bits: a key a lane, 16-bit caches only.
template <int DT, int KT>
__device__ __forceinline__ unsigned long long keys_with(const AttendParams& p, const Tile& t, int head, int k0, bool nan_too) {
    constexpr unsigned E = DT == DT_F16 ? 0x7c007c00u : 0x7f807f80u, ONE = DT == DT_F16 ? 0x04000400u : 0x00800080u;
    const int key = k0 + (int)(threadIdx.x & 63) % KT;
    const CacheRow<DT, false> row(p, t, head, key < t.len ? key : t.len - 1);
    unsigned hit = 0;
#pragma unroll 1
    for (int d = 0; d < p.c.dim; d += 16) {
        const uint4v v[2] = {load16(row.v + 2 * d), load16(row.v + 2 * d + 16)};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned u = v[i / 4][i % 4];
            // both halves: all ones in the exponent carry, and so does what is not E's pattern
            hit |= nan_too ? (u & E) + ONE : ~(((u & 0x7fff7fffu) ^ E) + 0x7fff7fffu);
        }
    }
    const unsigned long long all = __ballot((hit & 0x80008000u) && key < t.len);
    return KT == 64 ? all : all & ((1ull << KT) - 1);
}

// An infinity of V that a row sees makes its sum infinite, however small its weight.
// But a weight that rounds to 0 (below 2^-31 of the largest in fp16) gives NaN in the
// product, as does an infinite sum whose scale falls to 0; and which keys share a
// maximum depends on how they are divided.  So if there are infinities in the wave's
// stages from, from + step, ... below to, sums (column + off(d, e) in o[d][e]) that have
// become NaN are made anew from what is not finite in the cache; those in which
// nothing is stay NaN.  (To look for infinities in every stage as V is brought to LDS
// cost 5 to 12%.)
template <int DT, int KT, typename V, int N, typename F>
__device__ __forceinline__ void mend_nan(const AttendParams& p, const Tile& t, const Row& row, const Keys& keys, int head, int from,
                                         int to, int step, V (&o)[N], float l, int column, F off) {
    constexpr int E = sizeof(V) / 4;
    float sum = 0.0f;  // NaN if any of them is, or is infinite
#pragma unroll
    for (int d = 0; d < N; ++d)
#pragma unroll
        for (int e = 0; e < E; ++e) sum = fmaf(o[d][e], 0.0f, sum);
    // where the weights are NaN, all is
    if (__builtin_expect(!__any(sum != sum && l == l && row.token >= 0), 1)) return;
    unsigned made[(N * E + 31) / 32] = {}, any = 0;
#pragma unroll
    for (int d = 0; d < N; ++d)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int n = d * E + e;
            made[n / 32] |= (o[d][e] != o[d][e] ? 1u : 0u) << n % 32;
        }
#pragma unroll
    for (unsigned m : made) any |= m;
    if (!__any(any && row.token >= 0)) return;
    bool infinite = false;
#pragma unroll 1
    for (int i = from; i < to && !infinite; i += step) infinite = keys_with<DT, KT>(p, t, head, keys.at(i) * KT, false) != 0;
    if (!infinite) return;
#pragma unroll
    for (int d = 0; d < N; ++d)
#pragma unroll
        for (int e = 0; e < E; ++e) o[d][e] = o[d][e] != o[d][e] ? 0.0f : o[d][e];
#pragma unroll 1
    for (int i = from; i < to; i += step) {
        const int k0 = keys.at(i) * KT;
        const unsigned long long bits = seen(p, t, row, k0);
#pragma unroll 1
        for (unsigned long long bad = keys_with<DT, KT>(p, t, head, k0, true); bad; bad &= bad - 1) {
            const int k = __builtin_ctzll(bad);
            const CacheRow<DT, false> v(p, t, head, k0 + k);
            const unsigned on = 0u - (unsigned)(bits >> k & 1);
            const int d0 = in_place(column);
#pragma unroll
            for (int d = 0; d < N; ++d) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int n = d * E + e;
                    const unsigned mask = on & (0u - (made[n / 32] >> n % 32 & 1));
                    o[d][e] = in_place(o[d][e] + __uint_as_float(__float_as_uint(v.not_finite(d0 + off(d, e))) & mask));
                }
            }
        }
    }
#pragma unroll
    for (int d = 0; d < N; ++d)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int n = d * E + e;
            o[d][e] = (made[n / 32] >> n % 32 & 1) && o[d][e] == 0.0f ? __builtin_nanf("") : o[d][e];
        }
}

// ------------------------------------------------------------- the results --
// Four neighbouring elements of a row's sums from d.
template <int DT>
__device__ __forceinline__ void put4(const AttendParams& p, const Row& row, int part, int d, float a, float b, float c,
                                     float e, float inv) {
    if (row.token < 0 || d >= p.c.dim) return;
    if (p.parts > 1) {
        const long long at = ((long long)part * p.b.tokens + row.token) * (p.c.heads * p.group) + row.head;
        *reinterpret_cast<floatx4*>(p.part_o + at * p.c.dim + d) = floatx4{a, b, c, e};
    } else {
        const uint2v w = {pack2<DT>(a * inv, b * inv), pack2<DT>(c * inv, e * inv)};
        __builtin_memcpy(p.y + row.token * p.y_token + row.head * p.y_head + d * 2, &w, 8);
    }
}

__device__ __forceinline__ void put_weight(const AttendParams& p, const Row& row, int part, float m, float l) {
    if (row.token < 0 || p.parts <= 1) return;
    const long long at = ((long long)part * p.b.tokens + row.token) * (p.c.heads * p.group) + row.head;
    p.part_ml[2 * at] = m;
    p.part_ml[2 * at + 1] = l;
}

// 1 / l, 0 for a row that sees nothing (whose maximum is none).  With fp16 and 8 bits
// V is half (above).
template <int DT, bool Q8>
__device__ __forceinline__ float inverse(float l, float m) {
    return m == -INFINITY ? 0.0f : (DT == DT_F16 && Q8 ? 2.0f : 1.0f) / l;
}

// Key tiles of a part: none for the last parts where there are few.
__device__ __forceinline__ void part_of(const AttendParams& p, int total, int part, int& from, int& to) {
    const int each = (total + p.parts - 1) / p.parts;
    from = scalar(part * each < total ? part * each : total);
    to = scalar(from + each < total ? from + each : total);
}

// -------------------------------------------------------------- tile kernel --
// WAVES x 32 rows; KT keys a stage, brought to LDS in 16 bits (through registers,
// where 8-bit rows widen), two stages' room.  Rows of K in LDS are 16 bytes longer
// than dim: 16 neighbouring keys, read 16 bytes each, then cover all 64 banks.  Those
// of V lie 64 bytes (mod 256) apart: a transposing read takes 64 bytes of 8 keys.
//
// Measured: a prompt of 8192 tokens, 32 heads on 8, dim 128 bf16 575 us (550 GFLOP,
// 956 TFLOP/s; a library product of 8192^3 reaches 1227), matrix units 44% busy at
// the 1.9 GHz that the chip holds.  What bounds it is the products themselves at
// that clock: without the exponentials a copy took 539 us, without any weights
// 521, without reading LDS 541.  Long 16-bit caches of single tokens run at
// 5.1 TB/s.  Other forms of it took, for that prompt: two halves of the waves that
// take turns at products and weights, with two barriers a turn, 606 to 651 us; the
// second product's instructions between the exponentials 643 (a wave that waits for
// the matrix unit holds its own other work up); stages of 32 keys 890, workgroups of
// 4 waves 887 (against 747 then); more priority for the products 617.
template <int DT, bool Q8, int DP, int WAVES, int KT>
__global__ __launch_bounds__(WAVES * 64, (DP > 128 ? 1 : 2)) void attend_tile_kernel(AttendParams p) {
    constexpr int NT = WAVES * 64, ROWS = WAVES * 32, NK = KT / 32;
    constexpr int KP = DP + 8, VP = DP == 96 ? DP : DP + 32;  // elements
    constexpr int PIECE = Q8 ? 16 : 8;             // elements of 16 bytes of the cache
    constexpr int PR = DP / PIECE, ALL = KT * PR;  // pieces of a row, of a stage
    constexpr int NP = (ALL + NT - 1) / NT;        // a thread's
    constexpr int DS = DP / 16, DO = DP / 32;
    __shared__ __attribute__((aligned(16))) uint16_t s_k[2][KT * KP], s_v[2][KT * VP];
    __shared__ int s_dirty[2], s_bad[2][KT];  // the stage in which V, and a key's, was not finite
    __shared__ long long s_at[4 * WAVES][KT];  // where a stage's keys lie
    __shared__ float s_scale[Q8 ? 2 * WAVES : 1][KT][2];

    const int head = blockIdx.x % p.c.heads;
    const int rest = blockIdx.x / p.c.heads;
    const int part = rest % p.parts;
    // the last rows of a sequence see the most keys: first
    const Tile t = find_tile(p, p.tiles - 1 - rest / p.parts, ROWS);
    if (t.seq < 0) return;
    const int wave = wave_of(), lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    const Row row = row_of(p, t, head * p.group, t.r0 + wave * 32 + col);
    const Keys keys = keys_of<KT>(p, t, t.r0, ROWS);
    int from, to;
    part_of(p, keys.total(), part, from, to);
    // tokens of the wave's rows, and of the workgroup's
    const int most = t.count * p.group - 1, w0 = t.r0 + wave * 32;
    const int i0 = scalar(w0 / p.group), i1 = scalar((w0 + 31 < most ? w0 + 31 : most) / p.group);
    const int a0 = scalar(t.r0 / p.group), a1 = scalar((t.r0 + ROWS - 1 < most ? t.r0 + ROWS - 1 : most) / p.group);

    uint4v q[DS];
#pragma unroll
    for (int s = 0; s < DS; ++s) {
        q[s] = uint4v{0, 0, 0, 0};
        const int d = s * 16 + half * 8;
        if (row.token >= 0 && d < p.c.dim) q[s] = load16(p.q + row.token * p.q_token + row.head * p.q_head + d * 2);
    }
    floatx16 o[DO];
#pragma unroll
    for (int i = 0; i < DO; ++i) o[i] = floatx16{};
    float m = -INFINITY, l = 0.0f;

    // Staging.  Where a stage's keys lie is looked up some blocks of WAVES stages ahead,
    // a stage a wave and a key a lane, and left in LDS with the scales: at the first
    // turn of block b its waves ask for the pages of block b + 3, make the places of
    // b + 2 and have the scales of b + 1.
    const char* const kbase = p.c.k + head * p.c.ld_head;
    const char* const vbase = p.c.v + head * p.c.ld_head;
    const float* const ksbase = Q8 ? p.c.ks + head * p.c.lds_head : nullptr;
    const float* const vsbase = Q8 ? p.c.vs + head * p.c.lds_head : nullptr;
    int page = 0;
    float ks = 1.0f, vs = 1.0f;
    auto place = [&](int i) {
        const int key = keys.at(i) * KT + in_place(lane) % KT;
        return place_of(p.c, key < t.len ? key : t.len - 1);
    };
    auto ask_page = [&](int i) { return i < to ? page_of(p.b, t.seq, place(i).index) : 0; };
    auto put_place = [&](int i, int page) {
        if (i >= to) return;
        // a page that the pool does not have is read as its first
        const int pg = (unsigned)page < (unsigned)p.c.pages ? page : 0, in = place(i).in;
        s_at[(i - from) % (4 * WAVES)][in_place(lane) % KT] = pg * p.c.ld_page + in * p.c.ld_token;
        if constexpr (Q8) {
            const long long soff = pg * p.c.lds_page + in * p.c.lds_token;
            ks = used_scale<DT, Q8>(ksbase[soff]);
            vs = used_scale<DT, Q8>(vsbase[soff]);
        }
    };
    auto put_scales = [&](int i) {
        if constexpr (Q8) {
            if (i >= to) return;
            s_scale[(i - from) % (2 * WAVES)][lane % KT][0] = ks;
            s_scale[(i - from) % (2 * WAVES)][lane % KT][1] = vs;
        }
    };
    auto look_up = [&](int i) {  // i: a block's first stage
        put_scales(i + WAVES + wave);
        put_place(i + 2 * WAVES + wave, page);
        page = ask_page(i + 3 * WAVES + wave);
    };
    // A thread's pieces of K and of V: piece j of key key_of(j).
    constexpr bool EVEN = NT % PR == 0;
    uint4v rk[NP], rv[NP];
    const int key0 = (int)threadIdx.x / PR, piece0 = (int)threadIdx.x % PR;
    auto key_of = [&](int j) { return EVEN ? key0 + j * (NT / PR) : (j * NT + (int)threadIdx.x) / PR; };
    auto piece_of = [&](int j) { return EVEN ? piece0 : (j * NT + (int)threadIdx.x) % PR; };
#pragma unroll
    for (int j = 0; j < NP; ++j) rk[j] = rv[j] = uint4v{0, 0, 0, 0};  // those past dim stay so
    auto load_rows = [&](int i, const char* base, uint4v (&r)[NP]) {
        long long at[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) at[j] = s_at[(i - from) % (4 * WAVES)][key_of(j) % KT] + piece_of(j) * 16;
        if constexpr (EVEN && ALL % NT == 0) {
            if (piece0 * PIECE < p.c.dim) {
#pragma unroll
                for (int j = 0; j < NP; ++j) r[j] = load16(base + at[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NP; ++j)
                if (key_of(j) < KT && piece_of(j) * PIECE < p.c.dim) r[j] = load16(base + at[j]);
        }
    };
    auto store_k = [&](int i) {
        uint16_t* const to_k = s_k[(i - from) & 1];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            if (ALL % NT && key_of(j) >= KT) continue;
            const float f = Q8 ? s_scale[(i - from) % (2 * WAVES)][key_of(j)][0] : 1.0f;
#pragma unroll
            for (int e = 0; e < (Q8 ? 2 : 1); ++e)
                *reinterpret_cast<uint4v*>(to_k + key_of(j) * KP + piece_of(j) * PIECE + 8 * e) = Q8 ? widen8<DT>(rk[j], e, f) : rk[j];
        }
    };
    auto store_v = [&](int i) {
        const int k0 = keys.at(i) * KT, buf = (i - from) & 1;
        const bool whole = all_seen<KT>(p, t, a0, a1, k0);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            if (ALL % NT && key_of(j) >= KT) continue;
            const float f = Q8 ? s_scale[(i - from) % (2 * WAVES)][key_of(j)][1] : 1.0f;
            unsigned bad = 0;
#pragma unroll
            for (int e = 0; e < (Q8 ? 2 : 1); ++e) {
                uint4v v = Q8 ? widen8<DT>(rv[j], e, f) : rv[j];
                if (!whole) {
                    if (k0 + key_of(j) >= t.len) v = uint4v{0, 0, 0, 0};
                    bad |= clear_not_finite<DT, Q8>(v);
                }
                *reinterpret_cast<uint4v*>(s_v[buf] + key_of(j) * VP + piece_of(j) * PIECE + 8 * e) = v;
            }
            if (bad) s_dirty[buf] = s_bad[buf][key_of(j)] = i;
        }
    };
    if (threadIdx.x < 2) s_dirty[threadIdx.x] = -1;
    if (threadIdx.x < 2 * KT) (&s_bad[0][0])[threadIdx.x] = -1;

    // A turn: the first product of stage i and the second of stage i - 1, in one run;
    // the weights of stage i; then K of stage i + 1 and V of stage i to LDS, from
    // registers that were loaded in the turn before.  One barrier a turn.  A SIMD's two
    // waves soon run against each other, one's products beside the other's weights.
    //
    // Scheduling barriers hold the order of the run: each product has its operand read
    // from LDS AHEAD products before.  Left to itself the compiler reads, waits and
    // multiplies.
    constexpr int AHEAD = 6, FIRST = NK * DS, SECOND = 2 * NK * DO;
    floatx16 z[NK];
    uint4v w[2 * NK];  // the weights of 16 keys each
    auto products = [&](int i, auto with_first, auto with_second) {
        constexpr int BEGIN = decltype(with_first)::value ? 0 : FIRST, END = decltype(with_second)::value ? FIRST + SECOND : FIRST;
        const int ln = in_place(lane);  // made anew: registers are short
        const uint16_t* const krow = &s_k[(i - from) & 1][(ln & 31) * KP + (ln >> 5) * 8];
        const uint16_t* const vrow = &s_v[(i - from + 1) & 1][(4 * (ln >> 5) + (ln & 15) / 4) * VP + 16 * ((ln >> 4) & 1) + 4 * (ln & 3)];
        uint4v f[AHEAD];
        auto read = [&](int n) {
            if (n < FIRST) {
                f[n % AHEAD] = *reinterpret_cast<const uint4v*>(krow + n / DS * 32 * KP + n % DS * 16);
            } else {
                const uint16_t* const at = vrow + (n - FIRST) / DO * 16 * VP + (n - FIRST) % DO * 32;
                const uint2v a = read_transposed(at), b = read_transposed(at + 8 * VP);
                f[n % AHEAD] = uint4v{a[0], a[1], b[0], b[1]};
            }
        };
        if constexpr (BEGIN == 0) {
#pragma unroll
            for (int kt = 0; kt < NK; ++kt) z[kt] = floatx16{};
        }
#pragma unroll
        for (int n = BEGIN; n < BEGIN + AHEAD; ++n) read(n);
#pragma unroll
        for (int n = BEGIN; n < END; ++n) {
            __builtin_amdgcn_sched_barrier(0);
            if (n < FIRST) z[n / DS] = mma32<DT>(f[n % AHEAD], q[n % DS], z[n / DS]);
            else o[(n - FIRST) % DO] = mma32<DT>(f[n % AHEAD], w[(n - FIRST) / DO], o[(n - FIRST) % DO]);
            if (n + AHEAD < END) read(n + AHEAD);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto weights = [&](int i) {
        const int k0 = keys.at(i) * KT;
        if (!all_seen<KT>(p, t, i0, i1, k0)) {
            const unsigned long long bits = seen(p, t, row, k0) >> (4 * half);
#pragma unroll
            for (int kt = 0; kt < NK; ++kt)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (!(bits >> (kt * 32 + 8 * (e / 4) + e % 4) & 1)) z[kt][e] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int kt = 0; kt < NK; ++kt)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, z[kt][e]);
        top = max_of_halves(top) * p.scale;
        if (__any(top > m + kLag)) {
            const float next = fmaxf(m, top);
            const float fall = fall_to(m, next);
            l *= fall;
#pragma unroll
            for (int d = 0; d < DO; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= fall;
            m = next;
        }
        const float base = m == -INFINITY ? 0.0f : m - p_shift<DT>();
#pragma unroll
        for (int kt = 0; kt < NK; ++kt)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                z[kt][e] = __builtin_amdgcn_exp2f(fmaf(z[kt][e], p.scale, -base));
                l += z[kt][e];
            }
#pragma unroll
        for (int u = 0; u < 2 * NK; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[u][e] = pack2<DT>(z[u / 2][8 * (u % 2) + 2 * e], z[u / 2][8 * (u % 2) + 2 * e + 1]);
    };
    // what of stage i is not finite
    auto add_not_finite = [&](int i) {
        const int buf = (i - from) & 1;
        if (s_dirty[buf] != i) return;
        const int k0 = keys.at(i) * KT;
        const unsigned long long bits = seen(p, t, row, k0);
#pragma unroll 1
        for (int k = 0; k < KT; ++k) {
            if (s_bad[buf][k] != i) continue;
            const CacheRow<DT, Q8> v(p, t, head, k0 + k);
            if (!(bits >> k & 1)) continue;
            const int d0 = in_place(4 * half);
#pragma unroll
            for (int d = 0; d < DO; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] = in_place(o[d][e] + v.not_finite(d0 + d * 32 + 8 * (e / 4) + e % 4));
        }
    };
    // K of stage i + 1 and V of stage i, whose room is free while stage i's turn lasts
    auto load = [&](int i) {
        if (i < to) load_rows(i, vbase, rv);
        if (i + 1 < to) load_rows(i + 1, kbase, rk);
    };
    auto store = [&](int i) {
        if (i + 1 < to) store_k(i + 1);
        if (i < to) store_v(i);
    };
    // the blocks before the first
    const int page0 = ask_page(from + wave), page1 = ask_page(from + WAVES + wave);
    page = ask_page(from + 2 * WAVES + wave);
    put_place(from + wave, page0);
    put_scales(from + wave);
    put_place(from + WAVES + wave, page1);
    __syncthreads();
    if (from < to) {
        load_rows(from, kbase, rk);
        store_k(from);
        load(from);
    }
    __syncthreads();
    const bool idle = w0 > most;  // no rows
#pragma unroll
    for (int s = 0; s < DS; ++s) q[s] = in_place(q[s]);  // waited for here, not in the loop
    for (int i = from; i < to; ++i) {
        if ((i - from) % WAVES == 0) look_up(i);
        if (!idle) {
            if (i > from) {
                products(i, std::true_type{}, std::true_type{});
                add_not_finite(i - 1);
            } else {
                products(i, std::true_type{}, std::false_type{});
            }
            weights(i);
        }
        store(i);
        load(i + 1);
        end_turn();
    }
    if (from < to && !idle) {
        products(to, std::false_type{}, std::true_type{});
        add_not_finite(to - 1);
    }
    l += __shfl_xor(l, 32);
    if constexpr (!Q8)  // within the type's range 8 bits have NaN only, which stays NaN
        mend_nan<DT, KT>(p, t, row, keys, head, from, to, 1, o, l, 4 * half, [](int d, int e) { return d * 32 + 8 * (e / 4) + e % 4; });
    if (__builtin_expect(__any(m == -INFINITY), 0)) least_maximum<KT>(p, t, row, keys, from, to, m, l);
    const float inv = inverse<DT, Q8>(l, m);
#pragma unroll
    for (int d = 0; d < DO; ++d)
#pragma unroll
        for (int e = 0; e < 16; e += 4)
            put4<DT>(p, row, part, d * 32 + 2 * e + 4 * half, o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3], inv);
    if (half == 0) put_weight(p, row, part, m, l);
}

// --------------------------------------------------------------- row kernel --
// Up to 16 rows.  Memory bounds it, so a wave keeps its own keys: 32 at a time,
// K straight to the registers of the first product, V through the wave's own
// piece of LDS; no barrier until the waves' sums are joined.  Two workgroups a CU
// are enough: registers for three or four (__launch_bounds__) took 64 sequences of
// up to 8192 tokens in e4m3 from 161 to 176 and 206 us.  Measured: that 157 us
// (723 MB, 4.6 TB/s), 100 windows of 1024 fp16 24.5 (106 MB), 64 sequences of up to 8192
// bf16 333, one token of 1200 bf16 11.5 with the join, a chain of five reads that wait
// for each other.
template <int DT, bool Q8, int DP>
__global__ __launch_bounds__(256) void attend_rows_kernel(AttendParams p) {
    constexpr int WAVES = 4, KT = 32, ROWS = 16;
    constexpr int PITCH = DP + 16;         // of V in LDS: a transposing read takes 32 bytes of 16 keys
    constexpr int PIECE = Q8 ? 16 : 8;
    constexpr int PR = DP / PIECE;
    constexpr int NK = (PR + 3) / 4;       // pieces of a key that a lane loads
    constexpr int DS = NK * (Q8 ? 2 : 1);  // instructions of the first product
    constexpr int DO = DP / 16;
    constexpr int VLDS = KT * PITCH * 2, OLDS = ROWS * (DP + 4) * 4;
    static_assert(OLDS <= VLDS, "all waves' sums have room side by side at the end");
    __shared__ __attribute__((aligned(16))) char s_mem[VLDS * WAVES];
    __shared__ float s_ml[WAVES][ROWS][2];

    const int head = blockIdx.x % p.c.heads;
    const int rest = blockIdx.x / p.c.heads;
    const int part = rest % p.parts;
    const Tile t = find_tile(p, p.tiles - 1 - rest / p.parts, ROWS);
    if (t.seq < 0) return;
    const int wave = wave_of(), lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    uint16_t* const s_v = reinterpret_cast<uint16_t*>(s_mem + wave * VLDS);
    const Keys keys = keys_of<KT>(p, t, t.r0, ROWS);
    int from, to;
    part_of(p, keys.total(), part, from, to);
    const int most = t.count * p.group - 1;
    const int i0 = t.r0 / p.group, i1 = (t.r0 + ROWS - 1 < most ? t.r0 + ROWS - 1 : most) / p.group;

    const Row row = row_of(p, t, head * p.group, t.r0 + col);
    uint4v q[DS];
#pragma unroll
    for (int s = 0; s < DS; ++s) {
        q[s] = uint4v{0, 0, 0, 0};
        const int d = Q8 ? 16 * (4 * (s / 2) + quad) + 8 * (s % 2) : 8 * (4 * s + quad);
        if (row.token >= 0 && d < p.c.dim) q[s] = load16(p.q + row.token * p.q_token + row.head * p.q_head + d * 2);
    }
    floatx4 o[DO];
#pragma unroll
    for (int d = 0; d < DO; ++d) o[d] = floatx4{};
    float m = -INFINITY, l = 0.0f;

    const char* const kbase = p.c.k + head * p.c.ld_head;
    const char* const vbase = p.c.v + head * p.c.ld_head;
    // of a tile, a lane has keys col and 16 + col, and of those every fourth piece,
    // of K and of V: 64 bytes of 16 rows a load
    uint4v rk[2][NK], rv[2][NK];
    float sk[2] = {1.0f, 1.0f}, sv[2] = {1.0f, 1.0f};
    int pages[2] = {0, 0};
    auto place = [&](int i, int h) {
        const int key = keys.at(i) * KT + h * 16 + col;
        return place_of(p.c, key < t.len ? key : t.len - 1);
    };
    auto load_pages = [&](int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) pages[h] = page_of(p.b, t.seq, place(i, h).index);
    };
    auto load_rows = [&](int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // a page that the pool does not have is read as its first
            const int page = (unsigned)pages[h] < (unsigned)p.c.pages ? pages[h] : 0, in = place(i, h).in;
            const long long off = page * p.c.ld_page + in * p.c.ld_token + quad * 16;
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                rk[h][j] = rv[h][j] = uint4v{0, 0, 0, 0};
                if ((4 * j + quad) * PIECE < p.c.dim) {
                    rk[h][j] = load16(kbase + off + j * 64);
                    rv[h][j] = load16(vbase + off + j * 64);
                }
            }
            if constexpr (Q8) {
                const long long soff = page * p.c.lds_page + in * p.c.lds_token + head * p.c.lds_head;
                sk[h] = used_scale<DT, Q8>(p.c.ks[soff]);
                sv[h] = used_scale<DT, Q8>(p.c.vs[soff]);
            }
        }
    };

    if (from + wave < to) {
        load_pages(from + wave);
        load_rows(from + wave);
        if (from + wave + WAVES < to) load_pages(from + wave + WAVES);
    }
    for (int i = from + wave; i < to; i += WAVES) {
        const int k0 = keys.at(i) * KT;
        const bool whole = all_seen<KT>(p, t, i0, i1, k0);
        unsigned hit[2] = {0, 0};  // whether V of the lane's keys is not finite
        // V to LDS, and the first product: both free their registers
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const int k = h * 16 + col;
                if (PR % 4 && 4 * j + quad >= PR) continue;
#pragma unroll
                for (int e = 0; e < (Q8 ? 2 : 1); ++e) {
                    uint4v v = Q8 ? widen8<DT>(rv[h][j], e, sv[h]) : rv[h][j];
                    if (!whole) {
                        if (k0 + k >= t.len) v = uint4v{0, 0, 0, 0};
                        hit[h] |= clear_not_finite<DT, Q8>(v);
                    }
                    *reinterpret_cast<uint4v*>(s_v + k * PITCH + (4 * j + quad) * PIECE + 8 * e) = v;
                }
            }
        floatx4 z[2];
        z[0] = z[1] = floatx4{};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < DS; ++s) {
                const uint4v a = Q8 ? widen8<DT>(rk[h][s / 2], s % 2, sk[h]) : rk[h][s];
                z[h] = mma16<DT>(a, q[s], z[h]);
            }
        if (i + WAVES < to) {
            load_rows(i + WAVES);
            if (i + 2 * WAVES < to) load_pages(i + 2 * WAVES);
        }
        uint4v w;
        if (!whole) {
            const unsigned bits = (unsigned)seen(p, t, row, k0) >> (4 * quad);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(bits >> (h * 16 + e) & 1)) z[h][e] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, z[h][e]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32)) * p.scale;
        if (__any(top > m + kLag)) {
            const float next = fmaxf(m, top);
            const float fall = fall_to(m, next);
            l *= fall;
#pragma unroll
            for (int d = 0; d < DO; ++d) o[d] *= fall;
            m = next;
        }
        const float base = m == -INFINITY ? 0.0f : m - p_shift<DT>();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                z[h][e] = __builtin_amdgcn_exp2f(fmaf(z[h][e], p.scale, -base));
                l += z[h][e];
            }
            w[2 * h] = pack2<DT>(z[h][0], z[h][1]);
            w[2 * h + 1] = pack2<DT>(z[h][2], z[h][3]);
        }
        wave_fence();  // V is read by other lanes than those that wrote it
        const uint16_t* vrow = s_v + (4 * quad + col / 4) * PITCH + 4 * (col & 3);
#pragma unroll
        for (int d = 0; d < DO; ++d) {
            const uint2v a = read_transposed(vrow + d * 16), b = read_transposed(vrow + 16 * PITCH + d * 16);
            const uint4v v = {a[0], a[1], b[0], b[1]};
            o[d] = mma16<DT>(v, w, o[d]);
        }
        wave_fence();  // and written anew once they have
        const unsigned bad = (hit[0] ? 1u << col : 0) | (hit[1] ? 0x10000u << col : 0);
        if (__any(bad)) {
#pragma unroll 1
            for (int k = 0; k < KT; ++k) {
                if (!__any(bad >> k & 1)) continue;
                const CacheRow<DT, Q8> v(p, t, head, k0 + k);
                if (!(seen(p, t, row, k0) >> k & 1)) continue;
                const int d0 = in_place(4 * quad);
#pragma unroll
                for (int d = 0; d < DO; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[d][e] = in_place(o[d][e] + v.not_finite(d0 + d * 16 + e));
            }
        }
    }
    // the waves' sums, brought to their common maximum and added in order
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if constexpr (!Q8)  // as above
        mend_nan<DT, KT>(p, t, row, keys, head, from + wave, to, WAVES, o, l, 4 * quad, [](int d, int e) { return d * 16 + e; });
    if (quad == 0) {
        s_ml[wave][col][0] = m;
        s_ml[wave][col][1] = l;
    }
    __syncthreads();  // V in LDS is no longer needed either
    float* const s_o = reinterpret_cast<float*>(s_mem);
    float total = 0.0f, mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) mx = fmaxf(mx, s_ml[w][col][0]);
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const float mw = s_ml[w][col][0];
        total += mw == -INFINITY ? 0.0f : s_ml[w][col][1] * __builtin_amdgcn_exp2f(mw - mx);
    }
    const float fall = fall_to(m, mx);
    if (__builtin_expect(__any(mx == -INFINITY), 0)) least_maximum<KT>(p, t, row, keys, from, to, mx, total);
    if (!Q8 && __builtin_expect(__any(fall == 0.0f), 0)) {
#pragma unroll
        for (int d = 0; d < DO; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] = fallen(o[d][e], fall);
    } else {
#pragma unroll
        for (int d = 0; d < DO; ++d) o[d] *= fall;
    }
#pragma unroll
    for (int d = 0; d < DO; ++d)
        *reinterpret_cast<floatx4*>(s_o + wave * OLDS / 4 + col * (DP + 4) + d * 16 + quad * 4) = o[d];
    __syncthreads();
    const float inv = inverse<DT, Q8>(total, mx);
#pragma unroll
    for (int d = 0; d < DO; ++d) {
        if (d % WAVES != wave) continue;
        floatx4 v = {};
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            v += *reinterpret_cast<const floatx4*>(s_o + w * OLDS / 4 + col * (DP + 4) + d * 16 + quad * 4);
        put4<DT>(p, row, part, d * 16 + quad * 4, v[0], v[1], v[2], v[3], inv);
    }
    if (wave == 0 && quad == 0) put_weight(p, row, part, mx, total);
}

// --------------------------------------------------------------------- join --
// W waves a row: the parts' sums, brought to their common maximum and added in
// order, every wave's W-th part by itself first.  All of a row's maxima are read
// at once, a part a lane.  (64 parts of 32 rows: 25 us read one after another, 4 so.)
template <int DT, bool Q8, int W>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams p) {
    static_assert(W == 1 || W == 4, "a workgroup has 4 waves");
    __shared__ floatx4 s_o[W > 1 ? W : 1][64];
    const int heads = p.c.heads * p.group, wave = wave_of(), lane = threadIdx.x & 63;
    const long long rows = p.b.tokens * heads;  // below 2^26
    const int r = W > 1 ? (int)blockIdx.x : (int)blockIdx.x * 4 + wave;
    if (r >= rows) return;
    const int token = r / heads, head = r - token * heads;
    if (sequence_of(p.b, token) < 0) return;  // no row: nobody wrote its parts
    float m[2], l[2], mx = -INFINITY;  // parts lane and lane + 64
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = lane + 64 * i;
        m[i] = -INFINITY, l[i] = 0.0f;
        if (s < p.parts) m[i] = p.part_ml[2 * (s * rows + r)], l[i] = p.part_ml[2 * (s * rows + r) + 1];
        mx = fmaxf(mx, m[i]);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        m[i] = fall_to(m[i], mx);  // sums of no key are zeros
        total += l[i] * m[i];
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) total += __shfl_xor(total, o);
    floatx4 sum = {};
    const bool on = lane * 4 < p.c.dim;
    const float* const at = p.part_o + (long long)r * p.c.dim + lane * 4;
    constexpr int U = 8;  // parts whose rows are on their way together
    auto add = [&](auto far) {
        for (int s0 = W > 1 ? wave : 0; s0 < p.parts; s0 += U * W) {
            floatx4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = s0 + u * W;
                v[u] = floatx4{};
                if (on && s < p.parts) v[u] = *reinterpret_cast<const floatx4*>(at + s * rows * p.c.dim);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = s0 + u * W;
                const float fall = __shfl(s < 64 ? m[0] : m[1], s & 63);
                if constexpr (!decltype(far)::value) sum += v[u] * fall;
                else
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[e] += fallen(v[u][e], fall);
            }
        }
    };
    // maxima so far apart that a part's scale is 0 are rare (1 us a call if all went that way)
    if (!Q8 && __builtin_expect(__any(m[0] == 0.0f || m[1] == 0.0f), 0)) add(std::true_type{});
    else add(std::false_type{});
    if constexpr (W > 1) {
        s_o[wave][lane] = sum;
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int w = 1; w < W; ++w) sum += s_o[w][lane];
    }
    const float inv = inverse<DT, Q8>(total == 0.0f ? __builtin_nanf("") : total, mx);  // 0 / 0 where V is infinite too
    if (!on) return;
    const uint2v w = {pack2<DT>(sum[0] * inv, sum[1] * inv), pack2<DT>(sum[2] * inv, sum[3] * inv)};
    __builtin_memcpy(p.y + token * p.y_token + head * p.y_head + lane * 8, &w, 8);
}

// ------------------------------------------------------------------- launch --
template <int DT, bool Q8, int DP>
void launch_dim(const AttendPlan& plan, const AttendParams& p, hipStream_t stream) {
    const dim3 grid((unsigned)((long long)p.tiles * p.parts * p.c.heads));
    constexpr int WAVES = DP > 128 ? 4 : 8;
    if (plan.form == ATT_TILE)
        attend_tile_kernel<DT, Q8, DP, WAVES, 64><<<grid, dim3(WAVES * 64), 0, stream>>>(p);
    else
        attend_rows_kernel<DT, Q8, DP><<<grid, dim3(256), 0, stream>>>(p);
}

template <int DT, bool Q8>
hipError_t launch_type(const AttendPlan& plan, const AttendParams& p, hipStream_t stream) {
    if (p.c.dim <= 64) launch_dim<DT, Q8, 64>(plan, p, stream);
    else if (p.c.dim <= 96) launch_dim<DT, Q8, 96>(plan, p, stream);
    else if (p.c.dim <= 128) launch_dim<DT, Q8, 128>(plan, p, stream);
    else if (p.c.dim <= 192) launch_dim<DT, Q8, 192>(plan, p, stream);
    else launch_dim<DT, Q8, 256>(plan, p, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.parts <= 1) return e;
    const long long rows = (long long)p.b.tokens * p.c.heads * p.group;
    // a wave a row where the parts are few, a workgroup where they are many
    if (p.parts <= 8)
        attend_join_kernel<DT, Q8, 1><<<dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream>>>(p);
    else
        attend_join_kernel<DT, Q8, 4><<<dim3((unsigned)rows), dim3(256), 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attend(const AttendPlan& plan, const AttendParams& p, int cache_dt, int dt, hipStream_t stream) {
    (void)hipGetLastError();
    if (dt == DT_F16) return cache_dt == DT_E4M3 ? launch_type<DT_F16, true>(plan, p, stream) : launch_type<DT_F16, false>(plan, p, stream);
    return cache_dt == DT_E4M3 ? launch_type<DT_BF16, true>(plan, p, stream) : launch_type<DT_BF16, false>(plan, p, stream);
}

}  // namespace ct
