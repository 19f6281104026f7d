// Linear layer: y = act(scale * x w^T + bias) * gate + residual.
//
// x [M][K] and w [N][K] both hold the reduction contiguously, so every type
// is read the same way, in 16-byte chunks of a row: a chunk is 4 fp32, 8
// half-precision or 16 e4m3 elements, a stage of the reduction is 128 bytes
// of every row of a tile, and only the matrix instruction differs.  Which
// element of the reduction a lane's registers hold does not matter as long as
// both operands hold the same one, so the chunks go to the instructions as
// they lie: no operand is rearranged.
//
// The weights are the instruction's first operand (its rows) and x the second
// (its columns): a lane's results then belong to one row of x, and the rows
// of w are dealt to the instruction's rows so that they are neighbours in it
// (4, or 16 with 32 x 32 instructions), which go on to LDS in 16-byte vectors
// and come back as whole lines of y, gate and residual.
#include "ct_device.hpp"
#include "block_kernels.hpp"

#include <atomic>
#include <type_traits>

namespace ct {

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int uint4v __attribute__((ext_vector_type(4)));
typedef int int8v __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void_t;

// 8-bit operands: DT_E4M3 on the 8-bit instruction, which aligns the products
// of every 8 neighbours of the reduction to the largest of them and cuts what
// lies 2^-13 below it (a product of 4 beside one of 2^16 is lost whole;
// measured, with the cut the same on the older 8-bit instructions): sums off by
// 1.5e-5 of their size in the 2-norm on normally distributed rows, whatever K.
// That is 1/130 of the rounding of a bf16 result and 1/16 of an fp16 one, for
// twice the rate; a cut is at most 1/512 of what rounding a factor to e4m3 may
// have moved the group's largest product by.  DT_E4M3_WIDE widens the operands
// to fp16, exactly, and takes its instruction, whose sums keep fp32: for fp32
// results (4096 x 8192 x 4096 221 us, 112 to bf16 on the other), and for up to 32
// rows of x, whatever form the sizes choose, so that a token's sums do not
// depend on the layer's (the weights' reading bounds those products: tiles of
// 8 x 256 x 16384 8.8 us, 8.0 on the 8-bit instruction, 32 x 4096 x 4096 8.8 and 8.6).
enum { DT_E4M3 = 3, DT_E4M3_WIDE = 4 };
enum { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

constexpr int kBufRaw = 0x00020000;        // raw buffer descriptor
constexpr unsigned kBufOut = 0x80000000u;  // an offset past every buffer here (all below 2 GiB): reads zeros

template <int DT> constexpr int elem_size() { return DT == DT_F32 ? 4 : DT >= DT_E4M3 ? 1 : 2; }

__device__ __forceinline__ int8v join(uint4v lo, uint4v hi) {
    return __builtin_bit_cast(int8v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Elements 8 i .. 8 i + 7 of a chunk of 8-bit elements as fp16.
__device__ __forceinline__ halfx8 widen(uint4v v, int i) {
    typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
    const halfx2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * i], 1.0f, false);
    const halfx2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * i], 1.0f, true);
    const halfx2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * i + 1], 1.0f, false);
    const halfx2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * i + 1], 1.0f, true);
    return halfx8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The products of two pairs of chunks, 32 x 32 results: lane l holds chunks of
// row l % 32 of each operand; lanes l / 32 hold different ones.
template <int DT>
__device__ __forceinline__ floatx16 mma32(uint4v a0, uint4v a1, uint4v b0, uint4v b1, floatx16 c) {
    if constexpr (DT == DT_E4M3) {
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(a0, a1), join(b0, b1), c, 0, 0, 0, 0, 0, 0);
    } else if constexpr (DT == DT_E4M3_WIDE) {
#pragma unroll
        for (int i = 0; i < 2; ++i) c = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen(a0, i), widen(b0, i), c, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) c = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen(a1, i), widen(b1, i), c, 0, 0, 0);
        return c;
    } else if constexpr (DT == DT_F16) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(halfx8, a0), __builtin_bit_cast(halfx8, b0), c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(halfx8, a1), __builtin_bit_cast(halfx8, b1), c, 0, 0, 0);
    } else if constexpr (DT == DT_BF16) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a0), __builtin_bit_cast(bf16x8, b0), c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a1), __builtin_bit_cast(bf16x8, b1), c, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a0[i]), __uint_as_float(b0[i]), c, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a1[i]), __uint_as_float(b1[i]), c, 0, 0, 0);
        return c;
    }
}

// The same for 16 x 16 results: lane l holds chunks of row l % 16.
template <int DT>
__device__ __forceinline__ floatx4 mma16(uint4v a0, uint4v a1, uint4v b0, uint4v b1, floatx4 c) {
    if constexpr (DT == DT_E4M3_WIDE) {
#pragma unroll
        for (int i = 0; i < 2; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(a0, i), widen(b0, i), c, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(a1, i), widen(b1, i), c, 0, 0, 0);
        return c;
    } else if constexpr (DT == DT_F16) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, a0), __builtin_bit_cast(halfx8, b0), c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, a1), __builtin_bit_cast(halfx8, b1), c, 0, 0, 0);
    } else if constexpr (DT == DT_BF16) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a0), __builtin_bit_cast(bf16x8, b0), c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a1), __builtin_bit_cast(bf16x8, b1), c, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a0[i]), __uint_as_float(b0[i]), c, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a1[i]), __uint_as_float(b1[i]), c, 0, 0, 0);
        return c;
    }
}

// ---------------------------------------------------------------- epilogue --
// z / (1 + exp(-u)); exp and the reciprocal run on the hardware units, about 1 ulp
// each.  WHOLE: with e = exp(-|u|) it is z e / (1 + e) for negative u, so a small
// result keeps its digits until e leaves the range of fp32 (2^-126), and the
// exponent's rounding, |u| 2^-24 of the result by itself, is carried along.
// Not WHOLE: neither, for 16-bit results, where that rounding is below 2^-17 of
// the result, and results below 2^-119 become zeros (8192 x 8192 x 1024 bf16 with
// silu 140 us, 151 WHOLE).
template <bool WHOLE>
__device__ __forceinline__ float sigmoid_times(float z, float u) {
    if constexpr (!WHOLE) return z * __builtin_amdgcn_rcpf(1.0f + dev_exp(-u));
    const float t = fmaxf(-fabsf(u), -128.0f);  // exp2 of it is 0, and infinities have no remainder
    const float hi = t * 1.44269504f;           // log2(e) to 24 bits, and the rest of it
    const float lo = fmaf(t, 1.925963e-8f, fmaf(t, 1.44269504f, -hi));
    const float e0 = __builtin_amdgcn_exp2f(hi);
    const float e = fmaf(e0, lo * 0.69314718f, e0);
    return z * (u < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e);
}

// erfc(a / sqrt 2) / 2, the normal distribution's tail beyond a >= 0, to a few
// units in the last place of a value that falls as exp(-a^2 / 2): that exponential
// times a polynomial in t = 1 / (1 + 0.3 a) (the form of Hastings, "Approximations
// for Digital Computers", 1955).  The coefficients are a least-squares fit of
// the relative error, reweighted until it is even: 1.5e-7 over 0 <= a <= 14.
// 4096 x 8192 x 4096 bf16 with gelu 239 us (249 with the device library's erff, whose
// 1 + erf loses the tail, 262 with its erfcf).
__device__ __forceinline__ float normal_tail(float a) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, a, 1.0f));
    float p = 0.0356747732f;
    p = fmaf(p, t, -0.157203078f);
    p = fmaf(p, t, 0.206353515f);
    p = fmaf(p, t, -0.053683646f);
    p = fmaf(p, t, 0.128561631f);
    p = fmaf(p, t, 0.0999134928f);
    p = fmaf(p, t, 0.120753959f);
    p = fmaf(p, t, 0.119629301f);
    return p * t * __builtin_amdgcn_exp2f(-0.72134752f * (a * a));  // log2(e) / 2
}

// z times the normal distribution function.  For negative z that is its tail:
// as (1 + erf) / 2 the digits would cancel.
__device__ __forceinline__ float gelu(float z) {
    const float q = normal_tail(fabsf(z));
    return z * (z < 0.0f ? q : 1.0f - q);
}

template <int ACT, bool WHOLE>
__device__ __forceinline__ float activated(float z) {
    if constexpr (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays
    if constexpr (ACT == ACT_GELU) return gelu(z);
    // 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)), u = sqrt(2 / pi) (z + 0.044715 z^3)
    if constexpr (ACT == ACT_GELU_TANH) return sigmoid_times<WHOLE>(z, 1.5957691f * fmaf(0.044715f * z * z, z, z));
    if constexpr (ACT == ACT_SILU) return sigmoid_times<WHOLE>(z, z);
    return z;
}

// f(a constant of the activation's value)
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f) {
    switch (act) {
        case ACT_RELU: f(std::integral_constant<int, ACT_RELU>{}); break;
        case ACT_GELU: f(std::integral_constant<int, ACT_GELU>{}); break;
        case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>{}); break;
        case ACT_SILU: f(std::integral_constant<int, ACT_SILU>{}); break;
        default: f(std::integral_constant<int, ACT_NONE>{}); break;
    }
}

template <int V>
__device__ __forceinline__ void activate(float (&z)[V], int act) {
    with_activation(act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = activated<decltype(a)::value, true>(z[i]);
    });
}

__device__ __forceinline__ float load_out(const char* p, int dt) {
    if (dt == DT_F32) return *reinterpret_cast<const float*>(p);
    const uint16_t u = *reinterpret_cast<const uint16_t*>(p);
    return dt == DT_BF16 ? Elem<DT_BF16>::to_f32(u) : (float)__builtin_bit_cast(_Float16, u);
}

__device__ __forceinline__ uint16_t round_half(float f, int dt) {
    return dt == DT_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)f) : __builtin_bit_cast(uint16_t, (_Float16)f);
}

__device__ __forceinline__ void store_out(char* p, int dt, float v) {
    if (dt == DT_F32)
        *reinterpret_cast<float*>(p) = v;
    else
        *reinterpret_cast<uint16_t*>(p) = round_half(v, dt);
}

// V neighbouring elements, at any address their type allows: one access of up
// to 16 bytes each, whatever its alignment (1011 x 1500 x 2047 fp16, whose rows of
// y are 8-byte aligned: 28 us with an access an element, 26 so).
template <int V>
__device__ __forceinline__ void load_out_vec(const char* p, int dt, float (&f)[V]) {
    if (dt == DT_F32) {
        __builtin_memcpy(f, p, V * 4);
    } else {
        uint16_t u[V];
        __builtin_memcpy(u, p, V * 2);
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] = dt == DT_BF16 ? Elem<DT_BF16>::to_f32(u[i]) : (float)__builtin_bit_cast(_Float16, u[i]);
    }
}

template <int V>
__device__ __forceinline__ void store_out_vec(char* p, int dt, const float (&f)[V]) {
    if (dt == DT_F32) {
        __builtin_memcpy(p, f, V * 4);
    } else {
        uint16_t u[V];
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = round_half(f[i], dt);
        __builtin_memcpy(p, u, V * 2);
    }
}

// What finishing V neighbouring results of row m from column n reads beside
// them: gate (1 without one), residual (0) and the row's scale, loaded ahead.
template <int V>
struct Side {
    float g[V], r[V], xs;
    __device__ __forceinline__ void load(const LinearParams& p, int m, int n) {
        const int oes = p.out_dt == DT_F32 ? 4 : 2;
        const bool in = m < p.M && n < p.N, vec = n + V <= p.N;
        xs = p.xs && in ? p.xs[m] : 1.0f;
        get(p.gate, m * p.ldg + (long long)n * oes, p, n, in, vec, 1.0f, g);
        get(p.res, m * p.ldr + (long long)n * oes, p, n, in, vec, 0.0f, r);
    }
    __device__ __forceinline__ void get(const char* base, long long at, const LinearParams& p, int n, bool in, bool vec,
                                        float none, float (&f)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = none;
        if (!base || !in) return;
        if (vec) {
            load_out_vec<V>(base + at, p.out_dt, f);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (n + i < p.N) f[i] = load_out(base + at + i * (p.out_dt == DT_F32 ? 4 : 2), p.out_dt);
        }
    }
};

// Finish V neighbouring results of row m from column n, whose column scales
// and bias values are cs and cb: the one rounding to y's type is the last step.
template <int V>
__device__ __forceinline__ void finish(const LinearParams& p, int m, int n, const float (&acc)[V], const float (&cs)[V],
                                       const float (&cb)[V], const Side<V>& side) {
    if (m >= p.M || n >= p.N) return;
    const int oes = p.out_dt == DT_F32 ? 4 : 2;
    char* y = p.y + m * p.ldy + (long long)n * oes;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = acc[i] * side.xs * cs[i] + cb[i];
    activate<V>(v, p.act);
    if (p.gate) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= side.g[i];
    }
    if (p.res) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += side.r[i];
    }
    if (n + V <= p.N) {
        store_out_vec<V>(y, p.out_dt, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (n + i < p.N) store_out(y + i * oes, p.out_dt, v[i]);
    }
}

// Column values of V neighbours from n: scales and bias.
template <int V>
__device__ __forceinline__ void column_values(const LinearParams& p, int n, float (&s)[V], float (&b)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 1.0f, b[i] = 0.0f;
    if (n + V <= p.N) {
        if (p.ws) __builtin_memcpy(s, p.ws + n, V * 4);
        if (p.bias) __builtin_memcpy(b, p.bias + n, V * 4);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (p.ws && n + i < p.N) s[i] = p.ws[n + i];
        if (p.bias && n + i < p.N) b[i] = p.bias[n + i];
    }
}

// A chunk of a row from byte k of it (zeros from byte kbytes on), at any
// alignment: gfx950 takes a 16-byte global load at any address.
template <int ES>
__device__ __forceinline__ uint4v load_chunk(const char* row, long long k, int kbytes) {
    uint4v v = {0, 0, 0, 0};
    const long long left = kbytes - k;
    if (left >= 16) {
        __builtin_memcpy(&v, row + k, 16);
    } else if (left > 0) {
#pragma unroll
        for (int i = 0; i < 16 / ES; ++i) {
            if (i * ES >= left) continue;
            unsigned e;
            if constexpr (ES == 4)
                e = reinterpret_cast<const uint32_t*>(row + k)[i];
            else if constexpr (ES == 2)
                e = reinterpret_cast<const uint16_t*>(row + k)[i];
            else
                e = reinterpret_cast<const uint8_t*>(row + k)[i];
            v[i * ES / 4] |= e << (8 * (i * ES % 4));
        }
    }
    return v;
}

// 32 bytes from `sh` bits into the dword at p.  Loads at any dword address run
// at full rate, loads at other addresses at less than half (8 x 4096 x 4095 fp16
// 24 us with them, 13 with these and the shifts), so rows that start inside a
// dword are read in whole dwords, all of them holding bytes of the row.
__device__ __forceinline__ void load_shifted(const char* p, unsigned sh, uint4v& v0, uint4v& v1) {
    uint4v a, b;
    unsigned c;
    __builtin_memcpy(&a, __builtin_assume_aligned(p, 4), 16);
    __builtin_memcpy(&b, __builtin_assume_aligned(p + 16, 4), 16);
    __builtin_memcpy(&c, __builtin_assume_aligned(p + (sh ? 32 : 28), 4), 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v0[i] = __builtin_amdgcn_alignbit(i < 3 ? a[i + 1] : b[0], a[i], sh);
        v1[i] = __builtin_amdgcn_alignbit(i < 3 ? b[i + 1] : c, b[i], sh);
    }
}

// -------------------------------------------------------------- row form --
// Few rows of x (MF groups of 16).  Bound by reading the weights once.  A
// workgroup takes 16 rows of w; its waves share the reduction, wave v taking
// every NW-th stage, and lanes load both operands straight to registers in
// the order the 16 x 16 instruction takes them, 32 bytes of a stage of row l %
// 16 (chunks l / 16 and 4 + l / 16, or, AL false, the neighbours 2 (l / 16)
// and the next), so every load of w is used once and nothing passes through
// LDS before the waves' sums are joined there.  AL: rows start at dwords.
// Measured: one row, bf16, 8192 x 8192 weights (not in the caches) 28 us, 4.8
// TB/s, where a device copy moves 5.1 to 5.2; 4096 x 4096 (in them) 8.1 us.
constexpr int kRowWaves = 8;

template <int DT, int MF, bool AL>
__global__ __launch_bounds__(kRowWaves * 64) void linear_rows_kernel(LinearParams p) {
    constexpr int ES = elem_size<DT>();
    constexpr int U = (AL ? 8 : 4) / MF;  // stages in flight (bf16 1 x 4096 x 4096: 7.9 us with 8, 8.8 with 4)
    constexpr int R = MF + 1;           // rows a lane reads: w's, then x's
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16;
    const int lr = lane & 15, lg = lane >> 4;
    const char* row[R];
    row[0] = p.w + (n0 + lr < p.N ? n0 + lr : p.N - 1) * p.ldw;
#pragma unroll
    for (int f = 0; f < MF; ++f) row[1 + f] = p.x + (f * 16 + lr < p.M ? f * 16 + lr : p.M - 1) * p.ldx;
    const char* from[R];  // the lane's place in a stage (AL false: the dword it lies in)
    unsigned sh[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        from[r] = row[r] + lg * (AL ? 16 : 32);
        sh[r] = AL ? 0 : ((unsigned)(uintptr_t)from[r] & 3) * 8;
        from[r] -= sh[r] / 8;
    }
    floatx4 acc[MF] = {};
    struct Stage {
        uint4v v[R][2];
    };
    auto load = [&](Stage& g, int st) {  // a whole stage
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const char* at = from[r] + (long long)st * kStage;
            if constexpr (AL) {
                __builtin_memcpy(&g.v[r][0], __builtin_assume_aligned(at, 4), 16);
                __builtin_memcpy(&g.v[r][1], __builtin_assume_aligned(at + 64, 4), 16);
            } else {
                load_shifted(at, sh[r], g.v[r][0], g.v[r][1]);
            }
        }
    };
    auto multiply = [&](const Stage& g) {
#pragma unroll
        for (int f = 0; f < MF; ++f) acc[f] = mma16<DT>(g.v[0][0], g.v[0][1], g.v[1 + f][0], g.v[1 + f][1], acc[f]);
    };
    const int whole = p.kbytes / kStage;
    int st = wave;
    auto batch = [&](auto count) {  // that many of the wave's stages, all loaded before the first is used
        constexpr int C = decltype(count)::value;
        Stage g[C];
#pragma unroll
        for (int u = 0; u < C; ++u) load(g[u], st + u * kRowWaves);
#pragma unroll
        for (int u = 0; u < C; ++u) multiply(g[u]);
        st += C * kRowWaves;
    };
    while (st + (U - 1) * kRowWaves < whole) batch(std::integral_constant<int, U>{});
    if (U > 4 && st + 3 * kRowWaves < whole) batch(std::integral_constant<int, 4>{});
    if (U > 2 && st + kRowWaves < whole) batch(std::integral_constant<int, 2>{});
    if (st < whole) batch(std::integral_constant<int, 1>{});
    if (st == whole && whole * kStage < p.kbytes) {  // the rows' ends
        Stage g;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                g.v[r][h] = load_chunk<ES>(row[r], (long long)whole * kStage + lg * (AL ? 16 : 32) + h * (AL ? 64 : 16), p.kbytes);
        multiply(g);
    }
    // join the waves' sums: results [row of x][row of w], wave after wave
    __shared__ __align__(16) float red[kRowWaves][MF * 256];
#pragma unroll
    for (int f = 0; f < MF; ++f)
        *reinterpret_cast<floatx4*>(&red[wave][f * 256 + lr * 16 + lg * 4]) = acc[f];
    __syncthreads();
    for (int o = threadIdx.x; o < MF * 256; o += kRowWaves * 64) {
        const int m = o >> 4, n = n0 + (o & 15);
        if (m >= p.M || n >= p.N) continue;
        float v[1] = {0.0f}, s[1], b[1];
#pragma unroll
        for (int i = 0; i < kRowWaves; ++i) v[0] += red[i][o];
        column_values<1>(p, n, s, b);
        Side<1> side;
        side.load(p, m, n);
        finish<1>(p, m, n, v, s, b, side);
    }
}

// ------------------------------------------------------------- tile form --
// B x B results a workgroup (rows of x, rows of w), WM x WN waves of 32 MF x
// 32 NF each, on 32 x 32 instructions; KG such groups of waves share the
// reduction, each with stages, slots and sums of its own, joined at the end.
// A stage of an operand, 128 bytes of each of the tile's B rows, is an item;
// items lie in a ring of 2 L + 1 slots of LDS, x's of stage s at place 2 s, w's
// at 2 s + 1.  A wave reads its operands half a stage (64 bytes) ahead of the
// instructions that use them:
//
//   A(s):  start loading x of stage s + L | read half 1 of stage s | instructions on half 0
//          wait for stage s + 1, barrier
//   B(s):  start loading w of stage s + L | read half 0 of stage s + 1 | instructions on half 1
//
// so every LDS read has half a stage of matrix instructions to arrive, every
// load L - 1/2 stages or more, and one barrier a stage both ends the reads of
// a stage and publishes the next.  The slot that A(s) fills is that of w of
// stage s - 1, B(s)'s that of x of stage s, both read to the end before the
// barrier ahead.  Loads are spread over both halves because a CU takes them
// at 64 bytes a cycle: a stage's, started together, held the waves that
// issued them back from their matrix instructions.
//
// The 256 x 256 tile is bound by the matrix units (70% busy) and the issue of
// loads: 4096 x 8192 x 4096 bf16 217 to 229 us with the boxes' clocks (1.2 to 1.27
// PFLOP/s), 8192 x 8192 x 8192 bf16 814 (1.35), e4m3 416 (2.64), fp32 4096 x 4096 x
// 4096 945 (145 TFLOP/s).  The smaller ones, taken where that would leave CUs
// idle, are bound by what a CU takes in from L2, 75 GB/s (1024 x 1024 x 4096 bf16,
// 64 x 64, 15.7 us; 2048 x 2048 x 2048, 128 x 128, 21 to 23).
//
// LDS banks: a cycle serves 16 lanes of a 16-byte read from 64 banks (two
// 128-byte rows).  Chunk c of a row is stored at c ^ f(row), f giving the 8
// rows of equal parity among the 16 that are read together 8 different places:
// f = (row / 2) % 8 for x; for w, whose instruction rows 8 q + 4 h + i are its
// rows 16 h + 4 q + i of each 32 (a lane of half h then holds 16 neighbours),
// f = 4 (row / 16 % 2) + 2 (row / 4 % 2) + row / 2 % 2.
__device__ __forceinline__ int rot_x(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int rot_w(int row) { return ((row >> 2) & 4) | ((row >> 1) & 2) | ((row >> 1) & 1); }

// 16 bytes a lane from base + off (zeros where off is kBufOut or above) to the
// wave's 1024 bytes of LDS at `to`; base and `to` are wave-uniform.
__device__ __forceinline__ void load_to_lds(const char* base, unsigned off, char* to) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, 0x7fffffff, kBufRaw);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)to, 16, off, 0, 0, 0);
}

// Tile t in bands of 8 row tiles, row tiles fastest: what runs at one time on
// an XCD shares its L2.
__device__ __forceinline__ void tile_at(const LinearParams& p, unsigned t, int& tm, int& tn) {
    const unsigned band = 8u * p.tiles_n;
    const unsigned b = t / band, in = t - b * band;
    const unsigned rows = (unsigned)p.tiles_m - b * 8 < 8 ? p.tiles_m - b * 8 : 8;
    tn = in / rows;
    tm = b * 8 + (in - tn * rows);
}

// The work of this workgroup: a whole tile for the first p.full of them, a
// part of the reduction of one of the p.rest others after that (part -1: the
// whole).  XCD b % 8 takes one run of either.
__device__ __forceinline__ unsigned work_of(const LinearParams& p, int& part) {
    const bool whole = blockIdx.x < (unsigned)p.full;
    const unsigned nb = whole ? p.full : p.rest * p.S, b = blockIdx.x - (whole ? 0 : p.full);
    const unsigned xcd = b & 7, q = nb >> 3, r = nb & 7;
    const unsigned id = xcd * q + (xcd < r ? xcd : r) + (b >> 3);
    part = whole ? -1 : id / p.rest;
    return whole ? id : p.full + (id - part * p.rest);
}

// The results' way through LDS (the end of the kernel): floats between the
// rows of a wave's area (the vectors of 16 lanes in different banks), groups of
// 32 rows it holds, and the bytes a workgroup needs for that or the ring.
template <int NF> constexpr int row_stride() { return 32 * NF + 4; }
template <int MF> constexpr int turn_groups() { return MF < 2 ? MF : 2; }
template <int WM, int WN, int MF, int NF, int KG, int L>
constexpr int tile_lds() {
    const int ring = KG * (2 * L + 1) * WM * MF * 32 * kStage;
    const int turn = KG * WM * WN * turn_groups<MF>() * 32 * row_stride<NF>() * 4;
    return ring > turn ? ring : turn;
}

// The order of a half stage's instructions: the loads (LOADS) and LDS reads
// (READS) spread evenly between the matrix instructions (MMAS).  Where two
// waves share a SIMD over long runs of short instructions, as in the 256 x 256
// tile of two-byte types, the compiler's own order is the better one (bf16 4096 x
// 8192 x 4096 221 us spread, 217 not; 1024 x 1024 x 4096 on 64 x 64 tiles 15.5
// spread, 16.3 not; fp32 4096 x 4096 x 4096 945 and 949).
template <int LOADS, int READS, int MMAS, bool LEAVE>
__device__ __forceinline__ void spread() {
    if constexpr (LEAVE) return;
    constexpr int G = LOADS < MMAS ? LOADS : MMAS;  // groups
    constexpr int RG = (READS + G - 1) / G, MG = MMAS / G;
#pragma unroll
    for (int i = 0; i < G; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x010, (LOADS + G - 1) / G, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, RG, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, MG, 0);
    }
}

template <int DT, int WM, int WN, int MF, int NF, int KG, int L, bool AL>
__global__ __launch_bounds__(KG* WM* WN * 64) void linear_tile_kernel(LinearParams p) {
    constexpr int ES = elem_size<DT>();
    constexpr int NW = WM * WN;
    constexpr int B = WM * MF * 32;
    static_assert(B == WN * NF * 32, "square tiles: every item has the same size");
    constexpr int LPI = B / 8 / NW;  // 8-row loads of a wave an item
    static_assert(LPI * NW * 8 == B, "whole loads");
    constexpr int ITEM = B * kStage, RING = (2 * L + 1) * ITEM;
    constexpr int READS = 2 * (MF + NF), MMAS = MF * NF * (DT == DT_E4M3 ? 1 : DT == DT_F32 ? 8 : DT == DT_E4M3_WIDE ? 4 : 2);
    extern __shared__ __align__(16) char all_lds[];

    const int lane = threadIdx.x & 63;
    const int wave_of_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = KG > 1 ? wave_of_all / NW : 0, wave = wave_of_all - kg * NW;
    char* const lds = all_lds + kg * RING;
    const int wm = wave % WM, wn = wave / WM;
    int tm, tn, part;
    const unsigned tile = work_of(p, part);
    if (B == 256) part = -1;  // never split
    tile_at(p, tile, tm, tn);
    const int m0 = tm * B, n0 = tn * B;
    // this workgroup's stages, of which group kg takes every KG-th
    const int st0 = part < 0 ? 0 : part * p.stages_per_split;
    const int all = (p.kbytes + kStage - 1) / kStage;
    const int end = part < 0 || all - st0 < p.stages_per_split ? all : st0 + p.stages_per_split;
    const int stages = (end - st0 + KG - 1) / KG;

    // ---- loads: a wave's load j of an item fills rows (wave + NW j) * 8 .. + 7,
    // lane l place l % 8 of row l / 8.  Rows past the end are the last row again
    // (their results are not stored).  A lane's place is the same in all its
    // loads (its rows differ by multiples of 32), so the chunk it loads is too:
    // byte cx (cw) of the stage.
    static_assert(NW % 4 == 0, "rows of one lane's loads differ by multiples of 32");
    const char* const xb = p.x + m0 * p.ldx + (long long)(st0 + kg) * kStage;
    const char* const wb = p.w + n0 * p.ldw + (long long)(st0 + kg) * kStage;
    const int cx = ((lane & 7) ^ rot_x(wave * 8 + (lane >> 3))) << 4;
    const int cw = ((lane & 7) ^ rot_w(wave * 8 + (lane >> 3))) << 4;
    unsigned xo[LPI], wo[LPI];
#pragma unroll
    for (int j = 0; j < LPI; ++j) {
        const int row = (wave + NW * j) * 8 + (lane >> 3);
        xo[j] = (unsigned)((m0 + row < p.M ? row : p.M - 1 - m0) * (int)p.ldx) + (AL ? cx : 0);
        wo[j] = (unsigned)((n0 + row < p.N ? row : p.N - 1 - n0) * (int)p.ldw) + (AL ? cw : 0);
    }
    // bytes of the rows from stage st on (none past the last: those loads bring
    // zeros that nothing reads, so that every stage waits for the same count)
    auto left_at = [&](int st) {
        const int at = st0 + kg + st * KG;
        return at < end ? p.kbytes - at * kStage : 0;
    };
    // aligned rows go to LDS directly
    auto load_item = [&](const char* base, const unsigned (&o)[LPI], int c, int st, int slot) {
        const unsigned past = c >= left_at(st) ? kBufOut : 0;
        char* to = lds + slot + wave * 1024;
#pragma unroll
        for (int j = 0; j < LPI; ++j) load_to_lds(base + (long long)st * (KG * kStage), o[j] | past, to + j * NW * 1024);
    };
    // others pass through registers, two stages of them in flight
    struct Held {
        uint4v v[LPI];
    };
    Held hx[AL ? 1 : 2], hw[AL ? 1 : 2];
    auto hold_item = [&](Held& h, const char* base, const unsigned (&o)[LPI], int c, int st) {
        const int left = left_at(st);
        const char* from = base + (long long)st * (KG * kStage);
        if (left >= kStage) {
#pragma unroll
            for (int j = 0; j < LPI; ++j) __builtin_memcpy(&h.v[j], from + o[j] + c, 16);
        } else {
#pragma unroll
            for (int j = 0; j < LPI; ++j) h.v[j] = load_chunk<ES>(from + o[j], c, left);
        }
    };
    auto put_item = [&](const Held& h, int slot) {
        char* to = lds + slot + wave * 1024 + lane * 16;
#pragma unroll
        for (int j = 0; j < LPI; ++j) *reinterpret_cast<uint4v*>(to + j * NW * 1024) = h.v[j];
    };

    // ---- operand reads: half s of a stage, chunks 4 s + h and 4 s + 2 + h
    const int lj = lane & 31, lh = lane >> 5;
    const int wrow = 16 * ((lj >> 2) & 1) + 4 * (lj >> 3) + (lj & 3);
    const int xa = (wm * MF * 32 + lj) * kStage + ((lh ^ rot_x(lj)) << 4);
    const int wa = (wn * NF * 32 + wrow) * kStage + ((lh ^ rot_w(wrow)) << 4);
    struct Half {
        uint4v x[MF][2], w[NF][2];
    };
    auto read_half = [&](Half& h, int xslot, int wslot, int s) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int flip = s * 64 + c * 32;
#pragma unroll
            for (int f = 0; f < NF; ++f)
                h.w[f][c] = *reinterpret_cast<const uint4v*>(lds + wslot + (wa ^ flip) + f * 32 * kStage);
#pragma unroll
            for (int f = 0; f < MF; ++f)
                h.x[f][c] = *reinterpret_cast<const uint4v*>(lds + xslot + (xa ^ flip) + f * 32 * kStage);
        }
    };
    floatx16 acc[MF][NF] = {};
    auto products = [&](const Half& h) {
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j)
                acc[i][j] = mma32<DT>(h.w[j][0], h.w[j][1], h.x[i][0], h.x[i][1], acc[i][j]);
    };
    // all but the last PENDING items this wave started have arrived, everywhere
    auto arrive = [&](auto pending) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(pending)::value * LPI) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    auto next = [](int slot) { return slot + ITEM < RING ? slot + ITEM : 0; };

    Half h0, h1;
    int xs = 0, ws = ITEM;  // the slots of stage s
    if constexpr (AL) {
#pragma unroll
        for (int st = 0; st < L; ++st) {
            load_item(xb, xo, cx, st, 2 * st * ITEM);
            load_item(wb, wo, cw, st, (2 * st + 1) * ITEM);
        }
        arrive(std::integral_constant<int, 2 * L - 2>{});
        read_half(h0, xs, ws, 0);
        int free = 2 * L * ITEM;  // the slot to fill next: the one ahead of x's of stage s
        for (int s = 0; s < stages - 1; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            load_item(xb, xo, cx, s + L, free);
            read_half(h1, xs, ws, 1);
            products(h0);
            spread<LPI, READS, MMAS, (B == 256 && DT != DT_F32)>();
            __builtin_amdgcn_sched_barrier(0);
            arrive(std::integral_constant<int, 2 * L - 3>{});
            free = xs;
            xs = next(ws);
            ws = next(xs);
            load_item(wb, wo, cw, s + L, free);
            free = next(free);
            read_half(h0, xs, ws, 0);
            products(h1);
            spread<LPI, READS, MMAS, (B == 256 && DT != DT_F32)>();
            __builtin_amdgcn_sched_barrier(0);
        }
        // what is left on its way is not read
    } else {
        // an item is loaded two stages before it is put into its slot, half a
        // stage before the barrier that publishes it: two stages' slots at once
        static_assert(L >= 2, "slots of the stage that is read and of the next");
        hold_item(hx[0], xb, xo, cx, 0);
        hold_item(hw[0], wb, wo, cw, 0);
        hold_item(hx[1], xb, xo, cx, 1);
        hold_item(hw[1], wb, wo, cw, 1);
        put_item(hx[0], 0);
        put_item(hw[0], ITEM);
        hold_item(hx[0], xb, xo, cx, 2);
        hold_item(hw[0], wb, wo, cw, 2);
        arrive(std::integral_constant<int, 63 / LPI>{});
        read_half(h0, xs, ws, 0);
        // stage s: hx[(s + 1) % 2] holds stage s + 1
        int px = 2 * ITEM;
        auto stage = [&](int s, Held& x1, Held& w1) {
            put_item(x1, px);
            px = next(px);
            put_item(w1, px);
            px = next(px);
            hold_item(x1, xb, xo, cx, s + 3);
            read_half(h1, xs, ws, 1);
            products(h0);
            arrive(std::integral_constant<int, 63 / LPI>{});
            xs = next(ws);
            ws = next(xs);
            hold_item(w1, wb, wo, cw, s + 3);
            read_half(h0, xs, ws, 0);
            products(h1);
        };
        int s = 0;
        for (; s + 1 < stages - 1; s += 2) {
            stage(s, hx[1], hw[1]);
            stage(s + 1, hx[0], hw[0]);
        }
        if (s < stages - 1) stage(s, hx[1], hw[1]);
    }
    read_half(h1, xs, ws, 1);
    products(h0);
    products(h1);

    // ---- results.  Lane l holds, of tile (i, j), row l % 32 of x and the 16
    // rows of w from 16 (l / 32).  Each wave turns its 32 rows of tiles (i, .)
    // through LDS of its own, so that lanes hold 8 neighbours of a row and a
    // row's lanes are neighbours too: whole 128-byte lines of y, gate and
    // residual with NF = 2 and two-byte elements.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();  // the ring is free
    asm volatile("" ::: "memory");
    constexpr int RS = row_stride<NF>();
    constexpr int LPR = 32 * NF / 8;      // lanes a row
    constexpr int RPS = 64 / LPR;         // rows a step
    constexpr int GR = turn_groups<MF>();
    constexpr int SHARE = GR * 32 / KG;   // rows of the area that this wave finishes: each group of waves a share
    constexpr int STEPS = SHARE < 2 * RPS ? 1 : 2;  // steps whose side values are loaded ahead
    const int row_first = kg * SHARE;
    static_assert(SHARE % (RPS * STEPS) == 0, "whole steps");
    constexpr int AREA = GR * 32 * RS;
    static_assert(KG == 1 || GR == MF, "groups join their sums in one turn");
    float* const area = reinterpret_cast<float*>(all_lds) + wave * AREA;
    const int lrow = lane / LPR, lcol = (lane % LPR) * 8;
    const int mw = m0 + wm * MF * 32, nw = n0 + wn * NF * 32;  // the wave's first row and column
    const int n = nw + lcol;
    auto turn = [&](int i0) {
#pragma unroll
        for (int i = 0; i < GR; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j)
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    *reinterpret_cast<floatx4*>(area + kg * NW * AREA + (i * 32 + lj) * RS + j * 32 + lh * 16 + r) =
                        floatx4{acc[i0 + i][j][r], acc[i0 + i][j][r + 1], acc[i0 + i][j][r + 2], acc[i0 + i][j][r + 3]};
        if constexpr (KG > 1)
            __syncthreads();
        else
            asm volatile("" ::: "memory");  // a wave's LDS operations complete in order: no barrier
    };
    auto turned = [&](int row, float (&v)[8]) {  // row: of the area, of which lanes read RPS from here
        __builtin_memcpy(v, __builtin_assume_aligned(area + (row + lrow) * RS + lcol, 16), 32);
#pragma unroll
        for (int g = 1; g < KG; ++g) {
            float w[8];
            __builtin_memcpy(w, __builtin_assume_aligned(area + g * NW * AREA + (row + lrow) * RS + lcol, 16), 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += w[i];
        }
    };
    // A tile inside y, of two-byte elements: 16 bytes a lane of y, gate and
    // residual, whose rows a step are RPS, at a uniform address and a 32-bit
    // offset of the lane; gate, residual and row scales of the next STEPS steps
    // are on their way while these are finished.  Instructions are few and
    // straight, one copy for each activation and type, because a workgroup runs
    // them cold: on a 4096 x 8192 x 4096 product with a check per element and a
    // choice of activation per step they took 10 us a tile of 256 x 256, a
    // sixth of the whole.
    auto inside = [&](auto act, auto type) {
        constexpr int ACT = decltype(act)::value, ODT = decltype(type)::value;
        constexpr int GROUP = RPS * STEPS;  // rows
        const unsigned yo = (unsigned)lrow * (unsigned)p.ldy + lcol * 2;
        const unsigned go = (unsigned)lrow * (unsigned)p.ldg + lcol * 2;
        const unsigned ro = (unsigned)lrow * (unsigned)p.ldr + lcol * 2;
        char* const yw = p.y + mw * p.ldy + nw * 2LL;
        const char* const gw = p.gate ? p.gate + mw * p.ldg + nw * 2LL : nullptr;
        const char* const rw = p.res ? p.res + mw * p.ldr + nw * 2LL : nullptr;
        float cs[8], cb[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 1.0f, cb[i] = 0.0f;
        if (DT == DT_E4M3) __builtin_memcpy(cs, p.ws + n, 32);
        if (p.bias) __builtin_memcpy(cb, p.bias + n, 32);
        struct Ahead {
            uint4v g[STEPS], r[STEPS];
            float xs[STEPS];
        };
        auto fetch = [&](Ahead& a, int row0) {
#pragma unroll
            for (int t = 0; t < STEPS; ++t) a.g[t] = a.r[t] = uint4v{0, 0, 0, 0}, a.xs[t] = 1.0f;
            if (gw) {
#pragma unroll
                for (int t = 0; t < STEPS; ++t)
                    __builtin_memcpy(&a.g[t], gw + (row0 + t * RPS) * p.ldg + go, 16);
            }
            if (rw) {
#pragma unroll
                for (int t = 0; t < STEPS; ++t)
                    __builtin_memcpy(&a.r[t], rw + (row0 + t * RPS) * p.ldr + ro, 16);
            }
            if (DT == DT_E4M3) {
#pragma unroll
                for (int t = 0; t < STEPS; ++t) a.xs[t] = p.xs[mw + row0 + t * RPS + lrow];
            }
        };
        auto halves = [&](uint4v u, float (&f)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint16_t h = (uint16_t)(u[i / 2] >> (16 * (i & 1)));
                f[i] = ODT == DT_BF16 ? Elem<DT_BF16>::to_f32(h) : (float)__builtin_bit_cast(_Float16, h);
            }
        };
        Ahead now;
        fetch(now, row_first);
#pragma unroll
        for (int i0 = 0; i0 < MF; i0 += GR) {
            turn(i0);
#pragma unroll 1
            for (int row0 = row_first; row0 < row_first + SHARE; row0 += GROUP) {
                Ahead then;
                const int after = i0 * 32 + row0 + GROUP;
                fetch(then, after < (KG > 1 ? row_first + SHARE : MF * 32) ? after : row_first);  // at the end: again the first
#pragma unroll
                for (int t = 0; t < STEPS; ++t) {
                    float v[8], f[8];
                    turned(row0 + t * RPS, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = activated<ACT, false>(DT == DT_E4M3 ? fmaf(v[i] * now.xs[t], cs[i], cb[i]) : v[i] + cb[i]);
                    if (gw) {
                        halves(now.g[t], f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] *= f[i];
                    }
                    if (rw) {
                        halves(now.r[t], f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] += f[i];
                    }
                    store_out_vec<8>(yw + (i0 * 32 + row0 + t * RPS) * p.ldy + yo, ODT, v);
                }
                now = then;
            }
        }
    };
    if (part < 0 && p.near && m0 + B <= p.M && n0 + B <= p.N) {
        // fp32 operands with two-byte results are left to the general form
        if constexpr (DT == DT_BF16 || DT == DT_E4M3)
            if (p.out_dt == DT_BF16)
                return with_activation(p.act, [&](auto act) { inside(act, std::integral_constant<int, DT_BF16>{}); });
        if constexpr (DT == DT_F16 || DT == DT_E4M3)
            if (p.out_dt == DT_F16)
                return with_activation(p.act, [&](auto act) { inside(act, std::integral_constant<int, DT_F16>{}); });
    }
    float cs[8], cb[8];
    if (part < 0) column_values<8>(p, n, cs, cb);
    float* const parts = part < 0 ? nullptr : p.part + ((long long)part * p.rest + (tile - p.full)) * B * B;
#pragma unroll
    for (int i0 = 0; i0 < MF; i0 += GR) {
        turn(i0);
#pragma unroll 1
        for (int row = row_first; row < row_first + SHARE; row += RPS * STEPS) {
            const int mt = (wm * MF + i0) * 32 + row + lrow;  // row of the tile
            float v[8];
            if (part >= 0) {
#pragma unroll
                for (int t = 0; t < STEPS; ++t) {
                    turned(row + t * RPS, v);
                    __builtin_memcpy(__builtin_assume_aligned(parts + (mt + t * RPS) * B + wn * NF * 32 + lcol, 16), v, 32);
                }
                continue;
            }
            Side<8> side[STEPS];
#pragma unroll
            for (int t = 0; t < STEPS; ++t) side[t].load(p, m0 + mt + t * RPS, n);
#pragma unroll
            for (int t = 0; t < STEPS; ++t) {
                turned(row + t * RPS, v);
                finish<8>(p, m0 + mt + t * RPS, n, v, cs, cb, side[t]);
            }
        }
    }
}

// Join the parts of the split tiles (B x B floats each, [S][rest]), part after
// part, and finish: 4 neighbours a thread.
template <int B>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearParams p) {
    const unsigned id = blockIdx.x * 256 + threadIdx.x;
    constexpr unsigned PT = B * B / 4;  // threads a tile, a multiple of the workgroup
    const unsigned t = id / PT, in = id - t * PT;
    int tm, tn;
    tile_at(p, p.full + t, tm, tn);
    const int row = in / (B / 4), col = (in - row * (B / 4)) * 4;
    const int m = tm * B + row, n = tn * B + col;
    if (m >= p.M || n >= p.N) return;
    Side<4> side;
    side.load(p, m, n);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s[4], b[4];
    column_values<4>(p, n, s, b);
    const float* part = p.part + (long long)t * B * B + row * B + col;
#pragma unroll 4
    for (int k = 0; k < p.S; ++k) {
        float f[4];
        __builtin_memcpy(f, __builtin_assume_aligned(part + (long long)k * p.rest * B * B, 16), 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += f[i];
    }
    finish<4>(p, m, n, v, s, b, side);
}

// The rows of x and w, one after the other, at a pitch of whole stages, zeros
// behind their ends.  A workgroup takes every gridDim.x-th row.
__global__ __launch_bounds__(256) void linear_pack_kernel(LinearParams p, char* to, int pitch) {
    for (int r = blockIdx.x; r < p.M + p.N; r += gridDim.x) {
        const char* from = r < p.M ? p.x + r * p.ldx : p.w + (r - p.M) * p.ldw;
        const unsigned in = (unsigned)(uintptr_t)from & 3;
        char* row = to + (long long)r * pitch;
        for (int k = threadIdx.x * 16; k < pitch; k += 256 * 16) {
            const int left = p.kbytes - k;
            // whole dwords, all holding bytes of the row
            unsigned d[5] = {0, 0, 0, 0, 0};
            if (left >= 16) {
                __builtin_memcpy(d, __builtin_assume_aligned(from + k - in, 4), 16);
                if (in) __builtin_memcpy(d + 4, __builtin_assume_aligned(from + k - in + 16, 4), 4);
            } else {
#pragma unroll
                for (int i = 0; i < 5; ++i)
                    if (4 * i - (int)in < left) __builtin_memcpy(d + i, __builtin_assume_aligned(from + k - in + 4 * i, 4), 4);
            }
            uint4v v;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __builtin_amdgcn_alignbit(d[i + 1], d[i], in * 8);
                const int bytes = left - 4 * i;  // of the row in this dword
                if (bytes < 4) v[i] = bytes <= 0 ? 0 : v[i] & ((1u << (8 * bytes)) - 1);
            }
            *reinterpret_cast<uint4v*>(row + k) = v;
        }
    }
}

template <int DT, int WM, int WN, int MF, int NF, int KG, int L, bool AL>
hipError_t launch_tile(LinearParams p, const LinearPlan& plan, hipStream_t stream) {
    constexpr int B = WM * MF * 32;
    constexpr int LDS = tile_lds<WM, WN, MF, NF, KG, L>();
    static_assert(LDS <= 160 * 1024, "one workgroup a CU at least");
    p.tiles_m = (p.M + B - 1) / B;
    p.tiles_n = (p.N + B - 1) / B;
    p.full = plan.full;
    p.rest = p.tiles_m * p.tiles_n - plan.full;
    p.S = plan.S;
    p.stages_per_split = linear_part_stages(p.kbytes, p.S);
    auto* kernel = linear_tile_kernel<DT, WM, WN, MF, NF, KG, L, AL>;
    static std::atomic<unsigned long long> lds_set{0};  // a bit per device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(lds_set.load(std::memory_order_relaxed) & bit)) {
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
        if (e != hipSuccess) {
            (void)hipGetLastError();
            return e;
        }
        lds_set.fetch_or(bit, std::memory_order_relaxed);
    }
    (void)hipGetLastError();
    kernel<<<dim3((unsigned)(p.full + p.rest * p.S)), dim3(KG * WM * WN * 64), LDS, stream>>>(p);
    e = hipGetLastError();
    if constexpr (B < 256) {  // the largest tiles are never split
        if (e != hipSuccess || p.rest == 0) return e;
        linear_join_kernel<B><<<dim3((unsigned)(p.rest * (B * B / 1024))), dim3(256), 0, stream>>>(p);
        e = hipGetLastError();
    }
    return e;
}

template <int DT>
hipError_t launch_dt(const LinearPlan& plan, const LinearParams& p, bool aligned, hipStream_t stream) {
    (void)hipGetLastError();
    const dim3 rows_grid((unsigned)((p.N + 15) / 16)), rows_block(kRowWaves * 64);
    constexpr int ROW_DT = DT == DT_E4M3 ? DT_E4M3_WIDE : DT;
    const bool at_dwords = ((uintptr_t)p.x | (uintptr_t)p.w | (uintptr_t)p.ldx | (uintptr_t)p.ldw) % 4 == 0;
    switch (plan.form) {
        case LIN_ROW16:
            if (at_dwords)
                linear_rows_kernel<ROW_DT, 1, true><<<rows_grid, rows_block, 0, stream>>>(p);
            else
                linear_rows_kernel<ROW_DT, 1, false><<<rows_grid, rows_block, 0, stream>>>(p);
            return hipGetLastError();
        case LIN_ROW32:
            if (at_dwords)
                linear_rows_kernel<ROW_DT, 2, true><<<rows_grid, rows_block, 0, stream>>>(p);
            else
                linear_rows_kernel<ROW_DT, 2, false><<<rows_grid, rows_block, 0, stream>>>(p);
            return hipGetLastError();
        case LIN_T64:
            if (!aligned) return launch_tile<DT, 2, 2, 1, 1, 2, 2, false>(p, plan, stream);
            // a workgroup with a CU to itself takes a deeper ring (1024 x 1024 x 4096
            // bf16 20.5 -> 15.7 us); two share the CU's LDS (512 x 4096 x 4096 28.9 us,
            // 31.4 with the deeper one, which leaves room for one)
            if (linear_workgroups(plan, p.M, p.N) <= 256) return launch_tile<DT, 2, 2, 1, 1, 2, 3, true>(p, plan, stream);
            return launch_tile<DT, 2, 2, 1, 1, 2, 2, true>(p, plan, stream);
        case LIN_T128K:
            return aligned ? launch_tile<DT, 2, 2, 2, 2, 2, 2, true>(p, plan, stream)
                           : launch_tile<DT, 2, 2, 2, 2, 2, 2, false>(p, plan, stream);
        case LIN_T128:
            // fp32 comes here only in the place of 256 x 256 tiles that are not aligned
            if constexpr (DT != DT_F32)
                if (aligned) return launch_tile<DT, 2, 2, 2, 2, 1, 2, true>(p, plan, stream);
            return launch_tile<DT, 2, 2, 2, 2, 1, 2, false>(p, plan, stream);
        default: return launch_tile<DT, 2, 4, 4, 2, 1, 2, true>(p, plan, stream);
    }
}

}  // namespace

hipError_t launch_linear(LinearPlan plan, LinearParams p, int dtype, bool aligned, hipStream_t stream) {
    if (plan.pack) {
        const int pitch = linear_pack_pitch(p.kbytes);
        char* const to = (char*)p.part + linear_workspace_bytes(plan, p.M, p.N, p.kbytes) - ((long long)p.M + p.N) * pitch;
        (void)hipGetLastError();
        linear_pack_kernel<<<dim3((unsigned)(p.M + p.N < 1 << 20 ? p.M + p.N : 1 << 20)), dim3(256), 0, stream>>>(p, to, pitch);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        p.x = to;
        p.w = to + (long long)p.M * pitch;
        p.ldx = p.ldw = p.kbytes = pitch;
        aligned = true;
    } else if (plan.form == LIN_T256 && !aligned) {
        // passing through registers leaves too few for the largest tile
        plan = {LIN_T128, ((p.M + 127) / 128) * ((p.N + 127) / 128), 1, 0};
    }
    switch (dtype) {
        case DT_F32: return launch_dt<DT_F32>(plan, p, aligned, stream);
        case DT_F16: return launch_dt<DT_F16>(plan, p, aligned, stream);
        case DT_BF16: return launch_dt<DT_BF16>(plan, p, aligned, stream);
        default:
            return p.out_dt == DT_F32 || p.M <= 32 ? launch_dt<DT_E4M3_WIDE>(plan, p, aligned, stream)
                                                   : launch_dt<DT_E4M3>(plan, p, aligned, stream);
    }
}

}  // namespace ct
