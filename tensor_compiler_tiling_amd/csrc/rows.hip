// Row operators: the root-mean-square norm with the residual's addition, and
// the 8-bit quantization of rows.
//
//   h = x + residual                      (fp32; stored rounded to x's type)
//   y = (h * gain) * r,  r = 1 / sqrt(mean h^2 + eps)      (norm; else y = h)
//   e4m3:  a = max(max |y|, 2^-100),  scale = a / 448,  q = rne(y / scale)
//
// The sum of squares and the maximum of |t|, t = h * gain, are reduced
// together, over one reading of the row, which stays in registers: max |y| is
// max |t| times r, rounded, since rounding keeps the order.
//
// y, scale and the quotient are fp32, each rounded to nearest, so the codes of
// a norm are those of its fp32 values.  The quotient has to be rounded as one:
// rows of two-byte types put many of them half way between two codes, and a
// product with a rounded 448 / a in its place moves all of a row's the same
// way (0.1% of a bf16 row's codes).  A product with 1 / scale and corrections by
// the remainder (Divisor, below) gives the quotient's bits in 3 or 5 operations
// (16384 x 8192 fp16 70 us, with a division an element 85).
//
// The maximum is taken over the bit patterns of |t| as unsigned integers:
// the order is that of the values, infinity above every finite value and NaN
// above infinity, so a NaN anywhere in a row reaches its scale.
//
// Bound by memory: about 10 operations an element.  A row is held by TPR
// threads, 16 bytes of the input's type a load and C loads a thread, all
// issued before the first is used.  Measured: rmsnorm of 8192 x 8192 bf16 with a
// residual 95.0 us (537 MB, 5.65 TB/s; a device copy moves 5.1 to 5.2), to e4m3 92
// (5.1 TB/s), 16384 x 8192 fp16 to e4m3 68.6 us (403 MB, 5.9 TB/s); one row of
// 4096 3.6 us on the device.
#include "ct_device.hpp"
#include "block_kernels.hpp"

namespace ct {

namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kFloor = 0x1p-100f;

enum { OUT_E4M3 = 3 };  // out_dt beyond DT_F32, DT_F16, DT_BF16

// n elements of type DT at p (n < V: the row's end) as floats, zeros beyond.
// A whole vector is one 16-byte load at whatever alignment the row has: gfx950
// takes global accesses at any byte address.
template <int DT> struct Vec;
template <> struct Vec<DT_F32> { static constexpr int V = 4; };
template <> struct Vec<DT_F16> { static constexpr int V = 8; };
template <> struct Vec<DT_BF16> { static constexpr int V = 8; };

template <int DT, int V>
__device__ __forceinline__ void load_vec(const char* p, int n, float (&f)[V]) {
    using T = typename Elem<DT>::T;
    T v[V];
    if (n >= V) {
        __builtin_memcpy(v, p, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = T(0);
            if (i < n) v[i] = reinterpret_cast<const T*>(p)[i];
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = Elem<DT>::to_f32(v[i]);
}

__device__ __forceinline__ uint16_t to_bf16(float f) {
    // round to nearest even; a NaN stays one
    return __builtin_bit_cast(uint16_t, (__bf16)f);
}

template <int V, typename T>
__device__ __forceinline__ void store_elems(char* p, int n, const T (&v)[V]) {
    if (n >= V) {
        __builtin_memcpy(p, v, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) reinterpret_cast<T*>(p)[i] = v[i];
    }
}

template <int V>
__device__ __forceinline__ void store_vec(char* p, int n, int dt, const float (&f)[V]) {
    if (dt == DT_F32) {
        store_elems<V, float>(p, n, f);
    } else {
        uint16_t v[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = dt == DT_BF16 ? to_bf16(f[i]) : __builtin_bit_cast(uint16_t, (_Float16)f[i]);
        store_elems<V, uint16_t>(p, n, v);
    }
}

// V values to e4m3 (round to nearest even).
template <int V>
__device__ __forceinline__ void store_e4m3(char* p, int n, const float (&f)[V]) {
    uint8_t b[V];
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        int u = __builtin_amdgcn_cvt_pk_fp8_f32(f[i], f[i + 1], 0, false);
        u = __builtin_amdgcn_cvt_pk_fp8_f32(f[i + 2], f[i + 3], u, true);
        __builtin_memcpy(b + i, &u, 4);
    }
    store_elems<V, uint8_t>(p, n, b);
}

__device__ __forceinline__ int elem_bytes(int dt) { return dt == DT_F32 ? 4 : dt == OUT_E4M3 ? 1 : 2; }

// Quotients by a row's scale s, rounded to nearest.  With inv = 1 / s rounded to
// nearest, v * inv is off by at most 1.5 steps; adding the remainder times inv
// leaves the quotient's neighbour on either side or the quotient itself, and
// from there a second such step rounds it correctly (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  The
// remainders are exact while the products of their last places are normal: for
// s between 2^-80 and 2^100 they are wherever the quotient is 2^-11 or more,
// and below that its code is a zero whatever its last bits.  Rows outside
// (zeros and nearly so, infinities, NaN) divide.
// A row of a two-byte type that is brought to 8 bits as it is needs one step
// (STEPS): it gives the quotient for all pairs of 11-bit significands of v and
// of the row's maximum, and exponents only scale them (16384 x 8192 fp16 71.4
// us with two steps, 70.2 with one).
template <int STEPS>
struct Divisor {
    float s, inv;
    bool usual;
    __device__ __forceinline__ explicit Divisor(float scale)
        : s(scale), inv(1.0f / scale), usual(scale >= 0x1p-80f && scale <= 0x1p100f) {}
    // The remainder is taken negative so that a zero keeps its sign.
    __device__ __forceinline__ float near(float v) const {
        float q = v * inv;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) q = fmaf(-fmaf(q, s, -v), inv, q);
        return q;
    }
    __device__ __forceinline__ float any(float v) const { return v / s; }
};

template <int DT, bool NORM>
constexpr int quotient_steps() {
    return !NORM && DT != DT_F32 ? 1 : 2;
}

// What a row's statistics give: y = t * r, and the scale of 8-bit output.
struct RowFactors {
    float r, scale;
};

// ss: the sum of squares, tbits: the bits of max |t|.
template <bool NORM>
__device__ __forceinline__ RowFactors row_factors(float ss, uint32_t tbits, int D, int out_dt, float eps, float* scale) {
    const float r = NORM ? 1.0f / sqrtf(ss / (float)D + eps) : 1.0f;
    if (out_dt != OUT_E4M3) return {r, 1.0f};
    const float a0 = r * __uint_as_float(tbits);
    const float a = a0 < kFloor ? kFloor : a0;  // NaN stays
    const float s = a / kE4m3Max;
    if (scale) *scale = s;
    return {r, s};
}

// Reductions over the TPR threads of a row (whole waves): the sum of squares
// and the maximum, every thread getting both.
template <int TPR>
__device__ __forceinline__ void reduce_row(float& ss, uint32_t& tb) {
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        ss += __shfl_xor(ss, o);
        const uint32_t u = __shfl_xor(tb, o);
        tb = u > tb ? u : tb;
    }
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        __shared__ float s_ss[W];
        __shared__ uint32_t s_tb[W];
        if ((threadIdx.x & 63) == 0) {
            s_ss[threadIdx.x >> 6] = ss;
            s_tb[threadIdx.x >> 6] = tb;
        }
        __syncthreads();
        ss = 0.0f;
        tb = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            ss += s_ss[w];
            tb = s_tb[w] > tb ? s_tb[w] : tb;
        }
    }
}

// One row by TPR threads, in registers: D <= TPR * C * V.
template <int DT, int TPR, int C, bool NORM>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void rows_kernel(RowsParams p, int M) {
    constexpr int V = Vec<DT>::V;
    constexpr int RPB = TPR == 64 ? 4 : 1;  // rows a workgroup
    const int lt = RPB > 1 ? threadIdx.x % TPR : threadIdx.x;
    const long long row = (long long)blockIdx.x * RPB + (RPB > 1 ? threadIdx.x / TPR : 0);
    if (row >= M) return;  // whole waves, and no barrier where a workgroup has several rows
    const char* x = p.x + row * p.ldx;
    constexpr int ES = sizeof(typename Elem<DT>::T);

    float h[C][V];
    uint32_t tb = 0;
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (c * TPR + lt) * V;
        load_vec<DT, V>(x + (long long)e * ES, p.D - e, h[c]);
    }
    if (p.res) {
        const char* res = p.res + row * p.ldres;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * TPR + lt) * V;
            float f[V];
            load_vec<DT, V>(res + (long long)e * ES, p.D - e, f);
#pragma unroll
            for (int i = 0; i < V; ++i) h[c][i] += f[i];
        }
    }
    if (p.h) {
        char* ho = p.h + row * p.ldh;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * TPR + lt) * V;
            store_vec<V>(ho + (long long)e * ES, p.D - e, DT, h[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (c * TPR + lt) * V;
        if constexpr (NORM) {
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(h[c][i], h[c][i], ss);
            if (p.gain) {
                float g[V];
                load_vec<DT_F32, V>(reinterpret_cast<const char*>(p.gain + e), p.D - e, g);
#pragma unroll
                for (int i = 0; i < V; ++i) h[c][i] *= g[i];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t u = __float_as_uint(h[c][i]) & 0x7fffffffu;
            tb = u > tb ? u : tb;
        }
    }
    reduce_row<TPR>(ss, tb);
    const RowFactors f = row_factors<NORM>(ss, tb, p.D, p.out_dt, p.eps, lt == 0 && p.scale ? p.scale + row : nullptr);
    char* y = p.y + row * p.ldy;
    auto put = [&](auto store) {  // store(address, elements, values)
        const int oes = elem_bytes(p.out_dt);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * TPR + lt) * V;
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = NORM ? h[c][i] * f.r : h[c][i];
            store(y + (long long)e * oes, p.D - e, o);
        }
    };
    if (p.out_dt == OUT_E4M3) {
        const Divisor<quotient_steps<DT, NORM>()> d(f.scale);
        if (d.usual)
            put([&](char* at, int n, float (&o)[V]) {
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = d.near(o[i]);
                store_e4m3<V>(at, n, o);
            });
        else
            put([&](char* at, int n, float (&o)[V]) {
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = d.any(o[i]);
                store_e4m3<V>(at, n, o);
            });
    } else {
        put([&](char* at, int n, const float (&o)[V]) { store_vec<V>(at, n, p.out_dt, o); });
    }
}

// A row of any length, read twice: statistics, then outputs.  h is written in
// the second reading, after the elements it may replace.
template <int DT, bool NORM>
__global__ __launch_bounds__(1024) void rows_long_kernel(RowsParams p) {
    constexpr int V = Vec<DT>::V, TPR = 1024;
    constexpr int ES = sizeof(typename Elem<DT>::T);
    const long long row = blockIdx.x;
    const char* x = p.x + row * p.ldx;
    const char* res = p.res ? p.res + row * p.ldres : nullptr;
    float ss = 0.0f;
    uint32_t tb = 0;
    auto load_h = [&](long long e, float (&h)[V]) {
        const int n = (int)((long long)p.D - e < V ? (long long)p.D - e : V);
        load_vec<DT, V>(x + e * ES, n, h);
        if (res) {
            float f[V];
            load_vec<DT, V>(res + e * ES, n, f);
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] += f[i];
        }
    };
    auto times_gain = [&](long long e, float (&h)[V]) {
        if (!NORM || !p.gain) return;
        const int n = (int)((long long)p.D - e < V ? (long long)p.D - e : V);
        float g[V];
        load_vec<DT_F32, V>(reinterpret_cast<const char*>(p.gain + e), n, g);
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] *= g[i];
    };
    for (long long e = (long long)threadIdx.x * V; e < p.D; e += TPR * V) {
        float h[V];
        load_h(e, h);
        if constexpr (NORM) {
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(h[i], h[i], ss);
        }
        times_gain(e, h);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t u = __float_as_uint(h[i]) & 0x7fffffffu;
            tb = u > tb ? u : tb;
        }
    }
    reduce_row<TPR>(ss, tb);
    const RowFactors f =
        row_factors<NORM>(ss, tb, p.D, p.out_dt, p.eps, threadIdx.x == 0 && p.scale ? p.scale + row : nullptr);
    char* y = p.y + row * p.ldy;
    const int oes = elem_bytes(p.out_dt);
    const Divisor<quotient_steps<DT, NORM>()> d(f.scale);
    for (long long e = (long long)threadIdx.x * V; e < p.D; e += TPR * V) {
        const int n = (int)((long long)p.D - e < V ? (long long)p.D - e : V);
        float h[V], o[V];
        load_h(e, h);
        if (p.h) store_vec<V>(p.h + row * p.ldh + e * ES, n, DT, h);
        times_gain(e, h);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = NORM ? h[i] * f.r : h[i];
        if (p.out_dt == OUT_E4M3) {
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = d.usual ? d.near(o[i]) : d.any(o[i]);
            store_e4m3<V>(y + e * oes, n, o);
        } else {
            store_vec<V>(y + e * oes, n, p.out_dt, o);
        }
    }
}

template <int DT, int TPR, int C>
hipError_t launch_one(const RowsParams& p, int M, bool norm, hipStream_t stream) {
    constexpr int RPB = TPR == 64 ? 4 : 1;
    const dim3 grid((unsigned)(((long long)M + RPB - 1) / RPB)), block(TPR * RPB);
    if (norm)
        rows_kernel<DT, TPR, C, true><<<grid, block, 0, stream>>>(p, M);
    else
        rows_kernel<DT, TPR, C, false><<<grid, block, 0, stream>>>(p, M);
    return hipGetLastError();
}

// Two 16-byte loads a thread are in flight where its count allows: with a
// residual one of each operand, if that leaves at most a quarter of the
// threads idle, else two (8192 rows of 4096 bf16 with a residual: 512 threads x 1
// load 46.7 us, 256 x 2 51.3; 16384 without: 44.2 and 37.5; 32768 of 1024 with a
// residual on half-idle 256 x 1 61.8, 128 x 2 50).  The longest rows take 1024
// threads with two or four loads (2048 rows of 16384 bf16 51.2 us, 52.8 on 512 x 4).
template <int DT, int TPR>
bool fits(int D) {
    return D <= TPR * Vec<DT>::V;
}

template <int DT, int TPR>
hipError_t launch_fitted(const RowsParams& p, int M, bool norm, hipStream_t stream) {
    if (p.res && 4LL * p.D >= 3LL * TPR * Vec<DT>::V) return launch_one<DT, TPR, 1>(p, M, norm, stream);
    return launch_one<DT, TPR / 2, 2>(p, M, norm, stream);
}

template <int DT>
hipError_t launch_dt(const RowsParams& p, int M, bool norm, hipStream_t stream) {
    constexpr int V = Vec<DT>::V;
    const int D = p.D;
    if (fits<DT, 64>(D)) return launch_one<DT, 64, 1>(p, M, norm, stream);
    if (fits<DT, 128>(D)) return launch_fitted<DT, 128>(p, M, norm, stream);
    if (fits<DT, 256>(D)) return launch_fitted<DT, 256>(p, M, norm, stream);
    if (fits<DT, 512>(D)) return launch_fitted<DT, 512>(p, M, norm, stream);
    if (fits<DT, 1024>(D)) return launch_fitted<DT, 1024>(p, M, norm, stream);
    if (D <= 1024 * V * 2) return launch_one<DT, 1024, 2>(p, M, norm, stream);
    if (D <= 1024 * V * 4) return launch_one<DT, 1024, 4>(p, M, norm, stream);
    if (norm)
        rows_long_kernel<DT, true><<<dim3((unsigned)M), dim3(1024), 0, stream>>>(p);
    else
        rows_long_kernel<DT, false><<<dim3((unsigned)M), dim3(1024), 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rows(const RowsParams& q, int M, int dtype, bool norm, hipStream_t stream) {
    (void)hipGetLastError();
    // a grid holds fewer than 2^32 threads: at most 2^21 rows of up to 1024
    constexpr int MOST = 1 << 21;
    RowsParams p = q;
    for (int m = 0; m < M; m += MOST) {
        const int rows = M - m < MOST ? M - m : MOST;
        const hipError_t e = dtype == DT_F32   ? launch_dt<DT_F32>(p, rows, norm, stream)
                             : dtype == DT_F16 ? launch_dt<DT_F16>(p, rows, norm, stream)
                                               : launch_dt<DT_BF16>(p, rows, norm, stream);
        if (e != hipSuccess || M - m <= MOST) return e;
        p.x += MOST * p.ldx;
        p.y += MOST * p.ldy;
        if (p.res) p.res += MOST * p.ldres;
        if (p.h) p.h += MOST * p.ldh;
        if (p.scale) p.scale += MOST;
    }
    return hipSuccess;
}

}  // namespace ct
