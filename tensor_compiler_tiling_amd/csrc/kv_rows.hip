// New tokens into the key-value cache, and tokens of it back out.
//
// A row is a token's key or value in one head.  In 16 bits it is stored as it
// is (rounded to the cache's type); in 8 bits as e4m3 codes with a scale:
//
//   a = max(largest finite |v|, 2^-100)
//   s = the least power of two with a <= 448 s,  code = rne_e4m3(v / s)
//
// A power of two costs no precision (e4m3 keeps its three fraction bits from
// 2^-6 up to 448, so a row loses at most one of its 17 binades to a scale that
// is not a / 448) and makes both directions exact: v / s is a shift of the
// exponent, and s * code a value of bf16 that one instruction gives
// (v_cvt_scalef32_pk_bf16_fp8), which is what attention multiplies.
// In bits: 448 = 0.875 * 2^9 = 1.75 * 2^8, so s has the exponent of a, less 8,
// and one more where a's fraction is above 0.75.
//
// Not finite values stay where they are: an infinity or NaN becomes the NaN
// code and leaves its row's scale to the others.
//
// Bound by memory.  LPR lanes hold a row, 8 elements each, and a group of them
// does a token's key and its value, so that two loads are in flight and the
// place is looked up once.  Measured: 32768 tokens of 8 heads of 128 from bf16 to
// e4m3 48 us (203 MB, 4.2 TB/s; 50 with a token's heads in a workgroup, whose
// scales' lines several then write), back 45 us (4.5 TB/s); 2 and 4 tokens a group
// of lanes 50 and 58 us; a step of 48 tokens 3.6 us on the device.
#include "kv_device.hpp"

namespace ct {

namespace {

enum { DT_E4M3 = 3 };
constexpr int kThreads = 256;
constexpr int kV = 8;  // elements a lane

template <int DT>
__device__ __forceinline__ void load8(const char* p, float (&f)[kV]) {
    using T = typename Elem<DT>::T;
    T v[kV];
    __builtin_memcpy(v, p, sizeof(v));  // one or two 16-byte loads, at any alignment
#pragma unroll
    for (int i = 0; i < kV; ++i) f[i] = Elem<DT>::to_f32(v[i]);
}

template <int DT>
__device__ __forceinline__ void store8(char* p, const float (&f)[kV]) {
    if constexpr (DT == DT_F32) {
        __builtin_memcpy(p, f, sizeof(f));
    } else {
        uint16_t v[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = to_half(f[i], DT);
        __builtin_memcpy(p, v, sizeof(v));
    }
}

// The largest finite |v| of the lanes that hold a row, as bits: their order is
// that of the values, and what is not finite is left out.
template <int LPR>
__device__ __forceinline__ uint32_t row_top(const float (&f)[kV]) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const uint32_t u = __float_as_uint(f[i]) & 0x7fffffffu;
        t = u < 0x7f800000u && u > t ? u : t;
    }
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) {
        const uint32_t u = __shfl_xor(t, o);
        t = u > t ? u : t;
    }
    return t;
}

// Exponent field of s; the inverse has 254 minus it.
__device__ __forceinline__ int scale_field(uint32_t top) {
    const uint32_t least = 27u << 23;  // 2^-100
    return (int)(((top > least ? top : least) + 0x1fffffu) >> 23) - 8;
}

// e4m3 of 8 values that are at most 448 or not finite.
__device__ __forceinline__ void store_codes(char* p, const float (&f)[kV], float inv) {
    uint32_t u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i] * inv, f[4 * i + 1] * inv, 0, false);
        u[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2] * inv, f[4 * i + 3] * inv, w, true);
    }
    __builtin_memcpy(p, u, 8);
}

__device__ __forceinline__ void load_codes(const char* p, float (&f)[kV], float scale) {
    uint32_t u[2];
    __builtin_memcpy(u, p, 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __builtin_amdgcn_cvt_f32_fp8(u[i], 0) * scale;
        f[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(u[i], 1) * scale;
        f[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(u[i], 2) * scale;
        f[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(u[i], 3) * scale;
    }
}

// Where a token's rows lie: its page, or -1 for none (a token of no sequence,
// before the sequence's first place or past its pages, or a page that the pool
// does not have).
struct Slot {
    int page, in, seq;
};

__device__ __forceinline__ Slot slot_of(const KvRowsParams& p, int token) {
    Slot s{-1, 0, sequence_of(p.b, token)};
    if (s.seq < 0) return s;
    const Span sp = span_of(p.b, s.seq);
    const int pos = length_of(p.b, s.seq) - (sp.first + sp.count - token);
    if (pos < 0 || pos >= p.b.width * p.c.page) return s;
    const Place at = place_of(p.c, pos);
    const int page = page_of(p.b, s.seq, at.index);
    if ((unsigned)page < (unsigned)p.c.pages) s.page = page, s.in = at.in;
    return s;
}

template <int CDT, int DT, int LPR, bool WRITE>
__global__ __launch_bounds__(kThreads) void kv_rows_kernel(KvRowsParams p) {
    constexpr int RPB = kThreads / LPR;
    constexpr int ES = DT == DT_F32 ? 4 : 2, CS = CDT == DT_E4M3 ? 1 : 2;
    const int lane = threadIdx.x % LPR;
    // a workgroup has neighbouring tokens of one head: whole lines of the cache and of its scales
    const int block = blockIdx.x / p.c.heads, head = blockIdx.x - block * p.c.heads;
    const int token = block * RPB + (int)threadIdx.x / LPR;
    // the lanes of a row go together; those past its elements help in its maximum
    const bool on = token < p.b.tokens && lane * kV < p.c.dim;
    char* const k = p.k + token * p.k_token + head * p.k_head + lane * kV * ES;
    char* const v = p.v + token * p.v_token + head * p.v_head + lane * kV * ES;
    float fk[kV] = {}, fv[kV] = {};
    if (WRITE && on) {
        load8<DT>(k, fk);
        load8<DT>(v, fv);
    }
    Slot s{-1, 0, -1};
    if (token < p.b.tokens) s = slot_of(p, token);
    const long long at = s.page * p.c.ld_page + s.in * p.c.ld_token + head * p.c.ld_head + lane * kV * CS;
    const long long sat = s.page * p.c.lds_page + s.in * p.c.lds_token + head * p.c.lds_head;
    if constexpr (WRITE) {
        if constexpr (CDT == DT_E4M3) {
            const int ek = scale_field(row_top<LPR>(fk)), ev = scale_field(row_top<LPR>(fv));
            if (!on || s.page < 0) return;
            store_codes(p.c.k + at, fk, __uint_as_float((uint32_t)(254 - ek) << 23));
            store_codes(p.c.v + at, fv, __uint_as_float((uint32_t)(254 - ev) << 23));
            if (lane == 0) {
                p.c.ks[sat] = __uint_as_float((uint32_t)ek << 23);
                p.c.vs[sat] = __uint_as_float((uint32_t)ev << 23);
            }
        } else {
            if (!on || s.page < 0) return;
            store8<CDT>(p.c.k + at, fk);
            store8<CDT>(p.c.v + at, fv);
        }
    } else {
        if (!on || s.seq < 0) return;
        if (s.page >= 0) {
            if constexpr (CDT == DT_E4M3) {
                load_codes(p.c.k + at, fk, p.c.ks[sat]);
                load_codes(p.c.v + at, fv, p.c.vs[sat]);
            } else {
                load8<CDT>(p.c.k + at, fk);
                load8<CDT>(p.c.v + at, fv);
            }
        }
        store8<DT>(k, fk);
        store8<DT>(v, fv);
    }
}

template <int CDT, int DT, bool WRITE>
hipError_t launch_lanes(const KvRowsParams& p, hipStream_t stream) {
    auto go = [&](auto lanes) {
        constexpr int LPR = decltype(lanes)::value, RPB = kThreads / LPR;
        const dim3 blocks((unsigned)((p.b.tokens + RPB - 1) / RPB * p.c.heads));
        kv_rows_kernel<CDT, DT, LPR, WRITE><<<blocks, dim3(kThreads), 0, stream>>>(p);
        return hipGetLastError();
    };
    if (p.c.dim <= 64) return go(std::integral_constant<int, 8>{});
    if (p.c.dim <= 128) return go(std::integral_constant<int, 16>{});
    return go(std::integral_constant<int, 32>{});
}

template <int CDT, bool WRITE>
hipError_t launch_type(const KvRowsParams& p, int dt, hipStream_t stream) {
    if (dt == DT_F32) return launch_lanes<CDT, DT_F32, WRITE>(p, stream);
    if (dt == DT_F16) return launch_lanes<CDT, DT_F16, WRITE>(p, stream);
    return launch_lanes<CDT, DT_BF16, WRITE>(p, stream);
}

template <bool WRITE>
hipError_t launch_rows_of(const KvRowsParams& p, int cache_dt, int dt, hipStream_t stream) {
    (void)hipGetLastError();
    if (cache_dt == DT_E4M3) return launch_type<DT_E4M3, WRITE>(p, dt, stream);
    if (cache_dt == DT_F16) return launch_type<DT_F16, WRITE>(p, dt, stream);
    return launch_type<DT_BF16, WRITE>(p, dt, stream);
}

}  // namespace

hipError_t launch_kv_write(const KvRowsParams& p, int cache_dt, int dt, hipStream_t stream) {
    return launch_rows_of<true>(p, cache_dt, dt, stream);
}

hipError_t launch_kv_read(const KvRowsParams& p, int cache_dt, int dt, hipStream_t stream) {
    return launch_rows_of<false>(p, cache_dt, dt, stream);
}

}  // namespace ct
