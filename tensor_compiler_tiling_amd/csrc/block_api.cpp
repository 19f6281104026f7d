// C entry points of the transformer-block kernels (include/convtile.h):
// argument checks, the choice of kernel and the launch.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "../../include/convtile.h"
#include "block_kernels.hpp"
#include "ct_kernels.hpp"

namespace ct {

namespace {

constexpr int kMaxRows = 1 << 30;            // M, N, and bytes of a row
constexpr long long kMaxStride = 8LL << 20;  // bytes between rows that a product reads

bool plain_dtype(int dt) { return dt == CT_F32 || dt == CT_F16 || dt == CT_BF16; }
int elem_bytes(int dt) { return dt == CT_F32 ? 4 : dt == CT_E4M3 ? 1 : 2; }

// A matrix argument: not NULL, aligned to its element, rows apart.
int check_matrix(const char* name, const void* p, long long ld, int cols, int dt) {
    if (!p) return fail(CT_ERR_INVALID_ARG, "%s must not be NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % elem_bytes(dt))
        return fail(CT_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    if (ld < cols) return fail(CT_ERR_INVALID_ARG, "%s: row stride %lld below the row's %d elements", name, ld, cols);
    if (ld > (1LL << 40)) return fail(CT_ERR_INVALID_ARG, "%s: row stride %lld is too large", name, ld);
    return CT_OK;
}

int check_floats(const char* name, const float* p) {
    if (!p) return fail(CT_ERR_INVALID_ARG, "%s must not be NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % 4) return fail(CT_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    return CT_OK;
}

// An output on an input's place: every element must fall on the one it is made
// from (one type, and one stride where there are rows to be apart), or a row's
// results land on another's inputs before they are read.
int check_in_place(const char* out, const void* o, long long ldo, int odt, const char* in, const void* i, long long ldi,
                   int idt, int M) {
    if (!i || o != i || (odt == idt && (M == 1 || ldo == ldi))) return CT_OK;
    return fail(CT_ERR_INVALID_ARG, "%s is in the place of %s with another type or stride", out, in);
}

bool aligned16(const void* p, long long ld_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld_bytes % 16 == 0;
}

int rows_call(const void* x, long long ldx, const void* residual, long long ldr, const float* gain, void* h,
              long long ldh, void* y, long long ldy, float* scale, int M, int D, int dtype, int out_dtype, float eps,
              bool norm, void* stream) {
    if (M < 0 || D < 1) return fail(CT_ERR_INVALID_ARG, "M must not be negative and D must be positive");
    if (!plain_dtype(dtype)) return fail(CT_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (!plain_dtype(out_dtype) && out_dtype != CT_E4M3) return fail(CT_ERR_INVALID_ARG, "unknown out_dtype %d", out_dtype);
    if (norm && !(eps >= 0.0f && eps <= FLT_MAX)) return fail(CT_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (h && !residual) return fail(CT_ERR_INVALID_ARG, "h is the sum with residual, which is NULL");
    if (M == 0) return CT_OK;
    const char* yname = norm ? "y" : "q";
    int st = check_matrix("x", x, ldx, D, dtype);
    if (st == CT_OK) st = check_matrix(yname, y, ldy, D, out_dtype);
    if (st == CT_OK && residual) st = check_matrix("residual", residual, ldr, D, dtype);
    if (st == CT_OK && h) st = check_matrix("h", h, ldh, D, dtype);
    if (st == CT_OK && gain) st = check_floats("gain", gain);
    if (st == CT_OK) st = check_in_place(yname, y, ldy, out_dtype, "x", x, ldx, dtype, M);
    if (st == CT_OK) st = check_in_place(yname, y, ldy, out_dtype, "residual", residual, ldr, dtype, M);
    if (st == CT_OK && h) st = check_in_place("h", h, ldh, dtype, "x", x, ldx, dtype, M);
    if (st == CT_OK && h) st = check_in_place("h", h, ldh, dtype, "residual", residual, ldr, dtype, M);
    if (st == CT_OK && h == y) return fail(CT_ERR_INVALID_ARG, "h and y must not be the same");
    if (st != CT_OK) return st;
    if (out_dtype == CT_E4M3) {
        st = check_floats("scale", scale);
        if (st != CT_OK) return st;
    } else if (scale) {
        return fail(CT_ERR_INVALID_ARG, "scale belongs to CT_E4M3 output");
    }
    RowsParams p{};
    const int es = elem_bytes(dtype);
    p.x = static_cast<const char*>(x);
    p.res = static_cast<const char*>(residual);
    p.gain = gain;
    p.h = static_cast<char*>(h);
    p.y = static_cast<char*>(y);
    p.scale = scale;
    p.ldx = ldx * es;
    p.ldres = residual ? ldr * es : 0;
    p.ldh = h ? ldh * es : 0;
    p.ldy = ldy * elem_bytes(out_dtype);
    p.D = D;
    p.out_dt = out_dtype;
    p.eps = eps;
    const hipError_t e = launch_rows(p, M, dtype, norm, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? CT_OK : hip_fail(e, norm ? "rmsnorm launch" : "quantize launch");
}

// Sizes and type of a product, whose plan goes to `plan` (not for M = 0).
int check_product(int M, int N, int K, int dtype, bool q8, LinearPlan* plan) {
    if (M < 0 || N < 1 || K < 1) return fail(CT_ERR_INVALID_ARG, "M must not be negative, N and K must be positive");
    if (q8 ? dtype != CT_E4M3 : !plain_dtype(dtype)) return fail(CT_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (M > kMaxRows || N > kMaxRows || (long long)K * elem_bytes(dtype) > kMaxRows)
        return fail(CT_ERR_UNSUPPORTED, "M, N and the bytes of a row must be at most 2^30");
    if (((M + 63LL) / 64) * ((N + 63LL) / 64) > 0x7fffffffLL) return fail(CT_ERR_UNSUPPORTED, "too many tiles");
    if (M == 0) return CT_OK;
    *plan = linear_plan(M, N, K * elem_bytes(dtype), dtype);
    // 512 threads each: fewer than 2^32 in a launch
    const long long groups = linear_workgroups(*plan, M, N);
    if (groups >= 1LL << 23) return fail(CT_ERR_UNSUPPORTED, "%lld tiles: more than one launch takes", groups);
    return CT_OK;
}

int linear_call(const void* x, long long ldx, const float* xs, const void* w, long long ldw, const float* ws, void* y,
                long long ldy, int M, int N, int K, int dtype, int out_dtype, const ct_linear_epilogue* epi,
                void* workspace, long long workspace_bytes, void* stream) {
    const bool q8 = dtype == CT_E4M3;
    LinearPlan plan{};
    int st = check_product(M, N, K, dtype, q8, &plan);
    if (st != CT_OK) return st;
    if (!plain_dtype(out_dtype)) return fail(CT_ERR_INVALID_ARG, "unknown out_dtype %d", out_dtype);
    const ct_linear_epilogue none{CT_ACT_NONE, nullptr, nullptr, 0, nullptr, 0};
    const ct_linear_epilogue& ep = epi ? *epi : none;
    if (ep.act < CT_ACT_NONE || ep.act > CT_ACT_SILU) return fail(CT_ERR_INVALID_ARG, "unknown activation %d", ep.act);
    if (M == 0) return CT_OK;
    st = check_matrix("x", x, ldx, K, dtype);
    if (st == CT_OK) st = check_matrix("w", w, ldw, K, dtype);
    if (st == CT_OK) st = check_matrix("y", y, ldy, N, out_dtype);
    if (st == CT_OK && (y == x || y == w)) return fail(CT_ERR_INVALID_ARG, "y must not be x or w");
    if (st == CT_OK && ep.gate) st = check_matrix("gate", ep.gate, ep.ldg, N, out_dtype);
    if (st == CT_OK && ep.residual) st = check_matrix("residual", ep.residual, ep.ldr, N, out_dtype);
    if (st == CT_OK) st = check_in_place("y", y, ldy, out_dtype, "gate", ep.gate, ep.ldg, out_dtype, M);
    if (st == CT_OK) st = check_in_place("y", y, ldy, out_dtype, "residual", ep.residual, ep.ldr, out_dtype, M);
    if (st == CT_OK && ep.bias) st = check_floats("bias", ep.bias);
    if (st == CT_OK && q8) st = check_floats("xs", xs);
    if (st == CT_OK && q8) st = check_floats("ws", ws);
    if (st != CT_OK) return st;
    const int es = elem_bytes(dtype), oes = elem_bytes(out_dtype);
    LinearParams p{};
    // a single row has no stride to speak of
    p.ldx = (M > 1 ? ldx : K) * es;
    p.ldw = (N > 1 ? ldw : K) * es;
    // the tiles address a row by its 32-bit offset from the tile's first
    if ((M > 1 && p.ldx > kMaxStride) || (N > 1 && p.ldw > kMaxStride))
        return fail(CT_ERR_UNSUPPORTED, "rows of x and w must be at most 8 MiB apart");
    p.kbytes = K * es;
    const long long need = linear_workspace_bytes(plan, M, N, p.kbytes);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(CT_ERR_INVALID_ARG, "this product needs a workspace of %lld bytes (got %lld)", need,
                        workspace ? workspace_bytes : 0LL);
        if (reinterpret_cast<uintptr_t>(workspace) % 16) return fail(CT_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    }
    p.x = static_cast<const char*>(x);
    p.w = static_cast<const char*>(w);
    p.y = static_cast<char*>(y);
    p.bias = ep.bias;
    p.gate = static_cast<const char*>(ep.gate);
    p.res = static_cast<const char*>(ep.residual);
    p.xs = q8 ? xs : nullptr;
    p.ws = q8 ? ws : nullptr;
    p.part = static_cast<float*>(workspace);
    p.ldy = ldy * oes;
    p.ldg = p.gate ? ep.ldg * oes : 0;
    p.ldr = p.res ? ep.ldr * oes : 0;
    p.M = M;
    p.N = N;
    p.act = ep.act;
    p.out_dt = out_dtype;
    const long long near = 1 << 20;
    p.near = oes == 2 && p.ldy <= near && p.ldg <= near && p.ldr <= near;
    const bool aligned = aligned16(x, p.ldx) && aligned16(w, p.ldw) && p.kbytes % 16 == 0;
    const hipError_t e = launch_linear(plan, p, dtype, aligned, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? CT_OK : hip_fail(e, "linear launch");
}

}  // namespace
}  // namespace ct

extern "C" {

int ct_rmsnorm_fwd(const void* x, long long ldx, const void* residual, long long ldr, const float* gain, void* h,
                   long long ldh, void* y, long long ldy, float* scale, int M, int D, int dtype, int out_dtype,
                   float eps, void* stream) {
    return ct::rows_call(x, ldx, residual, ldr, gain, h, ldh, y, ldy, scale, M, D, dtype, out_dtype, eps, true, stream);
}

int ct_quantize_rows(const void* x, long long ldx, void* q, long long ldq, float* scale, int M, int D, int dtype,
                     void* stream) {
    return ct::rows_call(x, ldx, nullptr, 0, nullptr, nullptr, 0, q, ldq, scale, M, D, dtype, CT_E4M3, 0.0f, false,
                         stream);
}

int ct_linear_fwd(const void* x, long long ldx, const void* w, long long ldw, void* y, long long ldy, int M, int N,
                  int K, int dtype, int out_dtype, const ct_linear_epilogue* epi, void* workspace,
                  long long workspace_bytes, void* stream) {
    if (dtype == CT_E4M3) return ct::fail(CT_ERR_INVALID_ARG, "8-bit rows have scales: call ct_linear_q8_fwd");
    return ct::linear_call(x, ldx, nullptr, w, ldw, nullptr, y, ldy, M, N, K, dtype, out_dtype, epi, workspace,
                           workspace_bytes, stream);
}

int ct_linear_q8_fwd(const void* x, long long ldx, const float* xs, const void* w, long long ldw, const float* ws,
                     void* y, long long ldy, int M, int N, int K, int out_dtype, const ct_linear_epilogue* epi,
                     void* workspace, long long workspace_bytes, void* stream) {
    return ct::linear_call(x, ldx, xs, w, ldw, ws, y, ldy, M, N, K, CT_E4M3, out_dtype, epi, workspace, workspace_bytes,
                           stream);
}

long long ct_linear_workspace_bytes(int M, int N, int K, int dtype) {
    ct::LinearPlan plan{};
    const int st = ct::check_product(M, N, K, dtype, dtype == CT_E4M3, &plan);
    if (st != CT_OK) return st;
    return M == 0 ? 0 : ct::linear_workspace_bytes(plan, M, N, K * ct::elem_bytes(dtype));
}

}  // extern "C"
