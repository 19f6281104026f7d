// Host-visible declarations of the transformer-block kernels: the linear
// layer (linear.hip, its plan linear_plan.cpp) and the row operators (rows.hip).  Arguments are checked
// by the C entry points (block_api.cpp) before they get here.
#pragma once

#include <hip/hip_runtime.h>

namespace ct {

// ---------------------------------------------------------------- linear --
// y = act(scale * x w^T + bias) * gate + residual (include/convtile.h).
// Pointers and strides are in bytes: a stage of the reduction is 128 bytes of
// a row whatever the type.
constexpr int kStage = 128;

struct LinearParams {
    const char* x;       // [M] rows of K elements, ldx bytes apart
    const char* w;       // [N] rows of K elements, ldw bytes apart
    char* y;             // [M] rows of N elements of out_dt
    const float* bias;   // [N] or null
    const char* gate;    // [M] rows of N elements of out_dt, or null
    const char* res;     // the same
    const float* xs;     // [M], [N] row scales of 8-bit operands, or null
    const float* ws;
    float* part;         // workspace: partial sums of the split tiles
    long long ldx, ldw, ldy, ldg, ldr;  // bytes
    int M, N;
    int kbytes;          // bytes of a row of x and w
    int act, out_dt;
    int near;            // y, gate and residual: two-byte elements, rows at most 1 MiB apart
    int tiles_m, tiles_n;
    int full, rest;      // tiles computed whole, and the others, whose
    int S;               // reduction is split into S parts
    int stages_per_split;
};

// The kernel that runs a product.
enum LinearForm {
    LIN_ROW16 = 0,  // at most 16 rows of x: weights straight to registers
    LIN_ROW32 = 1,  // at most 32
    LIN_T64 = 2,    // 64 x 64 tiles through LDS, two groups of waves sharing the reduction
    LIN_T128K = 3,  // 128 x 128, the same: a tile has a CU to itself
    LIN_T128 = 4,   // 128 x 128, two workgroups a CU
    LIN_T256 = 5,   // 256 x 256
};

struct LinearPlan {
    int form;
    int full;  // tiles that one workgroup computes whole (the tile forms)
    int S;     // workgroups that share each of the others, with parts of its reduction
    int pack;  // copy x and w to rows of whole stages first
};

// Stages of each of the S parts of a sum over rows of kbytes (the last may have
// fewer, none has none: S comes from the plan).
inline int linear_part_stages(int kbytes, int S) { return ((kbytes + kStage - 1) / kStage + S - 1) / S; }
// Bytes between rows that are copied to whole stages.
inline int linear_pack_pitch(int kbytes) { return (kbytes + kStage - 1) / kStage * kStage; }

// The form and split for a product of these sizes (kbytes: bytes of a row).
LinearPlan linear_plan(int M, int N, int kbytes, int dtype);
// Workgroups (of at most 512 threads) the plan launches for the product itself.
long long linear_workgroups(const LinearPlan& plan, int M, int N);
// Bytes of workspace (partial sums, or rows copied to a pitch) the plan needs.
long long linear_workspace_bytes(const LinearPlan& plan, int M, int N, int kbytes);
// p holds everything but the tiling fields, which are filled in here.
// aligned: rows of x and w are whole numbers of 16 bytes, 16-byte aligned.
hipError_t launch_linear(LinearPlan plan, LinearParams p, int dtype, bool aligned, hipStream_t stream);

// ------------------------------------------------------------------ rows --
// h = x + residual; y = h * rsqrt(mean h^2 + eps) * gain, or y = h where no
// norm is asked for; to out_dt, or to e4m3 with a scale a row.
struct RowsParams {
    const char* x;
    const char* res;    // or null
    const float* gain;  // or null
    char* h;            // or null
    char* y;
    float* scale;       // e4m3 only
    long long ldx, ldres, ldh, ldy;  // bytes
    int D;
    int out_dt;
    float eps;
};

hipError_t launch_rows(const RowsParams& p, int M, int dtype, bool norm, hipStream_t stream);

}  // namespace ct
