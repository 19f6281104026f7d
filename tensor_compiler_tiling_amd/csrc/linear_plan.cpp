// Which kernel runs a product, how its work is divided and what workspace it
// needs (linear.hip has the kernels): host arithmetic on sizes alone.
#include <algorithm>

#include "../../include/convtile.h"
#include "block_kernels.hpp"

namespace ct {

namespace {

// A tile's rows and columns.
int tile_of_form(int form) { return form == LIN_T64 ? 64 : form == LIN_T256 ? 256 : 128; }

// Microseconds of a stage on a CU that runs n workgroups of a form together
// or one after another, measured on this card with operands in the caches: the
// small tiles are bound by what a CU takes in (16 KB a stage of a 64 x 64
// tile, 32 KB of a 128 x 128 one, at 70 to 90 GB/s), the large one by LDS and
// the matrix units together, fp32 by the matrix units alone.
double stage_us(int form, bool f32, long long n) {
    switch (form) {
        case LIN_T64: return f32 ? 0.45 * n : n == 1 ? 0.18 : 0.15 * n;
        case LIN_T128K: return f32 ? 1.75 * n : n == 1 ? 0.40 : 0.48 * n;
        case LIN_T128: return f32 ? 1.75 * n : 0.46 * n;
        default: return f32 ? 7.0 * n : 1.5 * n;
    }
}

// What a workgroup takes beside its stages (the first loads, the results).
double edge_us(int form) { return form == LIN_T64 ? 2.0 : form == LIN_T256 ? 7.0 : 3.0; }

// Microseconds of a row form: its waves' turns of 8 stages (0.7 us, 1.2 with two
// groups of rows), or the weights' bytes, or, with two groups, the weights' and
// twice as many of x's from L2.
double row_us(int M, int N, int kbytes) {
    const double turns = (kbytes + 8 * kStage - 1) / (8 * kStage), bytes = (double)N * kbytes;
    return M <= 16 ? std::max(2.5 + 0.7 * turns, 1.5 + bytes / 4.8e6) : std::max(2.5 + 1.2 * turns, 2.0 + 3.0 * bytes / 10e6);
}

}  // namespace

long long linear_workgroups(const LinearPlan& plan, int M, int N) {
    if (plan.form < LIN_T64) return (N + 15LL) / 16;
    const long long b = tile_of_form(plan.form);
    return plan.full + ((M + b - 1) / b * ((N + b - 1) / b) - plan.full) * plan.S;
}

long long linear_workspace_bytes(const LinearPlan& plan, int M, int N, int kbytes) {
    if (plan.form < LIN_T64) return 0;
    const long long b = tile_of_form(plan.form);
    const long long rest = (M + b - 1) / b * ((N + b - 1) / b) - plan.full;
    return rest * plan.S * b * b * 4 + (plan.pack ? ((long long)M + N) * linear_pack_pitch(kbytes) : 0);
}

// The tile, and what of it is split, that the measured rates above expect to
// end first.
// Whole rounds of tiles (one a CU) are computed whole; the rest, or all where
// they do not fill the device, may be split over k so that every CU has a
// share, at the price of writing and reading the parts (4 bytes a result and
// part, at about 4 TB/s) and of a second launch (2.5 us; 4 after whole tiles,
// whose CUs the parts share).  Measured, whole against split: 640 x 2048 x 2048
// fp32 72 against 49 us (tiles past the first 256 in 4 parts), 64 x 4096 x 12288
// bf16 71 against 28 (all in 4), 256 x 1024 x 1024 bf16 10 against 13.
//
// Up to 32 rows of x, a row form where that is expected to take less, or less
// than the 11 us that the host needs for a split product's two launches (it
// splits no sum over workgroups and reads the weights once; in a captured graph
// the tiles would be up to 1 us ahead on some of these).  Measured on the
// device, row form against tiles: 8 rows, bf16, 4096 x 4096 8.9 and 10.1, 1024 x
// 4096 8.3 and 7.4, 1024 x 8192 14.0 and 9.9, 256 x 16384 24.9 and 8.7; 24 rows, 1024
// x 1024 4.8 and 5.8, 4096 x 4096 12.3 and 11.8, 16384 x 1024 12.2 and 9.2; fp32 4096
// x 4096 22.3 and 25.9, 1000 x 16000 73.5 and 27.3.
LinearPlan linear_plan(int M, int N, int kbytes, int dtype) {
    const bool f32 = dtype == CT_F32;
    const LinearPlan rows{M <= 16 ? LIN_ROW16 : LIN_ROW32, 0, 1, 0};
    if (M <= 32 && row_us(M, N, kbytes) <= 11.0) return rows;
    const int stages = (kbytes + kStage - 1) / kStage;
    constexpr int CUS = 256;
    auto rounds = [](long long t) { return (t + CUS - 1) / CUS; };
    LinearPlan best{LIN_T64, 0, 1, 0};
    double best_us = 1e300;
    for (int form = LIN_T64; form <= LIN_T256; ++form) {
        const long long b = tile_of_form(form);
        const long long t = (M + b - 1) / b * ((N + b - 1) / b);
        const double whole = stages * stage_us(form, f32, rounds(t)) + edge_us(form) * rounds(t);
        if (whole < best_us) best_us = whole, best = {form, (int)t, 1, 0};
        if (form == LIN_T256) continue;  // its parts are too large to pay
        const long long full = t / CUS * CUS, rest = t - full;
        if (rest == 0 || full > 8 * CUS) continue;
        for (int want = 2; want <= 16; ++want) {
            // every part has stages of its own, at least 4
            const int per = (stages + want - 1) / want, S = (stages + per - 1) / per;
            if (per < 4 || S < 2) break;
            const double parts = (double)rest * S * b * b * 8 / 4e6;
            const double us = stages * (full ? stage_us(form, f32, full / CUS) : 0.0) +
                              per * stage_us(form, f32, rounds(rest * S)) +
                              edge_us(form) * (full / CUS + rounds(rest * S)) + parts + (full ? 4.0 : 2.5);
            if (us < best_us) best_us = us, best = {form, (int)full, S, 0};
        }
    }
    if (M <= 32) {
        const double tiles = std::max(best_us, (double)N * kbytes / 4.8e6) + 2.0;
        if (row_us(M, N, kbytes) <= tiles) return rows;
    }
    // Rows whose length is no multiple of 16 bytes cannot go to LDS directly.
    // Passing through registers costs a product about 0.7 of its time more
    // (100 x 4096 x 4095 fp16 23 us, 16 for K = 4096; 2048 x 4096 x 4095 106 and
    // 69), the largest tile, which has no registers to spare, more than that, and
    // fp32, which the matrix units bound, a sixth (2048 x 2048 x 2047 145 us, 127;
    // 1472 x 169 x 11597 69, 99 copied);
    // copying both operands to whole stages costs their bytes twice at about
    // 4.5 TB/s and a launch (4096 x 4096 x 4095 fp16 204 us through registers,
    // 150 copied; e4m3 133 and 74).  Rows of whole chunks that start off 16 bytes go
    // through registers too (4096 x 4096 x 4096 fp16 240 us, 116 aligned), never
    // copied: the plan, and with it the workspace, goes by the sizes alone.
    if (kbytes % 16) best.pack = 2.0 * (M + (double)N) * kbytes / 4.5e6 + 2.5 < (f32 ? 0.17 : 0.7) * best_us;
    return best;
}

}  // namespace ct
