// Host-side checks of the transformer-block entry points, built like
// host_check.cpp: the refusals of ct_rmsnorm_fwd, ct_quantize_rows,
// ct_linear_fwd and ct_linear_q8_fwd (nothing here launches), the answers of
// ct_linear_workspace_bytes at the ends of its range, and the plan behind
// them: every part of a split sum has a stage, the parts cover the sum, and
// the workspace holds the parts and the copied rows.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "block_kernels.hpp"
#include "convtile.h"

static int g_fail = 0;
#define CHECK(cond)                                                              \
    do {                                                                         \
        if (!(cond)) {                                                           \
            std::fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond); \
            ++g_fail;                                                            \
        }                                                                        \
    } while (0)

namespace {

// addresses that no call here reads
char* at(int mib) { return reinterpret_cast<char*>(static_cast<uintptr_t>(mib) << 20); }
float* floats(int mib) { return reinterpret_cast<float*>(at(mib)); }

int norm(const void* x, long long ldx, void* h, long long ldh, void* y, long long ldy, int M, int D, int dt, int odt,
         float eps, float* scale = nullptr) {
    return ct_rmsnorm_fwd(x, ldx, at(2), D, floats(9), h, ldh, y, ldy, scale, M, D, dt, odt, eps, nullptr);
}

void refusals() {
    CHECK(norm(at(1), 64, at(3), 64, at(4), 64, -1, 64, CT_BF16, CT_BF16, 0) == CT_ERR_INVALID_ARG);
    CHECK(norm(at(1), 64, at(3), 64, at(4), 64, 4, 0, CT_BF16, CT_BF16, 0) == CT_ERR_INVALID_ARG);
    CHECK(norm(at(1), 63, at(3), 64, at(4), 64, 4, 64, CT_BF16, CT_BF16, 0) == CT_ERR_INVALID_ARG);
    CHECK(norm(at(1), LLONG_MAX, at(3), 64, at(4), 64, 4, 64, CT_BF16, CT_BF16, 0) == CT_ERR_INVALID_ARG);
    CHECK(norm(at(1), LLONG_MIN, at(3), 64, at(4), 64, 4, 64, CT_BF16, CT_BF16, 0) == CT_ERR_INVALID_ARG);
    CHECK(norm(at(1), 64, at(3), 64, at(4), 64, 4, 64, CT_BF16, CT_BF16, NAN) == CT_ERR_INVALID_ARG);
    CHECK(norm(at(1), 64, at(3), 64, at(3), 64, 4, 64, CT_BF16, CT_BF16, 0) == CT_ERR_INVALID_ARG);
    CHECK(norm(at(1), 64, at(3), 64, at(1), 64, 4, 64, CT_BF16, CT_E4M3, 0, floats(8)) == CT_ERR_INVALID_ARG);
    CHECK(norm(at(1), 64, at(1), 72, at(4), 64, 4, 64, CT_BF16, CT_BF16, 0) == CT_ERR_INVALID_ARG);
    CHECK(norm(at(1), INT_MAX, at(3), INT_MAX, at(4), INT_MAX - 1LL, INT_MAX, INT_MAX, CT_F32, CT_F32, 0) ==
          CT_ERR_INVALID_ARG);
    CHECK(std::strlen(ct_last_error()) > 0);
    CHECK(norm(nullptr, 0, nullptr, 0, nullptr, 0, 0, 64, CT_BF16, CT_BF16, 0) == CT_OK);
    CHECK(ct_quantize_rows(at(1), 64, at(1), 64, floats(8), 4, 64, CT_F32, nullptr) == CT_ERR_INVALID_ARG);
    CHECK(ct_quantize_rows(at(1), 64, at(2), 64, nullptr, 4, 64, CT_F32, nullptr) == CT_ERR_INVALID_ARG);
    CHECK(ct_quantize_rows(at(1), 64, at(2), 64, floats(8), 4, 64, CT_E4M3, nullptr) == CT_ERR_INVALID_ARG);
    CHECK(ct_quantize_rows(nullptr, 0, nullptr, 0, nullptr, 0, 64, CT_F32, nullptr) == CT_OK);

    auto linear = [](int M, int N, int K, int dt, const ct_linear_epilogue* ep, long long ldx, long long space) {
        return ct_linear_fwd(at(1), ldx, at(2), K, at(3), N, M, N, K, dt, CT_F32, ep, space ? at(7) : nullptr, space, nullptr);
    };
    ct_linear_epilogue ep{};
    ep.act = 99;
    CHECK(linear(4, 32, 64, CT_BF16, &ep, 64, 0) == CT_ERR_INVALID_ARG);
    ep.act = INT_MIN;
    CHECK(linear(4, 32, 64, CT_BF16, &ep, 64, 0) == CT_ERR_INVALID_ARG);
    ep = ct_linear_epilogue{};
    ep.gate = at(3);
    ep.ldg = 40;
    CHECK(linear(4, 32, 64, CT_BF16, &ep, 64, 0) == CT_ERR_INVALID_ARG);
    CHECK(linear(4, 32, 64, CT_E4M3, nullptr, 64, 0) == CT_ERR_INVALID_ARG);
    CHECK(linear(4, 32, 64, CT_BF16, nullptr, 63, 0) == CT_ERR_INVALID_ARG);
    CHECK(linear(4, 32, 64, CT_BF16, nullptr, (4LL << 20) + 1, 0) == CT_ERR_UNSUPPORTED);
    CHECK(linear(INT_MAX, INT_MAX, INT_MAX, CT_F32, nullptr, INT_MAX, 0) == CT_ERR_UNSUPPORTED);
    CHECK(linear(1 << 30, 1 << 30, 1, CT_F32, nullptr, 1, 0) == CT_ERR_UNSUPPORTED);
    CHECK(linear(1 << 30, 64, 1, CT_F32, nullptr, 1, 0) == CT_ERR_UNSUPPORTED);
    const long long need = ct_linear_workspace_bytes(64, 512, 8192, CT_BF16);
    CHECK(need > 0);
    CHECK(linear(64, 512, 8192, CT_BF16, nullptr, 8192, need - 1) == CT_ERR_INVALID_ARG);
    CHECK(linear(64, 512, 8192, CT_BF16, nullptr, 8192, LLONG_MIN) == CT_ERR_INVALID_ARG);
    CHECK(ct_linear_q8_fwd(at(1), 64, nullptr, at(2), 64, floats(8), at(3), 32, 4, 32, 64, CT_BF16, nullptr, nullptr, 0,
                           nullptr) == CT_ERR_INVALID_ARG);
    CHECK(ct_linear_q8_fwd(nullptr, 0, nullptr, nullptr, 0, nullptr, nullptr, 0, 0, 32, 64, CT_BF16, nullptr, nullptr, 0,
                           nullptr) == CT_OK);
}

// The plan of one product, against its own description.
void plan(int M, int N, int K, int dt, long long* forms) {
    const int es = dt == CT_F32 ? 4 : dt == CT_E4M3 ? 1 : 2;
    const long long need = ct_linear_workspace_bytes(M, N, K, dt);
    if ((long long)K * es > 1 << 30 || M > 1 << 30 || N > 1 << 30 || ((M + 63LL) / 64) * ((N + 63LL) / 64) > INT_MAX) {
        CHECK(need == CT_ERR_UNSUPPORTED);
        return;
    }
    const int kbytes = K * es;
    const ct::LinearPlan p = ct::linear_plan(M, N, kbytes, dt);
    if (ct::linear_workgroups(p, M, N) >= 1 << 23) {  // the product refuses: so does the question
        CHECK(need == CT_ERR_UNSUPPORTED);
        return;
    }
    CHECK(need == ct::linear_workspace_bytes(p, M, N, kbytes));
    CHECK(p.form >= ct::LIN_ROW16 && p.form <= ct::LIN_T256 && p.S >= 1 && p.S <= 16);
    ++forms[p.form];
    if (p.form < ct::LIN_T64) {
        CHECK(M <= (p.form == ct::LIN_ROW16 ? 16 : 32) && need == 0 && p.pack == 0);
        CHECK(ct::linear_workgroups(p, M, N) == (N + 15LL) / 16);
        return;
    }
    const long long b = p.form == ct::LIN_T64 ? 64 : p.form == ct::LIN_T256 ? 256 : 128;
    const long long tiles = ((M + b - 1) / b) * ((N + b - 1) / b), rest = tiles - p.full;
    CHECK(p.full >= 0 && rest >= 0 && rest < 256);
    CHECK((rest == 0) == (p.S == 1));
    CHECK(ct::linear_workgroups(p, M, N) == p.full + rest * p.S);
    // one workgroup past the last stage would have nothing to add
    const int stages = (kbytes + ct::kStage - 1) / ct::kStage, per = ct::linear_part_stages(kbytes, p.S);
    CHECK((long long)per * p.S >= stages && (long long)per * (p.S - 1) < stages);
    long long space = rest * p.S * b * b * 4;
    if (p.pack) {
        ++forms[6];
        const long long pitch = ct::linear_pack_pitch(kbytes);
        CHECK(kbytes % 16 != 0 && pitch >= kbytes && pitch % ct::kStage == 0);
        CHECK((pitch + ct::kStage - 1) / ct::kStage == stages);
        space += ((long long)M + N) * pitch;
    }
    CHECK(need == space);
}

// fp32 takes 128 x 128 tiles with two groups of waves whenever it takes such tiles.
void every_form(int dt, const long long* forms) {
    for (int f = 0; f < 7; ++f) CHECK((forms[f] > 0) == !(dt == CT_F32 && f == ct::LIN_T128));
}

void plans() {
    const int rows[] = {1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 128, 255, 257, 640, 1011, 2049, 4097, 8192, 65537,
                        1 << 20, (1 << 30) - 1, 1 << 30};
    const int lengths[] = {1, 7, 31, 32, 63, 64, 65, 127, 129, 512, 515, 999, 2047, 4096, 4095, 12000, 16384, 65537, 1 << 20,
                           (1 << 23) + 1, 1 << 28, (1 << 29) - 1, 1 << 29, 1 << 30};
    const int types[] = {CT_F32, CT_F16, CT_BF16, CT_E4M3};
    for (int dt : types) {
        long long forms[7] = {};
        for (int M : rows)
            for (int N : rows)
                for (int K : lengths) plan(M, N, K, dt, forms);
        every_form(dt, forms);
    }
    // the sizes that tests/test_gpu_block_forms.py multiplies reach every form
    // and the copy in every type
    const int sizes[][3] = {{5, 100, 129}, {24, 1024, 1024}, {24, 515, 130}, {70, 90, 515}, {8, 256, 16383}, {640, 2048, 1024},
                            {1100, 2048, 999}, {1500, 1500, 200}, {2049, 2050, 200}, {2500, 2048, 131}, {4097, 4090, 264},
                            {4100, 4097, 139}, {4090, 4000, 272}, {3900, 4090, 139}};
    for (int dt : types) {
        long long forms[7] = {};
        for (const auto& s : sizes) plan(s[0], s[1], s[2], dt, forms);
        std::printf("forms of type %d: %lld %lld %lld %lld %lld %lld, copied %lld\n", dt, forms[0], forms[1], forms[2],
                    forms[3], forms[4], forms[5], forms[6]);
        every_form(dt, forms);
    }
    CHECK(ct_linear_workspace_bytes(0, 32, 64, CT_BF16) == 0);
    for (int bad : {0, -1, INT_MIN}) {
        CHECK(ct_linear_workspace_bytes(4, bad, 64, CT_BF16) == CT_ERR_INVALID_ARG);
        CHECK(ct_linear_workspace_bytes(4, 32, bad, CT_BF16) == CT_ERR_INVALID_ARG);
    }
    CHECK(ct_linear_workspace_bytes(-1, 32, 64, CT_BF16) == CT_ERR_INVALID_ARG);
    CHECK(ct_linear_workspace_bytes(INT_MAX, INT_MAX, INT_MAX, CT_E4M3) == CT_ERR_UNSUPPORTED);
}

}  // namespace

int main() {
    refusals();
    plans();
    std::printf("block checks: %d failed\n", g_fail);
    return g_fail ? 1 : 0;
}
