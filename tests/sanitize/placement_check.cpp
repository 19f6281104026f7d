// Host-side check of what the workgroup-placement probe accepts, built like
// host_check.cpp: every order of the XCDs that repeats after eight workgroups,
// and nothing else.
#include <cstdio>
#include <vector>

#include "ct_kernels.hpp"

static int g_fail = 0;
#define CHECK(cond)                                                              \
    do {                                                                         \
        if (!(cond)) {                                                           \
            std::fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond); \
            ++g_fail;                                                            \
        }                                                                        \
    } while (0)

int main() {
    constexpr int kBlocks = 4096;
    std::vector<int> h(kBlocks);
    for (int first = 0; first < 8; ++first) {
        for (int b = 0; b < kBlocks; ++b) h[b] = (b + first) % 8;
        CHECK(ct::placed_round_robin(h.data(), kBlocks));
        for (int at : {0, 7, 8, 100, kBlocks - 1}) {  // one workgroup elsewhere, or not heard of
            const int was = h[at];
            for (int bad : {(was + 1) % 8, -1, 8, 15}) {
                h[at] = bad;
                CHECK(!ct::placed_round_robin(h.data(), kBlocks));
            }
            h[at] = was;
        }
    }
    const int order[8] = {3, 0, 7, 1, 6, 2, 5, 4};
    for (int b = 0; b < kBlocks; ++b) h[b] = order[b % 8];
    CHECK(ct::placed_round_robin(h.data(), kBlocks));
    for (int b = 0; b < kBlocks; ++b) h[b] = b % 4;  // fewer XCDs
    CHECK(!ct::placed_round_robin(h.data(), kBlocks));
    for (int b = 0; b < kBlocks; ++b) h[b] = b / 8 % 8;  // in runs
    CHECK(!ct::placed_round_robin(h.data(), kBlocks));
    for (int b = 0; b < kBlocks; ++b) h[b] = b % 8 + b / 2048 % 2;  // a shift on the way
    CHECK(!ct::placed_round_robin(h.data(), kBlocks));
    CHECK(!ct::placed_round_robin(h.data(), 7));
    std::printf("placement checks: %d failed\n", g_fail);
    return g_fail != 0;
}
