// Host-side checks of the key-value cache's entry points, built like
// host_check.cpp: refusals at the ends of the range (nothing here launches), the
// numbers that stand for a division by the page size, and the plan: the
// workspace holds every part, the tiles cover every row, and the launch is
// within its limits.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "attention_kernels.hpp"
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

ct_kv_cache cache_of(int pages, int heads, int page, int dim, int dtype) {
    ct_kv_cache c{};
    c.k = at(1), c.v = at(2);
    c.dtype = dtype, c.pages = pages, c.heads = heads, c.page = page, c.dim = dim;
    c.ld_token = dim, c.ld_head = (long long)dim * page, c.ld_page = c.ld_head * heads;
    if (dtype == CT_E4M3) {
        c.k_scale = reinterpret_cast<float*>(at(3)), c.v_scale = reinterpret_cast<float*>(at(4));
        c.lds_token = 1, c.lds_head = page, c.lds_page = (long long)page * heads;
    }
    return c;
}

ct_kv_batch batch_of(int tokens, int sequences, int width) {
    ct_kv_batch b{};
    b.tokens = tokens, b.sequences = sequences;
    b.lens = reinterpret_cast<int*>(at(5));
    b.table = reinterpret_cast<int*>(at(6));
    b.ldt = b.width = width;
    return b;
}

int attend(const ct_kv_cache& c, const ct_kv_batch& b, const ct_kv_mask* m, int heads, float scale, long long max_len,
           long long space) {
    return ct_kv_attention_fwd(&c, &b, m, at(7), (long long)heads * c.dim, c.dim, at(8), (long long)heads * c.dim, c.dim, heads,
                               CT_BF16, scale, max_len, space ? at(9) : nullptr, space, nullptr);
}

void refusals() {
    const ct_kv_cache c = cache_of(100, 2, 16, 64, CT_BF16), q8 = cache_of(100, 2, 16, 64, CT_E4M3);
    const ct_kv_batch b = batch_of(4, 2, 10);
    for (int bad : {INT_MIN, -1, 0}) {
        ct_kv_cache x = c;
        x.pages = bad;
        CHECK(ct_kv_write(&x, &b, at(7), 128, 64, at(8), 128, 64, CT_BF16, nullptr) == CT_ERR_INVALID_ARG);
        x = c, x.dim = bad;
        CHECK(ct_kv_read(&x, &b, at(7), 128, 64, at(8), 128, 64, CT_BF16, nullptr) == CT_ERR_INVALID_ARG);
        x = c, x.ld_page = bad;
        CHECK(attend(x, b, nullptr, 4, 1.0f, 0, 0) == CT_ERR_INVALID_ARG);
    }
    for (long long bad : {LLONG_MIN, LLONG_MAX, -1LL, 1LL << 62}) {
        ct_kv_cache x = q8;
        x.ld_head = bad;
        CHECK(attend(x, b, nullptr, 4, 1.0f, 0, 0) == CT_ERR_INVALID_ARG);
        x = q8, x.lds_token = bad;
        CHECK(attend(x, b, nullptr, 4, 1.0f, 0, 0) == CT_ERR_INVALID_ARG);
        CHECK(ct_kv_write(&c, &b, at(7), bad, 64, at(8), 128, 64, CT_BF16, nullptr) == CT_ERR_INVALID_ARG);
        CHECK(ct_kv_read(&c, &b, at(7), 128, 64, at(8), 128, bad, CT_BF16, nullptr) == CT_ERR_INVALID_ARG);
        ct_kv_batch y = b;
        y.ldt = bad;
        CHECK(attend(c, y, nullptr, 4, 1.0f, 0, 0) == CT_ERR_INVALID_ARG);
    }
    // strides as large as they may be, in every axis
    ct_kv_cache wide = c;
    wide.pages = INT_MAX, wide.ld_page = 1LL << 40, wide.ld_head = 1LL << 39, wide.ld_token = 1LL << 34;
    wide.page = 16;
    ct_kv_batch y = b;
    y.lens = nullptr;
    CHECK(attend(wide, y, nullptr, 4, 1.0f, 0, 0) == CT_ERR_INVALID_ARG);
    CHECK(std::strstr(ct_last_error(), "lens"));
    for (float bad : {0.0f, -1.0f, INFINITY, NAN}) CHECK(attend(c, b, nullptr, 4, bad, 0, 0) == CT_ERR_INVALID_ARG);
    CHECK(attend(c, b, nullptr, 4, 3e38f, 0, 0) == CT_ERR_UNSUPPORTED);
    for (int heads : {INT_MIN, -1, 0, 3, 5}) CHECK(attend(c, b, nullptr, heads, 1.0f, 0, 0) == CT_ERR_INVALID_ARG);
    CHECK(attend(c, b, nullptr, INT_MAX - 1, 1.0f, 0, 0) == CT_ERR_UNSUPPORTED);
    CHECK(attend(c, b, nullptr, 4, 1.0f, LLONG_MIN, 0) == CT_ERR_INVALID_ARG);
    ct_kv_mask m{INT_MIN, 0, nullptr, 0};
    CHECK(attend(c, b, &m, 4, 1.0f, 0, 0) == CT_ERR_INVALID_ARG);
    m = ct_kv_mask{1, INT_MIN, nullptr, 0};
    CHECK(attend(c, b, &m, 4, 1.0f, 0, 0) == CT_ERR_INVALID_ARG);
    m = ct_kv_mask{0, 0, reinterpret_cast<long long*>(at(10)), INT_MAX};
    CHECK(attend(c, b, &m, 4, 1.0f, 0, 0) == CT_ERR_INVALID_ARG);
    y = batch_of(INT_MAX, 1, 10);
    CHECK(attend(c, y, nullptr, 4, 1.0f, 0, 0) == CT_ERR_UNSUPPORTED);
    y = batch_of(4, 2, INT_MAX);
    CHECK(attend(c, y, nullptr, 4, 1.0f, 0, 0) == CT_ERR_UNSUPPORTED);
    y = batch_of(0, 0, 0);
    CHECK(attend(c, y, nullptr, 4, 1.0f, 0, 0) == CT_OK);
    CHECK(ct_kv_attention_workspace_bytes(INT_MAX, INT_MAX, INT_MAX, 1, 256, LLONG_MAX, INT_MAX, INT_MAX, CT_F16) == CT_ERR_UNSUPPORTED);
    CHECK(ct_kv_attention_workspace_bytes(INT_MIN, 1, 1, 1, 16, 0, 0, 0, CT_F16) == CT_ERR_INVALID_ARG);
}

void division() {
    for (int page : {1, 2, 3, 5, 7, 16, 24, 50, 64, 100, 1000, 4097, 65535, 65536, 1 << 20, (1 << 20) + 1, 1 << 30, INT_MAX}) {
        ct::KvPages c{};
        c.page = page;
        ct::page_magic(c);
        auto check = [&](long long n) {
            if (n < 0 || n > INT_MAX) return;
            CHECK((long long)(((unsigned long long)n * c.magic) >> c.shift) == n / page);
        };
        for (long long q : {0LL, 1LL, 2LL, 77LL, (long long)INT_MAX / page - 1, (long long)INT_MAX / page, (1LL << 30) / page})
            for (long long d : {-1LL, 0LL, 1LL}) check(q * page + d);
        check(INT_MAX);
        check(1 << 30);
    }
}

void plans() {
    for (int tokens : {1, 2, 7, 48, 64, 1000, 8192, 100000, (1 << 20) + 3})
        for (int sequences : {1, 2, 7, 64, 1000})
            for (int heads : {1, 3, 8, 32})
                for (int group : {1, 2, 5, 8, 16})
                    for (int dim : {16, 64, 80, 128, 192, 256})
                        for (long long len : {1LL, 100LL, 5000LL, 131072LL, 1LL << 30})
                            for (int window : {ct::kNoWindow, 1, 1024}) {
                                if ((long long)tokens * heads * group >= 1 << 26) continue;
                                const ct::AttendPlan p = ct::attend_plan(tokens, sequences, heads, group, dim, len, window, 4, tokens % 2 == 0);
                                CHECK(p.parts >= 1 && p.parts <= 128);
                                CHECK(p.form == ct::ATT_ROWS || p.form == ct::ATT_TILE);
                                CHECK(p.rows == ct::attend_rows(p.form, dim));
                                const long long space = ct::attend_workspace_bytes(p, tokens, heads * group, dim);
                                CHECK(space == (p.parts > 1 ? (long long)p.parts * tokens * heads * group * (dim + 2) * 4 : 0));
                                // never many parts of few keys, nor more of them than memory bears
                                CHECK(space < 1LL << 33);
                                ct::KvBatch b{};
                                b.tokens = tokens, b.sequences = sequences, b.even = tokens / sequences;
                                if (tokens % sequences == 0) {
                                    const long long t = ct::attend_tiles(p, b, group);
                                    CHECK(t * p.rows >= (long long)tokens * group && t % sequences == 0);
                                }
                                const int starts[1] = {0};
                                b.starts = starts;
                                // a whole sequence beside sequences of one token each
                                const long long t = ct::attend_tiles(p, b, group), ones = sequences - 1 < tokens ? sequences - 1 : tokens;
                                CHECK(t >= ((tokens - ones) * group + p.rows - 1) / p.rows + ones * ((group + p.rows - 1) / p.rows));
                            }
}

}  // namespace

int main() {
    refusals();
    division();
    plans();
    std::printf("attention checks: %d failed\n", g_fail);
    return g_fail != 0;
}
