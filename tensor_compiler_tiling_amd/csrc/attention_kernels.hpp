// Host-visible declarations of the key-value cache's kernels (kv_rows.hip) and
// of attention over it (attention.hip, its plan attention_plan.cpp).
// Arguments are checked by the C entry points (attention_api.cpp) before they
// get here.
#pragma once

#include <hip/hip_runtime.h>

namespace ct {

// The pages of a cache, as one kv head's rows of k and v: strides in bytes,
// those of the scales in floats.
struct KvPages {
    char* k;
    char* v;
    float* ks;  // 8-bit caches only
    float* vs;
    long long ld_page, ld_head, ld_token;
    long long lds_page, lds_head, lds_token;
    int pages, heads, page, dim;
    // place / page = (place * magic) >> shift for 0 <= place < 2^31
    unsigned magic;
    int shift;
};

// magic = ceil(2^shift / page), shift = 31 + ceil(log2 page): the excess of
// magic * page over 2^shift is below page <= 2^(shift - 31), so that it stays
// below a whole quotient for every place below 2^31.
inline void page_magic(KvPages& c) {
    c.shift = 31;
    while ((1LL << (c.shift - 31)) < c.page) ++c.shift;
    c.magic = (unsigned)(((1ULL << c.shift) + c.page - 1) / c.page);
}

// Whose tokens they are, and in which pages.
struct KvBatch {
    const int* lens;
    const int* starts;  // or null: `even` tokens a sequence
    const int* table;   // or null: sequence b has page b
    long long ldt;
    int width;
    int tokens, sequences, even;
};

// ------------------------------------------------------------- kv rows ----
struct KvRowsParams {
    KvPages c;
    KvBatch b;
    char* k;  // [tokens][heads][dim] of dt: read when writing the cache
    char* v;
    long long k_token, k_head, v_token, v_head;  // bytes
};

hipError_t launch_kv_write(const KvRowsParams& p, int cache_dt, int dt, hipStream_t stream);
hipError_t launch_kv_read(const KvRowsParams& p, int cache_dt, int dt, hipStream_t stream);

// ----------------------------------------------------------- attention ----
struct AttendParams {
    KvPages c;
    KvBatch b;
    const char* q;  // [tokens][heads * group][dim] of the kernel's type
    char* y;
    long long q_token, q_head, y_token, y_head;  // bytes
    const long long* tree;                       // [tokens][words] or null
    int words;
    int group;
    int window;  // kNoWindow without one
    int sinks;
    float scale;     // of q . k, times log2 e
    int tiles;       // tiles of rows in the launch (an upper bound where starts are given)
    int parts;       // workgroups that share a tile's keys
    float* part_o;   // parts > 1: [parts][tokens][heads * group][dim] sums,
    float* part_ml;  // and their maximum and weight, [..][2]
};

constexpr int kNoWindow = 1 << 30;  // past every distance

// The kernel that attends.
enum AttendForm {
    ATT_ROWS = 0,  // up to 16 rows (tokens x heads of a group) a tile, a wave's keys its own
    ATT_TILE = 1,  // 32 rows a wave, the workgroup's keys shared through LDS
};

struct AttendPlan {
    int form;
    int rows;   // rows of a tile
    int parts;
};

// Rows of a form's tile.
inline int attend_rows(int form, int dim) {
    return form == ATT_ROWS ? 16 : dim > 128 ? 128 : 256;
}

AttendPlan attend_plan(int tokens, int sequences, int heads, int group, int dim, long long max_len, int window, int sinks, bool q8);
// Tiles of rows to launch.
long long attend_tiles(const AttendPlan& plan, const KvBatch& b, int group);
long long attend_workspace_bytes(const AttendPlan& plan, int tokens, int heads, int dim);

hipError_t launch_attend(const AttendPlan& plan, const AttendParams& p, int cache_dt, int dt, hipStream_t stream);

}  // namespace ct
