// Which kernel attends, and how many workgroups share a tile's keys: host
// arithmetic on sizes alone.
#include <algorithm>

#include "attention_kernels.hpp"

namespace ct {

// The row form for up to 16 rows (a sequence's new tokens x the heads of a group)
// over an 8-bit cache, or over fewer than 4096 keys.  Measured on the device, row
// form against tiles, us: 64 x 8192 e4m3 159 and 363, one of 131072 e4m3 64 and 100,
// of 1200 bf16 12.7 and 17.9, 100 windows of 1024 fp16 30 and 50; but 16-bit rows
// of long caches, which the tiles bring to LDS in whole rows, one of 131072 115
// and 105, 16 x 4096 x 32 heads 209 and 197, 4 x 4096 25 and 21, 8 x 8192 of 256 wide 81
// and 60.  More rows than 16 take tiles: 32 rows of 16 x 4096 in a row form for 32
// bf16 87 and 59, e4m3 61 and 58, 64 rows in one for 64 156 and 64.
//
// Parts, so that all CUs have work: a workgroup a CU for the tiles, whose registers
// leave no room for two, and for the row form of wide heads, else two (one of
// 131072 bf16: 512 workgroups 129 us, 768 159); to the next whole number below or
// above, since 400 tiles in two parts take 34 us and whole 30.  A part has 512 keys
// in a tile, 128 in a row form at least (one of 1200: parts of 256 17.7 us, of 128
// 16.3, of 64 19.4).
AttendPlan attend_plan(int tokens, int sequences, int heads, int group, int dim, long long max_len, int window, int sinks, bool q8) {
    const long long each = std::max(1LL, ((long long)tokens + sequences - 1) / sequences) * group;
    // keys that a token sees, at most
    const long long keys = std::min(max_len, (long long)window + sinks + 64);
    const int form = each <= 16 && (q8 || keys < 4096) ? ATT_ROWS : ATT_TILE;
    AttendPlan plan{form, attend_rows(form, dim), 1};
    const long long tiles = (each + plan.rows - 1) / plan.rows * sequences * heads;
    const long long want = form == ATT_TILE || dim > 128 ? 256 : 512;
    const long long least = form == ATT_TILE ? 512 : 128;
    const long long parts = std::min((want + tiles / 2) / tiles, (keys + least - 1) / least);
    plan.parts = (int)std::max(1LL, std::min(parts, 128LL));
    return plan;
}

long long attend_tiles(const AttendPlan& plan, const KvBatch& b, int group) {
    if (!b.starts) return ((long long)b.even * group + plan.rows - 1) / plan.rows * b.sequences;
    return (long long)b.tokens * group / plan.rows + b.sequences;
}

long long attend_workspace_bytes(const AttendPlan& plan, int tokens, int heads, int dim) {
    return plan.parts > 1 ? (long long)plan.parts * tokens * heads * (dim + 2) * 4 : 0;
}

}  // namespace ct
