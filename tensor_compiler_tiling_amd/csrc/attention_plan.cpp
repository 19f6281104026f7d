// Which kernel attends, and how many workgroups share a tile's keys: host
// arithmetic on sizes alone.
#include <algorithm>

#include "attention_kernels.hpp"

namespace ct {

// The row form for up to 16 rows (a sequence's new tokens x the heads of a group), tiles
// for more.  Measured on the device, row form against tiles, us: 64 x 8192 e4m3 159 and
// 363, one of 1200 bf16 11.5 and 17.9, 100 windows of 1024 fp16 24 and 50; bf16 batches of
// unequal lengths up to 8192, 32 sequences 64 wide 87 and 144, 96 wide 135 and 182, 128
// wide 175 and 190, 64 sequences 128 wide 333 and 370, 256 wide 328 and 372.  Tiles, which
// bring 16-bit rows to LDS whole, are ahead where all lengths are equal, rows wide and
// there are many (64 x 8192 of 128 410 and 392, 8 x 8192 60.5 and 57, of 256 64 and 62,
// one of 131072 113 and 106).  The host knows lengths to be equal where there is one: tiles
// from 2^19 keys in all heads (one of 32768 on 8 heads 33.4 and 33.6, of 65536 61 and 58; 96
// wide and less the row form leads at any length, one of 32768 25 and 32).  More rows than
// 16 take tiles: 32 rows of 16 x 4096 in a row form for 32 bf16 87 and 59, e4m3 61 and 58,
// 64 rows in one for 64 156 and 64.
//
// Parts, so that all CUs have work: a workgroup a CU for the tiles, whose registers
// leave no room for two, and for the row form of heads wider than 128, else two (one
// of 131072 bf16: 512 workgroups 129 us, 768 159; two for 256 wide, 8 x 3000 e4m3 23 -> 31,
// bf16 29.5 -> 37; for 192 wide e4m3 8 x 16000 52 -> 49, but one of 32768 22 -> 23, bf16
// 8 x 3000 24 -> 30); to the next whole number below or above, since 400 tiles in two
// parts take 34 us and whole 30.  A part has 512 keys in a tile, 128 in a row form at least
// (one of 1200: parts of 256 17.7 us, of 128 16.3, of 64 19.4).
AttendPlan attend_plan(int tokens, int sequences, int heads, int group, int dim, long long max_len, int window, int sinks, bool q8) {
    const long long each = std::max(1LL, ((long long)tokens + sequences - 1) / sequences) * group;
    // keys that a token sees, at most
    const long long keys = std::min(max_len, (long long)window + sinks + 64);
    const bool one_long = !q8 && sequences == 1 && dim > 96 && keys * heads >= 1 << 19;
    const int form = each <= 16 && !one_long ? ATT_ROWS : ATT_TILE;
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
