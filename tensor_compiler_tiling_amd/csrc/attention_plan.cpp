// Which kernel attends, and how many workgroups share a tile's keys: host
// arithmetic on sizes alone.
#include <algorithm>

#include "attention_kernels.hpp"

namespace ct {

AttendPlan attend_plan(int tokens, int sequences, int heads, int group, int dim, long long max_len, int window, int sinks) {
    const long long each = std::max(1LL, ((long long)tokens + sequences - 1) / sequences) * group;
    AttendPlan plan{ATT_TILE, dim > 128 ? 128 : 256, 1};
    if (each <= 16) plan = {ATT_ROW16, 16, 1};
    else if (each <= 32) plan = {ATT_ROW32, 32, 1};
    else if (each <= 64 && dim <= 128) plan = {ATT_ROW64, 64, 1};
    const long long tiles = (each + plan.rows - 1) / plan.rows * sequences * heads;
    // keys that a tile's rows see, at most
    const long long span = (plan.rows + group - 1) / group;
    const long long keys = std::min(max_len, (long long)window + sinks + span + 64);
    const long long want = plan.form == ATT_TILE || dim > 128 ? 256 : 512;  // workgroups that fill the device
    const long long least = plan.form == ATT_TILE ? 512 : 128; // keys that are worth a part
    long long parts = std::min((want + tiles / 2) / tiles, (keys + least - 1) / least);
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
