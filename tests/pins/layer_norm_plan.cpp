// Layer norm's forward cuts for every width, format and place of rows.
//
// Where a call is cut for two blocks an SM, both fit there: their shared memory, static
// and dynamic, and what the device keeps for each.  All of a row's chunks belong to a
// thread, and every class of rows to a block.  Each kernel that is compiled for units of
// several warps is some width's.
#include <cstdio>
#include <initializer_list>

#include "wgs_layer_norm_plan.h"

using namespace wgs;

int main() {
    long long cuts = 0;
    bool seen[2][2][8] = {};        // [bytes][whole][chunks a thread]
    for (int bytes : {4, 2})
        for (int place = 0; place < 3; ++place)         // whole chunks; ragged, alike; ragged, apart
            for (int width = 1; width <= kMaxWidth; ++width) {
                const int v = 16 / bytes;
                if (place == 0 && width % v) continue;
                const bool whole = place == 0;
                int period = 1;
                while (place == 1 && period < v && width * period % v) period *= 2;
                const int chunks = static_cast<int>(ceil_div(width + (place == 1 ? v - 1 : 0), v));
                const Unit u = forward_unit(chunks, bytes, whole);
                if (u.team == 0) seen[bytes == 4][whole][u.each] = true;
                for (int tensors : {1, 2})
                    for (int sms : {152, 20})
                        for (int64_t rows : {1, 7, 300, 5000, 131040}) {
                            const ForwardCut f = forward_cut(u, chunks, tensors, bytes, whole, rows, period, sms);
                            const int fixed = forward_static_bytes(u.team, bytes, whole) + kBlockReserve, blocks = f.two ? 2 : 1;
                            const int lanes = u.team ? u.team : 32 * f.team_warps;
                            const bool ok = blocks * (f.smem + fixed) <= kSmBytes && f.smem <= kMostOfSm && f.stages >= 1 &&
                                            (!f.two || f.stages >= 2) && lanes * u.each >= chunks && f.cut.units >= 1 &&
                                            f.cut.threads <= 32 * forward_warps(u.each, bytes) &&
                                            f.cut.blocks >= (rows < period ? rows : period) &&
                                            (f.cut.blocks <= blocks * sms || f.cut.blocks <= period);
                            if (!ok)
                                return std::printf("[%lld, %d] of %d bytes, place %d, %d tensors, %d SMs: units of %d chunks, "
                                                   "%d lanes; %d blocks an SM of %d bytes and %d, %d stages\n",
                                                   static_cast<long long>(rows), width, bytes, place, tensors, sms, u.each,
                                                   lanes, blocks, f.smem, fixed, f.stages),
                                       1;
                            ++cuts;
                        }
            }
    for (int bytes : {4, 2})
        for (bool whole : {false, true})
            for (int each = 0; each < 8; ++each)
                if (forward_has_warps(each, bytes, whole) != seen[bytes == 4][whole][each])
                    return std::printf("%d chunks a thread of %d bytes, whole %d: compiled %d, called %d\n", each, bytes,
                                       whole, forward_has_warps(each, bytes, whole), seen[bytes == 4][whole][each]),
                           1;
    std::printf("cuts %lld\n", cuts);
    return 0;
}
