// embedding_bwd's cuts of many sizes, on devices of few and many SMs.
//
// The zeros of the table's gradient belong to blocks behind the sort's own: every byte
// to one launch, a block at least in each that has any, and never fewer blocks in a
// launch than the sort needs.
//
// Where one block may have all of a call's few indices in one row of the table, it has 1 KB
// of their columns at most, and all columns belong to a block.
#include <cstdio>
#include <initializer_list>

#include "wgs_embedding_plan.h"

using namespace wgs;

int main() {
    const int64_t indices[] = {1, 7, 180, 1024, 1025, 2049, 4096, 9000, 131040, 131072, 131073, 200000, 262144, 262145,
                               1000000, 8500000, 100000000, 2147483646};
    const int64_t rows[] = {1, 2, 24, 300, 511, 512, 32768, 262144, 1 << 28, 2147483646};
    const int widths[] = {1, 5, 64, 192, 771, 2048, 32768};
    long long plans = 0;
    for (int64_t n : indices)
        for (int64_t r : rows)
            for (int w : widths)
                for (int v : {4, 8}) {
                    const Plan z = plan_of(n, r, w, v);
                    if (z.few && (z.cols * 16 > 1024 || z.slices < 1 || static_cast<int64_t>(z.slices) * z.cols * v < w ||
                                  static_cast<int64_t>(z.slices - 1) * z.cols * v >= w))
                        return std::printf("%lld indices of width %d: %d slices of %d threads\n", static_cast<long long>(n), w,
                                           z.slices, z.cols),
                               1;
                    if (z.few || z.tile) continue;
                    for (int sms = 1; sms <= 160; ++sms) {
                        for (int64_t bytes : {r * w * 2, r * w * 4}) {
                            int64_t end = 0;
                            for (int p = -1; p < z.passes; ++p) {
                                const ZeroShare s = zero_share(z, p, bytes, sms);
                                const bool ok = s.blocks >= 0 && s.blocks < 1 << 30 && (s.bytes == 0) == (s.blocks == 0) &&
                                                (s.bytes == 0 || (s.first == end && s.first % 16 == 0 && s.bytes > 0));
                                if (!ok) {
                                    std::printf("%lld indices, %lld rows of %d, %d SMs, pass %d: %lld blocks for %lld bytes from %lld\n",
                                                static_cast<long long>(n), static_cast<long long>(r), w, sms, p,
                                                static_cast<long long>(s.blocks), static_cast<long long>(s.bytes),
                                                static_cast<long long>(s.first));
                                    return 1;
                                }
                                end += s.bytes;
                            }
                            if (end != bytes) return std::printf("%lld of %lld bytes\n", static_cast<long long>(end), static_cast<long long>(bytes)), 1;
                            ++plans;
                        }
                    }
                }
    std::printf("plans %lld\n", plans);
    return 0;
}
