// Host threads that share a PerDevice table, run under the thread sanitizer:
// every thread sees the whole value or fills it, one fill succeeds per device,
// and a failed fill is tried again.
#include <cstdio>
#include <thread>
#include <vector>

#include "per_device.h"

struct Table {
    int a[3];
};

int main()
{
    static razer::PerDevice<Table> table;
    std::atomic<int> fills{0}, wrong{0};
    for (int dev = 0; dev < 66; dev++) {  // 64 and 65: beyond the table, filled by every call
        std::atomic<bool> go{false};
        std::vector<std::thread> threads;
        for (int t = 0; t < 8; t++)
            threads.emplace_back([&, dev] {
                while (!go.load()) {
                }
                Table v = {};
                const bool ok = table.get(dev, v, [&](Table &w) {
                    if (fills.fetch_add(1) == 0) return false;  // the very first one cannot tell
                    for (int i = 0; i < 3; i++) w.a[i] = 10 * dev + i + 1;
                    return true;
                });
                if (!ok) return;
                for (int i = 0; i < 3; i++)
                    if (v.a[i] != 10 * dev + i + 1) wrong++;
            });
        go = true;
        for (auto &t : threads) t.join();
    }
    const int want = 1 + 64 + 2 * 8;
    if (fills != want || wrong != 0) {
        std::printf("%d fills (%d expected), %d values torn\n", fills.load(), want, wrong.load());
        return 1;
    }
    std::printf("all checks passed\n");
    return 0;
}
