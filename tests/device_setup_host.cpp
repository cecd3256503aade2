// First calls of many threads at once through DeviceSetup (csrc/bsa_device_setup.h),
// built by test_device_setup_host.py with the thread sanitizer where there is one.
#include <stdio.h>

#include <atomic>
#include <chrono>
#include <thread>
#include <vector>

#include "bsa_device_setup.h"

static bsa::DeviceSetup setup;
static int value[bsa::kMaxDevices];  // plain, as a launch's number of SMs
static int runs[bsa::kMaxDevices];

static bool use(int dev, bool fail) {
    return setup.once(dev, [&] {
        ++runs[dev];
        if (fail) return false;
        std::this_thread::sleep_for(std::chrono::milliseconds(20));
        value[dev] = 100 + dev;
        return true;
    });
}

int main() {
    if (use(5, true) || use(5, true) || runs[5] != 2) return printf("a failed set-up counts as done\n"), 1;
    for (int dev : {-1, bsa::kMaxDevices})
        if (use(dev, true)) return printf("device %d taken\n", dev), 1;
    std::atomic<int> waiting{0}, wrong{0};
    std::vector<std::thread> threads;
    const int n = 16;
    for (int i = 0; i < n; ++i)
        threads.emplace_back([&, i] {
            ++waiting;
            while (waiting < n) std::this_thread::yield();
            for (int k = 0; k < 3; ++k)
                for (int dev : {i % 2, 5, 63})
                    if (!use(dev, false) || value[dev] != 100 + dev) ++wrong;
        });
    for (auto& t : threads) t.join();
    if (wrong) return printf("%d calls went on before the set-up was done\n", wrong.load()), 1;
    if (runs[0] != 1 || runs[1] != 1 || runs[5] != 3 || runs[63] != 1) return printf("set up more than once\n"), 1;
    printf("ok\n");
    return 0;
}
