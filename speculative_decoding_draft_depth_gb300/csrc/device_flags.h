// device_flags.h -- devices for which a kernel's attributes have been set (setting them
// twice does no harm, so two threads may come at once).
#pragma once

#include <stdint.h>

#include <atomic>

struct DeviceFlags {
    std::atomic<uint64_t> bits{0};
    bool test(int dev) const { return dev < 64 && ((bits.load(std::memory_order_relaxed) >> dev) & 1); }
    void set(int dev)
    {
        if (dev < 64)
            bits.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    }
};
