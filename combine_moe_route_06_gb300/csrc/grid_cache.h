// grid_cache.h -- what resident_grid has found out: a table of fixed size, filled
// once per key and never emptied (host code only, one lock around it).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

// A kernel at one block size and dynamic shared memory on one device.  Kernels whose
// shared memory follows the shape have a key per shape, so the table is far larger
// than the number of kernels.
struct GridKey {
    const void *kernel;
    int dev, threads;
    size_t smem;
    bool operator==(const GridKey &o) const
    {
        return kernel == o.kernel && dev == o.dev && threads == o.threads && smem == o.smem;
    }
};

class GridCache {
public:
    static constexpr int kSlots = 4096;              // a power of two
    static constexpr int kMost = kSlots / 4 * 3;     // keys held: a search ends at a free slot

    // The value of `key`, or -1.
    int find(const GridKey &key) const
    {
        for (unsigned i = slot(key); vals_[i]; i = (i + 1) % kSlots)
            if (keys_[i] == key) return vals_[i];
        return -1;
    }
    // Adds a key that find() does not know, with a value > 0, while there is room.
    void add(const GridKey &key, int value)
    {
        if (used_ == kMost || value <= 0) return;
        unsigned i = slot(key);
        while (vals_[i]) i = (i + 1) % kSlots;
        keys_[i] = key;
        vals_[i] = value;
        used_++;
    }

private:
    static unsigned slot(const GridKey &key)
    {
        uint64_t h = (uint64_t)(uintptr_t)key.kernel;
        h = (h ^ (h >> 29)) * 0x9e3779b97f4a7c15ull;
        h = (h ^ key.smem) * 0x9e3779b97f4a7c15ull;
        h = (h ^ ((uint64_t)key.dev << 32 | (uint32_t)key.threads)) * 0x9e3779b97f4a7c15ull;
        return (unsigned)(h >> 40) % kSlots;
    }

    GridKey keys_[kSlots] = {};
    int vals_[kSlots] = {};       // 0: a free slot
    int used_ = 0;
};

}  // namespace moe
