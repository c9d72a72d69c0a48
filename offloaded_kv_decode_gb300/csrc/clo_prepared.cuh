// clo_prepared.cuh -- which kernels have had their launch attributes set: a hash
// table of (kernel, context) with the dynamic shared memory that was asked for.
// Host code without allocations; the caller holds a lock.
#pragma once

#include <stdint.h>

namespace clo {

class PreparedKernels {
public:
    // True if `func` was prepared in the context for at least `smem` bytes.
    bool has(const void* func, unsigned long long ctx, int smem) const {
        const Entry& e = entries_[find(func, ctx)];
        return e.func == func && e.smem >= smem;
    }
    void add(const void* func, unsigned long long ctx, int smem) {
        int at = find(func, ctx);
        if (entries_[at].func == nullptr && ++used_ > MOST) {
            // Many contexts came and went: all are prepared again.
            for (Entry& e : entries_) e = Entry{};
            used_ = 1;
            at = find(func, ctx);
        }
        entries_[at] = Entry{func, ctx, smem};
    }

private:
    // The library has about 100 kernels.
    static constexpr int SLOTS = 1024, MOST = SLOTS / 2;
    struct Entry {
        const void* func = nullptr;
        unsigned long long ctx = 0;
        int smem = 0;
    };
    // Its slot, or the free one that it would get.
    int find(const void* func, unsigned long long ctx) const {
        const uint64_t key = (reinterpret_cast<uintptr_t>(func) >> 4) + ctx * 0x9E3779B97F4A7C15ull;
        unsigned at = static_cast<unsigned>((key * 0x9E3779B97F4A7C15ull) >> 54);  // the top 10 bits
        while (entries_[at].func != nullptr && (entries_[at].func != func || entries_[at].ctx != ctx))
            at = (at + 1) % SLOTS;
        return static_cast<int>(at);
    }
    Entry entries_[SLOTS];
    int used_ = 0;
};

}  // namespace clo
