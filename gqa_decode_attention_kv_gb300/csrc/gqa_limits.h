// gqa_limits.h -- what the runtime was told and asked about kernels, remembered: the
// dynamic shared-memory limit set for each, and the CTAs of it that an SM holds. Host
// code without CUDA headers; the callers give the two runtime calls and hold a lock.
#pragma once

#include <algorithm>
#include <cstddef>
#include <map>
#include <tuple>
#include <utility>

namespace gqa {

class KernelLimits {
  public:
    // Sets fn's limit on the device to at least smem; set(smem) makes the runtime call.
    // A limit only grows: one set for a size serves every smaller one, and another thread
    // may be about to launch at the size it asked for before. Every kernel keeps an entry.
    template <class Set>
    bool raise(int device, const void* fn, int smem, Set&& set) {
        const auto key = std::make_pair(device, fn);
        const auto it = limit_.find(key);
        if (it != limit_.end() && it->second >= smem) return true;
        if (!set(smem)) return false;
        limit_[key] = smem;
        return true;
    }

    // CTAs per SM at (threads, smem), ask() the first time (0 or less: no answer, not kept).
    template <class Ask>
    int ctas(int device, const void* fn, int threads, int smem, Ask&& ask) {
        const auto key = std::make_tuple(device, fn, threads, smem);
        const auto it = ctas_.find(key);
        if (it != ctas_.end()) return it->second;
        const int n = ask();
        if (n <= 0) return n;
        if (ctas_.size() >= kMostAnswers) ctas_.clear();      // sizes go by batch: some hundred entries each
        ctas_[key] = n;
        return n;
    }

  private:
    static constexpr std::size_t kMostAnswers = 1 << 16;
    std::map<std::pair<int, const void*>, int> limit_;
    std::map<std::tuple<int, const void*, int, int>, int> ctas_;
};

}  // namespace gqa
