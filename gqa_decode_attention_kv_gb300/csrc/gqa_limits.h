// gqa_limits.h -- what the runtime was told and asked about kernels, remembered: the
// dynamic shared-memory limit set for each, and the CTAs of it that an SM holds. Host
// code without CUDA headers; the callers give the two runtime calls and hold a lock. Both
// methods are reached from C entry points: no exception leaves them.
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
    // may be about to launch at the size it asked for before. Every kernel keeps an entry,
    // made before the call: a limit that could not be remembered is not set.
    template <class Set>
    bool raise(int device, const void* fn, int smem, Set&& set) noexcept {
        try {
            int& now = limit_.try_emplace(std::make_pair(device, fn), -1).first->second;
            if (now >= smem) return true;
            if (!set(smem)) return false;
            now = smem;
            return true;
        } catch (...) {
            return false;
        }
    }

    // CTAs per SM at (threads, smem), ask() the first time (0 or less: no answer, not kept).
    template <class Ask>
    int ctas(int device, const void* fn, int threads, int smem, Ask&& ask) noexcept {
        const auto key = std::make_tuple(device, fn, threads, smem);
        const auto it = ctas_.find(key);
        if (it != ctas_.end()) return it->second;
        const int n = ask();
        if (n <= 0) return n;
        if (ctas_.size() >= kMostAnswers) ctas_.clear();      // sizes go by batch: some hundred entries each
        try {
            ctas_.try_emplace(key, n);
        } catch (...) {                                       // asked for again the next time
        }
        return n;
    }

  private:
    static constexpr std::size_t kMostAnswers = 1 << 16;
    std::map<std::pair<int, const void*>, int> limit_;
    std::map<std::tuple<int, const void*, int, int>, int> ctas_;
};

}  // namespace gqa
