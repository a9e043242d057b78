// How many CTAs or clusters of a kernel are resident at once, by device and
// cluster size: asked of the runtime once each, as the query takes longer than a
// launch. Host code without CUDA types, so that it can be tested alone.
#pragma once

#include <atomic>

namespace fl {

template <int Devices, int Sizes>
class Resident {
    std::atomic<int> kept_[Devices][Sizes + 1] = {};  // the answer plus one; 0: not known yet

  public:
    // The number for clusters of `size` on `device`. ask(&n) fetches it and returns 0,
    // or an error code, which is handed on and not kept: the next call asks again.
    template <typename Ask>
    int get(int device, int size, Ask ask, int* n) {
        std::atomic<int>& kept = kept_[device][size];
        const int known = kept.load(std::memory_order_relaxed);
        if (known > 0) {
            *n = known - 1;
            return 0;
        }
        *n = 0;
        const int e = ask(n);
        if (e == 0) kept.store(*n + 1, std::memory_order_relaxed);
        else *n = 0;
        return e;
    }
};

}  // namespace fl
