// Host: what is looked up once and kept, but only if the lookup worked.
#pragma once
#include <atomic>

namespace gqh {

// The first value of look() that is not T{}; until there is one, look() is asked on every call.  Safe from
// several threads, which may ask at the same time.
template <typename T>
class KeepFound {
    std::atomic<T> kept_{};

public:
    template <typename Look>
    T get(Look look) {
        T v = kept_.load(std::memory_order_acquire);
        if (v == T{}) {
            v = look();
            if (v != T{}) kept_.store(v, std::memory_order_release);
        }
        return v;
    }
};

}  // namespace gqh
