// hs_shared.h -- per-device facts that host threads share.  The Python binding
// makes its calls without the interpreter's lock, so two threads can be in the
// launch code of one kernel at a time.  Plain C++, no CUDA.
#pragma once

#include <mutex>

namespace hs_host {

// Raises the limit in force, *known, to at least `want` by set(want), which
// returns a status (0: done).  It never lowers it: a thread that finds a larger
// one by the time that it holds the lock leaves it alone.
template <typename Set>
int raise_limit(int* known, int want, Set set) {
    if (__atomic_load_n(known, __ATOMIC_ACQUIRE) >= want) return 0;
    static std::mutex lock;
    const std::lock_guard<std::mutex> hold(lock);
    if (__atomic_load_n(known, __ATOMIC_RELAXED) >= want) return 0;
    const int rc = set(want);
    if (rc == 0) __atomic_store_n(known, want, __ATOMIC_RELEASE);
    return rc;
}

// A value that is asked for once and is the same for every thread (several may
// ask at a time); *known is 0 until it is known, and ask() never returns 0.
template <typename Ask>
int ask_once(int* known, Ask ask) {
    int n = __atomic_load_n(known, __ATOMIC_RELAXED);
    if (n == 0) {
        n = ask();
        __atomic_store_n(known, n, __ATOMIC_RELAXED);
    }
    return n;
}

}  // namespace hs_host
