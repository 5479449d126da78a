/* Walks a wave's search for the last of n places at or below a value, with a
 * place's own number (and, for runs of equal ones, its half or 1000th) as what
 * stands there, and checks that it looks at places of 1 .. n - 1 only, ends, and
 * finds the place.  Given an argument, walks the same in signed numbers that wrap,
 * which have to go wrong at the largest n. */
#include <algorithm>
#include <cstdio>

#include "echo_search.hpp"

static unsigned long long looked = 0, outside = 0, wrong = 0;

template <typename F>
static bool look(int64_t at, int64_t n, int64_t v, F f)
{
    ++looked;
    if (at < 1 || at >= n) {
        ++outside;
        return false;
    }
    return f(at) <= v;
}

template <typename F>
static int64_t search(int64_t n, int64_t v, F f)
{
    echo::WaveSearch s((uint32_t)n);
    for (int turn = 0; s.turn(); ++turn) {
        if (turn == 8) return -1;
        uint32_t below = 0;
        for (uint32_t lane = 0; lane < 64; ++lane)
            if (s.place(lane) < s.hi) below += look(s.place(lane), n, v, f);
        s.narrow(below);
    }
    return s.lo;
}

static int32_t wrap(int64_t v) { return (int32_t)(uint32_t)v; }

template <typename F>
static int64_t signed_search(int64_t n, int64_t v, F f)
{
    int32_t lo = 0, hi = (int32_t)n;
    for (int turn = 0; wrap((int64_t)hi - lo) > 1; ++turn) {
        if (turn == 8) return -1;
        const int32_t step = wrap((int64_t)hi - lo + 63) / 64;
        int32_t below = 0;
        for (int lane = 0; lane < 64; ++lane) {
            const int64_t at = lo + (int64_t)(lane + 1) * step;
            if (at < hi) below += look(at, n, v, f);
        }
        lo = wrap(lo + (int64_t)below * step);
        hi = std::min(wrap((int64_t)lo + step), hi);
    }
    return lo;
}

int main(int argc, char**)
{
    const int64_t top = (int64_t(1) << 31) - 1;
    const int64_t sizes[] = {1, 2, 3, 63, 64, 65, 66, 127, 128, 129, 4095, 4096, 4097, 4161, 262144, 262145, 1 << 24, (1 << 30) - 1,
                             1 << 30, top - (1 << 25), top - 64, top - 63, top - 62, top - 1, top};
    for (int64_t n : sizes)
        for (int64_t run : {int64_t(1), int64_t(2), int64_t(1000)}) {
            auto f = [&](int64_t i) { return i / run; };
            for (int64_t p : {int64_t(0), int64_t(1), int64_t(62), int64_t(63), int64_t(64), n / 64, n / 64 + 1, n / 3, n / 2, n - 66, n - 65, n - 64,
                              n - 2, n - 1, n, n + 1000}) {
                if (p < 0) continue;
                const int64_t v = p / run, want = std::min(n - 1, v * run + run - 1);
                wrong += (argc > 1 ? signed_search(n, v, f) : search(n, v, f)) != want;
            }
            wrong += (argc > 1 ? signed_search(n, -1, f) : search(n, -1, f)) != 0;
        }
    std::printf("looked=%llu outside=%llu wrong=%llu\n", looked, outside, wrong);
    return outside || wrong;
}
