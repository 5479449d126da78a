// echo_search.hpp — where a wave looks for the last of n places at or below a
// value, 64 places at a time.  Plain arithmetic without HIP, so that a host
// test can walk it.
#pragma once

#include <cstdint>

#include "echo_stage.hpp"

namespace echo {

// The place is in lo .. hi - 1.  A turn looks at lo + step, lo + 2 step, ...,
// one a lane, as far as they are below hi, and counts those at or below the
// value.  Unsigned: for n up to 2^31 - 1 the last lane's place is up to
// hi + 62 and a run's end up to 2^25 behind hi, past a signed number's range.
struct WaveSearch {
    uint32_t lo, hi, step;
    ECHO_HD explicit WaveSearch(uint32_t n) : lo(0), hi(n), step(0) {}
    ECHO_HD bool turn()                          // whether there is more to look at; sets the step
    {
        if (hi <= lo + 1) return false;
        step = (hi - lo + 63) / 64;
        return true;
    }
    ECHO_HD uint32_t place(uint32_t lane) const { return lo + (lane + 1) * step; }
    ECHO_HD void narrow(uint32_t below)          // places of the turn that are at or below the value
    {
        lo += below * step;
        hi = lo + step < hi ? lo + step : hi;
    }
};

}  // namespace echo
