// echo_stage.hpp — where the loads of a stage of K lie in an operand's panel.
// Plain arithmetic without HIP, so that a host test can walk all of it.
#pragma once

#include <cstdint>

#if defined(__HIPCC__)
#define ECHO_HD __host__ __device__ __forceinline__
#else
#define ECHO_HD inline
#endif

namespace echo {

// 16-byte chunk c of stage row r lies at chunk c ^ key(r): the rows of a
// fragment (one row per lane, 128 bytes apart) then start on distinct banks
ECHO_HD uint32_t i8_key(uint32_t r) { return (r & 7u) ^ ((r >> 3) & 1u); }

// Byte offset of 16-byte chunk `chunk` of row `row` in a panel of `rows` rows.
// A row past the last one repeats it (its sums are not stored), so that every
// load lies inside the panel by itself: a buffer load's range check subtracts
// the scalar offset from the record count, and what it does where the scalar
// offset alone (a later load's first row) is past the count is not documented.
ECHO_HD uint32_t stage_offset(uint32_t row, uint32_t rows, uint32_t ld, uint32_t chunk)
{
    return (row < rows ? row : rows - 1) * ld + 16 * chunk;
}

}  // namespace echo
