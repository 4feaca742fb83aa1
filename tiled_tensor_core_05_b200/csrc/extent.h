// Sizes of operands in bytes and whether they lie in an allocation: host
// arithmetic that holds for every size and stride an entry point is given
// (rows below 2^31 that are up to 2^40 bytes apart pass 2^64).
#pragma once

#include <stdint.h>

namespace ttc {

// Bytes from the first to the last unit of `rows` rows (at least 1) of `used`
// units, `ld` units of `unit` bytes apart; UINT64_MAX, which no allocation
// holds, if there are more than 64 bits can count.
inline uint64_t matrix_span(int64_t rows, int64_t used, int64_t ld, int64_t unit) {
  const unsigned __int128 units =
      static_cast<unsigned __int128>(static_cast<uint64_t>(rows - 1)) *
          static_cast<uint64_t>(ld) + static_cast<uint64_t>(used);
  // (rows, ld and used are below 2^63: units is below 2^127)
  const unsigned __int128 limit = UINT64_MAX / static_cast<uint64_t>(unit);
  return units > limit ? UINT64_MAX : static_cast<uint64_t>(units) * static_cast<uint64_t>(unit);
}

// The bytes [start, start + span) lie in the allocation [base, base + size).
inline bool span_inside(uint64_t start, uint64_t span, uint64_t base, uint64_t size) {
  return start >= base && start - base <= size && span <= size - (start - base);
}

}  // namespace ttc
