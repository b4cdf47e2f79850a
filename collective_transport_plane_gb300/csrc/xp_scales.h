// Scale bytes of a matrix in 8 bits, four blocks at a time (host and device).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define XP_BOTH __host__ __device__ __forceinline__
#else
#define XP_BOTH inline
#endif

namespace xp {

// The bytes of blocks 4 group .. 4 group + 3 of a row's `blocks`, the first lowest.
// Rows begin at multiples of 4 bytes, so behind a row's last byte a word has what
// lies between rows; behind the last row, which may end with its buffer, it has
// zeros and nothing is read.  (Every row by bytes: 300 x 300 x 300 7.0 us where it
// took 6.0 so; loads that conditions leave out in place of the branch: 762 x 2152 x
// 15524 44 us, 27 so.)
XP_BOTH unsigned scale_word(const uint8_t* row, unsigned group, unsigned blocks, bool last_row) {
  const unsigned left = blocks - 4 * group;
  row += 4ull * group;
  if (left >= 4 || !last_row) return *reinterpret_cast<const unsigned*>(row);
  const unsigned low = left > 1 ? *reinterpret_cast<const uint16_t*>(row) : row[0];
  return left > 2 ? low | (unsigned)row[2] << 16 : low;
}

}  // namespace xp
