// fp4q_tma.h -- tensor maps of byte matrices (host side).
#pragma once

#include <cstdint>
#include <cuda.h>

namespace fp4q {

// Tensor map of a [rows][row_bytes] byte matrix (row_bytes a multiple of 16,
// base 16-byte aligned) in boxes of box_rows x 128 bytes with the 128-byte
// swizzle: one swizzle row per matrix row, the layout a K-major operand of
// tcgen05.mma has in shared memory.  False if the driver refuses it.
bool make_byte_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t row_bytes, int box_rows);

}  // namespace fp4q
