// mx_stage.h -- which 16-byte piece of a row each thread of the MX tile
// kernel requests, and where it lies in the operand's buffer.
//
// A stage brings RB bytes of every row of a tile to LDS.  Thread `tid` of TH
// requests, in round k, LDS slot tid % (RB / 16) of row tid / (RB / 16) +
// k * (rows a round); the slot's piece is the slot's number XOR the row's
// swizzle.  Each round has a buffer of its own, the round's valid rows one
// after another, so a row past the last lies past the buffer's end, and the
// lane's offset, which the range check compares with the buffer's size, is
// the whole offset.  (A uniform offset beside it is documented as taken off
// the size first, below zero where a tile has few valid rows, or as left out
// of the check.)
// Plain constant expressions: the same code on the device and on the host.
#pragma once
#include <stdint.h>

namespace oq {

// beyond every buffer (256 rows of 16 KB)
constexpr uint32_t kMxOutside = 0x7ffffff0u;

// XOR swizzle of a row's 16-byte pieces in LDS (rows lie one after another).
// A 16-byte LDS read serves lanes {0-3, 12-15, 20-23, 24-27} of 32 together,
// then the others: of those, rows equal modulo 256 bytes differ in these bits.
template <int RB>
constexpr int mx_swizzle(int row) {
  return RB == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
}

template <int RB, int TH>
struct MxPieces {
  static constexpr int C = RB / 16;    // pieces of a row in a stage
  static constexpr int ROWS = TH / C;  // rows a round
  static constexpr int row(int tid) { return tid / C; }
  static constexpr int byte(int tid) { return 16 * ((tid % C) ^ mx_swizzle<RB>(row(tid))); }
  // bytes from the tile's first row to the buffer of round k, and its size
  static constexpr int base(int row_bytes, int k) { return k * ROWS * row_bytes; }
  static constexpr int size(int valid_rows, int row_bytes, int k) {
    return valid_rows > k * ROWS ? (valid_rows - k * ROWS) * row_bytes : 0;
  }
  // offset of the thread's piece of stage t in it; at = row(tid) * row_bytes + byte(tid)
  static constexpr uint32_t offset(uint32_t at, int byte, int row_bytes, int t) {
    return byte < row_bytes - t * RB ? at + (uint32_t)(t * RB) : kMxOutside;
  }
};

}  // namespace oq
