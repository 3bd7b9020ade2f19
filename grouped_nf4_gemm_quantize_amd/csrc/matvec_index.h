// Where the matrix-vector kernel reads packed codes: plain arithmetic, no device code.
#pragma once

namespace nf4moe {

constexpr int kMvChunk = 128;  // k of one read of a wave: 64 bytes of each row

// Byte of a row of `row_bytes` (a multiple of 16) at which the lanes of quarter q (0..3)
// read their 16 bytes of a chunk.  A last chunk can be cut: the quarters beyond
// the end read the row's last 16 bytes again (x is zero there).
constexpr int mv_code_byte(int chunk, int q, int row_bytes) {
  const int at = chunk * (kMvChunk / 2) + 16 * q;
  return at < row_bytes ? at : row_bytes - 16;
}

}  // namespace nf4moe
