// arnq_matmul_shape.h -- the split kernel's shared memory and TMEM by its tile
// (plain C++, no CUDA).
#pragma once

namespace arnq {

constexpr int kTmemColumns = 512;          // of an SM
constexpr int kSmemPerSm = 228 * 1024;     // of which a CTA takes 1 KB besides its own
constexpr int kSmemLimit = 227 * 1024;     // of a CTA

// Every CTA takes at least this much shared memory for each of its TMEM
// columns, so that CTAs which fit an SM together by shared memory fit it by
// TMEM too, whichever kernel of this library and stream they come from, and no
// tcgen05.alloc waits for another CTA's columns.  (Columns are handed out in
// multiples of 32: more than 512 are at least 544.)  Two CTAs of 256 columns,
// or four of 128, still fit.
constexpr int kSmemPerColumn = 430;
static_assert((kTmemColumns + 32) * kSmemPerColumn > kSmemPerSm, "");

// TMEM columns of a tile of `tokens`: a power of two, 32 at least.
inline int split_columns(int tokens) {
  int columns = 32;
  while (columns < tokens) columns *= 2;
  return columns;
}

// Bytes of dynamic shared memory: the stages (128 channels and the tokens, by
// 128 codes), over which the partial sums (128 channels by the tokens) lie
// later, and 1 KB to align them.
inline int split_smem(int tokens, int stages) {
  int bytes = stages * (16384 + tokens * 128);
  if (bytes < tokens * 512) bytes = tokens * 512;
  bytes += 1024;
  const int least = split_columns(tokens) * kSmemPerColumn;
  return bytes < least ? least : bytes;
}

}  // namespace arnq
