// linear_plan.h -- the FP8 product's arithmetic on sizes that needs no GPU: plain
// C++, shared by the kernels and by checks on the CPU.
#pragma once

namespace dsa {
namespace lin {

// Bytes that exist of a row of out (N values of `size` bytes) from feature n on, at
// most `most` of them; 0 or less where n is not a feature.  N may be near 2^30: the
// features left are cut before they become bytes, whose number may pass 32 bits.
constexpr int row_bytes_left(int N, int n, int size, int most) {
  const int left = N - n, fit = most / size;
  return (left < fit ? left : fit) * size;
}

}  // namespace lin
}  // namespace dsa
