// linear_plan.h -- the FP8 product's arithmetic on sizes that needs no GPU: plain
// C++, shared by the kernels and by checks on the CPU.
#pragma once
#include <cstdint>

namespace dsa {
namespace lin {

// Bytes that exist of a row of out (N values of `size` bytes) from feature n on, at
// most `most` of them; 0 or less where n is not a feature.  N may be near 2^30: the
// features left are cut before they become bytes, whose number may pass 32 bits.
constexpr int row_bytes_left(int N, int n, int size, int most) {
  const int left = N - n, fit = most / size;
  return (left < fit ? left : fit) * size;
}

// The split kernel's tiles and their numbers of K slices (above 8 only where a GPC
// holds such a cluster without needing 16 free SMs).
constexpr struct {
  int nt, ctas;      // the tile's tokens, its CTAs per SM
  double block[3];   // time per block of K with 1, 2, 3 CTAs on the SM
} kTile[] = {{16, 3, {0.152, 0.275, 0.364}}, {32, 2, {0.19, 0.293}}, {64, 2, {0.273, 0.366}},
             {96, 1, {0.284}}, {128, 1, {0.33}}};
constexpr struct {
  int S;
  double reach;      // the part of the SMs that clusters of S fill
} kSlices[] = {{1, 1.0}, {2, 1.0}, {3, 0.91}, {4, 0.95}, {5, 0.92}, {6, 0.91}, {8, 0.79},
               {12, 0.7}, {16, 0.7}};
constexpr int kPortable = 8, kLargest = 16;   // CTAs of a cluster: on any GPU, on this one
inline int most_slices(int ctas, int kb, int cluster = kLargest) {
  const int most = ctas == 1 ? kPortable : cluster;
  return most < kb ? most : kb;
}
inline int64_t split_tiles(int M, int N, int nt) {
  return static_cast<int64_t>((N + 127) / 128) * ((M + nt - 1) / nt);
}

// Which kernel, tile and number of K slices: the cheapest by an estimate of the
// time in microseconds, whose terms were fitted to the measured time of every
// combination at 220 sizes (1 to 4,096 tokens, 64 to 8,192 features, K 256 to
// 12,288): the choice is on average 0.7 % slower than the fastest combination,
// at most 17 % (0.4 us at 4 x 64 x 512); at 70 other sizes (up to 16,384 tokens) 2 %
// and 19 % (1.7 us at 7 x 6,432 x 7,792).  There is no term for the memory's rate:
// 64 x 55,296 x 7,168 is put at 48 us and takes 67, by the best kernel all the same.
// The terms: a CTA's time per block of K,
// by how many CTAs share its SM (its bytes at an SM's share of L2 bandwidth, 59 a
// cycle, or the epilogue's latency); a start; the join of K slices, a cluster
// barrier and the partial tiles' way through distributed shared memory (about 12
// bytes a cycle at 1.9 GHz); the part of the SMs that clusters of a size can fill; the wide
// kernel's way of storing rows that TMA cannot.  Examples (us; tokens x features
// x K): 1 x 8,192 x 7,168: 16 tokens and 4 slices 11.6, unsliced 17; and with the
// operands in L2, 64 x 128 x 7,168: 16 tokens and 16 slices 3.7, 64 tokens and 8
// slices 5.3; 777 x 1,001 x 1,040: 64 tokens unsliced 5.1, with 2 slices 8; 2,048 x
// 576 x 7,168: 96 tokens 15.4, 128 tokens 18, wide 25; 512 x 7,168 x 12,288: wide 42,
// 128 tokens 60.
struct Pick {
  int nt, S;   // nt = 0: the pair kernel
};
// cluster: the most CTAs that a cluster may have.
inline Pick pick(int M, int N, int kb, int sms, int64_t row_bytes, int cluster = kLargest) {
  const int64_t pairs = sms / 2;
  const int64_t wt = static_cast<int64_t>((M + 255) / 256) * ((N + 255) / 256);
  const double rows = row_bytes % 4 != 0 ? 8.3 : row_bytes % 16 != 0 ? 1.3 : 0.0;
  double best = 1.98 + static_cast<double>((wt + pairs - 1) / pairs) * (kb * 0.40 + 1.79 + rows);
  Pick at{0, 1};
  for (const auto& t : kTile) {
    const int64_t tiles = split_tiles(M, N, t.nt);
    for (const auto& s : kSlices) {
      if (s.S > most_slices(t.ctas, kb, cluster)) break;
      const int64_t n = tiles * s.S, reach = static_cast<int64_t>(sms * s.reach),
                    slots = static_cast<int64_t>(sms * t.ctas * s.reach);
      const double rounds = n <= slots ? 1.0 : static_cast<double>((n + slots - 1) / slots);
      const int on = n <= reach ? 1 : n <= 2 * reach ? (t.ctas < 2 ? 1 : 2) : t.ctas;
      const double join = s.S > 1 ? 0.49 + on * t.nt * 512 / 21.9e3 : on * t.nt * 0.0021;
      const double us = rounds * (3.17 + (kb + s.S - 1) / s.S * t.block[on - 1] + join);
      if (us < best) {
        best = us;
        at = Pick{t.nt, s.S};
      }
    }
  }
  return at;
}

// Takes the choice, where clusters of more than kPortable CTAs may not fit: a process
// that has a part of the SMs only (a partition's, a shared server's) may have no GPC with
// so many.  take(at) is false where the cluster does not fit.
template <typename Take>
void take_one_that_fits(int M, int N, int kb, int sms, int64_t row_bytes, Take take) {
  const Pick at = pick(M, N, kb, sms, row_bytes);
  if (!take(at) && at.S > kPortable) take(pick(M, N, kb, sms, row_bytes, kPortable));
}

// Whether a kernel can be asked for by its tile and slices at these sizes (a grid
// has fewer than 2^31 CTAs; what pick() takes never comes near).
inline bool offered(const Pick& at, int M, int N, int kb) {
  if (at.nt == 0) return at.S == 1;
  for (const auto& t : kTile)
    if (t.nt == at.nt)
      for (const auto& s : kSlices)
        if (s.S == at.S)
          return s.S <= most_slices(t.ctas, kb) &&
                 split_tiles(M, N, t.nt) * s.S < (int64_t(1) << 31);
  return false;
}

}  // namespace lin
}  // namespace dsa
