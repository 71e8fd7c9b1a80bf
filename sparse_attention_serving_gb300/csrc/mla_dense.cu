// mla_dense.cu -- dense attention over latent rows: a tree of drafted tokens over
// a cache, and a sliding window with first tokens that stay visible.
//
//   z_s = scale * q_lat[t,h,:] . KV[s,:]  over the rows s that query t sees,
//   o = sum_s softmax(z)_s KV[s, 0:512],   lse = log sum_s exp(z_s)
//
// One warp per (query, head): each lane holds dims 64c + 2 lane (+1) of the query,
// the running maximum and sum of the softmax go along with the rows.
#include <cmath>

#include <cuda_bf16.h>

#include "dense_mask.cuh"
#include "sm103.cuh"

namespace dsa {
namespace dense {

constexpr int WARPS = 8;

struct Params {
  const uint16_t* q;
  Store kv;
  Mask m;
  int B, H;
  float scale_log2;
  uint16_t* o;
  float* lse;
  uint32_t* status;
};

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(WARPS * 32) rows_kernel(const Params p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(p.B) * p.m.T * p.H) return;
  const int64_t qi = row / p.H;
  const int b = static_cast<int>(qi / p.m.T), i = static_cast<int>(qi % p.m.T);
  const Seq s = seq_of(p.m, b);
  if (row % (static_cast<int64_t>(p.m.T) * p.H) == 0 && lane == 0) report_seq(p.m, s, b, p.status);
  if (i >= s.n) return;
  const uint64_t bits = p.m.tree != nullptr ? __ldg(p.m.tree + qi) : 0;
  float q[18], acc[16];
  const uint32_t* qr = reinterpret_cast<const uint32_t*>(p.q + row * kRlat) + lane;
#pragma unroll
  for (int c = 0; c < 9; ++c) {
    const uint32_t v = __ldg(qr + 32 * c);
    q[2 * c] = lo_f(v), q[2 * c + 1] = hi_f(v);
  }
#pragma unroll
  for (int d = 0; d < 16; ++d) acc[d] = 0.f;
  float top = -INFINITY, sum = 0.f;
  const Pages pages = pages_of(p.m, s, i, i);
  for (int k = 0; k < pages.count(); ++k) {
    const int pg = pages.page(k);
    uint64_t see = row_mask(p.m, s, i, bits, pg * 64);
    if (see == 0) continue;
    const int64_t r0 = page_row(p.kv, b, pg);
    if (r0 < 0) {
      if (lane == 0) status_raise(p.status, DSA_ERR_BAD_INDEX, SITE_PAGE, static_cast<uint32_t>(pg));
      continue;
    }
    for (; see != 0; see &= see - 1) {
      const int64_t r = r0 + __ffsll(static_cast<long long>(see)) - 1;
      const uint32_t* kr = reinterpret_cast<const uint32_t*>(p.kv.base + r * kRlat) + lane;
      float x[18], z = 0.f;
#pragma unroll
      for (int c = 0; c < 9; ++c) {
        const uint32_t v = __ldg(kr + 32 * c);
        x[2 * c] = lo_f(v), x[2 * c + 1] = hi_f(v);
        z = fmaf(q[2 * c], x[2 * c], fmaf(q[2 * c + 1], x[2 * c + 1], z));
      }
      z = warp_sum(z) * p.scale_log2;
      if (z > top) {
        const float f = exp2f(top - z);
        sum *= f;
#pragma unroll
        for (int d = 0; d < 16; ++d) acc[d] *= f;
        top = z;
      }
      const float e = z == -INFINITY ? 0.f : exp2f(z - top);
      sum += e;
#pragma unroll
      for (int d = 0; d < 16; ++d) acc[d] = fmaf(e, x[d], acc[d]);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  uint32_t* o = reinterpret_cast<uint32_t*>(p.o + row * kVlat) + lane;
#pragma unroll
  for (int c = 0; c < 8; ++c) o[32 * c] = pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace dense

size_t dense_scratch_bytes(int B, int T, int H, int64_t span) {
  (void)B, (void)T, (void)H, (void)span;
  return 0;
}

dsa_status_t dense_fwd_launch(const DenseArgs& a, cudaStream_t stream) {
  using namespace dense;
  const Params p{a.q_lat, store_of(a), mask_of(a), a.B, a.H, a.scale * 1.4426950408889634f,
                 a.o_lat, a.lse, a.status};
  const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.H;
  rows_kernel<<<static_cast<unsigned>((rows + WARPS - 1) / WARPS), WARPS * 32, 0, stream>>>(p);
  return launch_status("rows_kernel");
}

}  // namespace dsa
