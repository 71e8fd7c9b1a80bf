// mla_window_bwd.cu -- backward pass of windowed dense attention over latent rows.
//
// Given the forward's o_lat and lse, and d_o, with z and p as there:
//   p_s = exp(z_s - lse),  D = d_o . o_lat,  dz_s = scale * p_s (d_o . KV[s, 0:512] - D)
//   dq = sum_s dz_s KV[s, :],   dkv[s] = sum over the queries that see s of dz_s q + p_s d_o
//
// A warp per (query, head) for dq and per row for dkv, dims over the lanes.
#include <cmath>

#include <cuda_bf16.h>

#include "dense_mask.cuh"
#include "sm103.cuh"

namespace dsa {
namespace wbw {

using namespace dense;
constexpr int WARPS = 8;

struct Params {
  const uint16_t* q;
  Store kv;
  Mask m;
  int B, H;
  float scale;
  const uint16_t* o;
  const float* lse;
  const uint16_t* d_o;
  uint16_t* dq;
  uint16_t* dkv;
  uint32_t* status;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// C chunks of 64 dims of a row: dims 64c + 2 lane (+1)
template <int C>
__device__ __forceinline__ void load_row(const uint16_t* row, int lane, float (&x)[2 * C]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(row) + lane;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t v = __ldg(r + 32 * c);
    x[2 * c] = __uint_as_float(v << 16), x[2 * c + 1] = __uint_as_float(v & 0xffff0000u);
  }
}
template <int N, int M, int K>
__device__ __forceinline__ float dot(const float (&x)[M], const float (&y)[K]) {
  float z = 0.f;
#pragma unroll
  for (int d = 0; d < N; ++d) z = fmaf(x[d], y[d], z);
  return warp_sum(z);
}
__device__ __forceinline__ void store_row(uint16_t* row, int lane, const float (&x)[18]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(row) + lane;
#pragma unroll
  for (int c = 0; c < 9; ++c) r[32 * c] = pack_bf16x2(x[2 * c], x[2 * c + 1]);
}

__global__ void __launch_bounds__(WARPS * 32) dq_kernel(const Params p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(p.B) * p.m.T * p.H) return;
  const int64_t qi = row / p.H;
  const int b = static_cast<int>(qi / p.m.T), i = static_cast<int>(qi % p.m.T);
  const Seq s = seq_of(p.m, b);
  if (row % (static_cast<int64_t>(p.m.T) * p.H) == 0 && lane == 0) report_seq(p.m, s, b, p.status);
  float q[18], d_o[16], o[16], acc[18], x[18];
  load_row<9>(p.q + row * kRlat, lane, q);
  load_row<8>(p.d_o + row * kVlat, lane, d_o);
  load_row<8>(p.o + row * kVlat, lane, o);
#pragma unroll
  for (int d = 0; d < 18; ++d) acc[d] = 0.f;
  const float D = dot<16>(d_o, o), lse = __ldg(p.lse + row);
  const Pages pages = pages_of(p.m, s, i, i);
  for (int k = 0; k < pages.count(); ++k) {
    const int pg = pages.page(k);
    for (uint64_t see = row_mask(p.m, s, i, 0, pg * 64); see != 0; see &= see - 1) {
      const int64_t r = page_row(p.kv, b, pg) + __ffsll(static_cast<long long>(see)) - 1;
      load_row<9>(p.kv.base + r * kRlat, lane, x);
      const float e = expf(dot<18>(q, x) * p.scale - lse);
      const float dz = e * (dot<16>(d_o, x) - D) * p.scale;
#pragma unroll
      for (int d = 0; d < 18; ++d) acc[d] = fmaf(dz, x[d], acc[d]);
    }
  }
  store_row(p.dq + row * kRlat, lane, acc);
}

__global__ void __launch_bounds__(WARPS * 32) dkv_kernel(const Params p) {
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  const int b = static_cast<int>(w / p.m.max_kv_len), r = static_cast<int>(w % p.m.max_kv_len);
  if (b >= p.B) return;
  const Seq s = seq_of(p.m, b);
  if (!s.ok || r >= s.L) return;
  const int64_t row = static_cast<int64_t>(b) * p.kv.seq_stride + r;
  float x[18], acc[18], q[18], d_o[16], o[16];
  load_row<9>(p.kv.base + row * kRlat, lane, x);
#pragma unroll
  for (int d = 0; d < 18; ++d) acc[d] = 0.f;
  const int last = min(s.n, s.L - s.pos0);
  for (int i = max(0, r - s.pos0); i < last; ++i) {
    if (r >= p.m.n_first && s.pos0 + i - r >= p.m.window) break;
    for (int h = 0; h < p.H; ++h) {
      const int64_t qr = (static_cast<int64_t>(b) * p.m.T + i) * p.H + h;
      load_row<9>(p.q + qr * kRlat, lane, q);
      load_row<8>(p.d_o + qr * kVlat, lane, d_o);
      load_row<8>(p.o + qr * kVlat, lane, o);
      const float e = expf(dot<18>(q, x) * p.scale - __ldg(p.lse + qr));
      const float dz = e * (dot<16>(d_o, x) - dot<16>(d_o, o)) * p.scale;
#pragma unroll
      for (int d = 0; d < 18; ++d) acc[d] = fmaf(dz, q[d], acc[d]);
#pragma unroll
      for (int d = 0; d < 16; ++d) acc[d] = fmaf(e, d_o[d], acc[d]);
    }
  }
  store_row(p.dkv + row * kRlat, lane, acc);
}

}  // namespace wbw

size_t window_bwd_scratch_bytes(int B, int T, int H, int max_kv_len, int64_t span) {
  (void)B, (void)T, (void)H, (void)max_kv_len, (void)span;
  return 0;
}

dsa_status_t window_bwd_launch(const WindowBwdArgs& a, cudaStream_t stream) {
  using namespace wbw;
  const Params p{a.f.q_lat, store_of(a.f), mask_of(a.f), a.f.B, a.f.H, a.f.scale, a.f.o_lat,
                 a.f.lse, a.d_o, a.dq, a.dkv, a.f.status};
  const int64_t rows = static_cast<int64_t>(a.f.B) * a.f.T * a.f.H;
  const int64_t keys = static_cast<int64_t>(a.f.B) * a.f.max_kv_len;
  dq_kernel<<<static_cast<unsigned>((rows + WARPS - 1) / WARPS), WARPS * 32, 0, stream>>>(p);
  dkv_kernel<<<static_cast<unsigned>((keys + WARPS - 1) / WARPS), WARPS * 32, 0, stream>>>(p);
  return launch_status("dkv_kernel");
}

}  // namespace dsa
