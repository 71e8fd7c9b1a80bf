// rmsnorm_fp8.cu -- the head of a layer on sm_103a: residual addition, RMS norm
// and E4M3 quantisation in one pass over the row (KimiK3TextConfig: hidden_size
// 7168, rms_norm_eps 1e-5).
//
//   h = x + r,  y = h / sqrt(mean(h^2) + eps) * g
//   residual_out = BF16(h),  y_out = BF16(y)
//   scale_b = max(max_b |y|, 2^-100) / 448,  code = E4M3(y * (1 / scale_b)),  b = 128 values
//
// A row is held in registers as FP32 between the two halves (sum of squares,
// then scaling), so each input is read once and each output written once.
// Thread t of a row's T threads holds the 16-byte vectors t, t + T, ...; T is a
// multiple of 32, so the 16 lanes of a half-warp hold one scale block each time
// and its maximum is four shuffles away.  HBM-bound where there are many rows
// (16,384 x 7,168 with residual and y in 155 us, 6.8 TB/s, the rate of a copy),
// else by the launch and one row's way through an SM (2.5 us for one row).
#include <cuda_bf16.h>

#include <type_traits>

#include "cluster.cuh"
#include "dsa_status.cuh"
#include "projection.h"

namespace dsa {
namespace rms {

struct Params {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* gain;
  int64_t n_rows;
  int nvec;      // hid / 8
  int nblk;      // ceil(hid / 128)
  float inv_hid, eps;
  uint16_t* residual_out;
  uint16_t* y;
  uint8_t* codes;
  float* scale;
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// Squares that FP32 cannot hold, up to 2^16 of them below 2^-126, are off by less than
// 2^-134 together, which counts only beside a sum and an eps below kLow.  Calls with
// such an eps take the kernels with SMALL, which sum such a row again, its values times
// 2^100 (16,384 x 7,168 with eps = 0: 148 us, 141.5 without the second look; x = residual).
constexpr float kLow = 0x1p-100f;

// One row per CTA, or (MANY) several of T threads each; VPT vectors per thread.
template <int VPT, bool MANY, bool SMALL>
__global__ void __launch_bounds__(1024, VPT <= 2 ? 2 : 1) rmsnorm_kernel(const Params p, int T) {
  __shared__ float s_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!MANY) T = blockDim.x;
  const int slot = MANY ? threadIdx.x / T : 0, tid = threadIdx.x - slot * T;
  const int64_t row = MANY ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / T) + slot : blockIdx.x;
  const int nvec = !MANY || row < p.n_rows ? p.nvec : 0;   // no row: nothing is read or written
  const int64_t base = row * p.nvec;
  // x, residual and the outputs may be the same memory: no read-only loads
  const uint4* x = reinterpret_cast<const uint4*>(p.x) + base;
  float h[VPT][8];
  float q = 0.f;
  pdl_wait();
  pdl_start_next();
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * T;
    if (v < nvec) {
      unpack8(x[v], h[i]);
      if (p.residual != nullptr) {
        float r[8];
        unpack8(reinterpret_cast<const uint4*>(p.residual)[base + v], r);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] += r[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(h[i][e], h[i][e], q);
  }
  const int nw = T >> 5;                                   // the row's warps
  auto sum_row = [&](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) s_sum[warp] = v;
    __syncthreads();
    v = lane < nw ? s_sum[slot * nw + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  q = sum_row(q);
  float up = 1.f;                                          // what h is multiplied by
  if constexpr (SMALL) {
    if (q < kLow) up = 0x1p100f;
    if (__syncthreads_or(q < kLow)) {                      // a CTA's rows go together
      float again = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) again = fmaf(h[i][e] * up, h[i][e] * up, again);
      q = sum_row(again);
    }
  }
  const float inv = 1.f / sqrtf(fmaf(q, p.inv_hid, p.eps * up * up));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * T;
    const bool in = v < nvec;
    if (in && p.residual_out != nullptr)
      reinterpret_cast<uint4*>(p.residual_out)[base + v] = pack8(h[i]);
    float y[8];
    uint32_t top = 0;
    if (in) {
      unpack8(reinterpret_cast<const uint4*>(p.gain)[v], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] *= h[i][e] * up * inv;
        // magnitudes order like their bit patterns, a NaN above everything
        top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
      }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (in) {
      const float scale = __fdiv_rn(__uint_as_float(max(top, __float_as_uint(0x1p-100f))), 448.f);
      const float k = __frcp_rn(scale);
      if (p.y != nullptr) reinterpret_cast<uint4*>(p.y)[base + v] = pack8(y);
      uint2 c;
      c.x = e4m3x2(__fmul_rn(y[1], k), __fmul_rn(y[0], k)) |
            (e4m3x2(__fmul_rn(y[3], k), __fmul_rn(y[2], k)) << 16);
      c.y = e4m3x2(__fmul_rn(y[5], k), __fmul_rn(y[4], k)) |
            (e4m3x2(__fmul_rn(y[7], k), __fmul_rn(y[6], k)) << 16);
      reinterpret_cast<uint2*>(p.codes)[base + v] = c;
      if ((v & 15) == 0) p.scale[row * p.nblk + (v >> 4)] = scale;
    }
  }
}

}  // namespace rms

dsa_status_t rmsnorm_fp8_launch(const RmsNormArgs& a, cudaStream_t stream) {
  using namespace rms;
  const Params p{a.x, a.residual, a.gain, a.n_rows, a.hid / 8, (a.hid + 127) / 128,
                 1.f / static_cast<float>(a.hid), a.eps, a.residual_out, a.y, a.codes, a.scale};
  // Vectors per thread: one (the shortest way through a row) unless a row's
  // threads crowd an SM, when two let twice as many rows be in flight
  // (16,384 x 7,168 with everything on: 180 us with one, 156 with two, 172 with
  // four; 16,384 x 1,024: 23.8 against 24.7; one row of 7,168: 2.5 against 3.1),
  // or the row needs more (with eight the values do not all fit the registers: 4,096 x
  // 65,536 with everything on 530 us, 4.6 TB/s).  Short rows share a CTA.
  const int vpt = p.nvec > 4096 ? 8 : p.nvec > 2048 ? 4
                  : p.nvec > 1024 || (p.nvec > 512 && a.n_rows > 2 * num_sms()) ? 2 : 1;
  const int T = ((p.nvec + vpt - 1) / vpt + 31) / 32 * 32;
  const int R = T <= 128 ? 256 / T : 1;
  const unsigned grid = static_cast<unsigned>((a.n_rows + R - 1) / R), block = static_cast<unsigned>(T * R);
  auto launch = [&](auto kernel) { launch_overlapped(kernel, grid, block, 0, 0, stream, p, T); };
  auto launch_eps = [&](auto SMALL) {
    constexpr bool small = decltype(SMALL)::value;
    if (R > 1) launch(rmsnorm_kernel<1, true, small>);
    else if (vpt == 1) launch(rmsnorm_kernel<1, false, small>);
    else if (vpt == 2) launch(rmsnorm_kernel<2, false, small>);
    else if (vpt == 4) launch(rmsnorm_kernel<4, false, small>);
    else launch(rmsnorm_kernel<8, false, small>);
  };
  if (a.eps < kLow) launch_eps(std::true_type{});
  else launch_eps(std::false_type{});
  return launch_status("rmsnorm_kernel");
}

}  // namespace dsa
