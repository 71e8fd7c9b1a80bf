// linear_fp8.cu -- projections in E4M3 on sm_103a: the quantisation of a weight
// with one FP32 scale per 128 x 128 block, and the product with activations that
// carry one scale per 128 values of a row:
//   out[m,n] = sum_b a_scale[m,b] * w_scale[n/128,b] * sum_{k in b} a[m,k] * w[n,k]
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsa_status.cuh"
#include "internal.h"
#include "sm103.cuh"

namespace dsa {
namespace lin {

// One CTA per 128 x 128 block, held in registers between the maximum and the
// rounding: 16 lanes read a row's 256 bytes, 8 passes of 16 rows.
__global__ void __launch_bounds__(256)
    quant_weight_kernel(const uint16_t* __restrict__ w, int N, int K, uint8_t* __restrict__ codes,
                        float* __restrict__ scale) {
  __shared__ uint32_t s_top[8];
  const int tid = threadIdx.x;
  const int kb = (K + 127) / 128;
  const int col = static_cast<int>(blockIdx.x % kb) * 128 + (tid & 15) * 8;
  const int row0 = static_cast<int>(blockIdx.x / kb) * 128 + (tid >> 4);
  uint4 u[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    u[i] = make_uint4(0, 0, 0, 0);
    if (row < N && col < K)
      u[i] = __ldg(reinterpret_cast<const uint4*>(w + static_cast<int64_t>(row) * K + col));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)   // BF16 magnitudes order like their bits, a NaN above everything
      top = max(top, max((x[e] << 16) & 0x7fff0000u, x[e] & 0x7fff0000u));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, s_top[k]);
  const float sc = __fdiv_rn(__uint_as_float(max(top, __float_as_uint(0x1p-100f))), 448.f);
  const float inv = __frcp_rn(sc);
  if (tid == 0) scale[blockIdx.x] = sc;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    if (row < N && col < K) {
      const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      uint32_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c[e] = e4m3x2(__fmul_rn(__uint_as_float(x[e] & 0xffff0000u), inv),
                      __fmul_rn(__uint_as_float(x[e] << 16), inv));
      *reinterpret_cast<uint2*>(codes + static_cast<int64_t>(row) * K + col) =
          make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
  }
}

struct Params {
  const uint8_t* a;
  const float* a_scale;
  const uint8_t* w;
  const float* w_scale;
  int M, N, K, kb;
  void* out;
};

// 32 x 32 outputs per CTA, one per thread, on the FP32 pipes.
template <bool FP32>
__global__ void __launch_bounds__(1024) linear_kernel(const Params p) {
  __shared__ float s_a[32][33], s_w[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int m0 = blockIdx.y * 32, n0 = blockIdx.x * 32;
  auto decode = [](uint8_t c) {
    __nv_fp8_e4m3 v;
    v.__x = c;
    return static_cast<float>(v);
  };
  const int m = m0 + ty, n = n0 + tx;
  float acc = 0.f;
  for (int b = 0; b < p.kb; ++b) {
    float part = 0.f;
    for (int k0 = b * 128; k0 < min(p.K, b * 128 + 128); k0 += 32) {
      const int k = k0 + tx;
      const bool in = k < p.K;
      s_a[ty][tx] = in && m0 + ty < p.M ? decode(p.a[static_cast<int64_t>(m0 + ty) * p.K + k]) : 0.f;
      s_w[ty][tx] = in && n0 + ty < p.N ? decode(p.w[static_cast<int64_t>(n0 + ty) * p.K + k]) : 0.f;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 32; ++k) part = fmaf(s_a[ty][k], s_w[tx][k], part);
      __syncthreads();
    }
    if (m < p.M && n < p.N)
      acc = fmaf(part, p.a_scale[static_cast<int64_t>(m) * p.kb + b] *
                           p.w_scale[static_cast<int64_t>(n >> 7) * p.kb + b], acc);
  }
  if (m < p.M && n < p.N) {
    const int64_t o = static_cast<int64_t>(m) * p.N + n;
    if constexpr (FP32)
      static_cast<float*>(p.out)[o] = acc;
    else
      static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(acc);
  }
}

}  // namespace lin

dsa_status_t quant_fp8_weight_launch(const uint16_t* w, int N, int K, uint8_t* codes, float* scale,
                                     cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((K + 127) / 128) * static_cast<unsigned>((N + 127) / 128);
  lin::quant_weight_kernel<<<grid, 256, 0, stream>>>(w, N, K, codes, scale);
  return launch_status("quant_weight_kernel");
}

dsa_status_t linear_fp8_launch(const LinearArgs& a, cudaStream_t stream) {
  const lin::Params p{a.a, a.a_scale, a.w, a.w_scale, a.M, a.N, a.K, (a.K + 127) / 128, a.out};
  const dim3 grid(static_cast<unsigned>((a.N + 31) / 32), static_cast<unsigned>((a.M + 31) / 32));
  if (a.fp32)
    lin::linear_kernel<true><<<grid, 1024, 0, stream>>>(p);
  else
    lin::linear_kernel<false><<<grid, 1024, 0, stream>>>(p);
  return launch_status("linear_kernel");
}

}  // namespace dsa
