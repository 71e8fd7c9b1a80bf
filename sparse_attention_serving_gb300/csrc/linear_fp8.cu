// linear_fp8.cu -- projections in E4M3 on sm_103a: the quantisation of a weight
// with one FP32 scale per 128 x 128 block, and the product with activations that
// carry one scale per 128 values of a row:
//   out[m,n] = sum_b a_scale[m,b] * w_scale[n/128,b] * sum_{k in b} a[m,k] * w[n,k]
#include <cuda_bf16.h>

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
  const float* a_scale;
  const float* w_scale;
  int M, N, kb;       // kb = ceil(K / 128) blocks of K
  void* out;
  bool fp32;
  uint32_t* status;
};

__device__ __forceinline__ void store_out(const Params& p, int m, int n, float v) {
  const int64_t o = static_cast<int64_t>(m) * p.N + n;
  if (p.fp32)
    static_cast<float*>(p.out)[o] = v;
  else
    static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------------------
// Split kernel: Dt[128 features x NT tokens] = W . A^T over a slice of K per CTA,
// the slices of a tile on one cluster and joined through its shared memory.
//
// The weight is the M side of the MMA, so a few tokens cost few columns (N = NT
// from 16) and every weight byte is read once.  Each block of K = 128 goes into a
// TMEM buffer of its own (four MMAs of K = 32); the epilogue warps add it, times
// w_scale * a_scale[token], to FP32 registers: a lane is a feature, a register a
// token, the token's factor comes from shared memory as a broadcast.
// ---------------------------------------------------------------------------
enum : uint32_t { SITE_S_E = 0x700, SITE_S_F = 0x701, SITE_S_ACC = 0x702, SITE_S_FREE = 0x703,
                  SITE_S_DRAIN = 0x704 };

template <int NT>
struct Split {
  static constexpr int EW = NT > 64 ? 8 : 4;             // epilogue warps
  static constexpr int COLS = NT / (EW / 4);             // tokens per epilogue thread
  static constexpr int NTHREADS = 64 + EW * 32;
  static constexpr int STAGE = (128 + NT) * 128;
  // three CTAs per SM up to 16 tokens, two up to 64, one above
  static constexpr int CTAS = NT <= 16 ? 3 : NT <= 64 ? 2 : 1;
  static constexpr int NST = NT == 32 ? 5 : NT == 128 ? 6 : 4;
  static constexpr int NB = NT <= 128 ? 4 : 2;           // TMEM buffers
  static constexpr int TCOLS = NT * NB;
  static constexpr int OFF_MISC = NST * STAGE;           // barriers, then two sets of factors
  static constexpr int OFF_FACT = OFF_MISC + 256;
  static constexpr int SMEM = 1024 + OFF_FACT + 2 * NT * 4;
  static_assert(TCOLS >= 32 && TCOLS * CTAS <= 512, "TMEM columns");
  static_assert(NT * 128 * 4 <= NST * STAGE, "the partial tile reuses the stages");
  static_assert((SMEM + 1024) * CTAS <= 228 * 1024, "shared memory");
};

template <int NT>
__global__ void __launch_bounds__(Split<NT>::NTHREADS, Split<NT>::CTAS)
    split_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                 const Params p, const int S) {
  using C = Split<NT>;
  constexpr uint32_t IDESC = idesc_e4m3(128, NT);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OFF_MISC);
  uint64_t* empty = full + C::NST;
  uint64_t* acc_full = empty + C::NST;
  uint64_t* acc_free = acc_full + C::NB;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(acc_free + C::NB);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tslot + 1);
  float* fact = reinterpret_cast<float*>(sm + C::OFF_FACT);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = blockIdx.x / S, rank = blockIdx.x - tile * S;   // the cluster is S CTAs along x
  const int ntn = (p.N + 127) / 128;
  const int nb = tile % ntn;
  const int n0 = nb * 128, m0 = (tile / ntn) * NT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / S);
  const int nkb = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / S) - kb0;

  if (tid == 0) {
    for (int k = 0; k < 2 * C::NST + C::NB; ++k) mbar_init(&full[k], 1);
    for (int k = 0; k < C::NB; ++k) mbar_init(&acc_free[k], C::EW);
    s_abort[0] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tslot, C::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  float acc[C::COLS];
#pragma unroll
  for (int c = 0; c < C::COLS; ++c) acc[c] = 0.f;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_w);
      tma_prefetch_desc(&tm_a);
      int i = 0;
      for (; i < nkb; ++i) {
        const int st = i % C::NST, use = i / C::NST;
        if (use > 0 && !mbar_wait(&empty[st], (use - 1) & 1, p.status, kWaitLimitNs, SITE_S_E)) break;
        if (s_abort[0]) break;
        uint8_t* w = sm + st * C::STAGE;
        mbar_expect_tx(&full[st], C::STAGE);
        tma_load_2d(w, &tm_w, &full[st], 64 * (kb0 + i), n0);
        tma_load_2d(w + 128 * 128, &tm_a, &full[st], 64 * (kb0 + i), m0);
      }
      if (i < nkb) s_abort[0] = 1;
      // the copies in flight have landed before anything else touches the stages
      for (int k = max(0, i - C::NST); k < i; ++k)
        mbar_wait(&full[k % C::NST], (k / C::NST) & 1, p.status, kWaitLimitNs, SITE_S_F);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int i = 0;
      for (; i < nkb; ++i) {
        const int st = i % C::NST, bu = i % C::NB, use = i / C::NB;
        if (!mbar_wait(&full[st], (i / C::NST) & 1, p.status, kWaitLimitNs, SITE_S_F)) break;
        if (use > 0 &&
            !mbar_wait(&acc_free[bu], (use - 1) & 1, p.status, kWaitLimitNs, SITE_S_FREE))
          break;
        tc_fence_after();
        const uint64_t wd = smem_desc(smem_u32(sm + st * C::STAGE), 16, 1024);
        const uint64_t ad = desc_add(wd, 128 * 128);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_e4m3(tmem + bu * NT, desc_add(wd, kk * 32), desc_add(ad, kk * 32), IDESC, kk ? 1u : 0u);
        umma_commit(&empty[st]);
        umma_commit(&acc_full[bu]);
      }
      if (i < nkb) s_abort[0] = 1;
      // every MMA issued has finished before the stages or the TMEM are given up
      for (int k = max(0, i - C::NST); k < i; ++k)
        mbar_wait(&empty[k % C::NST], (k / C::NST) & 1, p.status, kWaitLimitNs, SITE_S_DRAIN);
    }
    __syncwarp();
  } else {
    const int et = tid - 64;                               // epilogue thread
    const int sub = warp & 3;                              // TMEM lane quarter of this warp
    const int c0 = (et >> 7) * C::COLS;                    // its first token
    const uint32_t taddr = tmem + (static_cast<uint32_t>(sub * 32) << 16) + c0;
    // factors w_scale * a_scale of token m0 + et, two blocks ahead of their use
    const bool has = et < NT && m0 + et < p.M;
    const float* as = p.a_scale + static_cast<int64_t>(has ? m0 + et : 0) * p.kb + kb0;
    const float* ws = p.w_scale + static_cast<int64_t>(nb) * p.kb + kb0;
    auto factor = [&](int i) { return has && i < nkb ? __ldg(as + i) * __ldg(ws + i) : 0.f; };
    float f0 = factor(0), f1 = factor(1);
    bool ok = true;
    for (int i = 0; i < nkb; ++i) {
      const int bu = i % C::NB;
      float* fb = fact + (i & 1) * NT;
      if (et < NT) fb[et] = f0;
      f0 = f1;
      f1 = factor(i + 2);
      // all epilogue warps leave together if one of them gave up
      if (named_bar_or(1, C::EW * 32, !ok)) {
        ok = false;
        break;
      }
      ok = mbar_wait(&acc_full[bu], (i / C::NB) & 1, p.status, kWaitLimitNs, SITE_S_ACC);
      __syncwarp();
      tc_fence_after();
      constexpr int STEP = C::COLS < 32 ? 16 : 32;
#pragma unroll
      for (int c = 0; c < C::COLS; c += STEP) {
        uint32_t d[STEP];
        if constexpr (STEP == 16)
          tmem_ld16(taddr + bu * NT + c, d);
        else
          tmem_ld32(taddr + bu * NT + c, d);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < STEP; e += 4) {
          const float4 f = *reinterpret_cast<const float4*>(fb + c0 + c + e);
          fma2_rn(acc[c + e], acc[c + e + 1], __uint_as_float(d[e]), __uint_as_float(d[e + 1]), f.x, f.y);
          fma2_rn(acc[c + e + 2], acc[c + e + 3], __uint_as_float(d[e + 2]),
                  __uint_as_float(d[e + 3]), f.z, f.w);
        }
      }
      tc_fence_before();
      mbar_arrive_warp(&acc_free[bu]);
    }
    if (!ok) s_abort[0] = 1;
    const int n = n0 + sub * 32 + lane;
    if (S == 1) {
      if (n < p.N) {
#pragma unroll
        for (int c = 0; c < C::COLS; ++c)
          if (m0 + c0 + c < p.M) store_out(p, m0 + c0 + c, n, acc[c]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) {
    // every copy and MMA of this CTA is done: its stages hold the partial tile now
    float* part = reinterpret_cast<float*>(sm);            // [NT][128]
    const int et = tid - 64, row = ((warp & 3) << 5) + lane, grp = et >> 7;
    if (warp >= 2) {
#pragma unroll
      for (int c = 0; c < C::COLS; ++c) part[(grp * C::COLS + c) * 128 + row] = acc[c];
    }
    cluster_sync();
    if (warp >= 2 && n0 + row < p.N) {
      // this CTA's share of the tokens, the slices of K added in their order
      const int live = min(NT, p.M - m0);
      for (int c = rank + grp * S; c < live; c += S * (C::EW / 4)) {
        float v = 0.f;
        const uint32_t at = smem_u32(part + c * 128 + row);
        for (int r = 0; r < S; ++r) v += ld_cluster_f32(at, r);
        store_out(p, m0 + c, n0 + row, v);
      }
    }
    cluster_sync();   // no CTA leaves while another still reads its shared memory
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TCOLS);
  }
}

template <int NT>
dsa_status_t launch_split(const LinearArgs& a, int S, cudaStream_t stream) {
  using C = Split<NT>;
  CUtensorMap ta, tw;
  // pairs of codes as 16-bit elements: copies only move them
  const uint64_t K = static_cast<uint64_t>(a.K);
  if (!encode_tmap_2d(&ta, a.a, a.M, K / 2, K, 64, NT, true) ||
      !encode_tmap_2d(&tw, a.w, a.N, K / 2, K, 64, 128, true))
    return DSA_ERR_CUDA;
  const Params p{a.a_scale, a.w_scale, a.M, a.N, (a.K + 127) / 128, a.out, a.fp32, a.status};
  if (cudaFuncSetAttribute(split_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
      cudaSuccess)
    return launch_status("cudaFuncSetAttribute");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(((a.N + 127) / 128) * ((a.M + NT - 1) / NT) * S));
  cfg.blockDim = dim3(C::NTHREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(S);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, split_kernel<NT>, ta, tw, p, S);
  return launch_status("split_kernel");
}

}  // namespace lin

dsa_status_t quant_fp8_weight_launch(const uint16_t* w, int N, int K, uint8_t* codes, float* scale,
                                     cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((K + 127) / 128) * static_cast<unsigned>((N + 127) / 128);
  lin::quant_weight_kernel<<<grid, 256, 0, stream>>>(w, N, K, codes, scale);
  return launch_status("quant_weight_kernel");
}

dsa_status_t linear_fp8_launch(const LinearArgs& a, cudaStream_t stream) {
  const int kb = (a.K + 127) / 128;
  const int nt = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : a.M <= 128 ? 128 : 256;
  const int per_sm = nt <= 16 ? 3 : nt <= 64 ? 2 : 1;
  const int64_t tiles = static_cast<int64_t>((a.N + 127) / 128) * ((a.M + nt - 1) / nt);
  // as many slices of K as fill the GPU, up to the portable cluster size
  int64_t S = num_sms() * per_sm / tiles;
  S = S < 1 ? 1 : S > 8 ? 8 : S;
  if (S > kb) S = kb;
  switch (nt) {
    case 16: return lin::launch_split<16>(a, static_cast<int>(S), stream);
    case 32: return lin::launch_split<32>(a, static_cast<int>(S), stream);
    case 64: return lin::launch_split<64>(a, static_cast<int>(S), stream);
    case 128: return lin::launch_split<128>(a, static_cast<int>(S), stream);
    default: return lin::launch_split<256>(a, static_cast<int>(S), stream);
  }
}

}  // namespace dsa
