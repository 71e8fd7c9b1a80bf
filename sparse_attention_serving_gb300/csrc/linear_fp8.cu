// linear_fp8.cu -- projections in E4M3 on sm_103a: the quantisation of a weight
// with one FP32 scale per 128 x 128 block, and the product with activations that
// carry one scale per 128 values of a row:
//   out[m,n] = sum_b a_scale[m,b] * w_scale[n/128,b] * sum_{k in b} a[m,k] * w[n,k]
#include <cuda_bf16.h>

#include <type_traits>

#include "cluster.cuh"
#include "dsa_status.cuh"
#include "projection.h"

namespace dsa {
namespace lin {

// One CTA per 128 x 128 block, held in registers between the maximum and the
// rounding (one pass over the weight): 16 lanes read a row's 256 bytes, 8 passes
// of 16 rows, all loads in flight before the first is used.  HBM-bound: 7,168 x
// 12,288 in 41 us, 6.5 TB/s of the 3 bytes per weight it cannot do without.
__global__ void __launch_bounds__(256)
    quant_weight_kernel(const uint16_t* w, int N, int K, uint8_t* codes, float* scale) {
  __shared__ uint32_t s_top[8];
  const int tid = threadIdx.x;
  const int kb = (K + 127) / 128;
  const int col = static_cast<int>(blockIdx.x % kb) * 128 + (tid & 15) * 8;
  const int row0 = static_cast<int>(blockIdx.x / kb) * 128 + (tid >> 4);
  uint4 u[8];
  uint32_t top = 0;
  pdl_wait();
  pdl_start_next();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    u[i] = make_uint4(0, 0, 0, 0);
    if (row < N && col < K)
      u[i] = *reinterpret_cast<const uint4*>(w + static_cast<int64_t>(row) * K + col);
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

// Features n .. n+3 of token m (n a multiple of 4), those that exist.
__device__ __forceinline__ void store_out4(const Params& p, int m, int n, const float4& v) {
  const int64_t o = static_cast<int64_t>(m) * p.N + n;
  if ((p.N & 3) == 0) {
    if (n >= p.N) return;
    if (p.fp32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  } else {
    const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < p.N) store_out(p, m, n + k, e[k]);
  }
}

// The factor a_scale * w_scale of a block's sum d (0 or 2^-18 to 2^25 in magnitude).
// The scales are FP32 of any size, so their product may leave FP32's normal range
// though d times it does not.  Then it is applied as pre * mul with mul a power of
// two, (d * pre) * mul: below the range pre = product * 2^32 (where that is not normal
// its error, 2^-150, comes to less than 2^-156 of out); above it pre = product * 2^-127,
// cut to the largest number where it overflows (d * product is then infinite or 0
// either way).  In the range pre = 1 and mul is the product.  A set of factors that
// has one out of range takes the loop with pre: with no other sets 64 x 7,168 x 12,288
// takes 22.5 us instead of 15.6 (the weight in L2), 16,384 x 7,168 x 12,288 1.29 ms
// instead of 0.93; products all in range take no longer than without it.  (A token of
// zeros has the least scale, 2^-109: in range for weights' scales above 2^-17.)
struct Factor {
  float pre, mul;
};
constexpr float kLeastNormal = 0x1p-126f, kMost = 0x1.fffffep127f;
__device__ __forceinline__ Factor factor(float a, float w) {
  const float f = a * w;
  if (fabsf(f) < kLeastNormal)
    return fabsf(a) < fabsf(w) ? Factor{(a * 0x1p32f) * w, 0x1p-32f} : Factor{(w * 0x1p32f) * a, 0x1p-32f};
  if (fabsf(f) > kMost && fmaxf(fabsf(a), fabsf(w)) <= kMost) {   // two numbers, so both above 1
    const float pre = (a * 0x1p-64f) * (w * 0x1p-63f);
    return {fmaxf(-kMost, fminf(kMost, pre)), 0x1p127f};
  }
  return {1.f, f};
}
// The least and the largest magnitude of some numbers (a NaN does not count: no
// Factor changes what it gives).
struct Span {
  float least = kMost, most = 0.f;
  template <int N>
  __device__ __forceinline__ void add(const float (&v)[N]) {
    float lo[N], hi[N];                    // a tree: a chain of 16 is what a set waits for
#pragma unroll
    for (int k = 0; k < N; ++k) lo[k] = hi[k] = fabsf(v[k]);
#pragma unroll
    for (int d = 1; d < N; d *= 2)
#pragma unroll
      for (int k = 0; k + d < N; k += 2 * d) {
        lo[k] = fminf(lo[k], lo[k + d]);
        hi[k] = fmaxf(hi[k], hi[k + d]);
      }
    least = fminf(least, lo[0]);
    most = fmaxf(most, hi[0]);
  }
  // Whether all of them times w are normal numbers.
  __device__ __forceinline__ bool normal_times(float w) const {
    return fabsf(least * w) >= kLeastNormal && fabsf(most * w) <= kMost;
  }
};

// A value that is the same in every lane, known to be so by the compiler.  Warps
// that issue copies and MMAs run their loops whole, on such values, and elect a
// lane for the instructions themselves: with one lane running the loop, every
// MMA and every commit cost about 45 cycles more (a block of 128 x 16 x 128 276
// cycles instead of 160).
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// ---------------------------------------------------------------------------
// Split kernel: Dt[128 features x NT tokens] = W . A^T over a slice of K per CTA,
// the slices of a tile on one cluster and joined through its shared memory.
//
// The weight is the M side of the MMA, so a few tokens cost few columns (N = NT
// from 16) and every weight byte is read once.  Each block of K = 128 goes into a
// TMEM buffer of its own (four MMAs of K = 32, the codes' products and their sum
// in FP32); the epilogue warps add it, times w_scale * a_scale[token], to FP32
// registers: a lane is a feature, a register a token, the token's factor comes
// from shared memory as a broadcast.
//
// A few tokens are bound by the weight's bytes (1 x 7,168 x 12,288 in 15.8 us,
// 5.6 TB/s; 64 tokens in 18.7), small products by their latencies (64 x 128 x
// 7,168 in 3.7 us), more tokens by the way from L2 into an SM's shared memory,
// about 61 bytes a cycle, and by the epilogue's loop (2,048 x 576 x 7,168 in 16.0 us:
// (128 + 96) * 128 bytes a block and CTA).
// ---------------------------------------------------------------------------
enum : uint32_t { SITE_S_E = 0x700, SITE_S_F = 0x701, SITE_S_ACC = 0x702, SITE_S_FREE = 0x703,
                  SITE_S_DRAIN = 0x704 };

template <int NT>
struct Split {
  static constexpr int EW = NT == 96 ? 12 : NT > 64 ? 8 : 4;    // epilogue warps
  static constexpr int COLS = NT / (EW / 4);             // tokens per epilogue thread
  static constexpr int NTHREADS = 64 + EW * 32;
  static constexpr int STAGE = (128 + NT) * 128;
  static constexpr int CTAS = NT <= 16 ? 3 : NT <= 64 ? 2 : 1;  // per SM
  static constexpr int NST = NT == 32 ? 5 : NT > 64 ? 6 : 4;
  static constexpr int NB = 4;                           // TMEM buffers
  static constexpr int STEP = COLS % 32 == 0 ? 32 : 16;  // columns per TMEM load
  static constexpr int TCOLS = NT == 96 ? 512 : NT * NB; // a power of two
  static constexpr int OFF_MISC = NST * STAGE;           // barriers, then two sets of factors
  static constexpr int OFF_FACT = OFF_MISC + 256;
  static constexpr int CH = 8;                           // blocks of K per set of factors
  static constexpr int FROW = NT + 4;
  static constexpr int OFF_PRE = OFF_FACT + 2 * CH * FROW * 4;   // one set's Factor::pre
  static constexpr int SMEM = 1024 + OFF_PRE + CH * NT * 4;
  static_assert(NT <= EW * 32 && TCOLS >= 32 && TCOLS * CTAS <= 512, "TMEM columns");
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
  float* pre = reinterpret_cast<float*>(sm + C::OFF_PRE);

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int tile = blockIdx.x / S, rank = blockIdx.x - tile * S;   // the cluster is S CTAs along x
  const int ntn = (p.N + 127) / 128;
  const int nb = tile % ntn;
  const int n0 = nb * 128, m0 = (tile / ntn) * NT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / S);
  const int nkb = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / S) - kb0;

  auto load = [&](int i) {
    const int st = i % C::NST;
    uint8_t* w = sm + st * C::STAGE;
    mbar_expect_tx(&full[st], C::STAGE);
    tma_load_2d(w, &tm_w, &full[st], 64 * (kb0 + i), n0);
    tma_load_2d(w + 128 * 128, &tm_a, &full[st], 64 * (kb0 + i), m0);
  };
  if (tid == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_a);
    for (int k = 0; k < 2 * C::NST + C::NB; ++k) mbar_init(&full[k], 1);
    for (int k = 0; k < C::NB; ++k) mbar_init(&acc_free[k], C::EW);
    s_abort[0] = 0;
    fence_mbar_init();
    pdl_wait();
    // the copying thread fills the ring before the other warps are set up
    for (int i = 0; i < min(C::NST, nkb); ++i) load(i);
  }
  if (warp == 1) {
    tmem_alloc(tslot, C::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tslot);
  pdl_wait();
  pdl_start_next();

  float acc[C::COLS];
#pragma unroll
  for (int c = 0; c < C::COLS; ++c) acc[c] = 0.f;

  if (warp == 0) {
    int i = min(C::NST, nkb);
    for (; i < nkb; ++i) {
      const bool ok = mbar_wait(&empty[i % C::NST], (i / C::NST - 1) & 1, p.status, kWaitLimitNs,
                                SITE_S_E) && !s_abort[0];
      if (!__all_sync(0xffffffffu, ok)) break;
      if (elect_one_lane()) load(i);
      __syncwarp();
    }
    if (i < nkb) s_abort[0] = 1;
    // the copies in flight have landed before anything else touches the stages
    for (int k = max(0, i - C::NST); k < i; ++k)
      mbar_wait(&full[k % C::NST], (k / C::NST) & 1, p.status, kWaitLimitNs, SITE_S_F);
  } else if (warp == 1) {
    const uint64_t desc0 = smem_desc(smem_u32(sm), 16, 1024);
    int i = 0;
    bool ok = true;
    for (; i < nkb; ++i) {
      const int st = i % C::NST, bu = i % C::NB, use = i / C::NB;
      ok = mbar_wait(&full[st], (i / C::NST) & 1, p.status, kWaitLimitNs, SITE_S_F) &&
           (use == 0 || mbar_wait(&acc_free[bu], (use - 1) & 1, p.status, kWaitLimitNs, SITE_S_FREE));
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint64_t wd = desc_add(desc0, st * C::STAGE), ad = desc_add(wd, 128 * 128);
      if (elect_one_lane()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_e4m3(tmem + bu * NT, desc_add(wd, kk * 32), desc_add(ad, kk * 32), IDESC, kk ? 1u : 0u);
        umma_commit(&empty[st]);
        umma_commit(&acc_full[bu]);
      }
      __syncwarp();
    }
    if (i < nkb) s_abort[0] = 1;
    // every MMA issued has finished before the stages or the TMEM are given up
    for (int k = max(0, i - C::NST); k < i; ++k)
      mbar_wait(&empty[k % C::NST], (k / C::NST) & 1, p.status, kWaitLimitNs, SITE_S_DRAIN);
  } else {
    const int et = tid - 64;                               // epilogue thread
    const int sub = warp & 3;                              // TMEM lane quarter of this warp
    const int c0 = (et >> 7) * C::COLS;                    // its first token
    const uint32_t taddr = tmem + (static_cast<uint32_t>(sub * 32) << 16) + c0;
    // Factors a_scale * w_scale, CH blocks of K at a time: loaded into registers
    // one chunk ahead, multiplied and put into shared memory at the chunk's start.
    // A thread always holds the same block of a chunk.
    constexpr int T = C::EW * 32, PER = C::CH * NT / T;
    const int fk = et % C::CH;
    const float* ws = p.w_scale + static_cast<int64_t>(nb) * p.kb + kb0;
    // Tokens and blocks that do not exist have the factor 1 (and codes of 0).
    float fa[PER], fw = 1.f;
    auto token_scale = [&](int m, int i) {
      return m < p.M ? p.a_scale[static_cast<int64_t>(m) * p.kb + kb0 + i] : 1.f;
    };
    auto fetch = [&](int i0) {
      const bool in = i0 + fk < nkb;
      fw = in ? ws[i0 + fk] : 1.f;
#pragma unroll
      for (int k = 0; k < PER; ++k)
        fa[k] = in ? token_scale(m0 + (et + k * T) / C::CH, i0 + fk) : 1.f;
    };
    fetch(0);
    int bu = 0;
    uint32_t ph = 0;
    bool ok = true;
    // Blocks i .. end - 1 with their factors from fb on; RARE: and Factor::pre from pr on.
    auto add_blocks = [&](auto RARE, int i, int end, const float* fb, const float* pr) {
#pragma unroll 1
      for (; ok && i != end; ++i, fb += C::FROW, pr += NT) {
        ok = !__any_sync(0xffffffffu, !mbar_wait(&acc_full[bu], ph, p.status, kWaitLimitNs, SITE_S_ACC));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C::COLS; c += C::STEP) {
          uint32_t d[C::STEP];
          if constexpr (C::STEP == 16)
            tmem_ld16(taddr + bu * NT + c, d);
          else
            tmem_ld32(taddr + bu * NT + c, d);
          float4 f[C::STEP / 4];                           // on their way beside the load
#pragma unroll
          for (int e = 0; e < C::STEP / 4; ++e) f[e] = reinterpret_cast<const float4*>(fb + c)[e];
          tmem_ld_wait_regs(d);
          if (c + C::STEP == C::COLS) {
            tc_fence_before();
            mbar_arrive_warp(&acc_free[bu]);
          }
          if constexpr (RARE.value) {
            const volatile float* pb = pr + c;
#pragma unroll
            for (int e = 0; e < C::STEP; ++e) d[e] = __float_as_uint(__uint_as_float(d[e]) * pb[e]);
          }
#pragma unroll
          for (int e = 0; e < C::STEP; e += 4) {
            const float4 g = f[e / 4];
            fma2_rn(acc[c + e], acc[c + e + 1], __uint_as_float(d[e]), __uint_as_float(d[e + 1]), g.x, g.y);
            fma2_rn(acc[c + e + 2], acc[c + e + 3], __uint_as_float(d[e + 2]),
                    __uint_as_float(d[e + 3]), g.z, g.w);
          }
        }
        if (++bu == C::NB) bu = 0, ph ^= 1;
      }
    };
#pragma unroll 1
    for (int i = 0; i < nkb; i += C::CH) {
      float* set = fact + ((i / C::CH) & 1) * (C::CH * C::FROW);
      Span span;
#pragma unroll
      for (int k = 0; k < PER; ++k) set[fk * C::FROW + (et + k * T) / C::CH] = fa[k] * fw;
      span.add(fa);
      const bool far = !span.normal_times(fw);
      // One vote for what is rare: a factor out of range, or a warp that gave up, when
      // all epilogue warps leave together.  (A warp's vote makes the result known to be
      // the same in all lanes, as the loops' counts are: 2,048 x 576 x 7,168 takes 16.1
      // us, 17.4 with the barrier's result itself.)
      const bool rare = __any_sync(0xffffffffu, named_bar_or(1, T, far || !ok));
      if (rare) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int c = (et + k * T) / C::CH;
          const Factor g = factor(fa[k], fw);
          set[fk * C::FROW + c] = g.mul;
          pre[fk * NT + c] = g.pre;
        }
        if (__any_sync(0xffffffffu, named_bar_or(1, T, !ok))) {
          ok = false;
          break;
        }
      }
      fetch(i + C::CH);
      const int end = min(nkb, i + C::CH);
      if (rare)
        add_blocks(std::true_type{}, i, end, set + c0, pre + c0);
      else
        add_blocks(std::false_type{}, i, end, set + c0, pre + c0);
    }
    if (!ok) s_abort[0] = 1;
    if (S == 1) {
      const int n = n0 + sub * 32 + lane;
      if (ok && n < p.N) {
#pragma unroll
        for (int c = 0; c < C::COLS; ++c)
          if (m0 + c0 + c < p.M) store_out(p, m0 + c0 + c, n, acc[c]);
      }
    } else if (ok) {
      // the last block is summed, so every copy and MMA of this CTA is done: its
      // stages hold the partial tile [NT][128] now
      float* part = reinterpret_cast<float*>(sm) + c0 * 128 + sub * 32 + lane;
#pragma unroll
      for (int c = 0; c < C::COLS; ++c) part[c * 128] = acc[c];
    }
  }
  // lanes leave a wait one by one; the cluster barriers and the release of the TMEM
  // are for whole warps
  __syncwarp();
  tc_fence_before();
  if (S == 1) {
    __syncthreads();
  } else {
    cluster_sync();
    if (warp >= 2) {
      // this CTA's share of the tokens, a warp per token and four features per
      // lane, the slices of K added in their order, eight loads in flight
      const int live = min(NT, p.M - m0);
      for (int c = rank + (warp - 2) * S; c < live; c += S * C::EW) {
        const uint32_t at = smem_u32(sm) + (c * 128 + lane * 4) * 4;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r0 = 0; r0 < S; r0 += 8) {
          float4 v[8];
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r0 + r < S) v[r] = ld_cluster_f32x4(at, r0 + r);
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r0 + r < S) {
              sum.x += v[r].x;
              sum.y += v[r].y;
              sum.z += v[r].z;
              sum.w += v[r].w;
            }
        }
        store_out4(p, m0 + c, n0 + lane * 4, sum);
      }
    }
    // no CTA leaves while another may still read its shared memory; the reads
    // are over (their values are in the stores), so nothing has to be ordered
    __syncwarp();
    cluster_arrive_relaxed();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TCOLS);
  }
  if (S > 1) cluster_wait();
}

// Whether one cluster of S CTAs fits on the SMs that this context has (0.25 us).
template <int NT>
bool split_fits(int S, cudaStream_t stream) {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(S);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(S));
  cfg.blockDim = dim3(Split<NT>::NTHREADS);
  cfg.dynamicSmemBytes = Split<NT>::SMEM;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, split_kernel<NT>, &cfg) == cudaSuccess)
    return clusters > 0;
  cudaGetLastError();   // an answer, not a failure of the call
  return false;
}

// DSA_ERR_UNSUPPORTED: a cluster of S CTAs, more than kPortable, does not fit.
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
  if (S > kPortable) {
    if (cudaFuncSetAttribute(split_kernel<NT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
        cudaSuccess)
      return launch_status("cudaFuncSetAttribute");
    if (!split_fits<NT>(S, stream)) return DSA_ERR_UNSUPPORTED;
  }
  launch_overlapped(split_kernel<NT>, static_cast<unsigned>(split_tiles(a.M, a.N, NT) * S),
                    C::NTHREADS, C::SMEM, static_cast<unsigned>(S), stream, ta, tw, p, S);
  return launch_status("split_kernel");
}

// ---------------------------------------------------------------------------
// Wide kernel: 256 tokens x 256 features per pair of CTAs (cta_group::2).
//
// One SM alone would move 48 KB into and out of its shared memory for every
// 128 x 256 x 128 block, about 750 cycles of its port against 512 of the tensor
// core.  The pair splits the weight tile: each SM stages its own 128 tokens and
// half of the 256 features (32 KB) and multiplies against both halves, so the
// port needs no longer than the MMA.  Tokens are the M side: a lane is a token,
// whose factor a_scale * w_scale is one scalar per block of K.  Persistent: a
// pair walks the tiles, and the epilogue's store of one tile overlaps the first
// blocks of the next.
//
// 16,384 x 7,168 x 12,288 in 0.93 to 0.95 ms by the box, 3.0 to 3.1 PFLOP/s (1.04 ms
// in a row of 600 calls, at the power cap's 1.7 GHz); a library product of the same
// codes with one scale for the whole matrix takes 0.77 to 0.83 ms.  A block takes
// about 780 cycles of a pair, its MMAs 512: the rest is the chain through the two
// TMEM buffers (all 512 columns): commit, the epilogue's 128 columns a thread, the
// buffer's return to the issuing CTA.  A third buffer would need a narrower tile,
// and the MMAs of one take as long per feature (128 features: 418 cycles).
// ---------------------------------------------------------------------------
enum : uint32_t { SITE_P_E = 0x710, SITE_P_F = 0x711, SITE_P_ACC = 0x712, SITE_P_FREE = 0x713,
                  SITE_P_DRAIN = 0x714, SITE_P_FACT = 0x715 };

struct Wide {
  static constexpr int NST = 4;
  static constexpr int STAGE = 2 * 128 * 128;            // 128 tokens, 128 features
  static constexpr int EW = 8;                           // epilogue warps 0..7, two warpgroups
  static constexpr int NTHREADS = EW * 32 + 128;         // and one warpgroup for copies and MMA
  static constexpr int BOX = 32 * 128;                   // 32 tokens x 128 bytes of out
  static constexpr int OFF_OUT = NST * STAGE;            // two boxes per epilogue warp
  static constexpr int OFF_MISC = OFF_OUT + EW * 2 * BOX;
  static constexpr int CH = 16;                          // blocks of K per set of factors
  static constexpr int FROW = 132;                       // 128 tokens, 2 weight blocks, padding
  static constexpr int FSET = CH * FROW;
  static constexpr int OFF_FACT = OFF_MISC + 256;
  static constexpr int NF = 2;                           // sets of factors
  static constexpr int SMEM = 1024 + OFF_FACT + NF * FSET * 4;
  static constexpr int GROUP = 8;                        // token tiles that share a weight sweep
};

// Tiles in groups of GROUP token tiles, token tiles fastest: the pairs at work
// at one time share few weight and token tiles, which stay in L2.
__device__ __forceinline__ void wide_tile(int tile, int ntm, int ntn, int& mt, int& nt) {
  const int per = Wide::GROUP * ntn, g = tile / per, rem = tile - g * per;
  const int gm = min(Wide::GROUP, ntm - g * Wide::GROUP);
  nt = rem / gm;
  mt = g * Wide::GROUP + rem - nt * gm;
}

// A lane's row of a 128-byte-swizzled box.
__device__ __forceinline__ void put_box_f32(uint8_t* box, int lane, const float* v) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    *reinterpret_cast<float4*>(box + sw128_unit(lane, u)) =
        make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
}
__device__ __forceinline__ void put_box_bf16(uint8_t* box, int lane, const float* v) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    *reinterpret_cast<uint4*>(box + sw128_unit(lane, u)) =
        make_uint4(pack_bf16x2(v[8 * u], v[8 * u + 1]), pack_bf16x2(v[8 * u + 2], v[8 * u + 3]),
                   pack_bf16x2(v[8 * u + 4], v[8 * u + 5]), pack_bf16x2(v[8 * u + 6], v[8 * u + 7]));
}

// The box's 32 rows to tokens m0 .. of out, features n .. (128 bytes of them), one
// row at a time: 4 bytes a lane, or 2 where rows start on 2-byte boundaries.
__device__ __forceinline__ void store_rows(const Params& p, const uint8_t* box, int m0, int n, int lane) {
  const int rows = min(32, p.M - m0);
  const int size = p.fp32 ? 4 : 2, width = row_bytes_left(p.N, n, size, 128);
  uint8_t* out = static_cast<uint8_t*>(p.out) + (static_cast<int64_t>(m0) * p.N + n) * size;
  const int64_t pitch = static_cast<int64_t>(p.N) * size;
  if (pitch % 4 == 0) {
#pragma unroll 8
    for (int r = 0; r < rows; ++r)
      if (lane * 4 < width)
        *reinterpret_cast<uint32_t*>(out + r * pitch + lane * 4) =
            *reinterpret_cast<const uint32_t*>(box + sw128_unit(r, lane >> 2) + (lane & 3) * 4);
  } else {
#pragma unroll 8
    for (int r = 0; r < rows; ++r)
#pragma unroll
      for (int c = lane * 2; c < 128; c += 64)
        if (c < width)
          *reinterpret_cast<uint16_t*>(out + r * pitch + c) =
              *reinterpret_cast<const uint16_t*>(box + sw128_unit(r, c >> 4) + (c & 15));
  }
}

// TMA: rows of out start on 16-byte boundaries, so that TMA can store it.
template <bool TMA>
__global__ void __launch_bounds__(Wide::NTHREADS, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_out, const Params p) {
  using C = Wide;
  constexpr uint32_t IDESC = idesc_e4m3(256, 256);
  extern __shared__ uint8_t smem_raw[];
  cluster_arrive_relaxed();
  uint8_t* sm = smem_align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OFF_MISC);   // used in the even CTA
  uint64_t* done = full + C::NST;      // a stage's MMAs are complete: it is empty and its block summed
  uint64_t* acc_free = done + C::NST;                                // used in the even CTA
  uint64_t* f_full = acc_free + 2;
  uint64_t* f_free = f_full + C::NF;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(f_free + C::NF);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tslot + 1);
  int* s_far = reinterpret_cast<int*>(tslot + 2);   // per set and staging warp: far factors
  float* fact = reinterpret_cast<float*>(sm + C::OFF_FACT);

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int rank = blockIdx.x & 1;
  const int ntm = (p.M + 255) / 256, ntn = (p.N + 255) / 256;
  const int ntiles = ntm * ntn, step = gridDim.x >> 1;

  if (tid == 0) {
    for (int k = 0; k < 2 * C::NST; ++k) mbar_init(&full[k], 1);
    for (int k = 0; k < 2; ++k) mbar_init(&acc_free[k], 2 * C::EW);
    for (int k = 0; k < C::NF; ++k) {
      mbar_init(&f_full[k], 2);                                      // the two staging warps
      mbar_init(&f_free[k], C::EW);
    }
    s_abort[0] = 0;
    fence_mbar_init();
  }
  __syncwarp();
  cluster_wait();                      // the other CTA runs
  if (warp == C::EW + 1) {
    tmem_alloc_pair(tslot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = uniform(*tslot);
  pdl_wait();
  pdl_start_next();

  if (warp >= C::EW) {
    regs_dec<56>();
    if (warp == C::EW) {
      if (elect_one_lane()) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_w);
        if (TMA) tma_prefetch_desc(&tm_out);
      }
      __syncwarp();
      int st = 0, i = 0;
      uint32_t ph = 0;       // parity of the stage's current use
      bool ok = true;
      for (int tile = blockIdx.x >> 1; ok && tile < ntiles; tile += step) {
        int mt, nt;
        wide_tile(tile, ntm, ntn, mt, nt);
        for (int b = 0; b < p.kb; ++b) {
          ok = (i < C::NST || mbar_wait(&done[st], ph ^ 1, p.status, kWaitLimitNs, SITE_P_E)) &&
               !s_abort[0];
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* a = sm + st * C::STAGE;
          if (elect_one_lane()) {
            if (rank == 0) mbar_expect_tx(&full[st], 2 * C::STAGE);   // both CTAs' bytes
            const uint32_t bar = mapa_u32(smem_u32(&full[st]), 0);
            tma_load_2d_pair(a, &tm_a, bar, 64 * b, mt * 256 + rank * 128);
            tma_load_2d_pair(a + 128 * 128, &tm_w, bar, 64 * b, nt * 256 + rank * 128);
          }
          __syncwarp();
          if (i < C::NST) ++i;
          if (++st == C::NST) st = 0, ph ^= 1;
        }
      }
      if (!ok) s_abort[0] = 1;
      // the pair's copies in flight (the last i uses of the ring) have landed
      // before either CTA leaves
      if (rank == 0)
        for (; i > 0; --i) {
          if (--st < 0) st = C::NST - 1, ph ^= 1;
          mbar_wait(&full[st], ph, p.status, kWaitLimitNs, SITE_P_F);
        }
    } else if (warp == C::EW + 1 && rank == 0) {
      const uint64_t desc0 = smem_desc(smem_u32(sm), 16, 1024);
      int st = 0, i = 0;
      uint32_t ph = 0, fph = 1, bu = 0;
      bool ok = true;
      for (int tile = blockIdx.x >> 1; ok && tile < ntiles; tile += step) {
        for (int b = 0; b < p.kb; ++b) {
          ok = mbar_wait(&full[st], ph, p.status, kWaitLimitNs, SITE_P_F) &&
               (i < 2 || mbar_wait(&acc_free[bu], fph, p.status, kWaitLimitNs, SITE_P_FREE));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = desc_add(desc0, st * C::STAGE), wd = desc_add(ad, 128 * 128);
          if (elect_one_lane()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_e4m3_pair(tmem + bu * 256, desc_add(ad, kk * 32), desc_add(wd, kk * 32), IDESC,
                             kk ? 1u : 0u);
            umma_commit_pair(&done[st]);
          }
          __syncwarp();
          if (i < C::NST) ++i;
          if (bu) fph ^= 1;
          bu ^= 1;
          if (++st == C::NST) st = 0, ph ^= 1;
        }
      }
      if (!ok) s_abort[0] = 1;
      // every MMA issued has finished before the stages or the TMEM are given up
      for (; i > 0; --i) {
        if (--st < 0) st = C::NST - 1, ph ^= 1;
        mbar_wait(&done[st], ph, p.status, kWaitLimitNs, SITE_P_DRAIN);
      }
    } else if (warp >= C::EW + 2) {
      // Factors: sets of CH blocks of K, in a ring of NF; each of two warps stages
      // 64 tokens.  CH lanes read CH neighbouring scales of a token, the warp RP
      // tokens a load, 16 loads in flight (a set's latency is what a tile of few
      // blocks waits for).
      constexpr int RP = 32 / C::CH;
      static_assert(RP >= 2, "a lane for each of the two weight blocks");
      const int fk = lane % C::CH, fr = lane / C::CH, first = (warp - (C::EW + 2)) * 64;
      int ch = 0;
      bool ok = true;
      for (int tile = blockIdx.x >> 1; ok && tile < ntiles; tile += step) {
        int mt, nt;
        wide_tile(tile, ntm, ntn, mt, nt);
        const int m0 = mt * 256 + rank * 128 + fr;
        const float* as = p.a_scale + static_cast<int64_t>(m0) * p.kb + fk;
        for (int b = 0; b < p.kb; b += C::CH, ++ch) {
          const int fs = ch % C::NF;
          ok = ch < C::NF ||
               mbar_wait(&f_free[fs], (ch / C::NF - 1) & 1, p.status, kWaitLimitNs, SITE_P_FACT);
          ok = __all_sync(0xffffffffu, ok) && !s_abort[0];
          if (!ok) break;
          float* to = fact + fs * C::FSET + fk * C::FROW + fr;
          const bool in = b + fk < p.kb;
          const float* wsc = p.w_scale + static_cast<int64_t>(nt * 2) * p.kb + b + fk;
          const float w0 = in ? wsc[0] : 1.f, w1 = in && nt * 256 + 128 < p.N ? wsc[p.kb] : 1.f;
          Span span;
#pragma unroll 1
          for (int r0 = first; r0 < first + 64; r0 += 16 * RP) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int r = r0 + RP * k;
              v[k] = in && m0 + r < p.M ? as[static_cast<int64_t>(r) * p.kb + b] : 1.f;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) to[r0 + RP * k] = v[k];
            span.add(v);
          }
          if (first == 0 && fr < 2) to[128] = fr == 0 ? w0 : w1;
          const bool any_far = __any_sync(0xffffffffu, !span.normal_times(w0) || !span.normal_times(w1));
          if (lane == 0) s_far[fs * 2 + (first != 0)] = any_far;
          mbar_arrive_warp(&f_full[fs]);
        }
      }
      if (!ok) s_abort[0] = 1;
    }
    __syncwarp();
  } else {
    regs_inc<224>();
    const int sub = warp & 3, half = warp >> 2, row = sub * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(sub * 32) << 16) + half * 128;
    const uint32_t free0 = mapa_u32(smem_u32(&acc_free[0]), 0);
    // The block's columns leave TMEM in two halves; only the first half's sums
    // stand between the block's completion and the buffer's return, the second
    // half's overlap the wait for the next block.  A lane that gave up keeps its
    // warp together until the vote at the next set of factors.
    int st = 0, fs = 0, bu = 0;
    uint32_t ph = 0, fph = 0;
    bool ok = true, live = true;   // live: the same in all lanes
    for (int tile = blockIdx.x >> 1; live && tile < ntiles; tile += step) {
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.f;
#pragma unroll 1
      for (int b = 0; b < p.kb; b += C::CH) {
        ok = ok && mbar_wait(&f_full[fs], fph, p.status, kWaitLimitNs, SITE_P_FACT);
        live = ok = __all_sync(0xffffffffu, ok);
        if (!live) break;
        const float* fb = fact + fs * C::FSET;
        const float* const fe = fb + min(C::CH, p.kb - b) * C::FROW;
        auto add_block = [&](auto FAR) {
          const float fa = fb[row], fw = fb[128 + half];
          ok = ok && mbar_wait(&done[st], ph, p.status, kWaitLimitNs, SITE_P_ACC);
          __syncwarp();
          tc_fence_after();
          Factor f{1.f, fa * fw};
          if constexpr (FAR.value) f = factor(fa, fw);
          const uint32_t ta = taddr + bu * 256;
          uint32_t d[2][32];
          auto add = [&](int c, uint32_t (&x)[32]) {
            if constexpr (FAR.value) {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f.pre);
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              fma2_rn(acc[c + e], acc[c + e + 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]),
                      f.mul, f.mul);
          };
          tmem_ld32(ta, d[0]);
          tmem_ld32(ta + 32, d[1]);
          tmem_ld_wait_regs(d[0]);
          tmem_ld_wait_regs(d[1]);
          add(0, d[0]);
          tmem_ld32(ta + 64, d[0]);
          add(32, d[1]);
          tmem_ld32(ta + 96, d[1]);
          tmem_ld_wait_regs(d[0]);
          tmem_ld_wait_regs(d[1]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (rank == 0)
              mbar_arrive(&acc_free[bu]);
            else
              mbar_arrive_cluster_relaxed(free0 + bu * 8);
          }
          add(64, d[0]);
          add(96, d[1]);
          bu ^= 1;
          if (++st == C::NST) st = 0, ph ^= 1;
          fb += C::FROW;
        };
        const int2 far = reinterpret_cast<const int2*>(s_far)[fs];
        if ((far.x | far.y) == 0) {
#pragma unroll 1
          do add_block(std::false_type{});
          while (fb != fe);
        } else {
#pragma unroll 1
          do add_block(std::true_type{});
          while (fb != fe);
        }
        mbar_arrive_warp(&f_free[fs]);
        if (++fs == C::NF) fs = 0, fph ^= 1;
      }
      int mt, nt;
      wide_tile(tile, ntm, ntn, mt, nt);
      const int m = mt * 256 + rank * 128 + row, n = nt * 256 + half * 128;
      if (live) {
        // A box of 128 bytes of 32 tokens at a time through this warp's shared
        // memory and out by TMA, or, where rows of out do not start on 16-byte
        // boundaries, row by row.  Stored straight from the registers, 16 bytes
        // of 32 different rows at a time, a tile's output took 7,000 cycles.
        const int m0 = m - lane, per = p.fp32 ? 32 : 64;     // features per box
        for (int q = 0; q < 128 / per; ++q) {
          uint8_t* box = sm + C::OFF_OUT + (warp * 2 + (q & 1)) * C::BOX;
          const int nq = n + q * per;
          if (TMA && lane == 0) bulk_wait_read<1>();         // the box's last store has read it
          __syncwarp();
          if (p.fp32) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              if (q == s) put_box_f32(box, lane, acc + 32 * s);
          } else {
#pragma unroll
            for (int s = 0; s < 2; ++s)
              if (q == s) put_box_bf16(box, lane, acc + 64 * s);
          }
          if constexpr (TMA) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (m0 < p.M && nq < p.N) tma_store_2d(&tm_out, box, nq, m0);
              bulk_commit();
            }
          } else {
            __syncwarp();
            store_rows(p, box, m0, nq, lane);
          }
        }
      }
    }
    if (TMA && lane == 0) bulk_wait_all();
    __syncwarp();
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) s_abort[0] = 1;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the pair's MMAs, copies and TMEM reads are done
  if (warp == C::EW + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

dsa_status_t launch_wide(const LinearArgs& a, cudaStream_t stream) {
  using C = Wide;
  CUtensorMap ta, tw, to;
  const uint64_t K = static_cast<uint64_t>(a.K), N = static_cast<uint64_t>(a.N);
  // the output goes out by TMA where its rows start on 16-byte boundaries
  const bool by_tma = N * (a.fp32 ? 4 : 2) % 16 == 0;
  if (!encode_tmap_2d(&ta, a.a, a.M, K / 2, K, 64, 128, true) ||
      !encode_tmap_2d(&tw, a.w, a.N, K / 2, K, 64, 128, true))
    return DSA_ERR_CUDA;
  if (!by_tma)
    to = ta;   // not used
  else if (!(a.fp32 ? encode_tmap_2d_f32(&to, a.out, a.M, N, 4 * N, 32, 32, true)
                    : encode_tmap_2d(&to, a.out, a.M, N, 2 * N, 64, 32, true)))
    return DSA_ERR_CUDA;
  const Params p{a.a_scale, a.w_scale, a.M, a.N, (a.K + 127) / 128, a.out, a.fp32, a.status};
  const auto kernel = by_tma ? wide_kernel<true> : wide_kernel<false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return launch_status("cudaFuncSetAttribute");
  const int64_t tiles = static_cast<int64_t>((a.M + 255) / 256) * ((a.N + 255) / 256);
  const int64_t pairs = num_sms() / 2;
  launch_overlapped(kernel, static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)), C::NTHREADS,
                    C::SMEM, 2, stream, ta, tw, to, p);
  return launch_status("wide_kernel");
}

}  // namespace lin

dsa_status_t quant_fp8_weight_launch(const uint16_t* w, int N, int K, uint8_t* codes, float* scale,
                                     cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((K + 127) / 128) * static_cast<unsigned>((N + 127) / 128);
  launch_overlapped(lin::quant_weight_kernel, grid, 256, 0, 0, stream, w, N, K, codes, scale);
  return launch_status("quant_weight_kernel");
}

dsa_status_t linear_fp8_launch(const LinearArgs& a, const lin::Pick* forced, cudaStream_t stream) {
  auto launch = [&](const lin::Pick& at) {
    switch (at.nt) {
      case 16: return lin::launch_split<16>(a, at.S, stream);
      case 32: return lin::launch_split<32>(a, at.S, stream);
      case 64: return lin::launch_split<64>(a, at.S, stream);
      case 96: return lin::launch_split<96>(a, at.S, stream);
      case 128: return lin::launch_split<128>(a, at.S, stream);
      default: return lin::launch_wide(a, stream);
    }
  };
  if (forced != nullptr) return launch(*forced);
  dsa_status_t st = DSA_OK;
  lin::take_one_that_fits(a.M, a.N, (a.K + 127) / 128, num_sms(),
                          static_cast<int64_t>(a.N) * (a.fp32 ? 4 : 2), [&](const lin::Pick& at) {
                            st = launch(at);
                            return st != DSA_ERR_UNSUPPORTED;
                          });
  return st;
}

}  // namespace dsa
