// mla_window_bwd.cu -- backward pass of windowed dense attention over latent rows.
//
// Given the forward's o_lat and lse, and d_o, with z as there:
//   p_s = exp(z_s - lse),  D = d_o . o_lat,  dz_s = scale * p_s (d_o . KV[s, 0:512] - D)
//   dq = sum_s dz_s KV[s, :],   dkv[s] = sum over the queries that see s of dz_s q + p_s d_o
//
// The (query, head) rows of a sequence are packed into tiles of 128; a tile sees a
// list of pages (64 rows of the cache).  P and dZ of a (tile, page) are 128 x 64 BF16
// blocks in the workspace, 128-byte swizzled as the tensor core reads them (rows of
// 64 keys), so each product below takes them by plain box copies in either order.
//   prep     D and lse (base 2) of every row
//   pz       [S^T | dP^T] [256 keys x (128 + 128)] = K . [Q | dO]^T for a tile and four
//            of its pages: one MMA, M = 256, N = 256 on a pair of CTAs, of which the
//            even one holds the tile's q and the odd one its d_o (and zeros for the
//            rotated dims, which have no value part), so neither needs room for both.
//            A thread has a key and both of its products with a row: p and dz need
//            no exchange.  Blocks leave from registers.
//   product  dq: [256 rows x 256 or 320 dims] = dZ . K over the pages of two tiles;
//            dkv: [256 keys x 256 or 320 dims] = dZ^T . q + P^T . dO over those tiles of
//            a segment that see the keys.  M = 256 on a pair of CTAs; the 576 dims are
//            two tasks (0..255; 256..575), as 512 TMEM columns do not hold them.
//   reduce   dkv's segments, added in order (no atomics: equal calls give equal bits)
// dkv's tasks stand in the order of the segments, so that the key tiles that see a
// segment run through its q and d_o at the same time and read them from L2 (by key
// tile they came from HBM for each: 5.5 GB instead of 2.7 at 4096 tokens x 96 heads,
// window 1024, and 0.88 ms at 6.4 TB/s).  pz and dq are persistent (dkv's tasks differ
// in length and are dealt out as SMs fall free): the next task's
// copies (pz: of its q and d_o too, chunk by chunk beside the first keys) and first
// products run while the last one's results are written out.
// Tiles go in chunks where P and dZ of all would take more than kChunkBytes.
// P and dZ are rounded to BF16 once, whatever the call's sizes: each of the products that
// add up to a gradient is off by up to 2^-8, independently, so that dq and dkv are off by
// sqrt(2) times their own final rounding (root mean square; 1.0 to 1.7 times for a few rows
// of a few keys).  A second BF16 number for what that leaves would double what the products
// multiply, 1,664 of a pair's 2,816 dims, and P and dZ in the workspace.
#include <cmath>

#include <cuda_bf16.h>

#include "dense_mask.cuh"
#include "dense_pair.cuh"

namespace dsa {
namespace wbw {

using namespace dense;

constexpr int X = 128;                              // rows of a tile
constexpr int BLOCK = X * 128;                      // bytes of a block: 128 rows x 64 keys
constexpr int64_t kChunkBytes = int64_t(4) << 30;   // P and dZ at a time
constexpr int TASKS = 600;                          // dkv tasks aimed at: about eight a pair of SMs

enum : uint32_t {
  SITE_KF = 0x721, SITE_KE = 0x722, SITE_AF = 0x723, SITE_AE = 0x724,
  SITE_F = 0x725, SITE_E = 0x726, SITE_LAND = 0x727, SITE_DONE = 0x728,
  SITE_DF = 0x72a
};

struct Plan {
  int RT, RC, np;        // tiles of a sequence, of a chunk; pages a tile may see at most
  int KT, KF;            // tiles of 256 keys; those that hold first tokens
  int seg, G, nk;        // tiles of a segment; segments of a chunk; key tiles that a segment's
                         // windows reach
  __host__ __device__ int per_seg() const { return nk + KF; }
};

struct Params {
  Store kv;
  Mask m;
  int B, H;
  Plan q;
  int rt0;               // first tile of the chunk
  float scale, scale_log2;
  const uint16_t* o;
  const uint16_t* d_o;
  const float* lse;
  float2* rows;          // [B, T * H] lse (base 2), D
  uint8_t* pz;           // a block of zeros, then [B, RC, np, P | dZ] blocks
  float* part;           // [B, G, nk + KF, 256, 576]
  float* acc;            // [B, max_kv_len, 576] between chunks
  uint16_t* dq;
  uint16_t* dkv;
  int first_chunk, last_chunk;
  uint32_t* status;

  // first row (128 bytes each) of a block in the workspace's tensor map; which: P, dZ
  __device__ __forceinline__ int64_t block_row(int b, int rt, int k, int which) const {
    return X + (((static_cast<int64_t>(b) * q.RC + rt - rt0) * q.np + k) * 2 + which) * X;
  }
};

__device__ __forceinline__ Pages tile_pages(const Params& p, const Seq& s, int rt) {
  const int rows = s.n * p.H, g = rt * X;
  if (g >= rows) return Pages{0, 0, 0};
  return pages_of(p.m, s, g / p.H, (min(g + X, rows) - 1) / p.H);
}
// Where a page stands in a list, or -1.
__device__ __forceinline__ int place(const Pages& l, int pg) {
  return pg < l.head ? pg : pg >= l.tail && pg < l.end ? l.head + pg - l.tail : -1;
}
// The chunk's tiles that see some of the keys 256 kt .. 256 kt + 255.
__device__ __forceinline__ int2 tiles_of(const Params& p, const Seq& s, int kt) {
  const int64_t s0 = 256ll * kt;
  const int64_t n = min(s.n, s.L - s.pos0);
  int64_t lo = max(s0 - s.pos0, int64_t(0));
  int64_t hi = s0 < p.m.n_first ? n : min(n, s0 + 255 + p.m.window - s.pos0);
  if (!s.ok || lo >= hi) return make_int2(0, 0);
  lo = max(lo * p.H / X, static_cast<int64_t>(p.rt0));
  hi = min((hi * p.H + X - 1) / X, static_cast<int64_t>(p.rt0 + p.q.RC));
  return lo < hi ? make_int2(static_cast<int>(lo), static_cast<int>(hi)) : make_int2(0, 0);
}
// The first key tile that the windows of segment g reach.
__device__ __forceinline__ int first_key_tile(const Params& p, const Seq& s, int g) {
  const int t = s.pos0 + (p.rt0 + g * p.q.seg) * X / p.H;
  return max(t - p.m.window + 1, 0) >> 8;
}
// Where the sums of segment g for key tile kt stand: the windows' key tiles, then those
// of first tokens that no window reaches.
__device__ __forceinline__ int64_t part_row(const Params& p, const Seq& s, int b, int g, int kt) {
  const int k0 = first_key_tile(p, s, g);
  const int at = kt >= k0 ? kt - k0 : p.q.nk + kt;
  return ((static_cast<int64_t>(b) * p.q.G + g) * p.q.per_seg() + at) * 256;
}

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// A warp per row; also the block of zeros.
__global__ void __launch_bounds__(256) prep_kernel(const Params p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_start_next();
  if (blockIdx.x < BLOCK / (256 * 16))
    reinterpret_cast<uint4*>(p.pz)[blockIdx.x * 256 + threadIdx.x] = make_uint4(0, 0, 0, 0);
  const int per = p.m.T * p.H;
  if (row >= static_cast<int64_t>(p.B) * per) return;
  if (row % per == 0 && lane == 0) {
    const int b = static_cast<int>(row / per);
    report_seq(p.m, seq_of(p.m, b), b, p.status);
  }
  const uint4* x = reinterpret_cast<const uint4*>(p.o + row * kVlat) + lane;
  const uint4* y = reinterpret_cast<const uint4*>(p.d_o + row * kVlat) + lane;
  float d = 0.f;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint4 a = x[32 * c], g = y[32 * c];
    d = fmaf(lo_f(a.x), lo_f(g.x), fmaf(hi_f(a.x), hi_f(g.x), d));
    d = fmaf(lo_f(a.y), lo_f(g.y), fmaf(hi_f(a.y), hi_f(g.y), d));
    d = fmaf(lo_f(a.z), lo_f(g.z), fmaf(hi_f(a.z), hi_f(g.z), d));
    d = fmaf(lo_f(a.w), lo_f(g.w), fmaf(hi_f(a.w), hi_f(g.w), d));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) p.rows[row] = make_float2(p.lse[row] * 1.4426950408889634f, d);
}

// ---------------------------------------------------------------------------
// pz
// ---------------------------------------------------------------------------
struct Pz {
  static constexpr int NS = 4;                       // slots: 64 dims of 128 keys
  static constexpr int OFF_B = 0;                    // q or d_o of the tile: 9 chunks of 128 rows
  static constexpr int OFF_K = 9 * BLOCK;
  static constexpr int OFF_ROW = OFF_K + NS * BLOCK;
  static constexpr int OFF_MISC = OFF_ROW + 2 * X * 16;
  static constexpr int SMEM = OFF_MISC + 256 + 1024;
  static constexpr int THREADS = 384;                // 0 copies, 1 issues, 4..11 form P and dZ
  static_assert(SMEM <= 232448, "shared memory");
};

// A tile of the chunk and what it sees.
struct Tile {
  int b, rt, g0, rows;   // rows: of the sequence
  Seq s;
  Pages pages;
  int np, ng;            // pages, groups of four
};
__device__ __forceinline__ Tile tile_at(const Params& p, int task) {
  Tile t;
  t.b = task / p.q.RC;
  t.rt = p.rt0 + task % p.q.RC;
  t.s = seq_of(p.m, t.b);
  t.pages = tile_pages(p, t.s, t.rt);
  t.np = t.pages.count();
  t.ng = (t.np + 3) / 4;
  t.g0 = t.rt * X;
  t.rows = t.s.n * p.H;
  return t;
}

__global__ void __launch_bounds__(Pz::THREADS, 1)
    pz_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
              const __grid_constant__ CUtensorMap tm_kv, const Params p) {
  using C = Pz;
  constexpr uint32_t IDESC = idesc_bf16(256, 256, false, false);
  const int rank = blockIdx.x & 1, tasks = p.B * p.q.RC, step = gridDim.x >> 1;

  extern __shared__ uint8_t smem_raw[];
  cluster_arrive_relaxed();
  uint8_t* sm = smem_align1024(smem_raw);
  uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + C::OFF_MISC);   // even CTA
  uint64_t* kempty = kfull + C::NS;
  uint64_t* afull = kempty + C::NS;
  uint64_t* afree = afull + 2;                                       // even CTA
  uint64_t* drain = afree + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tslot + 1);
  float4* s_row = reinterpret_cast<float4*>(sm + C::OFF_ROW);        // [2][X] lse, D, position

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int k = 0; k < C::NS; ++k) mbar_init(&kfull[k], 1), mbar_init(&kempty[k], 1);
    for (int k = 0; k < 2; ++k) mbar_init(&afull[k], 1), mbar_init(&afree[k], 16);
    mbar_init(drain, 1);
    s_abort[0] = s_abort[1] = 0;
    fence_mbar_init();
    tma_prefetch_desc(rank == 0 ? &tm_q : &tm_do);
    tma_prefetch_desc(&tm_kv);
  }
  __syncwarp();
  cluster_wait();                                    // the other CTA runs
  if (warp == 1) {
    tmem_alloc_pair(tslot, 512);
    tmem_relinquish_pair();
  }
  if (rank == 1) {                                   // no value part for the rotated dims
    for (int e = tid; e < BLOCK / 16; e += C::THREADS)
      reinterpret_cast<uint4*>(sm + C::OFF_B + 8 * BLOCK)[e] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait();
  pdl_start_next();

  if (warp == 0) {
    Ring<C::NS> r;
    int used = 0;
    bool ok = true;
    for (int task = blockIdx.x >> 1; task < tasks && ok; task += step) {
      const Tile t = tile_at(p, task);
      for (int j = 0; j < t.ng && ok; ++j) {
        int row[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {                // pages that are not there: any rows
          const int k = 4 * j + 2 * rank + h;
          row[h] = static_cast<int>(page_row(p.kv, t.b, t.pages.page(k < t.np ? k : 0)));
        }
        for (int c = 0; c < 9; ++c) {
          // a tile's first keys bring its q and d_o along: the products that read the
          // last tile's chunk c came before those that free this slot
          ok = used < C::NS || wait(&kempty[r.slot], r.ph ^ 1, s_abort, p.status, SITE_KE);
          if (!ok) break;
          if (elect_one_lane()) {
            uint8_t* dst = sm + C::OFF_K + r.slot * BLOCK;
            const uint32_t bar = mapa_u32(smem_u32(&kfull[r.slot]), 0);
            if (rank == 0)
              mbar_expect_tx(&kfull[r.slot], (2 + (j > 0 ? 0 : c < 8 ? 2 : 1)) * BLOCK);
            if (j == 0 && (c < 8 || rank == 0))
              tma_load_3d_pair(sm + C::OFF_B + c * BLOCK, rank == 0 ? &tm_q : &tm_do, bar, 64 * c, t.g0, t.b);
            tma_load_2d_pair(dst, &tm_kv, bar, 64 * c, row[0]);
            tma_load_2d_pair(dst + CHUNK, &tm_kv, bar, 64 * c, row[1]);
          }
          __syncwarp();
          if (used < C::NS) ++used;
          r.next();
        }
      }
    }
    for (; used > 0; --used) {
      if (--r.slot < 0) r.slot = C::NS - 1, r.ph ^= 1;
      if (rank == 0) settle(&kfull[r.slot], r.ph);
      if (ok) settle(&kempty[r.slot], r.ph);
    }
  } else if (warp == 1 && rank == 0) {
    const uint64_t kd = smem_desc(smem_u32(sm + C::OFF_K), 16, 1024);
    const uint64_t bd = smem_desc(smem_u32(sm + C::OFF_B), 16, 1024);
    Ring<C::NS> r;
    int n = 0;                                       // groups so far
    bool ok = true;
    for (int task = blockIdx.x >> 1; task < tasks && ok; task += step) {
      const int ng = tile_at(p, task).ng;
      for (int j = 0; j < ng && ok; ++j, ++n) {
        const int bu = n & 1;
        if (n > 1) ok = wait(&afree[bu], ((n >> 1) - 1) & 1, s_abort, p.status, SITE_AE);
        tc_fence_after();
        for (int c = 0; c < 9 && ok; ++c) {
          ok = wait(&kfull[r.slot], r.ph, s_abort, p.status, SITE_KF);
          if (!ok) break;
          tc_fence_after();
          if (elect_one_lane()) {
            const uint64_t a = desc_add(kd, r.slot * BLOCK), w = desc_add(bd, c * BLOCK);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16_pair(tmem + bu * 256, desc_add(a, kk * 32), desc_add(w, kk * 32), IDESC,
                             c > 0 || kk > 0);
            umma_commit_pair(&kempty[r.slot]);
            if (c == 8) umma_commit_pair(&afull[bu]);
          }
          __syncwarp();
          r.next();
        }
      }
    }
    if (elect_one_lane()) umma_commit_pair_own(drain);
    __syncwarp();
    settle(drain, 0);
  } else if (warp >= 4) {
    // ---- a key a thread, 64 of the tile's rows a warp ----
    const int sub = warp & 3, r0 = (warp - 4) / 4 * 64, key = sub * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(sub * 32) << 16) + r0;
    const uint32_t free_bar = mapa_u32(smem_u32(afree), 0);
    const uint32_t unit = (key & 63) >> 3;
    const int mine = tid - 128;                      // a row of the tile for the first half of the threads
    auto row_at = [&](int task) {                    // lse, D and position of that row
      float4 v = make_float4(0.f, 0.f, __int_as_float(-1), 0.f);
      if (task < tasks && mine < X) {
        const int b = task / p.q.RC, g = (p.rt0 + task % p.q.RC) * X + mine;
        const Seq s = seq_of(p.m, b);
        if (g < s.n * p.H) {
          const float2 r = p.rows[static_cast<int64_t>(b) * p.m.T * p.H + g];
          const int t = s.pos0 + g / p.H;
          v = make_float4(r.x, r.y, __int_as_float(t < s.L ? t : -1), 0.f);
        }
      }
      return v;
    };
    float4 next = row_at(blockIdx.x >> 1);
    int n = 0, at = 0;
    bool ok = true;
    for (int task = blockIdx.x >> 1; task < tasks; task += step, at ^= 1) {
      const Tile t = tile_at(p, task);
      const float4* rows = s_row + at * X;
      if (mine < X) s_row[at * X + mine] = next;
      if (named_bar_or(1, 256, !ok)) break;          // rows written; two tiles back: read
      next = row_at(task + step);
      const int t0 = t.s.pos0 + t.g0 / p.H, t1 = t.s.pos0 + (min(t.g0 + X, t.rows) - 1) / p.H;
      const bool whole = t.g0 + X <= t.rows && t1 < t.s.L;
      for (int j = 0; j < t.ng && ok; ++j, ++n) {
        const int bu = n & 1, k = 4 * j + 2 * rank + (sub >> 1);
        const int kb = k < t.np ? t.pages.page(k) * 64 + (sub & 1) * 32 : 0;   // the warp's first key
        const int kp = kb + lane;
        const bool all = whole && kb + 31 <= t0 && (kb > t1 - p.m.window || kb + 31 < p.m.n_first);
        ok = wait(&afull[bu], (n >> 1) & 1, s_abort, p.status, SITE_AF);
        if (!ok) break;
        tc_fence_after();
        // the lane pair's two keys in the two blocks: row r at 128 r, 16-byte units xor r
        uint8_t* dst = p.pz + 128 * p.block_row(t.b, t.rt, k, 0) + (key & 6) * 2;
#pragma unroll 1
        for (int q = 0; q < 64; q += 16) {
          uint32_t z[16], dp[16];
          tmem_ld16(taddr + bu * 256 + q, z);
          tmem_ld16(taddr + bu * 256 + 128 + q, dp);
          tmem_ld_wait_regs(z);
          tmem_ld_wait_regs(dp);
          if (q == 48) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (rank == 0) mbar_arrive(&afree[bu]);
              else mbar_arrive_cluster_relaxed(free_bar + bu * 8);
            }
          }
          if (k < t.np) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int r = r0 + q + e;
              const float2 w = *reinterpret_cast<const float2*>(&rows[r]);
              float pr = ex2(fmaf(__uint_as_float(z[e]), p.scale_log2, -w.x));
              float dz = p.scale * pr * (__uint_as_float(dp[e]) - w.y);
              if (!all) {
                const int tt = __float_as_int(rows[r].z);
                const bool sees = kp <= tt && (tt - kp < p.m.window || kp < p.m.n_first);
                pr = sees ? pr : 0.f;
                dz = sees ? dz : 0.f;
              }
              // two rows of a key become two keys of a row, between two lanes: 4-byte
              // stores (2-byte ones: pz 0.10 ms more at 4096 tokens)
              z[e] = pack_bf16x2(pr, dz);
              if (e & 1) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 1 ? z[e - 1] : z[e], 1);
                const uint32_t k0 = lane & 1 ? got : z[e - 1], k1 = lane & 1 ? z[e] : got;
                const int rr = r - 1 + (lane & 1);
                uint8_t* to = dst + rr * 128 + ((unit ^ (rr & 7)) << 4);
                *reinterpret_cast<uint32_t*>(to) = __byte_perm(k0, k1, 0x5410);
                *reinterpret_cast<uint32_t*>(to + BLOCK) = __byte_perm(k0, k1, 0x7632);
              }
            }
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
struct Prod {
  static constexpr int NS = 5;
  static constexpr int OFF_W = 2 * CHUNK;            // in a stage: A 16 KB, then 64 x 128 dims, then 64 more
  static constexpr int STAGE = 5 * CHUNK;
  static constexpr int OFF_MISC = NS * STAGE;
  static constexpr int SMEM = OFF_MISC + 256 + 1024;
  static constexpr int THREADS = 384;                // 0 copies, 1 issues, 4..11 write out
};

// Columns c of D are dims 256 * upper + c, in TMEM columns c or (upper) 192 + c: the
// next task's products may start once the 64 columns that both use have been read.
// The rotated dims are an MMA of their own, N = 64, 32 dims from each CTA.
// dkv: of a stage's 64 rows, the first products take dZ and q, the second P and d_o.
template <bool DKV>
struct Task {
  int b, upper, kt, g, x0, x1;   // dkv: tiles x0..x1-1 of segment g; dq: tiles x0, x0 + 1
  Seq s;
  Pages list;                    // dq: pages of the two tiles
  bool there;

  // n: tasks that the pair has had so far.  Its dims alternate; of two neighbouring pairs,
  // which have the same rows throughout, one has the upper ones.
  __device__ __forceinline__ Task(const Params& p, int task, int n) {
    upper = (task ^ n) & 1;
    int u = task >> 1;
    kt = g = 0;
    list = Pages{0, 0, 0};
    if constexpr (DKV) {
      const int at = u % p.q.per_seg();
      u /= p.q.per_seg();
      g = u % p.q.G;
      b = u / p.q.G;
      s = seq_of(p.m, b);
      const int k0 = first_key_tile(p, s, g);
      kt = at < p.q.nk ? k0 + at : at - p.q.nk;
      there = s.ok && kt < p.q.KT && (at < p.q.nk || kt < k0);
      const int2 tiles = there ? tiles_of(p, s, kt) : make_int2(0, 0);
      x0 = max(tiles.x, p.rt0 + g * p.q.seg);
      x1 = min(tiles.y, p.rt0 + (g + 1) * p.q.seg);
      there = x0 < x1;
    } else {
      b = u / (p.q.RC / 2);
      x0 = p.rt0 + 2 * (u % (p.q.RC / 2));
      x1 = x0 + 2;
      s = seq_of(p.m, b);
      const int rows = s.n * p.H;
      there = x0 * X < rows;
      if (there) list = pages_of(p.m, s, x0 * X / p.H, (min(x1 * X, rows) - 1) / p.H);
    }
  }
  // dkv: whether a tile sees any of the task's keys
  __device__ __forceinline__ bool sees(const Pages& l) const {
    return place(l, 4 * kt) >= 0 || place(l, 4 * kt + 1) >= 0 || place(l, 4 * kt + 2) >= 0 ||
           place(l, 4 * kt + 3) >= 0;
  }
  // Whether there is anything to add up.
  __device__ __forceinline__ bool some(const Params& p) const {
    if constexpr (DKV) {
      for (int x = x0; x < x1; ++x)
        if (sees(tile_pages(p, s, x))) return true;
      return false;
    }
    return list.count() > 0;
  }
};

// The tasks first, first + step, ... of one kind.
template <bool DKV>
__device__ __forceinline__ void product(const CUtensorMap& tm_pz, const CUtensorMap& tm_kv, const CUtensorMap& tm_q,
                                        const CUtensorMap& tm_do, const Params& p, uint8_t* sm, int first,
                                        int step, int tasks) {
  using C = Prod;
  constexpr uint32_t IDESC = idesc_bf16(256, 256, DKV, true), IDESC_ROT = idesc_bf16(256, 64, DKV, true);
  const int rank = blockIdx.x & 1;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OFF_MISC);    // even CTA
  uint64_t* empty = full + C::NS;
  uint64_t* land = empty + C::NS;
  uint64_t* done = land + 1;                                         // a task's sums are complete
  uint64_t* dfree = done + 1;                                        // even CTA: and those that the next uses read
  uint64_t* drain = dfree + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tslot + 1);

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int k = 0; k < C::NS; ++k) mbar_init(&full[k], 2), mbar_init(&empty[k], 1);
    mbar_init(land, 1);
    mbar_init(done, 1);
    mbar_init(dfree, 16);
    mbar_init(drain, 1);
    s_abort[0] = s_abort[1] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_pz);
    tma_prefetch_desc(DKV ? &tm_q : &tm_kv);
    if (DKV) tma_prefetch_desc(&tm_do);
  }
  __syncwarp();
  cluster_wait();                                    // the other CTA runs
  if (warp == 1) {
    tmem_alloc_pair(tslot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait();
  pdl_start_next();

  if (warp == 0) {
    Ring<C::NS> r;
    int used = 0, n = 0;
    uint32_t lph = 0;
    bool ok = true;
    auto acquire = [&] {
      ok = used < C::NS || wait(&empty[r.slot], r.ph ^ 1, s_abort, p.status, SITE_E);
      return ok;
    };
    auto advance = [&] {
      __syncwarp();
      if (used < C::NS) ++used;
      r.next();
    };
    for (int task = first; task < tasks && ok; task += step) {
      const Task<DKV> t(p, task, n);
      if (!t.there) continue;
      ++n;
      const int col = 256 * t.upper + 128 * rank;
      if constexpr (DKV) {
        for (int x = t.x0; x < t.x1 && ok; ++x) {
          const Pages l = tile_pages(p, t.s, x);
          if (!t.sees(l)) continue;
          const int c0 = place(l, 4 * t.kt + 2 * rank), c1 = place(l, 4 * t.kt + 2 * rank + 1);
#pragma unroll 1
          for (int st = 0; st < 4 && ok; ++st) {     // dZ and q or P and d_o, 64 rows
            const int dz = 1 - (st & 1), y = 64 * (st >> 1);
            if (!acquire()) break;
            if (elect_one_lane()) {
              uint8_t* a = sm + r.slot * C::STAGE;
              uint8_t* w = a + C::OFF_W;
              const uint32_t bar = mapa_u32(smem_u32(&full[r.slot]), 0);
              const bool rot = t.upper && dz;
              mbar_expect_tx_cluster(bar, (rot ? 5 : 4) * CHUNK);
              tma_load_2d_pair(a, &tm_pz, bar, 0,
                               c0 < 0 ? 0 : static_cast<int>(p.block_row(t.b, x, c0, dz)) + y);
              tma_load_2d_pair(a + CHUNK, &tm_pz, bar, 0,
                               c1 < 0 ? 0 : static_cast<int>(p.block_row(t.b, x, c1, dz)) + y);
              const CUtensorMap* tm = dz ? &tm_q : &tm_do;
              tma_load_3d_pair(w, tm, bar, col, x * X + y, t.b);
              tma_load_3d_pair(w + CHUNK, tm, bar, col + 64, x * X + y, t.b);
              if (rot) tma_load_3d_pair(w + 2 * CHUNK, tm, bar, kVlat + 32 * rank, x * X + y, t.b);
            }
            advance();
          }
        }
      } else {
        const Pages l = tile_pages(p, t.s, t.x0 + rank);
        for (int k = 0; k < t.list.count() && ok; ++k) {
          const int pg = t.list.page(k), c = place(l, pg), row = static_cast<int>(page_row(p.kv, t.b, pg));
          const uint64_t any = range_bits(0, t.s.L, pg * 64);
          if (!acquire()) break;
          uint8_t* a = sm + r.slot * C::STAGE;
          uint8_t* w = a + C::OFF_W;
          const uint32_t bar = mapa_u32(smem_u32(&full[r.slot]), 0);
          const bool rot = t.upper;
          const int boxes = rot ? 3 : 2;
          if (any != ~0ull) {
            // rows behind the sequence become zeros: whatever they hold must not meet
            // the zeros of dZ
            if (elect_one_lane()) {
              mbar_expect_tx(land, boxes * CHUNK);
              tma_load_2d(w, &tm_kv, land, col, row);
              tma_load_2d(w + CHUNK, &tm_kv, land, col + 64, row);
              if (rot) tma_load_2d(w + 2 * CHUNK, &tm_kv, land, kVlat + 32 * rank, row);
            }
            __syncwarp();
            ok = wait(land, lph, s_abort, p.status, SITE_LAND);
            lph ^= 1;
            if (!ok) break;
            for (int e = lane; e < boxes * CHUNK / 16; e += 32)
              if (!(any >> ((e >> 3) & 63) & 1)) reinterpret_cast<uint4*>(w)[e] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (elect_one_lane()) {
            if (any == ~0ull) {
              mbar_expect_tx_cluster(bar, (2 + boxes) * CHUNK);
            } else {
              mbar_expect_tx_cluster_release(bar, 2 * CHUNK);
            }
            const int br = c < 0 ? 0 : static_cast<int>(p.block_row(t.b, t.x0 + rank, c, 1));
            tma_load_2d_pair(a, &tm_pz, bar, 0, br);
            tma_load_2d_pair(a + CHUNK, &tm_pz, bar, 0, br + 64);
            if (any == ~0ull) {
              tma_load_2d_pair(w, &tm_kv, bar, col, row);
              tma_load_2d_pair(w + CHUNK, &tm_kv, bar, col + 64, row);
              if (rot) tma_load_2d_pair(w + 2 * CHUNK, &tm_kv, bar, kVlat + 32 * rank, row);
            }
          }
          advance();
        }
      }
    }
    for (; used > 0; --used) {
      if (--r.slot < 0) r.slot = C::NS - 1, r.ph ^= 1;
      if (rank == 0) settle(&full[r.slot], r.ph);
      if (ok) settle(&empty[r.slot], r.ph);
    }
  } else if (warp == 1 && rank == 0) {
    const uint64_t ad = DKV ? smem_desc(smem_u32(sm), CHUNK, 1024) : smem_desc(smem_u32(sm), 16, 1024);
    const uint64_t wd = smem_desc(smem_u32(sm + C::OFF_W), CHUNK, 1024);
    Ring<C::NS> r;
    int n = 0;                                       // tasks so far
    bool ok = true;
    uint32_t more = 0;                               // accumulate
    auto multiply = [&](uint32_t d, bool rot) {
      ok = wait(&full[r.slot], r.ph, s_abort, p.status, SITE_F);
      if (!ok) return;
      tc_fence_after();
      if (elect_one_lane()) {
        const uint64_t a = desc_add(ad, r.slot * C::STAGE), w = desc_add(wd, r.slot * C::STAGE);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t ak = desc_add(a, kk * (DKV ? 2048 : 32));
          umma_bf16_pair(d, ak, desc_add(w, kk * 2048), IDESC, more | (kk > 0));
          if (rot)
            umma_bf16_pair(d + 256, ak, desc_add(w, 2 * CHUNK + kk * 2048), IDESC_ROT, more | (kk > 0));
        }
        umma_commit_pair(&empty[r.slot]);
      }
      __syncwarp();
      more = 1;
      r.next();
    };
    for (int task = first; task < tasks && ok; task += step) {
      const Task<DKV> t(p, task, n);
      if (!t.there) continue;
      if (n > 0) ok = wait(dfree, (n - 1) & 1, s_abort, p.status, SITE_DF);
      tc_fence_after();
      ++n;
      more = 0;
      const uint32_t d = tmem + (t.upper ? 192 : 0);
      if constexpr (DKV) {
        for (int x = t.x0; x < t.x1 && ok; ++x) {
          if (!t.sees(tile_pages(p, t.s, x))) continue;
          for (int st = 0; st < 4 && ok; ++st) multiply(d, t.upper && !(st & 1));
        }
      } else {
        for (int k = 0; k < t.list.count() && ok; ++k) multiply(d, t.upper);
      }
      if (elect_one_lane()) umma_commit_pair(done);
      __syncwarp();
    }
    if (elect_one_lane()) umma_commit_pair_own(drain);
    __syncwarp();
    settle(drain, 0);
  } else if (warp >= 4) {
    // ---- out: a row (key) a thread; warps 4..7 the lower half of the columns ----
    const int sub = warp & 3, half = (warp >> 2) - 1, r = 128 * rank + 32 * sub + lane;
    const uint32_t free_bar = mapa_u32(smem_u32(dfree), 0);
    auto give = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(dfree);
        else mbar_arrive_cluster_relaxed(free_bar);
      }
    };
    int n = 0;
    bool ok = true;
    for (int task = first; task < tasks && ok; task += step) {
      const Task<DKV> t(p, task, n);
      if (!t.there) continue;
      const bool some = t.some(p);
      const int g = t.x0 * X + r;                    // dq: row of the sequence
      ok = wait(done, n & 1, s_abort, p.status, SITE_DONE);
      if (!ok) break;
      ++n;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(sub * 32) << 16) + (t.upper ? 192 : 0);
      const bool shared = half != t.upper;           // this warp reads the columns that the next task uses
      if (!shared) give();
#pragma unroll 1
      for (int i = 0; i < (t.upper ? 5 : 4); ++i) {
        const int q = i < 4 && !t.upper ? (i + 2) & 3 : i;
        const int c = q < 4 ? 128 * half + 32 * q : 256 + 32 * half;
        uint32_t v[32];
        if (some) {
          tmem_ld32(taddr + c, v);
          tmem_ld_wait_regs(v);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0;
        }
        if (shared && i == 1) give();
        if constexpr (DKV) {
          float4* to = reinterpret_cast<float4*>(
              p.part + (part_row(p, t.s, t.b, t.g, t.kt) + r) * kRlat + 256 * t.upper + c);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            to[e] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
        } else if (g < t.s.n * p.H) {
          uint4* to = reinterpret_cast<uint4*>(
              p.dq + (static_cast<int64_t>(t.b) * p.m.T * p.H + g) * kRlat + 256 * t.upper + c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int f = 0; f < 4; ++f)
              w[f] = pack_bf16x2(__uint_as_float(v[8 * e + 2 * f]), __uint_as_float(v[8 * e + 2 * f + 1]));
            to[e] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Both products in one launch: neither needs the other's results.  The first dq_pairs pairs
// share dq's tasks, the others have a task of dkv each and follow as SMs fall free (a launch
// for each: 3 x 301 tokens, 8 heads 49.0 us instead of 45.3, 4096 tokens 1.99 ms instead of
// 1.97).
__global__ void __launch_bounds__(Prod::THREADS, 1)
    product_kernel(const __grid_constant__ CUtensorMap tm_pz, const __grid_constant__ CUtensorMap tm_kv,
                   const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                   const __grid_constant__ Params p, int dq_pairs, int dq_tasks, int dkv_tasks) {
  extern __shared__ uint8_t smem_raw[];
  cluster_arrive_relaxed();
  uint8_t* sm = smem_align1024(smem_raw);
  const int pair = blockIdx.x >> 1;
  if (pair < dq_pairs)
    product<false>(tm_pz, tm_kv, tm_q, tm_do, p, sm, pair, dq_pairs, dq_tasks);
  else
    product<true>(tm_pz, tm_kv, tm_q, tm_do, p, sm, pair - dq_pairs, dkv_tasks, dkv_tasks);
}

// dkv of a row: its segments in order (and what earlier chunks left), four dims a thread.
__global__ void __launch_bounds__(144) reduce_kernel(const Params p) {
  const int b = blockIdx.x / p.m.max_kv_len, key = blockIdx.x % p.m.max_kv_len, kt = key >> 8;
  pdl_wait();
  pdl_start_next();
  const Seq s = seq_of(p.m, b);
  // (rows of a sequence whose queries are all behind its end get their zeros)
  if (s.pos0 < 0 || s.L > p.m.max_kv_len || key >= s.L) return;
  const int2 tiles = tiles_of(p, s, kt);
  float4* acc = reinterpret_cast<float4*>(p.acc + (static_cast<int64_t>(b) * p.m.max_kv_len + key) * kRlat) +
                threadIdx.x;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!p.first_chunk) v = *acc;
  if (tiles.x < tiles.y) {
    const int g1 = (tiles.y - 1 - p.rt0) / p.q.seg;
#pragma unroll 4
    for (int g = (tiles.x - p.rt0) / p.q.seg; g <= g1; ++g) {
      const float4 w = reinterpret_cast<const float4*>(
          p.part + (part_row(p, s, b, g, kt) + (key & 255)) * kRlat)[threadIdx.x];
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
  }
  if (!p.last_chunk) {
    *acc = v;
    return;
  }
  reinterpret_cast<uint2*>(p.dkv + (static_cast<int64_t>(b) * p.kv.seq_stride + key) * kRlat)[threadIdx.x] =
      make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// span: keys that one query may see at most (window + n_first, or every row).  All but
// KF and nk follow from the sizes and the span alone, and nk + KF stays within
// most_key_tiles().
int64_t seg_tokens(int seg, int H) { return (static_cast<int64_t>(seg) * X + H - 2) / H + 1; }
int64_t most_key_tiles(int seg, int H, int64_t span) { return (span + seg_tokens(seg, H) + 509) / 256 + 2; }
Plan plan(int B, int T, int H, int max_kv_len, int64_t span, int64_t window, int64_t n_first) {
  Plan q{};
  const int64_t rows = static_cast<int64_t>(T) * H, S = max_kv_len;
  q.RT = static_cast<int>((rows + 2 * X - 1) / (2 * X) * 2);
  const int64_t tokens = (X + H - 2) / H + 1;
  const int64_t np = (span + tokens) / 64 + 4, most = (S + 63) / 64;
  q.np = static_cast<int>(np < most ? np : most);
  int64_t rc = kChunkBytes / (static_cast<int64_t>(B) * q.np * 2 * BLOCK) / 2 * 2;
  if (rc < 2) rc = 2;
  q.RC = static_cast<int>(rc < q.RT ? rc : q.RT);
  q.KT = static_cast<int>((S + 255) / 256);
  // segments: as many tasks as keep the pairs evenly busy, but the sums of each are
  // 590 KB to write and add
  int64_t seg = (2ll * B * q.RC * (span / 256 + 2) + TASKS - 1) / TASKS;
  if (seg < 4) seg = 4;
  q.seg = static_cast<int>(seg < q.RC ? seg : q.RC);
  q.G = (q.RC + q.seg - 1) / q.seg;
  const int64_t kf = (n_first + 255) / 256, nk = (window + seg_tokens(q.seg, H) + 254) / 256 + 1;
  q.KF = static_cast<int>(kf < q.KT ? kf : q.KT);
  q.nk = static_cast<int>(nk < q.KT ? nk : q.KT);
  return q;
}

// Bytes by part, from the sizes and the span alone.
struct Sizes {
  size_t rows, pz, part, acc;
  size_t total() const { return rows + pz + part + acc; }
};
Sizes sizes(const Plan& q, int B, int T, int H, int max_kv_len, int64_t span) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  Sizes z{};
  z.rows = up(static_cast<size_t>(B) * T * H * sizeof(float2));
  z.pz = BLOCK + static_cast<size_t>(B) * q.RC * q.np * 2 * BLOCK;
  const int64_t all = most_key_tiles(q.seg, H, span), twice = 2ll * q.KT;
  z.part = static_cast<size_t>(B) * q.G * (all < twice ? all : twice) * 256 * kRlat * sizeof(float);
  z.acc = q.RC < q.RT ? up(static_cast<size_t>(B) * max_kv_len * kRlat * sizeof(float)) : 0;
  return z;
}

template <typename Kernel, typename... Args>
dsa_status_t launch_pairs(const char* what, Kernel kernel, int64_t pairs, int threads, int smem,
                          cudaStream_t stream, Args... args) {
  if (pairs > (1 << 30) - 1) return DSA_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return launch_status("cudaFuncSetAttribute");
  launch_overlapped(kernel, static_cast<unsigned>(2 * pairs), threads, smem, 2, stream, args...);
  return launch_status(what);
}

}  // namespace wbw

// What these and all smaller calls with as many heads need at most; sizes() itself goes up and down
// with the segments.  With N = B RC tiles and s = span / 256 + 2, a segment has seg =
// max(4, N s / 300) tiles (or all of its sequence's) and reaches at most r = s + 3 + seg / 2H key
// tiles, 2 KT where that is less, so that there are B G <= min(N / 4, 300 / s) + B segments and
// B G r <= min(N / 4, 300 / s) (s + 3) + N / H + B (s + 3), where s >= 2.
size_t window_bwd_scratch_bytes(int B, int T, int H, int max_kv_len, int64_t span) {
  using namespace wbw;
  const Plan q = plan(B, T, H, max_kv_len, span, span, 0);
  Sizes z = sizes(q, B, T, H, max_kv_len, span);
  const int64_t tiles = static_cast<int64_t>(B) * q.RT, tile = static_cast<int64_t>(q.np) * 2 * BLOCK;
  const int64_t least = 2 * B * tile, some = kChunkBytes > least ? kChunkBytes : least;
  z.pz = BLOCK + static_cast<size_t>(tiles < some / tile ? tiles * tile : some);
  const int64_t twice = 2ll * q.KT, far = span / 256 + 5, reach = far < twice ? far : twice;
  const int64_t few = (tiles * reach + 3) / 4;
  const int64_t sums = (few < 750 ? few : 750) + tiles / H + 1 + B * reach;
  const int64_t segs = static_cast<int64_t>(B) * ((q.RT + 3) / 4);
  const int64_t all = (segs < 150 + B ? segs : 150 + B) * twice;
  z.part = static_cast<size_t>(sums < all ? sums : all) * 256 * kRlat * sizeof(float);
  const size_t acc = static_cast<size_t>(B) * max_kv_len * kRlat * sizeof(float);
  z.acc = q.RT > 2 && tiles > kChunkBytes / tile ? (acc + 255) / 256 * 256 : 0;
  return z.total();
}

dsa_status_t window_bwd_launch(const WindowBwdArgs& a, cudaStream_t stream) {
  using namespace wbw;
  const DenseArgs& f = a.f;
  const int64_t S = f.max_kv_len, both = static_cast<int64_t>(f.window) + f.n_first;
  const int64_t span = both == 0 ? 1 : both < S ? both : S;
  // a window and first tokens that meet at every position: the window alone
  const int window = both >= S ? f.max_kv_len : f.window, n_first = both >= S ? 0 : f.n_first;
  const Plan q = plan(f.B, f.T, f.H, f.max_kv_len, span, window, n_first);
  const Sizes z = sizes(q, f.B, f.T, f.H, f.max_kv_len, span);
  if (f.scratch_bytes < z.total()) return DSA_ERR_WORKSPACE_TOO_SMALL;
  const int64_t per = static_cast<int64_t>(f.T) * f.H;
  uint8_t* ws = static_cast<uint8_t*>(f.scratch);
  Params p{};
  p.kv = store_of(f);
  p.m = mask_of(f);
  p.m.window = window;
  p.m.n_first = n_first;
  p.B = f.B;
  p.H = f.H;
  p.q = q;
  p.scale = f.scale;
  p.scale_log2 = f.scale * 1.4426950408889634f;
  p.o = f.o_lat;
  p.d_o = a.d_o;
  p.lse = f.lse;
  p.rows = reinterpret_cast<float2*>(ws);
  p.pz = ws + z.rows;
  p.part = reinterpret_cast<float*>(p.pz + z.pz);
  p.acc = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.part) + z.part);
  p.dq = a.dq;
  p.dkv = a.dkv;
  p.status = f.status;
  const uint64_t pz_rows = z.pz / 128;
  if (pz_rows >= (uint64_t(1) << 31)) return DSA_ERR_UNSUPPORTED;
  // boxes of 64 rows for the products, of a tile for pz
  CUtensorMap tq, td, tq_tile, td_tile, tk, tp;
  const uint64_t kv_rows = static_cast<uint64_t>((f.B - 1) * f.kv.seq_stride + f.max_kv_len);
  if (!encode_tmap_2d(&tk, f.kv.base, kv_rows, kRlat, kRlat * 2, 64, 64, true) ||
      !encode_tmap_2d(&tp, p.pz, pz_rows, 64, 128, 64, 64, false) ||
      !encode_tmap_3d(&tq, f.q_lat, f.B, per, kRlat, 64, 64) ||
      !encode_tmap_3d(&td, a.d_o, f.B, per, kVlat, 64, 64) ||
      !encode_tmap_3d(&tq_tile, f.q_lat, f.B, per, kRlat, 64, X) ||
      !encode_tmap_3d(&td_tile, a.d_o, f.B, per, kVlat, 64, X))
    return DSA_ERR_CUDA;
  const int64_t ctas = (f.B * per + 7) / 8;
  launch_overlapped(prep_kernel, static_cast<unsigned>(ctas > 4 ? ctas : 4), 256, 0, 0, stream, p);
  if (launch_status("prep_kernel") != DSA_OK) return DSA_ERR_CUDA;
  for (int rt0 = 0; rt0 < q.RT; rt0 += q.RC) {
    p.rt0 = rt0;
    p.first_chunk = rt0 == 0;
    p.last_chunk = rt0 + q.RC >= q.RT;
    const int64_t pairs = num_sms() / 2, tiles = static_cast<int64_t>(f.B) * q.RC;
    const int64_t sums = 2ll * f.B * q.G * q.per_seg();
    if (sums > (1 << 30) || tiles > (1 << 30)) return DSA_ERR_UNSUPPORTED;
    const int64_t some = tiles < pairs ? tiles : pairs / 2 * 2;   // (even, as the tiles are)
    dsa_status_t st = launch_pairs("pz_kernel", pz_kernel, some, Pz::THREADS, Pz::SMEM, stream, tq_tile, td_tile,
                                   tk, p);
    if (st == DSA_OK)
      st = launch_pairs("product_kernel", product_kernel, some + sums, Prod::THREADS, Prod::SMEM, stream, tp, tk,
                        tq, td, p, static_cast<int>(some), static_cast<int>(tiles), static_cast<int>(sums));
    if (st != DSA_OK) return st;
    launch_overlapped(reduce_kernel, static_cast<unsigned>(static_cast<int64_t>(f.B) * f.max_kv_len), 144, 0,
                      0, stream, p);
    if (launch_status("reduce_kernel") != DSA_OK) return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

}  // namespace dsa
