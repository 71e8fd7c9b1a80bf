// mla_dense.cu -- dense attention over latent rows: a tree of drafted tokens over
// a cache, and a sliding window with first tokens that stay visible.
//
//   z_s = scale * q_lat[t,h,:] . KV[s,:]  over the rows s that query t sees,
//   o = sum_s softmax(z)_s KV[s, 0:512],   lse = log sum_s exp(z_s)
//
// The (query, head) rows of a sequence are packed: a unit is 2R consecutive ones
// (R = 96, 64 or 48: plan()), done by a pair of CTAs.
// Rows of the cache come 64 at a time (a page), a block is two such pages.
//   S [R rows per CTA x 128 keys] = Q . K^T      cta_group::2, N = 128, M = 256 (R = 96)
//        or 128 (64, 48): each CTA holds its own R queries (the MMA's other rows alias what
//        lies behind them and are not read) and the keys of one of the two pages
//   O^T [512 x 2R] += V^T . P^T                  cta_group::2, M = 256, N = 2R, twice:
//        CTA c holds dims 256c .. 256c+255 of all 128 keys and P of its own rows,
//        and accumulates its dims of all 2R rows
// in TMEM columns 0 .. 4R-1 (O^T) and 128 more (S; R <= 64: 64, twice).  Transposing the value product
// is what makes room: 512 dims of 96 rows would be all of a CTA's TMEM the other
// way round.  Sharing the keys between two CTAs halves what the score product reads
// of them through the shared-memory port: per block 216 KB (S) + 112 KB (O^T) are
// read, 136 KB copied in and 24 KB of P written, about 3,800 cycles at 128 bytes,
// beside 3,840 cycles of MMAs (R = 96).
//
// Roles (12 warps): 0 copies Q (chunk by chunk beside a unit's first K) and K, 1 copies
// V, 2 and 3 of the even CTA issue the two products, 4..7 hold a row (R <= 64: and one
// of the two pages) a thread: its scores, P = 2^(z - m) to BF16 in shared memory; 8..11
// write O^T / l out while the next unit's first products run.
// m is the maximum of the first block in which the row sees anything, so O^T is
// never rescaled.  A row whose later scores exceed it by 2^80 leaves the maximum that it
// met where its output goes, and its unit is done a second time with that, after all
// others of the pair (512 queries, 96 heads, window 1024: 0.14 ms, every unit twice 0.24;
// row by row it was 34).  The second time stands behind the kernel's end, in a function of
// its own: units put back into the line cost every call 1.1 us at that end.  A unit some of
// whose queries do not see a row of the sequence that holds an infinity or a NaN (0 * NaN
// would reach them) goes to attend_row (33 ms there); the waits of the others last as long
// as it moves on.  So does one with a reference that FP32 rounds too coarsely: from 2^28 on it
// is off the maximum by up to 16 and more, from 2^31 on by more than an exponent holds (LOST).
// P up to 2^80 leaves the FP32 sums 2^47 for the values: where a row's P passed 2^20 and its
// O^T is not finite although its sum of P is, its unit is marked, and all warps do the marked
// units' rows by attend_row at the end (looking for it in every unit's outputs took 1 % of
// a call; in those alone 2,048 queries 408 -> 409 us, 417 -> 421 where all have such a row).
// Rows behind the sequence, in its last page, are zeroed in V before use.
//
// Persistent: the blocks of all units stand in one line, and every pair of SMs takes
// an equal stretch of it (whole units where there are many).  A unit that is cut has
// its pieces' normalised FP32 outputs joined by their log-sum-exps, in order, by
// combine_kernel.
//
// 96 heads: 2 x 8192 queries, window 1024: 3.1 ms, 1.07 PFLOP/s; 16 x 8 drafted tokens over
// 4096 to 16384 rows: 235 us, 1.16 PFLOP/s (the port); 4 x 1 over up to 131072: 126 us,
// 4.0 TB/s (499 MB); 64 windows of one query: 20 us.  pair_kernel<96> spills
// (168 registers, 48 bytes): 0.4 % of its instructions are for that (2,048 queries).
#include <cmath>

#include <cuda_bf16.h>

#include "dense_mask.cuh"
#include "dense_pair.cuh"

namespace dsa {
namespace dense {

constexpr int THREADS = 384;
constexpr int REDO = 1024;                // units of a pair that may be done twice; more: attend_row
constexpr float FAR = 80.f;               // exponents that P may reach: 2^80 times 2^47 is FP32's range
constexpr float RISE = 20.f;              // above it, P may be what takes P V out of FP32's range
constexpr float LOST = 0x1p-16f;          // a sum of P that only a reference above the maximum leaves

template <int R_>
struct Cfg {
  static constexpr int R = R_;
  static constexpr int HALVES = R <= 64 ? 2 : 1;      // threads that share a row's scores
  // K slots: a chunk of own keys; V slots: 64 keys x 128 dims (48 rows, 7 + 5: 4 x 1 over
  // 131072 128.1 us instead of 126.3; 64 rows, 8 + 3: 5 trees of 33 27.1 instead of 25.8)
  static constexpr int NK = R == 96 ? 5 : R == 64 ? 6 : 9;
  static constexpr int NV = R == 96 ? 3 : 4;
  static constexpr int QCH = R * 128;                 // 64 dims of the queries
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = OFF_Q + 9 * QCH;
  static constexpr int NP = R == 96 ? 1 : 2;          // P of as many blocks (4 x 1 over 131072: 131.6 -> 129.3 us)
  static constexpr int OFF_K = OFF_P + 2 * NP * QCH;
  static constexpr int OFF_V = OFF_K + NK * CHUNK;
  static constexpr int OFF_MISC = OFF_V + NV * 2 * CHUNK;
  static constexpr int MISC = 1024 + 16 * R + (HALVES == 2 ? 2048 : 0) + 6 * REDO / 8;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;
  static constexpr uint32_t S_COL = 4 * R;
  static constexpr int SW = 128 / HALVES;             // columns of a score buffer
  static constexpr int NB = R == 96 ? 1 : 2;          // score buffers
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(OFF_Q + 8 * QCH + 128 * 128 / HALVES <= OFF_K, "the aliased rows stay inside Q and P");
  static_assert(4 * R + SW * NB <= 512, "TMEM columns");
};

enum : uint32_t {
  SITE_KF = 0x711, SITE_KE = 0x712, SITE_VF = 0x713, SITE_VE = 0x714,
  SITE_SF = 0x715, SITE_SE = 0x716, SITE_P = 0x717, SITE_O = 0x718, SITE_VT = 0x719,
  SITE_OE = 0x71b, SITE_L = 0x71c, SITE_U = 0x71d
};

// A pair's stretch of the line, as combine_kernel needs it: the unit and the block
// that it starts with, the unit that it begins but does not end (or -1) and the slot
// of that piece.
struct Stretch {
  int first, j0, head, slot;
};

struct Params {
  const uint16_t* q;
  Store kv;
  Mask m;
  int B, H, tiles, pairs;
  int nominal;        // window: blocks that a unit counts for; tree: 0, what it has
  int cut;            // units may be cut
  float scale_log2;
  uint16_t* o;
  float* lse;
  float* part_o;      // [pairs, 2, 2R, 512] normalised
  float* part_lse;    // [pairs, 2, 2R] base 2
  Stretch* stretch;   // [pairs]
  uint32_t* status;
};

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// One row by a warp over pages k0..k1-1 of `pages`, in FP32 with a running maximum:
// for what the products above cannot give.  Into o / lse, or (part) the partials.
__device__ __noinline__ void attend_row(const Params& p, const Seq& s, const Pages& pages, int k0,
                                        int k1, int b, int row, float* part_o, float* part_lse) {
  const int lane = threadIdx.x & 31, i = row / p.H;
  const int64_t at = static_cast<int64_t>(b) * p.m.T * p.H + row;
  const uint64_t bits = p.m.tree != nullptr ? p.m.tree[static_cast<int64_t>(b) * p.m.T + i] : 0;
  float q[18], acc[16];
  const uint32_t* qr = reinterpret_cast<const uint32_t*>(p.q + at * kRlat) + lane;
#pragma unroll
  for (int c = 0; c < 9; ++c) {
    const uint32_t v = qr[32 * c];
    q[2 * c] = lo_f(v), q[2 * c + 1] = hi_f(v);
  }
#pragma unroll
  for (int d = 0; d < 16; ++d) acc[d] = 0.f;
  float top = -INFINITY, sum = 0.f;
  for (int k = k0; k < k1; ++k) {
    const int pg = pages.page(k);
    const int64_t r0 = page_row(p.kv, b, pg);
    if (r0 < 0) continue;
    for (uint64_t see = row_mask(p.m, s, i, bits, pg * 64); see != 0; see &= see - 1) {
      const int64_t r = r0 + __ffsll(static_cast<long long>(see)) - 1;
      const uint32_t* kr = reinterpret_cast<const uint32_t*>(p.kv.base + r * kRlat) + lane;
      float x[18], z = 0.f;
#pragma unroll
      for (int c = 0; c < 9; ++c) {
        const uint32_t v = kr[32 * c];
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
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum);
  if (part_o != nullptr) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      reinterpret_cast<float2*>(part_o)[32 * c + lane] = make_float2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
    if (lane == 0) *part_lse = lse2;
  } else {
    uint32_t* o = reinterpret_cast<uint32_t*>(p.o + at * kVlat) + lane;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[32 * c] = pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
    if (lane == 0 && p.lse != nullptr) p.lse[at] = lse2 * 0.6931471805599453f;
  }
}

// A piece of a unit: its pages k0 .. k1-1, nb blocks.
struct Unit {
  int b, id, g0, rows, i0, i1;    // rows: of the sequence
  Seq s;
  Pages pages;
  int k0, k1, nb;
  int j0, j1, of;                 // blocks j0 .. j1-1 of `of`
  int no;                         // which of its pair's
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == of; }
};

// A pair's stretch of the line, unit by unit.  Every warp walks it by itself (all
// lanes alike); the sequences' lengths stay in L1.
template <int R>
struct Line {
  const Params& p;
  int b = 0, tile = 0, j = 0, tiles = 0, cost = 0;   // tiles and blocks per tile of sequence b
  int64_t left = 0;
  Seq s;

  __device__ __forceinline__ void measure(int at, Seq& sq, int& n_tiles, int& n_blocks) const {
    sq = seq_of(p.m, at);
    n_tiles = (sq.n * p.H + 2 * R - 1) / (2 * R);
    n_blocks = p.nominal;
    if (p.nominal == 0) n_blocks = sq.ok ? max(((sq.L + 63) / 64 + 1) / 2, 1) : 1;
  }
  // Blocks of the sequences at .. at + 31, a lane each, summed from `at` on.
  __device__ __forceinline__ int64_t sums(int at, int& mine) const {
    const int lane = threadIdx.x & 31;
    Seq sq;
    int n = 0, c = 0;
    if (at + lane < p.B) measure(at + lane, sq, n, c);
    mine = n * c;
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    return sum;
  }
  // The sequence, tile and block at x (or behind the last sequence).
  __device__ __forceinline__ void seek(int64_t x) {
    if (p.nominal > 0) {
      const int64_t u = x / p.nominal;
      j = static_cast<int>(x - u * p.nominal);
      b = static_cast<int>(u / p.tiles);
      tile = static_cast<int>(u % p.tiles);
      if (b < p.B) measure(b, s, tiles, cost);
      return;
    }
    for (b = 0; b < p.B; b += 32) {
      int mine;
      const int64_t sum = sums(b, mine);
      const unsigned over = __ballot_sync(0xffffffffu, sum > x);
      if (over != 0) {
        const int at = __ffs(over) - 1;
        const unsigned in = static_cast<unsigned>(x - __shfl_sync(0xffffffffu, sum - mine, at));
        b += at;
        measure(b, s, tiles, cost);
        tile = in / static_cast<unsigned>(cost);
        j = in % static_cast<unsigned>(cost);
        return;
      }
      x -= __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  __device__ __forceinline__ int64_t total() const {
    if (p.nominal > 0) return static_cast<int64_t>(p.B) * p.tiles * p.nominal;
    int64_t sum = 0;
    int mine;
    for (int at = 0; at < p.B; at += 32) sum += __shfl_sync(0xffffffffu, sums(at, mine), 31);
    return sum;
  }
  __device__ __forceinline__ Line(const Params& pp, int pair) : p(pp) {
    if (!p.cut && p.pairs == p.B * p.tiles) {          // a unit each
      b = pair / p.tiles;
      tile = pair % p.tiles;
      measure(b, s, tiles, cost);
      left = tile < tiles ? cost : 0;
      return;
    }
    // at least two blocks each (5 trees of 33 tokens, 120 blocks: 34 us with all 76 pairs
    // at work, 28 with 60): the last pairs may have nothing
    const int64_t all = total();
    const int n = static_cast<int>(min((all + 1) / 2, static_cast<int64_t>(p.pairs)));
    if (pair >= n) return;
    // the first pairs have one block more
    int64_t each, more;
    if (all < (1ll << 31)) {
      each = static_cast<unsigned>(all) / static_cast<unsigned>(n);
      more = static_cast<unsigned>(all) % static_cast<unsigned>(n);
    } else {
      each = all / n, more = all % n;
    }
    int64_t x0 = each * pair + min(static_cast<int64_t>(pair), more), x1 = x0 + each + (pair < more);
    if (!p.cut) {                 // whole units: to the next unit's start
      seek(x1);
      if (x1 < all && j > 0) x1 += cost - j;
      seek(x0);
      if (x0 < all && j > 0) x0 += cost - j;
    }
    if (x0 < x1) seek(x0);
    left = x1 - x0;
  }
  __device__ __forceinline__ bool next(Unit& u) {
    if (left <= 0) return false;
    while (tile >= tiles) {
      if (++b >= p.B) return false;
      tile = j = 0;
      measure(b, s, tiles, cost);
    }
    u.b = b;
    u.id = b * p.tiles + tile;
    u.s = s;
    u.g0 = tile * 2 * R;
    u.rows = s.n * p.H;
    u.i0 = u.g0 / p.H;
    u.i1 = (min(u.g0 + 2 * R, u.rows) - 1) / p.H;
    u.pages = pages_of(p.m, s, u.i0, u.i1);
    u.of = cost;
    u.j0 = j;
    u.j1 = static_cast<int>(min(static_cast<int64_t>(cost), j + left));
    const int np = u.pages.count();
    u.k0 = min(2 * u.j0, np);
    u.k1 = min(2 * u.j1, np);
    u.nb = (u.k1 - u.k0 + 1) / 2;
    left -= u.j1 - u.j0;
    j = 0;
    ++tile;
    return true;
  }
};

// The units of a CTA's stretch in shared memory: the K warp walks the line and
// publishes them, the others read them there (and keep their registers).
constexpr int UNITS = 4;
struct Feed {
  const Unit* ring;
  uint64_t* full;
  uint64_t* empty;
  volatile int* s_abort;
  uint32_t* status;
  int at = -1;
  // The next unit, the one before given back; null at the end or once the CTA has given up.
  __device__ __forceinline__ const Unit* next() {
    if (at >= 0) mbar_arrive_warp(&empty[at % UNITS]);
    ++at;
    if (!wait(&full[at % UNITS], (at / UNITS) & 1, s_abort, status, SITE_U)) return nullptr;
    const Unit* u = ring + at % UNITS;
    return u->b >= 0 ? u : nullptr;
  }
};

// Whether every query of the unit sees all of the 64 rows from kb on.
__device__ __forceinline__ bool all_see(const Mask& m, const Unit& u, int kb) {
  if (m.tree != nullptr) return kb + 63 < u.s.pos0;
  const int t0 = u.s.pos0 + u.i0, t1 = u.s.pos0 + u.i1;
  return kb + 63 <= t0 && t1 < u.s.L && (kb > t1 - m.window || kb + 63 < m.n_first);
}

// What a CTA keeps in shared memory beside its operands.
template <int R>
struct Shared {
  using C = Cfg<R>;
  static constexpr int BARS = 2 * C::NK + 2 * C::NV + 21 + 2 * UNITS;
  uint64_t *kfull, *kempty;      // kfull, vfull, sfree, ofree: the even CTA's
  uint64_t *vfull, *vempty;
  uint64_t *sfull, *sfree;       // [NB]
  uint64_t* pready;              // [NP] odd CTA: for its warp 3
  uint64_t *odone, *ofull;       // [NP] a block's values added; a unit's
  uint64_t *ofree;               // [2] 2R columns read
  uint64_t *lfull, *lpeer;       // [2] a unit's sums, of this CTA's rows, of the other's
  uint64_t *lfree;               // [2]
  uint64_t *vland;               // [2] this CTA's own copies
  uint64_t *drain;               // [2]
  uint64_t *ufull, *uempty;      // [UNITS]
  uint32_t* tslot;
  volatile int* s_abort;         // [2] the second moves while attend_row goes on
  volatile int* s_slow;          // [2] x unit + 1 of which a row is far, needs attend_row, is above RISE
  volatile int *s_any, *s_go;    // units are to be done again; the other CTA says so too
  volatile uint32_t* s_past;     // units stand in s_beyond (of either CTA: both are told)
  Unit* s_unit;                  // [UNITS]
  float* s_inv;                  // [2][2R]
  float *s_top, *s_sum;          // HALVES = 2: [2][2][64] maxima, sums
  uint32_t* s_redo;              // a bit a unit
  uint32_t* s_noted;             // [4 warps] the warp's rows have left their maxima
  uint32_t* s_beyond;            // a bit a unit, the last for all from there on: P times V left FP32's range
  static_assert(BARS * 8 + 48 <= 512, "misc");
  static_assert(UNITS * sizeof(Unit) <= 512, "misc");

  __device__ __forceinline__ explicit Shared(uint8_t* sm) {
    kfull = reinterpret_cast<uint64_t*>(sm + C::OFF_MISC);
    kempty = kfull + C::NK;
    vfull = kempty + C::NK;
    vempty = vfull + C::NV;
    sfull = vempty + C::NV;
    sfree = sfull + 2;
    pready = sfull + 4;
    odone = sfull + 6;
    ofull = sfull + 8;
    ofree = sfull + 9;
    lfull = sfull + 11;
    lpeer = sfull + 13;
    lfree = sfull + 15;
    vland = sfull + 17;
    drain = sfull + 19;
    ufull = sfull + 21;
    uempty = ufull + UNITS;
    tslot = reinterpret_cast<uint32_t*>(uempty + UNITS);
    s_abort = reinterpret_cast<volatile int*>(tslot + 1);
    s_slow = reinterpret_cast<volatile int*>(tslot + 3);
    s_any = reinterpret_cast<volatile int*>(tslot + 9);
    s_go = s_any + 1;
    s_past = reinterpret_cast<volatile uint32_t*>(s_any + 2);
    s_unit = reinterpret_cast<Unit*>(sm + C::OFF_MISC + 512);
    s_inv = reinterpret_cast<float*>(sm + C::OFF_MISC + 1024);
    s_top = s_inv + 4 * R;
    s_sum = s_top + 256;
    s_redo = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC + C::MISC - 6 * REDO / 8);
    s_noted = s_redo + REDO / 32;
    s_beyond = s_noted + 4 * (REDO / 32);
  }
  __device__ __forceinline__ void barriers(int rank) const {
    for (int k = 0; k < C::NK; ++k) mbar_init(&kfull[k], 1), mbar_init(&kempty[k], 1);
    for (int k = 0; k < C::NV; ++k) mbar_init(&vfull[k], 2), mbar_init(&vempty[k], 1);
    mbar_init(ofull, 1);
    for (int k = 0; k < 2; ++k) {
      mbar_init(&sfull[k], 1);
      mbar_init(&sfree[k], 8);
      mbar_init(&pready[k], rank == 0 ? 5 : 4);
      mbar_init(&odone[k], 1);
      mbar_init(&ofree[k], 8);
      mbar_init(&lfull[k], 4);
      mbar_init(&lpeer[k], 1);
      mbar_init(&lfree[k], 8);
      mbar_init(&vland[k], 1);
      mbar_init(&drain[k], 1);
    }
    for (int k = 0; k < UNITS; ++k) mbar_init(&ufull[k], 1), mbar_init(&uempty[k], rank == 0 ? 11 : 10);
    fence_mbar_init();
  }
};

// Whether P V, of 32 dims and `here` rows, is an infinity or a NaN in a row whose sum of P is
// neither: marks the unit in both CTAs.  By a warp.
__device__ __noinline__ void mark_beyond(uint32_t taddr, int here, const float* inv, int no, uint32_t* beyond,
                                         volatile uint32_t* past) {
  bool some = false;
#pragma unroll 1
  for (int c = 0; c < here; c += 32) {
    uint32_t x[32];
    tmem_ld32(taddr + c, x);
    tmem_ld_wait_regs(x);
    float sum = 0.f;                                     // NaN with an infinity or a NaN
#pragma unroll
    for (int e = 0; e < 32; ++e) sum = fmaf(__uint_as_float(x[e]), 0.f, sum);
    if (!__any_sync(0xffffffffu, sum != 0.f)) continue;
#pragma unroll
    for (int e = 0; e < 32; ++e)
      some |= c + e < here && inv[c + e] < INFINITY && !(fabsf(__uint_as_float(x[e])) < INFINITY);
  }
  if (__any_sync(0xffffffffu, some)) {
    const int k = min(no, REDO - 1), lane = threadIdx.x & 31;
    if (lane < 2) {
      or_cluster_u32(smem_u32(beyond + (k >> 5)), lane, 1u << (k & 31));
      or_cluster_u32(smem_u32(const_cast<uint32_t*>(past)), lane, 1u);
    }
    __syncwarp();
  }
}

// What the warps do from the first unit to the last.  AGAIN: only the units that have to
// be done a second time.
template <int R, bool AGAIN>
__device__ __forceinline__ void roles(const CUtensorMap& tm_q, const CUtensorMap& tm_kv, const Params& p,
                                      uint8_t* sm, uint32_t tmem) {
  using C = Cfg<R>;
  constexpr uint32_t IDESC_S = idesc_bf16(256 / C::HALVES, 128, false, false);
  constexpr uint32_t IDESC_O = idesc_bf16(256, 2 * R, true, false);
  const auto [kfull, kempty, vfull, vempty, sfull, sfree, pready, odone, ofull, ofree, lfull, lpeer, lfree,
              vland, drain, ufull, uempty, tslot, s_abort, s_slow, s_any, s_go, s_past, s_unit, s_inv, s_top,
              s_sum, s_redo, s_noted, s_beyond] = Shared<R>(sm);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1;
  // An issuer that gives up: its MMAs are complete before the pair leaves.  (Otherwise those
  // who waited for what they gave have seen that.)
  auto give_up = [&](uint64_t* bar) {
    if (elect_one_lane()) umma_commit_pair_own(bar);
    __syncwarp();
    settle(bar, 0);
  };
  Feed feed{s_unit, ufull, uempty, s_abort, p.status};

  if (warp < 4) {
    if (warp == 0) {
      // ---- the own page's K, chunk by chunk; beside the first block's, Q's: the
      // products that read a chunk of the unit before are those that free K's slot ----
      // (the lengths are looked up while the other warps and the other CTA get ready)
      if (!AGAIN) {
        pdl_wait();
        pdl_start_next();
      }
      Line<R> line(p, pair);
      if (!AGAIN) cluster_wait();
      Unit u;
      Ring<C::NK> r;
      Stretch mine{-1, 0, -1, 0};
      int used = 0;
      bool ok = true;
      for (int at = 0, no = 0;; ++at) {
        bool more = line.next(u);
        if (AGAIN)
          for (; more && !(no < REDO && s_redo[no >> 5] >> (no & 31) & 1); ++no) more = line.next(u);
        u.no = no++;
        if (!more) u.b = -1;
        if (at >= UNITS) ok = wait(&uempty[at % UNITS], (at / UNITS - 1) & 1, s_abort, p.status, SITE_U);
        if (!ok) break;
        if (lane == 0) {
          s_unit[at % UNITS] = u;
          mbar_arrive(&ufull[at % UNITS]);
        }
        __syncwarp();
        if (!more) break;
        if (at == 0) mine.first = u.id, mine.j0 = u.j0;
        if (u.j0 == 0 && u.j1 < u.of) mine.head = u.id, mine.slot = 2 * pair + (at > 0);
        const int qrow = static_cast<int>(static_cast<int64_t>(u.b) * p.m.T * p.H) + u.g0 + rank * R;
        for (int j = 0; j < u.nb && ok; ++j) {
          const int k = u.k0 + 2 * j + rank;
          int64_t row = 0;
          if (k < u.k1) {
            row = page_row(p.kv, u.b, u.pages.page(k));
            if (row < 0) {                                 // nobody sees it
              if (lane == 0)
                status_raise(p.status, DSA_ERR_BAD_INDEX, SITE_PAGE, static_cast<uint32_t>(u.pages.page(k)));
              row = 0;
            }
          }
          for (int c = 0; c < 9; ++c) {
            ok = used < C::NK || wait(&kempty[r.slot], r.ph ^ 1, s_abort, p.status, SITE_KE);
            if (!ok) break;
            if (elect_one_lane()) {
              const uint32_t bar = mapa_u32(smem_u32(&kfull[r.slot]), 0);
              if (rank == 0) mbar_expect_tx(&kfull[r.slot], 2 * CHUNK + (j == 0 ? 2 * C::QCH : 0));
              if (j == 0) tma_load_2d_pair(sm + C::OFF_Q + c * C::QCH, &tm_q, bar, 64 * c, qrow);
              if (k < u.k1)
                tma_load_2d_pair(sm + C::OFF_K + r.slot * CHUNK, &tm_kv, bar, 64 * c, static_cast<int>(row));
              else    // no second page: the slot keeps what it holds.  Counted all the same: products
                      // that did not need this CTA could free the slot twice between two of its looks
                mbar_complete_tx_cluster(bar, CHUNK);
            }
            __syncwarp();
            if (used < C::NK) ++used;
            r.next();
          }
        }
        if (!ok) break;
      }
      if (!AGAIN && rank == 0 && lane == 0 && p.cut) p.stretch[pair] = mine;
      // the pair's copies have landed and the last arrivals of the MMAs have come
      // before either CTA leaves
      for (; used > 0; --used) {
        if (--r.slot < 0) r.slot = C::NK - 1, r.ph ^= 1;
        if (rank == 0) settle(&kfull[r.slot], r.ph);
        if (ok) settle(&kempty[r.slot], r.ph);
      }
    } else if (warp == 1) {
      // ---- V: the own 256 dims of both pages, 128 at a time ----
      Ring<C::NV> r;
      int used = 0;
      uint32_t vph = 0;
      bool ok = true;
      while (const Unit* up = ok ? feed.next() : nullptr) {
        const Unit& u = *up;
#pragma unroll 1
        for (int k = u.k0; k < u.k1 && ok; ++k) {
          const int64_t row = page_row(p.kv, u.b, u.pages.page(k));
          const uint64_t any = row < 0 ? 0 : range_bits(0, u.s.L, u.pages.page(k) * 64);
          Ring<C::NV> z = r;
#pragma unroll 1
          for (int m = 0; m < 2; ++m) {
            ok = used < C::NV || wait(&vempty[r.slot], r.ph ^ 1, s_abort, p.status, SITE_VE);
            if (!ok) break;
            uint8_t* dst = sm + C::OFF_V + r.slot * 2 * CHUNK;
            const int col = 256 * rank + 128 * m;
            if (any != 0 && elect_one_lane()) {
              if (any == ~0ull) {
                const uint32_t bar = mapa_u32(smem_u32(&vfull[r.slot]), 0);
                mbar_expect_tx_cluster(bar, 2 * CHUNK);
                tma_load_2d_pair(dst, &tm_kv, bar, col, static_cast<int>(row));
                tma_load_2d_pair(dst + CHUNK, &tm_kv, bar, col + 64, static_cast<int>(row));
              } else {
                mbar_expect_tx(&vland[m], 2 * CHUNK);
                tma_load_2d(dst, &tm_kv, &vland[m], col, static_cast<int>(row));
                tma_load_2d(dst + CHUNK, &tm_kv, &vland[m], col + 64, static_cast<int>(row));
              }
            }
            __syncwarp();
            if (used < C::NV) ++used;
            r.next();
          }
          if (!ok || any == ~0ull) continue;
          // rows behind the sequence become zeros: whatever they hold must not meet
          // the zeros of P
#pragma unroll 1
          for (int m = 0; m < 2; ++m) {
            if (any != 0) {
              ok = wait(&vland[m], vph, s_abort, p.status, SITE_VT);
              if (!ok) break;
            }
            uint8_t* dst = sm + C::OFF_V + z.slot * 2 * CHUNK;
#pragma unroll 4
            for (int e = lane; e < 1024; e += 32)       // 16 bytes of row (e >> 3) & 63
              if (!(any >> ((e >> 3) & 63) & 1))
                reinterpret_cast<uint4*>(dst)[e] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_u32(smem_u32(&vfull[z.slot]), 0));
            z.next();
          }
          if (any != 0) vph ^= 1;
        }
      }
      for (; used > 0; --used) {
        if (--r.slot < 0) r.slot = C::NV - 1, r.ph ^= 1;
        if (rank == 0) settle(&vfull[r.slot], r.ph);
        if (ok) settle(&vempty[r.slot], r.ph);
      }
    } else if (warp == 2) {
      if (rank == 0) {
        // ---- scores ----
        const uint64_t qd = smem_desc(smem_u32(sm + C::OFF_Q), 16, 1024);
        const uint64_t kd = smem_desc(smem_u32(sm + C::OFF_K), 16, 1024);
        Ring<C::NK> r;
        int blk = 0;
        bool ok = true;
        while (const Unit* up = ok ? feed.next() : nullptr) {
        const Unit& u = *up;
          for (int j = 0; j < u.nb && ok; ++j, ++blk) {
            const int bu = blk % C::NB;
            if (blk >= C::NB) ok = wait(&sfree[bu], (blk / C::NB - 1) & 1, s_abort, p.status, SITE_SE);
            tc_fence_after();
            for (int c = 0; c < 9 && ok; ++c) {
              ok = wait(&kfull[r.slot], r.ph, s_abort, p.status, SITE_KF);
              if (!ok) break;
              tc_fence_after();
              if (elect_one_lane()) {
                const uint64_t a = desc_add(qd, c * C::QCH), w = desc_add(kd, r.slot * CHUNK);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_bf16_pair(tmem + C::S_COL + C::SW * bu, desc_add(a, kk * 32), desc_add(w, kk * 32), IDESC_S,
                                 c > 0 || kk > 0);
                umma_commit_pair(&kempty[r.slot]);
                if (c == 8) umma_commit_pair(&sfull[bu]);
              }
              __syncwarp();
              r.next();
            }
          }
        }
        if (!ok) give_up(&drain[0]);
      } else if (!AGAIN) {
        // every sequence, whether it has a unit or not
        for (int b = pair * 32 + lane; b < p.B; b += p.pairs * 32) report_seq(p.m, seq_of(p.m, b), b, p.status);
      }
    } else if (rank == 0) {
      // ---- values ----
      const uint64_t pd = smem_desc(smem_u32(sm + C::OFF_P), 16, 1024);
      const uint64_t vd = smem_desc(smem_u32(sm + C::OFF_V), CHUNK, 1024);
      Ring<C::NV> r;
      int n = 0, blk = 0;
      bool ok = true;
      while (const Unit* up = ok ? feed.next() : nullptr) {
        const Unit& u = *up;
        if (u.nb == 0) continue;
        for (int j = 0; j < u.nb && ok; ++j, ++blk) {
          const int pb = blk % C::NP;
          ok = wait(&pready[pb], blk / C::NP & 1, s_abort, p.status, SITE_P);
          const int nt = u.k0 + 2 * j + 1 < u.k1 ? 4 : 2;
          for (int t = 0; t < nt && ok; ++t) {           // page t >> 1, dims 128 (t & 1)
            // the unit before has been read out
            if (j == 0 && t < 2 && n > 0) ok = wait(&ofree[t], (n - 1) & 1, s_abort, p.status, SITE_OE);
            ok = ok && wait(&vfull[r.slot], r.ph, s_abort, p.status, SITE_VF);
            if (!ok) break;
            tc_fence_after();
            if (elect_one_lane()) {
              const uint64_t a = desc_add(vd, r.slot * 2 * CHUNK), w = desc_add(pd, (2 * pb + (t >> 1)) * C::QCH);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16_pair(tmem + (t & 1) * 2 * R, desc_add(a, kk * 2048), desc_add(w, kk * 32),
                               IDESC_O, j > 0 || t > 1 || kk > 0);
              umma_commit_pair(&vempty[r.slot]);
              if (t == nt - 1) umma_commit_pair(&odone[pb]);
              if (t == nt - 1 && j == u.nb - 1) umma_commit_pair(ofull);
            }
            __syncwarp();
            r.next();
          }
        }
        ++n;
      }
      if (!ok) give_up(&drain[1]);
    } else {
      // ---- tells the even CTA that this one's P is written: a release at cluster scope
      // takes 0.5 us, in the softmax warps it set the pace of the pair ----
      const uint32_t bar = mapa_u32(smem_u32(pready), 0);
      int blk = 0;
      bool ok = true;
      while (const Unit* up = ok ? feed.next() : nullptr) {
        const int nb = up->nb;
        for (int j = 0; j < nb && ok; ++j, ++blk) {
          const int pb = blk % C::NP;
          ok = wait(&pready[pb], blk / C::NP & 1, s_abort, p.status, SITE_P);
          if (ok && lane == 0) mbar_arrive_cluster(bar + 8 * pb);
          __syncwarp();
        }
      }
    }
  } else if (warp < 8) {
    // ---- softmax: a row a thread, or (HALVES = 2) a row and one of the block's pages:
    // the MMA of 128 rows leaves a CTA's 64 in lanes 0..63 (first page) and 64..127 ----
    constexpr int PG = 2 / C::HALVES, CH = 2 * PG;       // pages and 32-column chunks of a thread
    const int sub = warp & 3, half = C::HALVES == 2 ? sub >> 1 : 0;
    const int r = (C::HALVES == 2 ? sub & 1 : sub) * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(sub * 32) << 16) + C::S_COL;
    const uint32_t free_bar = mapa_u32(smem_u32(sfree), 0);
    uint8_t* prow = sm + C::OFF_P + half * C::QCH + (r >> 3) * 1024 + (r & 7) * 128;
    int blk = 0, met = 0;                                // met: exchanges of the two halves so far
    bool ok = true;
    // the other half's value of what this thread gives (HALVES = 2)
    auto exchange = [&](float* s_buf, int turn, float v) {
      float* buf = s_buf + (turn & 1) * 128;
      buf[half * 64 + r] = v;
      named_bar_sync(2 + (sub & 1), 64);
      return buf[(half ^ 1) * 64 + r];
    };
    while (true) {
      const Unit* up = ok ? feed.next() : nullptr;
      // (HALVES = 2: the two warps that share rows come and leave together, by votes)
      if (C::HALVES == 2 ? named_bar_or(2 + (sub & 1), 64, up == nullptr) : up == nullptr) break;
      const Unit& u = *up;
      const int at = feed.at;
      const int g = u.g0 + rank * R + r;
      const bool live = r < R && g < u.rows;
      const int i = live ? g / p.H : 0;
      const uint64_t bits =
          live && p.m.tree != nullptr ? p.m.tree[static_cast<int64_t>(u.b) * p.m.T + i] : 0;
      // where the row leaves its maximum (HALVES = 2: its two threads theirs)
      auto note = [&] {
        return u.whole() ? reinterpret_cast<float*>(p.o + (static_cast<int64_t>(u.b) * p.m.T * p.H + g) * kVlat)
                         : p.part_o + (static_cast<int64_t>(2 * pair + (u.no > 0)) * 2 * R + rank * R + r) * kVlat;
      };
      float l_sum = 0.f, m_ref = -INFINITY, peak = 0.f;  // peak: of z - m; infinite: for attend_row
      if (AGAIN && live)
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h)
          if (s_noted[((C::HALVES == 2 ? sub & 1 : sub) + 2 * h) * (REDO / 32) + (u.no >> 5)] >> (u.no & 31) & 1)
            m_ref = fmaxf(m_ref, note()[h]);
      bool good[PG];                       // the block's pages are there: looked up a block ahead
      auto look = [&](int j) {
#pragma unroll
        for (int h = 0; h < PG; ++h) {
          const int k = u.k0 + 2 * j + half + h;
          good[h] = k < u.k1 && page_row(p.kv, u.b, u.pages.page(k)) >= 0;
        }
      };
      look(0);
      for (int j = 0; j < u.nb && (C::HALVES == 2 || ok); ++j, ++blk) {
        // who sees what of the pages (a row that is not there: all)
        uint64_t see[PG], any[PG], all = ~0ull, some = 0;
#pragma unroll
        for (int h = 0; h < PG; ++h) {
          see[h] = any[h] = 0;
          if (good[h]) {
            const int kb = u.pages.page(u.k0 + 2 * j + half + h) * 64;
            if (all_see(p.m, u, kb)) {
              see[h] = any[h] = ~0ull;
            } else {
              any[h] = range_bits(0, u.s.L, kb);
              see[h] = live ? row_mask(p.m, u.s, i, bits, kb) : any[h];
            }
          }
          all &= see[h];
          some |= see[h];
        }
        const int sb = blk % C::NB;
        ok = ok && wait(&sfull[sb], (blk / C::NB) & 1, s_abort, p.status, SITE_SF);
        if (C::HALVES == 2) ok = !named_bar_or(2 + (sub & 1), 64, !ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t z[CH][32];
#pragma unroll
        for (int c = 0; c < CH; ++c) tmem_ld32(taddr + C::SW * sb + 32 * c, z[c]);
#pragma unroll
        for (int c = 0; c < CH; ++c) tmem_ld_wait_regs(z[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(&sfree[sb]);
          else mbar_arrive_cluster_relaxed(free_bar + 8 * sb);
        }
        look(j + 1);
        if (!__all_sync(0xffffffffu, all == ~0ull)) {
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const uint32_t sees = static_cast<uint32_t>(see[c >> 1] >> (32 * (c & 1)));
            const uint32_t others = static_cast<uint32_t>(any[c >> 1] >> (32 * (c & 1))) & ~sees;
            float hidden = 0.f;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (others >> e & 1) hidden = fmaf(__uint_as_float(z[c][e]), 0.f, hidden);
              if (!(sees >> e & 1)) z[c][e] = 0xff800000u;
            }
            if (hidden != 0.f) peak = INFINITY;          // a NaN: somebody else's row holds one
          }
        }
        // the row's reference, once it sees something (both of its threads know m_ref and
        // live, so both warps come here or neither)
        if (__any_sync(0xffffffffu, m_ref == -INFINITY && (C::HALVES == 2 ? live : some != 0))) {
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(z[c][e]));
          if (C::HALVES == 2) top = fmaxf(top, exchange(s_top, met++, top));
          if (m_ref == -INFINITY) m_ref = top * p.scale_log2;
        }
        const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
        float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float a0 = fmaf(__uint_as_float(z[c][e]), p.scale_log2, neg);
            const float a1 = fmaf(__uint_as_float(z[c][e + 1]), p.scale_log2, neg);
            peak = fmaxf(peak, fmaxf(a0, a1));
            const float p0 = ex2(a0), p1 = ex2(a1);
            sums[(e >> 1) & 3] += p0 + p1;
            z[c][e >> 1] = pack_bf16x2(p0, p1);
          }
        l_sum += (sums[0] + sums[1]) + (sums[2] + sums[3]);
        // P is free once the block that had its place has been multiplied
        const int pb = blk % C::NP;
        if (blk >= C::NP) ok = wait(&odone[pb], (blk / C::NP - 1) & 1, s_abort, p.status, SITE_O);
        if (ok && r < R) {
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(prow + (2 * pb + (c >> 1)) * C::QCH + (((4 * (c & 1) + q) ^ (r & 7)) << 4)) =
                  make_uint4(z[c][4 * q], z[c][4 * q + 1], z[c][4 * q + 2], z[c][4 * q + 3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&pready[pb]);
      }
      // what the epilogues of both CTAs need of this row, once they are done with the
      // unit before the last
      const int bu = at & 1;
      if (ok && at > 1) ok = wait(&lfree[bu], ((at >> 1) - 1) & 1, s_abort, p.status, SITE_L);
      if (C::HALVES == 2) ok = !named_bar_or(2 + (sub & 1), 64, !ok);
      if (!ok) break;
      if (C::HALVES == 2) {
        const float other = exchange(s_sum, at, l_sum);
        l_sum = half == 0 ? l_sum + other : other + l_sum;
      }
      // P of the maximum is 2^0 but for the reference's rounding: one that is far too high shows in
      // the sum, one far too low in the peak
      if (m_ref > -INFINITY && l_sum < LOST) peak = INFINITY;
      if (live && half == 0) {
        const float lse2 = l_sum == 0.f ? -INFINITY : m_ref + log2f(l_sum);
        if (!u.whole())
          p.part_lse[(2 * pair + (u.no > 0)) * 2 * R + rank * R + r] = lse2;
        else if (p.lse != nullptr)
          p.lse[static_cast<int64_t>(u.b) * p.m.T * p.H + g] = lse2 * 0.6931471805599453f;
      }
      if (r < R && half == 0) {
        const float inv = l_sum != 0.f ? 1.f / l_sum : 0.f;
        float* to = &s_inv[bu * 2 * R + rank * R + r];
        *to = inv;
        st_cluster_u32(smem_u32(to), rank ^ 1, __float_as_uint(inv));
      }
      if (__any_sync(0xffffffffu, live && peak > RISE)) {
        const bool far = __any_sync(0xffffffffu, live && peak > FAR);
        const bool bad = __any_sync(0xffffffffu, live && peak == INFINITY);
        if (far && live) note()[half] = m_ref + peak;
        if (lane == 0) {
          if (far && u.no < REDO) s_noted[sub * (REDO / 32) + (u.no >> 5)] |= 1u << (u.no & 31);
          for (int k = 0; k < 3; ++k) {
            if (k == 0 ? !far : k == 1 && !bad) continue;
            s_slow[3 * bu + k] = at + 1;
            st_cluster_u32(smem_u32(const_cast<int*>(s_slow + 3 * bu + k)), rank ^ 1, at + 1);
          }
        }
      }
      mbar_arrive_warp(&lfull[bu]);
    }
    for (int k = max(blk - C::NP, 0); k < blk; ++k)      // (not waited for above)
      settle(&odone[k % C::NP], k / C::NP & 1);
  } else {
    // ---- out: lane = dim 256 rank + 128 m + 32 sub + lane, a row a column ----
    const int sub = warp & 3;
    const uint32_t free_bar = mapa_u32(smem_u32(ofree), 0);
    int n = 0;
    bool ok = true;
    while (const Unit* up = ok ? feed.next() : nullptr) {
      const Unit& u = *up;
      const int at = feed.at;
      const int bu = at & 1, here = min(2 * R, u.rows - u.g0);   // rows that are there
      const int64_t first = static_cast<int64_t>(u.b) * p.m.T * p.H + u.g0;
      const int64_t part = static_cast<int64_t>(2 * pair + (u.no > 0)) * 2 * R;
      const bool parts = !u.whole();
      const float* inv = s_inv + bu * 2 * R;
      // this CTA's sums have gone to both; its first warp says so to the other
      ok = wait(&lfull[bu], (at >> 1) & 1, s_abort, p.status, SITE_L);
      if (ok && sub == 0 && lane == 0) mbar_arrive_cluster(mapa_u32(smem_u32(&lpeer[bu]), rank ^ 1));
      __syncwarp();
      if (ok) ok = wait<true>(&lpeer[bu], (at >> 1) & 1, s_abort, p.status, SITE_L);
      if (ok && u.nb > 0) ok = wait(ofull, n & 1, s_abort, p.status, SITE_O);
      if (!ok) break;
      tc_fence_after();
      const bool slow = s_slow[3 * bu] == at + 1, rise = s_slow[3 * bu + 2] == at + 1;
#pragma unroll 1
      for (int m = 0; m < 2; ++m) {
        const int dim = 256 * rank + 128 * m + 32 * sub + lane;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(sub * 32) << 16) + m * 2 * R;
#pragma unroll 1
        for (int c0 = 0; c0 < here && !slow; c0 += 32) {
          uint32_t x[32];
          if (u.nb > 0) {
            tmem_ld32(taddr + c0, x);
            tmem_ld_wait_regs(x);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 w = *reinterpret_cast<const float4*>(inv + c0 + e);
            x[e] = u.nb > 0 ? __float_as_uint(__uint_as_float(x[e]) * w.x) : 0;
            x[e + 1] = u.nb > 0 ? __float_as_uint(__uint_as_float(x[e + 1]) * w.y) : 0;
            x[e + 2] = u.nb > 0 ? __float_as_uint(__uint_as_float(x[e + 2]) * w.z) : 0;
            x[e + 3] = u.nb > 0 ? __float_as_uint(__uint_as_float(x[e + 3]) * w.w) : 0;
          }
          if (parts) {
            float* to = p.part_o + (part + c0) * kVlat + dim;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c0 + e < here) to[e * kVlat] = __uint_as_float(x[e]);
          } else {
            // two rows of a dim become two dims of a row, between two lanes: 4-byte stores
            const int odd = lane & 1;
            uint16_t* to = p.o + (first + c0 + odd) * kVlat + dim - odd;
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const uint32_t w = pack_bf16x2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
              const uint32_t v = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), odd ? 0x3276 : 0x5410);
              if (c0 + e + odd < here) *reinterpret_cast<uint32_t*>(to + e * kVlat) = v;
            }
          }
        }
        if (rise && u.nb > 0 && !slow) mark_beyond(taddr, here, inv, u.no, s_beyond, s_past);
        tc_fence_before();
        __syncwarp();
        if (u.nb > 0 && lane == 0) {                     // these columns may be overwritten
          if (rank == 0) mbar_arrive(&ofree[m]);
          else mbar_arrive_cluster_relaxed(free_bar + 8 * m);
        }
      }
      if (u.nb > 0) ++n;
      if (slow) {
        // (both CTAs come to the same)
        const bool again = !AGAIN && u.no < REDO && s_slow[3 * bu + 1] != at + 1;
        for (int r = rank * R + sub; !again && r < min(here, rank * R + R); r += 4) {
          attend_row(p, u.s, u.pages, u.k0, u.k1, u.b, u.g0 + r, parts ? p.part_o + (part + r) * kVlat : nullptr,
                     parts ? p.part_lse + part + r : nullptr);
          if (lane == 0) {                               // whoever waits, here or there, waits on
            const uint32_t beat = static_cast<uint32_t>(globaltimer_ns());
            s_abort[1] = static_cast<int>(beat);
            st_cluster_u32(smem_u32(const_cast<int*>(s_abort + 1)), rank ^ 1, beat);
          }
        }
        if (again && sub == 0 && lane == 0) s_redo[u.no >> 5] |= 1u << (u.no & 31), s_any[0] = 1;
        __syncwarp();
      }
      if (lane == 0) {                                   // the sums may be overwritten
        const uint32_t there = mapa_u32(smem_u32(&lfree[bu]), rank ^ 1);
        mbar_arrive(&lfree[bu]);
        mbar_arrive_cluster_relaxed(there);
      }
    }
  }
}

template <int R>
__device__ __noinline__ void roles_again(const CUtensorMap& tm_q, const CUtensorMap& tm_kv, const Params& p,
                                         uint8_t* sm, uint32_t tmem) {
  roles<R, true>(tm_q, tm_kv, p, sm, tmem);
}

// The pair's units marked in s_beyond, row by row: means of finite values, of which P V (P up
// to 2^FAR) was not finite.  By all warps of both CTAs.
template <int R>
__device__ __noinline__ void by_rows(const Params& p, uint8_t* sm) {
  const Shared<R> x(sm);
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, warp = threadIdx.x >> 5;
  Line<R> line(p, pair);
  Unit next;
  for (int no = 0; line.next(next); ++no) {
    const int k = min(no, REDO - 1);
    if (!(x.s_beyond[k >> 5] >> (k & 31) & 1)) continue;
    __syncthreads();
    if (threadIdx.x == 0) x.s_unit[0] = next;
    __syncthreads();
    const Unit& u = x.s_unit[0];
    const int64_t part = static_cast<int64_t>(2 * pair + (no > 0)) * 2 * R;
    for (int r = 2 * warp + rank; r < min(2 * R, u.rows - u.g0); r += 2 * (THREADS / 32))
      attend_row(p, u.s, u.pages, u.k0, u.k1, u.b, u.g0 + r, u.whole() ? nullptr : p.part_o + (part + r) * kVlat,
                 u.whole() ? nullptr : p.part_lse + part + r);
  }
}

template <int R>
__global__ void __launch_bounds__(THREADS, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_align1024(smem_raw);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), rank = blockIdx.x & 1;
  uint32_t tmem;
  cluster_arrive_relaxed();
  {
    const Shared<R> x(sm);
    if (tid == 0) {
      x.barriers(rank);
      x.s_abort[0] = x.s_abort[1] = 0;
      x.s_any[0] = x.s_go[0] = 0;
      x.s_past[0] = 0;
      for (int k = 0; k < 6; ++k) x.s_slow[k] = 0;
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_kv);
    }
    if (tid < 6 * REDO / 32) x.s_redo[tid] = 0;
    __syncwarp();
    cluster_wait();             // the other CTA runs
    if (warp == 2) {
      tmem_alloc_pair(x.tslot, 512);
      tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_arrive();
    if (warp != 0) {            // warp 0: in roles
      cluster_wait();
      pdl_wait();
      pdl_start_next();
    }
    tc_fence_after();
    tmem = warp != 0 ? *x.tslot : 0;
  }
  roles<R, false>(tm_q, tm_kv, p, sm, tmem);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  const Shared<R> x(sm);
  const bool again = x.s_any[0] != 0 && x.s_abort[0] == 0;
  if (again && tid == 0) st_cluster_u32(smem_u32(const_cast<int*>(x.s_go)), rank ^ 1, 1);
  cluster_sync();               // nothing of the pair's is read or arrived at any more
  if (again && x.s_go[0] != 0) {
    // all copies, products and arrivals of both CTAs are in: the barriers start over
    if (tid == 0) {
      for (int k = 0; k < Shared<R>::BARS; ++k) mbar_inval(&x.kfull[k]);
      x.barriers(rank);
      for (int k = 0; k < 6; ++k) x.s_slow[k] = 0;
    }
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    roles_again<R>(tm_q, tm_kv, p, sm, tmem);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  if (x.s_past[0] != 0 && x.s_abort[0] == 0) by_rows<R>(p, sm);
}

// Joins the pieces of the unit that pair blockIdx.x / 2R begins and does not end:
// lse = log2 sum 2^lse_k, o = sum 2^(lse_k - lse) o_k, in FP32 and in order.  A warp
// per row, 16 dims a lane (a CTA per row: 22 us for the 14,592 rows of 76 pairs).
template <int R>
__global__ void __launch_bounds__(128) combine_kernel(const Params p) {
  const int pair = blockIdx.x / (R / 2), r = blockIdx.x % (R / 2) * 4 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_start_next();
  // the pieces: the pair's last one, then the first ones of the next pairs for as long as they
  // go on with the unit.  What may be wanted is read at once (pairs that have had no unit
  // hold anything: not used)
  const int lane = threadIdx.x & 31, next = pair + lane;
  Stretch mine{-1, 0, -1, 0};
  float l = -INFINITY;
  if (next < p.pairs) {
    mine = p.stretch[next];
    if (lane > 0) l = p.part_lse[static_cast<int64_t>(next) * 4 * R + r];
  }
  const int head = __shfl_sync(0xffffffffu, mine.head, 0), slot = __shfl_sync(0xffffffffu, mine.slot, 0);
  if (head < 0) return;
  const int b = head / p.tiles, g = head % p.tiles * 2 * R + r;
  if (lane == 0) l = p.part_lse[static_cast<int64_t>(slot) * 2 * R + r];
  if (g >= seq_of(p.m, b).n * p.H) return;
  unsigned off = ~__ballot_sync(0xffffffffu, lane == 0 || (mine.first == head && mine.j0 > 0));
  int n = off != 0 ? __ffs(off) - 1 : 32;
  for (int k = next + 32; off == 0; k += 32) {
    const bool on = k < p.pairs && p.stretch[k].first == head && p.stretch[k].j0 > 0;
    off = ~__ballot_sync(0xffffffffu, on);
    n += off != 0 ? __ffs(off) - 1 : 32;
  }
  auto at = [&](int k) { return static_cast<int64_t>(k == 0 ? slot : 2 * (pair + k)) * 2 * R + r; };
  // their weights, a lane each
  if (lane >= n) l = -INFINITY;
  float top = l;
  for (int k = lane + 32; k < n; k += 32) top = fmaxf(top, p.part_lse[at(k)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int k0 = 0; k0 < n; k0 += 32) {
    if (k0 > 0) l = k0 + lane < n ? p.part_lse[at(k0 + lane)] : -INFINITY;
    const float w = l == -INFINITY ? 0.f : exp2f(l - top);
    const int m = min(32, n - k0);
#pragma unroll 2
    for (int k = 0; k < m; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float4* from = reinterpret_cast<const float4*>(p.part_o + at(k0 + k) * kVlat) + lane;
      float4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = from[32 * c];
      if (wk == 0.f) continue;
      sum += wk;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[4 * c] = fmaf(wk, v[c].x, acc[4 * c]);
        acc[4 * c + 1] = fmaf(wk, v[c].y, acc[4 * c + 1]);
        acc[4 * c + 2] = fmaf(wk, v[c].z, acc[4 * c + 2]);
        acc[4 * c + 3] = fmaf(wk, v[c].w, acc[4 * c + 3]);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t row = static_cast<int64_t>(b) * p.m.T * p.H + g;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    reinterpret_cast<uint2*>(p.o + row * kVlat)[32 * c + lane] =
        make_uint2(pack_bf16x2(acc[4 * c] * inv, acc[4 * c + 1] * inv),
                   pack_bf16x2(acc[4 * c + 2] * inv, acc[4 * c + 3] * inv));
  if (lane == 0 && p.lse != nullptr)
    p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

struct Plan {
  int R, tiles, blocks, pairs;      // blocks: of a unit, at most
  bool cut;
};
// span: the keys that one query may see at most; tree: they are all of the sequence's, from
// row 0.  Units are cut where the pair with the most whole ones would have three blocks more
// to do than the mean, and more than four: the pieces' outputs and their joining take about
// as long (1 x 1 over 400 rows, four blocks: 15.3 us whole, 15.6 cut; over 600, five: 17.8
// whole, 15.8 cut; 4 x 1 over 300: 13.6 whole, 17.8 cut).
Plan plan(int B, int T, int H, int64_t span, bool tree) {
  Plan q{};
  const int64_t rows = static_cast<int64_t>(T) * H, most = num_sms() / 2;
  auto set = [&](int R) {
    q.R = R;
    q.tiles = static_cast<int>((rows + 2 * R - 1) / (2 * R));
    const int64_t tokens = (2 * R + H - 2) / H + 1;      // of a unit
    q.blocks = static_cast<int>(tree ? (span + 127) / 128 : (span + tokens + 64) / 128 + 2);
  };
  // 96 rows a CTA copy the least per row; 64 have the shorter chain from a block to the
  // next, which counts where a pair has few blocks (5 trees of 33 tokens, 8 heads: 25.5
  // us against 28.8; 2048 queries, window 1024: 438 against 409)
  set(rows <= 96 ? 48 : rows <= 128 ? 64 : 96);
  if (q.R == 96 && static_cast<int64_t>(B) * q.tiles * q.blocks < 4 * most) set(64);
  const int64_t units = static_cast<int64_t>(B) * q.tiles;
  const int64_t whole = (units + most - 1) / most * q.blocks * most;
  q.cut = whole > units * q.blocks + 3 * most && whole > 4 * most;
  const int64_t pieces = units * (q.cut ? q.blocks : 1);
  q.pairs = static_cast<int>(pieces < most ? pieces : most);
  return q;
}
size_t part_bytes(const Plan& q) {
  if (!q.cut) return 0;
  return static_cast<size_t>(q.pairs) * (2 * 2 * q.R * (kVlat + 1) * sizeof(float) + sizeof(Stretch));
}

template <int R>
dsa_status_t launch(const DenseArgs& a, const Plan& q, const Params& p, cudaStream_t stream) {
  using C = Cfg<R>;
  CUtensorMap tq, tk;
  // contiguous rows: none behind the last sequence's max_kv_len is read
  const int64_t kv_rows = a.kv.block_table != nullptr
                              ? a.kv.total_rows
                              : (a.B - 1) * a.kv.seq_stride + a.max_kv_len;
  if (!encode_tmap_2d(&tq, a.q_lat, static_cast<uint64_t>(a.B) * a.T * a.H, kRlat, kRlat * 2, 64, R, true) ||
      !encode_tmap_2d(&tk, a.kv.base, static_cast<uint64_t>(kv_rows), kRlat, kRlat * 2, 64, 64, true))
    return DSA_ERR_CUDA;
  if (cudaFuncSetAttribute(pair_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
      cudaSuccess)
    return launch_status("cudaFuncSetAttribute");
  launch_overlapped(pair_kernel<R>, static_cast<unsigned>(2 * q.pairs), THREADS, C::SMEM, 2, stream, tq, tk, p);
  const dsa_status_t st = launch_status("pair_kernel");
  if (st != DSA_OK || !q.cut) return st;
  launch_overlapped(combine_kernel<R>, static_cast<unsigned>(q.pairs * R / 2), 128, 0, 0, stream, p);
  return launch_status("combine_kernel");
}

}  // namespace dense

// What these and all smaller calls need at most: whether units are cut, and for how many pairs,
// goes up and down with the sizes (76 sequences may stay whole where 75 are cut).
size_t dense_scratch_bytes(int B, int T, int H, int64_t span, bool tree) {
  const int64_t rows = static_cast<int64_t>(T) * H, most = num_sms() / 2;
  dense::Plan q{};
  q.R = rows <= 96 ? 48 : rows <= 128 ? 64 : 96;
  const int64_t units = B * ((rows + 127) / 128);
  const int64_t blocks = tree ? (span + 127) / 128 : (span + 2 * q.R + 64) / 128 + 2;
  q.cut = units > most || blocks > 4;
  q.pairs = static_cast<int>(units < most && units * blocks < most ? units * blocks : most);
  return dense::part_bytes(q);
}

dsa_status_t dense_fwd_launch(const DenseArgs& a, cudaStream_t stream) {
  using namespace dense;
  int64_t span = a.max_kv_len;
  if (a.tree == nullptr && static_cast<int64_t>(a.window) + a.n_first < span)
    span = a.window + a.n_first > 0 ? a.window + a.n_first : 1;
  const Plan q = plan(a.B, a.T, a.H, span, a.tree != nullptr);
  if (a.scratch_bytes < part_bytes(q)) return DSA_ERR_WORKSPACE_TOO_SMALL;
  Params p{};
  p.q = a.q_lat;
  p.kv = store_of(a);
  p.m = mask_of(a);
  p.B = a.B;
  p.H = a.H;
  p.tiles = q.tiles;
  p.pairs = q.pairs;
  p.nominal = a.tree != nullptr ? 0 : q.blocks;
  p.cut = q.cut;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.o = a.o_lat;
  p.lse = a.lse;
  p.part_o = static_cast<float*>(a.scratch);
  const size_t rows = static_cast<size_t>(q.pairs) * 2 * 2 * q.R;
  p.part_lse = p.part_o + rows * kVlat;
  p.stretch = reinterpret_cast<Stretch*>(p.part_lse + rows);
  p.status = a.status;
  return q.R == 96   ? launch<96>(a, q, p, stream)
         : q.R == 64 ? launch<64>(a, q, p, stream)
                     : launch<48>(a, q, p, stream);
}

}  // namespace dsa
