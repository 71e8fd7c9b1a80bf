// cache_append_rope.cu -- the append before the indexer for layers whose keys carry
// their position as a rotation: LayerNorm of the new indexer keys, rotation of the
// keys' and latent rows' position dims, append to the two caches, and the rotation
// of the queries that go with them, in one launch.
//
//   (a, b) -> (a cos - b sin, b cos + a sin) for the 32 dim pairs (i, i + 32) or
//   (2i, 2i + 1) of 64 dims, cos and sin from the caller's table at the token's
//   position; FP32, one rounding to BF16 (the key's after LayerNorm and rotation).
//
// Bound: HBM, or the launch for a few tokens.  Per token 12 KB + 12 KB of queries
// (96 heads) and 16 KB + 16 KB of indexer queries (64 x 128) go through beside
// 4.4 KB of key and rows, so the work is dealt out in items of 32 bytes in and 32
// out, one a thread: an item is two 16-byte units that hold both dims of eight
// pairs (units 2v and 2v + 1, or v and v + 4), so that either pairing needs no
// exchange between threads.  An item's eight angles are two 32-byte reads of the
// token's table row, which the heads of a token share in L1.
#include <cuda_bf16.h>

#include "dense.h"
#include "dsa_status.cuh"
#include "sm103.cuh"

namespace dsa {
namespace apr {

constexpr int THREADS = 128;                   // 64 to 1024 measured at 8192 tokens: 88.6 us at 128
enum : uint32_t { SITE_KROW = 0x610, SITE_VROW = 0x611, SITE_POS = 0x612, SITE_NEW = 0x613 };
enum { NONE = 0, HALVES = 1, PAIRS = 2 };
constexpr int KEY_ITEMS = 32;                  // the key: a warp
constexpr int ROW_ITEMS = 64;                  // the latent row: 32 copied, 4 rotated, the rest idle

struct Rows {
  uint16_t* base;
  const int32_t* bt;
  int64_t stride;
  int32_t max_pages, num_pages;
  int width;
};
struct Params {
  const float* k_pre;
  const uint16_t* kv_new;
  Rows k, kv;
  const int32_t* q_start;
  const float* rope;
  const int32_t* pos;
  const int32_t* n_new;
  const uint16_t* q_pe;
  uint16_t* q_lat;
  const uint16_t* q_idx;
  uint16_t* q_idx_out;
  int n_pos, B, Tq, H, H_I, kv_style, key_style;
  int pe_items, idx_items, items, chunks;      // per token; idx_items: 4 or 8 per head
  float eps;
  uint32_t* status;
};

// The row of position pos of sequence b, or null if the store has no such row.
__device__ __forceinline__ uint16_t* row_at(const Rows& s, int b, int pos) {
  if (pos < 0) return nullptr;
  int64_t r;
  if (s.bt == nullptr) {
    if (pos >= s.stride) return nullptr;
    r = static_cast<int64_t>(b) * s.stride + pos;
  } else {
    const int pg = pos >> 6;
    if (pg >= s.max_pages) return nullptr;
    const int id = __ldg(s.bt + static_cast<int64_t>(b) * s.max_pages + pg);
    if (id < 0 || id >= s.num_pages) return nullptr;
    r = static_cast<int64_t>(id) * kPage + (pos & (kPage - 1));
  }
  return s.base + r * s.width;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Two 16-byte units of a row, as an item moves them: u0 and u1, rotated by the eight
// angles 8v..8v+7 or (NONE) as they are.
struct Item {
  const uint16_t* src;
  int u0, u1, v, style;
};
__device__ __forceinline__ Item item_of(const uint16_t* src, int v, int style) {
  return style == HALVES ? Item{src, v, v + 4, v, style} : Item{src, 2 * v, 2 * v + 1, v, style};
}
__device__ __forceinline__ void put_item(const Item& it, uint4 w0, uint4 w1, uint16_t* dst,
                                         const float* angles) {
  const int v = it.v, style = it.style;
  uint4* to0 = reinterpret_cast<uint4*>(dst) + it.u0;
  uint4* to1 = reinterpret_cast<uint4*>(dst) + it.u1;
  if (style == NONE) {
    *to0 = w0;
    *to1 = w1;
    return;
  }
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float4 cc = __ldg(reinterpret_cast<const float4*>(angles + 8 * v) + e);
    const float4 ss = __ldg(reinterpret_cast<const float4*>(angles + 32 + 8 * v) + e);
    c[4 * e] = cc.x, c[4 * e + 1] = cc.y, c[4 * e + 2] = cc.z, c[4 * e + 3] = cc.w;
    s[4 * e] = ss.x, s[4 * e + 1] = ss.y, s[4 * e + 2] = ss.z, s[4 * e + 3] = ss.w;
  }
  float x[8], y[8], r0[8], r1[8];
  unpack(w0, x);
  unpack(w1, y);
  if (style == HALVES) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      r0[e] = x[e] * c[e] - y[e] * s[e];
      r1[e] = y[e] * c[e] + x[e] * s[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r0[2 * e] = x[2 * e] * c[e] - x[2 * e + 1] * s[e];
      r0[2 * e + 1] = x[2 * e + 1] * c[e] + x[2 * e] * s[e];
      r1[2 * e] = y[2 * e] * c[4 + e] - y[2 * e + 1] * s[4 + e];
      r1[2 * e + 1] = y[2 * e + 1] * c[4 + e] + y[2 * e] * s[4 + e];
    }
  }
  *to0 = pack(r0);
  *to1 = pack(r1);
}

// LayerNorm (unit gain, zero bias, population variance of the centred values) and
// rotation of one key by a warp; lane l holds dims PER l ... PER l + PER - 1.
template <int D>
__device__ __forceinline__ void key_row(const float* src, uint16_t* dst, int lane, int style,
                                        float eps, const float* angles) {
  constexpr int PER = D / 32;
  float x[PER];
#pragma unroll
  for (int e = 0; e < PER; e += 2) {
    const float2 v = __ldg(reinterpret_cast<const float2*>(src + PER * lane + e));
    x[e] = v.x, x[e + 1] = v.y;
  }
  float s = 0.f, q = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) s += x[e];
  const float mean = warp_sum(s) / static_cast<float>(D);
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    x[e] -= mean;
    q = fmaf(x[e], x[e], q);
  }
  const float inv = 1.f / sqrtf(warp_sum(q) / static_cast<float>(D) + eps);
#pragma unroll
  for (int e = 0; e < PER; ++e) x[e] *= inv;
  if (style != NONE) {
    float y[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) y[e] = __shfl_xor_sync(0xffffffffu, x[e], 32 / PER);
    if (PER * lane < 64) {
#pragma unroll
      for (int e = 0; e < PER; e += 2) {
        const int d = PER * lane + e;
        if (style == HALVES) {
          const float2 c = __ldg(reinterpret_cast<const float2*>(angles + (d & 31)));
          const float2 w = __ldg(reinterpret_cast<const float2*>(angles + 32 + (d & 31)));
          const float sg = d < 32 ? -1.f : 1.f;
          x[e] = x[e] * c.x + sg * (y[e] * w.x);
          x[e + 1] = x[e + 1] * c.y + sg * (y[e + 1] * w.y);
        } else {
          const float c = __ldg(angles + d / 2), w = __ldg(angles + 32 + d / 2);
          const float a = x[e], b = x[e + 1];
          x[e] = a * c - b * w;
          x[e + 1] = b * c + a * w;
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<uint32_t*>(dst + PER * lane + e) = pack_bf16x2(x[e], x[e + 1]);
}

// Chunk c of a token's items: CTAs token * chunks + c.  Items in the order key,
// latent row, q_pe, q_idx; the key's warp is whole (KEY_ITEMS and the chunk's start
// are multiples of 32).
template <int D>
__global__ void __launch_bounds__(THREADS) append_rope_kernel(const Params p) {
  const int64_t tok = blockIdx.x / static_cast<unsigned>(p.chunks);
  const int first = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.chunks)) * THREADS + threadIdx.x;
  const int b = static_cast<int>(tok / p.Tq), i = static_cast<int>(tok % p.Tq);

  // what the item reads does not depend on the token's place: its loads go out first
  Item it{nullptr, 0, 0, 0, NONE};
  uint16_t* dst = nullptr;                       // of a query's item
  const int row_item = first - KEY_ITEMS, pe = row_item - ROW_ITEMS, ix = pe - p.pe_items;
  if (row_item >= 0 && row_item < 32) {
    it = Item{p.kv_new + tok * kRlat, row_item, row_item + 32, 0, NONE};
  } else if (row_item >= 32 && row_item < 36) {
    it = item_of(p.kv_new + tok * kRlat + kVlat, row_item - 32, p.kv_style);
  } else if (pe >= 0 && pe < p.pe_items) {
    const int64_t h = tok * p.H + (pe >> 2);
    it = item_of(p.q_pe + h * 64, pe & 3, p.kv_style);
    dst = p.q_lat + h * kRlat + kVlat;
  } else if (ix >= 0 && ix < p.idx_items) {
    // a head's dims 0..63 rotated by four items; 64..127 copied by four more, unless
    // the queries are rotated where they are
    const int per = p.idx_items / p.H_I, v = ix % per;
    const int64_t at = (tok * p.H_I + ix / per) * D + (v < 4 ? 0 : 64);
    it = item_of(p.q_idx + at, v & 3, v < 4 ? p.key_style : NONE);
    dst = p.q_idx_out + at;
  } else if (first >= KEY_ITEMS) {
    return;
  }
  uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
  if (it.src != nullptr) {
    w0 = reinterpret_cast<const uint4*>(it.src)[it.u0];
    w1 = reinterpret_cast<const uint4*>(it.src)[it.u1];
  }

  const int n = p.n_new != nullptr ? __ldg(p.n_new + b) : p.Tq;
  const int row = __ldg(p.q_start + b) + i;
  const int at = p.pos != nullptr ? __ldg(p.pos + tok) : row;
  if (i == 0 && first == 0 && (n < 0 || n > p.Tq))
    status_raise(p.status, DSA_ERR_BAD_INDEX, SITE_NEW, static_cast<uint32_t>(b));
  if (i >= n) return;
  if (at < 0 || at >= p.n_pos) {
    if (first == 0) status_raise(p.status, DSA_ERR_BAD_INDEX, SITE_POS, static_cast<uint32_t>(at));
    return;
  }
  const float* angles = p.rope + static_cast<int64_t>(at) * 64;
  if (first < KEY_ITEMS) {
    uint16_t* key = row_at(p.k, b, row);
    if (key != nullptr)
      key_row<D>(p.k_pre + tok * D, key, first, p.key_style, p.eps, angles);
    else if (first == 0)
      status_raise(p.status, DSA_ERR_BAD_INDEX, SITE_KROW, static_cast<uint32_t>(row));
    return;
  }
  if (dst == nullptr) {
    dst = row_at(p.kv, b, row);
    if (dst == nullptr) {
      if (row_item == 0) status_raise(p.status, DSA_ERR_BAD_INDEX, SITE_VROW, static_cast<uint32_t>(row));
      return;
    }
    if (row_item >= 32) dst += kVlat;
  }
  put_item(it, w0, w1, dst, angles);
}

Rows rows_of(const RowStore& s, int width) {
  return Rows{const_cast<uint16_t*>(s.base), s.block_table, s.seq_stride, s.max_pages, s.num_pages,
              width};
}

}  // namespace apr

dsa_status_t cache_append_rope_launch(const AppendRopeArgs& a, cudaStream_t stream) {
  using namespace apr;
  Params p{};
  p.k_pre = a.k_pre;
  p.kv_new = a.kv_new;
  p.k = rows_of(a.k_cache, a.D_I);
  p.kv = rows_of(a.kv_cache, kRlat);
  p.q_start = a.q_start;
  p.rope = a.rope;
  p.pos = a.pos;
  p.n_new = a.n_new;
  p.q_pe = a.q_pe;
  p.q_lat = a.q_lat;
  p.q_idx = a.q_idx;
  p.q_idx_out = a.q_idx_out;
  p.n_pos = a.n_pos;
  p.B = a.B;
  p.Tq = a.Tq;
  p.H = a.H;
  p.H_I = a.H_I;
  p.kv_style = a.kv_style;
  p.key_style = a.key_style;
  p.pe_items = a.q_pe != nullptr ? 4 * a.H : 0;
  p.idx_items = a.q_idx == nullptr ? 0
                : a.D_I == 128 && a.q_idx != a.q_idx_out ? 8 * a.H_I : 4 * a.H_I;
  p.items = KEY_ITEMS + ROW_ITEMS + p.pe_items + p.idx_items;
  p.chunks = (p.items + THREADS - 1) / THREADS;
  p.eps = a.eps;
  p.status = a.status;
  const int64_t ctas = static_cast<int64_t>(a.B) * a.Tq * p.chunks;
  if (ctas > 0x7fffffff) return DSA_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(ctas);
  if (a.D_I == 128)
    append_rope_kernel<128><<<grid, THREADS, 0, stream>>>(p);
  else
    append_rope_kernel<64><<<grid, THREADS, 0, stream>>>(p);
  return launch_status("append_rope_kernel");
}

}  // namespace dsa
