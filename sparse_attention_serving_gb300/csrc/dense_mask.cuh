// dense_mask.cuh -- which rows a query sees in dense latent attention, 64 rows
// (a cache page) at a time.
#pragma once
#include "dense.h"
#include "dsa_status.cuh"

namespace dsa {
namespace dense {

enum : uint32_t { SITE_SEQ = 0x700, SITE_PAGE = 0x701, SITE_DRAFT = 0x702 };

struct Mask {
  const int32_t* pos0;
  const int32_t* lim;
  const uint64_t* tree;
  int T, max_kv_len, window, n_first;
};

// One sequence, as every role resolves it.
struct Seq {
  int pos0;   // window: position of query 0; tree: rows before the drafts
  int L;      // rows that exist
  int n;      // queries; those behind them are left alone
  bool ok;    // false: no query sees anything
};
__device__ __forceinline__ Seq seq_of(const Mask& m, int b) {
  Seq s;
  s.pos0 = m.pos0[b];
  if (m.tree != nullptr) {
    const int n = m.lim != nullptr ? m.lim[b] : m.T;
    s.n = min(max(n, 0), m.T);
    s.ok = s.pos0 >= 0 && s.pos0 <= m.max_kv_len - s.n;
    s.L = s.pos0 + s.n;
  } else {
    s.n = m.T;
    s.L = m.lim[b];
    s.ok = s.pos0 >= 0 && s.L <= m.max_kv_len && s.pos0 < s.L;
  }
  return s;
}
// What is wrong with the sequence, if anything: said once, by one thread.
__device__ __forceinline__ void report_seq(const Mask& m, const Seq& s, int b, uint32_t* status) {
  if (m.tree != nullptr) {
    if (m.lim != nullptr && s.n != m.lim[b])
      status_raise(status, DSA_ERR_BAD_INDEX, SITE_DRAFT, static_cast<uint32_t>(b));
    if (!s.ok && s.n > 0) status_raise(status, DSA_ERR_BAD_INDEX, SITE_SEQ, static_cast<uint32_t>(b));
  } else if (!s.ok || s.pos0 > s.L - s.n) {
    status_raise(status, DSA_ERR_BAD_INDEX, SITE_SEQ, static_cast<uint32_t>(b));
  }
}

// Bits of [lo, hi) that fall on the 64 rows from kb on.
__device__ __forceinline__ uint64_t range_bits(int lo, int hi, int kb) {
  lo = max(max(lo, 0) - kb, 0);
  hi = min(hi - kb, 64);
  if (lo >= hi) return 0;
  return (~0ull >> (64 - (hi - lo))) << lo;
}
// The rows kb..kb+63 that query i sees (kb >= 0); bits = tree[b, i], or not used.
__device__ __forceinline__ uint64_t row_mask(const Mask& m, const Seq& s, int i, uint64_t bits, int kb) {
  if (!s.ok || i >= s.n) return 0;
  if (m.tree != nullptr) {
    uint64_t v = range_bits(0, s.pos0, kb);
    bits &= s.n >= 64 ? ~0ull : (1ull << s.n) - 1;
    const int at = s.pos0 - kb;
    if (at >= 0)
      v |= at < 64 ? bits << at : 0;
    else
      v |= at > -64 ? bits >> -at : 0;
    return v;
  }
  const int t = s.pos0 + i;
  if (t >= s.L) return 0;
  return range_bits(t - m.window + 1, t + 1, kb) | range_bits(0, min(m.n_first, t + 1), kb);
}

// Pages (64 rows) that the queries i0..i1 of a sequence may see: [0, head) and
// [tail, end).
struct Pages {
  int head, tail, end;
  __device__ __forceinline__ int count() const { return head + end - tail; }
  __device__ __forceinline__ int page(int k) const { return k < head ? k : tail + k - head; }
};
__device__ __forceinline__ Pages pages_of(const Mask& m, const Seq& s, int i0, int i1) {
  Pages p{0, 0, 0};
  i1 = min(i1, s.n - 1);
  if (!s.ok || i0 > i1) return p;
  if (m.tree != nullptr) {
    p.end = (s.L + 63) >> 6;
    return p;
  }
  const int t0 = s.pos0 + i0, t1 = min(s.pos0 + i1, s.L - 1);
  if (t0 > t1) return p;
  p.end = m.window > 0 ? (t1 >> 6) + 1 : 0;
  p.tail = m.window > 0 ? max(t0 - m.window + 1, 0) >> 6 : 0;
  p.head = (min(m.n_first, t1 + 1) + 63) >> 6;
  if (p.head >= p.tail) {        // the ranges meet
    p.end = max(p.end, p.head);
    p.head = p.tail = 0;
  }
  return p;
}

struct Store {
  const uint16_t* base;
  int64_t seq_stride;
  const int32_t* block_table;
  int32_t max_pages, num_pages;
};
// First physical row of page `pg` of sequence b, or -1 (a page outside the pool).
__device__ __forceinline__ int64_t page_row(const Store& kv, int b, int pg) {
  if (kv.block_table == nullptr) return static_cast<int64_t>(b) * kv.seq_stride + pg * 64;
  if (pg >= kv.max_pages) return -1;
  const int id = kv.block_table[static_cast<int64_t>(b) * kv.max_pages + pg];
  return id < 0 || id >= kv.num_pages ? -1 : static_cast<int64_t>(id) * kPage;
}

inline Mask mask_of(const DenseArgs& a) {
  return Mask{a.pos0, a.lim, a.tree, a.T, a.max_kv_len, a.window, a.n_first};
}
inline Store store_of(const DenseArgs& a) {
  return Store{a.kv.base, a.kv.seq_stride, a.kv.block_table, a.kv.max_pages, a.kv.num_pages};
}

}  // namespace dense
}  // namespace dsa
