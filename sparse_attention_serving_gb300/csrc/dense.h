// dense.h -- host-side launch interfaces of the append with rotated positions and
// of dense attention over latent rows (drafted trees, windows with first tokens,
// the windows' backward pass), shared between the C ABI layer and the kernels.
#pragma once
#include "internal.h"

namespace dsa {

// A dense 3D BF16 tensor map [z, rows, cols] with a {box_cols, box_rows, 1} box and
// 128-byte swizzle: boxes end with the rows of their z.
bool encode_tmap_3d(CUtensorMap* map, const void* base, uint64_t z, uint64_t rows, uint64_t cols,
                    uint32_t box_cols, uint32_t box_rows);

struct AppendRopeArgs {
  const float* k_pre;
  const uint16_t* kv_new;
  RowStore k_cache;        // written through (base is cast to non-const)
  RowStore kv_cache;
  const int32_t* q_start;
  const float* rope;       // [n_pos, 64]: 32 cosines, 32 sines
  int n_pos;
  const int32_t* pos;      // [B, Tq] or null: q_start[b] + i
  const int32_t* n_new;    // [B] or null: Tq
  const uint16_t* q_pe;    // [B, Tq, H, 64] or null
  uint16_t* q_lat;         // [B, Tq, H, 576], dims 512..575 written
  int H;
  const uint16_t* q_idx;   // [B, Tq, H_I, D_I] or null
  uint16_t* q_idx_out;     // may be q_idx
  int H_I;
  int B, Tq, D_I, kv_style, key_style;
  float eps;
  uint32_t* status;
};
dsa_status_t cache_append_rope_launch(const AppendRopeArgs& a, cudaStream_t stream);

// Attention of every query of a sequence to a range of rows under a mask that
// follows from positions (window) or from the drafted tree.
struct DenseArgs {
  const uint16_t* q_lat;
  RowStore kv;
  const int32_t* pos0;     // [B] window: q_start; tree: kv_len (the prefix)
  const int32_t* lim;      // [B] window: kv_len; tree: n_draft, or null (T)
  const uint64_t* tree;    // [B, T] who each drafted token sees; null: window
  int B, T, H, max_kv_len;
  int window, n_first;
  float scale;
  uint16_t* o_lat;
  float* lse;              // or null
  uint32_t* status;
  void* scratch;           // split partials; may be null when there are none
  size_t scratch_bytes;
};
// span: the keys that one query may see at most
size_t dense_scratch_bytes(int B, int T, int H, int64_t span, bool tree);
dsa_status_t dense_fwd_launch(const DenseArgs& a, cudaStream_t stream);

struct WindowBwdArgs {
  DenseArgs f;             // q_lat, kv (contiguous), masks; o_lat and lse are inputs here
  const uint16_t* d_o;
  uint16_t* dq;
  uint16_t* dkv;           // [B, seq_stride, 576]
};
size_t window_bwd_scratch_bytes(int B, int T, int H, int max_kv_len, int64_t span);
dsa_status_t window_bwd_launch(const WindowBwdArgs& a, cudaStream_t stream);

}  // namespace dsa
