// Private interface between the C-ABI layer (gdr_attn_api.cpp) and the kernels of
// the softmax-attention layers: rotary positions, attention over packed documents,
// the cache held in 4 bits and the attention of new tokens over it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gdr.h"

namespace gdr {

// ---- rotary positions ----

// A block's share: `tokens` of one chunk (or of the row of tokens, with positions),
// whose sines and cosines it forms once for all heads of its part `hparts` of them.
// Few tokens are spread over blocks and heads, many take 8 a block.
struct RopePlan {
  int tokens, hparts;
  int64_t blocks;
};
inline RopePlan rope_plan(const gdr_rope &p) {
  RopePlan r;
  const int64_t rows = (int64_t)p.T * (p.H_q + p.H_k);
  r.tokens = p.T >= 2048 ? 8 : p.T >= 512 ? 4 : 1;
  // a block of few tokens takes at most 32 of their heads
  const int heads = p.H_q + p.H_k;
  r.hparts = rows < 65536 ? (heads + 31) / 32 : 1;
  r.blocks = (p.positions ? ((int64_t)p.T + r.tokens - 1) / r.tokens : (int64_t)p.n_chunks * (64 / r.tokens)) * r.hparts;
  return r;
}
hipError_t launch_rope(const gdr_rope &p, bool back, const void *q, int64_t q_stride, const void *k, int64_t k_stride, void *qo,
                       int64_t qo_stride, void *ko, int64_t ko_stride, hipStream_t stream);

// ---- attention over packed documents ----

// Rows of a query tile and keys of a key tile: a block's, 32 to each of its wavefronts.
constexpr int ATT_TILE = 128;
// A tile of the table (both kinds), 8 int32: its first row in the packed batch, its
// rows, the other side's first row in the batch and its document's rows there, the
// tile's first row within the document, Lk - Lq, two spare.
constexpr int ATT_ENTRY = 8;

// The dk, dv kernel's blocks: (key tile, kv head, part of the kv head's query heads).
// Where tiles and kv heads leave the chip half empty, the query heads of a kv head
// are dealt to `parts` blocks whose fp32 sums a second kernel adds in order.
inline int attn_parts(int64_t tiles, int H_kv, int group) {
  int parts = 1;
  while (parts < group && group % (2 * parts) == 0 && tiles * H_kv * parts < 384) parts *= 2;
  return parts;
}
// Workspace of the backward: lse and delta of every row and head as the matrix kernels take
// them, then the parts' sums.
struct AttnWorkspace {
  int64_t stats, partial, bytes;
  int parts;
};
inline AttnWorkspace attn_workspace(int32_t T_q, int32_t T_k, int32_t n_k_tiles, int32_t H_q, int32_t H_kv) {
  AttnWorkspace w;
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  w.parts = attn_parts(n_k_tiles, H_kv, H_q / H_kv);
  w.stats = up((int64_t)T_q * H_q * 4);
  w.partial = w.parts > 1 ? up((int64_t)T_k * H_kv * 128 * 4) : 0;
  w.bytes = 2 * w.stats + 2 * w.parts * w.partial;
  return w;
}
hipError_t launch_attn_fwd(const gdr_attn &p, uint16_t *o, float *lse, hipStream_t stream);
hipError_t launch_attn_dq(const gdr_attn &p, const uint16_t *o, const float *lse, const uint16_t *dout, uint16_t *dq,
                          int64_t dq_stride, void *ws, hipStream_t stream);
hipError_t launch_attn_dkv(const gdr_attn &p, const uint16_t *dout, uint16_t *dk, int64_t dk_stride, uint16_t *dv,
                           int64_t dv_stride, void *ws, hipStream_t stream);
hipError_t launch_attn_join(const gdr_attn &p, uint16_t *dk, int64_t dk_stride, uint16_t *dv, int64_t dv_stride, void *ws,
                            hipStream_t stream);

// ---- the cache and the attention over it ----

hipError_t launch_kv(const gdr_kv &p, bool store, int32_t T, const int32_t *cu, const int32_t *start, uint16_t *k,
                     int64_t k_stride, uint16_t *v, int64_t v_stride, hipStream_t stream);

// A sequence's tokens are shared by `splits` blocks for every kv head and 16 rows of
// its run (`row_tiles` of them are launched; longer runs loop).  A block takes at least
// STEP_UNIT tokens; a launch has about STEP_BLOCKS blocks.
constexpr int STEP_UNIT = 128;
constexpr int STEP_BLOCKS = 8192;
struct StepPlan {
  int splits, row_tiles;
  int64_t blocks;
  int64_t bytes;  // workspace
};
inline StepPlan step_plan(int32_t T, int32_t N, int32_t H_q, int32_t H_kv, int32_t max_pages, int32_t page) {
  StepPlan s;
  const int64_t run = N > 0 ? std::max<int64_t>(1, ((int64_t)T + N - 1) / N) : 1;
  s.row_tiles = (int)std::min<int64_t>((run * (H_q / H_kv) + 15) / 16, 4096);
  const int64_t items = std::max<int64_t>(1, (int64_t)N * H_kv * s.row_tiles);
  const int64_t most = ((int64_t)max_pages * page + STEP_UNIT - 1) / STEP_UNIT;
  s.splits = (int)std::max<int64_t>(1, std::min<int64_t>(most, STEP_BLOCKS / items));
  s.blocks = items * s.splits;
  s.bytes = s.splits > 1 ? ((int64_t)T * H_q * s.splits * 130 * 4 + 255) / 256 * 256 : 0;
  return s;
}
hipError_t launch_attn_step(const gdr_kv &c, const gdr_attn_step &p, uint16_t *o, void *ws, const StepPlan &plan, hipStream_t stream);
hipError_t launch_attn_step_join(const gdr_kv &c, const gdr_attn_step &p, uint16_t *o, void *ws, const StepPlan &plan,
                                 hipStream_t stream);

}  // namespace gdr
