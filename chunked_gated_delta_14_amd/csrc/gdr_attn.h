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

// Rows of a query tile, and keys of a key tile: 32 to each of a block's four and eight wavefronts.
constexpr int ATT_QTILE = 128, ATT_KTILE = 256;
// A tile of the table (both kinds), 8 int32: its first row in the packed batch, its
// rows, the other side's first row in the batch and its document's rows there, the
// tile's first row within the document, Lk - Lq, the other side's first row (a multiple
// of 64) and end that its rows meet.
constexpr int ATT_ENTRY = 8;

// The table: the entries of the query tiles and of the key tiles, then the lists of parts of
// either kind by level, an item of 2 int32: the tile, and the part + its tile's parts << 16.  Items with the most
// steps come first, a tile's parts in a row; an item's place in the list is its slot in the workspace.
constexpr int ATT_PARTS = 64;
inline int attn_parts(int64_t steps, int level) {
  return (int)std::min<int64_t>(std::max<int64_t>((steps + (int64_t(1) << level) - 1) >> level, 1), ATT_PARTS);
}
inline int64_t attn_items(const int32_t (&items)[GDR_ATTN_LEVELS], int levels) {
  int64_t n = 0;
  for (int i = 0; i < levels; ++i) n += items[i];
  return n;
}
// How a launch shares its tiles' steps.  Where tiles and heads would leave compute units
// idle, or a few long tiles would run on after the others, it takes the list of parts whose
// steps come nearest the mean load of `slots` blocks, but not fewer than `least`, which a block's start and
// its part's way through memory outweigh; a second kernel then joins the parts' fp32
// results in order, a block for a slot and head, which takes its share of its tile's rows.
struct AttnShare {
  int level;        // -1: whole tiles
  int parts;        // the longest tile's
  int64_t blocks;   // tiles or parts, of one head
  int64_t items;    // the list's place in the table, in int32
  int64_t slots;    // the list's first items, which hold all that are one of several parts
};
inline AttnShare attn_share(const gdr_attn_plan &p, bool keys, int64_t heads, int slots, int least) {
  const int32_t (&items)[GDR_ATTN_LEVELS] = keys ? p.k_items : p.q_items;
  const int32_t tiles = keys ? p.n_k_tiles : p.n_q_tiles, longest = keys ? p.k_longest : p.q_longest;
  const int64_t mean = std::max<int64_t>(least, ((keys ? p.k_steps : p.q_steps) * heads + slots - 1) / slots);
  AttnShare s{-1, 1, tiles, 0, 0};
  if (longest <= mean + mean / 2) return s;
  int level = 0;
  while (level < GDR_ATTN_LEVELS - 1 && (int64_t(4) << level) <= 3 * mean) ++level;  // the power of two within 3/4 and 3/2 of it
  if (!items[level]) return s;
  s.level = level;
  s.parts = attn_parts(longest, level);
  s.blocks = items[level];
  s.items = ((int64_t)p.n_q_tiles + p.n_k_tiles) * ATT_ENTRY + 2 * ((keys ? attn_items(p.q_items, GDR_ATTN_LEVELS) : 0) + attn_items(items, level));
  // one of several parts has more than half of 2^level steps, and so has what stands before it
  s.slots = std::min<int64_t>(items[level], 2 * (keys ? p.k_steps : p.q_steps) >> level);
  return s;
}
// Blocks of 128 query rows run two to a compute unit, and two rounds of them even out; blocks of 256 keys, whose
// steps are rows of all of a kv head's query heads, run one to a unit.
constexpr int ATT_Q_SLOTS = 1024, ATT_K_SLOTS = 384;
inline AttnShare attn_q_share(const gdr_attn &p) { return attn_share(p.plan, false, p.H_q, ATT_Q_SLOTS, 4); }
inline AttnShare attn_k_share(const gdr_attn &p) {
  const int group = p.H_q / p.H_kv;
  return attn_share(p.plan, true, p.H_kv, ATT_K_SLOTS, std::max(1, 4 / group));
}
// The workspace.  Forward: the parts' rows [slot][H_q][128][128], then their maxima and sums
// [slot][H_q][128][2].  Backward: lse and delta of every row and head as the
// matrix kernels take them, [H_q][T_q] each; the parts of dq [slot][H_q][128][128], of dk and of dv
// [slot][H_kv][256][128].  2^level is more than 3/4 of a block's mean load, so slots times heads are below 2731 (8/3 of
// 1024 blocks) and 1024: 182 MB forward, and 447 MB beside lse and delta backward, whatever a batch holds (of parts of up to 2^11 steps).
constexpr int64_t ATT_QPART = ATT_QTILE * 128, ATT_KPART = ATT_KTILE * 128;  // floats of a slot's head
struct AttnWorkspace {
  int64_t stats, fwd, bwd;  // bytes: a row of stats, the whole
  AttnShare q, k;
};
inline AttnWorkspace attn_workspace(const gdr_attn &p) {
  AttnWorkspace w;
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  w.q = attn_q_share(p);
  w.k = attn_k_share(p);
  w.stats = up((int64_t)p.T_q * p.H_q * 4);
  w.fwd = w.q.slots * p.H_q * (ATT_QPART + 2 * ATT_QTILE) * 4;
  w.bwd = 2 * w.stats + (w.q.slots * p.H_q * ATT_QPART + 2 * w.k.slots * p.H_kv * ATT_KPART) * 4;
  return w;
}
hipError_t launch_attn_fwd(const gdr_attn &p, uint16_t *o, float *lse, void *ws, hipStream_t stream);
hipError_t launch_attn_fwd_join(const gdr_attn &p, uint16_t *o, float *lse, void *ws, hipStream_t stream);
hipError_t launch_attn_dq(const gdr_attn &p, const uint16_t *o, const float *lse, const uint16_t *dout, uint16_t *dq,
                          int64_t dq_stride, void *ws, hipStream_t stream);
hipError_t launch_attn_dkv(const gdr_attn &p, const uint16_t *dout, uint16_t *dk, int64_t dk_stride, uint16_t *dv,
                           int64_t dv_stride, void *ws, hipStream_t stream);
hipError_t launch_attn_bwd_join(const gdr_attn &p, uint16_t *dq, int64_t dq_stride, uint16_t *dk, int64_t dk_stride, uint16_t *dv,
                                int64_t dv_stride, void *ws, hipStream_t stream);

// ---- the cache and the attention over it ----

hipError_t launch_kv(const gdr_kv &p, bool store, int32_t T, const int32_t *cu, const int32_t *start, uint16_t *k,
                     int64_t k_stride, uint16_t *v, int64_t v_stride, hipStream_t stream);

// A sequence's tokens are shared by `splits` blocks for every kv head and 16 rows of
// its run (`row_tiles` of them are launched; longer runs loop).  A block takes at least
// STEP_UNIT tokens.  Two rounds of blocks (768 run at once) fill the chip, and more of them only add
// starts and parts (256 sequences of 1000, 16 heads on 4: 29 us unsplit, 39 with 4096 blocks, 49 with 8192); where
// a table has room for sequences so long that each of them still gets STEP_LONG tokens, up to STEP_MOST
// blocks even out sequences of different lengths (64 of 1 to 32000, 32 heads on 8: 235 us with 1536, 221 with 4096).
// The table's width is all that the host knows of the lengths: short sequences in a wide one pay for blocks that find
// nothing and for the join (in one for 32768 tokens, 256 of 1000 take 38 us instead of 28, 512 of 300 34 instead of 14).
constexpr int STEP_UNIT = 128, STEP_LONG = 1024;
constexpr int STEP_BLOCKS = 1536, STEP_MOST = 4096;
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
  const int64_t room = (int64_t)max_pages * page, most = (room + STEP_UNIT - 1) / STEP_UNIT;
  const int64_t want = std::max<int64_t>(STEP_BLOCKS / items, std::min<int64_t>(STEP_MOST / items, room / STEP_LONG));
  s.splits = (int)std::max<int64_t>(1, std::min(most, want));
  s.blocks = items * s.splits;
  s.bytes = s.splits > 1 ? ((int64_t)T * H_q * s.splits * 130 * 4 + 255) / 256 * 256 : 0;
  return s;
}
hipError_t launch_attn_step(const gdr_kv &c, const gdr_attn_step &p, uint16_t *o, void *ws, const StepPlan &plan, hipStream_t stream);
hipError_t launch_attn_step_join(const gdr_kv &c, const gdr_attn_step &p, uint16_t *o, void *ws, const StepPlan &plan,
                                 hipStream_t stream);

}  // namespace gdr
