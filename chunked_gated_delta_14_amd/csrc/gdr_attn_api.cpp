// C ABI of the softmax-attention layers' operators: argument checks, the tile planner,
// rope frequencies, workspace sizes and launches.  See include/gdr.h for the contract
// of every entry point.
#include "gdr_attn.h"

#include <cmath>
#include <vector>

#include "gdr_check.h"

namespace {

using gdr::aliases;
using gdr::check_workspace;
using gdr::element_aligned;
using gdr::host_status;
using gdr::invalid;
using gdr::launch;
using gdr::stride_ok;
using gdr::unsupported;

// HIP's grids hold fewer than 2^32 threads.
bool grid_ok(int64_t blocks, int threads) { return blocks * threads < (int64_t(1) << 32); }
bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
constexpr int32_t kMostTokens = 1 << 30;

// ---- rotary positions ----

int32_t check_rope(const gdr_rope *p) {
  if (!p) return invalid("problem is NULL");
  if (p->T < 0 || p->N < 0) return invalid("T and N must be >= 0");
  if (p->H_q < 0 || p->H_k < 0) return invalid("H_q and H_k must be >= 0");
  if (p->H_q > 65536 || p->H_k > 65536) return unsupported("H above 65536");
  if (p->D < 2) return invalid("D must be at least 2");
  if (p->D > 1024) return unsupported("D above 1024");
  if (p->rot < 2 || p->rot > p->D || p->rot % 2) return invalid("rot must be even, from 2 to D");
  if (!gdr::is_dtype(p->dtype)) return invalid("unknown dtype");
  if (p->layout != GDR_ROPE_HALF && p->layout != GDR_ROPE_PAIRS) return invalid("unknown layout");
  if (!std::isfinite(p->magnitude)) return invalid("magnitude must be finite");
  if (p->T > 0 && !p->freqs) return invalid("freqs is NULL");
  if (!aligned(p->freqs, 8) || !element_aligned(p->positions, GDR_F32) || !element_aligned(p->chunk_table, GDR_F32))
    return invalid("freqs, positions and chunk_table must be aligned to their elements");
  if (!p->positions) {
    const int64_t least = ((int64_t)p->T + 63) / 64;
    if (p->n_chunks < 0 || p->n_chunks > p->T || p->n_chunks < least || p->n_chunks > least + p->N)
      return invalid("n_chunks is inconsistent with T and N");
    if (p->T > 0 && !p->chunk_table) return invalid("positions or chunk_table must be non-NULL");
  }
  if (!grid_ok(gdr::rope_plan(*p).blocks, 256)) return unsupported("too many rows for one launch");
  return GDR_OK;
}
// One side of a call: H heads from x to y.
int32_t check_rope_side(const gdr_rope *p, int32_t H, const void *x, int64_t xs, const void *y, int64_t ys) {
  if (p->T == 0 || H == 0) return GDR_OK;
  if (!x || !y) return invalid("rows of a side with heads must be non-NULL");
  if (!stride_ok(xs, (int64_t)H * p->D, p->T) || !stride_ok(ys, (int64_t)H * p->D, p->T)) return invalid("a stride is below H * D");
  if (!element_aligned(x, p->dtype) || !element_aligned(y, p->dtype)) return invalid("rows must be aligned to their elements");
  if (x == y && p->T > 1 && xs != ys) return invalid("in place, both strides must be the same");
  return GDR_OK;
}
int32_t rope(const gdr_rope *p, bool back, const void *q, int64_t qs, const void *k, int64_t ks, void *qo, int64_t qos, void *ko,
             int64_t kos, void *stream) {
  int32_t rc = check_rope(p);
  if (rc) return rc;
  if ((rc = check_rope_side(p, p->H_q, q, qs, qo, qos)) || (rc = check_rope_side(p, p->H_k, k, ks, ko, kos))) return rc;
  if (p->H_q && p->H_k && p->T > 0 && (qo == ko || aliases({qo}, {k}) || aliases({ko}, {q})))
    return invalid("an output is the other side's");
  if (aliases({p->H_q ? qo : nullptr, p->H_k ? ko : nullptr}, {p->positions, p->chunk_table, p->freqs}))
    return invalid("an output is an input");
  if ((rc = gdr::host_check_device())) return rc;
  if ((rc = launch(gdr::TK_ROPE, stream, "rope launch",
                   [&](hipStream_t s) { return gdr::launch_rope(*p, back, q, qs, k, ks, qo, qos, ko, kos, s); })))
    return rc;
  return host_status(GDR_OK, "");
}

// ---- attention over packed documents ----

bool tiles_ok(int32_t tiles, int32_t T, int32_t N, int rows) {
  const int64_t least = ((int64_t)T + rows - 1) / rows;
  return tiles >= least && tiles <= T && tiles <= least + N;
}
bool steps_ok(int32_t longest, int64_t steps, int32_t tiles, int32_t T, const int32_t (&items)[GDR_ATTN_LEVELS]) {
  for (int32_t n : items)
    if (n != 0 && (n < tiles || n > (int64_t)tiles * gdr::ATT_PARTS)) return false;
  return longest >= 0 && longest <= (T + 63) / 64 + 1 && steps >= longest && steps <= (int64_t)longest * tiles;
}
// 16-byte aligned rows of [T, H, 128], no wider than the kernels' 32-bit offsets within a tile.
bool rows_ok(const void *p, int64_t stride, int32_t H, int32_t T) {
  return aligned(p, 16) && (T < 2 || (stride >= (int64_t)H * 128 && stride % 8 == 0 && stride < (1 << 24)));
}
const char *const kRows = "rows must be 16-byte aligned, with strides that are multiples of 8, at least H * 128 and below 2^24";

int32_t check_attn(const gdr_attn *p) {
  if (!p) return invalid("problem is NULL");
  if (p->T_q < 0 || p->T_k < 0 || p->N < 0) return invalid("T_q, T_k and N must be >= 0");
  if (p->H_q < 1 || p->H_kv < 1) return invalid("head counts must be positive");
  if (p->H_q % p->H_kv) return unsupported("H_q must be a multiple of H_kv");
  if (p->H_q > 65536) return unsupported("H above 65536");
  if (p->T_q > kMostTokens || p->T_k > kMostTokens) return unsupported("more than 2^30 tokens");
  if (p->D != 128) return unsupported("only D = 128 is implemented");
  if (p->window < 0) return invalid("window must be >= 0");
  if (p->window > 0 && !p->causal) return unsupported("a window needs causal");
  if (!(p->scale > 0.f && p->scale <= 0x1p64f)) return invalid("scale must be positive, at most 2^64");
  const gdr_attn_plan &plan = p->plan;
  if (!tiles_ok(plan.n_q_tiles, p->T_q, p->N, gdr::ATT_QTILE) || !tiles_ok(plan.n_k_tiles, p->T_k, p->N, gdr::ATT_KTILE) ||
      !steps_ok(plan.q_longest, plan.q_steps, plan.n_q_tiles, p->T_k, plan.q_items) ||
      !steps_ok(plan.k_longest, plan.k_steps, plan.n_k_tiles, p->T_q, plan.k_items))
    return invalid("the plan is inconsistent with T_q, T_k and N");
  if (plan.n_q_tiles + (int64_t)plan.n_k_tiles > 0 && !p->tile_table) return invalid("tile_table must be non-NULL");
  if (p->T_q > 0 && !p->q) return invalid("q must be non-NULL");
  if (p->T_k > 0 && (!p->k || !p->v)) return invalid("k and v must be non-NULL");
  if (!element_aligned(p->tile_table, GDR_F32)) return invalid("tile_table must be aligned to its elements");
  if (!rows_ok(p->q, p->q_stride, p->H_q, p->T_q) || !rows_ok(p->k, p->k_stride, p->H_kv, p->T_k) ||
      !rows_ok(p->v, p->v_stride, p->H_kv, p->T_k))
    return invalid(kRows);
  if ((int64_t)p->H_q * 128 >= (1 << 24)) return unsupported("H_q * 128 of 2^24 or more");
  // a launch has a block for every part and head, and a block, or four, for every slot and head to join them
  const gdr::AttnShare q = gdr::attn_q_share(*p), k = gdr::attn_k_share(*p);
  const int64_t q_blocks = std::max(q.blocks, q.slots), k_blocks = std::max(k.blocks, 4 * k.slots);
  if (!grid_ok(q_blocks * p->H_q + k_blocks * p->H_kv, 512)) return unsupported("too many rows and heads for one launch");
  return GDR_OK;
}

int32_t attn_fwd(const gdr_attn *p, uint16_t *o, float *lse, void *ws, int64_t ws_bytes, void *stream) {
  int32_t rc = check_attn(p);
  if (rc) return rc;
  if (p->T_q > 0 && !o) return invalid("o is NULL");
  if (!aligned(o, 16) || !element_aligned(lse, GDR_F32)) return invalid("o must be 16-byte aligned and lse to its elements");
  const gdr::AttnWorkspace w = gdr::attn_workspace(*p);
  if (ws && (rc = check_workspace(ws, ws_bytes, w.fwd))) return rc;
  if (aliases({o, lse}, {p->q, p->k, p->v, p->tile_table})) return invalid("o or lse is an input");
  if (aliases({o}, {lse})) return invalid("o and lse are the same memory");
  if ((rc = gdr::host_check_device())) return rc;
  if ((rc = launch(gdr::TK_ATTN_FWD, stream, "attention launch",
                   [&](hipStream_t s) { return gdr::launch_attn_fwd(*p, o, lse, ws, s); })))
    return rc;
  if (ws && w.q.parts > 1 && (rc = launch(gdr::TK_ATTN_JOIN, stream, "attention join launch", [&](hipStream_t s) {
                                return gdr::launch_attn_fwd_join(*p, o, lse, ws, s);
                              })))
    return rc;
  return host_status(GDR_OK, "");
}

int32_t attn_bwd(const gdr_attn *p, const uint16_t *o, const float *lse, const uint16_t *dout, uint16_t *dq, int64_t dqs,
                 uint16_t *dk, int64_t dks, uint16_t *dv, int64_t dvs, void *ws, int64_t ws_bytes, void *stream) {
  int32_t rc = check_attn(p);
  if (rc) return rc;
  if (p->T_q > 0 && (!o || !lse || !dout || !dq)) return invalid("o, lse, dout and dq must be non-NULL");
  if (p->T_k > 0 && (!dk || !dv)) return invalid("dk and dv must be non-NULL");
  if (!aligned(o, 16) || !aligned(dout, 16) || !element_aligned(lse, GDR_F32))
    return invalid("o and dout must be 16-byte aligned and lse to its elements");
  if (!rows_ok(dq, dqs, p->H_q, p->T_q) || !rows_ok(dk, dks, p->H_kv, p->T_k) || !rows_ok(dv, dvs, p->H_kv, p->T_k))
    return invalid(kRows);
  const gdr::AttnWorkspace w = gdr::attn_workspace(*p);
  if ((rc = check_workspace(ws, ws_bytes, w.bwd))) return rc;
  if (aliases({dq, dk, dv}, {p->q, p->k, p->v, p->tile_table, o, lse, dout})) return invalid("dq, dk or dv is an input");
  if (aliases({dq}, {dk, dv}) || aliases({dk}, {dv})) return invalid("two of dq, dk and dv are the same memory");
  if ((rc = gdr::host_check_device())) return rc;
  if ((rc = launch(gdr::TK_ATTN_DQ, stream, "query gradient launch",
                   [&](hipStream_t s) { return gdr::launch_attn_dq(*p, o, lse, dout, dq, dqs, ws, s); })))
    return rc;
  if ((rc = launch(gdr::TK_ATTN_DKV, stream, "key gradient launch",
                   [&](hipStream_t s) { return gdr::launch_attn_dkv(*p, dout, dk, dks, dv, dvs, ws, s); })))
    return rc;
  if ((w.q.parts > 1 || w.k.parts > 1) && (rc = launch(gdr::TK_ATTN_JOIN, stream, "gradient sum launch", [&](hipStream_t s) {
                                             return gdr::launch_attn_bwd_join(*p, dq, dqs, dk, dks, dv, dvs, ws, s);
                                           })))
    return rc;
  return host_status(GDR_OK, "");
}

// A tile and the tiles of the other side that its rows meet.
struct Tile {
  int32_t entry[gdr::ATT_ENTRY];
  int64_t cost;
};
int32_t plan_attn(const int32_t *cu_q, const int32_t *cu_k, int32_t N, bool causal, int32_t window, int32_t *table,
                  int64_t capacity, gdr_attn_plan *plan) {
  if (N < 0) return invalid("N must be >= 0");
  if (!cu_q) return invalid("cu_q is NULL");
  if (!cu_k) cu_k = cu_q;
  if (window < 0) return invalid("window must be >= 0");
  if (window > 0 && !causal) return unsupported("a window needs causal");
  if (cu_q[0] != 0 || cu_k[0] != 0) return invalid("cu_q[0] and cu_k[0] must be 0");
  if (!plan) return invalid("plan is NULL");
  int64_t n_tiles[2] = {0, 0};
  for (int32_t n = 0; n < N; ++n) {
    const int64_t Lq = (int64_t)cu_q[n + 1] - cu_q[n], Lk = (int64_t)cu_k[n + 1] - cu_k[n];
    if (Lq < 0 || Lk < 0) return invalid("cu_q and cu_k must be non-decreasing");
    n_tiles[0] += (Lq + gdr::ATT_QTILE - 1) / gdr::ATT_QTILE;
    n_tiles[1] += (Lk + gdr::ATT_KTILE - 1) / gdr::ATT_KTILE;
  }
  if (cu_q[N] > kMostTokens || cu_k[N] > kMostTokens) return unsupported("more than 2^30 tokens");
  if (n_tiles[0] + n_tiles[1] > INT32_MAX / gdr::ATT_ENTRY) return unsupported("too many tiles");
  gdr_attn_plan out{};
  out.n_q_tiles = (int32_t)n_tiles[0];
  out.n_k_tiles = (int32_t)n_tiles[1];
  std::vector<Tile> tiles[2];
  int64_t len = (n_tiles[0] + n_tiles[1]) * gdr::ATT_ENTRY;
  for (int side = 0; side < 2; ++side) {
    std::vector<Tile> &list = tiles[side];
    list.reserve((size_t)n_tiles[side]);
    int64_t steps = 0, longest = 0;
    for (int32_t n = 0; n < N; ++n) {
      const int64_t Lq = cu_q[n + 1] - cu_q[n], Lk = cu_k[n + 1] - cu_k[n], shift = Lk - Lq;
      const int64_t mine = side ? Lk : Lq, rows_of_tile = side ? gdr::ATT_KTILE : gdr::ATT_QTILE;
      for (int64_t r = 0; r < mine; r += rows_of_tile) {
        const int64_t rows = std::min(rows_of_tile, mine - r);
        int64_t from = 0, to = side ? Lq : Lk;
        if (causal && side == 0) to = std::min(to, r + rows + shift);
        if (causal && side == 1) from = std::max<int64_t>(0, r - shift);
        if (window && side == 0) from = std::max<int64_t>(0, r + shift - window + 1);
        if (window && side == 1) to = std::min(to, r + rows - 1 - shift + window);
        from = from / 64 * 64;
        if (to < from) from = to = 0;
        Tile t{};
        const int64_t e[gdr::ATT_ENTRY] = {(side ? cu_k[n] : cu_q[n]) + r, rows, side ? cu_q[n] : cu_k[n], side ? Lq : Lk, r, shift, from, to};
        for (int i = 0; i < gdr::ATT_ENTRY; ++i) t.entry[i] = (int32_t)e[i];
        t.cost = (to - from + 63) / 64;
        steps += t.cost;
        longest = std::max(longest, t.cost);
        list.push_back(t);
      }
    }
    std::stable_sort(list.begin(), list.end(), [](const Tile &a, const Tile &b) { return a.cost > b.cost; });
    (side ? out.k_steps : out.q_steps) = steps;
    (side ? out.k_longest : out.q_longest) = (int32_t)longest;
    // lists of parts: those that a launch of one head or more can come to take
    const int slots = side ? gdr::ATT_K_SLOTS : gdr::ATT_Q_SLOTS;
    int32_t(&items)[GDR_ATTN_LEVELS] = side ? out.k_items : out.q_items;
    for (int level = 0; level < GDR_ATTN_LEVELS; ++level) {
      if ((int64_t(1) << level) >= longest || (int64_t(3) << level) < 2 * (steps / slots)) continue;
      int64_t n = 0;
      for (const Tile &t : list) n += gdr::attn_parts(t.cost, level);
      if (n > INT32_MAX / 4) continue;
      items[level] = (int32_t)n;
      len += 2 * n;
    }
  }
  if (len > INT32_MAX) return unsupported("too many tiles");
  out.table_len = len;
  *plan = out;
  if (!table) return host_status(GDR_OK, "");
  if (capacity < len) return invalid("table capacity too small");
  for (const std::vector<Tile> &list : tiles)
    for (const Tile &t : list) table = std::copy(t.entry, t.entry + gdr::ATT_ENTRY, table);
  struct Part {
    int32_t tile, part;
    int64_t cost;
  };
  std::vector<Part> parts;
  for (int side = 0; side < 2; ++side)
    for (int level = 0; level < GDR_ATTN_LEVELS; ++level) {
      if (!(side ? out.k_items : out.q_items)[level]) continue;
      parts.clear();
      for (size_t i = 0; i < tiles[side].size(); ++i) {
        const int n = gdr::attn_parts(tiles[side][i].cost, level);
        for (int x = 0; x < n; ++x) parts.push_back(Part{(int32_t)i, x | n << 16, (tiles[side][i].cost + n - 1) / n});
      }
      // a tile's parts cost the same, so a stable order keeps them in a row
      std::stable_sort(parts.begin(), parts.end(), [](const Part &a, const Part &b) { return a.cost > b.cost; });
      for (const Part &x : parts) *table++ = x.tile, *table++ = x.part;
    }
  return host_status(GDR_OK, "");
}

// ---- the cache in 4 bits ----

int32_t check_kv(const gdr_kv *p) {
  if (!p) return invalid("cache is NULL");
  if (p->n_pages < 0 || p->N < 0 || p->max_pages < 0) return invalid("n_pages, N and max_pages must be >= 0");
  if (p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128 && p->page != 256)
    return unsupported("page must be 16, 32, 64, 128 or 256");
  if (p->H_kv < 1) return invalid("H_kv must be positive");
  if (p->H_kv > 65536) return unsupported("H above 65536");
  if (p->D != 128) return unsupported("only D = 128 is implemented");
  if (p->n_pages > 0 && (!p->k_codes || !p->v_codes || !p->k_scale || !p->v_scale)) return invalid("the pool must be non-NULL");
  if (!aligned(p->k_codes, 16) || !aligned(p->v_codes, 16) || !aligned(p->k_scale, 16) || !aligned(p->v_scale, 16))
    return invalid("the pool must be 16-byte aligned");
  if (p->N > 0 && p->max_pages > 0 && !p->page_table) return invalid("page_table must be non-NULL");
  if (!element_aligned(p->page_table, GDR_F32)) return invalid("page_table must be aligned to its elements");
  return GDR_OK;
}

int32_t kv_move(bool store, const gdr_kv *p, int32_t T, const int32_t *cu, const int32_t *start, const uint16_t *k, int64_t ks,
                const uint16_t *v, int64_t vs, void *stream) {
  int32_t rc = check_kv(p);
  if (rc) return rc;
  if (T < 0) return invalid("T must be >= 0");
  if (!cu && p->N != T) return invalid("N must equal T without cu_seqlens");
  if (T > 0 && (!k || !v)) return invalid("k and v must be non-NULL");
  if (!stride_ok(ks, (int64_t)p->H_kv * 128, T) || !stride_ok(vs, (int64_t)p->H_kv * 128, T))
    return invalid("k_stride or v_stride below H_kv * 128");
  if (!element_aligned(k, GDR_BF16) || !element_aligned(v, GDR_BF16) || !element_aligned(cu, GDR_F32) || !element_aligned(start, GDR_F32))
    return invalid("k, v, cu_seqlens and start must be aligned to their elements");
  if (!grid_ok(((int64_t)T * p->H_kv + 15) / 16, 256)) return unsupported("too many rows for one launch");
  if (aliases({p->k_codes, p->v_codes, p->k_scale, p->v_scale}, {k, v, p->page_table, cu, start}) ||
      (!store && aliases({k, v}, {p->page_table, cu, start})))
    return invalid("an output is an input");
  if (aliases({p->k_codes}, {p->v_codes, p->k_scale, p->v_scale}) || aliases({p->v_codes}, {p->k_scale, p->v_scale}) ||
      aliases({p->k_scale}, {p->v_scale}) || (!store && aliases({k}, {v})))
    return invalid("two of the outputs are the same memory");
  if ((rc = gdr::host_check_device())) return rc;
  if ((rc = launch(store ? gdr::TK_KV_STORE : gdr::TK_KV_LOAD, stream, store ? "store launch" : "load launch", [&](hipStream_t s) {
         return gdr::launch_kv(*p, store, T, cu, start, const_cast<uint16_t *>(k), ks, const_cast<uint16_t *>(v), vs, s);
       })))
    return rc;
  return host_status(GDR_OK, "");
}

int32_t check_step_sizes(int32_t T, int32_t N, int32_t H_q, int32_t H_kv, int32_t max_pages, int32_t page) {
  if (T < 0 || N < 0 || max_pages < 0 || page < 1) return invalid("T, N and max_pages must be >= 0, page positive");
  if (H_q < 1 || H_kv < 1) return invalid("head counts must be positive");
  if (H_q % H_kv) return unsupported("H_q must be a multiple of H_kv");
  if (H_q > 65536) return unsupported("H above 65536");
  if ((int64_t)T * H_q > (int64_t(1) << 36)) return unsupported("more than 2^36 rows and heads");
  // places and rows are 32-bit in the kernel, sums of two of them and a block's share past the last among them
  if (T > kMostTokens || (int64_t)max_pages * page > kMostTokens) return unsupported("more than 2^30 rows, or places of a sequence");
  return GDR_OK;
}
int32_t step(const gdr_kv *c, const gdr_attn_step *p, uint16_t *o, void *ws, int64_t ws_bytes, void *stream) {
  int32_t rc = check_kv(c);
  if (rc) return rc;
  if (!p) return invalid("problem is NULL");
  if ((rc = check_step_sizes(p->T, c->N, p->H_q, c->H_kv, c->max_pages, c->page))) return rc;
  if (p->window < 0) return invalid("window must be >= 0");
  if (!(p->scale > 0.f && p->scale <= 0x1p64f)) return invalid("scale must be positive, at most 2^64");
  if (!p->cu_seqlens && c->N != p->T) return invalid("N must equal T without cu_seqlens");
  if (!stride_ok(p->q_stride, (int64_t)p->H_q * 128, p->T)) return invalid("q_stride below H_q * 128");
  if (p->T > 0 && (!p->q || !o)) return invalid("q and o must be non-NULL");
  if (c->N > 0 && !p->lens) return invalid("lens must be non-NULL");
  if (!element_aligned(p->q, GDR_BF16) || !element_aligned(p->lens, GDR_F32) || !element_aligned(p->cu_seqlens, GDR_F32) || !aligned(o, 16))
    return invalid("q, lens and cu_seqlens must be aligned to their elements, o to 16 bytes");
  const gdr::StepPlan plan = gdr::step_plan(p->T, c->N, p->H_q, c->H_kv, c->max_pages, c->page);
  if (!grid_ok(plan.blocks, 256) || !grid_ok((int64_t)c->N * p->H_q, 256)) return unsupported("too many sequences and heads for one launch");
  if ((rc = check_workspace(ws, ws_bytes, plan.bytes))) return rc;
  if (aliases({o}, {p->q, p->lens, p->cu_seqlens, c->page_table, c->k_codes, c->v_codes, c->k_scale, c->v_scale}))
    return invalid("o is an input");
  if ((rc = gdr::host_check_device())) return rc;
  if ((rc = launch(gdr::TK_ATTN_STEP, stream, "attention step launch",
                   [&](hipStream_t s) { return gdr::launch_attn_step(*c, *p, o, ws, plan, s); })))
    return rc;
  if (plan.splits > 1 && (rc = launch(gdr::TK_ATTN_JOIN, stream, "attention step join launch", [&](hipStream_t s) {
                            return gdr::launch_attn_step_join(*c, *p, o, ws, plan, s);
                          })))
    return rc;
  return host_status(GDR_OK, "");
}

}  // namespace

extern "C" {

int32_t gdr_rope_freqs(int32_t rot, double base, int32_t scaling, double factor, double original, double low, double high,
                       double *freqs) {
  if (rot < 2 || rot % 2 || rot > 1024) return invalid("rot must be even, from 2 to 1024");
  if (!freqs) return invalid("freqs is NULL");
  if (!(base > 0.) || !std::isfinite(base)) return invalid("base must be positive and finite");
  if (scaling < GDR_ROPE_PLAIN || scaling > GDR_ROPE_BLEND) return invalid("unknown scaling");
  if (scaling != GDR_ROPE_PLAIN && (!(factor > 0.) || !std::isfinite(factor))) return invalid("factor must be positive and finite");
  if (scaling == GDR_ROPE_BLEND && !(original > 0. && std::isfinite(original) && low < high && std::isfinite(high - low)))
    return invalid("original must be positive and low below high, all finite");
  if (scaling == GDR_ROPE_BASE && rot > 2) base *= std::pow(factor, (double)rot / (rot - 2));
  for (int32_t i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2. * i / rot) / 6.283185307179586476925286766559;  // turns a token
    if (scaling == GDR_ROPE_LINEAR) f /= factor;
    if (scaling == GDR_ROPE_BLEND) {
      const double r = original * f, c = std::min(std::max((r - low) / (high - low), 0.), 1.);
      f *= (1. - c) / factor + c;
    }
    freqs[i] = f;
  }
  return host_status(GDR_OK, "");
}
int32_t gdr_rope_fwd(const gdr_rope *p, void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream) {
  if (!p) return invalid("problem is NULL");
  return rope(p, false, p->q, p->q_stride, p->k, p->k_stride, q_out, q_out_stride, k_out, k_out_stride, stream);
}
int32_t gdr_rope_bwd(const gdr_rope *p, const void *dq_out, int64_t dq_out_stride, const void *dk_out, int64_t dk_out_stride,
                     void *dq, int64_t dq_stride, void *dk, int64_t dk_stride, void *stream) {
  return rope(p, true, dq_out, dq_out_stride, dk_out, dk_out_stride, dq, dq_stride, dk, dk_stride, stream);
}

int32_t gdr_plan_attn(const int32_t *cu_q, const int32_t *cu_k, int32_t N, int32_t causal, int32_t window, int32_t *table,
                      int64_t capacity, gdr_attn_plan *plan) {
  try {
    return plan_attn(cu_q, cu_k, N, causal != 0, window, table, capacity, plan);
  } catch (...) {
    return unsupported("no host memory for the tiles");
  }
}
int64_t gdr_attn_workspace_bytes(const gdr_attn *p, int32_t backward) {
  const int32_t rc = check_attn(p);
  if (rc) return -(int64_t)rc;
  const gdr::AttnWorkspace w = gdr::attn_workspace(*p);
  return backward ? w.bwd : w.fwd;
}
int32_t gdr_attn_fwd(const gdr_attn *p, uint16_t *o, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
  return attn_fwd(p, o, lse, workspace, workspace_bytes, stream);
}
int32_t gdr_attn_bwd(const gdr_attn *p, const uint16_t *o, const float *lse, const uint16_t *dout, uint16_t *dq,
                     int64_t dq_stride, uint16_t *dk, int64_t dk_stride, uint16_t *dv, int64_t dv_stride, void *workspace,
                     int64_t workspace_bytes, void *stream) {
  return attn_bwd(p, o, lse, dout, dq, dq_stride, dk, dk_stride, dv, dv_stride, workspace, workspace_bytes, stream);
}

int32_t gdr_kv_store(const gdr_kv *p, int32_t T, const int32_t *cu_seqlens, const int32_t *start, const uint16_t *k,
                     int64_t k_stride, const uint16_t *v, int64_t v_stride, void *stream) {
  return kv_move(true, p, T, cu_seqlens, start, k, k_stride, v, v_stride, stream);
}
int32_t gdr_kv_load(const gdr_kv *p, int32_t T, const int32_t *cu_seqlens, const int32_t *start, uint16_t *k, int64_t k_stride,
                    uint16_t *v, int64_t v_stride, void *stream) {
  return kv_move(false, p, T, cu_seqlens, start, k, k_stride, v, v_stride, stream);
}
int64_t gdr_attn_step_workspace_bytes(int32_t T, int32_t N, int32_t H_q, int32_t H_kv, int32_t max_pages, int32_t page) {
  const int32_t rc = check_step_sizes(T, N, H_q, H_kv, max_pages, page);
  return rc ? -(int64_t)rc : gdr::step_plan(T, N, H_q, H_kv, max_pages, page).bytes;
}
int32_t gdr_attn_step_fwd(const gdr_kv *cache, const gdr_attn_step *p, uint16_t *o, void *workspace, int64_t workspace_bytes,
                          void *stream) {
  return step(cache, p, o, workspace, workspace_bytes, stream);
}

}  // extern "C"
