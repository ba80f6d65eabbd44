// Attention over packed documents, backward, from the forward's log-sum-exp:
//   P = exp(scale Q K^T - lse),  delta_i = dO_i . O_i,  dS = P (dO V^T - delta),
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO.
//
// Two kernels, each with its own rows in registers and the other side's in LDS, form P and dS
// again for themselves: seven products instead of five, but every sum is one block's own
// (or, for few tiles, a fixed sequence of partial sums), so results repeat bit for bit and
// nothing is added in memory.
//   attn_dq:  32 query rows a wavefront, keys and values through LDS; forms delta, and leaves
//             lse and delta of every row as the other kernel takes them.
//   attn_dkv: 32 keys a wavefront, query rows and output gradients of all of the kv head's
//             query heads through LDS.
// Each forms S and dP as 32 x 32 tiles whose registers, rounded to bf16, are the next
// product's operand as they stand.  P and dS carry up to a relative 2^-8 from that, of either
// sign where scores differ, into sums that are rounded by up to 2^-8 at their end.
//
// Bound by the matrix units at the clock that their power leaves: 32674 causal rows of 16 heads on 4 take
// 5.55 ms (attn_dq: three products, 1.18 PFLOP/s, matrix units 0.66 of the cycles busy) and 8.1 ms (attn_dkv:
// four, 1.08 PFLOP/s, 0.60 busy, LDS 0.45, at 1.8 GHz), where a bf16 product of 8192^3 reaches 1.23-1.29.
#include "gdr_attn_device.h"

namespace gdr {
namespace {

struct BwdArgs {
  const u16 *q, *k, *v, *o, *go;
  const float *lse;
  const int32_t *tiles, *items;
  u16 *dq, *dk, *dv;
  float *lse2, *delta, *pq, *pk, *pv;
  int64_t qs, ks, vs, dqs, dks, dvs;
  int Hq, Hkv, group, Tq, Tk, causal, window;
  float scale;
};

// A row that sees no key gets this in lse's place, which leaves exp2 nothing.
constexpr float NO_KEYS = 3e38f;

__global__ __launch_bounds__(256, 2) void attn_dq_kernel(BwdArgs a) {
  __shared__ __align__(16) unsigned char lds[4 * TILE_BYTES];  // K, V; twice
  const int lane = threadIdx.x & 63, lr = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Share x(a.items, blockIdx.x, a.Hq);
  const TileEntry e(a.tiles, x.tile);
  const int head = x.head, kvh = head / a.group, steps = e.steps();
  const u16 *kb = a.k + e.other0 * a.ks + kvh * HD, *vb = a.v + e.other0 * a.vs + kvh * HD;
  const int Lk = e.other;
  const int rmax = min(32 * wave + 31, e.rows - 1);
  const int p0 = e.first + 32 * wave + e.shift, p1 = e.first + rmax + e.shift;
  const int begin = e.begin + (int)((int64_t)steps * x.part / x.parts) * KT;
  const int end = min(e.end, e.begin + (int)((int64_t)steps * (x.part + 1) / x.parts) * KT);
  const int row = min(32 * wave + lr, e.rows - 1);
  const bool live = 32 * wave + lr < e.rows;
  const int p = e.first + row + e.shift;
  const int hi = a.causal ? min(p, Lk - 1) : Lk - 1, lo = a.window ? p - a.window + 1 : 0;

  f32x16 D[4];
#pragma unroll
  for (int dt = 0; dt < 4; ++dt) D[dt] = zero16();
  const float c = a.scale * LOG2E;
  const uint32_t lds0 = lds_addr(lds);
  uint32_t ko[4], vo[4];
  copy_offsets(ko, wave, lane, KT - 1, (uint32_t)(a.ks * 2));
  copy_offsets(vo, wave, lane, KT - 1, (uint32_t)(a.vs * 2));
  auto copy = [&](int t, int buf) {
    if (t + KT > Lk) {
      copy_offsets(ko, wave, lane, Lk - 1 - t, (uint32_t)(a.ks * 2));
      copy_offsets(vo, wave, lane, Lk - 1 - t, (uint32_t)(a.vs * 2));
    }
    const uint32_t to = lds0 + buf * 2 * TILE_BYTES + wave * 4096;
    copy4(kb + t * a.ks, ko, to);
    copy4(vb + t * a.vs, vo, to + TILE_BYTES);
  };
  if (begin < end) copy(begin, 0);
  bf16x8 Q[8], G[8];
  const int64_t at = ((int64_t)(e.row0 + row) * a.Hq + head) * HD + 8 * h;
  // delta is the diagonal of O dO^T by the products that give dP, in their order: where a row sees one key, and o is
  // that key's v, dP - delta is then zero as the formula has it, not the difference of two sums' roundings.
  f32x16 OG = zero16();
  {
    const u16 *qp = a.q + (int64_t)(e.row0 + row) * a.qs + head * HD + 8 * h;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      Q[kk] = ld8(qp + 16 * kk);
      G[kk] = ld8(a.go + at + 16 * kk);
      OG = mfma32(ld8(a.o + at + 16 * kk), G[kk], OG);
    }
  }
  float delta = 0.f;  // row lr of column lr: register 4 (lr >> 3) + (lr & 3) of half (lr >> 2) & 1
#pragma unroll
  for (int i = 0; i < 16; ++i) delta = i == 4 * (lr >> 3) + (lr & 3) ? OG[i] : delta;
  const float other = other_half(delta);
  delta = h == ((lr >> 2) & 1) ? delta : other;
  const int64_t stat = (int64_t)head * a.Tq + e.row0 + row;
  const float given = a.lse[stat];
  const float lse = given == -INFINITY ? NO_KEYS : given * LOG2E;
  if (live && h == 0 && x.part == 0) a.lse2[stat] = lse, a.delta[stat] = delta;
  settle_loads();

  int buf = 0;
  for (int t = begin; t < end; t += KT, buf ^= 1) {
    drain_vmem();
    lds_barrier();
    if (t + KT < end) copy(t + KT, buf ^ 1);
    const uint32_t k0 = lds0 + buf * 2 * TILE_BYTES;
    const uint32_t kt = row_base(k0, lane), vt = row_base(k0 + TILE_BYTES, lane), kc = col_base(k0, lane);
    if ((a.causal && t > p1) || (a.window && t + KT <= p0 - a.window + 1) || 32 * wave >= e.rows) continue;
    const bool masked = t + KT > Lk || (a.causal && t + KT - 1 > p0) || (a.window && t <= p1 - a.window);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      f32x16 S = zero16(), P = zero16();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        S = mfma32(row_frag(kt, half, kk), Q[kk], S);
        P = mfma32(row_frag(vt, half, kk), G[kk], P);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) P[i] = __builtin_amdgcn_exp2f(fmaf(S[i], c, -lse)) * (P[i] - delta);
      if (masked) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = t + 32 * half + 8 * (i >> 2) + 4 * h + (i & 3);
          if (j > hi || j < lo) P[i] = 0.f;
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bf16x8 dS = acc_frag(P, s);
#pragma unroll
        for (int dt = 0; dt < 4; ++dt) D[dt] = mfma32(col_frag(kc, 2 * half + s, dt), dS, D[dt]);
      }
    }
  }
  if (x.parts == 1) store_row(a.dq + (int64_t)(e.row0 + row) * a.dqs + head * HD, D, a.scale, h, live);
  else if (live) store_floats(a.pq + ((int64_t)x.slot * a.Hq + head) * ATT_QPART + row * HD, D, h);
}

// Eight wavefronts, 32 keys each, share the tiles in LDS; the keys' sums take half of a wavefront's
// registers and the keys another eighth, and the values, which there is no room for, stay in LDS.  (Four
// wavefronts with the values in registers too spilled 50 of them, 16.8 ms on [32674, 16/4]; four of 64 keys each, one to a
// SIMD, whose products wait for its own softmax, 10.5 ms.)  S and dP are formed side by side: one after the other 4 % slower.
__global__ __launch_bounds__(512, 2) void attn_dkv_kernel(BwdArgs a) {
  __shared__ __align__(16) unsigned char lds[8 * TILE_BYTES];  // Q, dO; twice; the block's values
  __shared__ __align__(16) float stats[2][2][KT];              // lse, delta; twice
  const int lane = threadIdx.x & 63, lr = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Share x(a.items, blockIdx.x, a.Hkv);
  const TileEntry e(a.tiles, x.tile);
  const int kvh = x.head, Lq = e.other, key0 = 32 * wave;
  // the query rows that see key `first + x`: from f0 + x, and below f0 + x + window
  const int f0 = e.first - e.shift;
  const int begin = e.begin;
  // this part's share of the steps: KT rows of one of the kv head's query heads each
  const int steps = e.steps();
  const int64_t all = (int64_t)steps * a.group;
  int64_t it = all * x.part / x.parts;
  const int64_t last_it = all * (x.part + 1) / x.parts;
  const uint32_t lds0 = lds_addr(lds), stat0 = lds_addr(&stats[0][0][0]);
  const uint32_t v0 = lds0 + (4 + (wave >> 1)) * TILE_BYTES;

  {  // the copies first: what is loaded to registers after them is not waited for apart
    const u16 *vb = a.v + (int64_t)(e.row0 + (key0 & ~63)) * a.vs + kvh * HD;
    const int last = e.rows - 1 - (key0 & ~63);
    if (key0 < e.rows) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int sub = 2 * (wave & 1) + y;
        uint32_t vo[4];
        copy_offsets(vo, sub, lane, last, (uint32_t)(a.vs * 2));
        copy4(vb, vo, v0 + sub * 4096);
      }
    }
  }
  f32x16 dK[4], dV[4];
#pragma unroll
  for (int dt = 0; dt < 4; ++dt) dK[dt] = zero16(), dV[dt] = zero16();
  const float c = a.scale * LOG2E;
  const int64_t gs = (int64_t)a.Hq * HD;
  auto copy = [&](int g, int t, int buf) {  // the first four wavefronts bring Q, the others dO
    uint32_t off[4];
    const int ln = afresh(lane), last = min(KT, Lq - t) - 1, head = kvh * a.group + g, part = wave & 3;
    const bool q = wave < 4;
    const int64_t r = e.other0 + t, stride = q ? a.qs : gs;
    copy_offsets(off, part, ln, last, (uint32_t)(stride * 2));
    copy4((q ? a.q : a.go) + r * stride + head * HD, off, lds0 + (buf * 2 + !q) * TILE_BYTES + part * 4096);
    if (part == 0) lds_dma<4>((q ? a.lse2 : a.delta) + (int64_t)head * a.Tq + r + min(ln, last), stat0 + (buf * 2 + !q) * KT * 4);
  };
  // The rows from the document's last on: causal tiles begin at different rows and end at the same one,
  // so the blocks of an XCD read more of the same rows at a time ([32674, 16/4] 12.7 GB past the L2 instead
  // of 16.2, the time level).
  const int top = begin + (steps - 1) * KT;
  int g = steps ? (int)(it / steps) : 0, t = top - (int)(it - (int64_t)g * steps) * KT, buf = 0;
  if (it < last_it) copy(g, t, 0);
  bf16x8 K[8];
  {
    const int row = min(key0 + lr, e.rows - 1);
    const u16 *kp = a.k + (int64_t)(e.row0 + row) * a.ks + kvh * HD + 8 * h;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) K[kk] = ld8(kp + 16 * kk);
  }
  settle_loads();
  // rows that see this wavefront's first and last key, first ones
  const int x0 = f0 + key0, x1 = f0 + min(key0 + 31, e.rows - 1);
  for (; it < last_it; ++it, buf ^= 1) {
    drain_vmem();
    lds_barrier();
    int g2 = g, t2 = t - KT;
    if (t2 < begin) t2 = top, ++g2;
    if (it + 1 < last_it) copy(g2, t2, buf ^ 1);
    const uint32_t q0 = lds0 + buf * 2 * TILE_BYTES;
    if (!((a.causal && t + KT - 1 < x0) || (a.window && (int64_t)t > (int64_t)x1 + a.window - 1) || key0 >= e.rows)) {
      const bool masked = t + KT > Lq || (a.causal && t < x1) || (a.window && (int64_t)t + KT > (int64_t)x0 + a.window);
      const uint32_t qt = row_base(q0, lane), qc = col_base(q0, lane), vt = row_base(v0, lane) + 8192 * (wave & 1);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x16 S = zero16(), P = zero16();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          S = mfma32(row_frag(qt, half, kk), K[kk], S);
          P = mfma32(row_frag(qt + TILE_BYTES, half, kk), row_frag(vt, 0, kk), P);
        }
        const int hh = afresh(lane >> 5);
        const float *ls = stats[buf][0], *dl = stats[buf][1];
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const float4 L = *reinterpret_cast<const float4 *>(ls + 32 * half + 8 * i4 + 4 * hh);
          const float4 E = *reinterpret_cast<const float4 *>(dl + 32 * half + 8 * i4 + 4 * hh);
          const float ll[4] = {L.x, L.y, L.z, L.w}, ee[4] = {E.x, E.y, E.z, E.w};
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int i = 4 * i4 + b;
            S[i] = __builtin_amdgcn_exp2f(fmaf(S[i], c, -ll[b]));
            P[i] = S[i] * (P[i] - ee[b]);
          }
        }
        if (masked) {
          const int ln = afresh(lane), lr = ln & 31, h = ln >> 5;
          const int y = x0 + lr;  // this lane's key; those past the last are not stored
          const int lo = a.causal ? y : 0, hi = a.window ? (int)min((int64_t)Lq - 1, (int64_t)y + a.window - 1) : Lq - 1;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = t + 32 * half + 8 * (i >> 2) + 4 * h + (i & 3);
            if (r > hi || r < lo) S[i] = 0.f, P[i] = 0.f;
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bf16x8 p = acc_frag(S, s);
#pragma unroll
          for (int dt = 0; dt < 4; ++dt) dV[dt] = mfma32(col_frag(qc + TILE_BYTES, 2 * half + s, dt), p, dV[dt]);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bf16x8 d = acc_frag(P, s);
#pragma unroll
          for (int dt = 0; dt < 4; ++dt) dK[dt] = mfma32(col_frag(qc, 2 * half + s, dt), d, dK[dt]);
        }
      }
    }
    g = g2, t = t2;
  }
  drain_vmem();  // a block without steps has its values' copies still in flight
  const int ln = afresh(lane), lr2 = ln & 31, h2 = ln >> 5, row = min(key0 + lr2, e.rows - 1);
  const bool live = key0 + lr2 < e.rows;
  if (x.parts == 1) {
    store_row(a.dk + (int64_t)(e.row0 + row) * a.dks + kvh * HD, dK, a.scale, h2, live);
    store_row(a.dv + (int64_t)(e.row0 + row) * a.dvs + kvh * HD, dV, 1.f, h2, live);
  } else if (live) {
    const int64_t to = ((int64_t)x.slot * a.Hkv + kvh) * ATT_KPART + row * HD;
    store_floats(a.pk + to, dK, h2);
    store_floats(a.pv + to, dV, h2);
  }
}

// Adds the parts of a tile's rows in order: a block takes its slot's share of the rows, 16 threads a row, 8 channels
// each.  Blocks of both sides: dq of the query tiles (`qblocks` blocks, if they have parts), then the key tiles', which have
// four to a slot and head, dk's and dv's halves of the share.
struct JoinArgs {
  BwdArgs q, k;
  int64_t qblocks;
};
__global__ __launch_bounds__(ATT_JOIN) void attn_bwd_join_kernel(JoinArgs j) {
  const bool keys = blockIdx.x >= j.qblocks;
  const BwdArgs &a = keys ? j.k : j.q;
  const int b = blockIdx.x - (keys ? (int)j.qblocks : 0), heads = keys ? a.Hkv : a.Hq;
  const int pieces = keys ? 2 : 1;
  const Share x(a.items, keys ? b >> 2 : b, heads);
  if (x.parts == 1) return;
  const TileEntry e(a.tiles, x.tile);
  const int piece = x.part * pieces + (keys ? b & 1 : 0), c = (threadIdx.x & 15) * 8;
  const int last = e.rows * (piece + 1) / (x.parts * pieces);
  const bool values = keys && (b & 2);
  const int64_t part = keys ? ATT_KPART : ATT_QPART, next = heads * part;
  const float *src = (keys ? values ? a.pv : a.pk : a.pq) + ((int64_t)(x.slot - x.part) * heads + x.head) * part + c;
  u16 *to = (keys ? values ? a.dv : a.dk : a.dq) + x.head * HD + c;
  const int64_t stride = keys ? values ? a.dvs : a.dks : a.dqs;
  const float f = values ? 1.f : a.scale;
  for (int r = e.rows * piece / (x.parts * pieces) + (threadIdx.x >> 4); r < last; r += ATT_JOIN / 16) {
    f32x4 u = zero4(), v = zero4();
    for (int i = 0; i < x.parts; ++i) {
      const f32x4 *p = reinterpret_cast<const f32x4 *>(src + i * next + r * HD);
      u += p[0], v += p[1];
    }
    *reinterpret_cast<u32x4 *>(to + (int64_t)(e.row0 + r) * stride) =
        u32x4{pk2bf(u[0] * f, u[1] * f), pk2bf(u[2] * f, u[3] * f), pk2bf(v[0] * f, v[1] * f), pk2bf(v[2] * f, v[3] * f)};
  }
}

BwdArgs args(const gdr_attn &p, bool keys, void *ws) {
  const AttnWorkspace w = attn_workspace(p);
  char *base = static_cast<char *>(ws);
  BwdArgs a{};
  a.q = p.q, a.k = p.k, a.v = p.v;
  a.tiles = p.tile_table + (keys ? (int64_t)p.plan.n_q_tiles * ATT_ENTRY : 0);
  a.lse2 = reinterpret_cast<float *>(base);
  a.delta = reinterpret_cast<float *>(base + w.stats);
  a.pq = reinterpret_cast<float *>(base + 2 * w.stats);
  a.pk = a.pq + w.q.slots * p.H_q * ATT_QPART;
  a.pv = a.pk + w.k.slots * p.H_kv * ATT_KPART;
  const AttnShare &share = keys ? w.k : w.q;
  a.items = share.level < 0 ? nullptr : p.tile_table + share.items;
  a.qs = p.q_stride, a.ks = p.k_stride, a.vs = p.v_stride;
  a.Hq = p.H_q, a.Hkv = p.H_kv, a.group = p.H_q / p.H_kv, a.Tq = p.T_q, a.Tk = p.T_k;
  a.causal = p.causal, a.window = p.window < p.T_k ? p.window : 0, a.scale = p.scale;
  return a;
}

}  // namespace

hipError_t launch_attn_dq(const gdr_attn &p, const uint16_t *o, const float *lse, const uint16_t *dout, uint16_t *dq,
                          int64_t dq_stride, void *ws, hipStream_t stream) {
  if (p.plan.n_q_tiles == 0) return hipSuccess;
  BwdArgs a = args(p, false, ws);
  a.o = o, a.lse = lse, a.go = dout, a.dq = dq, a.dqs = dq_stride;
  attn_dq_kernel<<<dim3((uint32_t)(attn_q_share(p).blocks * p.H_q)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_attn_dkv(const gdr_attn &p, const uint16_t *dout, uint16_t *dk, int64_t dk_stride, uint16_t *dv,
                           int64_t dv_stride, void *ws, hipStream_t stream) {
  if (p.plan.n_k_tiles == 0) return hipSuccess;
  BwdArgs a = args(p, true, ws);
  a.go = dout, a.dk = dk, a.dv = dv, a.dks = dk_stride, a.dvs = dv_stride;
  attn_dkv_kernel<<<dim3((uint32_t)(attn_k_share(p).blocks * p.H_kv)), 512, 0, stream>>>(a);
  return hipGetLastError();
}
hipError_t launch_attn_bwd_join(const gdr_attn &p, uint16_t *dq, int64_t dq_stride, uint16_t *dk, int64_t dk_stride, uint16_t *dv,
                                int64_t dv_stride, void *ws, hipStream_t stream) {
  JoinArgs j{args(p, false, ws), args(p, true, ws), 0};
  j.q.dq = dq, j.q.dqs = dq_stride;
  j.k.dk = dk, j.k.dv = dv, j.k.dks = dk_stride, j.k.dvs = dv_stride;
  j.qblocks = attn_q_share(p).slots * p.H_q;
  const int64_t kblocks = attn_k_share(p).slots * p.H_kv * 4;
  if (j.qblocks + kblocks == 0) return hipSuccess;
  attn_bwd_join_kernel<<<dim3((uint32_t)(j.qblocks + kblocks)), ATT_JOIN, 0, stream>>>(j);
  return hipGetLastError();
}

}  // namespace gdr
