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
// product's operand as they stand.  P and dS carry a relative 2^-9 from that, of either
// sign, into sums that are rounded by 2^-9 at their end.
#include "gdr_attn_device.h"

namespace gdr {
namespace {

struct BwdArgs {
  const u16 *q, *k, *v, *o, *go;
  const float *lse;
  const int32_t *tiles;
  u16 *dq, *dk, *dv;
  float *lse2, *delta, *pk, *pv;
  int64_t qs, ks, vs, dqs, dks, dvs, partial;  // partial: floats of one part's sums
  int Hq, Hkv, group, Tq, Tk, parts, causal, window;
  float scale;
};

// A row that sees no key gets this in lse's place, which leaves exp2 nothing.
constexpr float NO_KEYS = 3e38f;

__global__ __launch_bounds__(256, 2) void attn_dq_kernel(BwdArgs a) {
  __shared__ __align__(16) unsigned char lds[4 * TILE_BYTES];  // K, V; twice
  const int lane = threadIdx.x & 63, lr = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tile, head;
  tile_of(blockIdx.x, a.Hq, tile, head);
  const TileEntry e(a.tiles, tile);
  const int kvh = head / a.group;
  const u16 *kb = a.k + e.other0 * a.ks + kvh * HD, *vb = a.v + e.other0 * a.vs + kvh * HD;
  const int Lk = e.other;
  const int rmax = min(32 * wave + 31, e.rows - 1);
  const int p0 = e.first + 32 * wave + e.shift, p1 = e.first + rmax + e.shift;
  const int end = a.causal ? min(Lk, e.first + e.rows + e.shift) : Lk;
  const int begin = a.window ? max(0, e.first + e.shift - a.window + 1) & ~(KT - 1) : 0;
  const int row = min(32 * wave + lr, e.rows - 1);
  const bool live = 32 * wave + lr < e.rows;
  const int p = e.first + row + e.shift;
  const int hi = a.causal ? min(p, Lk - 1) : Lk - 1, lo = a.window ? p - a.window + 1 : 0;

  bf16x8 Q[8], G[8];
  float delta = 0.f;
  const int64_t at = ((int64_t)(e.row0 + row) * a.Hq + head) * HD + 8 * h;
  {
    const u16 *qp = a.q + (int64_t)(e.row0 + row) * a.qs + head * HD + 8 * h;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      Q[kk] = ld8(qp + 16 * kk);
      G[kk] = ld8(a.go + at + 16 * kk);
      const bf16x8 o = ld8(a.o + at + 16 * kk);
#pragma unroll
      for (int j = 0; j < 8; ++j) delta = fmaf((float)G[kk][j], (float)o[j], delta);
    }
  }
  delta += other_half(delta);
  const int64_t stat = (int64_t)head * a.Tq + e.row0 + row;
  const float given = a.lse[stat];
  const float lse = given == -INFINITY ? NO_KEYS : given * LOG2E;
  if (live && h == 0) a.lse2[stat] = lse, a.delta[stat] = delta;

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
  drain_vmem();
  if (begin < end) copy(begin, 0);
  int buf = 0;
  for (int t = begin; t < end; t += KT, buf ^= 1) {
    drain_vmem();
    lds_barrier();
    if (t + KT < end) copy(t + KT, buf ^ 1);
    const unsigned char *kt = lds + buf * 2 * TILE_BYTES, *vt = kt + TILE_BYTES;
    if ((a.causal && t > p1) || (a.window && t + KT <= p0 - a.window + 1)) continue;
    const bool masked = t + KT > Lk || (a.causal && t + KT - 1 > p0) || (a.window && t <= p1 - a.window);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      f32x16 S = zero16(), P = zero16();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        S = mfma32(row_frag(kt, half, kk, lr, h), Q[kk], S);
        P = mfma32(row_frag(vt, half, kk, lr, h), G[kk], P);
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
        for (int dt = 0; dt < 4; ++dt) D[dt] = mfma32(col_frag(kt, 2 * half + s, dt, lane), dS, D[dt]);
      }
    }
  }
  store_row(a.dq + (int64_t)(e.row0 + row) * a.dqs + head * HD, D, a.scale, h, live);
}

__global__ __launch_bounds__(256, 2) void attn_dkv_kernel(BwdArgs a) {
  __shared__ __align__(16) unsigned char lds[4 * TILE_BYTES];  // Q, dO; twice
  __shared__ __align__(16) float stats[2][2][KT];              // lse, delta; twice
  const int lane = threadIdx.x & 63, lr = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tile, hp;
  tile_of(blockIdx.x, a.Hkv * a.parts, tile, hp);
  const int kvh = hp / a.parts, part = hp - kvh * a.parts;
  const TileEntry e(a.tiles, tile);
  const int Lq = e.other, per = a.group / a.parts;
  const int head0 = kvh * a.group + part * per;
  const int kmax = min(32 * wave + 31, e.rows - 1);
  const int row = min(32 * wave + lr, e.rows - 1);
  const bool live = 32 * wave + lr < e.rows;
  // the query rows that see key `first + x`: from f0 + x, and below f0 + x + window
  const int f0 = e.first - e.shift;
  const int begin = a.causal ? max(0, f0) & ~(KT - 1) : 0;
  const int end = a.window ? (int)min((int64_t)Lq, (int64_t)f0 + e.rows - 1 + a.window) : Lq;
  const int lo = a.causal ? f0 + row : 0, hi = a.window ? (int)min((int64_t)Lq - 1, (int64_t)f0 + row + a.window - 1) : Lq - 1;

  bf16x8 K[8], V[8];
  {
    const u16 *kp = a.k + (int64_t)(e.row0 + row) * a.ks + kvh * HD + 8 * h;
    const u16 *vp = a.v + (int64_t)(e.row0 + row) * a.vs + kvh * HD + 8 * h;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) K[kk] = ld8(kp + 16 * kk), V[kk] = ld8(vp + 16 * kk);
  }
  f32x16 dK[4], dV[4];
#pragma unroll
  for (int dt = 0; dt < 4; ++dt) dK[dt] = zero16(), dV[dt] = zero16();
  const float c = a.scale * LOG2E;
  const int64_t gs = (int64_t)a.Hq * HD;
  const uint32_t lds0 = lds_addr(lds), stat0 = lds_addr(&stats[0][0][0]);
  uint32_t qo[4], go[4];
  auto copy = [&](int g, int t, int buf) {
    const int last = min(KT, Lq - t) - 1, head = head0 + g;
    copy_offsets(qo, wave, lane, last, (uint32_t)(a.qs * 2));
    copy_offsets(go, wave, lane, last, (uint32_t)(gs * 2));
    const uint32_t to = lds0 + buf * 2 * TILE_BYTES + wave * 4096;
    const int64_t r = e.other0 + t;
    copy4(a.q + r * a.qs + head * HD, qo, to);
    copy4(a.go + r * gs + head * HD, go, to + TILE_BYTES);
    if (wave < 2) lds_dma<4>((wave ? a.delta : a.lse2) + (int64_t)head * a.Tq + r + min(lane, last), stat0 + (buf * 2 + wave) * KT * 4);
  };
  drain_vmem();
  int g = 0, t = begin, buf = 0;
  if (begin < end) copy(0, begin, 0);
  else g = per;
  while (g < per) {
    drain_vmem();
    lds_barrier();
    int g2 = g, t2 = t + KT;
    if (t2 >= end) t2 = begin, ++g2;
    if (g2 < per) copy(g2, t2, buf ^ 1);
    const unsigned char *qt = lds + buf * 2 * TILE_BYTES, *gt = qt + TILE_BYTES;
    const float *ls = stats[buf][0], *dl = stats[buf][1];
    const int x0 = f0 + 32 * wave, x1 = f0 + kmax;  // the first rows that see this wavefront's first and last key
    if (!((a.causal && t + KT - 1 < x0) || (a.window && (int64_t)t > (int64_t)x1 + a.window - 1) || 32 * wave >= e.rows)) {
      const bool masked = t + KT > Lq || (a.causal && t < x1) || (a.window && (int64_t)t + KT > (int64_t)x0 + a.window);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x16 S = zero16(), P = zero16();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) S = mfma32(row_frag(qt, half, kk, lr, h), K[kk], S);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) P = mfma32(row_frag(gt, half, kk, lr, h), V[kk], P);
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const float4 L = *reinterpret_cast<const float4 *>(ls + 32 * half + 8 * i4 + 4 * h);
          const float4 E = *reinterpret_cast<const float4 *>(dl + 32 * half + 8 * i4 + 4 * h);
          const float ll[4] = {L.x, L.y, L.z, L.w}, ee[4] = {E.x, E.y, E.z, E.w};
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int i = 4 * i4 + b;
            S[i] = __builtin_amdgcn_exp2f(fmaf(S[i], c, -ll[b]));
            P[i] = S[i] * (P[i] - ee[b]);
          }
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = t + 32 * half + 8 * (i >> 2) + 4 * h + (i & 3);
            if (r > hi || r < lo) S[i] = 0.f, P[i] = 0.f;
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bf16x8 p = acc_frag(S, s), ds = acc_frag(P, s);
#pragma unroll
          for (int dt = 0; dt < 4; ++dt) dV[dt] = mfma32(col_frag(gt, 2 * half + s, dt, lane), p, dV[dt]);
#pragma unroll
          for (int dt = 0; dt < 4; ++dt) dK[dt] = mfma32(col_frag(qt, 2 * half + s, dt, lane), ds, dK[dt]);
        }
      }
    }
    g = g2, t = t2, buf ^= 1;
  }
  if (a.parts == 1) {
    store_row(a.dk + (int64_t)(e.row0 + row) * a.dks + kvh * HD, dK, a.scale, h, live);
    store_row(a.dv + (int64_t)(e.row0 + row) * a.dvs + kvh * HD, dV, 1.f, h, live);
  } else if (live) {
    const int64_t to = part * a.partial + ((int64_t)(e.row0 + row) * a.Hkv + kvh) * HD + 4 * h;
#pragma unroll
    for (int dt = 0; dt < 4; ++dt)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int64_t x = to + 32 * dt + 2 * i;
        *reinterpret_cast<f32x4 *>(a.pk + x) = f32x4{dK[dt][i], dK[dt][i + 1], dK[dt][i + 2], dK[dt][i + 3]};
        *reinterpret_cast<f32x4 *>(a.pv + x) = f32x4{dV[dt][i], dV[dt][i + 1], dV[dt][i + 2], dV[dt][i + 3]};
      }
  }
}

// The parts' sums, added in order; a thread takes 4 channels of a row of dk or dv.
__global__ __launch_bounds__(256) void attn_join_kernel(BwdArgs a) {
  const int64_t n = (int64_t)a.Tk * a.Hkv * (HD / 4), i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= 2 * n) return;
  const bool v = i >= n;
  const int64_t x = v ? i - n : i;
  const float *src = (v ? a.pv : a.pk) + 4 * x;
  f32x4 s = *reinterpret_cast<const f32x4 *>(src);
  for (int part = 1; part < a.parts; ++part) s += *reinterpret_cast<const f32x4 *>(src + part * a.partial);
  const float f = v ? 1.f : a.scale;
  const int64_t r = x / (a.Hkv * (HD / 4)), y = x - r * (a.Hkv * (HD / 4));
  *reinterpret_cast<uint2 *>((v ? a.dv + r * a.dvs : a.dk + r * a.dks) + 4 * y) = make_uint2(pk2bf(s[0] * f, s[1] * f), pk2bf(s[2] * f, s[3] * f));
}

BwdArgs args(const gdr_attn &p, void *ws) {
  const AttnWorkspace w = attn_workspace(p.T_q, p.T_k, p.n_k_tiles, p.H_q, p.H_kv);
  char *base = static_cast<char *>(ws);
  BwdArgs a{};
  a.q = p.q, a.k = p.k, a.v = p.v;
  a.tiles = p.tile_table;
  a.lse2 = reinterpret_cast<float *>(base);
  a.delta = reinterpret_cast<float *>(base + w.stats);
  a.pk = reinterpret_cast<float *>(base + 2 * w.stats);
  a.pv = reinterpret_cast<float *>(base + 2 * w.stats + w.parts * w.partial);
  a.partial = w.partial / 4;
  a.qs = p.q_stride, a.ks = p.k_stride, a.vs = p.v_stride;
  a.Hq = p.H_q, a.Hkv = p.H_kv, a.group = p.H_q / p.H_kv, a.Tq = p.T_q, a.Tk = p.T_k, a.parts = w.parts;
  a.causal = p.causal, a.window = p.window < p.T_k ? p.window : 0, a.scale = p.scale;
  return a;
}

}  // namespace

hipError_t launch_attn_dq(const gdr_attn &p, const uint16_t *o, const float *lse, const uint16_t *dout, uint16_t *dq,
                          int64_t dq_stride, void *ws, hipStream_t stream) {
  if (p.n_q_tiles == 0) return hipSuccess;
  BwdArgs a = args(p, ws);
  a.o = o, a.lse = lse, a.go = dout, a.dq = dq, a.dqs = dq_stride;
  attn_dq_kernel<<<dim3((uint32_t)((int64_t)p.n_q_tiles * p.H_q)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_attn_dkv(const gdr_attn &p, const uint16_t *dout, uint16_t *dk, int64_t dk_stride, uint16_t *dv,
                           int64_t dv_stride, void *ws, hipStream_t stream) {
  if (p.n_k_tiles == 0) return hipSuccess;
  BwdArgs a = args(p, ws);
  a.tiles += (int64_t)p.n_q_tiles * ATT_ENTRY;
  a.go = dout, a.dk = dk, a.dv = dv, a.dks = dk_stride, a.dvs = dv_stride;
  attn_dkv_kernel<<<dim3((uint32_t)((int64_t)p.n_k_tiles * p.H_kv * a.parts)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_attn_join(const gdr_attn &p, uint16_t *dk, int64_t dk_stride, uint16_t *dv, int64_t dv_stride, void *ws,
                            hipStream_t stream) {
  BwdArgs a = args(p, ws);
  if (a.parts == 1 || p.T_k == 0) return hipSuccess;
  a.dk = dk, a.dv = dv, a.dks = dk_stride, a.dvs = dv_stride;
  const int64_t n = 2 * (int64_t)p.T_k * p.H_kv * (HD / 4);
  attn_join_kernel<<<dim3((uint32_t)((n + 255) / 256)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace gdr
