// Attention over packed documents, forward: one pass over the keys with the running
// maximum and sum of a softmax.
//
// A block takes 128 query rows of a head, 32 to each of four wavefronts, whose query
// rows stay in registers as B operands; keys and values come through LDS in tiles of 64, copied
// straight from memory while the tile before is worked on.  The products are formed
// transposed: S^T = K Q^T puts a row's scores into one lane (and its partner 32 lanes on), so the
// softmax needs one lane swap, and S^T's registers are the B operand of
// O^T += V^T P^T as they stand, V^T read from LDS by transposing reads.
// The running maximum is only moved, and the sums rescaled, when a row's grows by more
// than 2^8: until then the probabilities are up to 2^8 instead of 1, which costs neither
// fp32 nor bf16 any precision.  Probabilities go to bf16 for the second product, off by
// up to a relative 2^-8 each as the output is by its own rounding; their sum is taken in fp32 before.  Between different
// scores these errors have either sign; a row of equal ones has the same one throughout, and carries it to its output.
//
// Bound by the matrix units at the clock that their power leaves: 32674 causal rows of 16
// heads on 4 take 4.04 ms, 1.08 PFLOP/s, where a bf16 product of 8192^3 reaches 1.23-1.29 on the same cards;
// matrix units 0.57, vector units 0.49, LDS 0.28 of the cycles busy, at 1.9 GHz.  Two blocks of four wavefronts
// on a unit, at 220 registers, work on each other's waits.  s_setprio around the products changed nothing.
#include "gdr_attn_device.h"

namespace gdr {
namespace {

struct FwdArgs {
  const u16 *q, *k, *v;
  const int32_t *tiles, *items;
  u16 *o;
  float *lse;
  float *part, *ml;  // [slot][H_q][128][128], [slot][H_q][128][2]
  int64_t qs, ks, vs;
  int Hq, group, Tq, causal, window;
  float scale;
};

// Whether a tile holds an infinity or NaN: the largest magnitude's bits, over all its values.
__device__ __forceinline__ bool any_not_finite(uint32_t tile, int lane) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < TILE_BYTES / 1024; ++i) {
    const u32x4 w = *(const __attribute__((address_space(3))) u32x4 *)(tile + i * 1024 + lane * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[j] & 0x7fff7fffu));
  }
  return __any(max(m[0], m[1]) >= 0x7f80);
}

// For a tile with infinities or NaN, some of which not every row sees (0 times one of them would reach
// the rows it is hidden from), V^T P^T is formed in three goes: the finite values, with zeros in the
// others' places; then 2^127 for every +infinity or NaN, and -2^127 for every -infinity or NaN,
// times 2^127 where a row sees the key, which adds an infinity where it does and 0 where it does not.
__device__ __forceinline__ bf16x8 values_of_go(bf16x8 v, int go) {
  u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r = 0;
#pragma unroll
    for (int x = 0; x < 32; x += 16) {
      const uint32_t b = (w[i] >> x) & 0xffffu, mag = b & 0x7fffu;
      if (go == 0) r |= mag < 0x7f80u ? b << x : 0u;
      else if (mag > 0x7f80u || b == (go == 1 ? 0x7f80u : 0xff80u)) r |= (go == 1 ? 0x7f00u : 0xff00u) << x;
    }
    w[i] = r;
  }
  return __builtin_bit_cast(bf16x8, w);
}

__global__ __launch_bounds__(256, 2) void attn_fwd_kernel(FwdArgs a) {
  __shared__ __align__(16) unsigned char lds[4 * TILE_BYTES];  // K, V; twice
  const int lane = threadIdx.x & 63, lr = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Share x(a.items, blockIdx.x, a.Hq);
  const TileEntry e(a.tiles, x.tile);
  const int head = x.head, kvh = head / a.group, steps = e.steps();
  const u16 *kb = a.k + e.other0 * a.ks + kvh * HD, *vb = a.v + e.other0 * a.vs + kvh * HD;
  const int Lk = e.other;

  // the keys that this wavefront's first and last row see last, and this part's share of the tile's keys
  const int rmax = min(32 * wave + 31, e.rows - 1);
  const int p0 = e.first + 32 * wave + e.shift, p1 = e.first + rmax + e.shift;
  const int begin = e.begin + (int)((int64_t)steps * x.part / x.parts) * KT;
  const int end = min(e.end, e.begin + (int)((int64_t)steps * (x.part + 1) / x.parts) * KT);
  const int row = min(32 * wave + lr, e.rows - 1);
  const int p = e.first + row + e.shift;
  const int hi = a.causal ? min(p, Lk - 1) : Lk - 1, lo = a.window ? p - a.window + 1 : 0;  // this lane's row

  f32x16 O[4];
#pragma unroll
  for (int dt = 0; dt < 4; ++dt) O[dt] = zero16();
  const float c = a.scale * LOG2E;
  float m = LEAST, l = 0.f;  // of scores in powers of two

  const uint32_t lds0 = lds_addr(lds);
  uint32_t ko[4], vo[4];
  copy_offsets(ko, wave, lane, KT - 1, (uint32_t)(a.ks * 2));
  copy_offsets(vo, wave, lane, KT - 1, (uint32_t)(a.vs * 2));
  auto copy = [&](int t, int buf) {
    if (t + KT > Lk) {  // the document's last keys
      copy_offsets(ko, wave, lane, Lk - 1 - t, (uint32_t)(a.ks * 2));
      copy_offsets(vo, wave, lane, Lk - 1 - t, (uint32_t)(a.vs * 2));
    }
    const uint32_t to = lds0 + buf * 2 * TILE_BYTES + wave * 4096;
    copy4(kb + t * a.ks, ko, to);
    copy4(vb + t * a.vs, vo, to + TILE_BYTES);
  };
  if (begin < end) copy(begin, 0);
  bf16x8 Q[8];
  {
    const u16 *qp = a.q + (int64_t)(e.row0 + row) * a.qs + head * HD + 8 * h;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) Q[kk] = ld8(qp + 16 * kk);
  }
  settle_loads();
  // A tile's copies are there, and everyone is through with the other buffer, which the next tile's go to.
  auto arrive = [&](int t, int buf) {
    drain_vmem();
    lds_barrier();
    if (t + KT < end) copy(t + KT, buf ^ 1);
  };
  // a wavefront without rows, or none of whose rows sees a key of this tile
  auto idle = [&](int t) { return (a.causal && t > p1) || (a.window && t + KT <= p0 - a.window + 1) || 32 * wave >= e.rows; };
  auto is_masked = [&](int t) { return t + KT > Lk || (a.causal && t + KT - 1 > p0) || (a.window && t <= p1 - a.window); };
  // S^T of a tile, hidden scores at -infinity, and the row's largest over both of its lanes.
  auto scores = [&](f32x16 (&S)[2], int t, int buf) {
    const uint32_t kt = row_base(lds0 + buf * 2 * TILE_BYTES, lane);
    S[0] = zero16(), S[1] = zero16();
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int half = 0; half < 2; ++half) S[half] = mfma32(row_frag(kt, half, kk), Q[kk], S[half]);
    if (is_masked(t)) {
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = t + 32 * half + 8 * (i >> 2) + 4 * h + (i & 3);
          if (j > hi || j < lo) S[half][i] = -INFINITY;
        }
    }
    float top = S[0][0];
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(fmaxf(top, S[0][i]), S[1][i]);
    return fmaxf(top, other_half(top)) * c;
  };
  auto probabilities = [&](f32x16 (&S)[2]) {
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float x = __builtin_amdgcn_exp2f(fmaf(S[half][i], c, -m));
        S[half][i] = x;
        l += x;
      }
  };
  // the loop, until a masked tile holds a value that is not finite
  int t = begin, buf = 0;
  bool careful = false;
  for (; t < end; t += KT, buf ^= 1) {
    arrive(t, buf);
    if (idle(t)) continue;
    const uint32_t v0 = lds0 + (buf * 2 + 1) * TILE_BYTES;
    careful = is_masked(t) && any_not_finite(v0, lane);
    if (careful) break;
    const uint32_t vt = col_base(v0, lane);
    f32x16 S[2];
    const float top = scores(S, t, buf);
    if (__any(top > m + 8.f)) {
      const float to = fmaxf(top, m), f = __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
#pragma unroll
      for (int dt = 0; dt < 4; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[dt][i] *= f;
    }
    probabilities(S);
#pragma unroll
    for (int step = 0; step < 4; ++step) {
      const bf16x8 P = acc_frag(S[step >> 1], step & 1);
#pragma unroll
      for (int dt = 0; dt < 4; ++dt) O[dt] = mfma32(col_frag(vt, step, dt), P, O[dt]);
    }
  }
  if (careful) {  // from there on: the same with care, its sums in memory, so that it takes no registers from the loop above
    f32x16 X[4];
#pragma unroll
    for (int dt = 0; dt < 4; ++dt) X[dt] = O[dt];
    for (bool first = true; t < end; t += KT, buf ^= 1, first = false) {
      if (!first) arrive(t, buf);
      if (idle(t)) continue;
      const uint32_t vt = col_base(lds0 + (buf * 2 + 1) * TILE_BYTES, lane);
      f32x16 S[2];
      const float top = scores(S, t, buf), to = __any(top > m + 8.f) ? fmaxf(top, m) : m, f = __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
      probabilities(S);
      const int goes = is_masked(t) ? 3 : 0;  // 0: every row sees every key
#pragma unroll 1
      for (int go = 0; go < max(goes, 1); ++go) {
        bf16x8 P[4];
#pragma unroll
        for (int step = 0; step < 4; ++step) P[step] = acc_frag(S[step >> 1], step & 1);
#pragma unroll 1
        for (int dt = 0; dt < 4; ++dt) {
          f32x16 x = X[dt];
          if (go == 0) x *= f;
#pragma unroll
          for (int step = 0; step < 4; ++step) {
            const bf16x8 v = col_frag(vt, step, dt);
            x = mfma32(goes ? values_of_go(v, go) : v, P[step], x);
          }
          X[dt] = x;
        }
        const int j0 = afresh(t + 4 * h);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = j0 + 32 * half + 8 * (i >> 2) + (i & 3);
            S[half][i] = j > hi || j < lo ? 0.f : 0x1p127f;
          }
      }
    }
#pragma unroll
    for (int dt = 0; dt < 4; ++dt) O[dt] = X[dt];
  }
  l += other_half(l);
  const bool live = 32 * wave + lr < e.rows;
  if (x.parts == 1) {
    store_row(a.o + ((int64_t)(e.row0 + row) * a.Hq + head) * HD, O, l == 0.f ? 0.f : 1.f / l, h, live);
    if (a.lse && live && h == 0)
      a.lse[(int64_t)head * a.Tq + e.row0 + row] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * LN2;
  } else if (live) {
    const int64_t to = ((int64_t)x.slot * a.Hq + head) * ATT_QTILE + row;
    store_floats(a.part + to * HD, O, h);
    if (h == 0) *reinterpret_cast<float2 *>(a.ml + 2 * to) = make_float2(m, l);
  }
}

// Joins the parts of a tile's rows: a block takes its slot's share of the rows, 16 threads a row, 8 channels each.
__global__ __launch_bounds__(ATT_JOIN) void attn_fwd_join_kernel(FwdArgs a) {
  const Share x(a.items, blockIdx.x, a.Hq);
  if (x.parts == 1) return;
  const TileEntry e(a.tiles, x.tile);
  const int head = x.head, c = (threadIdx.x & 15) * 8, last = e.rows * (x.part + 1) / x.parts;
  const int64_t first = ((int64_t)(x.slot - x.part) * a.Hq + head) * ATT_QTILE, next = (int64_t)a.Hq * ATT_QTILE;  // rows of the parts
  for (int r = e.rows * x.part / x.parts + (threadIdx.x >> 4); r < last; r += ATT_JOIN / 16) {
    const int64_t row = e.row0 + r;
    const float *ml = a.ml + 2 * (first + r);
    float M = LEAST, L = 0.f, y[8] = {};
    for (int i = 0; i < x.parts; ++i) M = fmaxf(M, ml[2 * i * next]);
    for (int i = 0; i < x.parts; ++i) {
      const float f = __builtin_amdgcn_exp2f(ml[2 * i * next] - M);
      L = fmaf(ml[2 * i * next + 1], f, L);
      const f32x4 *src = reinterpret_cast<const f32x4 *>(a.part + (first + r + i * next) * HD + c);
      const f32x4 u = src[0], v = src[1];
#pragma unroll
      for (int z = 0; z < 4; ++z) y[z] = fmaf(u[z], f, y[z]), y[4 + z] = fmaf(v[z], f, y[4 + z]);
    }
    const float f = L == 0.f ? 0.f : 1.f / L;
    *reinterpret_cast<u32x4 *>(a.o + (row * a.Hq + head) * HD + c) =
        u32x4{pk2bf(y[0] * f, y[1] * f), pk2bf(y[2] * f, y[3] * f), pk2bf(y[4] * f, y[5] * f), pk2bf(y[6] * f, y[7] * f)};
    if (a.lse && c == 0) a.lse[(int64_t)head * a.Tq + row] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * LN2;
  }
}

FwdArgs args(const gdr_attn &p, uint16_t *o, float *lse, void *ws) {
  const AttnShare share = ws ? attn_q_share(p) : AttnShare{-1, 1, p.plan.n_q_tiles, 0, 0};
  float *part = static_cast<float *>(ws);
  return FwdArgs{p.q, p.k, p.v, p.tile_table, share.level < 0 ? nullptr : p.tile_table + share.items, o, lse, part,
                 part + share.slots * p.H_q * ATT_QPART, p.q_stride, p.k_stride, p.v_stride, p.H_q, p.H_q / p.H_kv, p.T_q, p.causal,
                 p.window < p.T_k ? p.window : 0, p.scale};
}

}  // namespace

hipError_t launch_attn_fwd(const gdr_attn &p, uint16_t *o, float *lse, void *ws, hipStream_t stream) {
  if (p.plan.n_q_tiles == 0) return hipSuccess;
  const int64_t blocks = ws ? attn_q_share(p).blocks : p.plan.n_q_tiles;
  attn_fwd_kernel<<<dim3((uint32_t)(blocks * p.H_q)), 256, 0, stream>>>(args(p, o, lse, ws));
  return hipGetLastError();
}
hipError_t launch_attn_fwd_join(const gdr_attn &p, uint16_t *o, float *lse, void *ws, hipStream_t stream) {
  if (p.plan.n_q_tiles == 0) return hipSuccess;
  attn_fwd_join_kernel<<<dim3((uint32_t)(attn_q_share(p).slots * p.H_q)), ATT_JOIN, 0, stream>>>(args(p, o, lse, ws));
  return hipGetLastError();
}

}  // namespace gdr
