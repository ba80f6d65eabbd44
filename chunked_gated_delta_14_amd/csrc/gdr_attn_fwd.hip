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
// fp32 nor bf16 any precision.  Probabilities go to bf16 for the second product (a
// relative 2^-9 each, of either sign, where the output is rounded by 2^-9 anyway); their sum is taken in fp32 before.
#include "gdr_attn_device.h"

namespace gdr {
namespace {

struct FwdArgs {
  const u16 *q, *k, *v;
  const int32_t *tiles;
  u16 *o;
  float *lse;
  int64_t qs, ks, vs;
  int Hq, group, Tq, causal, window;
  float scale;
};

__global__ __launch_bounds__(256, 2) void attn_fwd_kernel(FwdArgs a) {
  __shared__ __align__(16) unsigned char lds[4 * TILE_BYTES];  // K, V; twice
  const int lane = threadIdx.x & 63, lr = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tile, head;
  tile_of(blockIdx.x, a.Hq, tile, head);
  const TileEntry e(a.tiles, tile);
  const int kvh = head / a.group;
  const u16 *kb = a.k + e.other0 * a.ks + kvh * HD, *vb = a.v + e.other0 * a.vs + kvh * HD;
  const int Lk = e.other;

  // the keys this block's rows see: begin .. end - 1; those of this wavefront's first and last row
  const int rmax = min(32 * wave + 31, e.rows - 1);
  const int p0 = e.first + 32 * wave + e.shift, p1 = e.first + rmax + e.shift;
  const int end = a.causal ? min(Lk, e.first + e.rows + e.shift) : Lk;
  const int begin = a.window ? max(0, e.first + e.shift - a.window + 1) & ~(KT - 1) : 0;
  const int row = min(32 * wave + lr, e.rows - 1);
  const int p = e.first + row + e.shift;
  const int hi = a.causal ? min(p, Lk - 1) : Lk - 1, lo = a.window ? p - a.window + 1 : 0;  // this lane's row

  bf16x8 Q[8];
  {
    const u16 *qp = a.q + (int64_t)(e.row0 + row) * a.qs + head * HD + 8 * h;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) Q[kk] = ld8(qp + 16 * kk);
  }
  f32x16 O[4];
#pragma unroll
  for (int dt = 0; dt < 4; ++dt) O[dt] = zero16();
  const float c = a.scale * LOG2E;
  float m = -1.5e38f, l = 0.f;  // of scores in powers of two; finite, so that hidden scores stay at 0

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
  drain_vmem();  // the query rows are settled before the copies, which the compiler does not count
  if (begin < end) copy(begin, 0);
  int buf = 0;
  for (int t = begin; t < end; t += KT, buf ^= 1) {
    drain_vmem();
    lds_barrier();  // tile t is there, and everyone is through with the other buffer
    if (t + KT < end) copy(t + KT, buf ^ 1);
    const unsigned char *kt = lds + buf * 2 * TILE_BYTES, *vt = kt + TILE_BYTES;
    // a wavefront none of whose rows sees a key of this tile
    if ((a.causal && t > p1) || (a.window && t + KT <= p0 - a.window + 1)) continue;
    f32x16 S[2] = {zero16(), zero16()};
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int half = 0; half < 2; ++half) S[half] = mfma32(row_frag(kt, half, kk, lr, h), Q[kk], S[half]);
    const bool masked = t + KT > Lk || (a.causal && t + KT - 1 > p0) || (a.window && t <= p1 - a.window);
    if (masked) {
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
    top = fmaxf(top, other_half(top)) * c;
    if (__any(top > m + 8.f)) {
      const float to = fmaxf(top, m), f = __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
#pragma unroll
      for (int dt = 0; dt < 4; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[dt][i] *= f;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float x = __builtin_amdgcn_exp2f(fmaf(S[half][i], c, -m));
        S[half][i] = x;
        l += x;
      }
#pragma unroll
    for (int step = 0; step < 4; ++step) {
      const bf16x8 P = acc_frag(S[step >> 1], step & 1);
#pragma unroll
      for (int dt = 0; dt < 4; ++dt) O[dt] = mfma32(col_frag(vt, step, dt, lane), P, O[dt]);
    }
  }
  l += other_half(l);
  const bool live = 32 * wave + lr < e.rows;
  const float f = l == 0.f ? 0.f : 1.f / l;
  store_row(a.o + ((int64_t)(e.row0 + row) * a.Hq + head) * HD, O, f, h, live);
  if (a.lse && live && h == 0)
    a.lse[(int64_t)head * a.Tq + e.row0 + row] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * LN2;
}

}  // namespace

hipError_t launch_attn_fwd(const gdr_attn &p, uint16_t *o, float *lse, hipStream_t stream) {
  if (p.n_q_tiles == 0) return hipSuccess;
  const FwdArgs a{p.q, p.k, p.v, p.tile_table, o, lse, p.q_stride, p.k_stride, p.v_stride, p.H_q, p.H_q / p.H_kv, p.T_q,
                  p.causal, p.window < p.T_k ? p.window : 0, p.scale};
  attn_fwd_kernel<<<dim3((uint32_t)((int64_t)p.n_q_tiles * p.H_q)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace gdr
