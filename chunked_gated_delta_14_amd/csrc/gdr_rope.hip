// Rotary positions: pair i of a head's first R channels turns by the angle p f_i,
//   (a, b) -> m (a cos - b sin, b cos + a sin),
// the backward by -p f_i.
//
// Bound by the rows' bytes.  All heads of a token share their angles, so a block first
// forms the sines and cosines of its few tokens in LDS and then streams the heads.
// An angle is kept in turns: an fp64 fma takes the whole turns off p f_i before it rounds, and the fraction goes to
// fp32.  So sine and cosine are those of the frequency given, to a few roundings, at any position; that frequency's own
// rounding to fp64 grows with the position (2^-25 turn at p f = 2^28).  A thread of the second part owns up to 16
// bytes of a row's each side of the pairs: 8 (bf16) or 4 (fp32) pairs of half
// layout, half as many neighbouring pairs; what is left of R and of the channels that
// pass goes by single pairs and channels.  [261392, 16 + 4 heads] bf16 492 us, 5.4 TB/s, above what a large
// copy reaches (4.9-5.1); [32674, 8 + 8 heads] fp32 in neighbouring pairs 111 us, 4.8 TB/s; a token of 18 heads 2.9 us.
#include "gdr_attn.h"
#include "gdr_vec.h"

namespace gdr {
namespace {

struct RopeArgs {
  const void *q, *k;
  void *qo, *ko;
  int64_t qs, ks, qos, kos;
  const int32_t *pos, *table;
  const double *freqs;
  int T, N, n_chunks, Hq, Hk, D, R;
  int tokens, hparts;
  int pass;  // whether the channels from R on are copied (not in place)
  float magnitude, sign;
};

// One item of a head's row: `N` pairs at once.
template <class T, bool HALF, int N>
__device__ __forceinline__ void turn_pairs(const T *in, T *out, int i, int half, const float2 *cs) {
  if constexpr (HALF) {
    Raw<T, N> a, b;
    a.load(in + i);
    b.load(in + half + i);
    float x[N], y[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float2 t = cs[i + j];
      const float u = a.get(j), v = b.get(j);
      x[j] = fmaf(u, t.x, -(v * t.y));
      y[j] = fmaf(v, t.x, u * t.y);
    }
    a.set(x);
    b.set(y);
    a.store(out + i);
    b.store(out + half + i);
  } else {
    Raw<T, 2 * N> a;
    a.load(in + 2 * i);
    float x[2 * N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float2 t = cs[i + j];
      const float u = a.get(2 * j), v = a.get(2 * j + 1);
      x[2 * j] = fmaf(u, t.x, -(v * t.y));
      x[2 * j + 1] = fmaf(v, t.x, u * t.y);
    }
    a.set(x);
    a.store(out + 2 * i);
  }
}

template <class T, bool HALF>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  extern __shared__ float2 cs[];  // [tokens][R / 2] cosine and sine, times the magnitude
  constexpr int V = 16 / (int)sizeof(T);        // channels of a 16-byte piece
  constexpr int P = HALF ? V : V / 2;           // pairs of a whole item
  const int half = a.R / 2;
  const int part = blockIdx.x % a.hparts;
  const int64_t b = blockIdx.x / a.hparts;
  int64_t t0;
  int n;
  int first = 0;  // position of the block's first token, without positions
  if (a.pos) {
    t0 = b * a.tokens;
    n = (int)min((int64_t)a.tokens, a.T - t0);
  } else {
    const int per = 64 / a.tokens, c = (int)(b / per), i0 = (int)(b - (int64_t)c * per) * a.tokens;
    const ChunkTable table(a.table, a.n_chunks, a.N);
    n = min(a.tokens, table.len[c] - i0);
    t0 = table.start[c] + i0;
    first = (c - table.doc_ptr[table.doc[c]]) * CH + i0;
  }
  if (n <= 0) return;
  for (int e = threadIdx.x; e < n * half; e += 256) {
    const int t = e / half, i = e - t * half;
    const double p = (double)(a.pos ? a.pos[t0 + t] : first + t), f = a.freqs[i];
    float s, c;
    sincospif((float)(2.0 * fma(p, f, -rint(p * f))), &s, &c);
    cs[e] = make_float2(c * a.magnitude, s * a.magnitude * a.sign);
  }
  __syncthreads();
  const int H = a.Hq + a.Hk;
  const int h0 = (int)((int64_t)H * part / a.hparts), hn = (int)((int64_t)H * (part + 1) / a.hparts) - h0;
  const int whole = half / P, rest = half - whole * P;
  const int more = a.pass ? a.D - a.R : 0, pw = more / V, items = whole + rest + pw + more - pw * V;
  // item x of row y, rows ly apart: LX threads span the items, or 256 of them in turn
  const int lx = min(items, 256), ly = 256 / lx;
  const int tx = threadIdx.x % lx, ty = threadIdx.x / lx;
  if (ty >= ly) return;
  const int dt = ly / hn, dh = ly - dt * hn;
  int t = ty / hn, h = ty - t * hn;
  while (t < n) {
    const int hh = h0 + h;
    const bool is_q = hh < a.Hq;
    const int64_t row = t0 + t;
    const int64_t at = is_q ? row * a.qs + hh * a.D : row * a.ks + (hh - a.Hq) * a.D;
    const int64_t to = is_q ? row * a.qos + hh * a.D : row * a.kos + (hh - a.Hq) * a.D;
    const T *in = static_cast<const T *>(is_q ? a.q : a.k) + at;
    T *out = static_cast<T *>(is_q ? a.qo : a.ko) + to;
    const float2 *c = cs + t * half;
    for (int x = tx; x < items; x += lx) {
      if (x < whole) {
        turn_pairs<T, HALF, P>(in, out, x * P, half, c);
      } else if (x < whole + rest) {
        turn_pairs<T, HALF, 1>(in, out, whole * P + x - whole, half, c);
      } else if (x < whole + rest + pw) {
        Raw<T, V> r;
        const int i = a.R + (x - whole - rest) * V;
        r.load(in + i);
        r.store(out + i);
      } else {
        const int i = a.R + pw * V + x - whole - rest - pw;
        out[i] = in[i];
      }
    }
    t += dt;
    h += dh;
    if (h >= hn) h -= hn, ++t;
  }
}

template <class T, bool HALF>
hipError_t go(const RopeArgs &a, int64_t blocks, hipStream_t stream) {
  rope_kernel<T, HALF><<<dim3((uint32_t)blocks), 256, (size_t)a.tokens * (a.R / 2) * sizeof(float2), stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const gdr_rope &p, bool back, const void *q, int64_t q_stride, const void *k, int64_t k_stride, void *qo,
                       int64_t qo_stride, void *ko, int64_t ko_stride, hipStream_t stream) {
  if (p.T == 0 || p.H_q + p.H_k == 0) return hipSuccess;
  const RopePlan plan = rope_plan(p);
  if (plan.blocks == 0) return hipSuccess;
  RopeArgs a{q, k, qo, ko, q_stride, k_stride, qo_stride, ko_stride, p.positions, p.chunk_table, p.freqs,
             p.T, p.N, p.n_chunks, p.H_q, p.H_k, p.D, p.rot, plan.tokens, plan.hparts,
             (q != qo && p.H_q) || (k != ko && p.H_k), p.magnitude, back ? -1.f : 1.f};
  const bool half = p.layout == GDR_ROPE_HALF;
  if (p.dtype == GDR_BF16) return half ? go<u16, true>(a, plan.blocks, stream) : go<u16, false>(a, plan.blocks, stream);
  return half ? go<float, true>(a, plan.blocks, stream) : go<float, false>(a, plan.blocks, stream);
}

}  // namespace gdr
