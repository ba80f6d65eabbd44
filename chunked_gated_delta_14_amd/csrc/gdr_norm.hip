// RMS norm of rows of D values, before or after a block, with the block's gate and
// the residual stream:
//   n(u) = u rs w act(z),  rs = 1/sqrt(mean u^2 + eps)
//   none:   y = n(x)
//   before: s = res + alpha x,  y = n(s)       (the stream s is stored, y norms the unrounded sum)
//   after:  y = res + alpha n(x)
// Backward, with u the normed row, t = dy (alpha dy for `after`) and v = t act(z) w:
//   dz = t u rs w act'(z),  dw = sum over rows of t act(z) u rs
//   du = rs (v - u rs^2 mean(v u)),  before: du += ds, dres = du, dx = alpha du
// sum u^2 and sum v u come out of one pass, so a row is read once and held in
// registers; rs is formed again in the backward rather than kept.  Bound by HBM: heads
// with a gate, [4182272, 128] bf16, forward 598 us, 5.4 TB/s; residual [32674, 2048]
// with an fp32 stream 144 us forward and 194 us backward, 5.6 TB/s, on a card that
// copies 5.1 TB/s.
#include "gdr_layer.h"
#include "gdr_vec.h"

namespace gdr {
namespace {

struct NormArgs {
  const void *x, *z, *w, *res, *dy, *ds;
  void *y, *s, *dx, *dz, *dres;
  float *partial;
  int64_t rows, xs, zs, dxs, dzs;  // token strides of x, z, dx, dz
  int H, D, act;
  bool wbf;
  float alpha, eps;
};

// Threads of a block whose rows take LPR threads each.
constexpr int row_threads(int lpr) { return lpr <= 128 ? 256 : lpr; }

// A thread's groups of VEC values of a row.  Group i starts at column (i LPR + lane)
// VEC; the last group of a row whose width is no multiple of VEC, and the groups
// past it, start at D - VEC, so that every load is whole, and `skip` counts the
// leading values that belong to a group before (VEC: all of them).
template <int VEC, int LPR>
struct Cols {
  int lane, D;
  __device__ __forceinline__ int nominal(int i) const { return (i * LPR + lane) * VEC; }
  __device__ __forceinline__ int at(int i) const { return min(nominal(i), D - VEC); }
  __device__ __forceinline__ int skip(int i) const { return nominal(i) - at(i); }
  template <class T>
  __device__ __forceinline__ void store(T *row, int i, const float (&f)[VEC]) const {
    const int c = at(i), s = skip(i);
    if (s == 0) {
      Raw<T, VEC> r;
      r.set(f);
      r.store(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e >= s) {
          Raw<T, 1> one;
          const float v[1] = {f[e]};
          one.set(v);
          one.store(row + c + e);
        }
    }
  }
};

template <int N, int VEC, int LPR>
__device__ __forceinline__ void load_weight(const NormArgs &a, const Cols<VEC, LPR> &cols, float (&w)[N][VEC]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[i][e] = a.w ? ld_param(a.w, cols.at(i) + e, a.wbf) : 1.f;
}

// Sum of K values over the LPR threads of a row; every thread of the row gets it.
template <int LPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float *lds) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int d = 1; d < (LPR < 64 ? LPR : 64); d <<= 1) v[k] += __shfl_xor(v[k], d);
  }
  if constexpr (LPR > 64) {
    constexpr int WAVES = LPR / 64;
    const int wave = threadIdx.x >> 6;
    __syncthreads();  // the sums of the row before have been read
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) lds[wave * K + k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < WAVES; ++j) s += lds[((int)threadIdx.x / LPR * WAVES + j) * K + k];
      v[k] = s;
    }
  }
}

__device__ __forceinline__ int64_t row_at(int64_t row, int64_t stride, int H, int D) {
  if (stride == (int64_t)H * D) return row * D;
  const int64_t t = row / H;
  return t * stride + (row - t * H) * D;
}

// The row's values are loaded before any is used, and kept as they lie in memory
// until then: bf16 rows take half the registers.
template <class T, class R, int PLACE, bool GATE, int VEC, int LPR, int N>
__global__ __launch_bounds__(row_threads(LPR)) void norm_fwd_kernel(NormArgs a) {
  constexpr int THREADS = row_threads(LPR), RPB = THREADS / LPR;
  constexpr bool EXACT = sizeof(T) == 4;
  using Y = std::conditional_t<PLACE == GDR_RES_AFTER, R, T>;
  __shared__ float lds[THREADS / 64];
  const Cols<VEC, LPR> cols{(int)threadIdx.x % LPR, a.D};
  const int sub = threadIdx.x / LPR;
  float w[N][VEC];
  load_weight<N>(a, cols, w);
  const float inv = 1.f / (float)a.D;
  struct Row {
    Raw<T, VEC> x[N], z[GATE ? N : 1];
    Raw<R, VEC> res[PLACE == GDR_RES_NONE ? 1 : N];
  };
  auto fetch = [&](int64_t row0, Row &r) {
    const int64_t row = min(row0 + sub, a.rows - 1);
    const T *x = static_cast<const T *>(a.x) + row_at(row, a.xs, a.H, a.D);
    const T *z = GATE ? static_cast<const T *>(a.z) + row_at(row, a.zs, a.H, a.D) : nullptr;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = cols.at(i);
      r.x[i].load(x + c);
      if constexpr (PLACE != GDR_RES_NONE) r.res[i].load(static_cast<const R *>(a.res) + row * a.D + c);
      if constexpr (GATE) r.z[i].load(z + c);
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  constexpr bool AHEAD = LPR > 64;  // the next row is in flight while this one's sums cross the wavefronts
  Row r, ahead;
  if constexpr (AHEAD) fetch((int64_t)blockIdx.x * RPB, ahead);
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + sub;
    const bool mine = row < a.rows;
    if constexpr (AHEAD) {
      r = ahead;
      if (row0 + step < a.rows) fetch(row0 + step, ahead);
    } else {
      fetch(row0, r);
    }
    float q[1] = {0.f};
    float s[PLACE == GDR_RES_BEFORE ? N : 1][VEC];  // the unrounded stream
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int skip = cols.skip(i);
      float u[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        u[e] = r.x[i].get(e);
        if constexpr (PLACE == GDR_RES_BEFORE) s[i][e] = u[e] = fmaf(a.alpha, u[e], r.res[i].get(e));
        q[0] = e >= skip ? fmaf(u[e], u[e], q[0]) : q[0];
      }
      if constexpr (PLACE == GDR_RES_BEFORE) {
        if (mine) cols.store(static_cast<R *>(a.s) + row * a.D, i, u);
      }
    }
    row_sum<LPR, 1>(q, lds);
    const float rs = __builtin_amdgcn_rsqf(fmaf(q[0], inv, a.eps));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float u = 0.f;
        if constexpr (PLACE == GDR_RES_BEFORE) u = s[i][e];
        else u = r.x[i].get(e);
        y[e] = u * rs * w[i][e];
        if constexpr (GATE) {
          const float zz = r.z[i].get(e), g = sigmoid<EXACT>(zz);
          y[e] *= a.act == GDR_ACT_SILU ? zz * g : g;
        }
        if constexpr (PLACE == GDR_RES_AFTER) y[e] = fmaf(a.alpha, y[e], r.res[i].get(e));
      }
      if (mine) cols.store(static_cast<Y *>(a.y) + row * a.D, i, y);
    }
  }
}

// act(z) and act'(z).  sigma' = s (1 - s) takes 1 - s to its own precision, since a gate
// far from zero leaves little of it; SiLU' = s (1 + z (1 - s)) is of order one there.
template <int ACT, bool EXACT>
__device__ __forceinline__ void act_and_slope(float z, float &a, float &d) {
  if constexpr (ACT == GDR_ACT_SILU) {
    const float s = sigmoid<EXACT>(z);
    a = z * s;
    d = s * fmaf(z, 1.f - s, 1.f);
  } else {
    float c;
    sigmoid_both<EXACT>(z, a, c);
    d = a * c;
  }
}

template <class T, class R, int PLACE, int ACT, int VEC, int LPR, int N>
__global__ __launch_bounds__(row_threads(LPR)) void norm_bwd_kernel(NormArgs a) {
  constexpr int THREADS = row_threads(LPR), RPB = THREADS / LPR;
  constexpr bool EXACT = sizeof(T) == 4, GATE = ACT != GDR_ACT_NONE;
  using U = std::conditional_t<PLACE == GDR_RES_BEFORE, R, T>;  // the normed row as stored
  using Y = std::conditional_t<PLACE == GDR_RES_AFTER, R, T>;
  __shared__ float lds[2 * THREADS / 64];
  const Cols<VEC, LPR> cols{(int)threadIdx.x % LPR, a.D};
  const int sub = threadIdx.x / LPR;
  // The weight gradient's terms: in registers, or, for the widest rows, which need
  // those for the row itself, in LDS ([3000, 16000] with gate 187 us, from registers 303).
  constexpr bool LDS_DW = LPR >= 1024;
  __shared__ float dwl[LDS_DW ? THREADS * VEC * N : 1];
  float w[N][VEC], dw[LDS_DW ? 1 : N][VEC];
  load_weight<N>(a, cols, w);
  auto dw_at = [&](int i, int e) -> float & {
    if constexpr (LDS_DW) return dwl[(i * VEC + e) * THREADS + threadIdx.x];
    else return dw[i][e];
  };
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw_at(i, e) = 0.f;
  const float inv = 1.f / (float)a.D, ty = PLACE == GDR_RES_AFTER ? a.alpha : 1.f;
  struct Row {
    Raw<U, VEC> u[N];
    Raw<Y, VEC> t[N];
    Raw<T, VEC> z[GATE ? N : 1];
    Raw<R, VEC> d[PLACE == GDR_RES_BEFORE ? N : 1];
  };
  auto fetch = [&](int64_t row0, Row &r) {
    const int64_t row = min(row0 + sub, a.rows - 1);
    const U *x = PLACE == GDR_RES_BEFORE ? static_cast<const U *>(a.s) + row * a.D
                                         : static_cast<const U *>(a.x) + row_at(row, a.xs, a.H, a.D);
    const T *z = GATE ? static_cast<const T *>(a.z) + row_at(row, a.zs, a.H, a.D) : nullptr;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = cols.at(i);
      r.u[i].load(x + c);
      r.t[i].load(static_cast<const Y *>(a.dy) + row * a.D + c);
      if constexpr (GATE) r.z[i].load(z + c);
      if constexpr (PLACE == GDR_RES_BEFORE) {
        if (a.ds) r.d[i].load(static_cast<const R *>(a.ds) + row * a.D + c);
        else r.d[i].zero();
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  constexpr bool AHEAD = LPR > 64 && LPR < (GATE ? 640 : 1024);  // as in the forward, where registers allow
  Row r, ahead;
  if constexpr (AHEAD) fetch((int64_t)blockIdx.x * RPB, ahead);
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + sub;
    const bool mine = row < a.rows;
    if constexpr (AHEAD) {
      r = ahead;
      if (row0 + step < a.rows) fetch(row0 + step, ahead);
    } else {
      fetch(row0, r);
    }
    // t act(z) and t act'(z), kept where registers allow and formed again otherwise
    constexpr bool KEEP = GATE && N == 1;
    float ta[KEEP ? VEC : 1], tz[KEEP ? VEC : 1];
    float q[2] = {0.f, 0.f};  // sum u^2, sum v u
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int skip = cols.skip(i);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float u = r.u[i].get(e);
        float t = r.t[i].get(e) * ty;
        if constexpr (GATE) {
          float g, dg;
          act_and_slope<ACT, EXACT>(r.z[i].get(e), g, dg);
          if constexpr (KEEP) tz[e] = t * dg;
          t *= g;
          if constexpr (KEEP) ta[e] = t;
        }
        if (e >= skip) q[0] = fmaf(u, u, q[0]), q[1] = fmaf(u, t * w[i][e], q[1]);
      }
    }
    row_sum<LPR, 2>(q, lds);
    const float rs = __builtin_amdgcn_rsqf(fmaf(q[0], inv, a.eps));
    float m = q[1] * inv * rs * rs, k = rs;
    // A row of one value: v - u rs^2 (v u) = v eps rs^2, of which the subtraction would
    // leave only its rounding.
    if constexpr (VEC == 1)
      if (a.D == 1) m = 0.f, k = rs * (a.eps * (rs * rs));
    if (!mine) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float d[VEC], dz[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float u = r.u[i].get(e), n = u * rs;
        float t = r.t[i].get(e) * ty;
        if constexpr (KEEP) {
          dz[e] = tz[e] * w[i][e] * n;
          t = ta[e];
        } else if constexpr (GATE) {
          float g, dg;
          act_and_slope<ACT, EXACT>(r.z[i].get(e), g, dg);
          dz[e] = t * w[i][e] * n * dg;
          t *= g;
        }
        dw_at(i, e) = fmaf(t, n, dw_at(i, e));
        d[e] = k * fmaf(t, w[i][e], -u * m);
        if constexpr (PLACE == GDR_RES_BEFORE) d[e] += r.d[i].get(e);
      }
      if constexpr (PLACE == GDR_RES_BEFORE) {
        cols.store(static_cast<R *>(a.dres) + row * a.D, i, d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[e] *= a.alpha;
      }
      if (PLACE != GDR_RES_BEFORE || a.dx) cols.store(static_cast<T *>(a.dx) + row_at(row, a.dxs, a.H, a.D), i, d);
      if constexpr (GATE) cols.store(static_cast<T *>(a.dz) + row_at(row, a.dzs, a.H, a.D), i, dz);
    }
  }
  if (!a.partial) return;
  __shared__ float sums[RPB > 1 ? THREADS * VEC * N : 1];
  if constexpr (RPB > 1) {
    static_assert(N == 1, "rows shared by a block have one group per thread");
    add_sets<VEC>(dw[0], sums, cols.lane, sub, LPR, RPB);
  }
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[e] = dw_at(i, e);
      cols.store(a.partial + (int64_t)blockIdx.x * a.D, i, s);
    }
  }
}

NormArgs args_of(const gdr_norm &p) {
  NormArgs a{};
  a.x = p.x; a.z = p.gate; a.w = p.weight; a.res = p.residual; a.s = p.s;
  a.rows = (int64_t)p.T * p.H;
  a.xs = p.x_stride; a.zs = p.gate_stride;
  a.H = p.H; a.D = p.D; a.act = p.activation;
  a.wbf = p.w_dtype == GDR_BF16;
  a.alpha = p.scale; a.eps = p.eps;
  return a;
}

// Threads per row and groups per thread, the smallest that hold a row of D values:
// calls f with the kernels' compile-time values.
template <class T, class R, int PLACE, bool GATE, int VEC, int LPR, int N>
struct Shape {
  using Type = T;
  using Res = R;
  static constexpr int place = PLACE, vec = VEC, lpr = LPR, n = N, threads = row_threads(LPR);
  static constexpr bool gate = GATE;
};
template <class T, class R, int PLACE, bool GATE, int VEC, class F>
hipError_t with_rows(int D, F f) {
  if (D < VEC) return f(Shape<T, R, PLACE, GATE, 1, 16, 1>());
#define GDR_ROWS(LPR, N) \
  if (D <= LPR * N * VEC) return f(Shape<T, R, PLACE, GATE, VEC, LPR, N>())
  GDR_ROWS(16, 1);
  GDR_ROWS(32, 1);
  GDR_ROWS(64, 1);
  GDR_ROWS(128, 1);
  GDR_ROWS(192, 1);
  GDR_ROWS(256, 1);
  GDR_ROWS(256, 2);
  GDR_ROWS(384, 2);
  GDR_ROWS(512, 2);
  GDR_ROWS(640, 2);
  GDR_ROWS(768, 2);
  GDR_ROWS(1024, 2);
#undef GDR_ROWS
  if constexpr (VEC == 4) return f(Shape<T, R, PLACE, GATE, 8, 1024, 2>());  // fp32 rows up to 16384
  return hipErrorInvalidValue;
}
template <class T, class R, int PLACE, int VEC, class F>
hipError_t with_gate(const gdr_norm &p, F f) {
  return p.gate ? with_rows<T, R, PLACE, true, VEC>(p.D, f) : with_rows<T, R, PLACE, false, VEC>(p.D, f);
}
template <class F>
hipError_t with_types(const gdr_norm &p, F f) {
  const bool b = p.dtype == GDR_BF16, rb = p.res_dtype == GDR_BF16;
  switch (p.placement) {
    case GDR_RES_NONE: return b ? with_gate<u16, u16, GDR_RES_NONE, 8>(p, f) : with_gate<float, float, GDR_RES_NONE, 4>(p, f);
    case GDR_RES_BEFORE:
      return b ? (rb ? with_gate<u16, u16, GDR_RES_BEFORE, 8>(p, f) : with_gate<u16, float, GDR_RES_BEFORE, 8>(p, f))
               : with_gate<float, float, GDR_RES_BEFORE, 4>(p, f);
    default:
      return b ? (rb ? with_gate<u16, u16, GDR_RES_AFTER, 8>(p, f) : with_gate<u16, float, GDR_RES_AFTER, 8>(p, f))
               : with_gate<float, float, GDR_RES_AFTER, 4>(p, f);
  }
}

}  // namespace

namespace {
// Blocks for `rows` rows of D values, `each` bytes of input to a value: whole rounds
// of the 256 compute units, as few as keep `want` bytes in flight, so that the rows in
// flight lie close together and the weight is read seldom.  Measured on both sides:
//   rows that span wavefronts, whose next row is in flight too, 4 MB: [32674, 2048]
//   backward with an fp32 stream 184 us with one round, 200 with two, 209 with one and
//   a half; [40000, 2048] bf16 147 with two, 165 with four;
//   rows within a wavefront, 10 MB forward and 6 MB backward: heads [4182272, 128]
//   forward 595 us with four or five rounds, 670 with three, 843 with two; backward
//   985 with two, 1083 with four;
//   rows that leave lanes idle or start off a 128-byte line take longer to arrive,
//   9 MB: [40000, 1500] backward 133 us with four or more rounds, 158 with two;
//   [40000, 2049] 360 with two, 473 with one; [400000, 200] 160 with four, 182 with three.
constexpr int64_t AHEAD_BYTES = 4000000, FWD_BYTES = 10000000, BWD_BYTES = 6000000, ODD_BYTES = 9000000;
template <class S>
int64_t blocks_for(int64_t rows, int D, int each, int64_t want) {
  constexpr int rpb = S::threads / S::lpr;
  if (D != S::lpr * S::n * S::vec) want = ODD_BYTES;
  else if (S::lpr > 64) want = AHEAD_BYTES;
  const int64_t round = (int64_t)256 * rpb * D * each;
  return std::min<int64_t>((rows + rpb - 1) / rpb, 256 * std::min<int64_t>((want + round - 1) / round, 8));
}
}  // namespace

hipError_t launch_norm_fwd(const gdr_norm &p, void *y, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  NormArgs a = args_of(p);
  a.y = y;
  return with_types(p, [&](auto s) {
    using S = decltype(s);
    constexpr int each = (S::gate ? 2 : 1) * sizeof(typename S::Type) + (S::place == GDR_RES_NONE ? 0 : sizeof(typename S::Res));
    const int64_t blocks = blocks_for<S>(a.rows, a.D, each, FWD_BYTES);
    norm_fwd_kernel<typename S::Type, typename S::Res, S::place, S::gate, S::vec, S::lpr, S::n>
        <<<(unsigned)blocks, S::threads, 0, stream>>>(a);
    return hipGetLastError();
  });
}

int norm_bwd_workers(const gdr_norm &p) {
  if (p.T == 0) return 0;
  const int64_t rows = (int64_t)p.T * p.H;
  int64_t blocks = 0;
  (void)with_types(p, [&](auto s) {
    using S = decltype(s);
    constexpr int row = S::place == GDR_RES_BEFORE ? 2 * sizeof(typename S::Res) + sizeof(typename S::Type)
                        : S::place == GDR_RES_AFTER ? sizeof(typename S::Type) + sizeof(typename S::Res)
                                                    : 2 * sizeof(typename S::Type);
    constexpr int each = row + (S::gate ? sizeof(typename S::Type) : 0);
    blocks = blocks_for<S>(rows, p.D, each, BWD_BYTES);
    return hipSuccess;
  });
  return (int)std::min<int64_t>(norm_workers(rows, p.D), blocks);
}

// The backward's activation is a compile-time value (the forward's is not: HBM hides it).
template <int ACT>
using Act = std::integral_constant<int, ACT>;

hipError_t launch_norm_bwd(const gdr_norm &p, const void *dy, const void *ds, void *dx, int64_t dx_stride, void *dgate,
                           int64_t dgate_stride, void *dres, float *partial, int workers, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  NormArgs a = args_of(p);
  a.dy = dy; a.ds = ds; a.dx = dx; a.dz = dgate; a.dres = dres;
  a.dxs = dx_stride; a.dzs = dgate_stride;
  a.partial = partial;
  return with_types(p, [&](auto s) {
    using S = decltype(s);
    auto go = [&](auto act) {
      norm_bwd_kernel<typename S::Type, typename S::Res, S::place, decltype(act)::value, S::vec, S::lpr, S::n>
          <<<workers, S::threads, 0, stream>>>(a);
      return hipGetLastError();
    };
    if constexpr (!S::gate) return go(Act<GDR_ACT_NONE>());
    else return p.activation == GDR_ACT_SILU ? go(Act<GDR_ACT_SILU>()) : go(Act<GDR_ACT_SIGMOID>());
  });
}

}  // namespace gdr
