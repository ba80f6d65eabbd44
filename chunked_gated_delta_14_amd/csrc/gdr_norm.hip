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
// registers; rs is formed again in the backward rather than kept.  Bound by HBM.
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

// VEC values of a row from `p`, of which n are there (the rest read as zeros).
template <class T, int VEC>
__device__ __forceinline__ void ld(const T *p, int n, float (&f)[VEC]) {
  Raw<T, VEC> r;
  if (n >= VEC) {
    r.load(p);
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = r.get(e);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      Raw<T, 1> one;
      one.w[0] = 0;
      if (e < n) one.load(p + e);
      f[e] = one.get(0);
    }
  }
}
template <class T, int VEC>
__device__ __forceinline__ void st(T *p, int n, const float (&f)[VEC]) {
  if (n >= VEC) {
    Raw<T, VEC> r;
    r.set(f);
    r.store(p);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < n) {
        Raw<T, 1> one;
        const float v[1] = {f[e]};
        one.set(v);
        one.store(p + e);
      }
  }
}

template <int N, int VEC>
__device__ __forceinline__ void load_weight(const NormArgs &a, int lane, int lpr, float (&w)[N][VEC]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = (i * lpr + lane) * VEC + e;
      w[i][e] = c < a.D ? (a.w ? ld_param(a.w, c, a.wbf) : 1.f) : 0.f;
    }
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
      for (int j = 0; j < WAVES; ++j) s += lds[j * K + k];
      v[k] = s;
    }
  }
}

__device__ __forceinline__ int64_t row_at(int64_t row, int64_t stride, int H, int D) {
  if (stride == (int64_t)H * D) return row * D;
  const int64_t t = row / H;
  return t * stride + (row - t * H) * D;
}

template <class T, class R, int PLACE, int VEC, int LPR, int N>
__global__ __launch_bounds__(LPR > 256 ? LPR : 256) void norm_fwd_kernel(NormArgs a) {
  constexpr int THREADS = LPR > 256 ? LPR : 256, RPB = THREADS / LPR;
  constexpr bool EXACT = sizeof(T) == 4;
  using Y = std::conditional_t<PLACE == GDR_RES_AFTER, R, T>;
  __shared__ float lds[16];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float w[N][VEC];
  load_weight<N, VEC>(a, lane, LPR, w);
  const float inv = 1.f / (float)a.D;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = min(row0 + sub, a.rows - 1);
    const bool mine = row0 + sub < a.rows;
    const T *x = static_cast<const T *>(a.x) + row_at(row, a.xs, a.H, a.D);
    const T *z = a.z ? static_cast<const T *>(a.z) + row_at(row, a.zs, a.H, a.D) : nullptr;
    float u[N][VEC], zz[N][VEC], res[PLACE == GDR_RES_NONE ? 1 : N][VEC];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * LPR + lane) * VEC;
      ld<T, VEC>(x + c, a.D - c, u[i]);
      if (z) ld<T, VEC>(z + c, a.D - c, zz[i]);
      if constexpr (PLACE != GDR_RES_NONE) ld<R, VEC>(static_cast<const R *>(a.res) + row * a.D + c, a.D - c, res[i]);
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (PLACE == GDR_RES_BEFORE) {
        const int c = (i * LPR + lane) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[i][e] = fmaf(a.alpha, u[i][e], res[i][e]);
        if (mine) st<R, VEC>(static_cast<R *>(a.s) + row * a.D + c, a.D - c, u[i]);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) q[0] = fmaf(u[i][e], u[i][e], q[0]);
    }
    row_sum<LPR, 1>(q, lds);
    const float rs = __builtin_amdgcn_rsqf(fmaf(q[0], inv, a.eps));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * LPR + lane) * VEC;
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        y[e] = u[i][e] * rs * w[i][e];
        if (z) {
          const float g = sigmoid<EXACT>(zz[i][e]);
          y[e] *= a.act == GDR_ACT_SILU ? zz[i][e] * g : g;
        }
        if constexpr (PLACE == GDR_RES_AFTER) y[e] = fmaf(a.alpha, y[e], res[i][e]);
      }
      if (mine) st<Y, VEC>(static_cast<Y *>(a.y) + row * a.D + c, a.D - c, y);
    }
  }
}

template <class T, class R, int PLACE, int VEC, int LPR, int N>
__global__ __launch_bounds__(LPR > 256 ? LPR : 256) void norm_bwd_kernel(NormArgs a) {
  constexpr int THREADS = LPR > 256 ? LPR : 256, RPB = THREADS / LPR;
  constexpr bool EXACT = sizeof(T) == 4;
  using U = std::conditional_t<PLACE == GDR_RES_BEFORE, R, T>;  // the normed row as stored
  using Y = std::conditional_t<PLACE == GDR_RES_AFTER, R, T>;
  __shared__ float lds[32];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float w[N][VEC], dw[N][VEC];
  load_weight<N, VEC>(a, lane, LPR, w);
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = 0.f;
  const float inv = 1.f / (float)a.D, ty = PLACE == GDR_RES_AFTER ? a.alpha : 1.f;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = min(row0 + sub, a.rows - 1);
    const bool mine = row0 + sub < a.rows;
    const U *x = PLACE == GDR_RES_BEFORE ? static_cast<const U *>(a.s) + row * a.D
                                         : static_cast<const U *>(a.x) + row_at(row, a.xs, a.H, a.D);
    const T *z = a.z ? static_cast<const T *>(a.z) + row_at(row, a.zs, a.H, a.D) : nullptr;
    float u[N][VEC], t[N][VEC], zz[N][VEC], ds[PLACE == GDR_RES_BEFORE ? N : 1][VEC];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * LPR + lane) * VEC;
      ld<U, VEC>(x + c, a.D - c, u[i]);
      ld<Y, VEC>(static_cast<const Y *>(a.dy) + row * a.D + c, a.D - c, t[i]);
      if (z) ld<T, VEC>(z + c, a.D - c, zz[i]);
      if constexpr (PLACE == GDR_RES_BEFORE) {
        if (a.ds) {
          ld<R, VEC>(static_cast<const R *>(a.ds) + row * a.D + c, a.D - c, ds[i]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) ds[i][e] = 0.f;
        }
      }
    }
    float q[2] = {0.f, 0.f};  // sum u^2, sum v u
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        t[i][e] *= ty;
        q[0] = fmaf(u[i][e], u[i][e], q[0]);
        float v = t[i][e] * w[i][e];
        if (z) {
          const float g = sigmoid<EXACT>(zz[i][e]);
          const bool silu = a.act == GDR_ACT_SILU;
          const float act = silu ? zz[i][e] * g : g;
          // dz without rs, which is not known yet
          zz[i][e] = v * u[i][e] * (silu ? g * fmaf(zz[i][e], 1.f - g, 1.f) : g * (1.f - g));
          v *= act;
          t[i][e] *= act;
        }
        q[1] = fmaf(v, u[i][e], q[1]);
      }
    row_sum<LPR, 2>(q, lds);
    const float rs = __builtin_amdgcn_rsqf(fmaf(q[0], inv, a.eps)), m = q[1] * inv * rs * rs;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * LPR + lane) * VEC;
      float d[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (mine) dw[i][e] = fmaf(t[i][e], u[i][e] * rs, dw[i][e]);
        d[e] = rs * fmaf(t[i][e], w[i][e], -u[i][e] * m);
        if constexpr (PLACE == GDR_RES_BEFORE) d[e] += ds[i][e];
      }
      if (!mine) continue;
      if constexpr (PLACE == GDR_RES_BEFORE) {
        st<R, VEC>(static_cast<R *>(a.dres) + row * a.D + c, a.D - c, d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[e] *= a.alpha;
      }
      if (PLACE != GDR_RES_BEFORE || a.dx) st<T, VEC>(static_cast<T *>(a.dx) + row_at(row, a.dxs, a.H, a.D) + c, a.D - c, d);
      if (z) {
        float dz[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) dz[e] = zz[i][e] * rs;
        st<T, VEC>(static_cast<T *>(a.dz) + row_at(row, a.dzs, a.H, a.D) + c, a.D - c, dz);
      }
    }
  }
  if (!a.partial) return;
  __shared__ float sums[RPB > 1 ? 256 * VEC : 1];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = dw[i][e];
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) sums[threadIdx.x * VEC + e] = s[e];
      __syncthreads();
      if (sub == 0)
        for (int j = 1; j < RPB; ++j)
#pragma unroll
          for (int e = 0; e < VEC; ++e) s[e] += sums[(j * LPR + lane) * VEC + e];
    }
    const int c = (i * LPR + lane) * VEC;
    if (sub == 0) st<float, VEC>(a.partial + (int64_t)blockIdx.x * a.D + c, a.D - c, s);
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

// Threads per row and groups per thread, the smallest that hold a row of D values.
template <class T, class R, int PLACE, int VEC, class F>
hipError_t with_rows(int D, F f) {
#define GDR_ROWS(LPR, N) \
  if (D <= LPR * N * VEC) return f(T(), R(), std::integral_constant<int, PLACE>(), std::integral_constant<int, VEC>(), \
                                   std::integral_constant<int, LPR>(), std::integral_constant<int, N>())
  GDR_ROWS(16, 1);
  GDR_ROWS(32, 1);
  GDR_ROWS(64, 1);
  GDR_ROWS(256, 1);
  GDR_ROWS(256, 2);
  GDR_ROWS(256, 4);
  GDR_ROWS(1024, 2);
  GDR_ROWS(1024, 4);
#undef GDR_ROWS
  return hipErrorInvalidValue;
}
template <class F>
hipError_t with_types(const gdr_norm &p, F f) {
  const bool b = p.dtype == GDR_BF16, rb = p.res_dtype == GDR_BF16;
  switch (p.placement) {
    case GDR_RES_NONE: return b ? with_rows<u16, u16, GDR_RES_NONE, 8>(p.D, f) : with_rows<float, float, GDR_RES_NONE, 4>(p.D, f);
    case GDR_RES_BEFORE:
      return b ? (rb ? with_rows<u16, u16, GDR_RES_BEFORE, 8>(p.D, f) : with_rows<u16, float, GDR_RES_BEFORE, 8>(p.D, f))
               : with_rows<float, float, GDR_RES_BEFORE, 4>(p.D, f);
    default:
      return b ? (rb ? with_rows<u16, u16, GDR_RES_AFTER, 8>(p.D, f) : with_rows<u16, float, GDR_RES_AFTER, 8>(p.D, f))
               : with_rows<float, float, GDR_RES_AFTER, 4>(p.D, f);
  }
}

}  // namespace

hipError_t launch_norm_fwd(const gdr_norm &p, void *y, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  NormArgs a = args_of(p);
  a.y = y;
  return with_types(p, [&](auto t, auto r, auto place, auto vec, auto lpr, auto n) {
    constexpr int LPR = decltype(lpr)::value, threads = LPR > 256 ? LPR : 256, rpb = threads / LPR;
    const int64_t blocks = std::min<int64_t>((a.rows + rpb - 1) / rpb, 8192);
    norm_fwd_kernel<decltype(t), decltype(r), decltype(place)::value, decltype(vec)::value, LPR, decltype(n)::value>
        <<<(unsigned)blocks, threads, 0, stream>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_bwd(const gdr_norm &p, const void *dy, const void *ds, void *dx, int64_t dx_stride, void *dgate,
                           int64_t dgate_stride, void *dres, float *partial, int workers, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  NormArgs a = args_of(p);
  a.dy = dy; a.ds = ds; a.dx = dx; a.dz = dgate; a.dres = dres;
  a.dxs = dx_stride; a.dzs = dgate_stride;
  a.partial = partial;
  return with_types(p, [&](auto t, auto r, auto place, auto vec, auto lpr, auto n) {
    constexpr int LPR = decltype(lpr)::value, threads = LPR > 256 ? LPR : 256;
    norm_bwd_kernel<decltype(t), decltype(r), decltype(place)::value, decltype(vec)::value, LPR, decltype(n)::value>
        <<<workers, threads, 0, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace gdr
