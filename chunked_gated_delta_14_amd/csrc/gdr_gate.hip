// The log-decay from its raw projection, and its gradient.
//
//   u = x + b,  A = e^a
//   softplus: g = max(floor, -A softplus(u)),   dg/du = -A sigma(u),            dg/da = g     (0 below the floor)
//   sigmoid:  g = floor sigma(A u),             dg/du = floor A s(1-s),         dg/da = u dg/du
//
// a is one value per head, b one per channel.  softplus(u) = max(u,0) + log(1+e)
// with e = exp(-|u|) in (0,1], and log(1+e) = 2 artanh(v) = 2 (v + v^3/3 + ...)
// with v = e/(2+e) <= 1/3: the odd series keeps its relative accuracy for tiny e,
// where 1 + e would lose it; the first term left out, v^15/15, is at most 1.4e-8 of v,
// below half an fp32 step.
#include "gdr_layer.h"
#include "gdr_vec.h"

namespace gdr {
namespace {

struct GateArgs {
  const void *x;
  const float *a, *b;
  int T, C, D;
  int64_t xs;
  float floor;
  int lx, ly, nchb;
};

__device__ __forceinline__ float log1p01(float e) {  // e in [0, 1]
  const float v = e * __builtin_amdgcn_rcpf(2.f + e), q = v * v;
  float s = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  s = fmaf(s, q, 1.f / 9.f);
  s = fmaf(s, q, 1.f / 7.f);
  s = fmaf(s, q, 1.f / 5.f);
  s = fmaf(s, q, 1.f / 3.f);
  return 2.f * fmaf(v * q, s, v);
}

template <int KIND>
__device__ __forceinline__ float gate_value(float u, float A, float floor) {
  if constexpr (KIND == GDR_GATE_SOFTPLUS) {
    const float e = fast_exp<true>(-__builtin_fabsf(u));
    const float raw = -A * ((u > 0.f ? u : 0.f) + log1p01(e));
    return raw < floor ? floor : u == u ? raw : u;  // a NaN stays one
  } else {
    return floor * sigmoid<true>(A * u);
  }
}
// du = dg/du and da = dg/da at u.
template <int KIND>
__device__ __forceinline__ void gate_slopes(float u, float A, float floor, float &du, float &da) {
  if constexpr (KIND == GDR_GATE_SOFTPLUS) {
    const float e = fast_exp<true>(-__builtin_fabsf(u)), r = __builtin_amdgcn_rcpf(1.f + e);
    const float raw = -A * ((u > 0.f ? u : 0.f) + log1p01(e));
    const bool live = !(raw < floor);
    du = live ? -A * (u >= 0.f ? r : e * r) : 0.f;
    da = live ? raw : 0.f;
    if (u != u) du = da = u;
  } else {
    const float s = sigmoid<true>(A * u), c = sigmoid<true>(-A * u);  // 1 - s keeps its accuracy
    du = floor * A * (s * c);
    da = du * u;
    if (s == 0.f || c == 0.f) da = 0.f;  // the slope vanished: u itself may be infinite
  }
}

template <int VEC>
__device__ __forceinline__ void load_params(const GateArgs &p, int c, float (&A)[VEC], float (&b)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    A[e] = fast_exp<true>(p.a[(c + e) / p.D]);
    b[e] = p.b ? p.b[c + e] : 0.f;
  }
}

constexpr int U = 4;  // rows in flight per thread

template <class T, int VEC, int KIND>
__global__ __launch_bounds__(256) void gate_fwd_kernel(GateArgs p, int workers, float *__restrict__ g) {
  const int tx = threadIdx.x % p.lx, ty = threadIdx.x / p.lx;
  const int chb = blockIdx.x % p.nchb, worker = (blockIdx.x / p.nchb) * p.ly + ty;
  const int group = chb * p.lx + tx;
  if (ty >= p.ly || group >= (p.C + VEC - 1) / VEC) return;
  const int c = VEC == 1 ? group : min(group * VEC, p.C - VEC);
  float A[VEC], b[VEC];
  load_params<VEC>(p, c, A, b);
  const T *__restrict__ x = static_cast<const T *>(p.x) + c;
  g += c;
  for (int64_t t0 = worker; t0 < p.T; t0 += (int64_t)U * workers) {
    Raw<T, VEC> r[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t t = t0 + (int64_t)i * workers;
      r[i].load(x + (t < p.T ? t : t0) * p.xs);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t t = t0 + (int64_t)i * workers;
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = gate_value<KIND>(r[i].get(e) + b[e], A[e], p.floor);
      Raw<float, VEC> o;
      o.set(v);
      if (t < p.T) o.store(g + t * p.C);
    }
  }
}

template <class T, int VEC, int KIND>
__global__ __launch_bounds__(256) void gate_bwd_kernel(GateArgs p, int workers, const float *__restrict__ dg,
                                                       T *__restrict__ dx, int64_t dxs, float *__restrict__ partial) {
  const int tx = threadIdx.x % p.lx, ty = threadIdx.x / p.lx;
  const int chb = blockIdx.x % p.nchb, worker = (blockIdx.x / p.nchb) * p.ly + ty;
  const int group = chb * p.lx + tx;
  const bool live = ty < p.ly && group < (p.C + VEC - 1) / VEC;
  const int c = VEC == 1 ? min(group, p.C - 1) : min(group * VEC, p.C - VEC);
  float A[VEC], b[VEC], sa[VEC], sb[VEC];
  load_params<VEC>(p, c, A, b);
#pragma unroll
  for (int e = 0; e < VEC; ++e) sa[e] = sb[e] = 0.f;
  const T *__restrict__ x = static_cast<const T *>(p.x) + c;
  dg += c;
  dx += c;
  for (int64_t t0 = live ? worker : p.T; t0 < p.T; t0 += (int64_t)U * workers) {
    Raw<T, VEC> r[U];
    Raw<float, VEC> d[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t t = t0 + (int64_t)i * workers, at = t < p.T ? t : t0;
      r[i].load(x + at * p.xs);
      d[i].load(dg + at * p.C);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t t = t0 + (int64_t)i * workers;
      if (t < p.T) {
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float du, da;
          gate_slopes<KIND>(r[i].get(e) + b[e], A[e], p.floor, du, da);
          v[e] = d[i].get(e) * du;
          sb[e] += v[e];
          sa[e] = fmaf(d[i].get(e), da, sa[e]);
        }
        Raw<T, VEC> o;
        o.set(v);
        o.store(dx + t * dxs);
      }
    }
  }
  float *q = partial + (int64_t)(blockIdx.x / p.nchb) * 2 * p.C + c;
  __shared__ float sums[256 * VEC];
  block_partial<VEC>(sb, sums, tx, ty, p.lx, p.ly, live, q);
  block_partial<VEC>(sa, sums, tx, ty, p.lx, p.ly, live, q + p.C);
}

GateArgs args_of(const gdr_gate &p, const Lanes &l) {
  GateArgs a{};
  a.x = p.x; a.a = p.a_log; a.b = p.bias;
  a.T = p.T; a.C = p.H * p.D; a.D = p.D;
  a.xs = p.x_stride;
  a.floor = p.floor;
  a.lx = l.lx; a.ly = l.ly; a.nchb = l.nchb;
  return a;
}

template <class T, int VEC, class F>
hipError_t with_kind(int kind, F f) {
  if (kind == GDR_GATE_SOFTPLUS) return f(T(), std::integral_constant<int, VEC>(), std::integral_constant<int, GDR_GATE_SOFTPLUS>());
  return f(T(), std::integral_constant<int, VEC>(), std::integral_constant<int, GDR_GATE_SIGMOID>());
}
template <class F>
hipError_t with_types(const gdr_gate &p, int vec, F f) {
  if (p.dtype == GDR_BF16) return vec == 1 ? with_kind<u16, 1>(p.kind, f) : with_kind<u16, 8>(p.kind, f);
  return vec == 1 ? with_kind<float, 1>(p.kind, f) : with_kind<float, 4>(p.kind, f);
}

}  // namespace

hipError_t launch_gate_fwd(const gdr_gate &p, float *g, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  const int C = p.H * p.D, vec = vec_of(C, p.dtype);
  const Lanes l = lanes_for(groups_of(C, vec));
  const int workers = workers_for((p.T + U - 1) / U, l, 1 << 21);
  const GateArgs a = args_of(p, l);
  const unsigned blocks = (unsigned)((workers + l.ly - 1) / l.ly * l.nchb);
  return with_types(p, vec, [&](auto t, auto v, auto k) {
    using T = decltype(t);
    gate_fwd_kernel<T, decltype(v)::value, decltype(k)::value><<<blocks, l.threads, 0, stream>>>(a, workers, g);
    return hipGetLastError();
  });
}

hipError_t launch_gate_bwd(const gdr_gate &p, const float *dg, void *dx, int64_t dx_stride, float *partial, int workers,
                           hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  const int C = p.H * p.D, vec = vec_of(C, p.dtype);
  const Lanes l = lanes_for(groups_of(C, vec));
  const GateArgs a = args_of(p, l);
  const unsigned blocks = (unsigned)((workers + l.ly - 1) / l.ly * l.nchb);
  return with_types(p, vec, [&](auto t, auto v, auto k) {
    using T = decltype(t);
    gate_bwd_kernel<T, decltype(v)::value, decltype(k)::value><<<blocks, l.threads, 0, stream>>>(
        a, workers, dg, static_cast<T *>(dx), dx_stride, partial);
    return hipGetLastError();
  });
}

}  // namespace gdr
