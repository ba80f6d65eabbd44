// The log-decay from its raw projection, and its gradient.
//
//   u = x + b,  A = e^a
//   softplus: g = max(floor, -A softplus(u)),   dg/du = -A sigma(u),            dg/da = g     (0 below the floor)
//   sigmoid:  g = floor sigma(A u),             dg/du = floor A s(1-s),         dg/da = u dg/du
//
// a is one value per head, b one per channel.  softplus(u) = max(u,0) + log(1+e)
// with e = exp(-|u|) in (0,1], and log(1+e) = 2 artanh(v) with v = e/(2+e) <= 1/3:
// an odd function of v keeps its relative accuracy for tiny e, where 1 + e would
// lose it.  Bound by HBM; the arithmetic, about 30 lane operations per value, is up
// to 0.9 of what the vector units do in that time, so it is kept short.  On a card that
// copies 5.1 TB/s: forward [261392, 2048] from bf16 580 us, 5.5 TB/s; backward [32674,
// 2048] 103 us with its sums, 5.2 TB/s.
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

// log(1+e) / 2 for e in [0, 1]: artanh(v) = v + v^3 p(v^2), p fitted to degree 3 for
// v^2 in [0, 1/9] with a relative error of 5e-9, a twelfth of fp32's half step.
__device__ __forceinline__ float half_log1p(float e) {
  const float v = e * __builtin_amdgcn_rcpf(2.f + e), q = v * v;
  float p = fmaf(q, 0.140122339f, 0.139995694f);
  p = fmaf(p, q, 0.200108498f);
  p = fmaf(p, q, 0.333332062f);
  return fmaf(v * q, p, v);
}
// e^-|x|, the argument cut at 104 (the result is below fp32's smallest value
// there), which keeps infinities out of the correction; a NaN passes.
__device__ __forceinline__ float exp_neg_abs(float x) {
  float a = __builtin_fabsf(x);
  a = a > 104.f ? 104.f : a;
  const float t = a * -1.44269504088896341f, e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, fmaf(a, -1.44269504088896341f, -t) * 0.693147180559945309f, e);
}
// -A softplus(u) from e = exp(-|u|).
__device__ __forceinline__ float softplus_raw(float u, float e, float A) {
  return fmaf(-2.f * A, half_log1p(e), -A * fmaxf(u, 0.f));
}

template <int KIND>
__device__ __forceinline__ float gate_value(float u, float A, float floor) {
  if constexpr (KIND == GDR_GATE_SOFTPLUS) {
    const float raw = softplus_raw(u, exp_neg_abs(u), A);
    return raw < floor ? floor : raw;  // a NaN stays one
  } else {
    const float w = A * u, e = exp_neg_abs(w), r = floor * __builtin_amdgcn_rcpf(1.f + e);
    return w < 0.f ? e * r : r;
  }
}
// du = dg/du and da = dg/da at u.
template <int KIND>
__device__ __forceinline__ void gate_slopes(float u, float A, float floor, float &du, float &da) {
  if constexpr (KIND == GDR_GATE_SOFTPLUS) {
    const float e = exp_neg_abs(u), r = -A * __builtin_amdgcn_rcpf(1.f + e);
    const float raw = softplus_raw(u, e, A);
    const bool held = raw < floor;
    du = held ? 0.f : u < 0.f ? e * r : r;
    da = held ? 0.f : raw;
  } else {
    const float e = exp_neg_abs(A * u), r = __builtin_amdgcn_rcpf(1.f + e);
    // s (1 - s) = e / (1 + e)^2 on either side; floor A, like A, stays finite beside a zero
    du = fmaxf(floor * A, -0x1.fffffep126f) * (e * r * r);
    da = du == 0.f ? 0.f : du * u;      // the slope vanished: u itself may be infinite
  }
}

// A = e^a, cut at half of fp32's largest value: an infinite A times a softplus of zero, or
// times u = 0, would be NaN where g is the floor, or half of it.  A NaN passes.
__device__ __forceinline__ float rate(float a) {
  const float A = fast_exp<true>(a);
  return A > 0x1.fffffep126f ? 0x1.fffffep126f : A;
}

template <int VEC>
__device__ __forceinline__ void load_params(const GateArgs &p, int c, float (&A)[VEC], float (&b)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    A[e] = rate(p.a[p.D == 1 ? c + e : (c + e) >> 7]);
    b[e] = p.b ? p.b[c + e] : 0.f;
  }
}

constexpr int U = 4;  // rows in flight per thread

// First row of a thread set: a block takes U x LY neighbouring rows at a time, its
// sets' rows side by side, and the blocks follow one another, so that what is in
// flight lies close together.  ([261392, 2048], softplus: forward 580 us and backward
// 794; with a set's U rows a whole round of workers apart 621 and 887.)
__device__ __forceinline__ int64_t first_row(const GateArgs &p, int ty) {
  return (int64_t)(blockIdx.x / p.nchb) * U * p.ly + ty;
}

template <class T, int VEC, int KIND, bool UNI>
__global__ __launch_bounds__(256) void gate_fwd_kernel(GateArgs p, int workers, float *__restrict__ g) {
  const int tx = threadIdx.x % p.lx, ty = set_of<UNI>(p.lx);
  const int chb = blockIdx.x % p.nchb;
  const int group = chb * p.lx + tx;
  if (ty >= p.ly || group >= (p.C + VEC - 1) / VEC) return;
  const int c = first_channel<VEC>(group, p.C);
  float A[VEC], b[VEC];
  load_params<VEC>(p, c, A, b);
  const int64_t first = first_row(p, ty), step = (int64_t)U * workers;
  const T *__restrict__ x = static_cast<const T *>(p.x) + first * p.xs;
  float *__restrict__ out = g + first * p.C;
  const int64_t xstep = p.ly * p.xs, gstep = (int64_t)p.ly * p.C;
  for (int64_t t = first; t < p.T; t += step) {
    Raw<T, VEC> r[U];
#pragma unroll
    for (int i = 0; i < U; ++i) r[i].load((t + i * p.ly < p.T ? x + i * xstep : x) + c);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = gate_value<KIND>(r[i].get(e) + b[e], A[e], p.floor);
      Raw<float, VEC> o;
      o.set(v);
      if (t + i * p.ly < p.T) o.store(out + i * gstep + c);
    }
    x += step * p.xs;
    out += step * p.C;
  }
}

// A block leaves one partial row: the C sums of dg du, then the sums of dg da, per
// channel (D = 1) or per thread's VEC channels of one head (D = 128).
template <class T, int VEC, int KIND, bool UNI>
__global__ __launch_bounds__(256) void gate_bwd_kernel(GateArgs p, int workers, const float *__restrict__ dg,
                                                       T *__restrict__ dx, int64_t dxs, float *__restrict__ partial) {
  const int tx = threadIdx.x % p.lx, ty = set_of<UNI>(p.lx);
  const int chb = blockIdx.x % p.nchb;
  const int group = chb * p.lx + tx, groups = (p.C + VEC - 1) / VEC;
  const bool live = ty < p.ly && group < groups;
  const int c = first_channel<VEC>(min(group, groups - 1), p.C);
  float A[VEC], b[VEC], sa[VEC], sb[VEC];
  load_params<VEC>(p, c, A, b);
#pragma unroll
  for (int e = 0; e < VEC; ++e) sa[e] = sb[e] = 0.f;
  const int64_t first = first_row(p, ty), step = (int64_t)U * workers;
  const T *__restrict__ x = static_cast<const T *>(p.x) + first * p.xs;
  const float *__restrict__ d = dg + first * p.C;
  T *__restrict__ out = dx + first * dxs;
  const int64_t xstep = p.ly * p.xs, gstep = (int64_t)p.ly * p.C, ostep = p.ly * dxs;
  for (int64_t t = live ? first : p.T; t < p.T; t += step) {
    Raw<T, VEC> r[U];
    Raw<float, VEC> q[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool there = t + i * p.ly < p.T;
      r[i].load((there ? x + i * xstep : x) + c);
      q[i].load((there ? d + i * gstep : d) + c);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (t + i * p.ly < p.T) {
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float du, da;
          gate_slopes<KIND>(r[i].get(e) + b[e], A[e], p.floor, du, da);
          v[e] = q[i].get(e) * du;
          sb[e] += v[e];
          sa[e] = fmaf(q[i].get(e), da, sa[e]);
        }
        Raw<T, VEC> o;
        o.set(v);
        o.store(out + i * ostep + c);
      }
    }
    x += step * p.xs;
    d += step * p.C;
    out += step * dxs;
  }
  __shared__ float lds[2 * VEC * 256];
  float v[2 * VEC], s = 0.f;
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = sb[e], v[VEC + e] = sa[e], s += sa[e];
  if (p.D != 1) v[VEC] = s;  // one term per thread
  add_sets<2 * VEC>(v, lds, tx, ty, p.lx, p.ly);
  if (!live || ty != 0) return;
  float *q = partial + (int64_t)(blockIdx.x / p.nchb) * gate_partial_row(p.C, p.D, VEC);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    q[c + e] = v[e];
    if (p.D == 1) q[p.C + c + e] = v[VEC + e];
  }
  if (p.D != 1) q[p.C + c / VEC] = v[VEC];
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

// Calls f(type tag, VEC, KIND, UNI) with the compile-time values of the problem.
template <int N>
using Int = std::integral_constant<int, N>;
template <class T, int VEC, class F>
hipError_t with_flags(int kind, bool uniform, F f) {
  const T t{};
  const Int<VEC> v;
  if (kind == GDR_GATE_SOFTPLUS)
    return uniform ? f(t, v, Int<GDR_GATE_SOFTPLUS>(), Int<1>()) : f(t, v, Int<GDR_GATE_SOFTPLUS>(), Int<0>());
  return uniform ? f(t, v, Int<GDR_GATE_SIGMOID>(), Int<1>()) : f(t, v, Int<GDR_GATE_SIGMOID>(), Int<0>());
}
template <int VEC, class F>
hipError_t with_types(const gdr_gate &p, int vec, bool uniform, F f) {
  if (p.dtype == GDR_BF16) return vec == 1 ? with_flags<u16, 1>(p.kind, uniform, f) : with_flags<u16, VEC>(p.kind, uniform, f);
  return vec == 1 ? with_flags<float, 1>(p.kind, uniform, f) : with_flags<float, VEC>(p.kind, uniform, f);
}

// Channels per thread of the forward: a wavefront's stores then cover whole lines one
// after the other (bf16 [261392, 2048] 581 us, with 8 channels 678; fp32 [100000, 2048]
// 289 us, with 8 310).
constexpr int FWD_VEC = 4;

}  // namespace

hipError_t launch_gate_fwd(const gdr_gate &p, float *g, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  const int C = p.H * p.D;
  const int vec = C >= FWD_VEC ? FWD_VEC : 1;
  const Lanes l = lanes_for(groups_of(C, vec));
  // up to 4M threads: few rows each, no sums to share ([261392, 2048] 580 us; 0.5M 616,
  // 0.25M 603, 0.125M 830)
  const int workers = workers_for(((int64_t)p.T + U - 1) / U, l, 1 << 22);
  const GateArgs a = args_of(p, l);
  const unsigned blocks = (unsigned)(workers / l.ly * l.nchb);
  return with_types<FWD_VEC>(p, vec, l.uniform, [&](auto t, auto v, auto k, auto u) {
    using T = decltype(t);
    gate_fwd_kernel<T, decltype(v)::value, decltype(k)::value, decltype(u)::value><<<blocks, l.threads, 0, stream>>>(a, workers, g);
    return hipGetLastError();
  });
}

hipError_t launch_gate_bwd(const gdr_gate &p, const float *dg, void *dx, int64_t dx_stride, float *partial, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  const int C = p.H * p.D;
  const Lanes l = gate_lanes(C);
  const int workers = gate_rows(p.T, C) * l.ly;
  const GateArgs a = args_of(p, l);
  const unsigned blocks = (unsigned)(workers / l.ly * l.nchb);
  return with_types<GATE_VEC>(p, gate_vec(C), l.uniform, [&](auto t, auto v, auto k, auto u) {
    using T = decltype(t);
    gate_bwd_kernel<T, decltype(v)::value, decltype(k)::value, decltype(u)::value><<<blocks, l.threads, 0, stream>>>(
        a, workers, dg, static_cast<T *>(dx), dx_stride, partial);
    return hipGetLastError();
  });
}

}  // namespace gdr
