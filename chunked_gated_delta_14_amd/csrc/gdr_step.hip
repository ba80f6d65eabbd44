// The gated delta rule for single tokens and short runs of them, on a pool of
// states that stay in place:
//   S <- Diag(e^g) S;  r = S^T k;  S <- S + beta k (v - r)^T;  o = scale S^T q
//
// Both products need the decayed state only: with p = S^T q of the decayed state,
// o = scale (p + (k.q) beta (v - r)), so one reduction over the keys gives r, p
// and k.q together.  A wavefront takes 32 value columns of one head's state: lane
// (rg, qd) = (lane / 8, lane % 8) holds keys 16 rg .. +15 of columns 4 qd .. +3 in
// 64 registers, every load and store of a key's 32 columns covers a 128-byte line,
// and the reduction runs over the 8 lane groups.  Bound by the state's read and
// write, 2 x 64 KB per sequence and head.
#include "gdr_layer.h"
#include "gdr_vec.h"
#include "gdr_kernels.h"

namespace gdr {
namespace {

struct StepArgs {
  const u16 *q, *k, *v;
  const float *g;
  const void *beta;
  const int32_t *cu, *slots;
  float *state;
  u16 *o;
  int T, N, Hqk, Hv, group, n_slots;
  int64_t qs, ks, vs;
  float scale;
};

__device__ __forceinline__ float sum_groups(float x) {  // over the 8 lane groups
  x += __shfl_xor(x, 8);
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

template <bool GDN, bool NORM, bool SIGM>
__global__ __launch_bounds__(256) void step_kernel(StepArgs a) {
  const int lane = threadIdx.x & 63, rg = lane >> 3, qd = lane & 7;
  const int slice = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = blockIdx.x / a.Hv, h = blockIdx.x - n * a.Hv, hq = h / a.group;
  int t0 = n, t1 = n + 1;
  if (a.cu) t0 = max(a.cu[n], 0), t1 = min(a.cu[n + 1], a.T);
  const int slot = a.slots ? a.slots[n] : n;
  if (t0 >= t1 || slot < 0 || slot >= a.n_slots) return;
  float *sp = a.state + (((int64_t)slot * a.Hv + h) * HD + 16 * rg) * HD + 32 * slice + 4 * qd;
  f32x4 S[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) S[j] = *reinterpret_cast<const f32x4 *>(sp + j * HD);

  for (int t = t0; t < t1; ++t) {
    Raw<u16, 16> rk, rq;
    rk.load(a.k + (int64_t)t * a.ks + hq * HD + 16 * rg);
    rq.load(a.q + (int64_t)t * a.qs + hq * HD + 16 * rg);
    Raw<u16, 4> rv;
    rv.load(a.v + (int64_t)t * a.vs + h * HD + 32 * slice + 4 * qd);
    float dec[GDN ? 1 : 16];
    if constexpr (GDN) {
      dec[0] = fast_exp<true>(a.g[(int64_t)t * a.Hv + h]);
    } else {
      Raw<float, 16> rd;
      rd.load(a.g + ((int64_t)t * a.Hv + h) * HD + 16 * rg);
#pragma unroll
      for (int j = 0; j < 16; ++j) dec[j] = fast_exp<true>(rd.get(j));
    }
    float beta = ld_param(a.beta, (int64_t)t * a.Hv + h, !GDN);
    if constexpr (SIGM) beta = sigmoid<true>(beta);

    float r[4] = {}, p[4] = {}, kq = 0.f, kk = 0.f, qq = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float kj = rk.get(j), qj = rq.get(j);
      kq = fmaf(kj, qj, kq);
      if constexpr (NORM) kk = fmaf(kj, kj, kk), qq = fmaf(qj, qj, qq);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[j][e] *= dec[GDN ? 0 : j];
        r[e] = fmaf(kj, S[j][e], r[e]);
        p[e] = fmaf(qj, S[j][e], p[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = sum_groups(r[e]), p[e] = sum_groups(p[e]);
    kq = sum_groups(kq);
    float nk = 1.f, nq = 1.f;
    if constexpr (NORM) {
      nk = __builtin_amdgcn_rsqf(sum_groups(kk) + L2NORM_EPS);
      nq = __builtin_amdgcn_rsqf(sum_groups(qq) + L2NORM_EPS);
    }
    float out[4], coef[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c = beta * (rv.get(e) - nk * r[e]);
      coef[e] = c * nk;
      out[e] = a.scale * nq * fmaf(kq, coef[e], p[e]);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[j][e] = fmaf(rk.get(j), coef[e], S[j][e]);
    if (rg == 0) {
      Raw<u16, 4> ro;
      ro.set(out);
      ro.store(a.o + ((int64_t)t * a.Hv + h) * HD + 32 * slice + 4 * qd);
    }
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) *reinterpret_cast<f32x4 *>(sp + j * HD) = S[j];
}

}  // namespace

hipError_t launch_step(bool gdn, const gdr_step &p, uint16_t *o, hipStream_t stream) {
  if (p.T == 0 || p.N == 0) return hipSuccess;
  StepArgs a{};
  a.q = p.q; a.k = p.k; a.v = p.v; a.g = p.g; a.beta = p.beta;
  a.cu = p.cu_seqlens; a.slots = p.slots; a.state = p.state; a.o = o;
  a.T = p.T; a.N = p.N; a.Hqk = p.H_qk; a.Hv = p.H_v; a.group = p.H_v / p.H_qk; a.n_slots = p.n_slots;
  a.qs = p.q_stride; a.ks = p.k_stride; a.vs = p.v_stride;
  a.scale = p.scale;
  const unsigned blocks = (unsigned)p.N * (unsigned)p.H_v;
  const bool norm = p.input_flags & GDR_IN_QK_L2NORM, sigm = p.input_flags & GDR_IN_BETA_SIGMOID;
  auto go = [&](auto g, auto n, auto s) {
    step_kernel<decltype(g)::value, decltype(n)::value, decltype(s)::value><<<blocks, 256, 0, stream>>>(a);
    return hipGetLastError();
  };
  using Y = std::true_type;
  using X = std::false_type;
  if (gdn) return norm ? (sigm ? go(Y(), Y(), Y()) : go(Y(), Y(), X())) : (sigm ? go(Y(), X(), Y()) : go(Y(), X(), X()));
  return norm ? (sigm ? go(X(), Y(), Y()) : go(X(), Y(), X())) : (sigm ? go(X(), X(), Y()) : go(X(), X(), X()));
}

}  // namespace gdr
