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
// write, 2 x 64 KB per sequence and head: 256 sequences of 48 heads 317 us, 5.1 TB/s,
// what a copy reaches on that card; one sequence of 16 heads 4.4 us, its loads' latency.
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

// One token's operands for a lane's 16 keys and 4 columns, as they lie in memory.
template <bool GDN>
struct Token {
  Raw<u16, 16> k, q;
  Raw<u16, 4> v;
  Raw<float, GDN ? 1 : 16> g;
  float beta;
  __device__ __forceinline__ void load(const StepArgs &a, int64_t t, int h, int hq, int key, int col) {
    k.load(a.k + t * a.ks + hq * HD + key);
    q.load(a.q + t * a.qs + hq * HD + key);
    v.load(a.v + t * a.vs + h * HD + col);
    g.load(a.g + (GDN ? t * a.Hv + h : (t * a.Hv + h) * HD + key));
    beta = ld_param(a.beta, t * a.Hv + h, !GDN);
  }
};

// RUN: sequences given by cu_seqlens; otherwise one token each, whose operands do not
// wait for the slot.  (Reading a run's next token during the current one takes 177
// registers, two wavefronts per SIMD instead of three: 16 runs at 64 heads 30 us, not 26.)
template <bool GDN, bool NORM, bool SIGM, bool RUN>
__global__ __launch_bounds__(256) void step_kernel(StepArgs a) {
  const int lane = threadIdx.x & 63, rg = lane >> 3, qd = lane & 7;
  const int slice = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = blockIdx.x / a.Hv, h = blockIdx.x - n * a.Hv, hq = h / a.group;
  const int slot = a.slots ? a.slots[n] : n;
  int t0 = n, t1 = n + 1;
  if constexpr (RUN) {
    t0 = max(a.cu[n], 0), t1 = min(a.cu[n + 1], a.T);
    if (t0 >= t1) return;
  }
  const int key = 16 * rg, col = 32 * slice + 4 * qd;
  Token<GDN> x;
  if constexpr (!RUN) x.load(a, t0, h, hq, key, col);
  if (slot < 0 || slot >= a.n_slots) return;
  float *sp = a.state + (((int64_t)slot * a.Hv + h) * HD + key) * HD + col;
  f32x4 S[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) S[j] = *reinterpret_cast<const f32x4 *>(sp + j * HD);

  for (int t = t0; t < t1; ++t) {
    if constexpr (RUN) x.load(a, t, h, hq, key, col);
    float dec[GDN ? 1 : 16];
#pragma unroll
    for (int j = 0; j < (GDN ? 1 : 16); ++j) dec[j] = fast_exp<true>(x.g.get(j));
    const float beta = SIGM ? sigmoid<true>(x.beta) : x.beta;

    float r[4] = {}, p[4] = {}, kq = 0.f, kk = 0.f, qq = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float kj = x.k.get(j), qj = x.q.get(j);
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
      coef[e] = beta * (x.v.get(e) - nk * r[e]) * nk;
      out[e] = a.scale * nq * fmaf(kq, coef[e], p[e]);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[j][e] = fmaf(x.k.get(j), coef[e], S[j][e]);
    if (rg == 0) {
      Raw<u16, 4> ro;
      ro.set(out);
      ro.store(a.o + ((int64_t)t * a.Hv + h) * HD + col);
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
  using Y = std::true_type;
  using X = std::false_type;
  auto go = [&](auto g, auto n, auto s) {
    if (a.cu) step_kernel<decltype(g)::value, decltype(n)::value, decltype(s)::value, true><<<blocks, 256, 0, stream>>>(a);
    else step_kernel<decltype(g)::value, decltype(n)::value, decltype(s)::value, false><<<blocks, 256, 0, stream>>>(a);
    return hipGetLastError();
  };
  auto flags = [&](auto g) {
    const bool norm = p.input_flags & GDR_IN_QK_L2NORM, sigm = p.input_flags & GDR_IN_BETA_SIGMOID;
    return norm ? (sigm ? go(g, Y(), Y()) : go(g, Y(), X())) : (sigm ? go(g, X(), Y()) : go(g, X(), X()));
  };
  return gdn ? flags(Y()) : flags(X());
}

}  // namespace gdr
