// Device helpers of the layer kernels: rows of bf16 or fp32 read and written in
// groups of N neighbouring values as floats, and the activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_device.h"

namespace gdr {

// 16-, 8- and 4-byte pieces at any element's address: rows of odd width or stride
// start off their natural alignment, which gfx950's global accesses take.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));

// N values of type T as they lie in memory.
template <class T, int N>
struct Raw {
  static constexpr int WORDS = (N * (int)sizeof(T) + 3) / 4;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (N * sizeof(T) < 4) {
      w[0] = *reinterpret_cast<const u16 *>(p);
    } else {
      constexpr int Q = WORDS / 4;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const u32x4_any x = reinterpret_cast<const u32x4_any *>(p)[i];
        w[4 * i] = x[0]; w[4 * i + 1] = x[1]; w[4 * i + 2] = x[2]; w[4 * i + 3] = x[3];
      }
      if constexpr ((WORDS & 2) != 0) {
        const u32x2_any x = *reinterpret_cast<const u32x2_any *>(reinterpret_cast<const uint32_t *>(p) + 4 * Q);
        w[4 * Q] = x[0]; w[4 * Q + 1] = x[1];
      }
      if constexpr ((WORDS & 1) != 0) w[WORDS - 1] = *reinterpret_cast<const u32_any *>(reinterpret_cast<const uint32_t *>(p) + WORDS - 1);
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (N * sizeof(T) < 4) {
      *reinterpret_cast<u16 *>(p) = (u16)w[0];
    } else {
      constexpr int Q = WORDS / 4;
#pragma unroll
      for (int i = 0; i < Q; ++i)
        reinterpret_cast<u32x4_any *>(p)[i] = u32x4_any{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
      if constexpr ((WORDS & 2) != 0)
        *reinterpret_cast<u32x2_any *>(reinterpret_cast<uint32_t *>(p) + 4 * Q) = u32x2_any{w[4 * Q], w[4 * Q + 1]};
      if constexpr ((WORDS & 1) != 0) *reinterpret_cast<u32_any *>(reinterpret_cast<uint32_t *>(p) + WORDS - 1) = w[WORDS - 1];
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return (i & 1) ? __uint_as_float(w[i >> 1] & 0xffff0000u) : __uint_as_float(w[i >> 1] << 16);
  }
  __device__ __forceinline__ void set(const float (&f)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (N == 1) {
      w[0] = f2bf(f[0]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = pk2bf(f[2 * i], f[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0;
  }
};

// One parameter value stored as bf16 or fp32.
__device__ __forceinline__ float ld_param(const void *p, int64_t i, bool bf) {
  return bf ? bf2f(static_cast<const u16 *>(p)[i]) : static_cast<const float *>(p)[i];
}

// e^x by the hardware's 2^t.  With EXACT the rounding error of t = x log2(e), which
// grows with |x|, is carried into the result; without, it costs a relative |x| 2^-24.
// The convolution and the norm take EXACT for fp32 rows.  For bf16 rows they do not, also
// where an output is fp32 (the parameter sums, and y or dres beside an fp32 residual):
// the error stays below a bf16 half step for every |x| < 88, it is random from value to
// value, so a sum averages it, and the correction would cost the backwards what they
// have left of the vector units (convolution [241817, 6144] 1968 us, without 1792; gated
// norm [4000, 10240] with an fp32 stream 199 us, without 164).
template <bool EXACT>
__device__ __forceinline__ float fast_exp(float x) {
  const float t = x * 1.44269504088896341f;
  const float e = __builtin_amdgcn_exp2f(t);
  if constexpr (!EXACT) return e;
  float lo = fmaf(x, 1.44269504088896341f, -t);          // rounding of the product
  lo = fmaf(x, 1.92596299112661746e-8f, lo);             // log2(e) - float(log2(e))
  const float r = fmaf(e, lo * 0.693147180559945309f, e);
  return __builtin_fabsf(x) < 87.f ? r : e;              // infinities and the underflow range as they are
}
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + fast_exp<EXACT>(-x));
}

// sigma(x) and 1 - sigma(x), either to a few roundings of itself: with e = e^-x they are
// 1 / (1 + e) and e / (1 + e), where 1 - s would leave of a small one only the rounding of
// s.  Where e overflows, s is 0 and so is the c given, which is of use as a factor beside s.
template <bool EXACT>
__device__ __forceinline__ void sigmoid_both(float x, float &s, float &c) {
  const float e = fast_exp<EXACT>(-x);
  s = __builtin_amdgcn_rcpf(1.f + e);
  c = fminf(e, 0x1p126f) * s;
}

// The lane's first channel; the last group of a row whose width is no multiple of
// VEC starts early and repeats its neighbour's channels (the same values, written
// twice), so every access is whole.
template <int VEC>
__device__ __forceinline__ int first_channel(int group, int C) {
  return VEC == 1 ? group : min(group * VEC, C - VEC);
}

// The thread's set within its block.  With UNI a wavefront lies within one set
// (Lanes::uniform): its rows, their addresses and the document's bounds are then
// scalar values, and a row's access is one instruction with a scalar base.
template <bool UNI>
__device__ __forceinline__ int set_of(int lx) {
  const int ty = threadIdx.x / lx;
  return UNI ? __builtin_amdgcn_readfirstlane(ty) : ty;
}

// Adds a block's `ly` sets of K sums per thread (a set is lx threads wide) in a
// fixed tree, halving the sets; the sums of set 0's threads are the block's.  Every
// thread of the block calls it; `lds` holds K x (threads of the block) floats.
template <int K>
__device__ __forceinline__ void add_sets(float (&v)[K], float *lds, int tx, int ty, int lx, int ly) {
  const int threads = blockDim.x;
#pragma unroll
  for (int k = 0; k < K; ++k) lds[k * threads + threadIdx.x] = v[k];
  for (int n = ly; n > 1;) {
    const int h = (n + 1) / 2;
    __syncthreads();
    if (ty + h < n) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[k] += lds[k * threads + (ty + h) * lx + tx];
        lds[k * threads + threadIdx.x] = v[k];
      }
    }
    n = h;
  }
}

}  // namespace gdr
