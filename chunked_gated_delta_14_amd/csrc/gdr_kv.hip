// Keys and values to and from the cache in 4 bits.  32 channels of a token and head share
// the smallest power of two 2^e with max|x| <= 6 2^e; x 2^-e is then at most 6 and is
// rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code.  From
// bf16 everything but that rounding is exact: e is read off the largest magnitude's bits
// (the mantissa above or below 1.5), and the scaling moves an exponent.
//
// Bound by the bytes, 256 + 68 a token, head and side.  16 lanes take a row of 128 channels,
// 8 each: 16 bytes of bf16 and 4 of codes, so both sides' accesses are whole lines; four
// lanes share a block, whose maximum they find by two lane swaps.
#include "gdr_attn.h"
#include "gdr_vec.h"

namespace gdr {
namespace {

struct KvArgs {
  uint8_t *kc, *vc, *ksc, *vsc;
  const int32_t *table, *cu, *start;
  u16 *k, *v;
  int64_t ks, vs;
  int T, H, N, n_pages, page_shift, max_pages;
};

// The sequence of token t: the last n with cu[n] <= t (cu clipped to [0, T]); -1 without one.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int N, int T, int t) {
  int lo = 0, hi = N;  // cu[lo] <= t is open for lo == 0, cu[hi] > t for hi == N
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (min(max(cu[mid], 0), T) <= t) lo = mid;
    else hi = mid;
  }
  return N > 0 && max(cu[lo], 0) <= t && t < min(cu[lo + 1], T) ? lo : -1;
}

// Eight bf16 to eight codes; the block's exponent is over the quad of lanes.
__device__ __forceinline__ uint32_t to_codes(const u32x4 x, uint32_t &scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  if (m >= 0x7f80u) {  // infinite or NaN
    scale = 255;
    return 0;
  }
  // 6 2^e is 1.5 2^(e+2): the largest's exponent less 2, one more if its mantissa is past 1.5
  const int e = (int)(m >> 7) - 2 + ((m & 0x7f) > 0x40);
  scale = (uint32_t)max(e, 1);
  const float by = __uint_as_float((254u - scale) << 23);  // 2^-e; scale is 253 at most
  const uint32_t most = scale == 253 ? 5 : 7;  // 4 2^126 is past bf16
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t h = i & 1 ? x[i >> 1] >> 16 : x[i >> 1] & 0xffffu;
    const float a = __uint_as_float((h & 0x7fffu) << 16) * by;
    // the code is the number of borders passed; a tie goes up where the code above is even
    const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.f);
    out |= (min(c, most) | ((h >> 12) & 8u)) << (4 * i);
  }
  return out;
}
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x4 from_codes(uint32_t c, uint32_t scale) {
  const float s = __uint_as_float(scale << 23);
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, (bf16x2v)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
  r[1] = __builtin_bit_cast(uint32_t, (bf16x2v)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
  r[2] = __builtin_bit_cast(uint32_t, (bf16x2v)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
  r[3] = __builtin_bit_cast(uint32_t, (bf16x2v)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
  if (scale == 255) r = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
  return r;
}

template <bool STORE>
__global__ __launch_bounds__(256) void kv_kernel(KvArgs a) {
  const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int x = threadIdx.x & 15;
  if (row >= (int64_t)a.T * a.H) return;  // whole quads leave together
  const int t = (int)(row / a.H), h = (int)(row - (int64_t)t * a.H);
  u32x4_any k8, v8;
  u16 *kp = a.k + t * a.ks + h * HD + 8 * x, *vp = a.v + t * a.vs + h * HD + 8 * x;
  if constexpr (STORE) {  // these do not wait for the place
    k8 = *reinterpret_cast<const u32x4_any *>(kp);
    v8 = *reinterpret_cast<const u32x4_any *>(vp);
  }
  int n = t;
  int64_t at = 0;
  if (a.cu) {
    n = sequence_of(a.cu, a.N, a.T, t);
    if (n < 0) return;
    at = t - max(a.cu[n], 0);
  }
  if (a.start) at += a.start[n];
  const int64_t col = at >> a.page_shift;
  if (at < 0 || col >= a.max_pages) return;
  const int page = a.table[(int64_t)n * a.max_pages + col];
  if (page < 0 || page >= a.n_pages) return;
  const int64_t place = ((((int64_t)page * a.H + h) << a.page_shift) + (at & ((1 << a.page_shift) - 1)));
  uint32_t *kc = reinterpret_cast<uint32_t *>(a.kc + place * 64) + x, *vc = reinterpret_cast<uint32_t *>(a.vc + place * 64) + x;
  uint8_t *ksc = a.ksc + place * 4 + (x >> 2), *vsc = a.vsc + place * 4 + (x >> 2);
  if constexpr (STORE) {
    uint32_t s, u;
    *kc = to_codes(k8, s);
    *vc = to_codes(v8, u);
    if ((x & 3) == 0) *ksc = (uint8_t)s, *vsc = (uint8_t)u;
  } else {
    const uint32_t kw = *kc, vw = *vc, s = *ksc, u = *vsc;
    *reinterpret_cast<u32x4_any *>(kp) = from_codes(kw, s);
    *reinterpret_cast<u32x4_any *>(vp) = from_codes(vw, u);
  }
}

}  // namespace

hipError_t launch_kv(const gdr_kv &p, bool store, int32_t T, const int32_t *cu, const int32_t *start, uint16_t *k,
                     int64_t k_stride, uint16_t *v, int64_t v_stride, hipStream_t stream) {
  if (T == 0 || p.N == 0 || p.max_pages == 0 || p.n_pages == 0) return hipSuccess;
  const KvArgs a{p.k_codes, p.v_codes, p.k_scale, p.v_scale, p.page_table, cu, start, k, v, k_stride, v_stride, T, p.H_kv, p.N,
                 p.n_pages, __builtin_ctz((unsigned)p.page), p.max_pages};
  const dim3 grid((uint32_t)(((int64_t)T * p.H_kv + 15) / 16));
  if (store) kv_kernel<true><<<grid, 256, 0, stream>>>(a);
  else kv_kernel<false><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace gdr
