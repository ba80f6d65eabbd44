// Keys and values to and from the cache in 4 bits.  32 channels of a token and head share
// the smallest power of two 2^e with max|x| <= 6 2^e; x 2^-e is then at most 6 and is
// rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code.  From
// bf16 everything but that rounding is exact: e is read off the largest magnitude's bits
// (the mantissa above or below 1.5), and the scaling moves an exponent.
//
// Bound by the bytes, 256 + 68 a token, head and side.  16 lanes take a row of 128 channels,
// 8 each: 16 bytes of bf16 and 4 of codes, so both sides' accesses are whole lines; four
// lanes share a block, whose maximum they find by two lane swaps.  32674 tokens of 4 heads: stored in 21 us, 4.0 TB/s,
// read back in 17 us, 5.2 TB/s (the same tokens again; both calls 36 us, 43 on tokens that the caches do not hold).  (Codes
// by comparing with every border instead of the hardware's conversion: 35 us, the vector units' time.)
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

typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
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
  const float s = __uint_as_float(scale << 23);
  uint32_t w[4] = {x[0], x[1], x[2], x[3]};
  if (scale == 253) {  // 4 2^126 is past bf16: magnitudes past 3 2^126 count as that
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (w[i] & 0x80008000u) | min(w[i] & 0x7fffu, 0x7f40u) | min(w[i] & 0x7fff0000u, 0x7f400000u);
  }
  uint32_t out = 0;  // the hardware's conversion of w / s: to nearest, ties to the even code
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, __builtin_bit_cast(bf16x2v, w[0]), s, 0);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, __builtin_bit_cast(bf16x2v, w[1]), s, 1);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, __builtin_bit_cast(bf16x2v, w[2]), s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, __builtin_bit_cast(bf16x2v, w[3]), s, 3);
}
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

// Places of tokens t of kv heads h in the pool, in tokens; -1 where there is none (or t < 0).  The sequence
// is the last n with cu[n] <= t (cu clipped to [0, T]); ROWS searches go side by side.
template <int ROWS>
__device__ __forceinline__ void places_of(const KvArgs &a, const int (&t)[ROWS], const int (&h)[ROWS], int64_t (&place)[ROWS]) {
  int n[ROWS], end[ROWS];  // n: cu[n] <= t but for n == 0; cu[end] > t but for end == N
#pragma unroll
  for (int r = 0; r < ROWS; ++r) n[r] = a.cu ? 0 : max(t[r], 0), end[r] = a.N, place[r] = t[r] < 0 ? -1 : 0;
  if (a.cu) {
    for (int left = a.N; left > 1; left = (left + 1) >> 1)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const int mid = (n[r] + end[r]) >> 1;
        if (min(max(a.cu[mid], 0), a.T) <= t[r]) n[r] = mid;
        else end[r] = max(mid, n[r] + 1);
      }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int from = max(a.cu[n[r]], 0);
      if (t[r] < from || t[r] >= min(a.cu[n[r] + 1], a.T)) place[r] = -1;
      else place[r] = t[r] - from;
    }
  }
  int page[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    bool there = place[r] >= 0;
    if (a.start) place[r] += a.start[n[r]];
    there = there && place[r] >= 0 && place[r] >> a.page_shift < a.max_pages;
    if (!there) place[r] = -1;
    page[r] = a.table[(int64_t)n[r] * a.max_pages + (there ? place[r] >> a.page_shift : 0)];
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (place[r] < 0 || page[r] < 0 || page[r] >= a.n_pages) place[r] = -1;
    else place[r] = (((int64_t)page[r] * a.H + h[r]) << a.page_shift) + (place[r] & ((1 << a.page_shift) - 1));
  }
}

// A thread takes ROWS rows, 16 apart, so that their places' chains of loads run side by side: 2 to read
// back and to store many rows, 1 to store few (32674 tokens of 4 heads stored and read back 35.8 us; stored with
// 1 37.0; 10600 rows stored and 66000 read back 16.6 us, stored with 2 17.2).
template <bool STORE, int ROWS>
__global__ __launch_bounds__(256) void kv_kernel(KvArgs a) {
  const int x = threadIdx.x & 15;
  const uint32_t row0 = blockIdx.x * (16 * ROWS) + (threadIdx.x >> 4), rows = (uint32_t)a.T * a.H;  // a launch has fewer than 2^28
  u32x4_any k8[ROWS], v8[ROWS];
  u16 *kp[ROWS], *vp[ROWS];
  int64_t place[ROWS];
  int t[ROWS], h[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const uint32_t row = row0 + 16 * r, token = row / (uint32_t)a.H;
    t[r] = row < rows ? (int)token : -1, h[r] = (int)(row - token * a.H);
    if (row >= rows) continue;  // whole quads go together
    kp[r] = a.k + t[r] * a.ks + h[r] * HD + 8 * x, vp[r] = a.v + t[r] * a.vs + h[r] * HD + 8 * x;
    if constexpr (STORE) {
      k8[r] = *reinterpret_cast<const u32x4_any *>(kp[r]);
      v8[r] = *reinterpret_cast<const u32x4_any *>(vp[r]);
    }
  }
  places_of(a, t, h, place);
  if constexpr (STORE) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (place[r] < 0) continue;
      uint32_t s, u;
      reinterpret_cast<uint32_t *>(a.kc + place[r] * 64)[x] = to_codes(k8[r], s);
      reinterpret_cast<uint32_t *>(a.vc + place[r] * 64)[x] = to_codes(v8[r], u);
      if ((x & 3) == 0) a.ksc[place[r] * 4 + (x >> 2)] = (uint8_t)s, a.vsc[place[r] * 4 + (x >> 2)] = (uint8_t)u;
    }
  } else {
    uint32_t kw[ROWS], vw[ROWS], s[ROWS], u[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int64_t at = max(place[r], (int64_t)0);  // a token without a place reads the first one's
      kw[r] = reinterpret_cast<const uint32_t *>(a.kc + at * 64)[x], vw[r] = reinterpret_cast<const uint32_t *>(a.vc + at * 64)[x];
      s[r] = a.ksc[at * 4 + (x >> 2)], u[r] = a.vsc[at * 4 + (x >> 2)];
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (place[r] < 0) continue;
      *reinterpret_cast<u32x4_any *>(kp[r]) = from_codes(kw[r], s[r]);
      *reinterpret_cast<u32x4_any *>(vp[r]) = from_codes(vw[r], u[r]);
    }
  }
}

}  // namespace

hipError_t launch_kv(const gdr_kv &p, bool store, int32_t T, const int32_t *cu, const int32_t *start, uint16_t *k,
                     int64_t k_stride, uint16_t *v, int64_t v_stride, hipStream_t stream) {
  if (T == 0 || p.N == 0 || p.max_pages == 0 || p.n_pages == 0) return hipSuccess;
  const KvArgs a{p.k_codes, p.v_codes, p.k_scale, p.v_scale, p.page_table, cu, start, k, v, k_stride, v_stride, T, p.H_kv, p.N,
                 p.n_pages, __builtin_ctz((unsigned)p.page), p.max_pages};
  const int64_t rows = (int64_t)T * p.H_kv;
  auto blocks = [&](int each) { return dim3((uint32_t)((rows + 16 * each - 1) / (16 * each))); };
  const bool many = rows >= 65536;  // more than a round of blocks with 2 rows a thread
  if (store && many) kv_kernel<true, 2><<<blocks(2), 256, 0, stream>>>(a);
  else if (store) kv_kernel<true, 1><<<blocks(1), 256, 0, stream>>>(a);
  else kv_kernel<false, 2><<<blocks(2), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace gdr
