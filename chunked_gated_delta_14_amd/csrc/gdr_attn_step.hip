// Attention of a sequence's last tokens over keys and values held in 4 bits.
//
// Bound by the cache's bytes, 136 a token and kv head, which are read once: the query
// heads of a kv head and the tokens of a run are the columns of one matrix product.  A
// wavefront takes 32 tokens at a time and forms, with v_mfma_f32_16x16x32_bf16 and lane =
// 16 g + lr,
//   S^T (token, row) = K Q^T:    A lane: 32 channels 32 g .. of token lr, one 16-byte load;
//   O^T (channel, row) += V^T P^T: A lane: channels 8 lr .. 8 lr + 7 of tokens 4 g .. 4 g + 3
//       of either half of the 32, which is where S^T's registers hold the probabilities.
// Codes become bf16, exactly, by the hardware's scaled conversion, which makes NaN of the infinite scale that a byte
// of 255 gives; V's are then regrouped from pairs of channels to pairs of tokens.  The order of channels within a product is
// free, so both sides read the cache as it lies: row by row.
//
// A sequence's tokens are split over blocks, and over a block's wavefronts; each keeps a running
// maximum and sum, the block joins its wavefronts' in LDS, and a second kernel
// joins the blocks' where there are several.  64 sequences of 1 to 32000 tokens, 32 heads on 8: a call
// 221 us, 5.1 TB/s of the cache's bytes, a copy's rate, vector units half busy; one of 4096, 16 heads on 2: 5.0 us, its
// chain of loads, and 3.5 for the join.  (Two tiles' registers, the next loaded whole while one is worked on, leave two
// wavefronts to a SIMD instead of three: 276 us.  Four, which spills: 303.)
#include "gdr_attn_device.h"
#include "gdr_vec.h"

namespace gdr {
namespace {

struct StepArgs {
  const u16 *q;
  const uint8_t *kc, *vc, *ksc, *vsc;
  const int32_t *table, *lens, *cu;
  u16 *o;
  float *part, *ml;  // [rows][splits][128]; [rows][splits][2]
  int64_t qs;
  int T, N, Hq, Hkv, group, n_pages, page_shift, max_pages, window, splits, row_tiles;
  float c;  // scale log2(e)
};

// A sequence's rows and tokens, clipped to what there is.
struct Span {
  int t0, run, len, begin, per;
  __device__ __forceinline__ Span(const StepArgs &a, int n) {
    t0 = n, run = 1;
    if (a.cu) {
      t0 = max(a.cu[n], 0);
      run = min(a.cu[n + 1], a.T) - t0;
    }
    len = (int)min((int64_t)max(a.lens[n], 0), (int64_t)a.max_pages << a.page_shift);
    begin = a.window ? max(0, len - run - a.window + 1) : 0;
    const int share = (len - (begin & ~31) + a.splits - 1) / a.splits;
    per = max(STEP_UNIT, (share + STEP_UNIT - 1) & ~(STEP_UNIT - 1));
  }
};

typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
template <int SEL>
__device__ __forceinline__ uint32_t pair(uint32_t c, float s) {
  return __builtin_bit_cast(uint32_t, (bf16x2v)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, SEL));
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// RUNS: sequences may have several rows, which see different tokens (a row a sequence without: 256 sequences of 1000, 16
// heads on 4, 27.7 us for 28.2 with).
template <bool RUNS>
__global__ __launch_bounds__(256, 3) void attn_step_kernel(StepArgs a) {
  constexpr int PITCH = 132;
  __shared__ __align__(16) float so[4][16][PITCH];
  __shared__ float sm[4][16], sl[4][16];
  const int lane = threadIdx.x & 63, lr = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int b = blockIdx.x;
  const int rt0 = b % a.row_tiles;
  b /= a.row_tiles;
  const int split = b % a.splits;
  b /= a.splits;
  const int kvh = b % a.Hkv, n = b / a.Hkv;
  const Span s(a, n);
  if (s.run <= 0) return;
  const int from = (s.begin & ~31) + split * s.per, to = min(s.len, from + s.per);
  if (from >= to && a.splits > 1) return;
  const int rows = s.run * a.group;
  const int32_t *pages = a.table + (int64_t)n * a.max_pages;

  for (int rt = rt0; rt * 16 < rows; rt += a.row_tiles) {
    const int rr = min(rt * 16 + lr, rows - 1), i = rr / a.group;
    const int head = kvh * a.group + rr - i * a.group;
    const int hi = s.len - s.run + i, lo = a.window ? max(0, hi - a.window + 1) : 0;
    bf16x8 Q[4];
    {
      const u16 *qp = a.q + (s.t0 + i) * a.qs + head * HD + 32 * g;
#pragma unroll
      for (int x = 0; x < 4; ++x) Q[x] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4_any *>(qp + 8 * x));
    }
    f32x4 O[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) O[d] = zero4();
    float m = LEAST, l = 0.f;
    // Values that are NaN (a scale byte of 255) in tiles that not every row sees all of: there they count as finite, as 0
    // times them would reach rows that they are hidden from.  Bit 8 b + 7: this lane's row sees one in its channels 32 b .. .
    uint32_t bad = 0;

    // pages of this wavefront's next 32 tiles, two to a tile, one a lane
    int pv = -1;
    auto load_pages = [&](int it) {
      const int64_t j = (int64_t)from + 32 * (wave + 4 * (it + (lane >> 1))) + 16 * (lane & 1);
      pv = -1;
      if (j < to) {
        const int p = pages[j >> a.page_shift];
        if (p >= 0 && p < a.n_pages) pv = p;
      }
    };
    // Keys and values of a tile as they lie in memory.  The next tile's are loaded as soon as this one's
    // are used, the keys before the softmax and the values after it, into the same registers.
    u32x4 kc[2], vs[2];
    uint32_t ks[2], vc[8];
    auto place = [&](int it, int u) {
      const int p = max(__builtin_amdgcn_readlane(pv, 2 * (it & 31) + u), 0), j = from + 32 * (wave + 4 * it) + 16 * u;
      return (((int64_t)p * a.Hkv + kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
    };
    auto load_keys = [&](int it) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t at = place(it, u);
        kc[u] = *reinterpret_cast<const u32x4 *>(a.kc + at * 64 + (lr * 64 + g * 16));
        ks[u] = (a.ksc + at * 4)[lr * 4 + g];
      }
    };
    auto load_values = [&](int it) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t at = place(it, u);
#pragma unroll
        for (int r = 0; r < 4; ++r) vc[4 * u + r] = *reinterpret_cast<const uint32_t *>(a.vc + at * 64 + ((4 * g + r) * 64 + lr * 4));
        vs[u] = *reinterpret_cast<const u32x4 *>(a.vsc + at * 4 + g * 16);
      }
    };
    const int tiles = (to - from + 31) / 32, mine = tiles > wave ? (tiles - wave + 3) / 4 : 0;
    int pg0 = 0, pg1 = 0;
    if (mine > 0) {
      load_pages(0);
      pg0 = __builtin_amdgcn_readlane(pv, 0), pg1 = __builtin_amdgcn_readlane(pv, 1);
      load_keys(0);
      load_values(0);
    }
    for (int it = 0; it < mine; ++it) {
      const int j = from + 32 * (wave + 4 * it);
      const bool more = it + 1 < mine;
      if (more && ((it + 1) & 31) == 0) load_pages(it + 1);
      // tiles whose tokens not every row sees
      const bool masked = j + 32 > s.len - s.run + 1 || j < s.begin || (a.window && j < s.len - a.window) || pg0 < 0 || pg1 < 0;
      f32x4 S[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        S[u] = zero4();
        const float sc = scale_of(ks[u]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t w = kc[u][y];
          S[u] = mfma(__builtin_bit_cast(bf16x8, u32x4{pair<0>(w, sc), pair<1>(w, sc), pair<2>(w, sc), pair<3>(w, sc)}), Q[y], S[u]);
        }
      }
      if (more) load_keys(it + 1);
      if (masked) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = j + 16 * u + 4 * g + r;
            const bool there = (u ? pg1 : pg0) >= 0, seen = there && t <= hi && t >= lo;
            if (!seen) S[u][r] = -INFINITY;
            if (!there || t >= s.len || t < s.begin) vc[4 * u + r] = 0, vs[u][r] = 0x7f7f7f7fu;  // whatever lies there
            if constexpr (RUNS) {
              const uint32_t w = vs[u][r], nans = ((w & 0x7f7f7f7fu) + 0x01010101u) & w & 0x80808080u;
              vs[u][r] = w ^ nans;
              bad |= seen ? nans : 0u;
            }
          }
      }
      float top = fmaxf(fmaxf(fmaxf(S[0][0], S[0][1]), fmaxf(S[0][2], S[0][3])), fmaxf(fmaxf(S[1][0], S[1][1]), fmaxf(S[1][2], S[1][3])));
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32)) * a.c;
      if (__any(top > m + 8.f)) {
        const float up = fmaxf(top, m), f = __builtin_amdgcn_exp2f(m - up);
        m = up;
        l *= f;
#pragma unroll
        for (int d = 0; d < 8; ++d) O[d] *= f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          S[u][r] = __builtin_amdgcn_exp2f(fmaf(S[u][r], a.c, -m));
          l += S[u][r];
        }
      const bf16x8 P = __builtin_bit_cast(
          bf16x8, u32x4{pk2bf(S[0][0], S[0][1]), pk2bf(S[0][2], S[0][3]), pk2bf(S[1][0], S[1][1]), pk2bf(S[1][2], S[1][3])});
      float sc[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) sc[t] = scale_of((vs[t >> 2][t & 3] >> (8 * (lr >> 2))) & 0xffu);
      auto channels = [&](auto sel) {  // two channels of all tokens
        constexpr int SEL = decltype(sel)::value;
        uint32_t w[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) w[t] = pair<SEL>(vc[t], sc[t]);
        u32x4 even, odd;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          even[t] = __builtin_amdgcn_perm(w[2 * t + 1], w[2 * t], 0x05040100u);
          odd[t] = __builtin_amdgcn_perm(w[2 * t + 1], w[2 * t], 0x07060302u);
        }
        O[2 * SEL] = mfma(__builtin_bit_cast(bf16x8, even), P, O[2 * SEL]);
        O[2 * SEL + 1] = mfma(__builtin_bit_cast(bf16x8, odd), P, O[2 * SEL + 1]);
      };
      channels(std::integral_constant<int, 0>{});
      channels(std::integral_constant<int, 1>{});
      channels(std::integral_constant<int, 2>{});
      channels(std::integral_constant<int, 3>{});
      if (more) {
        load_values(it + 1);
        pg0 = __builtin_amdgcn_readlane(pv, 2 * ((it + 1) & 31)), pg1 = __builtin_amdgcn_readlane(pv, 2 * ((it + 1) & 31) + 1);
      }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    // the wavefronts' results: lane (g, lr) holds channels 32 g + 8 r .. +7 of row lr in O[0..7][r]
    if constexpr (RUNS) {
      bad |= __shfl_xor(bad, 16);
      bad |= __shfl_xor(bad, 32);
      if (bad >> (8 * g + 7) & 1)
#pragma unroll
        for (int d = 0; d < 8; ++d) O[d] = zero4() + __builtin_nanf("");
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      *reinterpret_cast<f32x4 *>(&so[wave][lr][32 * g + 8 * r]) = f32x4{O[0][r], O[1][r], O[2][r], O[3][r]};
      *reinterpret_cast<f32x4 *>(&so[wave][lr][32 * g + 8 * r + 4]) = f32x4{O[4][r], O[5][r], O[6][r], O[7][r]};
    }
    if (g == 0) sm[wave][lr] = m, sl[wave][lr] = l;
    __syncthreads();
    const int row = threadIdx.x >> 4, c = (threadIdx.x & 15) * 8, r2 = rt * 16 + row;
    if (r2 < rows) {
      float M = sm[0][row], L = 0.f, y[8] = {};
#pragma unroll
      for (int w = 1; w < 4; ++w) M = fmaxf(M, sm[w][row]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(sm[w][row] - M);
        L = fmaf(sl[w][row], f, L);
#pragma unroll
        for (int z = 0; z < 8; ++z) y[z] = fmaf(so[w][row][c + z], f, y[z]);
      }
      const int i2 = r2 / a.group;
      const int64_t at = (int64_t)(s.t0 + i2) * a.Hq + kvh * a.group + r2 - i2 * a.group;
      if (a.splits == 1) {
        const float f = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<u32x4 *>(a.o + at * HD + c) =
            u32x4{pk2bf(y[0] * f, y[1] * f), pk2bf(y[2] * f, y[3] * f), pk2bf(y[4] * f, y[5] * f), pk2bf(y[6] * f, y[7] * f)};
      } else {
        const int64_t x2 = at * a.splits + split;
        f32x4 *out = reinterpret_cast<f32x4 *>(a.part + x2 * HD + c);
        out[0] = f32x4{y[0], y[1], y[2], y[3]};
        out[1] = f32x4{y[4], y[5], y[6], y[7]};
        if (c == 0) a.ml[2 * x2] = M, a.ml[2 * x2 + 1] = L;
      }
    }
    __syncthreads();
  }
}

// Joins the splits of a sequence's rows: a block takes one head, 16 threads 8 channels each of every
// 16th split, and the 16 sums are joined in LDS.
__global__ __launch_bounds__(256) void attn_step_join_kernel(StepArgs a) {
  __shared__ float so[16][HD + 4], sm[16], sl[16];
  const int head = blockIdx.x % a.Hq, n = blockIdx.x / a.Hq, c = (threadIdx.x & 15) * 8, y = threadIdx.x >> 4;
  const Span s(a, n);
  const int used = (s.len - (s.begin & ~31) + s.per - 1) / s.per;
  for (int i = 0; i < s.run; ++i) {
    const int64_t row = (int64_t)(s.t0 + i) * a.Hq + head, at = row * a.splits;
    float m = LEAST, l = 0.f, o[8] = {};
    for (int x = y; x < used; x += 16) {
      const float mx = a.ml[2 * (at + x)], lx = a.ml[2 * (at + x) + 1];
      const f32x4 *src = reinterpret_cast<const f32x4 *>(a.part + (at + x) * HD + c);
      const f32x4 u = src[0], v = src[1];
      const float up = fmaxf(m, mx), f = __builtin_amdgcn_exp2f(m - up), e = __builtin_amdgcn_exp2f(mx - up);
      m = up;
      l = fmaf(l, f, lx * e);
#pragma unroll
      for (int z = 0; z < 4; ++z) o[z] = fmaf(o[z], f, u[z] * e), o[4 + z] = fmaf(o[4 + z], f, v[z] * e);
    }
#pragma unroll
    for (int z = 0; z < 8; ++z) so[y][c + z] = o[z];
    if (c == 0) sm[y] = m, sl[y] = l;
    __syncthreads();
    if (threadIdx.x < HD) {
      const int groups = min(used, 16);
      float M = LEAST, L = 0.f, z = 0.f;
      for (int x = 0; x < groups; ++x) M = fmaxf(M, sm[x]);
      for (int x = 0; x < groups; ++x) {
        const float f = __builtin_amdgcn_exp2f(sm[x] - M);
        L = fmaf(sl[x], f, L);
        z = fmaf(so[x][threadIdx.x], f, z);
      }
      a.o[row * HD + threadIdx.x] = f2bf(L == 0.f ? 0.f : z / L);
    }
    __syncthreads();
  }
}

StepArgs args(const gdr_kv &c, const gdr_attn_step &p, uint16_t *o, void *ws, const StepPlan &plan) {
  float *part = static_cast<float *>(ws);
  return StepArgs{p.q, c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.page_table, p.lens, p.cu_seqlens, o, part,
                  part + (int64_t)p.T * p.H_q * plan.splits * HD, p.q_stride, p.T, c.N, p.H_q, c.H_kv, p.H_q / c.H_kv, c.n_pages,
                  __builtin_ctz((unsigned)c.page), c.n_pages > 0 ? c.max_pages : 0,
                  p.window < (int64_t)c.max_pages * c.page ? p.window : 0, plan.splits, plan.row_tiles,
                  p.scale * LOG2E};
}

}  // namespace

hipError_t launch_attn_step(const gdr_kv &c, const gdr_attn_step &p, uint16_t *o, void *ws, const StepPlan &plan, hipStream_t stream) {
  if (p.T == 0 || c.N == 0) return hipSuccess;
  const StepArgs a = args(c, p, o, ws, plan);
  if (p.cu_seqlens) attn_step_kernel<true><<<dim3((uint32_t)plan.blocks), 256, 0, stream>>>(a);
  else attn_step_kernel<false><<<dim3((uint32_t)plan.blocks), 256, 0, stream>>>(a);
  return hipGetLastError();
}
hipError_t launch_attn_step_join(const gdr_kv &c, const gdr_attn_step &p, uint16_t *o, void *ws, const StepPlan &plan,
                                 hipStream_t stream) {
  if (p.T == 0 || c.N == 0) return hipSuccess;
  attn_step_join_kernel<<<dim3((uint32_t)((int64_t)c.N * p.H_q)), 256, 0, stream>>>(args(c, p, o, ws, plan));
  return hipGetLastError();
}

}  // namespace gdr
