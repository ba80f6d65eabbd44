// Short causal depthwise convolution over packed documents, with bias and SiLU.
//
//   z[t,c] = b[c] + sum_{i<W} w[c,i] X[t-(W-1)+i, c],     y = z or z sigma(z)
//
// X is the document preceded by W-1 carried-in rows (s0, or zeros).  Backward,
// with dz = dy act'(z) and dz = 0 past the document's end:
//   dX[s] = sum_{i<W} w[c,i] dz[s+(W-1)-i] (+ dst on the last W-1 rows of X)
//   dw[c,i] = sum_t dz[t] X[t-(W-1)+i],   db = sum_t dz[t]
// dX before the document's first row is ds0.
//
// Bound by HBM: about 17 (forward) and 34 (backward) lane operations a value against
// 4 and 6 bytes keep the vector units 0.6 and 0.8 busy.  W = 4, SiLU, bf16, on a card
// that copies 5.1 TB/s: forward [261392, 2048] 362 us, 6.0 TB/s; backward [241817,
// 6144] 1781 us, 5.2 TB/s, each with the 7 % that run starts read again.  Nothing is
// kept for the backward, since z costs less to form again than to read.
#include "gdr_layer.h"
#include "gdr_vec.h"

namespace gdr {
namespace {

struct ConvArgs {
  const void *x, *w, *b, *s0;
  const int32_t *table;
  int N, NC, C;
  int64_t xs;
  bool wbf;
  int lx, ly, nchb;
};

template <int VEC, int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c, float (&w)[W][VEC], float (&b)[VEC]) {
  if constexpr (VEC == 1) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i][0] = ld_param(a.w, (int64_t)c * W + i, a.wbf);
    b[0] = a.b ? ld_param(a.b, c, a.wbf) : 0.f;
  } else {
    if (a.wbf) {
      Raw<u16, VEC * W> r;
      r.load(static_cast<const u16 *>(a.w) + (int64_t)c * W);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
#pragma unroll
        for (int i = 0; i < W; ++i) w[i][e] = r.get(e * W + i);
    } else {
      Raw<float, VEC * W> r;
      r.load(static_cast<const float *>(a.w) + (int64_t)c * W);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
#pragma unroll
        for (int i = 0; i < W; ++i) w[i][e] = r.get(e * W + i);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) b[e] = a.b ? ld_param(a.b, c + e, a.wbf) : 0.f;
  }
}

// Row `pos` (-(W-1) <= pos < 0) of the carried-in rows of document `doc`.
template <class T, int VEC>
__device__ __forceinline__ void load_carried(const ConvArgs &a, int W, int doc, int pos, int c, Raw<T, VEC> &r) {
  if (a.s0) r.load(static_cast<const T *>(a.s0) + ((int64_t)doc * (W - 1) + (W - 1) + pos) * a.C + c);
  else r.zero();
}

// First token and token count of a document, from its chunks.
__device__ __forceinline__ void doc_span(const ChunkTable &tb, int doc, int &start, int &len) {
  const int c0 = tb.doc_ptr[doc], c1 = tb.doc_ptr[doc + 1];
  start = c0 < c1 ? tb.start[c0] : 0;
  len = c0 < c1 ? tb.start[c1 - 1] + tb.len[c1 - 1] - start : 0;
}

// The taps' products: z for one row, `win` holding the W-1 rows before it.
template <int VEC, int W>
__device__ __forceinline__ void taps(const float (&w)[W][VEC], const float (&b)[VEC], const float (&win)[W - 1][VEC],
                                     const float (&x)[VEC], float (&z)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float s = b[e];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) s = fmaf(w[i][e], win[i][e], s);
    z[e] = fmaf(w[W - 1][e], x[e], s);
  }
}
template <int VEC, int D>
__device__ __forceinline__ void push(float (&win)[D][VEC], const float (&x)[VEC]) {
#pragma unroll
  for (int i = 0; i + 1 < D; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) win[i][e] = win[i + 1][e];
#pragma unroll
  for (int e = 0; e < VEC; ++e) win[D - 1][e] = x[e];
}

// Blocks are dealt to the 8 XCDs in turn.  Within groups of 64 blocks the order is
// changed so that 8 neighbours, whose runs read each other's last rows, share an
// XCD's cache.  Of `total` blocks, those past the last whole group keep their place.
__device__ __forceinline__ int neighbours_on_one_xcd(int b, int total) {
  const int in = b & 63;
  return (b | 63) < total ? (b & ~63) + (in & 7) * 8 + (in >> 3) : b;
}

// Forward: a thread takes R consecutive tokens of one chunk.  Blocks past the
// `nrb` row blocks write the final rows st instead, LY documents each.
template <class T, int VEC, int W, bool SILU, bool UNI, int R>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a, int nrb, T *__restrict__ y, int64_t ys,
                                                       T *__restrict__ st) {
  const int tx = threadIdx.x % a.lx, ty = set_of<UNI>(a.lx);
  const int blk = neighbours_on_one_xcd(blockIdx.x, nrb * a.nchb);
  const int chb = blk % a.nchb, rb = blk / a.nchb;
  const int group = chb * a.lx + tx;
  if (ty >= a.ly || group >= (a.C + VEC - 1) / VEC) return;
  const int c = first_channel<VEC>(group, a.C);
  const ChunkTable tb(a.table, a.NC, a.N);
  const T *__restrict__ x = static_cast<const T *>(a.x);

  if (rb >= nrb) {
    const int doc = (rb - nrb) * a.ly + ty;
    if (doc >= a.N) return;
    int start, len;
    doc_span(tb, doc, start, len);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int pos = len - (W - 1) + j;
      Raw<T, VEC> r;
      if (pos >= 0) r.load(x + (int64_t)(start + pos) * a.xs + c);
      else load_carried<T, VEC>(a, W, doc, pos, c, r);
      r.store(st + ((int64_t)doc * (W - 1) + j) * a.C + c);
    }
    return;
  }

  constexpr int RUNS = 64 / R;
  const int run = rb * a.ly + ty, chunk = run / RUNS, sub = run % RUNS;
  if (chunk >= a.NC) return;
  const int len = min(R, tb.len[chunk] - sub * R);
  if (len <= 0) return;
  const int start = tb.start[chunk] + sub * R, doc = tb.doc[chunk];
  const int pos = (chunk - tb.doc_ptr[doc]) * 64 + sub * R;  // of the run's first token in its document

  Raw<T, VEC> in[R], hist[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int p = pos - (W - 1) + j;
    if (p >= 0) hist[j].load(x + (int64_t)(start - (W - 1) + j) * a.xs + c);
    else load_carried<T, VEC>(a, W, doc, p, c, hist[j]);
  }
  const T *__restrict__ px = x + (int64_t)start * a.xs;
  T *__restrict__ py = y + (int64_t)start * ys;
  // Whole runs go without a test per row, which keeps their loads and stores in one
  // stretch ([261392, 2048] 380 us, with the tests 399).
  auto all_rows = [&](auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
    for (int t = 0; t < R; ++t) {
      in[t].load(px + c);
      if (WHOLE || t < len - 1) px += a.xs;  // past the end: the last row again
    }
    float w[W][VEC], b[VEC], win[W - 1][VEC];
    load_taps<VEC, W>(a, c, w, b);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) win[j][e] = hist[j].get(e);
#pragma unroll
    for (int t = 0; t < R; ++t) {
      float xv[VEC], z[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) xv[e] = in[t].get(e);
      taps<VEC, W>(w, b, win, xv, z);
      if constexpr (SILU) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) z[e] *= sigmoid<sizeof(T) == 4>(z[e]);
      }
      Raw<T, VEC> out;
      out.set(z);
      if (WHOLE || t < len) out.store(py + c);
      py += ys;
      push<VEC, W - 1>(win, xv);
    }
  };
  if (len == R) all_rows(std::true_type());
  else all_rows(std::false_type());
}

// dz = dy act'(z).
template <bool EXACT, bool SILU>
__device__ __forceinline__ float act_grad(float dy, float z) {
  if constexpr (!SILU) return dy;
  const float s = sigmoid<EXACT>(z);
  return dy * (s * fmaf(z, 1.f - s, 1.f));
}

// Backward: the workers take the runs of R tokens in turn, keeping the last W-1 rows
// of x and dz in registers; z is formed again from x.  It reads W-1 rows past
// each run's end, whose dz reach back into the run.  The parameter terms stay in
// registers over all the worker's runs and leave as one partial row per block.
// Blocks past the `nwb` worker blocks form ds0, LY documents each.
template <class T, int VEC, int W, bool SILU, bool UNI>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a, int R, int nwb, int workers, const T *__restrict__ dy, int64_t ds,
                                                       const T *__restrict__ dst, T *__restrict__ dx, int64_t xs_out,
                                                       T *__restrict__ ds0, float *__restrict__ partial) {
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int B = 4;  // tokens per batch of loads; the next batch is in flight during one's arithmetic
  const int RUNS = 64 / R;
  const int tx = threadIdx.x % a.lx, ty = set_of<UNI>(a.lx);
  const int chb = blockIdx.x % a.nchb, wb = blockIdx.x / a.nchb;
  const int group = chb * a.lx + tx, groups = (a.C + VEC - 1) / VEC;
  const bool live = ty < a.ly && group < groups;
  const int c = first_channel<VEC>(min(group, groups - 1), a.C);
  const ChunkTable tb(a.table, a.NC, a.N);
  const T *__restrict__ x = static_cast<const T *>(a.x);
  float w[W][VEC], b[VEC];
  load_taps<VEC, W>(a, c, w, b);

  if (wb >= nwb) {
    const int doc = (wb - nwb) * a.ly + ty;
    if (!live || doc >= a.N) return;
    int start, len;
    doc_span(tb, doc, start, len);
    float win[W - 1][VEC], acc[W - 1][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Raw<T, VEC> r;
      load_carried<T, VEC>(a, W, doc, j - (W - 1), c, r);
#pragma unroll
      for (int e = 0; e < VEC; ++e) win[j][e] = r.get(e), acc[j][e] = 0.f;
      if (dst && j - len >= 0) {  // a document shorter than the history hands it on
        Raw<T, VEC> d;
        d.load(dst + ((int64_t)doc * (W - 1) + j - len) * a.C + c);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = d.get(e);
      }
    }
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
      if (t >= len) break;
      Raw<T, VEC> rx, rd;
      rx.load(x + (int64_t)(start + t) * a.xs + c);
      rd.load(dy + (int64_t)(start + t) * ds + c);
      float xv[VEC], z[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) xv[e] = rx.get(e);
      taps<VEC, W>(w, b, win, xv, z);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float dz = act_grad<EXACT, SILU>(rd.get(e), z[e]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
          if (j >= t) acc[j][e] = fmaf(w[j - t < 0 ? 0 : j - t][e], dz, acc[j][e]);
      }
      push<VEC, W - 1>(win, xv);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Raw<T, VEC> r;
      r.set(acc[j]);
      r.store(ds0 + ((int64_t)doc * (W - 1) + j) * a.C + c);
    }
    return;
  }

  const int worker = wb * a.ly + ty;
  const int64_t runs = (int64_t)a.NC * RUNS;
  float dw[W][VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) dw[i][e] = 0.f;
  }
  for (int run = live ? worker : (int)runs; run < (int)runs; run += workers) {
    const int chunk = run / RUNS, sub = run % RUNS;
    const int len = min(R, tb.len[chunk] - sub * R);
    if (len <= 0) continue;
    const int start = tb.start[chunk] + sub * R, doc = tb.doc[chunk];
    const int pos = (chunk - tb.doc_ptr[doc]) * 64 + sub * R;
    const int lastc = tb.doc_ptr[doc + 1] - 1;
    const int left = (lastc - chunk) * 64 + tb.len[lastc] - sub * R;  // tokens of the document from `start` on
    const int end = min(len + W - 1, left);                           // rows whose dz reach into the run
    float win[W - 1][VEC], dzw[W - 1][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int p = pos - (W - 1) + j;
      Raw<T, VEC> r;
      if (p >= 0) r.load(x + (int64_t)(start - (W - 1) + j) * a.xs + c);
      else load_carried<T, VEC>(a, W, doc, p, c, r);
#pragma unroll
      for (int e = 0; e < VEC; ++e) win[j][e] = r.get(e), dzw[j][e] = 0.f;
    }
    const T *__restrict__ px = x + (int64_t)start * a.xs;
    const T *__restrict__ pd = dy + (int64_t)start * ds;
    T *__restrict__ po = dx + (int64_t)start * xs_out;
    struct Batch {
      Raw<T, VEC> x[B], d[B];
    };
    auto fetch = [&](int t0, Batch &n) {
#pragma unroll
      for (int i = 0; i < B; ++i) {
        n.x[i].load(px + c);
        n.d[i].load(pd + c);
        if (t0 + i < end - 1) px += a.xs, pd += ds;  // past the end: the last row again
      }
    };
    auto walk = [&](int t0, const Batch &b4) {
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int t = t0 + i;
        float xv[VEC], z[VEC], dz[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) xv[e] = b4.x[i].get(e);
        taps<VEC, W>(w, b, win, xv, z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) dz[e] = act_grad<EXACT, SILU>(b4.d[i].get(e), z[e]);
        if (t >= end) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) dz[e] = 0.f;
        }
        if (t < len) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            db[e] += dz[e];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(dz[e], win[j][e], dw[j][e]);
            dw[W - 1][e] = fmaf(dz[e], xv[e], dw[W - 1][e]);
          }
        }
        const int s = t - (W - 1);  // dX[s]: dz[s .. s + W - 1] are dzw and dz
        if (s >= 0 && s < len) {
          float g[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            g[e] = w[0][e] * dz[e];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) g[e] = fmaf(w[W - 1 - j][e], dzw[j][e], g[e]);
          }
          const int q = s - (left - (W - 1));
          if (dst && q >= 0) {
            Raw<T, VEC> d;
            d.load(dst + ((int64_t)doc * (W - 1) + q) * a.C + c);
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[e] += d.get(e);
          }
          Raw<T, VEC> out;
          out.set(g);
          out.store(po + c);
          po += xs_out;
        }
        push<VEC, W - 1>(win, xv);
        push<VEC, W - 1>(dzw, dz);
      }
    };
    // two batches in turn, so that neither is copied ([241817, 6144] 1777 us, with one
    // and its copy 1827)
    const int stop = len + W - 1;
    Batch even, odd;
    fetch(0, even);
    for (int t0 = 0; t0 < stop; t0 += 2 * B) {
      if (t0 + B < stop) fetch(t0 + B, odd);
      walk(t0, even);
      if (t0 + B >= stop) break;
      if (t0 + 2 * B < stop) fetch(t0 + 2 * B, even);
      walk(t0 + B, odd);
    }
  }
  __shared__ float lds[(W + 1) * VEC * 256];
  float v[(W + 1) * VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i * VEC + e] = dw[i][e];
    v[W * VEC + e] = db[e];
  }
  add_sets<(W + 1) * VEC>(v, lds, tx, ty, a.lx, a.ly);
  if (!live || ty != 0) return;
  float *p = partial + (int64_t)wb * (W + 1) * a.C + c;
#pragma unroll
  for (int i = 0; i <= W; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) p[(int64_t)i * a.C + e] = v[i * VEC + e];
}

// One token per sequence ([64, 10240] 4.4 us, the latency of slot, state and store):
// the W-1 rows of the sequence's slot and the new row give
// y; the slot keeps the last W-1 rows.  Rows whose slot lies outside the pool are
// left alone.
template <class T, int VEC, int W, bool SILU>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a, T *__restrict__ y, int64_t ys, T *state,
                                                        const int32_t *__restrict__ slots, int n_slots) {
  const int tx = threadIdx.x % a.lx, ty = threadIdx.x / a.lx;
  const int chb = blockIdx.x % a.nchb, rb = blockIdx.x / a.nchb;
  const int group = chb * a.lx + tx, row = rb * a.ly + ty;
  if (ty >= a.ly || group >= a.C / VEC || row >= a.N) return;
  const int slot = slots ? slots[row] : row;
  if (slot < 0 || slot >= n_slots) return;
  const int c = group * VEC;
  T *s = state + (int64_t)slot * (W - 1) * a.C + c;
  Raw<T, VEC> in, hist[W - 1];
  in.load(static_cast<const T *>(a.x) + (int64_t)row * a.xs + c);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) hist[j].load(s + (int64_t)j * a.C);
  float w[W][VEC], b[VEC], win[W - 1][VEC], xv[VEC], z[VEC];
  load_taps<VEC, W>(a, c, w, b);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    xv[e] = in.get(e);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j][e] = hist[j].get(e);
  }
  taps<VEC, W>(w, b, win, xv, z);
  if constexpr (SILU) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) z[e] *= sigmoid<sizeof(T) == 4>(z[e]);
  }
  Raw<T, VEC> out;
  out.set(z);
  out.store(y + (int64_t)row * ys + c);
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j) hist[j + 1].store(s + (int64_t)j * a.C);
  in.store(s + (int64_t)(W - 2) * a.C);
}

ConvArgs args_of(const gdr_conv &p, const Lanes &l) {
  ConvArgs a{};
  a.x = p.x; a.w = p.weight; a.b = p.bias; a.s0 = p.s0;
  a.table = p.chunk_table;
  a.N = p.N; a.NC = p.n_chunks; a.C = p.C;
  a.xs = p.x_stride;
  a.wbf = p.w_dtype == GDR_BF16;
  a.lx = l.lx; a.ly = l.ly; a.nchb = l.nchb;
  return a;
}

// Calls f(type tag, VEC, W, SILU, UNI) with the compile-time values of the problem.
template <int N>
using Int = std::integral_constant<int, N>;
template <class T, int VEC, bool SILU, bool UNI, class F>
hipError_t with_width(int W, F f) {
  const T t{};
  const Int<VEC> v;
  const Int<SILU> s;
  const Int<UNI> u;
  switch (W) {
    case 2: return f(t, v, Int<2>(), s, u);
    case 3: return f(t, v, Int<3>(), s, u);
    case 4: return f(t, v, Int<4>(), s, u);
    case 5: return f(t, v, Int<5>(), s, u);
    case 6: return f(t, v, Int<6>(), s, u);
    case 7: return f(t, v, Int<7>(), s, u);
    case 8: return f(t, v, Int<8>(), s, u);
    default: return hipErrorInvalidValue;
  }
}
template <class T, int VEC, class F>
hipError_t with_flags(const gdr_conv &p, const Lanes &l, F f) {
  const bool silu = p.activation == GDR_ACT_SILU;
  if constexpr (VEC > 1) {
    if (l.uniform) return silu ? with_width<T, VEC, true, true>(p.W, f) : with_width<T, VEC, false, true>(p.W, f);
  }
  return silu ? with_width<T, VEC, true, false>(p.W, f) : with_width<T, VEC, false, false>(p.W, f);
}
template <int BF_VEC, class F>
hipError_t with_types(const gdr_conv &p, int vec, const Lanes &l, F f) {
  if (p.dtype == GDR_BF16) return vec == 1 ? with_flags<u16, 1>(p, l, f) : with_flags<u16, BF_VEC>(p, l, f);
  return vec == 1 ? with_flags<float, 1>(p, l, f) : with_flags<float, 4>(p, l, f);
}

}  // namespace

hipError_t launch_conv_fwd(const gdr_conv &p, void *y, int64_t y_stride, void *st, hipStream_t stream) {
  const ConvFwdPlan plan = conv_fwd_plan(p, st != nullptr);
  const Lanes &l = plan.lanes;
  const ConvArgs a = args_of(p, l);
  const unsigned blocks = (unsigned)(plan.rows() * l.nchb);
  if (blocks == 0) return hipSuccess;
  return with_types<8>(p, plan.vec, l, [&](auto t, auto v, auto w, auto s, auto u) {
    using T = decltype(t);
    conv_fwd_kernel<T, decltype(v)::value, decltype(w)::value, decltype(s)::value, decltype(u)::value,
                    conv_fwd_run(decltype(w)::value)>
        <<<blocks, l.threads, 0, stream>>>(a, (int)plan.runs, static_cast<T *>(y), y_stride, static_cast<T *>(st));
    return hipGetLastError();
  });
}

hipError_t launch_conv_bwd(const gdr_conv &p, const void *dy, int64_t dy_stride, const void *dst, void *dx,
                           int64_t dx_stride, void *ds0, float *partial, hipStream_t stream) {
  const int vec = conv_bwd_vec(p.C);
  const ConvBwdPlan plan = conv_bwd_plan(p.n_chunks, p.C);
  const Lanes &l = plan.lanes;
  const ConvArgs a = args_of(p, l);
  const int nwb = plan.rows();
  const unsigned blocks = (unsigned)((nwb + plan.docs(p.N, ds0 != nullptr)) * l.nchb);
  if (blocks == 0) return hipSuccess;
  return with_types<4>(p, vec, l, [&](auto t, auto v, auto w, auto s, auto u) {
    using T = decltype(t);
    conv_bwd_kernel<T, decltype(v)::value, decltype(w)::value, decltype(s)::value, decltype(u)::value>
        <<<blocks, l.threads, 0, stream>>>(a, plan.run, nwb, plan.workers, static_cast<const T *>(dy), dy_stride,
                                                     static_cast<const T *>(dst), static_cast<T *>(dx), dx_stride,
                                                     static_cast<T *>(ds0), partial);
    return hipGetLastError();
  });
}

hipError_t launch_conv_step(const gdr_conv &p, void *y, int64_t y_stride, void *state, const int32_t *slots,
                            int32_t n_slots, hipStream_t stream) {
  const ConvStepPlan plan = conv_step_plan(p);
  const Lanes &l = plan.lanes;
  const ConvArgs a = args_of(p, l);
  const unsigned blocks = (unsigned)(plan.rows * l.nchb);
  if (blocks == 0) return hipSuccess;
  return with_types<8>(p, plan.vec, l, [&](auto t, auto v, auto w, auto s, auto) {
    using T = decltype(t);
    conv_step_kernel<T, decltype(v)::value, decltype(w)::value, decltype(s)::value><<<blocks, l.threads, 0, stream>>>(
        a, static_cast<T *>(y), y_stride, static_cast<T *>(state), slots, n_slots);
    return hipGetLastError();
  });
}

}  // namespace gdr
