// Private interface between the C-ABI layer (gdr_layer_api.cpp) and the kernels
// around the recurrence: the short convolution, the decay gate, the
// single-token recurrence and the norm with gate and residual.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gdr.h"

namespace gdr {

// Lane map of the kernels whose rows are C channels wide: a thread owns one group
// of `vec` neighbouring channels, LX threads span LX groups, LY sets of LX threads
// take LY different rows (or runs of rows), nchb blocks span all groups.  Wide rows
// take LX in whole wavefronts (`uniform`: a wavefront's rows are scalar values) unless
// that leaves more than a fifth of the lanes idle; others take LX as it comes, so
// narrow and odd rows leave few lanes idle.
struct Lanes {
  int lx, ly, nchb, threads;
  bool uniform;
};
inline Lanes lanes_for(int groups) {
  Lanes l;
  const int waves = (groups + 63) / 64;
  l.uniform = groups * 5 >= waves * 64 * 4;
  if (l.uniform) {
    // the widest of 4, 3, 2, 1 wavefronts that adds no idle wavefront
    int k = 4;
    while (waves % k) --k;
    l.nchb = waves / k;
    l.lx = 64 * k;
  } else {
    l.nchb = (groups + 255) / 256;
    l.lx = (groups + l.nchb - 1) / l.nchb;
  }
  l.ly = std::max(1, 256 / l.lx);
  l.threads = (l.lx * l.ly + 63) / 64 * 64;
  return l;
}
// Channels per thread: 16 bytes of a row, or single channels for rows narrower than that.
inline int vec_of(int channels, int dtype) {
  const int v = dtype == GDR_BF16 ? 8 : 4;
  return channels >= v ? v : 1;
}
inline int groups_of(int channels, int vec) { return (channels + vec - 1) / vec; }

// What one launch takes: HIP's grids hold fewer than 2^32 threads, and the kernels
// count their sets (`ly` to a block, each one row, run or document) with 32 bits.
inline bool one_launch(int64_t blocks, int threads) { return blocks * threads < (int64_t(1) << 32); }
inline bool one_launch(int64_t row_blocks, const Lanes &l) {
  return row_blocks * l.ly <= INT32_MAX && one_launch(row_blocks * l.nchb, l.threads);
}

// Row workers of the parameter-gradient sums: each set of LX threads adds its rows'
// terms in registers, a block adds its LY sets and leaves one partial row, and a
// second kernel adds the blocks' partials in a fixed order, so the sums do not
// depend on scheduling.  `target` threads fill the chip.  A multiple of LY.
inline int workers_for(int64_t rows, const Lanes &l, int64_t target) {
  const int64_t n = std::max<int64_t>(1, target / ((int64_t)l.nchb * l.lx));
  const int64_t w = std::min<int64_t>(std::max<int64_t>(rows, 0), n);
  return (int)((w + l.ly - 1) / l.ly * l.ly);
}

// Tokens per thread of the convolution's forward: short runs keep the registers few,
// but each reads W-1 rows again ([261392, 2048] W = 4 361 us with 8, 380 with 16, 394
// with 32; [30000, 6144] W = 8 213 us with 16, 267 with 8).
constexpr int conv_fwd_run(int W) { return W <= 4 ? 8 : 16; }

// The forward's blocks: `runs` of them take the chunks' runs, `docs` the final rows.
struct ConvFwdPlan {
  Lanes lanes;
  int vec;
  int64_t runs, docs;
  int64_t rows() const { return runs + docs; }
};
inline ConvFwdPlan conv_fwd_plan(const gdr_conv &p, bool st) {
  ConvFwdPlan r;
  r.vec = vec_of(p.C, p.dtype);
  r.lanes = lanes_for(groups_of(p.C, r.vec));
  const int64_t ly = r.lanes.ly;
  r.runs = ((int64_t)p.n_chunks * (64 / conv_fwd_run(p.W)) + ly - 1) / ly;
  r.docs = st ? (p.N + ly - 1) / ly : 0;
  return r;
}

// The single-token call: whole groups of channels, since the pool's rows are rewritten in place.
struct ConvStepPlan {
  Lanes lanes;
  int vec;
  int64_t rows;
};
inline ConvStepPlan conv_step_plan(const gdr_conv &p) {
  ConvStepPlan r;
  const int full = vec_of(p.C, p.dtype);
  r.vec = p.C % full == 0 ? full : 1;
  r.lanes = lanes_for(p.C / r.vec);
  r.lanes.uniform = false;
  r.rows = ((int64_t)p.N + r.lanes.ly - 1) / r.lanes.ly;
  return r;
}

// The convolution's backward: 4 channels per thread, runs of 64 tokens, or shorter
// ones where the chunks are too few to fill the chip (each run reads W-1 rows
// before and after itself again).  Measured with 8 channels per thread (twice the
// registers, half the wavefronts) and one run per chunk: [16792, 3832] W = 2 117 us,
// [512, 128] 19 us, [40000, 37] 27 us; as here 94, 14 and 16 us, large packs level.
struct ConvBwdPlan {
  Lanes lanes;
  int run, workers;
  int rows() const { return workers / lanes.ly; }  // partial rows, one per block
  // blocks of ds0, which follow those of the workers
  int64_t docs(int N, bool ds0) const { return ds0 ? ((int64_t)N + lanes.ly - 1) / lanes.ly : 0; }
};
inline int conv_bwd_vec(int C) { return C >= 4 ? 4 : 1; }
inline ConvBwdPlan conv_bwd_plan(int n_chunks, int C) {
  ConvBwdPlan p;
  p.lanes = lanes_for(groups_of(C, conv_bwd_vec(C)));
  const int64_t target = 131072, threads = (int64_t)n_chunks * p.lanes.nchb * p.lanes.lx;
  p.run = 64;
  while (p.run > 8 && threads * (64 / p.run) < target * 3 / 4) p.run /= 2;
  p.workers = workers_for((int64_t)n_chunks * (64 / p.run), p.lanes, target);
  return p;
}

// The gate's backward: 8 channels per thread for either type.  A block's partial row holds
// the C sums of dbias and the terms of da, one per channel or per thread.
constexpr int GATE_VEC = 8;
inline int gate_vec(int C) { return C >= GATE_VEC ? GATE_VEC : 1; }
inline Lanes gate_lanes(int C) { return lanes_for(groups_of(C, gate_vec(C))); }
// Workers: 131072 threads ([261392, 2048] 799 us; 65536 or 262144 threads 935 and 824),
// for rows narrower than a wavefront twice that ([241817, 48] 36.0 us; half of it 38.3,
// twice 36.0: their blocks add up more sets, so the partials stay few).
inline int gate_rows(int64_t T, int C) {
  const Lanes l = gate_lanes(C);
  return workers_for((T + 7) / 8, l, l.lx < 64 ? 262144 : 131072) / l.ly;
}
__host__ __device__ inline int gate_partial_row(int C, int D, int vec) { return C + (D == 1 ? C : C / vec); }

// The norm's backward: a worker is a block (gdr_norm.hip).  At most this many, by
// which the workspace is sized: at least 2048 values or 64 rows for each and fewer
// for wide rows, whose blocks are larger, so that the partial rows stay a small part
// of the traffic.  The launch takes norm_bwd_workers of them.
inline int norm_workers(int64_t rows, int D) {
  const int64_t n = std::max<int64_t>(rows * D / 2048, (rows + 63) / 64);
  return (int)std::min<int64_t>(n, std::min(1024, (1 << 22) / D));
}
int norm_bwd_workers(const gdr_norm &p);

hipError_t launch_conv_fwd(const gdr_conv &p, void *y, int64_t y_stride, void *st, hipStream_t stream);
hipError_t launch_conv_bwd(const gdr_conv &p, const void *dy, int64_t dy_stride, const void *dst, void *dx,
                           int64_t dx_stride, void *ds0, float *partial, hipStream_t stream);
hipError_t launch_conv_step(const gdr_conv &p, void *y, int64_t y_stride, void *state, const int32_t *slots,
                            int32_t n_slots, hipStream_t stream);
hipError_t launch_gate_fwd(const gdr_gate &p, float *g, hipStream_t stream);
hipError_t launch_gate_bwd(const gdr_gate &p, const float *dg, void *dx, int64_t dx_stride, float *partial, hipStream_t stream);
hipError_t launch_step(bool gdn, const gdr_step &p, uint16_t *o, hipStream_t stream);
hipError_t launch_norm_fwd(const gdr_norm &p, void *y, hipStream_t stream);
hipError_t launch_norm_bwd(const gdr_norm &p, const void *dy, const void *ds, void *dx, int64_t dx_stride, void *dgate,
                           int64_t dgate_stride, void *dres, float *partial, int workers, hipStream_t stream);

// Sums of `rows` partial rows, in a fixed order.  conv: partial [rows][W + 1][C] ->
// dw [C][W], dbias [C].  gate: partial [rows][gate_partial_row] -> dbias [H D] and da
// [H] (D is 1 or 128).  norm: partial [rows][D] -> dw.  A NULL dbias is skipped.
constexpr int SUM_PARTS = 32, SUM_COLS = 32;  // threads of a block: sets and columns
inline int64_t sum_blocks(int64_t columns) { return (columns + SUM_COLS - 1) / SUM_COLS; }
hipError_t launch_conv_sum(const float *partial, int rows, int C, int W, float *dw, float *dbias, hipStream_t stream);
hipError_t launch_gate_sum(const float *partial, int rows, int H, int D, float *da, float *dbias, hipStream_t stream);
hipError_t launch_norm_sum(const float *partial, int rows, int D, float *dw, hipStream_t stream);

}  // namespace gdr
