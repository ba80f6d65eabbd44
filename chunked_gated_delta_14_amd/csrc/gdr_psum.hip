// Sums of partial rows: the second step of the layer kernels' parameter gradients.
// A block takes 32 neighbouring columns (128-byte lines) with 32 sets of threads;
// set k adds rows k, k + 32, ... and the sets' sums are added in a fixed order.  Bound
// by the read of the partials, a percent or two of what the first step moves, and
// by its latency where they are few ([85, 5 x 6144] 6 us, [256, 2048] 5 us).
#include "gdr_layer.h"
#include "gdr_vec.h"

namespace gdr {
namespace {

constexpr int PARTS = SUM_PARTS, COLS = SUM_COLS;

// The sum of column `col` of [rows][M], in fp64 (the caller rounds it once), returned to the
// threads of set 0.  (fp32 sums take the same time and leave a quarter more error in
// the gradients of [32674, 512], [32674, 2048].)
__device__ __forceinline__ double column_sum(const float *__restrict__ partial, int rows, int M, int col, double *lds) {
  const int tx = threadIdx.x % COLS, part = threadIdx.x / COLS;
  double s = 0.;
  if (col < M) {
#pragma unroll 8
    for (int r = part; r < rows; r += PARTS) s += partial[(int64_t)r * M + col];
  }
  s += __shfl_xor(s, 32);  // sets 2k and 2k + 1 share a wavefront
  if ((part & 1) == 0) lds[(part >> 1) * COLS + tx] = s;
  __syncthreads();
  if (part == 0) {
#pragma unroll
    for (int k = 1; k < PARTS / 2; ++k) s += lds[k * COLS + tx];
  }
  return s;
}

__global__ __launch_bounds__(PARTS *COLS) void conv_sum_kernel(const float *__restrict__ partial, int rows, int C, int W,
                                                               float *__restrict__ dw, float *__restrict__ dbias) {
  __shared__ double lds[PARTS / 2 * COLS];
  const int M = (W + 1) * C, col = blockIdx.x * COLS + threadIdx.x % COLS;
  const double s = column_sum(partial, rows, M, col, lds);
  if (threadIdx.x >= COLS || col >= M) return;
  const int i = col / C, c = col - i * C;
  if (i == W) {
    if (dbias) dbias[c] = (float)s;
  } else {
    dw[(int64_t)c * W + i] = (float)s;
  }
}

// Blocks [0, nb) take the C columns of dbias, the others the columns of da, G of
// them to a head (G divides COLS).
__global__ __launch_bounds__(PARTS *COLS) void gate_sum_kernel(const float *__restrict__ partial, int rows, int C, int M, int G,
                                                               int nb, float *__restrict__ da, float *__restrict__ dbias) {
  __shared__ double lds[PARTS / 2 * COLS], head[COLS];
  const int tx = threadIdx.x % COLS;
  const bool is_a = (int)blockIdx.x >= nb;
  const int col = is_a ? C + ((int)blockIdx.x - nb) * COLS + tx : (int)blockIdx.x * COLS + tx;
  const int end = is_a ? M : C;
  const double s = column_sum(partial, rows, M, col < end ? col : M, lds);
  if (!is_a) {
    if (threadIdx.x < COLS && col < end) dbias[col] = (float)s;
    return;
  }
  if (threadIdx.x < COLS) head[tx] = s;
  __syncthreads();
  if (threadIdx.x < COLS && tx % G == 0 && col < end) {
    double a = 0.;
    for (int k = 0; k < G; ++k) a += head[tx + k];
    da[(col - C) / G] = (float)a;
  }
}

__global__ __launch_bounds__(PARTS *COLS) void norm_sum_kernel(const float *__restrict__ partial, int rows, int D,
                                                               float *__restrict__ dw) {
  __shared__ double lds[PARTS / 2 * COLS];
  const int col = blockIdx.x * COLS + threadIdx.x % COLS;
  const double s = column_sum(partial, rows, D, col, lds);
  if (threadIdx.x < COLS && col < D) dw[col] = (float)s;
}

int blocks_for(int64_t columns) { return (int)sum_blocks(columns); }

}  // namespace

hipError_t launch_conv_sum(const float *partial, int rows, int C, int W, float *dw, float *dbias, hipStream_t stream) {
  conv_sum_kernel<<<blocks_for((int64_t)(W + 1) * C), PARTS * COLS, 0, stream>>>(partial, rows, C, W, dw, dbias);
  return hipGetLastError();
}

hipError_t launch_gate_sum(const float *partial, int rows, int H, int D, float *da, float *dbias, hipStream_t stream) {
  const int C = H * D, vec = gate_vec(C), M = gate_partial_row(C, D, vec);
  const int nb = dbias ? blocks_for(C) : 0;
  gate_sum_kernel<<<nb + blocks_for(M - C), PARTS * COLS, 0, stream>>>(partial, rows, C, M, D == 1 ? 1 : D / vec, nb, da, dbias);
  return hipGetLastError();
}

hipError_t launch_norm_sum(const float *partial, int rows, int D, float *dw, hipStream_t stream) {
  norm_sum_kernel<<<blocks_for(D), PARTS * COLS, 0, stream>>>(partial, rows, D, dw);
  return hipGetLastError();
}

}  // namespace gdr
