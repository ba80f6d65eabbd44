// Sums of partial rows: the second step of the layer kernels' parameter gradients.
// A block takes 64 neighbouring columns with 16 sets of threads; set k adds rows
// k, k + 16, ... and the sets' sums are added in set order.  Bound by the read of
// the partials, a percent or two of what the first step moves.
#include "gdr_layer.h"
#include "gdr_vec.h"

namespace gdr {
namespace {

constexpr int PARTS = 16, COLS = 64;

// The sum of column `col` of [rows][M], returned to the threads of set 0.
__device__ __forceinline__ float column_sum(const float *__restrict__ partial, int rows, int M, int col, float *lds) {
  const int tx = threadIdx.x % COLS, part = threadIdx.x / COLS;
  float s = 0.f;
  if (col < M) {
#pragma unroll 8
    for (int r = part; r < rows; r += PARTS) s += partial[(int64_t)r * M + col];
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  if (part == 0)
    for (int k = 1; k < PARTS; ++k) s += lds[k * COLS + tx];
  return s;
}

__global__ __launch_bounds__(PARTS *COLS) void conv_sum_kernel(const float *__restrict__ partial, int rows, int C, int W,
                                                               float *__restrict__ dw, float *__restrict__ dbias) {
  __shared__ float lds[PARTS * COLS];
  const int M = (W + 1) * C, col = blockIdx.x * COLS + threadIdx.x % COLS;
  const float s = column_sum(partial, rows, M, col, lds);
  if (threadIdx.x >= COLS || col >= M) return;
  const int i = col / C, c = col - i * C;
  if (i == W) {
    if (dbias) dbias[c] = s;
  } else if (dw) {
    dw[(int64_t)c * W + i] = s;
  }
}

// Columns [0, C) are dbias, [C, 2C) the per-channel terms of da.
__global__ __launch_bounds__(PARTS *COLS) void gate_sum_kernel(const float *__restrict__ partial, int rows, int C, int D,
                                                               float *__restrict__ da, float *__restrict__ dbias) {
  __shared__ float lds[PARTS * COLS], head[COLS];
  const int tx = threadIdx.x % COLS, M = 2 * C;
  // a block takes whole heads: 64 heads of one channel, or one head of 128
  const int per = D == 1 ? 1 : 2, first = blockIdx.x * COLS * per;
  float a = 0.f;
  for (int j = 0; j < per; ++j) {
    const int c = first + j * COLS + tx;
    const float b = column_sum(partial, rows, M, c < C ? c : M, lds);
    if (dbias && threadIdx.x < COLS && c < C) dbias[c] = b;
    __syncthreads();
    a += column_sum(partial, rows, M, c < C ? C + c : M, lds);
    __syncthreads();
  }
  if (D == 1) {
    if (threadIdx.x < COLS && first + tx < C) da[first + tx] = a;
    return;
  }
  if (threadIdx.x < COLS) head[tx] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
    for (int k = 0; k < COLS; ++k) s += head[k];
    da[blockIdx.x] = s;
  }
}

__global__ __launch_bounds__(PARTS *COLS) void norm_sum_kernel(const float *__restrict__ partial, int rows, int D,
                                                               float *__restrict__ dw) {
  __shared__ float lds[PARTS * COLS];
  const int col = blockIdx.x * COLS + threadIdx.x % COLS;
  const float s = column_sum(partial, rows, D, col, lds);
  if (threadIdx.x < COLS && col < D) dw[col] = s;
}

}  // namespace

hipError_t launch_conv_sum(const float *partial, int rows, int C, int W, float *dw, float *dbias, hipStream_t stream) {
  conv_sum_kernel<<<((W + 1) * C + COLS - 1) / COLS, PARTS * COLS, 0, stream>>>(partial, rows, C, W, dw, dbias);
  return hipGetLastError();
}

hipError_t launch_gate_sum(const float *partial, int rows, int H, int D, float *da, float *dbias, hipStream_t stream) {
  const int blocks = D == 1 ? (H + COLS - 1) / COLS : H;
  gate_sum_kernel<<<blocks, PARTS * COLS, 0, stream>>>(partial, rows, H * D, D, da, dbias);
  return hipGetLastError();
}

hipError_t launch_norm_sum(const float *partial, int rows, int D, float *dw, hipStream_t stream) {
  norm_sum_kernel<<<(D + COLS - 1) / COLS, PARTS * COLS, 0, stream>>>(partial, rows, D, dw);
  return hipGetLastError();
}

}  // namespace gdr
