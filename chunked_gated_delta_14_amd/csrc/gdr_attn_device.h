// What the attention kernels share: 32x32x16 matrix products, tiles of 64 rows of 128
// channels in LDS, and the copies that fill them.
//
// v_mfma_f32_32x32x16_bf16, lane = 32 h + lr:
//   A (32 x 16): lane holds A[lr][k(h, j)], j = 0..7;   B (16 x 32): B[k(h, j)][lr]
//   D (32 x 32): register i of the lane holds D[8 (i >> 2) + 4 h + (i & 3)][lr]
// A and B pair equal (h, j), so any order k of the 16 terms does if both take it.  Two do:
//   kstd(h, j) = 8 h + j: operands that lie along the reduction in memory;
//   kacc(h, j) = 4 h + (j & 3) + 8 (j >> 2): a lane's registers 8 s .. 8 s + 7 of a D tile,
//   rounded to bf16, are the B operand of the product over that tile's rows 16 s .. +15,
//   so probabilities go from one product into the next without leaving the lane.
#pragma once

#include "gdr_attn.h"
#include "gdr_device.h"

namespace gdr {

typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zero16() {
  return f32x16{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
}

// A tile in LDS: 64 rows of 256 bytes in 16 pieces of 16; piece c of row r lies at
// position c ^ swz(r).  swz takes 16 values over 16 rows, so a read of one piece of 16 rows (A operands
// along the rows) touches every bank once, and its high two bits 4 over 4 rows, so a read
// of four neighbouring pieces of 4 rows (half a transposed read) does too.  (With three high bits over
// 8 rows the transposed reads took twice as long: forward [32674, 16/4] 4.12 ms.)
constexpr int KT = 64;                 // rows of an LDS tile
constexpr int TILE_BYTES = KT * 2 * HD;
__device__ __forceinline__ int swz(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }

// Four copies of 1 KB each, straight from memory to LDS at m0 + 16 lane: rows
// 16 wave + 4 i + lane / 16 of the tile, i = 0..3, by a wavefront.  off[i] are the lanes' byte
// offsets from `base`.  In one block, as the compiler counts none of it: callers wait
// with vm_wait and a barrier before they read.
__device__ __forceinline__ void copy4(const void *base, const uint32_t (&off)[4], uint32_t lds_byte) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, %2\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %4, %2\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %5, %2\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %6, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds_byte), "s"(base), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3])
      : "memory", "scc");
}
// Offsets of a wavefront's rows of a tile of which rows 0 .. last are valid: the rows
// past them repeat the last (their scores are masked).  pitch: bytes a row, < 2^25.
__device__ __forceinline__ void copy_offsets(uint32_t (&off)[4], int wave, int lane, int last, uint32_t pitch) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 16 * wave + 4 * i + (lane >> 4);
    off[i] = (uint32_t)min(r, last) * pitch + (uint32_t)(((lane & 15) ^ swz(r)) * 16);
  }
}

// A lane's LDS byte address in a tile that begins at `tile`, from which its pieces for all
// kk, dt and steps follow by one exclusive or and a constant: the tile's bytes are
// 256 r + 16 (c ^ swz(r)), and kk or dt enter c as bits of their own.
__device__ __forceinline__ uint32_t row_base(uint32_t tile, int lane) {
  const int lr = lane & 31, h = lane >> 5;
  return tile + lr * 256 + (h ^ swz(lr)) * 16;
}
// ds_read_b64_tr_b16 hands lane 4 a + e of each 16 lanes element e of the 8-byte pieces that
// lanes a, 4 + a, 8 + a and 12 + a of them address.
__device__ __forceinline__ uint32_t col_base(uint32_t tile, int lane) {
  const int i = lane & 15, b = (lane >> 4) & 1, r = 4 * (lane >> 5) + (i >> 2);  // row within 8
  return tile + r * 256 + ((2 * b + ((i >> 1) & 1)) ^ swz(r)) * 16 + 8 * (i & 1);
}
// A operand along the rows: channels 16 kk + 8 h .. +7 of row 32 half + lr.
__device__ __forceinline__ bf16x8 row_frag(uint32_t base, int half, int kk) {
  return *(const __attribute__((address_space(3))) bf16x8 *)((base ^ (32u * kk)) + 8192u * half);
}
// A operand across the rows (the tile's transpose): channel 32 dt + lr of rows 16 step + kacc(h, j).
__device__ __forceinline__ bf16x8 col_frag(uint32_t base, int step, int dt) {
  typedef __attribute__((address_space(3))) bf16x4v *lds_v4;
  const uint32_t at = base ^ (64u * dt);
  const bf16x4v x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_v4)(at + 4096u * step));
  const bf16x4v y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_v4)((at ^ 32u) + 4096u * step + 2048u));
  const uint2 u = __builtin_bit_cast(uint2, x), v = __builtin_bit_cast(uint2, y);
  return __builtin_bit_cast(bf16x8, u32x4{u.x, u.y, v.x, v.y});
}
// Waits for every load, in a form that the compiler counts too: behind it, a loop holds no waits for
// registers loaded before it, which would wait for the loop's copies as well.
__device__ __forceinline__ void settle_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }
// A value as one that the compiler cannot keep from before: what follows from it is formed again here, for
// an instruction or two, where kept in a register it would be spilled.
__device__ __forceinline__ int afresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}
// Registers 8 s .. 8 s + 7 of a D tile as a B operand.
__device__ __forceinline__ bf16x8 acc_frag(const f32x16 &x, int s) {
  return __builtin_bit_cast(bf16x8, u32x4{pk2bf(x[8 * s], x[8 * s + 1]), pk2bf(x[8 * s + 2], x[8 * s + 3]),
                                          pk2bf(x[8 * s + 4], x[8 * s + 5]), pk2bf(x[8 * s + 6], x[8 * s + 7])});
}
// Largest or sum over the two lanes that share a column.
__device__ __forceinline__ float other_half(float x) {
  const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return __builtin_bit_cast(float, (threadIdx.x & 32) ? s[0] : s[1]);
}

// A transposed result (rows 32 dt + .. channels, column lr a row of the tensor), times f, to
// that row: 16 bytes a lane by swapping 8-byte pieces between the halves.
__device__ __forceinline__ void store_row(u16 *row, const f32x16 (&acc)[4], float f, int h, bool live) {
#pragma unroll
  for (int dt = 0; dt < 4; ++dt)
#pragma unroll
    for (int a = 0; a < 4; a += 2) {
      const f32x16 &x = acc[dt];
      const uint32_t x0 = pk2bf(x[4 * a] * f, x[4 * a + 1] * f), x1 = pk2bf(x[4 * a + 2] * f, x[4 * a + 3] * f);
      const uint32_t y0 = pk2bf(x[4 * a + 4] * f, x[4 * a + 5] * f), y1 = pk2bf(x[4 * a + 6] * f, x[4 * a + 7] * f);
      const auto s = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
      const auto t = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
      if (live) *reinterpret_cast<u32x4 *>(row + 32 * dt + 8 * (a + h)) = u32x4{s[0], t[0], s[1], t[1]};
    }
}

// The same in fp32, to a row of a part.
__device__ __forceinline__ void store_floats(float *row, const f32x16 (&acc)[4], int h) {
#pragma unroll
  for (int dt = 0; dt < 4; ++dt)
#pragma unroll
    for (int a = 0; a < 4; ++a)
      *reinterpret_cast<f32x4 *>(row + 32 * dt + 8 * a + 4 * h) =
          f32x4{acc[dt][4 * a], acc[dt][4 * a + 1], acc[dt][4 * a + 2], acc[dt][4 * a + 3]};
}

// The tile, its part and the head of a block, and the part's slot in the workspace.  Block ids go round the 8
// XCDs; where the heads divide by 8 an XCD takes neighbouring heads, which share keys in its L2.
struct Share {
  int tile, part, parts, head, slot;
  __device__ __forceinline__ Share(const int32_t *items, int b, int heads) {
    slot = tile = b / heads;
    const int r = b - tile * heads;
    head = (heads & 7) == 0 ? (r & 7) * (heads >> 3) + (r >> 3) : r;
    part = 0, parts = 1;
    if (items) {
      ConstI32 it = (ConstI32)(items + 2 * (int64_t)slot);
      tile = it[0];
      part = it[1] & 0xffff, parts = it[1] >> 16;
    }
  }
};

struct TileEntry {
  int row0, rows, other0, other, first, shift, begin, end;
  __device__ __forceinline__ TileEntry(const int32_t *table, int i) {
    ConstI32 e = (ConstI32)(table + (int64_t)i * ATT_ENTRY);
    row0 = e[0], rows = e[1], other0 = e[2], other = e[3], first = e[4], shift = e[5], begin = e[6], end = e[7];
  }
  // Steps of 64 of the other side's rows.
  __device__ __forceinline__ int steps() const { return begin < end ? (end - begin + KT - 1) / KT : 0; }
};

// The kernels that join parts: threads of a block, 16 to a row.
constexpr int ATT_JOIN = 512;

// Where a running maximum m starts: finite, so that a hidden score, -infinity, less it stays -infinity and gives a
// probability of 0, and below every score.  A probability's exponent S c - m is one fma and m a rounded product: what that
// rounding cuts off scales all of a row's probabilities, by 2^64 at most for scores of up to 2^30, which sums and quotient hold.
constexpr float LEAST = -3.402823466e38f;
constexpr float LOG2E = 1.44269504088896341f;
constexpr float LN2 = 0.693147180559945309f;

}  // namespace gdr
