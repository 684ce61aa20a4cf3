// Device pieces shared by the attention kernels.
//
// Tiles of rows lie in LDS as they lie in memory, [row][channel], filled by
// LDS-DMA (16 bytes per lane, no registers).  Both operand forms of the matrix
// instructions come from such a tile:
//   row fragment  operand rows = tile rows, K = channels: a lane reads 16
//                 contiguous bytes (ds_read_b128)
//   col fragment  operand rows = channels, K = tile rows: bf16 by the
//                 transposing read (ds_read_b64_tr_b16), fp32 by single words
// A 32x32 product leaves in lane l (half = l / 32) the column l % 32 and, in
// register r, the row 8 (r / 4) + 4 half + r % 4.  Fed back as the second
// operand of the next product its registers 8 t .. 8 t + 7 are the K slots of
// step t; which tile row a slot stands for is free as long as the col fragment
// uses the same one, so no lane ever exchanges scores with another.
//
// 16-byte chunk c of tile row r sits at chunk c ^ swizzle(r).  LDS serves 256
// bytes a clock, sixteen lanes of a 16-byte read or thirty-two of an 8-byte one:
// sixteen lanes that read one chunk of sixteen successive rows, and two groups of
// sixteen that each read 32 bytes of four successive rows, then touch every bank
// once (no conflict counted in any kernel here).
#pragma once

#include <algorithm>

#include "sequences.h"
#include "tokens.h"

namespace st {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_void;
typedef __attribute__((address_space(3))) v4s* lds_v4s;

constexpr uint32_t kOobOffset = 0x80000000u;    // past every num_records used: reads zeros
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t attn_rsrc(const void* base, int64_t bytes) {
  const int64_t n = bytes < 0 ? 0 : (bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)n, 0x00020000);
}

// LDS chunk permutation of a tile row, by the row's pitch in bytes
template <int PITCH> __device__ __forceinline__ constexpr int swizzle(int r) {
  return PITCH == 64 || PITCH == 192    ? (r >> 2) & 3
         : PITCH == 128 || PITCH == 384 ? (((r >> 1) & 1) << 2) | ((r >> 2) & 3)
                                        : ((r & 3) << 2) | ((r >> 2) & 3);
}

// max, sum over the two halves of a wave (the two lanes of one column): the
// swap of a value with itself leaves the lower half's in one result and the
// upper half's in the other, in all lanes
__device__ __forceinline__ float half_max(float v) {
  const u32x2_t r = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const u32x2_t r = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }

template <class T> struct Mma;
template <> struct Mma<BF16> {
  using Row = bf16x8;                      // 8 channels of one row: K = 16 per product
  using Col = bf16x8;                      // 8 rows of one channel
  static __device__ __forceinline__ f32x16 rows(Row a, Row b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 cols(Col a, Col b, f32x16 c) { return rows(a, b, c); }
  // Registers 8 t .. 8 t + 7 of a product as the next one's second operand: p or
  // ds rounded to bf16, since the matrix cores multiply bf16 by bf16 (fp32 products
  // run at a ninth of their rate).  The sums stay fp32 and the softmax's denominator
  // adds the unrounded p; the outputs' error is 1.1 to 1.45 times that of one
  // rounding at the end.
  static __device__ __forceinline__ Col regs(const f32x16& s, int t) {
    const u32x4_t w = {pack_bf16(s[8 * t], s[8 * t + 1]), pack_bf16(s[8 * t + 2], s[8 * t + 3]),
                       pack_bf16(s[8 * t + 4], s[8 * t + 5]), pack_bf16(s[8 * t + 6], s[8 * t + 7])};
    return __builtin_bit_cast(Col, w);
  }
  static __device__ __forceinline__ Row load_row(const char* p) { return *reinterpret_cast<const Row*>(p); }
};
template <> struct Mma<F32> {
  using Row = f32x4_t;                     // 4 channels of one row: K = 8 over four products
  using Col = f32x8;
  static __device__ __forceinline__ f32x16 rows(Row a, Row b, f32x16 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ f32x16 cols(Col a, Col b, f32x16 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ Col regs(const f32x16& s, int t) {
    Col v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s[8 * t + i];
    return v;
  }
  static __device__ __forceinline__ Row load_row(const char* p) { return *reinterpret_cast<const Row*>(p); }
};

// A tile of ROWS rows of DP channels in LDS
template <class T, int DP, int ROWS, int NW> struct Tile {
  using M = Mma<T>;
  static constexpr int PITCH = DP * T::kSize;
  static constexpr int CH = PITCH / 16;                 // 16-byte chunks of a row
  static constexpr int BYTES = ROWS * PITCH;
  static constexpr int NI = BYTES / 1024 / NW;          // DMA transfers per wave
  static constexpr int SR = CH / 2;                     // row-fragment steps over the channels
  static constexpr int DB = DP / 32;                    // 32-channel blocks
  static_assert(BYTES % (1024 * NW) == 0, "whole transfers");

  // tile row and source byte within the row of this lane's transfer i
  static __device__ __forceinline__ int dma_row(int wave, int lane, int i) {
    return ((i * NW + wave) * 64 + lane) / CH;
  }
  static __device__ __forceinline__ int dma_byte(int wave, int lane, int i) {
    const int c = (i * NW + wave) * 64 + lane, row = c / CH;
    return ((c - row * CH) ^ swizzle<PITCH>(row)) * 16;
  }
  static __device__ __forceinline__ char* dma_dst(char* tile, int wave, int i) {
    return tile + (i * NW + wave) * 1024;
  }
  // row fragment: rows 32 b + l % 32, channels of step s
  static __device__ __forceinline__ typename M::Row row(const char* tile, int b, int s, int lane) {
    const int l = lane & 31, half = lane >> 5;
    return M::load_row(tile + (32 * b + l) * PITCH + (((2 * s + half) ^ swizzle<PITCH>(l)) << 4));
  }
  // col fragment: channels 32 db + l % 32, rows of step t (16 rows) of block b
  static __device__ __forceinline__ typename M::Col col(const char* tile, int b, int t, int db, int lane) {
    if constexpr (T::kSize == 2) {
      const int g16 = lane >> 4, s16 = lane & 15, half = lane >> 5;
      const int c = db * 4 + 2 * (g16 & 1) + ((s16 & 3) >> 1);
      v4s w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * t + 8 * i + 4 * half + (s16 >> 2);
        w[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_v4s)(tile + (32 * b + r) * PITCH + ((c ^ swizzle<PITCH>(r)) << 4) + (s16 & 1) * 8));
      }
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(w[0], w[1], 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int l = lane & 31, half = lane >> 5;
      f32x8 v;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = 8 * t + i, r = 8 * (k / 4) + 4 * half + k % 4;
        v[i] = *reinterpret_cast<const float*>(tile + (32 * b + r) * PITCH +
                                               (((db * 8 + (l >> 2)) ^ swizzle<PITCH>(r)) << 4) + (l & 3) * 4);
      }
      return v;
    }
  }
};

struct AttnTensor {
  char* p;
  int64_t t, h;             // token and head strides in bytes
};
struct AttnArgs {
  AttnTensor q, k, v, out, dout, dq, dk, dv;
  const AttnItem* items;
  const AttnJoin* joins;
  float* lse;               // [token][head]
  float* delta;             // [token][head]: sum over channels of dout * out
  float* part;              // partial results, [slot][kv head][tile row][padded dim]
  float* part2;             // second partial (dv), or log2 of the partial denominators
  Div31 by_group;
  int32_t group, kv_heads, heads, dim, causal;
  float scale, scale_log2;
};

// channel of register r (first of four) in this lane's half, block db
__device__ __forceinline__ int reg_channel(int db, int r4, int lane) { return 32 * db + 8 * r4 + 4 * (lane >> 5); }

// Writes a column's channels (a 32-channel block in the product's layout,
// times `f`) to a row of the output, in its type.
template <class T> __device__ __forceinline__ void store_block(char* row, const f32x16& v, float f, int db, int dim, int lane) {
#pragma unroll
  for (int r4 = 0; r4 < 4; ++r4) {
    const int c = reg_channel(db, r4, lane);
    if (c < dim) {
      const float x[4] = {v[4 * r4] * f, v[4 * r4 + 1] * f, v[4 * r4 + 2] * f, v[4 * r4 + 3] * f};
      store_vec<T, 4>(row + c * T::kSize, x);
    }
  }
}

// ---- host side

// Work items of one launch, a workgroup per item and key-value head: list by
// list, in as many launches as the items need.  launch(first item, workgroups)
template <class F> st_status attn_launches(size_t items, int kv_heads, int threads, F launch) {
  const size_t most = (size_t)(max_blocks(threads) / kv_heads);
  for (size_t i = 0; i < items; i += most) {
    const st_status r = launch(i, (int)(std::min(items - i, most) * kv_heads));
    if (r != ST_OK) return r;
  }
  return ST_OK;
}

struct AttnLaunch {
  AttnArgs a;
  hipStream_t st;
};
st_status attn_tensor(AttnTensor& out, const st_tokens* v, int64_t tokens, int heads, int dim, int esize, int span,
                      const char* name);
size_t attn_forward_bytes(const st_seqs* s);
size_t attn_backward_bytes(const st_seqs* s);

}  // namespace st
