// Device pieces shared by the matrix products: operands in LDS or straight from
// memory, the matrix instructions, and the epilogue of a 32x32 block.
//
// A product's block has the output's channels along its rows and the output's
// rows (tokens) along its columns: lane l (half = l / 32) holds the token l % 32
// and, in register r, the channel 8 (r / 4) + 4 half + r % 4, so a token's 32
// channels lie in two lanes: bias, activation, residual and the 8-bit form's
// scale need at most one lane exchange, and stores run along the channels.
#pragma once

#include <algorithm>
#include <string>

#include "rows.h"

namespace st {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_void;
typedef __attribute__((address_space(3))) v4s* lds_v4s;

constexpr uint32_t kPastEnd = 0x80000000u;      // past every num_records used: reads zeros

// Chunk permutation of a tile row (16-byte chunks), by the row's pitch in bytes:
// sixteen lanes that read one chunk of sixteen successive rows, and two groups of
// sixteen that read 32 bytes of four successive rows, touch every bank once.
template <int PITCH> __device__ __forceinline__ constexpr int chunk_swizzle(int r) {
  return PITCH == 64 ? (r >> 2) & 3 : PITCH == 128 ? (((r >> 1) & 1) << 2) | ((r >> 2) & 3) : ((r & 3) << 2) | ((r >> 2) & 3);
}

// One operand's tile of a stage: 128 bytes of the contraction (a cache line) for W
// rows of the operand.  As it lies in memory: [W rows][128 bytes] where the
// contraction is contiguous (COL false), [128 / size contraction rows][W] where the
// operand's own rows are (COL true).
template <class T, bool COL, int W, int NW> struct Oper {
  static constexpr int KT = 128 / T::kSize;             // contraction steps of a stage
  static constexpr int PITCH = COL ? W * T::kSize : 128;
  static constexpr int CH = PITCH / 16;
  static constexpr int BYTES = W * 128;
  static constexpr int NI = BYTES / 1024 / NW;          // transfers of 1 KB per wave
  static_assert(BYTES % (1024 * NW) == 0, "whole transfers");
  // a wave's next transfer: so many rows on, and with the same chunks where the
  // permutation repeats by then
  static constexpr int ROWS_ON = 64 * NW / CH;
  static constexpr bool ALIKE = ROWS_ON % 16 == 0;

  static __device__ __forceinline__ int dma_row(int wave, int lane, int i) { return ((i * NW + wave) * 64 + lane) / CH; }
  static __device__ __forceinline__ int dma_byte(int wave, int lane, int i) {
    const int c = (i * NW + wave) * 64 + lane, row = c / CH;
    return ((c - row * CH) ^ chunk_swizzle<PITCH>(row)) * 16;
  }
  static __device__ __forceinline__ char* dma_dst(char* tile, int wave, int i) { return tile + (i * NW + wave) * 1024; }
  static __device__ __forceinline__ const char* at(const char* tile, int row, int chunk) {
    return tile + row * PITCH + ((chunk ^ chunk_swizzle<PITCH>(row)) << 4);
  }
};

// Fragments and products by type.  STEPS fragments cover a stage.
template <class T> struct Prod;
template <> struct Prod<BF16> {
  using Frag = bf16x8;                                  // 16 contraction steps, 8 a half
  static constexpr int STEPS = 4;
  template <bool COL, int W, int NW> static __device__ __forceinline__ Frag frag(const char* tile, int b, int s, int lane) {
    using O = Oper<BF16, COL, W, NW>;
    const int half = lane >> 5;
    if constexpr (!COL) {
      return *reinterpret_cast<const Frag*>(O::at(tile, 32 * b + (lane & 31), 2 * s + half));
    } else {
      // the transposing read: four contraction rows of sixteen operand rows a group
      const int g = lane >> 4, s16 = lane & 15;
      const int c = 4 * b + 2 * (g & 1) + ((s16 & 3) >> 1);
      v4s w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * s + 8 * half + 4 * i + (s16 >> 2);
        w[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(O::at(tile, r, c) + (s16 & 1) * 8));
      }
      return __builtin_bit_cast(Frag, __builtin_shufflevector(w[0], w[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  template <int S> static __device__ __forceinline__ f32x16 mul(const Frag& a, const Frag& b, f32x16 c, int, int) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Prod<F32> {
  using Frag = f32x4_t;                                 // 8 contraction steps, 4 a half, over four products
  static constexpr int STEPS = 4;
  template <bool COL, int W, int NW> static __device__ __forceinline__ Frag frag(const char* tile, int b, int s, int lane) {
    using O = Oper<F32, COL, W, NW>;
    const int l = lane & 31, half = lane >> 5;
    if constexpr (!COL) {
      return *reinterpret_cast<const Frag*>(O::at(tile, 32 * b + l, 2 * s + half));
    } else {
      Frag v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = *reinterpret_cast<const float*>(O::at(tile, 8 * s + 4 * half + i, 8 * b + (l >> 2)) + (l & 3) * 4);
      return v;
    }
  }
  template <int S> static __device__ __forceinline__ f32x16 mul(const Frag& a, const Frag& b, f32x16 c, int, int) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};
template <> struct Prod<MX8> {
  // 64 contraction steps: the instruction's layout has steps 16 half .. of either
  // block of 32 in a lane's first and second 16 bytes.  It takes the blocks' scales
  // from the lanes: block b's from half b.
  using Frag = i32x8;
  static constexpr int STEPS = 2;
  static __device__ __forceinline__ Frag join(u32x4_t lo, u32x4_t hi) {
    return Frag{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  }
  template <bool COL, int W, int NW> static __device__ __forceinline__ Frag frag(const char* tile, int b, int s, int lane) {
    static_assert(!COL, "blocks run along the contraction");
    using O = Oper<MX8, false, W, NW>;
    const int r = 32 * b + (lane & 31), half = lane >> 5;
    return join(*reinterpret_cast<const u32x4_t*>(O::at(tile, r, 4 * s + half)), *reinterpret_cast<const u32x4_t*>(O::at(tile, r, 4 * s + 2 + half)));
  }
  // sa, sb: scale bytes of this lane's row; block 2 S + half of the stage in byte 2 S.
  // Inside the instruction the products of eight steps are aligned to the largest of
  // them and cut 13 bits below its leading bit; beyond, the sums are fp32.  So outputs
  // in bf16 alone take it (16384 x 8192 x 2048: 2.2e-4 of the norm lands on a bf16
  // value's other side, against 1.7e-3 of the rounding itself); outputs in fp32, and in 8
  // bits, whose codes are to be those of the exact sums, take Prod<MX8X>.
  template <int S> static __device__ __forceinline__ f32x16 mul(const Frag& a, const Frag& b, f32x16 c, int sa, int sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 2 * S, sa, 2 * S, sb);
  }
};
// 8-bit operands whose products are summed in fp32 throughout: every value is
// widened to bf16 (which holds it exactly), at half the rate of the 8-bit instructions
// and, since every wave widens what it reads, a quarter of their products' speed.  A
// lane's 32 bytes are one block.
struct MX8X { static constexpr int kSize = 1; };
template <> struct Prod<MX8X> {
  struct Frag { bf16x8 v[4]; };
  static constexpr int STEPS = 2;
  template <bool COL, int W, int NW> static __device__ __forceinline__ i32x8 raw(const char* tile, int b, int s, int lane) {
    static_assert(!COL, "blocks run along the contraction");
    using O = Oper<MX8, false, W, NW>;
    const int r = 32 * b + (lane & 31), half = lane >> 5;
    return Prod<MX8>::join(*reinterpret_cast<const u32x4_t*>(O::at(tile, r, 4 * s + 2 * half)),
                           *reinterpret_cast<const u32x4_t*>(O::at(tile, r, 4 * s + 2 * half + 1)));
  }
  static __device__ __forceinline__ Frag widen(const i32x8& w, int scale) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
      mx_values((uint32_t)w[2 * i], scale, v);
      mx_values((uint32_t)w[2 * i + 1], scale, v + 4);
      const u32x4_t p = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
      f.v[i] = __builtin_bit_cast(bf16x8, p);
    }
    return f;
  }
  template <int S> static __device__ __forceinline__ f32x16 mul(const Frag& a, const Frag& b, f32x16 c, int, int) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
  }
};

// ------------------------------------------------------------- epilogue

struct Finish {
  Rows y, pre, res;                   // type -1: absent
  const float* bias;
  int32_t act;
  int32_t rows, cols;                 // of the output
};

__device__ __forceinline__ uint32_t swap_max(uint32_t v) {
  const u32x2_t r = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(v, v, false, false));
  return max(r[0], r[1]);
}

// A block of the epilogue: 32 tokens from m0 on (m0 + lane % 32) by 32 channels from
// n0 on, of which a lane holds 8 q + 4 half + e in v[4 q + e].  To memory and from it
// goes 16 bytes a lane, 64 contiguous bytes of a token (four lanes) at a time:
// swap_rows turns 32 tokens' first and second 32 bytes into 16 tokens' 64 and the
// other 16's (its own inverse).
__device__ __forceinline__ void swap_rows(u32x4_t& a, u32x4_t& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x2_t t = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(a[i], b[i], false, false));
    a[i] = t[0];
    b[i] = t[1];
  }
}
struct Spot {
  int64_t m;                          // of the first 16 tokens' register, of the second m + 16
  int at;                             // 16-byte piece of the token's 64
};
__device__ __forceinline__ Spot spot_of(int64_t m0, int lane) { return {m0 + (lane & 15), (lane >> 4 & 1) * 2 + (lane >> 5)}; }

// NT: outputs that pass the L2s by, larger than they are: operands stay there that
// are read again (16384 x 2048 x 8192 in bf16 482 -> 439 us, in 8 bits 283 -> 258).
template <bool NT> __device__ __forceinline__ void put16(char* p, u32x4_t w) {
  if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any*>(p));
  else *reinterpret_cast<u32x4_any*>(p) = w;
}

// A block to an output in bf16 or fp32
template <bool NT> __device__ __forceinline__ void put_float(const Rows& o, int64_t m0, int n0, int rows, int cols, int lane, const float (&v)[16]) {
  if (n0 + 32 <= cols) {
    const Spot at = spot_of(m0, lane);
    char* p = o.p + at.m * o.stride + (int64_t)n0 * (o.type == ST_F32 ? 4 : 2) + at.at * 16;
    const bool in0 = at.m < rows, in1 = at.m + 16 < rows;
    if (o.type == ST_BF16) {
      // the lanes of one token trade quads: 8 channels in a row each, twice
      u32x4_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t a0 = pack_bf16(v[8 * j], v[8 * j + 1]), a1 = pack_bf16(v[8 * j + 2], v[8 * j + 3]);
        const uint32_t b0 = pack_bf16(v[8 * j + 4], v[8 * j + 5]), b1 = pack_bf16(v[8 * j + 6], v[8 * j + 7]);
        const u32x2_t lo = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(a0, b0, false, false));
        const u32x2_t hi = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(a1, b1, false, false));
        w[j] = u32x4_t{lo[0], hi[0], lo[1], hi[1]};
      }
      swap_rows(w[0], w[1]);
      if (in0) put16<NT>(p, w[0]);
      if (in1) put16<NT>(p + 16 * o.stride, w[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u32x4_t w[2];
#pragma unroll
        for (int r = 0; r < 8; ++r) w[r / 4][r % 4] = __float_as_uint(v[8 * j + r]);
        swap_rows(w[0], w[1]);
        if (in0) put16<NT>(p + 64 * j, w[0]);
        if (in1) put16<NT>(p + 16 * o.stride + 64 * j, w[1]);
      }
    }
    return;
  }
  const int64_t m = m0 + (lane & 31);
  if (m >= rows) return;
  char* p = o.p + m * o.stride;
#pragma unroll
  for (int r = 0; r < 16; ++r) {                        // the last channels
    const int n = n0 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
    if (n < cols) {
      if (o.type == ST_F32) reinterpret_cast<float*>(p)[n] = v[r];
      else reinterpret_cast<uint16_t*>(p)[n] = (uint16_t)pack_bf16(v[r], 0.f);
    }
  }
}

// The same to an output in any type.
// (8-bit blocks are 32 bytes of a line, which the L2 joins: past it a product of 16384 x
// 2048 x 8192 in 8 bits took 311 us in place of 263)
template <bool NT> __device__ __forceinline__ void put_block(const Rows& o, int64_t m0, int n0, int rows, int cols, int lane, const float (&v)[16]) {
  if (o.type == ST_MX8) {
    const int half = lane >> 5;
    const int64_t m = m0 + (lane & 31);
    // (channels past the last are zeros here: they have no part in the scale)
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 16; ++r) top = max(top, mag_bits(v[r]));
    top = swap_max(top);
    uint32_t w[4];
    int s;
    if (__builtin_amdgcn_ballot_w64(top >= 0x7F800000u) == 0) {
      s = mx_scale(top);
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = mx_codes<false>(v + 4 * q, s);
    } else {                                            // NaN or infinity in some block of the wave
      top = 0;
#pragma unroll
      for (int r = 0; r < 16; ++r) top = max(top, mx_bits(v[r]));
      s = mx_scale(swap_max(top));
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = mx_codes<true>(v + 4 * q, s);
    }
    // the lanes of one token trade quads: 16 channels in a row each
    const u32x2_t a = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false));
    const u32x2_t b = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false));
    if (m >= rows) return;
    uint8_t* p = reinterpret_cast<uint8_t*>(o.p) + m * o.stride + n0;
    if (half == 0) o.scales[m * o.scale_stride + (n0 >> 5)] = (uint8_t)s;
    if (n0 + 32 <= cols) {
      *reinterpret_cast<u32x4_t*>(p + 16 * half) = u32x4_t{a[0], a[1], b[0], b[1]};
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int n = 8 * (r / 4) + 4 * half + r % 4;
        if (n0 + n < cols) p[n] = (uint8_t)(w[r / 4] >> (8 * (r % 4)));
      }
    }
    return;
  }
  put_float<NT>(o, m0, n0, rows, cols, lane, v);
}

// A block of the residual, as it lies: values come out of it when they are added,
// so that nothing waits for the loads before.
struct Res { u32x4_t w[4]; };
__device__ __forceinline__ void load_res(const Rows& o, int64_t m0, int n0, int rows, int cols, int lane, Res& t) {
  if (n0 + 32 <= cols) {
    const Spot at = spot_of(m0, lane);
    // (past the last token: its own again)
    const char* p = o.p + (int64_t)n0 * (o.type == ST_F32 ? 4 : 2) + at.at * 16;
    const char* p0 = p + min(at.m, (int64_t)rows - 1) * o.stride;
    const char* p1 = p + min(at.m + 16, (int64_t)rows - 1) * o.stride;
    t.w[0] = *reinterpret_cast<const u32x4_any*>(p0);
    t.w[1] = *reinterpret_cast<const u32x4_any*>(p1);
    if (o.type == ST_F32) {
      t.w[2] = *reinterpret_cast<const u32x4_any*>(p0 + 64);
      t.w[3] = *reinterpret_cast<const u32x4_any*>(p1 + 64);
    } else {
      t.w[2] = t.w[3] = u32x4_t{};
    }
    return;
  }
  const int64_t m = m0 + (lane & 31);
  const char* p = o.p + m * o.stride;
#pragma unroll
  for (int r = 0; r < 16; ++r) {                        // the last channels: as values
    const int n = n0 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
    float x = 0.f;
    if (m < rows && n < cols)
      x = o.type == ST_F32 ? reinterpret_cast<const float*>(p)[n] : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[n] << 16);
    t.w[r / 4][r % 4] = __float_as_uint(x);
  }
}
__device__ __forceinline__ void add_res(const Rows& o, int n0, int cols, Res& t, float (&v)[16]) {
  if (n0 + 32 <= cols) {
    swap_rows(t.w[0], t.w[1]);
    if (o.type == ST_BF16) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {                   // back to quads
          const u32x2_t u = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(t.w[j][i], t.w[j][2 + i], false, false));
          v[8 * j + 2 * i] += bf16_lo(u[0]);
          v[8 * j + 2 * i + 1] += bf16_hi(u[0]);
          v[8 * j + 4 + 2 * i] += bf16_lo(u[1]);
          v[8 * j + 4 + 2 * i + 1] += bf16_hi(u[1]);
        }
      return;
    }
    swap_rows(t.w[2], t.w[3]);
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) v[r] += __uint_as_float(t.w[r / 4][r % 4]);
}

// The bias of a block's channels, from memory
__device__ __forceinline__ void add_bias(const Finish& f, int n0, int lane, float (&v)[16]) {
  if (!f.bias) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int n = n0 + 8 * q + 4 * (lane >> 5);
    float t[4];
    load_some<F32, 4>(reinterpret_cast<const char*>(f.bias + n), f.cols - n, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * q + i] += t[i];
  }
}

// v = x w^T + bias: pre = v; y = act(v) + residual.  Every lane of the wave comes
// here; `t`: the block of the residual, if there is one.
// PLAIN: v alone, to bf16 or fp32.
template <bool PLAIN, bool NT = false> __device__ __forceinline__ void finish_block(const Finish& f, int64_t m0, int n0, int lane, Res& t, float (&v)[16]) {
  if (n0 >= f.cols) return;
  if constexpr (PLAIN) {
    put_float<NT>(f.y, m0, n0, f.rows, f.cols, lane, v);
    return;
  }
  if (f.pre.type >= 0) put_block<NT>(f.pre, m0, n0, f.rows, f.cols, lane, v);
  if (f.act != kActNone) activate(f.act, v);
  if (f.res.type >= 0) add_res(f.res, n0, f.cols, t, v);
  put_block<NT>(f.y, m0, n0, f.rows, f.cols, lane, v);
}

// ------------------------------------------------------------- launches

// One product: out[m][n] = sum over k of b[m][k] a[n][k] (a: the output's channel
// side, b: its row side; *_col: stored [k][.]), and what is done with it.
struct Product {
  Rows a, b;
  int type;                           // of both
  bool a_col, b_col;
  int64_t m, n, k;
  Finish f;
};
// Bytes of partial sums that a product of these sizes needs (0: none)
size_t product_bytes(int64_t m, int64_t n, int64_t k, int type, bool cols);
st_status product_launch(const Product& p, void* workspace, hipStream_t st);

}  // namespace st
