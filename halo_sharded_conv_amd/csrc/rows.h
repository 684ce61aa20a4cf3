// Rows of channels: the operand form of the MLP branch's operators (matrix
// products, RMS norm, 8-bit activations).  Host checks of st_rows and the device
// helpers for loads at any alignment, the 8-bit form and the activations.
#pragma once

#include <string>
#include <type_traits>

#include "tokens.h"

namespace st {

// One operand as the kernels take it: strides in bytes
struct Rows {
  char* p;
  uint8_t* scales;
  int64_t stride, scale_stride;
  int32_t type;                       // ST_F32, ST_BF16, ST_MX8; -1: absent
};

inline int type_size(int type) { return type == ST_F32 ? 4 : type == ST_BF16 ? 2 : 1; }
constexpr int kMxBlock = ST_MX_BLOCK;
struct MX8 { static constexpr int kSize = 1; };

// Checks of one operand of `rows` rows of `channels` channels.  Rows are 16-byte
// aligned, or lie back to back (where one row's length is off that grid); `types`:
// the bits 1 << type that the call takes.
// (messages are put together on failure only: a call's checks take a fraction of a
// microsecond)
inline st_status rows_fail(st_status s, const char* call, const char* name, const char* what) {
  return fail(s, std::string(call) + ": " + name + ": " + what);
}
inline st_status rows_of(Rows& out, const st_rows* v, int64_t rows, int64_t channels, uint32_t types, const char* call, const char* name) {
  out = Rows{};
  out.type = -1;
  if (!v) return rows_fail(ST_ERR_INVALID_ARG, call, name, "NULL operand");
  if (v->type < 0 || v->type > ST_MX8 || !(types >> v->type & 1)) return rows_fail(ST_ERR_INVALID_ARG, call, name, "type not taken here");
  const int es = type_size(v->type);
  if (rows > 0 && !v->data) return rows_fail(ST_ERR_INVALID_ARG, call, name, "NULL data");
  if (!aligned16(v->data)) return rows_fail(ST_ERR_ALIGNMENT, call, name, "data not 16-byte aligned");
  const int64_t stride = rows > 1 ? v->stride : channels;     // (one row: its stride is not looked at)
  if (rows > 1 && (stride < channels || stride > (1ll << 40)))
    return rows_fail(ST_ERR_BAD_SHAPE, call, name, "row stride below the channels, or too large");
  if (rows > 1 && stride * es % 16 != 0 && (stride != channels || v->type == ST_MX8))
    return rows_fail(ST_ERR_ALIGNMENT, call, name, "row stride neither a multiple of 16 bytes nor the row's own length");
  out.p = static_cast<char*>(v->data);
  out.stride = stride * es;
  out.type = v->type;
  if (v->type == ST_MX8) {
    const int64_t blocks = (channels + kMxBlock - 1) / kMxBlock;
    if (rows > 0 && !v->scales) return rows_fail(ST_ERR_INVALID_ARG, call, name, "NULL scales");
    if (!aligned16(v->scales)) return rows_fail(ST_ERR_ALIGNMENT, call, name, "scales not 16-byte aligned");
    const int64_t ss = rows > 1 ? v->scale_stride : (blocks + 3) / 4 * 4;
    if (rows > 1 && (ss < blocks || ss > (1ll << 40))) return rows_fail(ST_ERR_BAD_SHAPE, call, name, "scale stride below the blocks, or too large");
    if (ss % 4 != 0) return rows_fail(ST_ERR_ALIGNMENT, call, name, "scale stride not a multiple of 4");
    out.scales = v->scales;
    out.scale_stride = ss;
  }
  return ST_OK;
}
inline Rows no_rows() { Rows r{}; r.type = -1; return r; }

constexpr uint32_t kTakesFloat = 1u << ST_F32 | 1u << ST_BF16;
constexpr uint32_t kTakesAll = kTakesFloat | 1u << ST_MX8;

// True where two operands share bytes: `arows` rows of `ac` channels and `brows` of
// `bc`.  Views of one buffer with one stride and columns apart do not, nor does one
// row that lies between the rows of another operand.
inline bool bytes_meet(const void* ap, int64_t as, int64_t an, int64_t arows, const void* bp, int64_t bs, int64_t bn, int64_t brows) {
  const char *a = static_cast<const char*>(ap), *b = static_cast<const char*>(bp);
  if (!(a < b + (brows - 1) * bs + bn && b < a + (arows - 1) * as + an)) return false;
  if (arows == 1 && brows > 1) return bytes_meet(bp, bs, bn, brows, ap, as, an, arows);
  if (arows > 1 && (brows == 1 || as == bs)) {
    const int64_t d = ((b - a) % as + as) % as;             // b's rows start d bytes after a's
    return d < an || d + bn > as;
  }
  return true;
}
inline bool meet(const Rows& a, int64_t arows, int64_t ac, const Rows& b, int64_t brows, int64_t bc) {
  if (a.type < 0 || b.type < 0 || arows <= 0 || brows <= 0) return false;
  const void* p[2][2] = {{a.p, a.scales}, {b.p, b.scales}};
  const int64_t s[2][2] = {{a.stride, a.scale_stride}, {b.stride, b.scale_stride}};
  const int64_t n[2][2] = {{ac * type_size(a.type), (ac + kMxBlock - 1) / kMxBlock}, {bc * type_size(b.type), (bc + kMxBlock - 1) / kMxBlock}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (p[0][i] && p[1][j] && bytes_meet(p[0][i], s[0][i], n[0][i], arows, p[1][j], s[1][j], n[1][j], brows)) return true;
  return false;
}
// `n` floats beside the rows (a bias, a gamma, sums), as one row
inline Rows floats_of(const float* p, int64_t n) {
  Rows r = no_rows();
  if (!p) return r;
  r.p = reinterpret_cast<char*>(const_cast<float*>(p));
  r.stride = 4 * n;
  r.type = ST_F32;
  return r;
}
inline bool rows_meet(const Rows& a, const Rows& b, int64_t rows, int64_t channels) { return meet(a, rows, channels, b, rows, channels); }
// The same rows in the same type: what an operator that reads before it writes may take
inline bool same_rows(const Rows& a, const Rows& b) { return a.p == b.p && a.stride == b.stride && a.type == b.type; }

// ------------------------------------------------------------------ device

// vectors at any address: gfx950 takes unaligned global accesses, so rows of odd
// length cost no other code path
typedef f32x4_t f32x4_any __attribute__((aligned(4)));
typedef u32x4_t u32x4_any __attribute__((aligned(2)));
typedef u32x2_t u32x2_any __attribute__((aligned(2)));

// `n` (0 .. VEC) of VEC consecutive values at p, the others zero.  type: F32 or BF16
template <class T, int VEC> __device__ __forceinline__ void load_some(const char* p, int n, float (&x)[VEC]) {
  if (n >= VEC) {
    if constexpr (T::kSize == 4) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const f32x4_t v = reinterpret_cast<const f32x4_any*>(p)[i];
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
      }
    } else if constexpr (VEC == 8) {
      const u32x4_t w = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) { x[2 * i] = bf16_lo(w[i]); x[2 * i + 1] = bf16_hi(w[i]); }
    } else {
      const u32x2_t w = *reinterpret_cast<const u32x2_any*>(p);
#pragma unroll
      for (int i = 0; i < 2; ++i) { x[2 * i] = bf16_lo(w[i]); x[2 * i + 1] = bf16_hi(w[i]); }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      x[i] = 0.f;
      if (i < n) {
        if constexpr (T::kSize == 4) x[i] = reinterpret_cast<const float*>(p)[i];
        else x[i] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
      }
    }
  }
}

// A group as it lies in memory, unpacked when it is used: a load that is unpacked
// where its type is looked at would be waited for there, one after the other.
// EVEN: groups are whole or absent (the row's length is a multiple of VEC).
template <int VEC> struct Raw { uint32_t w[VEC]; };
template <bool EVEN, int VEC> __device__ __forceinline__ void load_raw(int type, const char* p, int n, Raw<VEC>& r) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) r.w[i] = 0;
  if (EVEN ? n > 0 : n >= VEC) {
    if (VEC == 8 || type == ST_F32) {
      const u32x4_t t = *reinterpret_cast<const u32x4_any*>(p);
      r.w[0] = t[0]; r.w[1] = t[1]; r.w[2] = t[2]; r.w[3] = t[3];
    } else {
      const u32x2_t t = *reinterpret_cast<const u32x2_any*>(p);
      r.w[0] = t[0]; r.w[1] = t[1];
    }
    if constexpr (VEC == 8) {
      if (type == ST_F32) {
        const u32x4_t t = *reinterpret_cast<const u32x4_any*>(p + 16);
        r.w[4] = t[0]; r.w[5] = t[1]; r.w[6] = t[2]; r.w[7] = t[3];
      }
    }
  } else if constexpr (!EVEN) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < n) {
        if (type == ST_F32) r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else r.w[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
      }
  }
}
template <int VEC> __device__ __forceinline__ void unpack(int type, const Raw<VEC>& r, float (&x)[VEC]) {
  if (type == ST_F32) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) { x[2 * i] = bf16_lo(r.w[i]); x[2 * i + 1] = bf16_hi(r.w[i]); }
  }
}

template <int VEC, bool NT = false> __device__ __forceinline__ void store_some(int type, char* p, int n, const float (&x)[VEC]) {
  if (type == ST_F32) {
    if (n >= VEC) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const f32x4_t v = {x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
        if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<f32x4_any*>(p) + i);
        else reinterpret_cast<f32x4_any*>(p)[i] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < n) reinterpret_cast<float*>(p)[i] = x[i];
    }
  } else if (n >= VEC) {
    if constexpr (VEC == 8) {
      const u32x4_t w = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
      if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any*>(p));
      else *reinterpret_cast<u32x4_any*>(p) = w;
    } else {
      const u32x2_t w = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
      if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<u32x2_any*>(p));
      else *reinterpret_cast<u32x2_any*>(p) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < n) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16(x[i], 0.f);
  }
}

// ---- the 8-bit form: e4m3 codes, one power of two per 32 channels

// Magnitude bits: those of a NaN or an infinity are 0x7F800000 or more, and do not
// count for their block's scale (their codes are NaN codes at any scale)
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t mx_bits(float v) {
  const uint32_t b = mag_bits(v);
  return b < 0x7F800000u ? b : 0u;
}
// Scale byte (k + 127) of a block whose largest magnitude has these bits: the
// smallest k with amax <= 448 * 2^k (448 = 1.75 * 2^8), so that no element
// saturates, as the scale of the largest power below amax would let a quarter of
// the blocks do; 1 .. 254, so that 2^k and 2^-k are normal numbers.
__device__ __forceinline__ int mx_scale(uint32_t amax_bits) {
  const int k = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(k, 1), 254);
}
__device__ __forceinline__ float pow2_of(int byte) { return __uint_as_float((uint32_t)byte << 23); }
// four values as codes of scale byte s: v * 2^-k (exact) rounded to nearest even.
// A NaN gives a NaN code by itself, an infinity where SPECIAL.
template <bool SPECIAL> __device__ __forceinline__ uint32_t mx_codes(const float* v, int s) {
  const float f = pow2_of(254 - s);
  float u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u[i] = v[i] * f;
    if constexpr (SPECIAL) u[i] = fabsf(u[i]) <= 448.f ? u[i] : __builtin_nanf("");
  }
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(u[2], u[3], w, true);
  return (uint32_t)w;
}
__device__ __forceinline__ void mx_values(uint32_t w, int s, float* v) {
  // byte 0 is 2^-127 and 255 NaN: below and above what a float's exponent field says
  const float f = (uint32_t)(s - 1) < 254u ? pow2_of(s) : s == 0 ? 0x1p-127f : __builtin_nanf("");
  const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = a.x * f; v[1] = a.y * f; v[2] = b.x * f; v[3] = b.y * f;
}

// max over the lanes of one block: lanes of VEC values each (quads at 8, eights at 4)
template <int C> __device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, C, 0xF, 0xF, false));
}
template <int VEC> __device__ __forceinline__ uint32_t block_max(uint32_t v) {
  v = max_dpp<0xB1>(v);                                 // quad_perm 1 0 3 2
  v = max_dpp<0x4E>(v);                                 // quad_perm 2 3 0 1
  if constexpr (VEC == 4) v = max_dpp<0x141>(v);        // row_half_mirror
  return v;
}

// VEC channels' codes of scale byte s at (row, c), of which n exist; the group that
// starts a block writes its scale.  Codes past the row's end are left as they are.
template <int VEC, bool NT = false> __device__ __forceinline__ void store_codes(const Rows& o, int64_t row, int c, int n, const float (&v)[VEC], int s) {
  if (n <= 0) return;
  uint8_t* p = reinterpret_cast<uint8_t*>(o.p) + row * o.stride + c;
  uint32_t w[VEC / 4];
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) w[i] = mx_codes<true>(v + 4 * i, s);
  if (n >= VEC) {
    if constexpr (VEC == 8 && NT) __builtin_nontemporal_store(u32x2_t{w[0], w[1]}, reinterpret_cast<u32x2_t*>(p));
    else if constexpr (VEC == 8) *reinterpret_cast<u32x2_t*>(p) = u32x2_t{w[0], w[1]};
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < n) p[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
  if ((c & (kMxBlock - 1)) == 0) o.scales[row * o.scale_stride + (c >> 5)] = (uint8_t)s;
}
// VEC channels' codes at (row, c), those past the n that exist zero; returns the scale byte
template <int VEC> __device__ __forceinline__ int load_codes(const Rows& x, int64_t row, int c, int n, uint32_t (&w)[VEC / 4]) {
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) w[i] = 0;
  if (n <= 0) return 127;
  const uint8_t* p = reinterpret_cast<const uint8_t*>(x.p) + row * x.stride + c;
  if (n >= VEC) {
    if constexpr (VEC == 8) {
      const u32x2_t t = *reinterpret_cast<const u32x2_t*>(p);
      w[0] = t[0]; w[1] = t[1];
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < n) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  }
  return x.scales[row * x.scale_stride + (c >> 5)];
}
template <int VEC> __device__ __forceinline__ void load_values(const Rows& x, int64_t row, int c, int n, float (&v)[VEC]) {
  uint32_t w[VEC / 4];
  const int s = load_codes<VEC>(x, row, c, n, w);
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) mx_values(w[i], s, v + 4 * i);
}

// ---- activations

enum { kActNone = ST_ACT_NONE, kActRelu = ST_ACT_RELU, kActGelu = ST_ACT_GELU, kActSilu = ST_ACT_SILU };

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float rcp_fast(float v) { return __builtin_amdgcn_rcpf(v); }

// Upper tail of the normal distribution, Q(a) = erfc(a / sqrt 2) / 2 for a >= 0, as
// exp(-a^2 / 2) R(t), t = 1 / (1 + 0.3 a).  R: a polynomial of degree 8 fitted to
// Q(a) exp(a^2 / 2) on 0 <= a <= 13 by weighted least squares to equal relative
// errors (6e-8; 3e-7 with fp32 steps and the hardware's exp2 and reciprocal).
// Returns R(t) and exp(-a^2 / 2) apart: the gradient needs both.
__device__ __forceinline__ float tail_poly(float a) {
  const float t = rcp_fast(fmaf(0.3f, a, 1.f));
  float r = 0.0382709876f;
  r = fmaf(r, t, -0.168643445f);
  r = fmaf(r, t, 0.227577806f);
  r = fmaf(r, t, -0.0752652735f);
  r = fmaf(r, t, 0.141675502f);
  r = fmaf(r, t, 0.0950512066f);
  r = fmaf(r, t, 0.121825859f);
  r = fmaf(r, t, 0.119501002f);
  return fmaf(r, t, 6.38292568e-06f);
}
constexpr float kHalfLog2e = 0.72134752044448170f, kLog2E = 1.4426950408889634f, kInvSqrt2Pi = 0.39894228040143268f;

// Infinities take the limits (exp2's argument and the clamped factor see to it), NaN
// stays NaN through exp2.
template <int ACT> __device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == kActRelu) return z > 0.f ? z : (z != z ? z : 0.f);
  if constexpr (ACT == kActGelu) {
    // z Phi(z) = max(z, 0) - |z| Q(|z|)
    const float a = __builtin_amdgcn_fmed3f(fabsf(z), 0.f, 13.f);
    return fmaf(-a * tail_poly(a), exp2_fast(-kHalfLog2e * z * z), __builtin_amdgcn_fmed3f(z, 0.f, INFINITY));
  }
  if constexpr (ACT == kActSilu) return __builtin_amdgcn_fmed3f(z, -200.f, INFINITY) * rcp_fast(1.f + exp2_fast(-kLog2E * z));
  return z;
}
// derivative of the activation
template <int ACT> __device__ __forceinline__ float slope_of(float z) {
  if constexpr (ACT == kActRelu) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == kActGelu) {
    // Phi(z) + z phi(z)
    const float a = __builtin_amdgcn_fmed3f(fabsf(z), 0.f, 13.f), e = exp2_fast(-kHalfLog2e * z * z);
    const float tail = fmaf(-e, tail_poly(a), 0.5f);    // 1/2 - Q(|z|)
    return fmaf(__builtin_amdgcn_fmed3f(z, -13.f, 13.f), e * kInvSqrt2Pi, 0.5f + copysignf(tail, z));
  }
  if constexpr (ACT == kActSilu) {
    const float s = rcp_fast(1.f + exp2_fast(-kLog2E * z)), c = __builtin_amdgcn_fmed3f(z, -200.f, 200.f);
    return s * fmaf(c, 1.f - s, 1.f);
  }
  return 1.f;
}
// one branch for N values
template <int N> __device__ __forceinline__ void activate(int act, float (&v)[N]) {
  if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_of<kActGelu>(v[i]);
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_of<kActSilu>(v[i]);
  } else if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_of<kActRelu>(v[i]);
  }
}
// Launches that other operators make (mx8.hip)
st_status mx8_store_rows(int64_t rows, int64_t channels, const Rows& x, const Rows& out, hipStream_t st);
st_status mx8_load_rows(int64_t rows, int64_t channels, const Rows& x, int act, const Rows& out, hipStream_t st);

// Sums `parts` rows of `columns` floats in order (rmsnorm.hip)
st_status add_rows_launch(const float* partial, int parts, int columns, float* out, hipStream_t st);

}  // namespace st
