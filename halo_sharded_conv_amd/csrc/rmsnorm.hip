// Root-mean-square norm of x + residual, forward and backward.
//
//   s  = x + residual, rounded to the type it is kept in
//   y  = s * r * gamma,  r = 1 / sqrt(mean(s^2) + eps)
//   dx = ds + r * (g - xh * mean(g * xh)),  g = dy * gamma, xh = s * r
//   dgamma = sum over rows of dy * xh
// The norm is of the rounded s, so that the backward pass, which reads it, has the
// same xh.
//
// Bound: HBM.  One pass: a row stays in registers between its loads and its
// stores, held by a power-of-two group of lanes (sums cross lanes by DPP and
// swaps), or by a workgroup when it is wider than a wave holds.  The 8-bit output
// is rounded from the fp32 y in the same pass: a block of 32 channels lies in four
// lanes of 8 channels or eight of 4, its largest magnitude crosses them by DPP.
// All sums are fp32.
//
// dgamma: every thread keeps the sums of its own columns over the rows it visits,
// a workgroup adds its threads in a fixed order and writes one partial row, and a
// second kernel adds the partial rows in order: no atomics.
//
// 1024 x 1792 x 256, fp32 + bf16 to fp32 and 8 bits: 979 us (5.3 TB/s); 65536 x 1000 in
// bf16: 109 us forward, 101 backward (4.8 and 5.2).
#include <algorithm>
#include <string>

#include "rows.h"

namespace st {
namespace {

constexpr int kRmsThreads = 256;
constexpr int kRmsMaxC = 16384;
// Workgroups (partial rows) of the backward pass, of which those of 16 waves take
// half: four a CU (65536 rows of 2048 in bf16, a row each: 2048 of them 227 us, 1024 196)
constexpr int kRmsMaxParts = 1024;

struct RmsArgs {
  Rows x, res, total, y, y8;          // forward; backward: s, dtotal, -, dx, dy in x, res, -, y, total
  int32_t rows, channels, lpr_log2, parts, blocks;
  float eps, count;
  const float* gamma;
  float* rstd;
  float* partial;
};

template <int C> __device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), C, 0xF, 0xF, false));
}

// sum over the lanes of one row: a power of two of them, or (WAVES > 0) those of a
// workgroup of so many waves
template <int WAVES> __device__ __forceinline__ float row_sum(float v, int lpr, float* red) {
  const int n = WAVES ? 64 : lpr;
  if (n > 1) v = add_dpp<0xB1>(v);                      // quad_perm 1 0 3 2
  if (n > 2) v = add_dpp<0x4E>(v);                      // quad_perm 2 3 0 1
  if (n > 4) v = add_dpp<0x141>(v);                     // row_half_mirror
  if (n > 8) v = add_dpp<0x140>(v);                     // row_mirror
  if (n > 16) {
    const u32x2_t r = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (n > 32) {
    const u32x2_t r = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (WAVES > 0) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();                                    // the last sum's readers are done
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; w += 4) v += (red[w] + red[w + 1]) + (red[w + 2] + red[w + 3]);
  }
  return v;
}

// rows of one lane group in flight per pass, by the values a lane holds of one
constexpr int rms_unroll(int per) { return per >= 32 ? 1 : per >= 16 ? 2 : 4; }
constexpr int kRmsBackUnroll = 2;

__device__ __forceinline__ int size_of(int type) { return type == ST_F32 ? 4 : 2; }

template <int VEC, int NV, bool BLOCK, bool EVEN> __global__ __launch_bounds__(kRmsThreads) void rms_forward(const RmsArgs a) {
  constexpr int U = BLOCK ? 1 : rms_unroll(NV * VEC);
  __shared__ float red[4];
  const int lpr = BLOCK ? kRmsThreads : 1 << a.lpr_log2;
  const int sub = threadIdx.x & (lpr - 1), slot = threadIdx.x / lpr, rp = kRmsThreads / lpr;
  const int C = a.channels;
  const int64_t r0 = (int64_t)blockIdx.x * (rp * U) + slot;
  float x[U][NV][VEC];
  {
    Raw<VEC> xr[U][NV], rr[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * rp;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (sub + k * lpr) * VEC, n = r < a.rows ? C - c : 0;
        load_raw<EVEN, VEC>(a.x.type, a.x.p + r * a.x.stride + (int64_t)c * size_of(a.x.type), n, xr[u][k]);
        if (a.res.type >= 0) load_raw<EVEN, VEC>(a.res.type, a.res.p + r * a.res.stride + (int64_t)c * size_of(a.res.type), n, rr[u][k]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < NV; ++k) unpack<VEC>(a.x.type, xr[u][k], x[u][k]);
    if (a.res.type >= 0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          float t[VEC];
          unpack<VEC>(a.res.type, rr[u][k], t);
#pragma unroll
          for (int i = 0; i < VEC; ++i) x[u][k][i] += t[i];
        }
    }
  }
  if (a.total.type == ST_BF16) {                        // the norm is of s as it is kept
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          const uint32_t w = pack_bf16(x[u][k][i], x[u][k][i + 1]);
          x[u][k][i] = bf16_lo(w);
          x[u][k][i + 1] = bf16_hi(w);
        }
  }
  float rstd[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) t = fmaf(x[u][k][i], x[u][k][i], t);
    rstd[u] = 1.f / sqrtf(row_sum<BLOCK ? 4 : 0>(t, lpr, red) / a.count + a.eps);
  }
  if (a.rstd && sub == 0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r0 + u * rp < a.rows) a.rstd[r0 + u * rp] = rstd[u];
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (sub + k * lpr) * VEC;
    float g[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = 1.f;
    if (a.gamma) {
      Raw<VEC> t;
      load_raw<EVEN, VEC>(ST_F32, reinterpret_cast<const char*>(a.gamma + c), C - c, t);
      unpack<VEC>(ST_F32, t, g);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * rp;
      const int n = r < a.rows ? C - c : 0;
      float y[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) y[i] = x[u][k][i] * rstd[u] * g[i];
      if (a.total.type >= 0 && n > 0) store_some<VEC, true>(a.total.type, a.total.p + r * a.total.stride + (int64_t)c * size_of(a.total.type), EVEN ? VEC : n, x[u][k]);
      if (a.y.type >= 0 && n > 0) store_some<VEC, true>(a.y.type, a.y.p + r * a.y.stride + (int64_t)c * size_of(a.y.type), EVEN ? VEC : n, y);
      if (a.y8.type >= 0) {                             // (every lane: a block's maximum crosses them)
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) top = max(top, EVEN || i < n ? mx_bits(y[i]) : 0u);   // (absent lanes hold zeros)
        const int s = mx_scale(block_max<VEC>(top));
        store_codes<VEC>(a.y8, r, c, EVEN && n > 0 ? VEC : n, y, s);
      }
    }
  }
}

// s, dy, dtotal -> dx, partial sums of dgamma.  TS: F32, BF16 or MX8 (s as it was kept)
// a group of s as it was kept, before it is unpacked
template <class TS, int VEC> struct Kept { Raw<VEC> r; int scale; };
template <class TS, bool EVEN, int VEC> __device__ __forceinline__ void load_kept(const Rows& s, int64_t r, int c, int n, Kept<TS, VEC>& k) {
  if constexpr (std::is_same<TS, MX8>::value) {
    uint32_t w[VEC / 4];
    k.scale = load_codes<VEC>(s, r, c, EVEN && n > 0 ? VEC : n, w);
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) k.r.w[i] = w[i];
  } else {
    load_raw<EVEN, VEC>(TS::kSize == 4 ? ST_F32 : ST_BF16, s.p + r * s.stride + (int64_t)c * TS::kSize, n, k.r);
  }
}
template <class TS, int VEC> __device__ __forceinline__ void unpack_kept(const Kept<TS, VEC>& k, float (&x)[VEC]) {
  if constexpr (std::is_same<TS, MX8>::value) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) mx_values(k.r.w[i], k.scale, x + 4 * i);
  } else {
    unpack<VEC>(TS::kSize == 4 ? ST_F32 : ST_BF16, k.r, x);
  }
}

// WAVES: of a workgroup that holds a row; 0: rows in lane groups of four waves
template <class TS, int VEC, int NV, int WAVES, bool EVEN> __global__ __launch_bounds__(WAVES ? 64 * WAVES : kRmsThreads) void rms_backward(const RmsArgs a) {
  constexpr bool BLOCK = WAVES > 0;
  constexpr int U = BLOCK ? 1 : kRmsBackUnroll, THREADS = BLOCK ? 64 * WAVES : kRmsThreads;
  __shared__ float red[BLOCK ? WAVES : 4];
  const int lpr = BLOCK ? THREADS : 1 << a.lpr_log2;
  const int sub = threadIdx.x & (lpr - 1), slot = threadIdx.x / lpr, rp = THREADS / lpr;
  const int C = a.channels;
  const Rows &S = a.x, &DY = a.total, &DT = a.res, &DX = a.y;
  float g[NV][VEC], dg[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (sub + k * lpr) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) { g[k][i] = 1.f; dg[k][i] = 0.f; }
    if (a.gamma) {
      Raw<VEC> t;
      load_raw<EVEN, VEC>(ST_F32, reinterpret_cast<const char*>(a.gamma + c), C - c, t);
      unpack<VEC>(ST_F32, t, g[k]);
    }
  }
  for (int blk = blockIdx.x; blk < a.blocks; blk += a.parts) {
    const int64_t r0 = (int64_t)blk * (rp * U) + slot;
    Kept<TS, VEC> sr[U][NV];
    Raw<VEC> yr[U][NV], tr[U][NV];
    float rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * rp;
      rstd[u] = r < a.rows ? a.rstd[r] : 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (sub + k * lpr) * VEC, n = r < a.rows ? C - c : 0;
        load_kept<TS, EVEN, VEC>(S, r, c, n, sr[u][k]);
        load_raw<EVEN, VEC>(DY.type, DY.p + r * DY.stride + (int64_t)c * size_of(DY.type), n, yr[u][k]);
        if (DT.type >= 0) load_raw<EVEN, VEC>(DT.type, DT.p + r * DT.stride + (int64_t)c * size_of(DT.type), n, tr[u][k]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * rp;
      float x[NV][VEC], dy[NV][VEC], t = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        unpack_kept<TS, VEC>(sr[u][k], x[k]);
        unpack<VEC>(DY.type, yr[u][k], dy[k]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float xh = x[k][i] * rstd[u], d = dy[k][i];
          x[k][i] = xh;
          dg[k][i] = fmaf(d, xh, dg[k][i]);
          dy[k][i] = d * g[k][i];
          t = fmaf(dy[k][i], xh, t);
        }
      }
      t = row_sum<WAVES>(t, lpr, red) / a.count;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (sub + k * lpr) * VEC, n = r < a.rows ? C - c : 0;
        if (n <= 0) continue;
        float dx[VEC], dt[VEC];
        if (DT.type >= 0) {
          unpack<VEC>(DT.type, tr[u][k], dt);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) dt[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) dx[i] = fmaf(rstd[u], dy[k][i] - x[k][i] * t, dt[i]);
        store_some<VEC, true>(DX.type, DX.p + r * DX.stride + (int64_t)c * size_of(DX.type), EVEN ? VEC : n, dx);
      }
    }
  }
  if (!a.partial) return;
  // this workgroup's partial row: over the slots of a wave, then over the waves
  float* out = a.partial + (int64_t)blockIdx.x * C;
  if constexpr (BLOCK) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (sub + k * lpr) * VEC;
      if (c < C) store_some<VEC>(ST_F32, reinterpret_cast<char*>(out + c), C - c, dg[k]);
    }
  } else {
    __shared__ float acc[4][64 * NV * VEC];
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        for (int m = lpr; m < 64; m <<= 1) dg[k][i] += __shfl_xor(dg[k][i], m);
        if ((threadIdx.x & 63) < lpr) acc[wave][(sub + k * lpr) * VEC + i] = dg[k][i];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += kRmsThreads) out[c] = (acc[0][c] + acc[1][c]) + (acc[2][c] + acc[3][c]);
  }
}

// ------------------------------------------------------------------ host

struct RmsPick {                      // how a row is held
  int vec, nv, lpr_log2;
  bool block;
  int waves;                          // backward: of the workgroup that holds a row (0: lane groups)
};

// Forward: whole rows per wave while a lane holds at most 64 values (32 with an fp32
// operand), by a workgroup beyond.  At least the lanes of one block of 32.
RmsPick rms_pick_forward(int C, bool wide) {
  RmsPick p{};
  p.vec = wide ? 8 : 4;
  const int nvec = (C + p.vec - 1) / p.vec;
  const int most = (wide ? 64 : 32) / p.vec;
  p.block = nvec > 64 * most;
  const int lanes = p.block ? 256 : 64;
  const int need = (nvec + lanes - 1) / lanes;
  p.nv = 1;
  while (p.nv < need) p.nv *= 2;
  int l = p.vec == 8 ? 2 : 3;
  while ((1 << l) < lanes && (1 << l) < nvec) ++l;
  p.lpr_log2 = p.block ? 8 : l;
  return p;
}
// Backward: few values a lane, so that many waves fit a SIMD: rows by a wave's lanes up
// to 1024 channels (two vectors of 8 a lane; 512 at 4), by 4, 8 or 16 waves beyond
// (65536 x 1000 in bf16: by a wave 105 us, by four 113; 8192 x 8192: four vectors a
// lane of four waves 163 us, one a lane of sixteen 105; 65536 x 500 in fp32: two vectors
// of 4 a lane 104 us, by four waves 98).  Above 8192 channels sixteen waves hold two
// vectors of 8 a lane or four of 4, and 3 to 22 registers of the 128 spill (16 to 92
// bytes a lane): 8192 x 16384 in bf16 211 us (5.1 TB/s), in fp32 428 (5.0), with s in 8
// bits 214 (4.4; 5.0 at 8192 channels).
RmsPick rms_pick_backward(int C, bool wide) {
  RmsPick p{};
  p.vec = wide ? 8 : 4;
  const int nvec = (C + p.vec - 1) / p.vec;
  p.block = nvec > (wide ? 128 : 64);
  p.waves = !p.block ? 0 : nvec <= 256 ? 4 : nvec <= 512 ? 8 : 16;
  p.nv = 1;
  while (p.nv * (p.block ? 64 * p.waves : 64) < nvec) p.nv *= 2;
  while ((1 << p.lpr_log2) < nvec && p.lpr_log2 < 6) ++p.lpr_log2;
  return p;
}

int rms_rows_per_block(const RmsPick& p, bool backward) {
  return p.block ? 1 : (kRmsThreads >> p.lpr_log2) * (backward ? kRmsBackUnroll : rms_unroll(p.nv * p.vec));
}

int rms_parts(int64_t rows) { return (int)std::max<int64_t>(1, std::min<int64_t>(kRmsMaxParts, rows)); }

st_status rms_forward_launch(const RmsArgs& a, const RmsPick& p, int blocks, hipStream_t st) {
#define RMS_CASE(V, N, B) \
  if (p.vec == V && p.nv == N && p.block == B) { \
    if (a.channels % V == 0) rms_forward<V, N, B, true><<<blocks, kRmsThreads, 0, st>>>(a); \
    else rms_forward<V, N, B, false><<<blocks, kRmsThreads, 0, st>>>(a); \
    return launch_check("rms_forward"); \
  }
  RMS_CASE(8, 1, false) RMS_CASE(8, 2, false) RMS_CASE(8, 4, false) RMS_CASE(8, 8, false)
  RMS_CASE(8, 4, true) RMS_CASE(8, 8, true)
  RMS_CASE(4, 1, false) RMS_CASE(4, 2, false) RMS_CASE(4, 4, false) RMS_CASE(4, 8, false)
  RMS_CASE(4, 4, true) RMS_CASE(4, 8, true) RMS_CASE(4, 16, true)
#undef RMS_CASE
  return fail(ST_ERR_UNSUPPORTED, "rms norm: no kernel for this width");
}

template <class TS> st_status rms_backward_launch(const RmsArgs& a, const RmsPick& p, hipStream_t st) {
#define RMS_CASE(V, N, W) \
  if (p.vec == V && p.nv == N && p.waves == W) { \
    if (a.channels % V == 0) rms_backward<TS, V, N, W, true><<<a.parts, W ? 64 * W : kRmsThreads, 0, st>>>(a); \
    else rms_backward<TS, V, N, W, false><<<a.parts, W ? 64 * W : kRmsThreads, 0, st>>>(a); \
    return launch_check("rms_backward"); \
  }
  RMS_CASE(8, 1, 0) RMS_CASE(8, 2, 0) RMS_CASE(8, 1, 4) RMS_CASE(8, 1, 8) RMS_CASE(8, 1, 16) RMS_CASE(8, 2, 16)
  if constexpr (std::is_same<TS, F32>::value) {         // (4 a lane: all sides fp32)
    RMS_CASE(4, 1, 0) RMS_CASE(4, 1, 4) RMS_CASE(4, 1, 8) RMS_CASE(4, 1, 16) RMS_CASE(4, 2, 16) RMS_CASE(4, 4, 16)
  }
#undef RMS_CASE
  return fail(ST_ERR_UNSUPPORTED, "rms norm: no kernel for this width");
}

st_status rms_sizes(int64_t rows, int64_t channels, const char* me) {
  if (rows < 0 || channels < 1) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": negative rows or no channels");
  if (channels > kRmsMaxC) return fail(ST_ERR_UNSUPPORTED, std::string(me) + ": more than 16384 channels");
  if (rows >= (1ll << 31) - kRmsMaxParts) return fail(ST_ERR_UNSUPPORTED, std::string(me) + ": 2^31 rows");
  return ST_OK;
}

}  // namespace

// Sums `parts` partial rows of `columns` floats in order into out (or zeros, parts == 0)
__global__ __launch_bounds__(256) void add_rows(const float* __restrict__ partial, int parts, int columns, float* __restrict__ out) {
  // 16 columns per workgroup, 16 threads add one column's rows (thread t rows t,
  // t + 16, ...), then the threads' sums in order
  __shared__ float acc[16][17];
  const int col = threadIdx.x & 15, t = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + col;
  float v = 0.f;
  if (c < columns) {
#pragma unroll 8
    for (int p = t; p < parts; p += 16) v += partial[(int64_t)p * columns + c];
  }
  acc[t][col] = v;
  __syncthreads();
  if (t == 0 && c < columns) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += acc[i][col];
    out[c] = sum;
  }
}
st_status add_rows_launch(const float* partial, int parts, int columns, float* out, hipStream_t st) {
  add_rows<<<(columns + 15) / 16, 256, 0, st>>>(partial, parts, columns, out);
  return launch_check("add_rows");
}

}  // namespace st

using namespace st;

extern "C" {

st_status st_rmsnorm(int64_t rows, int64_t channels, const st_rows* x, const st_rows* residual_or_null,
                     const float* gamma_or_null, float eps, const st_rows* total_or_null, const st_rows* y_or_null,
                     const st_rows* y8_or_null, float* rstd_or_null, void* stream) {
  const char* const me = "st_rmsnorm";
  st_status s = rms_sizes(rows, channels, me);
  if (s != ST_OK) return s;
  if (!(eps >= 0.f) || !(eps < 3.0e38f)) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": eps must be finite and >= 0");
  if (!aligned16(gamma_or_null) || !aligned16(rstd_or_null)) return fail(ST_ERR_ALIGNMENT, std::string(me) + ": gamma or rstd not 16-byte aligned");
  if (!total_or_null && !y_or_null && !y8_or_null && !rstd_or_null) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": no output");
  RmsArgs a{};
  a.res = a.total = a.y = a.y8 = no_rows();
  if ((s = rows_of(a.x, x, rows, channels, kTakesFloat, me, "x")) != ST_OK) return s;
  if (residual_or_null && (s = rows_of(a.res, residual_or_null, rows, channels, kTakesFloat, me, "residual")) != ST_OK) return s;
  if (total_or_null && (s = rows_of(a.total, total_or_null, rows, channels, kTakesFloat, me, "total")) != ST_OK) return s;
  if (y_or_null && (s = rows_of(a.y, y_or_null, rows, channels, kTakesFloat, me, "y")) != ST_OK) return s;
  if (y8_or_null && (s = rows_of(a.y8, y8_or_null, rows, channels, 1u << ST_MX8, me, "y8")) != ST_OK) return s;
  const Rows* in[2] = {&a.x, &a.res};
  const Rows* out[3] = {&a.total, &a.y, &a.y8};
  for (int i = 0; i < 3; ++i) {
    for (const Rows* r : in)
      if (rows_meet(*out[i], *r, rows, channels) && !(i == 0 && same_rows(*out[i], *r)))
        return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (rows_meet(*out[i], *out[j], rows, channels)) return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": two outputs overlap");
  }
  const Rows gv = floats_of(gamma_or_null, channels), rv = floats_of(rstd_or_null, rows);
  for (const Rows* r : {&a.total, &a.y, &a.y8})
    if (meet(*r, rows, channels, gv, 1, channels)) return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": an output overlaps gamma");
  for (const Rows* r : {&a.x, &a.res, &a.total, &a.y, &a.y8})
    if (meet(*r, rows, channels, rv, 1, rows)) return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": rstd overlaps an operand");
  if (rows > 0 && meet(gv, 1, channels, rv, 1, rows)) return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": rstd overlaps gamma");
  if (rows == 0) return ok();
  a.rows = (int32_t)rows;
  a.channels = (int32_t)channels;
  a.count = (float)channels;
  a.eps = eps;
  a.gamma = gamma_or_null;
  a.rstd = rstd_or_null;
  // 8 values a lane only where no operand is fp32: with one, 4 keep its accesses dense
  bool wide = true;
  for (const Rows* r : {&a.x, &a.res, &a.total, &a.y}) wide = wide && r->type != ST_F32;
  const RmsPick pick = rms_pick_forward((int)channels, wide);
  a.lpr_log2 = pick.lpr_log2;
  const int rpb = rms_rows_per_block(pick, false);
  // launches of fewer than 2^32 threads, whole workgroups of rows each
  const int64_t most = max_blocks(kRmsThreads) * rpb;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = std::min(most, rows - r);
    RmsArgs b = a;
    b.rows = (int32_t)n;
    for (Rows* v : {&b.x, &b.res, &b.total, &b.y, &b.y8}) {
      if (v->type < 0) continue;
      v->p += r * v->stride;
      if (v->type == ST_MX8) v->scales += r * v->scale_stride;
    }
    if (b.rstd) b.rstd += r;
    s = rms_forward_launch(b, pick, (int)((n + rpb - 1) / rpb), static_cast<hipStream_t>(stream));
    if (s != ST_OK) return s;
  }
  return ST_OK;
}

size_t st_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t channels) {
  if (rows < 0 || channels < 1 || channels > kRmsMaxC) return 0;
  return (size_t)rms_parts(rows) * (size_t)channels * sizeof(float);
}

st_status st_rmsnorm_backward(int64_t rows, int64_t channels, const st_rows* s_, const st_rows* dy,
                              const st_rows* dtotal_or_null, const float* gamma_or_null, const float* rstd,
                              const st_rows* dx, float* dgamma_or_null, void* workspace, size_t workspace_bytes,
                              void* stream) {
  const char* const me = "st_rmsnorm_backward";
  st_status s = rms_sizes(rows, channels, me);
  if (s != ST_OK) return s;
  if (rows > 0 && !rstd) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": NULL rstd");
  if (!aligned16(gamma_or_null) || !aligned16(rstd) || !aligned16(dgamma_or_null) || !aligned16(workspace))
    return fail(ST_ERR_ALIGNMENT, std::string(me) + ": gamma, rstd, dgamma or workspace not 16-byte aligned");
  RmsArgs a{};
  a.res = a.y8 = no_rows();
  if ((s = rows_of(a.x, s_, rows, channels, kTakesAll, me, "s")) != ST_OK) return s;
  if ((s = rows_of(a.total, dy, rows, channels, kTakesFloat, me, "dy")) != ST_OK) return s;
  if (dtotal_or_null && (s = rows_of(a.res, dtotal_or_null, rows, channels, kTakesFloat, me, "dtotal")) != ST_OK) return s;
  if ((s = rows_of(a.y, dx, rows, channels, kTakesFloat, me, "dx")) != ST_OK) return s;
  if (rows_meet(a.y, a.x, rows, channels) || (rows_meet(a.y, a.total, rows, channels) && !same_rows(a.y, a.total)) ||
      (rows_meet(a.y, a.res, rows, channels) && !same_rows(a.y, a.res)))
    return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": dx overlaps an input");
  const Rows gv = floats_of(gamma_or_null, channels), rv = floats_of(rstd, rows), dg = floats_of(dgamma_or_null, channels);
  if (meet(a.y, rows, channels, gv, 1, channels) || meet(a.y, rows, channels, rv, 1, rows))
    return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": dx overlaps gamma or rstd");
  bool shared = meet(dg, 1, channels, gv, 1, channels) || (rows > 0 && meet(dg, 1, channels, rv, 1, rows));
  for (const Rows* r : {&a.x, &a.total, &a.res, &a.y}) shared = shared || meet(*r, rows, channels, dg, 1, channels);
  if (shared) return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": dgamma overlaps an operand");
  if (dgamma_or_null && (!workspace || workspace_bytes < st_rmsnorm_backward_workspace_bytes(rows, channels)))
    return fail(ST_ERR_WORKSPACE, std::string(me) + ": workspace missing or too small");
  const hipStream_t st = static_cast<hipStream_t>(stream);
  a.channels = (int32_t)channels;
  float* partial = static_cast<float*>(workspace);
  if (rows == 0) return dgamma_or_null ? add_rows_launch(partial, 0, a.channels, dgamma_or_null, st) : ok();
  a.rows = (int32_t)rows;
  a.count = (float)channels;
  a.gamma = gamma_or_null;
  a.rstd = const_cast<float*>(rstd);
  a.partial = dgamma_or_null ? partial : nullptr;
  // 8 values a lane with any side below 32 bits, as the layer norm's backward pass
  bool wide = false;
  for (const Rows* r : {&a.x, &a.res, &a.total, &a.y}) wide = wide || (r->type >= 0 && r->type != ST_F32);
  const RmsPick pick = rms_pick_backward(a.channels, wide);
  a.lpr_log2 = pick.lpr_log2;
  const int rpb = rms_rows_per_block(pick, true);
  a.blocks = (int32_t)((rows + rpb - 1) / rpb);
  a.parts = std::min(std::min(rms_parts(rows), pick.waves == 16 ? kRmsMaxParts / 2 : kRmsMaxParts), a.blocks);
  s = a.x.type == ST_MX8 ? rms_backward_launch<MX8>(a, pick, st)
      : a.x.type == ST_F32 ? rms_backward_launch<F32>(a, pick, st) : rms_backward_launch<BF16>(a, pick, st);
  if (s != ST_OK || !dgamma_or_null) return s;
  return add_rows_launch(partial, a.parts, a.channels, dgamma_or_null, st);
}

}  // extern "C"
