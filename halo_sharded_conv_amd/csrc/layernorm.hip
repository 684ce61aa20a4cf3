// Layer norm over the channels of every cell of a sharded volume, forward and
// backward.
//
// With mu and the biased variance var of one cell's C channels,
// r = 1 / sqrt(var + eps), xhat = (x - mu) r:
//   y      = xhat * gamma + beta
//   dx     = r * (g - mean(g) - xhat * mean(g * xhat)),   g = dy * gamma
//   dgamma = sum over cells of dy * xhat,   dbeta = sum over cells of dy
// A cell needs no other cell, so a shard needs no halo and no statistics from
// its neighbours; only dgamma and dbeta are summed over the shards.
//
// Bound: HBM.  Forward reads x and writes y once, backward reads x and dy and
// writes dx once; a cell stays in registers between its load and its store,
// so the variance is the centred one (two passes over registers, none over
// memory; the backward pass of 4097 to 16383 channels off the 4-grid alone
// spills, 92 to 596 bytes a lane).  A cell is held by `lpr` lanes (a power of
// two, so sums cross lanes by DPP and swaps), or by the 256 threads of a
// workgroup when it is wider than ln_pick lets a wave hold.  All sums and statistics are fp32.  Measured: 2048^2
// cells of 64 channels in bf16 forward 182 us (5.9 TB/s), backward 322 us (5.0);
// 1024 x 1792 of 256, fp32 in and bf16 out, 460 us (6.1) and 907 us (5.2), where
// a large copy moves 4.8.
//
// dgamma and dbeta: every thread keeps the sums of its own columns over the
// cells it visits, a workgroup adds its threads in a fixed order and writes one
// partial row, and a second kernel adds the partial rows in order: no atomics,
// and the same bits for the same plan.
#include <algorithm>
#include <string>

#include "tokens.h"

namespace st {
namespace {

constexpr int kLnThreads = 256;
constexpr int kLnMaxC = 16384;
// workgroups (partial rows) of the backward pass: four a CU (2048: the partial
// rows' sums take 8 us in place of 5, the pass is no faster)
constexpr int kLnMaxParts = 1024;

struct LnTensor {                     // one tensor's view of a shard's interior
  char* p;                            // first interior cell
  int64_t sn, sd, sh;                 // strides in cells
};
struct LnShard {
  LnTensor t[3];                      // x, y | x, dy, dx
  Div31 w, h, d;                      // dividers by the interior extents
  int32_t rows;
  int32_t block_begin;                // first block of this shard
  int64_t row_begin;                  // first row in `stats`
};
struct LnArgs {
  int32_t nshards, channels, lpr_log2, flat;   // flat: bit i set where tensor i has no margins
  int32_t blocks, parts;
  int32_t block0;                     // forward: this launch's first block
  int32_t out_bf16;
  float eps, count;
  const float* gamma;
  const float* beta;
  float* stats;
  float* partial;
  LnShard sh[ST_MAX_SHARDS];
};
static_assert(sizeof(LnArgs) <= kMaxKernargBytes, "kernel argument struct too large");

__device__ __forceinline__ int64_t cell_of(const LnShard& s, int t, bool flat, uint32_t r) {
  if (flat) return r;
  const uint32_t q = quo(r, s.w), w = r - q * s.w.d;
  const uint32_t q2 = quo(q, s.h), h = q - q2 * s.h.d;
  const uint32_t n = quo(q2, s.d), d = q2 - n * s.d.d;
  return (int64_t)n * s.t[t].sn + (int64_t)d * s.t[t].sd + (int64_t)h * s.t[t].sh + w;
}

// v plus the value of the lane that DPP control C names
template <int C> __device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), C, 0xF, 0xF, false));
}

// sum over the lanes of one cell (a power of two of them): within 16 lanes by
// DPP (pairs, quads, then mirrors, whose partners hold whole quads and halves),
// beyond by lane swaps; no LDS round trips
template <bool BLOCK> __device__ __forceinline__ float cell_sum(float v, int lpr, float* red) {
  const int n = BLOCK ? 64 : lpr;
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
  if constexpr (BLOCK) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();                                    // the last sum's readers are done
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = (red[0] + red[1]) + (red[2] + red[3]);
  }
  return v;
}

// cells of one lane group in flight per pass, by the values a lane holds of one
constexpr int ln_unroll(int per) { return per >= 32 ? 1 : per >= 16 ? 2 : 4; }
constexpr int kLnBackUnroll = 2;      // (1: 373 us, 4: 340 us against 335 us on 2048^2 x 64 bf16; 4 is slower on fp32)

__device__ __forceinline__ int shard_of(const LnArgs& a, int block) {
  int s = 0;
  while (s + 1 < a.nshards && a.sh[s + 1].block_begin <= block) ++s;
  return s;
}

template <class TX, int VEC, int NV, bool BLOCK>
__global__ __launch_bounds__(kLnThreads) void ln_forward(const LnArgs a) {
  constexpr int U = BLOCK ? 1 : ln_unroll(NV * VEC);
  __shared__ float red[4];
  const int lpr = BLOCK ? kLnThreads : 1 << a.lpr_log2;
  const int sub = threadIdx.x & (lpr - 1), slot = threadIdx.x / lpr, rp = kLnThreads / lpr;
  const int C = a.channels;
  const int blk = a.block0 + (int)blockIdx.x;
  const LnShard& s = a.sh[shard_of(a, blk)];
  const int r0 = (blk - s.block_begin) * (rp * U) + slot;
  float x[U][NV][VEC], sum[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + u * rp;
    const char* px = s.t[0].p + (r < s.rows ? cell_of(s, 0, a.flat & 1, r) : 0) * C * TX::kSize;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (sub + k * lpr) * VEC;
      if (c < C && r < s.rows) {
        load_vec<TX, VEC>(px + (int64_t)c * TX::kSize, x[u][k]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[u][k][i] = 0.f;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) t += x[u][k][i];
    sum[u] = cell_sum<BLOCK>(t, lpr, red) / a.count;
  }
  float rstd[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool in = (sub + k * lpr) * VEC < C;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        x[u][k][i] = in ? x[u][k][i] - sum[u] : 0.f;
        t = fmaf(x[u][k][i], x[u][k][i], t);
      }
    }
    rstd[u] = 1.f / sqrtf(cell_sum<BLOCK>(t, lpr, red) / a.count + a.eps);
  }
  if (a.stats && sub == 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * rp;
      if (r < s.rows) *reinterpret_cast<f32x2_t*>(a.stats + 2 * (s.row_begin + r)) = f32x2_t{sum[u], rstd[u]};
    }
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (sub + k * lpr) * VEC;
    if (c >= C) continue;
    float g[VEC], b[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) { g[i] = 1.f; b[i] = 0.f; }
    if (a.gamma) load_vec<F32, VEC>(reinterpret_cast<const char*>(a.gamma + c), g);
    if (a.beta) load_vec<F32, VEC>(reinterpret_cast<const char*>(a.beta + c), b);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * rp;
      if (r >= s.rows) continue;
      float y[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) y[i] = fmaf(x[u][k][i] * rstd[u], g[i], b[i]);
      const int64_t e = cell_of(s, 1, a.flat & 2, r) * C + c;
      if (a.out_bf16) store_vec_nt<BF16, VEC>(s.t[1].p + e * 2, y);
      else store_vec_nt<F32, VEC>(s.t[1].p + e * 4, y);
    }
  }
}

template <class TX, class TY, int VEC, int NV, bool BLOCK>
__global__ __launch_bounds__(kLnThreads) void ln_backward(const LnArgs a) {
  constexpr int U = BLOCK ? 1 : kLnBackUnroll;
  __shared__ float red[4];
  const int lpr = BLOCK ? kLnThreads : 1 << a.lpr_log2;
  const int sub = threadIdx.x & (lpr - 1), slot = threadIdx.x / lpr, rp = kLnThreads / lpr;
  const int C = a.channels;
  float g[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (sub + k * lpr) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) { g[k][i] = 1.f; dg[k][i] = 0.f; db[k][i] = 0.f; }
    if (a.gamma && c < C) load_vec<F32, VEC>(reinterpret_cast<const char*>(a.gamma + c), g[k]);
  }
  for (int blk = blockIdx.x; blk < a.blocks; blk += a.parts) {
    const LnShard& s = a.sh[shard_of(a, blk)];
    const int r0 = (blk - s.block_begin) * (rp * U) + slot;
    float x[U][NV][VEC], dy[U][NV][VEC], mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * rp;
      const bool live = r < s.rows;
      const char* px = s.t[0].p + (live ? cell_of(s, 0, a.flat & 1, r) : 0) * C * TX::kSize;
      const char* py = s.t[1].p + (live ? cell_of(s, 1, a.flat & 2, r) : 0) * C * TY::kSize;
      mean[u] = rstd[u] = 0.f;
      if (live) {
        const f32x2_t st = *reinterpret_cast<const f32x2_t*>(a.stats + 2 * (s.row_begin + r));
        mean[u] = st.x; rstd[u] = st.y;
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (sub + k * lpr) * VEC;
        if (c < C && live) {
          load_vec<TX, VEC>(px + (int64_t)c * TX::kSize, x[u][k]);
          load_vec<TY, VEC>(py + (int64_t)c * TY::kSize, dy[u][k]);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) { x[u][k][i] = mean[u]; dy[u][k][i] = 0.f; }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * rp;
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float xh = (x[u][k][i] - mean[u]) * rstd[u], d = dy[u][k][i];
          x[u][k][i] = xh;
          dg[k][i] = fmaf(d, xh, dg[k][i]);
          db[k][i] += d;
          const float gd = d * g[k][i];
          dy[u][k][i] = gd;
          s1 += gd;
          s2 = fmaf(gd, xh, s2);
        }
      s1 = cell_sum<BLOCK>(s1, lpr, red) / a.count;
      s2 = cell_sum<BLOCK>(s2, lpr, red) / a.count;
      if (r >= s.rows) continue;
      const int64_t cell = cell_of(s, 2, a.flat & 4, r) * C;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (sub + k * lpr) * VEC;
        if (c >= C) continue;
        float dx[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) dx[i] = rstd[u] * (dy[u][k][i] - s1 - x[u][k][i] * s2);
        if (a.out_bf16) store_vec_nt<BF16, VEC>(s.t[2].p + (cell + c) * 2, dx);
        else store_vec_nt<F32, VEC>(s.t[2].p + (cell + c) * 4, dx);
      }
    }
  }
  // this workgroup's partial row: over the slots of a wave, then over the waves
  float* out = a.partial + (int64_t)blockIdx.x * 2 * C;
  if constexpr (BLOCK) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (sub + k * lpr) * VEC;
      if (c >= C) continue;
      store_vec<F32, VEC>(reinterpret_cast<char*>(out + c), dg[k]);
      store_vec<F32, VEC>(reinterpret_cast<char*>(out + C + c), db[k]);
    }
  } else {
    __shared__ float acc[4][2][64 * NV * VEC];
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        for (int m = lpr; m < 64; m <<= 1) {
          dg[k][i] += __shfl_xor(dg[k][i], m);
          db[k][i] += __shfl_xor(db[k][i], m);
        }
        const int c = (sub + k * lpr) * VEC + i;
        if ((threadIdx.x & 63) < lpr) {
          acc[wave][0][c] = dg[k][i];
          acc[wave][1][c] = db[k][i];
        }
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * C; c += kLnThreads) {
      const int w = c >= C, cc = c - w * C;
      out[c] = (acc[0][w][cc] + acc[1][w][cc]) + (acc[2][w][cc] + acc[3][w][cc]);
    }
  }
}

// dgamma, dbeta: 16 columns per workgroup, 16 threads add one column's partial
// rows (thread t rows t, t + 16, ...), then the threads' sums in order.
__global__ __launch_bounds__(256) void ln_columns(const float* __restrict__ partial, int parts, int C,
                                                  float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float acc[16][17];
  const int col = threadIdx.x & 15, t = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + col;
  float v = 0.f;
  if (c < 2 * C) {
#pragma unroll 8
    for (int p = t; p < parts; p += 16) v += partial[(int64_t)p * 2 * C + c];
  }
  acc[t][col] = v;
  __syncthreads();
  if (t == 0 && c < 2 * C) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += acc[i][col];
    float* out = c < C ? dgamma : dbeta;
    if (out) out[c < C ? c : c - C] = sum;
  }
}

// ------------------------------------------------------------------ host

struct LnPick {                       // how a cell is held
  int vec, nv, lpr_log2;
  bool block;
};

// Rows per pass and lane layout: the widest vector that divides C, whole cells
// per wave while a lane holds at most 8 vectors (16 single values) forward, 16
// values backward (x, dy, gamma and both column sums): up to 4096 channels at 8
// values a vector, 2048 at 4, 1024 at 1 forward, 1024 backward.
LnPick ln_pick(int C, bool wide, bool backward) {
  LnPick p{};
  p.vec = C % 8 == 0 && wide ? 8 : C % 4 == 0 ? 4 : 1;
  const int nvec = C / p.vec;
  const int most = backward ? (p.vec == 8 ? 2 : p.vec == 4 ? 4 : 16) : p.vec == 1 ? 16 : 8;
  p.block = nvec > 64 * most;
  const int lanes = p.block ? 256 : 64;
  const int need = (nvec + lanes - 1) / lanes;
  static const int steps8[] = {1, 2, 4, 8}, steps4[] = {1, 2, 4, 8, 16}, steps1[] = {1, 4, 16, 64};
  const int* st = p.vec == 8 ? steps8 : p.vec == 4 ? steps4 : steps1;
  int i = 0;
  while (st[i] < need) ++i;
  p.nv = st[i];
  int l = 0;
  while ((1 << l) < lanes && (1 << l) < nvec) ++l;
  p.lpr_log2 = p.block ? 8 : l;
  return p;
}

int ln_rows_per_block(const LnPick& p, bool backward) {
  const int per = p.nv * p.vec;
  return p.block ? 1 : (kLnThreads >> p.lpr_log2) * (backward ? kLnBackUnroll : ln_unroll(per));
}

int64_t shard_rows(const st_plan* p, const Shard& s) { return p->batch * s.ext[0] * s.ext[1] * s.ext[2]; }

// workgroups of the backward pass: from the plan alone (every dtype pairing
// takes the same number)
int ln_parts(const st_plan* p) {
  int64_t rows = 0;
  for (const Shard& s : p->shards) rows += shard_rows(p, s);
  return (int)std::max<int64_t>(1, std::min<int64_t>(kLnMaxParts, rows));
}

bool same_cells(const st_plan* a, const st_plan* b) {
  if (a->ndim != b->ndim || a->batch != b->batch || a->channels != b->channels ||
      a->shards.size() != b->shards.size())
    return false;
  for (int ax = 0; ax < kAxes; ++ax)
    if (a->sizes[ax] != b->sizes[ax]) return false;
  return true;
}

// Fills tensor t of every shard; false where a pointer is NULL or misaligned.
st_status ln_tensor(LnArgs& a, int t, const st_plan* p, const void* const* bufs, const char* name) {
  bool flat = true;
  for (int ax = 0; ax < kAxes; ++ax) flat = flat && p->halo[ax] == 0;
  if (flat) a.flat |= 1 << t;
  for (size_t i = 0; i < p->shards.size(); ++i) {
    if (!bufs[i]) return fail(ST_ERR_INVALID_ARG, std::string(name) + ": NULL shard buffer");
    if (!aligned16(bufs[i])) return fail(ST_ERR_ALIGNMENT, std::string(name) + ": shard buffer not 16-byte aligned");
    const Shard& s = p->shards[i];
    LnTensor& v = a.sh[i].t[t];
    v.sh = s.pad[2];
    v.sd = s.pad[1] * v.sh;
    v.sn = s.pad[0] * v.sd;
    const int64_t first = p->halo[0] * v.sd + p->halo[1] * v.sh + p->halo[2];
    v.p = static_cast<char*>(const_cast<void*>(bufs[i])) + first * p->channels * p->esize;
  }
  return ST_OK;
}

st_status ln_geometry(LnArgs& a, const st_plan* p, const LnPick& pick, bool backward) {
  a.nshards = (int32_t)p->shards.size();
  a.channels = (int32_t)p->channels;
  a.lpr_log2 = pick.lpr_log2;
  a.count = (float)p->channels;
  const int rpb = ln_rows_per_block(pick, backward);
  int64_t rows = 0, blocks = 0;
  for (size_t i = 0; i < p->shards.size(); ++i) {
    const Shard& s = p->shards[i];
    const int64_t n = shard_rows(p, s);
    if (n >= (1ll << 31)) return fail(ST_ERR_UNSUPPORTED, "layer norm: a shard of 2^31 cells or more");
    LnShard& v = a.sh[i];
    v.w = div31((uint32_t)s.ext[2]);
    v.h = div31((uint32_t)s.ext[1]);
    v.d = div31((uint32_t)s.ext[0]);
    v.rows = (int32_t)n;
    v.block_begin = (int32_t)blocks;
    v.row_begin = rows;
    rows += n;
    blocks += (n + rpb - 1) / rpb;
    // (the backward pass steps by up to kLnMaxParts past the last block)
    if (blocks >= (1ll << 31) - kLnMaxParts) return fail(ST_ERR_UNSUPPORTED, "layer norm: too many cells");
  }
  a.blocks = (int32_t)blocks;
  return ST_OK;
}

template <class TX> st_status ln_forward_launch(const LnArgs& a, const LnPick& p, int blocks, hipStream_t st) {
  const dim3 grid(blocks), block(kLnThreads);
#define LN_CASE(V, N, B) \
  if (p.vec == V && p.nv == N && p.block == B) { ln_forward<TX, V, N, B><<<grid, block, 0, st>>>(a); return launch_check("ln_forward"); }
  if constexpr (TX::kSize == 2) {                       // (8 a lane: both sides bf16)
    LN_CASE(8, 1, false) LN_CASE(8, 2, false) LN_CASE(8, 4, false) LN_CASE(8, 8, false)
    LN_CASE(8, 4, true) LN_CASE(8, 8, true)
  }
  LN_CASE(4, 1, false) LN_CASE(4, 2, false) LN_CASE(4, 4, false) LN_CASE(4, 8, false)
  LN_CASE(4, 4, true) LN_CASE(4, 8, true) LN_CASE(4, 16, true)
  LN_CASE(1, 1, false) LN_CASE(1, 4, false) LN_CASE(1, 16, false)
  LN_CASE(1, 16, true) LN_CASE(1, 64, true)
#undef LN_CASE
  return fail(ST_ERR_UNSUPPORTED, "layer norm: no kernel for this width");
}

template <class TX, class TY> st_status ln_backward_launch(const LnArgs& a, const LnPick& p, hipStream_t st) {
  const dim3 grid(a.parts), block(kLnThreads);
#define LN_CASE(V, N, B) \
  if (p.vec == V && p.nv == N && p.block == B) { ln_backward<TX, TY, V, N, B><<<grid, block, 0, st>>>(a); return launch_check("ln_backward"); }
  LN_CASE(8, 1, false) LN_CASE(8, 2, false)
  LN_CASE(8, 1, true) LN_CASE(8, 2, true) LN_CASE(8, 4, true) LN_CASE(8, 8, true)
  LN_CASE(4, 1, false) LN_CASE(4, 2, false) LN_CASE(4, 4, false)
  LN_CASE(4, 2, true) LN_CASE(4, 4, true) LN_CASE(4, 8, true) LN_CASE(4, 16, true)
  LN_CASE(1, 1, false) LN_CASE(1, 4, false) LN_CASE(1, 16, false)
  LN_CASE(1, 16, true) LN_CASE(1, 64, true)
#undef LN_CASE
  return fail(ST_ERR_UNSUPPORTED, "layer norm: no kernel for this width");
}

}  // namespace
}  // namespace st

using namespace st;

extern "C" {

st_status st_layernorm_sharded(const st_plan* x_plan, const void* const* x_bufs, const float* gamma_or_null,
                               const float* beta_or_null, float eps, const st_plan* y_plan, void* const* y_bufs,
                               float* stats_or_null, void* stream) {
  auto err = [](st_status s, const std::string& m) { return fail(s, "st_layernorm_sharded: " + m); };
  if (!x_plan || !x_bufs || !y_plan || !y_bufs) return err(ST_ERR_INVALID_ARG, "NULL argument");
  if (!(eps >= 0.f) || !(eps < 3.0e38f)) return err(ST_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!same_cells(x_plan, y_plan)) return err(ST_ERR_BAD_SHAPE, "x and y plans differ in shape or shard sizes");
  if (x_plan->channels > kLnMaxC) return err(ST_ERR_UNSUPPORTED, "more than 16384 channels");
  if (!aligned16(gamma_or_null) || !aligned16(beta_or_null) || !aligned16(stats_or_null))
    return err(ST_ERR_ALIGNMENT, "gamma, beta or stats not 16-byte aligned");
  LnArgs a{};
  st_status s = ln_tensor(a, 0, x_plan, x_bufs, "st_layernorm_sharded: x");
  if (s != ST_OK) return s;
  s = ln_tensor(a, 1, y_plan, y_bufs, "st_layernorm_sharded: y");
  if (s != ST_OK) return s;
  // 8 values a lane only where both sides are bf16: with an fp32 side, 4 keep its
  // loads dense (1024 x 1792 x 256, fp32 to bf16: 471 -> 458 us)
  const bool wide = x_plan->dtype == ST_BF16 && y_plan->dtype == ST_BF16;
  const LnPick pick = ln_pick((int)x_plan->channels, wide, false);
  s = ln_geometry(a, x_plan, pick, false);
  if (s != ST_OK) return s;
  a.eps = eps;
  a.gamma = gamma_or_null;
  a.beta = beta_or_null;
  a.stats = stats_or_null;
  a.out_bf16 = y_plan->dtype == ST_BF16;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  for (int64_t b = 0; b < a.blocks; b += max_blocks(kLnThreads)) {
    a.block0 = (int32_t)b;
    const int n = (int)std::min<int64_t>(a.blocks - b, max_blocks(kLnThreads));
    s = x_plan->dtype == ST_BF16 ? ln_forward_launch<BF16>(a, pick, n, st) : ln_forward_launch<F32>(a, pick, n, st);
    if (s != ST_OK) return s;
  }
  return ST_OK;
}

size_t st_layernorm_backward_workspace_bytes(const st_plan* x_plan) {
  if (!x_plan || x_plan->channels > kLnMaxC) return 0;
  return (size_t)ln_parts(x_plan) * 2 * (size_t)x_plan->channels * sizeof(float);
}

st_status st_layernorm_backward(const st_plan* x_plan, const void* const* x_bufs, const st_plan* dy_plan,
                                const void* const* dy_bufs, const float* gamma_or_null, const float* stats,
                                const st_plan* dx_plan, void* const* dx_bufs, float* dgamma_or_null,
                                float* dbeta_or_null, void* workspace, size_t workspace_bytes, void* stream) {
  auto err = [](st_status s, const std::string& m) { return fail(s, "st_layernorm_backward: " + m); };
  if (!x_plan || !x_bufs || !dy_plan || !dy_bufs || !dx_plan || !dx_bufs || !stats)
    return err(ST_ERR_INVALID_ARG, "NULL argument");
  if (!same_cells(x_plan, dy_plan) || !same_cells(x_plan, dx_plan))
    return err(ST_ERR_BAD_SHAPE, "x, dy and dx plans differ in shape or shard sizes");
  if (x_plan->channels > kLnMaxC) return err(ST_ERR_UNSUPPORTED, "more than 16384 channels");
  if (!aligned16(gamma_or_null) || !aligned16(stats) || !aligned16(dgamma_or_null) || !aligned16(dbeta_or_null) ||
      !aligned16(workspace))
    return err(ST_ERR_ALIGNMENT, "gamma, stats, dgamma, dbeta or workspace not 16-byte aligned");
  if (!workspace || workspace_bytes < st_layernorm_backward_workspace_bytes(x_plan))
    return err(ST_ERR_WORKSPACE, "workspace missing or too small");
  LnArgs a{};
  st_status s = ln_tensor(a, 0, x_plan, x_bufs, "st_layernorm_backward: x");
  if (s != ST_OK) return s;
  s = ln_tensor(a, 1, dy_plan, dy_bufs, "st_layernorm_backward: dy");
  if (s != ST_OK) return s;
  s = ln_tensor(a, 2, dx_plan, dx_bufs, "st_layernorm_backward: dx");
  if (s != ST_OK) return s;
  // 8 values a lane with any bf16 side: the same volume's backward pass takes
  // 906 us with 8 and 1028 us with 4 (half as many bytes in flight)
  const bool wide = x_plan->dtype == ST_BF16 || dy_plan->dtype == ST_BF16 || dx_plan->dtype == ST_BF16;
  const LnPick pick = ln_pick((int)x_plan->channels, wide, true);
  s = ln_geometry(a, x_plan, pick, true);
  if (s != ST_OK) return s;
  a.gamma = gamma_or_null;
  a.stats = const_cast<float*>(stats);
  a.partial = static_cast<float*>(workspace);
  a.parts = std::min(ln_parts(x_plan), a.blocks);
  a.out_bf16 = dx_plan->dtype == ST_BF16;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool xb = x_plan->dtype == ST_BF16, yb = dy_plan->dtype == ST_BF16;
  s = xb ? (yb ? ln_backward_launch<BF16, BF16>(a, pick, st) : ln_backward_launch<BF16, F32>(a, pick, st))
         : (yb ? ln_backward_launch<F32, BF16>(a, pick, st) : ln_backward_launch<F32, F32>(a, pick, st));
  if (s != ST_OK || (!dgamma_or_null && !dbeta_or_null)) return s;
  ln_columns<<<(2 * a.channels + 15) / 16, 256, 0, st>>>(a.partial, a.parts, a.channels, dgamma_or_null,
                                                         dbeta_or_null);
  return launch_check("ln_columns");
}

}  // extern "C"
