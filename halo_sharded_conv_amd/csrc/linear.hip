// Matrix products with bias, activation and residual in their epilogue, and the
// gradients' products.
//
//   forward  y[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n]
//   dx[m][k] = sum_n p[m][n] w[n][k]      (w read across its rows)
//   dw[n][k] = sum_m p[m][n] x[m][k]      (both read across their rows)
// One kernel for all three: an operand whose contraction is not contiguous lies in
// LDS as it lies in memory and is read by the transposing LDS read, so nothing is
// transposed in memory.
#include <cmath>

#include "linear.h"

namespace st {
namespace {

struct GemmArgs {
  Rows a, b;
  Finish f;
  float* part;                        // partial sums [split][m][ld], or NULL
  int64_t ld;
  int32_t m, n, k;
  int32_t kbytes;                     // k in bytes (contraction contiguous)
  int32_t tiles_a, tiles_b, splits, per_split, stages;
  int32_t blocks_k;                   // 8-bit: scale blocks along k
};

template <class T, bool AC, bool BC, int TA, int TB, int WA, int WB, int OCC>
__global__ __launch_bounds__(64 * WA * WB, OCC) void gemm(const GemmArgs g) {
  constexpr int NW = WA * WB, PA = TA / WA, PB = TB / WB, NA = PA / 32, NB = PB / 32;
  using P = Prod<T>;
  using OA = Oper<T, AC, TA, NW>;
  using OB = Oper<T, BC, TB, NW>;
  constexpr int KT = OA::KT, NI = OA::NI + OB::NI;
  constexpr bool EXACT = std::is_same<T, MX8X>::value, MX = std::is_same<T, MX8>::value || EXACT;
  __shared__ __attribute__((aligned(1024))) char a0[OA::BYTES];
  __shared__ __attribute__((aligned(1024))) char a1[OA::BYTES];
  __shared__ __attribute__((aligned(1024))) char a2[OA::BYTES];
  __shared__ __attribute__((aligned(1024))) char b0[OB::BYTES];
  __shared__ __attribute__((aligned(1024))) char b1[OB::BYTES];
  __shared__ __attribute__((aligned(1024))) char b2[OB::BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, wa = wave % WA, wb = wave / WA;

  // workgroups go round the 8 XCDs: each takes a run of tiles, eight row tiles
  // deep, so that what its L2 holds is shared
  int ta, tb, split;
  {
    const uint32_t total = gridDim.x, id = blockIdx.x, x = id & 7, per = total >> 3, more = total & 7;
    uint32_t t = x * per + min(x, more) + (id >> 3);
    const uint32_t tiles = (uint32_t)g.tiles_a * g.tiles_b;
    split = t / tiles;
    t -= split * tiles;
    const uint32_t deep = 8, group = deep * g.tiles_a, gi = t / group, first = gi * deep;
    const uint32_t in = t - gi * group, d = min(deep, g.tiles_b - first);
    tb = first + in % d;
    ta = in / d;
  }
  const int n0 = ta * TA, m0 = tb * TB;
  const int k_lo = split * g.per_split, k_hi = min(g.stages, k_lo + g.per_split);

  // this lane's transfers: byte offsets from a stage's base
  uint32_t offa[OA::NI], offb[OB::NI];
#pragma unroll
  for (int i = 0; i < OA::NI; ++i) {
    const int r = OA::dma_row(wave, lane, i), b = OA::dma_byte(wave, lane, i);
    offa[i] = AC && n0 * T::kSize + b >= g.n * T::kSize ? kPastEnd : (uint32_t)(r * (int)g.a.stride + b);
  }
#pragma unroll
  for (int i = 0; i < OB::NI; ++i) {
    const int r = OB::dma_row(wave, lane, i), b = OB::dma_byte(wave, lane, i);
    offb[i] = BC && m0 * T::kSize + b >= g.m * T::kSize ? kPastEnd : (uint32_t)(r * (int)g.b.stride + b);
  }
  const char* pa = AC ? g.a.p + (int64_t)n0 * T::kSize : g.a.p + (int64_t)n0 * g.a.stride;
  const char* pb = BC ? g.b.p + (int64_t)m0 * T::kSize : g.b.p + (int64_t)m0 * g.b.stride;
  // scale bytes of this lane's rows (8-bit operands)
  uint32_t soa[MX ? NA : 1], sob[MX ? NB : 1];
  int sa[MX ? NA : 1], sb[MX ? NB : 1];
  if constexpr (MX) {
#pragma unroll
    for (int i = 0; i < NA; ++i) soa[i] = (uint32_t)((wa * PA + 32 * i + (lane & 31)) * (int)g.a.scale_stride + half);
#pragma unroll
    for (int i = 0; i < NB; ++i) sob[i] = (uint32_t)((wb * PB + 32 * i + (lane & 31)) * (int)g.b.scale_stride + half);
  }

  // Stage kt's transfers.  Past the last stage nothing is read: the transfers write
  // zeros, so that every step waits for the same number of them.
  const int sta = (int)g.a.stride, stb = (int)g.b.stride;
  auto fetch = [&](char* as, char* bs, int kt) __attribute__((always_inline)) {
    const int left = g.kbytes - kt * 64;                // bytes of the contraction from here on
    const int rows = min(g.k - kt * KT, KT);            // its steps of this stage
    const int na = AC ? rows * sta : min(TA, g.n - n0) * sta, nb = BC ? rows * stb : min(TB, g.m - m0) * stb;
    const auto ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(AC ? pa + (int64_t)kt * KT * sta : pa), (short)0,
                                                      kt < k_hi ? na : 0, 0x00020000);
    const auto rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(BC ? pb + (int64_t)kt * KT * stb : pb), (short)0,
                                                      kt < k_hi ? nb : 0, 0x00020000);
#pragma unroll
    for (int i = 0; i < OA::NI; ++i) {
      const uint32_t at = !AC && OA::dma_byte(wave, lane, i) >= left ? kPastEnd : offa[i];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void)OA::dma_dst(as, wave, i), 16, at, AC ? 0 : kt * 64, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < OB::NI; ++i) {
      const uint32_t at = !BC && OB::dma_byte(wave, lane, i) >= left ? kPastEnd : offb[i];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void)OB::dma_dst(bs, wave, i), 16, at, BC ? 0 : kt * 64, 0, 0);
    }
  };
  auto scales = [&](int kt) __attribute__((always_inline)) {
    if constexpr (MX) {
      const auto ra = rows_rsrc(g.a.scales + (int64_t)n0 * g.a.scale_stride, (int64_t)min(TA, g.n - n0) * g.a.scale_stride);
      const auto rb = rows_rsrc(g.b.scales + (int64_t)m0 * g.b.scale_stride, (int64_t)min(TB, g.m - m0) * g.b.scale_stride);
      // (past the last block the codes are zero; a scale byte there may be NaN's)
      const uint32_t none = 2 * kt + half >= g.blocks_k ? kPastEnd : 0u;
#pragma unroll
      for (int i = 0; i < NA; ++i) sa[i] = __builtin_amdgcn_raw_buffer_load_b8(ra, none | soa[i], 2 * kt, 0);
#pragma unroll
      for (int i = 0; i < NB; ++i) sb[i] = __builtin_amdgcn_raw_buffer_load_b8(rb, none | sob[i], 2 * kt, 0);
    }
  };

  f32x16 acc[NA][NB];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};

  // Stage kt in (as, bs); stage kt + 2 goes to (an, bn), which every wave has
  // finished reading once it is past the barrier.  The NI transfers of stage kt + 1
  // may still be under way behind the barrier.
  auto step = [&](const char* as, const char* bs, char* an, char* bn, int kt) __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (NI & 15) | (NI >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    int ca[MX ? NA : 1], cb[MX ? NB : 1];
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < NA; ++i) ca[i] = sa[i];
#pragma unroll
      for (int i = 0; i < NB; ++i) cb[i] = sb[i];
      scales(kt + 1);
      asm volatile("" ::: "memory");                    // (ahead of the transfers: the next step's wait covers them)
    }
    fetch(an, bn, kt + 2);
#pragma unroll
    for (int s = 0; s < P::STEPS; ++s) {
      typename P::Frag fa[NA], fb[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if constexpr (EXACT) fb[j] = P::widen(P::template raw<BC, TB, NW>(bs, wb * NB + j, lane), cb[j]);
        else fb[j] = P::template frag<BC, TB, NW>(bs, wb * NB + j, s, lane);
      }
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        if constexpr (EXACT) fa[i] = P::widen(P::template raw<AC, TA, NW>(as, wa * NA + i, lane), ca[i]);
        else fa[i] = P::template frag<AC, TA, NW>(as, wa * NA + i, s, lane);
      }
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = P::mul(fa[i], fb[j], acc[i][j], MX ? ca[MX ? i : 0] : 0, MX ? cb[MX ? j : 0] : 0);
    }
  };

  scales(k_lo);
  fetch(a0, b0, k_lo);
  asm volatile("" ::: "memory");                        // (the first step's wait counts on this order)
  fetch(a1, b1, k_lo + 1);
  int kt = k_lo;
  for (; kt + 3 <= k_hi; kt += 3) {
    step(a0, b0, a2, b2, kt);
    step(a1, b1, a0, b0, kt + 1);
    step(a2, b2, a1, b1, kt + 2);
  }
  if (kt < k_hi) step(a0, b0, a2, b2, kt);
  if (kt + 1 < k_hi) step(a1, b1, a0, b0, kt + 1);
  __builtin_amdgcn_s_waitcnt(0x0070);                   // (no transfer outlives the workgroup's LDS)

#pragma unroll 1
  for (int t = 0; t < NA * NB; ++t) {                   // one copy of the epilogue for all blocks
    float v[16];
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if (t == i * NB + j) {
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] = acc[i][j][r];
        }
    const int64_t m = m0 + wb * PB + 32 * (t % NB) + (lane & 31);
    const int n = n0 + wa * PA + 32 * (t / NB);
    if (!g.part) {
      finish_block(g.f, m, n, half, v);
    } else if (m < g.m && n < g.n) {
      float* p = g.part + ((int64_t)split * g.m + m) * g.ld + n + 4 * half;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4_t*>(p + 8 * q) = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    }
  }
}

// Adds the splits' partial sums in order and finishes the blocks, one a wave
__global__ __launch_bounds__(256) void gemm_join(const float* __restrict__ part, int splits, int64_t ld, Finish f, int blocks_n, int64_t blocks) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int64_t blk = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (blk >= blocks) return;
  const int64_t m = blk / blocks_n * 32 + (lane & 31);
  const int n0 = (int)(blk % blocks_n) * 32;
  float v[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) v[r] = 0.f;
  if (m < f.rows) {
    const float* p = part + m * ld + n0 + 4 * half;
    for (int s = 0; s < splits; ++s, p += (int64_t)f.rows * ld) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t t = *reinterpret_cast<const f32x4_t*>(p + 8 * q);
        v[4 * q] += t.x; v[4 * q + 1] += t.y; v[4 * q + 2] += t.z; v[4 * q + 3] += t.w;
      }
    }
  }
  finish_block(f, m, n0, half, v);
}

// ------------------------------------------------------------------ host

struct Shape {                        // tile and what a compute unit holds of it
  int ta, tb, per_cu;
};
// large and small tile; fp32 (products a ninth as fast, twice the registers per
// fragment) stays with 128 x 128
constexpr Shape kShapes[2][2] = {{{256, 128, 2}, {128, 64, 4}}, {{128, 128, 2}, {128, 64, 4}}};
inline const Shape& shape_of(int type, int s) { return kShapes[type == ST_F32][s]; }
constexpr int kCus = 256;

struct Choice {
  int shape, splits, per_split;
};

// Tile shape and split of the contraction: the cheapest by rounds over the compute
// units (a stage's time goes with the tile's area; a tile's start and end cost
// as much as some stages) plus the partial sums' way through memory.
// exact: 8-bit operands with an fp32 output, which the small tile alone has.
Choice choose(int64_t m, int64_t n, int64_t k, int type, bool exact) {
  const int kt = type == ST_F32 ? 16 : type == ST_BF16 ? 32 : 64;
  const int64_t stages = (k + kt - 1) / kt;
  Choice best{};
  double least = INFINITY;
  for (int s = exact ? 1 : 0; s < 2; ++s) {
    const Shape& h = shape_of(type, s);
    const int64_t tiles = (n + h.ta - 1) / h.ta * ((m + h.tb - 1) / h.tb);
    // microseconds of one stage of a full compute unit
    const double stage = (type == ST_F32 ? 4.0 : 1.0) * h.ta * h.tb * h.per_cu / 65536.0 * (s ? 0.65 : 0.55);
    for (int64_t splits = 1; splits <= 64; splits = splits < 4 ? splits + 1 : splits * 5 / 4) {
      const int64_t per = (stages + splits - 1) / splits, real = (stages + per - 1) / per;
      if (splits > 1 && (real != splits || per < 4)) continue;
      const double rounds = std::ceil((double)tiles * splits / (kCus * h.per_cu));
      const double fill = std::min(1.0, (double)tiles * splits / (kCus * h.per_cu));
      double t = rounds * (per * stage * std::max(fill, 1.0 / h.per_cu) + 2.0);
      if (splits > 1) t += 4.0 + (double)m * n * 4 * (splits * 2) / 4.0e6;
      if (t < least) { least = t; best = Choice{s, (int)splits, (int)per}; }
    }
  }
  return best;
}
int64_t part_ld(int64_t n) { return (n + 31) / 32 * 32; }

template <class T, bool AC, bool BC> st_status gemm_launch(const GemmArgs& g, int shape, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)g.tiles_a * g.tiles_b * g.splits);
  if (shape == 0 && std::is_same<T, F32>::value) gemm<F32, AC, BC, 128, 128, 2, 2, 2><<<grid, 256, 0, st>>>(g);
  else if (shape == 0) gemm<typename std::conditional<std::is_same<T, F32>::value, BF16, T>::type, AC, BC, 256, 128, 2, 2, 2><<<grid, 256, 0, st>>>(g);
  else gemm<T, AC, BC, 128, 64, 2, 2, 4><<<grid, 256, 0, st>>>(g);
  return launch_check("gemm");
}

}  // namespace

size_t product_bytes(int64_t m, int64_t n, int64_t k, int type) {
  if (m <= 0 || n <= 0 || k <= 0) return 0;
  size_t most = 0;
  for (int exact = 0; exact <= (type == ST_MX8); ++exact) {
    const Choice c = choose(m, n, k, type, exact);
    if (c.splits > 1) most = std::max(most, (size_t)c.splits * (size_t)m * (size_t)part_ld(n) * 4);
  }
  return most;
}

st_status product_launch(const Product& p, void* workspace, hipStream_t st) {
  if (p.k == 0) {                                       // an empty sum: the epilogue of zeros
    const int bn = (int)(part_ld(p.n) / 32);
    const int64_t blocks = (p.m + 31) / 32 * bn;
    if ((blocks + 3) / 4 > max_blocks(256)) return fail(ST_ERR_UNSUPPORTED, "matrix product: too many blocks for one launch");
    gemm_join<<<(unsigned)((blocks + 3) / 4), 256, 0, st>>>(nullptr, 0, 0, p.f, bn, blocks);
    return launch_check("gemm_join");
  }
  const bool exact = p.type == ST_MX8 && (p.f.y.type == ST_F32 || p.f.pre.type == ST_F32);
  const Choice c = choose(p.m, p.n, p.k, p.type, exact);
  const Shape& h = shape_of(p.type, c.shape);
  const int es = type_size(p.type), kt = 64 / es;
  GemmArgs g{};
  g.a = p.a;
  g.b = p.b;
  g.f = p.f;
  g.m = (int32_t)p.m;
  g.n = (int32_t)p.n;
  g.k = (int32_t)p.k;
  g.kbytes = (int32_t)(p.k * es);
  g.blocks_k = (int32_t)((p.k + kMxBlock - 1) / kMxBlock);
  g.stages = (int32_t)((p.k + kt - 1) / kt);
  g.splits = c.splits;
  g.per_split = c.per_split;
  g.ld = part_ld(p.n);
  g.part = c.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  const int64_t ta = (p.n + h.ta - 1) / h.ta, tb = (p.m + h.tb - 1) / h.tb;
  if (ta * tb * c.splits > max_blocks(256)) return fail(ST_ERR_UNSUPPORTED, "matrix product: too many tiles for one launch");
  g.tiles_a = (int32_t)ta;
  g.tiles_b = (int32_t)tb;
  st_status s;
  if (exact) {
    gemm<MX8X, false, false, 128, 64, 2, 2, 2><<<(unsigned)(ta * tb * c.splits), 256, 0, st>>>(g);
    s = launch_check("gemm");
  } else if (p.type == ST_MX8) s = gemm_launch<MX8, false, false>(g, c.shape, st);
  else if (p.type == ST_BF16)
    s = p.b_col ? gemm_launch<BF16, true, true>(g, c.shape, st)
        : p.a_col ? gemm_launch<BF16, true, false>(g, c.shape, st) : gemm_launch<BF16, false, false>(g, c.shape, st);
  else
    s = p.b_col ? gemm_launch<F32, true, true>(g, c.shape, st)
        : p.a_col ? gemm_launch<F32, true, false>(g, c.shape, st) : gemm_launch<F32, false, false>(g, c.shape, st);
  if (s != ST_OK || c.splits == 1) return s;
  const int bn = (int)(g.ld / 32);
  const int64_t blocks = (p.m + 31) / 32 * bn;
  if ((blocks + 3) / 4 > max_blocks(256)) return fail(ST_ERR_UNSUPPORTED, "matrix product: too many blocks for one launch");
  gemm_join<<<(unsigned)((blocks + 3) / 4), 256, 0, st>>>(g.part, c.splits, g.ld, g.f, bn, blocks);
  return launch_check("gemm_join");
}

}  // namespace st
