// Attention over packed sequences: backward.
//
// With p = exp(s - lse) of the forward pass, D = sum over channels of
// dout * out, dp = dout v^T and ds = p * (dp - D):
//   dv = p^T dout,   dk = scale * ds^T q,   dq = scale * ds k
// Two kernels, each with its sums in registers from the first product to the
// store: attn_dq walks the keys for a tile of rows, attn_dkv the rows for a
// tile of keys.  The scores are formed in both (7 products where one kernel
// would need 5), and in return no sum is ever added to memory by several
// workgroups: no atomics, the same bits on every run.
//
// As in the forward pass a lane keeps one row (attn_dq) or one key (attn_dkv)
// of every product, and p and ds go from product to product in registers.
// Rows are (token, head of the group) pairs, so the gradients of a shared
// key-value head are summed over its group inside attn_dkv's loop.
//
// Bound: the matrix cores.  Measured with 4 x 4096 tokens, 16 heads of 128:
// attn_dq 720 us (1145 TFLOP/s of its 3 products), attn_dkv 1050 us (1045 of its
// 4); 2 x 8192 tokens, 16 heads of 64: 750 and 1090 us.  Causal 8192 tokens, 16 / 2
// heads of 128: 379 and 683 us; there the rows of a group (67 MB of q and dout)
// pass by every tile of keys from beyond the L2.  Walking the rows from the last
// one down, so that the tiles of keys share them, was no faster.
#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "attention.h"

namespace st {
namespace {

// ---------------------------------------------------------------------- dq

// waves per SIMD that the registers allow
template <class T, int DP> constexpr int dq_waves() { return DP * T::kSize > 256 ? 1 : DP * T::kSize > 128 ? 2 : 3; }

template <class T, int DP, int KT, int NW>
__global__ __launch_bounds__(64 * NW, (dq_waves<T, DP>())) void attn_dq(const AttnArgs a) {
  using M = Mma<T>;
  using Tl = Tile<T, DP, KT, NW>;
  constexpr int KB = KT / 32, SR = Tl::SR, DB = Tl::DB, NI = Tl::NI;
  __shared__ __attribute__((aligned(1024))) char k0s[Tl::BYTES];
  __shared__ __attribute__((aligned(1024))) char v0s[Tl::BYTES];
  __shared__ __attribute__((aligned(1024))) char k1s[Tl::BYTES];
  __shared__ __attribute__((aligned(1024))) char v1s[Tl::BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int kvh = blockIdx.x % a.kv_heads;
  const AttnItem it = a.items[blockIdx.x / a.kv_heads];

  const int row0 = it.at + wave * 32, row = row0 + l32;
  const int token = (int)quo(row, a.by_group), head = kvh * a.group + row - token * a.group;
  const bool live = token < it.lq;
  const int off = it.lk - it.lq;
  const int limit = a.causal ? min(it.lk, token + off + 1) : it.lk;
  const int all = min(it.hi, a.causal ? (int)quo(it.at, a.by_group) + off + 1 : it.lk);   // seen by every row
  const int wave_last = a.causal ? min(it.lk, (int)quo(row0 + 31, a.by_group) + off + 1) : it.lk;

  typename M::Row qf[SR], gf[SR];
  float delta = 0.f;
  {
    const char* pq = a.q.p + (int64_t)(it.q0 + token) * a.q.t + (int64_t)head * a.q.h;
    const char* pg = a.dout.p + (int64_t)(it.q0 + token) * a.dout.t + (int64_t)head * a.dout.h;
    const char* po = a.out.p + (int64_t)(it.q0 + token) * a.out.t + (int64_t)head * a.out.h;
#pragma unroll
    for (int s = 0; s < SR; ++s) {
      const int byte = (2 * s + half) * 16;
      const bool in = live && byte < a.dim * T::kSize;
      qf[s] = in ? *reinterpret_cast<const typename M::Row*>(pq + byte) : typename M::Row{};
      gf[s] = in ? *reinterpret_cast<const typename M::Row*>(pg + byte) : typename M::Row{};
      const typename M::Row of = in ? *reinterpret_cast<const typename M::Row*>(po + byte) : typename M::Row{};
#pragma unroll
      for (int i = 0; i < 16 / T::kSize; ++i) delta = fmaf((float)gf[s][i], (float)of[i], delta);
    }
  }
  delta = half_sum(delta);
  const int64_t stat = (int64_t)(it.q0 + token) * a.heads + head;
  // exp2(s - lse2): +inf (p = 0) for rows past the end and rows without keys
  float lse2 = INFINITY;
  if (live) {
    lse2 = a.lse[stat] * kLog2e;
    if (lse2 == -INFINITY) lse2 = INFINITY;
  }
  uint32_t koff[NI], voff[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = Tl::dma_row(wave, lane, i), b = Tl::dma_byte(wave, lane, i);
    const bool in = b < a.dim * T::kSize;
    koff[i] = in ? (uint32_t)(r * (int)a.k.t + b) : kOobOffset;
    voff[i] = in ? (uint32_t)(r * (int)a.v.t + b) : kOobOffset;
  }
  const char* kb = a.k.p + (int64_t)it.k0 * a.k.t + (int64_t)kvh * a.k.h;
  const char* vb = a.v.p + (int64_t)it.k0 * a.v.t + (int64_t)kvh * a.v.h;

  f32x16 dq[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) dq[d] = f32x16{};

  auto fetch = [&](char* ks, char* vs, int j0) __attribute__((always_inline)) {
    const int64_t left = min(KT, it.hi - j0);
    const auto rk = attn_rsrc(kb + (int64_t)j0 * a.k.t, left * a.k.t);
    const auto rv = attn_rsrc(vb + (int64_t)j0 * a.v.t, left * a.v.t);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t at = koff[i];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (lds_void)Tl::dma_dst(ks, wave, i), 16, at, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t at = voff[i];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (lds_void)Tl::dma_dst(vs, wave, i), 16, at, 0, 0, 0);
    }
  };
  auto step = [&](auto MASKED, const char* ks, const char* vs, char* kn, char* vn, int j0) __attribute__((always_inline)) {
    constexpr bool masked = decltype(MASKED)::value;
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    if (j0 + KT < it.hi) fetch(kn, vn, j0 + KT);
    if (masked && j0 >= wave_last) return;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
      for (int c = 0; c < SR; ++c) {
        s = M::rows(Tl::row(ks, b, c, lane), qf[c], s);
        dp = M::rows(Tl::row(vs, b, c, lane), gf[c], dp);
      }
      if constexpr (masked) {
        const int lim = limit - j0 - 4 * half;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const bool seen = 32 * b + 8 * (r / 4) + r % 4 < lim;
          s[r] = seen ? exp2_hw(fmaf(s[r], a.scale_log2, -lse2)) : 0.f;
          dp[r] = seen ? dp[r] : 0.f;
        }
        if (b == 0 && j0 == 0) {
          // A row with all its keys in these 32 takes D as the sum of p dp in
          // fp32: `out` is rounded to its type, and with few keys that rounding
          // is as large as all others together.  (32: the block of scores that a lane
          // pair holds at once; more keys would need a pass before the first ds.)  A
          // single key weighs exactly one, so that nothing is left of dq and dk.
          float d = (limit == 1 ? 1.f : s[0]) * dp[0];
#pragma unroll
          for (int r = 1; r < 16; ++r) d = fmaf(s[r], dp[r], d);
          d = half_sum(d);
          delta = limit <= 32 ? d : delta;
        }
        __builtin_amdgcn_sched_barrier(0);              // (few tiles: registers before speed)
#pragma unroll
        for (int r = 0; r < 16; ++r) dp[r] = s[r] * (dp[r] - delta);
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) dp[r] = exp2_hw(fmaf(s[r], a.scale_log2, -lse2)) * (dp[r] - delta);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const typename M::Col p = M::regs(dp, t);
#pragma unroll
        for (int d = 0; d < DB; ++d) dq[d] = M::cols(Tl::col(ks, b, t, d, lane), p, dq[d]);
      }
    }
  };
  if (it.lo < it.hi) {
    fetch(k0s, v0s, it.lo);
    const int first_masked = it.lo + max(0, (all - it.lo) / (2 * KT)) * (2 * KT);
    int j = it.lo;
    for (; j < first_masked; j += 2 * KT) {
      step(std::false_type{}, k0s, v0s, k1s, v1s, j);
      step(std::false_type{}, k1s, v1s, k0s, v0s, j + KT);
    }
    for (; j < it.hi; j += 2 * KT) {
      step(std::true_type{}, k0s, v0s, k1s, v1s, j);
      if (j + KT < it.hi) step(std::true_type{}, k1s, v1s, k0s, v0s, j + KT);
    }
  }
  if (live && half == 0 && it.lo == 0) a.delta[stat] = delta;   // the tile's first part writes it
  if (it.part >= 0) {
    const int64_t slot = ((int64_t)it.part * a.kv_heads + kvh) * (32 * NW) + wave * 32 + l32;
#pragma unroll
    for (int d = 0; d < DB; ++d)
      store_block<F32>(reinterpret_cast<char*>(a.part + slot * DP), dq[d], a.scale, d, DP, lane);
    return;
  }
  if (!live) return;
  char* p = a.dq.p + (int64_t)(it.q0 + token) * a.dq.t + (int64_t)head * a.dq.h;
#pragma unroll
  for (int d = 0; d < DB; ++d) store_block<T>(p, dq[d], a.scale, d, a.dim, lane);
}

// ------------------------------------------------------------------ dk, dv

// The lane index of a step.  The fp32 col fragments of a wide head have 64
// different LDS addresses: FRESH forms them in each step, a few instructions
// under long products, where held over the loop they spill (8 heads of 128,
// 4096 tokens: 2524 -> 1104 us).  Everywhere else the compiler's choice to hold
// them is 5 to 13% faster.
template <bool FRESH> struct LaneOf {
  static __device__ __forceinline__ int of(int lane) {
    if constexpr (FRESH) asm volatile("" : "+v"(lane));
    return lane;
  }
};

// waves per SIMD that the registers allow: K, V and the sums of dk and dv
template <class T, int DP> constexpr int dkv_waves() { return DP * T::kSize > 128 ? 1 : 2; }

template <class T, int DP, int RT, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(dkv_waves<T, DP>(), dkv_waves<T, DP>())))
void attn_dkv(const AttnArgs a) {
  using M = Mma<T>;
  using Tl = Tile<T, DP, RT, NW>;
  constexpr int RB = RT / 32, SR = Tl::SR, DB = Tl::DB, NI = Tl::NI;
  constexpr bool PIPE = T::kSize == 2 && RB == 2 && dkv_waves<T, DP>() == 1;
  // wide fp32 heads: V in LDS beside the tiles, its registers for the sums
  using Tv = Tile<T, DP, 32 * NW, NW>;
  constexpr bool VL = T::kSize == 4 && DP > 64;
  struct Stats { float lse2[RT], delta[RT]; int limit[RT]; };
  __shared__ __attribute__((aligned(1024))) char q0s[Tl::BYTES];
  __shared__ __attribute__((aligned(1024))) char g0s[Tl::BYTES];
  __shared__ __attribute__((aligned(1024))) char q1s[Tl::BYTES];
  __shared__ __attribute__((aligned(1024))) char g1s[Tl::BYTES];
  __shared__ __attribute__((aligned(1024))) char vls[VL ? Tv::BYTES : 16];
  __shared__ __attribute__((aligned(16))) Stats st0, st1;
  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int kvh = blockIdx.x % a.kv_heads;
  const AttnItem it = a.items[blockIdx.x / a.kv_heads];
  const int off = it.lk - it.lq;
  const int key0 = it.at + wave * 32, key = key0 + l32;
  const bool live = key < it.lk;

  typename M::Row kf[SR], vf[VL ? 1 : SR];
  {
    const char* pk = a.k.p + (int64_t)(it.k0 + key) * a.k.t + (int64_t)kvh * a.k.h;
    const char* pv = a.v.p + (int64_t)(it.k0 + key) * a.v.t + (int64_t)kvh * a.v.h;
#pragma unroll
    for (int s = 0; s < SR; ++s) {
      const int byte = (2 * s + half) * 16;
      const bool in = live && byte < a.dim * T::kSize;
      kf[s] = in ? *reinterpret_cast<const typename M::Row*>(pk + byte) : typename M::Row{};
      if constexpr (!VL) vf[s] = in ? *reinterpret_cast<const typename M::Row*>(pv + byte) : typename M::Row{};
    }
  }
  if (VL && it.lo < it.hi) {                            // (in LDS before the first tile is read: step's wait and barrier)
    const int64_t left = min(32 * NW, it.lk - it.at);
    const auto rv = attn_rsrc(a.v.p + (int64_t)(it.k0 + it.at) * a.v.t + (int64_t)kvh * a.v.h, left * a.v.t);
#pragma unroll
    for (int i = 0; i < Tv::NI; ++i) {
      const int r = Tv::dma_row(wave, lane, i), b = Tv::dma_byte(wave, lane, i);
      const uint32_t at = b < a.dim * T::kSize ? (uint32_t)(r * (int)a.v.t + b) : kOobOffset;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (lds_void)Tv::dma_dst(vls, wave, i), 16, at, 0, 0, 0);
    }
  }
  f32x16 dk[DB], dv[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) { dk[d] = f32x16{}; dv[d] = f32x16{}; }

  const char* qb = a.q.p + (int64_t)it.q0 * a.q.t + (int64_t)kvh * a.group * a.q.h;
  const char* gb = a.dout.p + (int64_t)it.q0 * a.dout.t + (int64_t)kvh * a.group * a.dout.h;
  const float* lb = a.lse + (int64_t)it.q0 * a.heads + kvh * a.group;
  const float* db = a.delta + (int64_t)it.q0 * a.heads + kvh * a.group;

  uint32_t byte[NI];                                    // this lane's byte of a row per transfer
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int b = Tl::dma_byte(wave, lane, i);
    byte[i] = b < a.dim * T::kSize ? (uint32_t)b : kOobOffset;
  }
  // rows [r0, r0 + RT): offsets from the tile's first token, zeros past the range
  auto fetch = [&](char* qs, char* gs, int r0) __attribute__((always_inline)) {
    const int t0 = __builtin_amdgcn_readfirstlane((int)quo(r0, a.by_group));
    const auto rq = attn_rsrc(qb + (int64_t)t0 * a.q.t, 0x7FFFFFFF);
    const auto rg = attn_rsrc(gb + (int64_t)t0 * a.dout.t, 0x7FFFFFFF);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = r0 + Tl::dma_row(wave, lane, i);
      const int token = (int)quo(r, a.by_group), g = r - token * a.group;
      const uint32_t tq = (uint32_t)((token - t0) * (int)a.q.t + g * (int)a.q.h) + byte[i];
      const uint32_t tg = (uint32_t)((token - t0) * (int)a.dout.t + g * (int)a.dout.h) + byte[i];
      const uint32_t oq = r < it.hi ? tq : kOobOffset, og = r < it.hi ? tg : kOobOffset;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (lds_void)Tl::dma_dst(qs, wave, i), 16, oq, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rg, (lds_void)Tl::dma_dst(gs, wave, i), 16, og, 0, 0, 0);
    }
  };
  // thread tid's row statistics of a tile: loaded ahead, put into LDS at the
  // end of the step before
  auto stats = [&](int r0, float& lse, float& delta) __attribute__((always_inline)) {
    const int r = r0 + tid;
    lse = -INFINITY;
    delta = 0.f;
    if (tid < RT && r < it.hi) {
      const int token = (int)quo(r, a.by_group), g = r - token * a.group;
      const int64_t at = (int64_t)token * a.heads + g;
      lse = lb[at];
      delta = db[at];
    }
  };
  auto put = [&](Stats& s, int r0, float lse, float delta) __attribute__((always_inline)) {
    if (tid < RT) {
      // p = 0 for rows past the range and rows without keys
      s.lse2[tid] = lse == -INFINITY ? INFINITY : lse * kLog2e;
      s.delta[tid] = delta;
      s.limit[tid] = a.causal ? (int)quo(r0 + tid, a.by_group) + off + 1 : it.lk;
    }
  };

  // one tile: MASKED where some row may not see some key
  auto step = [&](auto MASKED, const char* qs, const char* gs, const Stats& sc, char* qn, char* gn, Stats& sn, int r0)
      __attribute__((always_inline)) {
    constexpr bool masked = decltype(MASKED)::value;
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    const bool more = r0 + RT < it.hi;
    const int ln = LaneOf<VL>::of(lane);
    float lsen, deltan;
    if (more) {
      fetch(qn, gn, r0 + RT);
      stats(r0 + RT, lsen, deltan);
    }
    // (uniform) rows below all of this wave's keys see none of them
    const int last = min(it.hi, r0 + RT) - 1;
    {
      auto scores = [&](int b, f32x16& s, f32x16& dp) __attribute__((always_inline)) {
        s = f32x16{};
        dp = f32x16{};
#pragma unroll
        for (int c = 0; c < SR; ++c) {
          s = M::rows(Tl::row(qs, b, c, ln), kf[c], s);
          if constexpr (VL) dp = M::rows(Tl::row(gs, b, c, ln), Tv::row(vls, wave, c, ln), dp);
          else dp = M::rows(Tl::row(gs, b, c, ln), vf[c], dp);
          if constexpr (VL) __builtin_amdgcn_sched_barrier(0);   // no reads hoisted into registers that are not there
        }
      };
      auto weights = [&](int b, f32x16& s, f32x16& dp) __attribute__((always_inline)) {   // s -> p, dp -> ds
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const int at = 32 * b + 8 * r4 + 4 * half;
          const f32x4_t l4 = *reinterpret_cast<const f32x4_t*>(&sc.lse2[at]);
          const f32x4_t d4 = *reinterpret_cast<const f32x4_t*>(&sc.delta[at]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 4 * r4 + i;
            s[r] = exp2_hw(fmaf(s[r], a.scale_log2, -l4[i]));
            dp[r] = s[r] * (dp[r] - d4[i]);
            if constexpr (masked)
              if (key >= sc.limit[at + i]) { s[r] = 0.f; dp[r] = 0.f; }
          }
        }
      };
      auto sums = [&](int b, const f32x16& s, const f32x16& dp) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const typename M::Col p = M::regs(s, t), ds = M::regs(dp, t);
#pragma unroll
          for (int d = 0; d < DB; ++d) {
            dv[d] = M::cols(Tl::col(gs, b, t, d, ln), p, dv[d]);
            dk[d] = M::cols(Tl::col(qs, b, t, d, ln), ds, dk[d]);
            if constexpr (VL) __builtin_amdgcn_sched_barrier(0);
          }
        }
      };
      if constexpr (PIPE && !masked) {
        // One wave per SIMD hides nothing by itself: the order is written out.
        // A chunk is two products, the LDS reads of the chunk after the next,
        // and, under the products of the other block, two exponentials; a
        // barrier to the compiler's scheduler keeps each chunk together.
        constexpr int C2 = 2 * DB;                      // chunks of a block's sums
        f32x16 s0 = f32x16{}, dp0 = f32x16{}, s1 = f32x16{}, dp1 = f32x16{};
        typename M::Row fq[3], fg[3];
        typename M::Col cq[3], cg[3];
        f32x4_t l4[4], d4[4];
        // chunk n of both blocks' scores (sums) keeps its fragments in slot n % 3
        auto load_rows = [&](int n) __attribute__((always_inline)) {
          fq[n % 3] = Tl::row(qs, n / SR, n % SR, ln);
          fg[n % 3] = Tl::row(gs, n / SR, n % SR, ln);
        };
        auto load_cols = [&](int n) __attribute__((always_inline)) {
          cg[n % 3] = Tl::col(gs, n / C2, n % C2 / DB, n % DB, ln);
          cq[n % 3] = Tl::col(qs, n / C2, n % C2 / DB, n % DB, ln);
        };
        auto load_stats = [&](int b, int r4) __attribute__((always_inline)) {
          l4[r4] = *reinterpret_cast<const f32x4_t*>(&sc.lse2[32 * b + 8 * r4 + 4 * half]);
          d4[r4] = *reinterpret_cast<const f32x4_t*>(&sc.delta[32 * b + 8 * r4 + 4 * half]);
        };
        auto weigh = [&](f32x16& s, f32x16& dp, int r) __attribute__((always_inline)) {
          s[r] = exp2_hw(fmaf(s[r], a.scale_log2, -l4[r / 4][r % 4]));
          dp[r] = s[r] * (dp[r] - d4[r / 4][r % 4]);
        };
        load_rows(0);
        load_rows(1);
#pragma unroll
        for (int n = 0; n < 2 * SR; ++n) {              // scores; block 1's over the exponentials of block 0
          const int c = n % SR;
          if (n + 2 < 2 * SR) load_rows(n + 2);
          else load_cols(n + 2 - 2 * SR);
          if (n == SR - 2) { load_stats(0, 0); load_stats(0, 1); }
          if (n == SR - 1) { load_stats(0, 2); load_stats(0, 3); }
          f32x16 &s = n < SR ? s0 : s1, &dp = n < SR ? dp0 : dp1;
          s = M::rows(fq[n % 3], kf[c], s);
          dp = M::rows(fg[n % 3], vf[c], dp);
          if (n >= SR) {
#pragma unroll
            for (int r = c * 16 / SR; r < (c + 1) * 16 / SR; ++r) weigh(s0, dp0, r);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) load_stats(1, r4);
        typename M::Col p, ds;
#pragma unroll
        for (int n = 0; n < 2 * C2; ++n) {              // sums; block 0's over the exponentials of block 1
          const int i = n % C2, d = n % DB;
          if (d == 0) { p = M::regs(n < C2 ? s0 : s1, i / DB); ds = M::regs(n < C2 ? dp0 : dp1, i / DB); }
          if (n + 2 < 2 * C2) load_cols(n + 2);
          dv[d] = M::cols(cg[n % 3], p, dv[d]);
          dk[d] = M::cols(cq[n % 3], ds, dk[d]);
          if (n < C2) {
#pragma unroll
            for (int r = i * 16 / C2; r < (i + 1) * 16 / C2; ++r) weigh(s1, dp1, r);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          f32x16 s, dp;
          scores(b, s, dp);
          weights(b, s, dp);
          sums(b, s, dp);
        }
      }
    }
    if (more) put(sn, r0 + RT, lsen, deltan);
  };

  if (it.lo < it.hi) {
    fetch(q0s, g0s, it.lo);
    float lse, delta;
    stats(it.lo, lse, delta);
    put(st0, it.lo, lse, delta);
    // rows at or past `whole` see all of the workgroup's keys: masked tiles
    // first, in pairs, then the rest
    const int whole =
        a.causal ? (int)min((int64_t)max(0, it.at + 32 * NW - 1 - off) * a.group, (int64_t)it.hi) : it.lo;
    int r = it.lo;
    for (; r < whole && r + RT < it.hi; r += 2 * RT) {
      step(std::true_type{}, q0s, g0s, st0, q1s, g1s, st1, r);
      step(std::true_type{}, q1s, g1s, st1, q0s, g0s, st0, r + RT);
    }
    for (; r + RT < it.hi; r += 2 * RT) {
      step(std::false_type{}, q0s, g0s, st0, q1s, g1s, st1, r);
      step(std::false_type{}, q1s, g1s, st1, q0s, g0s, st0, r + RT);
    }
    if (r < it.hi) step(std::true_type{}, q0s, g0s, st0, q1s, g1s, st1, r);
  }
  if (it.part >= 0) {
    const int64_t slot = ((int64_t)it.part * a.kv_heads + kvh) * (32 * NW) + wave * 32 + l32;
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      store_block<F32>(reinterpret_cast<char*>(a.part + slot * DP), dk[d], a.scale, d, DP, lane);
      store_block<F32>(reinterpret_cast<char*>(a.part2 + slot * DP), dv[d], 1.f, d, DP, lane);
    }
    return;
  }
  if (!live) return;
  char* pk = a.dk.p + (int64_t)(it.k0 + key) * a.dk.t + (int64_t)kvh * a.dk.h;
  char* pv = a.dv.p + (int64_t)(it.k0 + key) * a.dv.t + (int64_t)kvh * a.dv.h;
#pragma unroll
  for (int d = 0; d < DB; ++d) {
    store_block<T>(pk, dk[d], a.scale, d, a.dim, lane);
    store_block<T>(pv, dv[d], 1.f, d, a.dim, lane);
  }
}

// Adds the parts of a split tile.  ROWS: dq (tile rows are query rows);
// otherwise dk and dv (tile rows are keys).  A workgroup takes one tile row:
// DP / 4 threads hold four channels each, 1024 / DP of them add every so-many-th
// part, then their sums in order.
template <class T, int DP, bool ROWS>
__global__ __launch_bounds__(256) void attn_add(const AttnArgs a, int tile) {
  constexpr int CT = DP / 4, LANES = 256 / CT;
  __shared__ f32x4_t acc[ROWS ? 1 : 2][LANES][CT];
  const int r = blockIdx.x % tile, unit = blockIdx.x / tile;
  const int kvh = unit % a.kv_heads;
  const AttnJoin j = a.joins[unit / a.kv_heads];
  const int at = j.at + r, token = ROWS ? (int)quo(at, a.by_group) : at;
  if (token >= (ROWS ? j.lq : j.lk)) return;
  const int ct = threadIdx.x % CT, g = threadIdx.x / CT, c = 4 * ct;
  f32x4_t x = f32x4_t{}, y = f32x4_t{};
  if (g < LANES) {
#pragma unroll 4
    for (int p = g; p < j.count; p += LANES) {
      const int64_t e = (((int64_t)(j.first + p) * a.kv_heads + kvh) * tile + r) * DP + c;
      x += *reinterpret_cast<const f32x4_t*>(a.part + e);
      if constexpr (!ROWS) y += *reinterpret_cast<const f32x4_t*>(a.part2 + e);
    }
    acc[0][g][ct] = x;
    if constexpr (!ROWS) acc[1][g][ct] = y;
  }
  __syncthreads();
  const int n = min(LANES, j.count);
  const bool second = !ROWS && threadIdx.x >= 64;       // dv by another wave
  const int t = threadIdx.x - (second ? 64 : 0);
  if (t >= CT || 4 * t >= a.dim || (second && threadIdx.x >= 128)) return;
  x = f32x4_t{};
  for (int i = 0; i < n; ++i) x += acc[ROWS ? 0 : second][i][t];
  const float v[4] = {x.x, x.y, x.z, x.w};
  char* p;
  if constexpr (ROWS) p = a.dq.p + (int64_t)(j.q0 + token) * a.dq.t + (int64_t)(kvh * a.group + at - token * a.group) * a.dq.h;
  else if (second) p = a.dv.p + (int64_t)(j.k0 + at) * a.dv.t + (int64_t)kvh * a.dv.h;
  else p = a.dk.p + (int64_t)(j.k0 + at) * a.dk.t + (int64_t)kvh * a.dk.h;
  store_vec<T, 4>(p + 4 * t * T::kSize, v);
}

template <class T, int DP> st_status backward_dim(st_seqs* s, AttnArgs a, hipStream_t st) {
  constexpr int KT = T::kSize == 2 ? 64 : 32;
  for (int which : {kListDq, kListDkv}) {
    const AttnList& l = s->list[which];
    const bool rows = which == kListDq;
    for (int w = 0; w < 2; ++w) {                       // one list at a time: they share the partial buffer
      if (l.item[w].empty()) continue;
      const int tile = l.tile[w];
      a.joins = l.d_join[w];
      a.part2 = a.part + l.parts[w] * s->kv_heads * tile * (int64_t)DP;
      st_status r = attn_launches(l.item[w].size(), s->kv_heads, w == 0 ? 256 : 64, [&](size_t first, int grid) {
        a.items = l.d_item[w] + first;
        if (rows) {
          if (w == 0) attn_dq<T, DP, KT, 4><<<grid, 256, 0, st>>>(a);
          else attn_dq<T, DP, 32, 1><<<grid, 64, 0, st>>>(a);
        } else {
          if (w == 0) attn_dkv<T, DP, KT, 4><<<grid, 256, 0, st>>>(a);
          else attn_dkv<T, DP, 32, 1><<<grid, 64, 0, st>>>(a);
        }
        return launch_check(rows ? "attn_dq" : "attn_dkv");
      });
      if (r != ST_OK) return r;
      if (l.join[w].empty()) continue;
      const int jg = (int)(l.join[w].size() * s->kv_heads * tile);
      if (rows) attn_add<T, DP, true><<<jg, 256, 0, st>>>(a, tile);
      else attn_add<T, DP, false><<<jg, 256, 0, st>>>(a, tile);
      r = launch_check("attn_add");
      if (r != ST_OK) return r;
    }
  }
  return ST_OK;
}

size_t delta_floats(const st_seqs* s) { return ((size_t)s->total_q * s->heads + 63) / 64 * 64; }

}  // namespace

size_t attn_backward_bytes(const st_seqs* s) {
  size_t most = 0;
  for (int w = 0; w < 2; ++w) {
    const AttnList &q = s->list[kListDq], &k = s->list[kListDkv];
    most = std::max(most, (size_t)(q.parts[w] * s->kv_heads * q.tile[w]) * s->dp);
    most = std::max(most, (size_t)(k.parts[w] * s->kv_heads * k.tile[w]) * s->dp * 2);
  }
  return (delta_floats(s) + most) * sizeof(float);
}

}  // namespace st

using namespace st;

extern "C" st_status st_attention_packed_backward(st_seqs* seqs, const st_tokens* q, const st_tokens* k,
                                                  const st_tokens* v, const st_tokens* out, const float* lse,
                                                  const st_tokens* dout, float scale, const st_tokens* dq,
                                                  const st_tokens* dk, const st_tokens* dv, void* workspace,
                                                  size_t workspace_bytes, void* stream) {
  auto err = [](st_status s, const std::string& m) { return fail(s, "st_attention_packed_backward: " + m); };
  if (!seqs || !q || !k || !v || !out || !dout || !dq || !dk || !dv) return err(ST_ERR_INVALID_ARG, "NULL argument");
  if (!(scale > 0.f) || !std::isfinite(scale)) return err(ST_ERR_INVALID_ARG, "scale must be positive and finite");
  const int es = seqs->dtype == ST_F32 ? 4 : 2;
  // tokens of a tile that is read with 31-bit offsets: attn_dq's of k and v,
  // attn_dkv's of q and dout, and of v where it lies in LDS (wide fp32 heads)
  const int tile = 64, vtile = seqs->dtype == ST_F32 && seqs->dp > 64 ? 128 : 64;
  const int64_t tq = seqs->total_q, tk = seqs->total_k;
  AttnArgs a{};
  struct { AttnTensor* t; const st_tokens* v; bool keys; int span; const char* name; } const all[] = {
      {&a.q, q, false, tile, "st_attention_packed_backward: q"}, {&a.k, k, true, tile, "st_attention_packed_backward: k"},
      {&a.v, v, true, vtile, "st_attention_packed_backward: v"}, {&a.out, out, false, 1, "st_attention_packed_backward: out"},
      {&a.dout, dout, false, tile, "st_attention_packed_backward: dout"},
      {&a.dq, dq, false, 1, "st_attention_packed_backward: dq"}, {&a.dk, dk, true, 1, "st_attention_packed_backward: dk"},
      {&a.dv, dv, true, 1, "st_attention_packed_backward: dv"}};
  for (const auto& e : all) {
    const st_status s = attn_tensor(*e.t, e.v, e.keys ? tk : tq, e.keys ? seqs->kv_heads : seqs->heads, seqs->dim, es, e.span, e.name);
    if (s != ST_OK) return s;
  }
  // one group's heads lie within a tile's 31-bit offsets
  for (const AttnTensor* t : {&a.q, &a.dout})
    if (seqs->group > 1 && t->h >= (1ll << 30) / seqs->group)
      return err(ST_ERR_UNSUPPORTED, "head stride of q or dout too large for grouped heads");
  if (tq > 0 && !lse) return err(ST_ERR_INVALID_ARG, "NULL lse");
  if (!aligned16(lse) || !aligned16(workspace)) return err(ST_ERR_ALIGNMENT, "lse or workspace not 16-byte aligned");
  const size_t need = attn_backward_bytes(seqs);
  if (need && (!workspace || workspace_bytes < need)) return err(ST_ERR_WORKSPACE, "workspace missing or too small");
  if (tq == 0 && tk == 0) return ok();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  st_status s = seqs_device_table(seqs, st);
  if (s != ST_OK) return s;
  a.lse = const_cast<float*>(lse);
  a.delta = static_cast<float*>(workspace);
  a.part = a.delta + delta_floats(seqs);
  a.group = seqs->group;
  a.by_group = div31((uint32_t)seqs->group);
  a.kv_heads = seqs->kv_heads;
  a.heads = seqs->heads;
  a.dim = seqs->dim;
  a.causal = seqs->causal;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  if (seqs->dtype == ST_BF16) switch (seqs->dp) {
      case 32: return backward_dim<BF16, 32>(seqs, a, st);
      case 64: return backward_dim<BF16, 64>(seqs, a, st);
      case 96: return backward_dim<BF16, 96>(seqs, a, st);
      default: return backward_dim<BF16, 128>(seqs, a, st);
    }
  switch (seqs->dp) {
    case 32: return backward_dim<F32, 32>(seqs, a, st);
    case 64: return backward_dim<F32, 64>(seqs, a, st);
    case 96: return backward_dim<F32, 96>(seqs, a, st);
    default: return backward_dim<F32, 128>(seqs, a, st);
  }
}
