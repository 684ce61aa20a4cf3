// Matrix products with bias, activation and residual in their epilogue, and the
// gradients' products.
//
//   forward  y[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n]
//   dx[m][k] = sum_n p[m][n] w[n][k]      (w read across its rows)
//   dw[n][k] = sum_m p[m][n] x[m][k]      (both read across their rows)
// One kernel for all three: an operand whose contraction is not contiguous lies in
// LDS as it lies in memory and is read by the transposing LDS read, so nothing is
// transposed in memory.
//
// Bound: the matrix cores; 256 x 256 tiles read each operand's stage (32 KB) once for
// 8 MFLOP.  16384 x 8192 x 2048 in bf16 419 us (1313 TFLOP/s), in 8 bits 238 (2308); 16384 x
// 2048 x 8192 475 us (1156: eight tiles a compute unit, whose stores of 128 KB each
// are partly waited for); dw of it 438 us (1257).  Up to 64 rows: the weights' bytes
// (1 x 2048 x 8192 in bf16 9.6 us, 3.5 TB/s).
#include "linear.h"
#include "linear_plan.h"

namespace st {
namespace {

template <int I> using Int = std::integral_constant<int, I>;
template <int N, int I = 0, class F> __device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(Int<I>{});
    static_for<N, I + 1>(f);
  }
}

// 64 lanes' B (16 or 4) bytes from base + offset (past `bytes`: zeros) to LDS, in the order
// of the lanes.  BYHAND: not by the builtin, whose transfers the compiler waits for before
// LDS is read again, with every store that it cannot count; the caller waits himself.
// (An SGPR that a vector instruction wrote is read by the fifth instruction after it at
// the earliest.)
typedef int i32x4_t __attribute__((ext_vector_type(4)));
template <int B, bool BYHAND> __device__ __forceinline__ void to_lds(const void* base, int bytes, const void* dst, uint32_t offset, int soffset) {
#ifdef __HIP_DEVICE_COMPILE__
  if constexpr (BYHAND) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    const i32x4_t r = {(int)(uint32_t)p, (int)(uint32_t)(p >> 32 & 0xFFFF), bytes, 0x00020000};
    const uint32_t at = (uint32_t)(uintptr_t)(lds_void)dst;
    int kept;                                           // (the compiler's m0)
    if constexpr (B == 16)
      asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
                   : "=&s"(kept) : "s"(at), "v"(offset), "s"(r), "s"(soffset) : "memory");
    else
      asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 4\n\tbuffer_load_dword %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
                   : "=&s"(kept) : "s"(at), "v"(offset), "s"(r), "s"(soffset) : "memory");
  } else {
    static_assert(B == 16, "16 bytes a lane");
    __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000),
                                             (lds_void)dst, 16, offset, soffset, 0, 0);
  }
#endif
}
// Waits for all but the newest N vector memory operations and for LDS
template <int N> __device__ __forceinline__ void wait_vm() { asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"(N) : "memory"); }

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

// PLAIN: partial sums, or an output in bf16 or fp32 with nothing but a bias; the
// epilogue is laid out for every block, so that it is worth keeping short.
template <class T, bool AC, bool BC, int TA, int TB, int WA, int WB, int OCC, bool PLAIN>
__global__ __launch_bounds__(64 * WA * WB, OCC) void gemm(const GemmArgs g) {
#ifdef __HIP_DEVICE_COMPILE__                           // (the host pass needs the name alone)
  constexpr int NW = WA * WB, PA = TA / WA, PB = TB / WB, NA = PA / 32, NB = PB / 32;
  using P = Prod<T>;
  using OA = Oper<T, AC, TA, NW>;
  using OB = Oper<T, BC, TB, NW>;
  constexpr int KT = OA::KT, STEPS = P::STEPS;
  constexpr bool EXACT = std::is_same<T, MX8X>::value, MX = std::is_same<T, MX8>::value || EXACT;
  constexpr int SCALES = MX ? (TA + TB) * 16 : 16;      // 16 scale bytes of every row: four stages
  __shared__ __attribute__((aligned(1024))) char a0[OA::BYTES];
  __shared__ __attribute__((aligned(1024))) char a1[OA::BYTES];
  __shared__ __attribute__((aligned(1024))) char b0[OB::BYTES];
  __shared__ __attribute__((aligned(1024))) char b1[OB::BYTES];
  __shared__ __attribute__((aligned(1024))) char sc[2 * SCALES];
  __shared__ __attribute__((aligned(1024))) float bias[2][TA];          // this tile's, the next one's
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, wa = wave % WA, wb = wave / WA;
  // (what depends on it is formed anew for each tile: no registers held meanwhile)
  auto lane_anew = [&]() __attribute__((always_inline)) -> int {
    int l = lane;
    asm("" : "+v"(l));
    return l;
  };

  // Workgroups go round the 8 XCDs: each XCD takes a run of tiles, eight row tiles
  // deep, so that what its L2 holds is shared; a workgroup takes every so many-th of
  // its XCD's run.
  const uint32_t xcd = blockIdx.x & 7, tiles = (uint32_t)g.tiles_a * g.tiles_b, total = tiles * g.splits;
  const uint32_t t_step = (gridDim.x + 7 - xcd) >> 3, t_end = (xcd + 1) * (total >> 3) + min(xcd + 1, total & 7);
  uint32_t t = xcd * (total >> 3) + min(xcd, total & 7) + (blockIdx.x >> 3);
  int n0, m0, split, k_lo, k_hi, turn = 0;
  // this lane's transfers: byte offsets from a stage's base, of the first one where
  // the others are rows on
  constexpr int QA = OA::ALIKE ? 1 : OA::NI, QB = OB::ALIKE ? 1 : OB::NI;
  uint32_t offa[QA], offb[QB];
  const char *pa, *pb;
  auto place = [&]() __attribute__((always_inline)) -> void {
    const int l = lane_anew();
    split = t / tiles;
    const uint32_t u = t - split * tiles, deep = 8, group = deep * g.tiles_a, gi = u / group, first = gi * deep;
    const uint32_t in = u - gi * group, d = min(deep, g.tiles_b - first);
    m0 = (first + in % d) * TB;
    n0 = in / d * TA;
    k_lo = split * g.per_split;
    k_hi = min(g.stages, k_lo + g.per_split);
#pragma unroll
    for (int i = 0; i < QA; ++i) {
      const int r = OA::dma_row(wave, l, i), b = OA::dma_byte(wave, l, i);
      offa[i] = AC && n0 * T::kSize + b >= g.n * T::kSize ? kPastEnd : (uint32_t)(r * (int)g.a.stride + b);
    }
#pragma unroll
    for (int i = 0; i < QB; ++i) {
      const int r = OB::dma_row(wave, l, i), b = OB::dma_byte(wave, l, i);
      offb[i] = BC && m0 * T::kSize + b >= g.m * T::kSize ? kPastEnd : (uint32_t)(r * (int)g.b.stride + b);
    }
    pa = AC ? g.a.p + (int64_t)n0 * T::kSize : g.a.p + (int64_t)n0 * g.a.stride;
    pb = BC ? g.b.p + (int64_t)m0 * T::kSize : g.b.p + (int64_t)m0 * g.b.stride;
  };

  // Stage kt's transfers.  Past the last stage nothing is read: they write zeros.
  const int sta = (int)g.a.stride, stb = (int)g.b.stride;
  auto fetch = [&](auto SWITCH, char* as, char* bs, int kt) __attribute__((always_inline)) -> void {
    constexpr bool sw = decltype(SWITCH)::value != 0;
    const int left = g.kbytes - kt * 128;               // bytes of the contraction from here on
    const int rows = min(g.k - kt * KT, KT);            // its steps of this stage
    const int na = AC ? rows * sta : min(TA, g.n - n0) * sta, nb = BC ? rows * stb : min(TB, g.m - m0) * stb;
    const char* ba = AC ? pa + (int64_t)kt * KT * sta : pa;
    const char* bb = BC ? pb + (int64_t)kt * KT * stb : pb;
    // (kPastEnd stays past every end with the rows added)
    static_assert((AC || OA::ALIKE) && (BC || OB::ALIKE), "one byte offset for all transfers along the contraction");
    const uint32_t a_first = !AC && OA::dma_byte(wave, lane, 0) >= left ? kPastEnd : offa[0];
    const uint32_t b_first = !BC && OB::dma_byte(wave, lane, 0) >= left ? kPastEnd : offb[0];
#pragma unroll
    for (int i = 0; i < OA::NI; ++i)
      to_lds<16, sw>(ba, kt < k_hi ? na : 0, OA::dma_dst(as, wave, i), OA::ALIKE ? a_first + (uint32_t)(i * OA::ROWS_ON * sta) : offa[i % QA], AC ? 0 : kt * 128);
#pragma unroll
    for (int i = 0; i < OB::NI; ++i)
      to_lds<16, sw>(bb, kt < k_hi ? nb : 0, OB::dma_dst(bs, wave, i), OB::ALIKE ? b_first + (uint32_t)(i * OB::ROWS_ON * stb) : offb[i % QB], BC ? 0 : kt * 128);
  };
  // 8-bit operands: the scale bytes of stages kt .. kt + 3, 16 of every row (a row's
  // may end before; the bytes past it are not used, and none past the last row's are read)
  auto fetch_scales = [&](auto SWITCH, int kt) __attribute__((always_inline)) -> void {
    if constexpr (MX) {
      if (wave < (TA + TB) / 64) {
        int w = wave;
        asm("" : "+s"(w));                              // (formed anew: no scalar registers held from stage to stage)
        const bool of_a = w < TA / 64;
        const Rows& o = of_a ? g.a : g.b;
        const int row0 = of_a ? n0 : m0, rows = of_a ? min(TA, g.n - n0) : min(TB, g.m - m0), first = of_a ? w * 64 : w * 64 - TA;
        to_lds<16, decltype(SWITCH)::value != 0>(o.scales + (int64_t)row0 * o.scale_stride, kt < k_hi ? scale_span(rows, (int)o.scale_stride, g.blocks_k) : 0,
                                                 sc + ((kt - k_lo) >> 2 & 1) * SCALES + wave * 1024, (uint32_t)((first + lane_anew()) * (int)o.scale_stride + kt * 4), 0);
      }
    }
  };
  // The tile's bias (zeros past the last channel).  It is added to the whole sum, at the
  // end: against a bias that the sums start from, the matrix instructions cut the
  // products' lowest bits (5092 x 11 x 3264: 21 of the 8-bit codes on the other side in
  // place of 2).
  auto fetch_bias = [&]() __attribute__((always_inline)) -> void {
    if (wave < TA / 64) {
      to_lds<4, true>(g.f.bias, g.f.bias ? g.n * 4 : 0, bias[turn] + wave * 64, (uint32_t)(n0 + wave * 64 + lane_anew()) * 4, 0);
    }
  };

  f32x16 acc[NA][NB];
  typename P::Frag fa[2][NA], fb[2][NB];
  int sa[2][MX ? NA : 1], sb[2][MX ? NB : 1];           // scale bytes of a stage: block 2 s + half in byte 2 s
  auto read_scales = [&](auto SET, int kt) __attribute__((always_inline)) -> void {
    if constexpr (MX) {
      constexpr int set = decltype(SET)::value;
      const char* p = sc + ((kt - k_lo) >> 2 & 1) * SCALES + ((kt - k_lo) & 3) * 4;
      // (past the last block the codes are zero; a byte there may be NaN's)
      const int blocks = g.blocks_k - 4 * kt;
      const uint32_t mask = blocks >= 4 ? 0xFFFFFFFFu : blocks <= 0 ? 0u : (1u << 8 * blocks) - 1;
#pragma unroll
      for (int i = 0; i < NA; ++i)
        sa[set][i] = (int)((*reinterpret_cast<const uint32_t*>(p + (wa * PA + 32 * i + (lane & 31)) * 16) & mask) >> 8 * half);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        sb[set][i] = (int)((*reinterpret_cast<const uint32_t*>(p + (TA + wb * PB + 32 * i + (lane & 31)) * 16) & mask) >> 8 * half);
    }
  };
  auto read = [&](auto SET, auto STEP, auto SCSET, const char* as, const char* bs) __attribute__((always_inline)) -> void {
    constexpr int set = decltype(SET)::value, s = decltype(STEP)::value, c = decltype(SCSET)::value;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if constexpr (EXACT) fb[set][j] = P::widen(P::template raw<BC, TB, NW>(bs, wb * NB + j, s, lane), sb[c][j] >> 16 * s & 255);
      else fb[set][j] = P::template frag<BC, TB, NW>(bs, wb * NB + j, s, lane);
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      if constexpr (EXACT) fa[set][i] = P::widen(P::template raw<AC, TA, NW>(as, wa * NA + i, s, lane), sa[c][i] >> 16 * s & 255);
      else fa[set][i] = P::template frag<AC, TA, NW>(as, wa * NA + i, s, lane);
    }
  };
  auto multiply = [&](auto SET, auto STEP, auto SCSET) __attribute__((always_inline)) -> void {
    constexpr int set = decltype(SET)::value, s = decltype(STEP)::value, c = decltype(SCSET)::value;
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        acc[i][j] = P::template mul<s>(fa[set][i], fb[set][j], acc[i][j], MX ? sa[c][MX ? i : 0] : 0, MX ? sb[c][MX ? j : 0] : 0);
  };
  // The order of a step: a product, then the reads of one of the next step's
  // fragments: b's first, a's as soon as the one in its place has had its last
  // product (so that they share registers); a transfer behind every product.
  auto order = [&](auto MORE) __attribute__((always_inline)) -> void {
    if constexpr (!EXACT && T::kSize < 4) {
      constexpr int RA = MX || AC ? 2 : 1, RB = MX || BC ? 2 : 1;      // LDS reads of a fragment
      static_for<NA * NB>([&](auto S) __attribute__((always_inline)) -> void {
        constexpr int t = decltype(S)::value, last = NA * NB - 1;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);             // a product
        if constexpr (t < NB) __builtin_amdgcn_sched_group_barrier(0x100, RB, 0);
        static_for<NA>([&](auto I) __attribute__((always_inline)) -> void {
          constexpr int at = (decltype(I)::value + 1) * NB;
          if constexpr (t == (at < last ? at : last)) __builtin_amdgcn_sched_group_barrier(0x100, RA, 0);
        });
        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);             // a transfer
        if constexpr (t == last / 2 && decltype(MORE)::value > 0) __builtin_amdgcn_sched_group_barrier(0x100, decltype(MORE)::value, 0);   // scale bytes
      });
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // Transfers and stores end in the order in which they set out, so waiting for all
  // but the newest `STORES` of a whole tile, which has at least that many, waits for the next
  // tile's transfers and not for the stores behind them.  They have until the end of the
  // second stage, whose transfers set out after them (8-bit 16384 x 2048 x 8192: 313 -> 285 us).
  constexpr int STORES = 2 * NA * NB;
  bool behind = false;

  // Stage kt in (as, bs), stage kt + 1 on its way to (an, bn).  Fragments are read one
  // step ahead of the products; before the last step's products every wave has read
  // all of stage kt, so the workgroup meets there, stage kt + 2 sets out into the
  // buffers of stage kt, and the first fragments of stage kt + 1 are on their way
  // while the matrix cores still have a step to do.
  // FIRST: of a tile.
  auto stage = [&](auto CUR, auto FIRST, char* as, char* bs, const char* an, const char* bn, int kt) __attribute__((always_inline)) -> void {
    constexpr int cur = decltype(CUR)::value;
    // (its buffer's last readers are two meetings back, its first three ahead)
    if constexpr (MX && cur == 0) {
      if ((kt - k_lo & 3) == 0) fetch_scales(Int<0>{}, kt + 4);
    }
    static_for<STEPS>([&](auto S) __attribute__((always_inline)) -> void {
      constexpr int s = decltype(S)::value;
      if constexpr (s == 0) read_scales(Int<1 - cur>{}, kt + 1);
      if constexpr (s + 1 < STEPS) {
        read(Int<(s + 1) & 1>{}, Int<s + 1>{}, Int<cur>{}, as, bs);
      } else {
        asm volatile("" ::: "memory");
        if (decltype(FIRST)::value && behind) wait_vm<STORES>();
        else __builtin_amdgcn_s_waitcnt(0x0070);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        read(Int<0>{}, Int<0>{}, Int<1 - cur>{}, an, bn);
        fetch(Int<0>{}, as, bs, kt + 2);
      }
      multiply(Int<s & 1>{}, Int<s>{}, Int<cur>{});
      order(Int<MX && s == 0 ? NA + NB : 0>{});
    });
  };

  // Two stages of the first tile set out; from then on the next tile's two do before
  // a tile's epilogue.  (Their buffers' last readers are behind the last meeting; what
  // is read after it is not used.)
  place();
  fetch_scales(Int<1>{}, k_lo);
  fetch_bias();
  fetch(Int<1>{}, a0, b0, k_lo);
  fetch(Int<1>{}, a1, b1, k_lo + 1);
  for (;;) {
    asm volatile("" ::: "memory");
    if (behind) wait_vm<STORES + OA::NI + OB::NI>();
    else wait_vm<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};
    read_scales(Int<0>{}, k_lo);
    read(Int<0>{}, Int<0>{}, Int<0>{}, a0, b0);
    int kt = k_lo;
    if (!MX && kt + 2 <= k_hi) {                        // (8-bit operands: no registers for a second copy)
      stage(Int<0>{}, Int<1>{}, a0, b0, a1, b1, kt);
      stage(Int<1>{}, Int<0>{}, a1, b1, a0, b0, kt + 1);
      kt += 2;
    }
    for (; kt + 2 <= k_hi; kt += 2) {
      stage(Int<0>{}, Int<0>{}, a0, b0, a1, b1, kt);
      stage(Int<1>{}, Int<0>{}, a1, b1, a0, b0, kt + 1);
    }
    if (kt < k_hi) stage(Int<0>{}, Int<0>{}, a0, b0, a1, b1, kt);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);                 // (no transfer of this tile meets one of the next)
    asm volatile("" ::: "memory");
    const int em = m0 + wb * PB, en = n0 + wa * PA, es = split;
    const float* ebias = bias[turn] + wa * PA;
    turn ^= 1;                                          // (the other's readers were the epilogue before this one)
    const bool added = !PLAIN && g.f.res.type >= 0;
    constexpr bool AHEAD = !MX;                         // (8-bit operands: no registers for it)
    Res res[2];                                         // the block's, the next one's
    behind = m0 + TB <= g.m && n0 + TA <= g.n;
    t += t_step;
    const bool more = t < t_end;
    if (more) {
      place();
      fetch_scales(Int<1>{}, k_lo);
      fetch_bias();
      fetch(Int<1>{}, a0, b0, k_lo);
      fetch(Int<1>{}, a1, b1, k_lo + 1);
    }
    asm volatile("" ::: "memory");
    int l = lane_anew();
    if (AHEAD && added) load_res(g.f.res, em, en, g.f.rows, g.f.cols, l, res[0]);
    static_for<NA * NB>([&](auto U) __attribute__((always_inline)) -> void {
      constexpr int i = decltype(U)::value / NB, j = decltype(U)::value % NB;
      constexpr int u = decltype(U)::value, in = (u + 1) / NB, jn = (u + 1) % NB;
      const int64_t m = em + 32 * j;
      const int n = en + 32 * i;
      if constexpr (!AHEAD) {
        l = lane_anew();
        res[0] = Res{};
        if (added) load_res(g.f.res, m, n, g.f.rows, g.f.cols, l, res[0]);
      } else if constexpr (u + 1 < NA * NB) {
        if (added) load_res(g.f.res, em + 32 * jn, en + 32 * in, g.f.rows, g.f.cols, l, res[(u + 1) & 1]);
      }
      float v[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] = acc[i][j][r];
      if (PLAIN && g.part) {
        if (m + (l & 31) < g.m && n < g.n) {
          float* p = g.part + ((int64_t)es * g.m + m + (l & 31)) * g.ld + n + 4 * (l >> 5);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4_t*>(p + 8 * q) = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 t = *reinterpret_cast<const float4*>(ebias + 32 * i + 8 * q + 4 * (l >> 5));
          v[4 * q] += t.x; v[4 * q + 1] += t.y; v[4 * q + 2] += t.z; v[4 * q + 3] += t.w;
        }
        finish_block<PLAIN, TA == 256>(g.f, m, n, l, res[AHEAD ? u & 1 : 0], v);
      }
    });
    if (!more) break;
  }
#endif
}

// Adds the splits' partial sums in order and finishes the blocks, a wave and a
// workgroup each.  Four splits are on their way at once: with few blocks the pass
// is as long as its loads are late (33 x 2048 in 4 splits: 5.7 -> 4.1 us).
__global__ __launch_bounds__(64) void gemm_join(const float* __restrict__ part, int splits, int64_t ld, Finish f, int blocks_n) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int64_t m0 = (int64_t)(blockIdx.x / blocks_n) * 32, m = m0 + (lane & 31);
  const int n0 = (int)(blockIdx.x % blocks_n) * 32;
  Res t;
  if (f.res.type >= 0) load_res(f.res, m0, n0, f.rows, f.cols, lane, t);
  float v[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) v[r] = 0.f;
  if (m < f.rows) {
    const float* p = part + m * ld + n0 + 4 * half;
    const int64_t next = (int64_t)f.rows * ld;
    int s = 0;
    for (; s + 4 <= splits; s += 4, p += 4 * next) {
      f32x4_t t[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) t[i][q] = *reinterpret_cast<const f32x4_t*>(p + i * next + 8 * q);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] += t[i][r / 4][r % 4];
    }
    for (; s < splits; ++s, p += next) {
      f32x4_t t[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) t[q] = *reinterpret_cast<const f32x4_t*>(p + 8 * q);
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] += t[r / 4][r % 4];
    }
  }
  add_bias(f, n0, lane, v);
  finish_block<false>(f, m0, n0, lane, t, v);
}

// ------------------------------------------------------------------ few rows

// Up to 64 rows of x: what counts is the weights' way from memory, once.  A
// workgroup takes 32 channels of the output, its eight waves take turns along the
// contraction in units of 128 bytes (a cache line of every weight row) and read
// both operands' fragments straight into registers; their sums meet in LDS and are
// added in the order of the waves.
template <class T> struct Unit;                         // fragments of a 128-byte unit, raw
template <> struct Unit<BF16> { u32x4_t v[4]; };
template <> struct Unit<F32> { u32x4_t v[4]; };
template <> struct Unit<MX8> { u32x4_t v[4]; int scale; };
template <> struct Unit<MX8X> { u32x4_t v[4]; int scale; };

template <class T, int MB> __global__ __launch_bounds__(64 * kFewWaves, 2) void few_rows(const GemmArgs g) {
#ifdef __HIP_DEVICE_COMPILE__
  using P = Prod<T>;
  constexpr bool EXACT = std::is_same<T, MX8X>::value, MX = std::is_same<T, MX8>::value || EXACT;
  constexpr int DEEP = MB == 1 ? 4 : 2;                 // units of a wave in flight
  __shared__ float4 sums[kFewWaves][MB][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int split = blockIdx.x / g.tiles_a, n0 = (blockIdx.x - split * g.tiles_a) * 32;
  const int u_lo = split * g.per_split, u_hi = min(g.stages, u_lo + g.per_split);

  const auto ra = __builtin_amdgcn_make_buffer_rsrc(g.a.p + (int64_t)n0 * g.a.stride, (short)0, min(32, g.n - n0) * (int)g.a.stride, 0x00020000);
  const auto rb = __builtin_amdgcn_make_buffer_rsrc(g.b.p, (short)0, g.m * (int)g.b.stride, 0x00020000);
  const uint32_t at_a = l32 * (int)g.a.stride;
  uint32_t at_b[MB];
#pragma unroll
  for (int j = 0; j < MB; ++j) at_b[j] = (32 * j + l32) * (int)g.b.stride;
  // the 16-byte chunks of a unit that this lane holds, in the order of the steps
  auto chunk = [&](int i) __attribute__((always_inline)) -> int {
    return std::is_same<T, MX8>::value ? 4 * (i >> 1) + 2 * (i & 1) + half : EXACT ? 4 * (i >> 1) + 2 * half + (i & 1) : 2 * i + half;
  };
  auto load = [&](Unit<T>& f, auto rs, uint32_t row, int r, const Rows& o, const uint8_t* sp, int rows, int u) __attribute__((always_inline)) -> void {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int byte = u * 128 + chunk(i) * 16;
      const uint32_t at = u < u_hi && byte < g.kbytes ? row + byte : kPastEnd;
      f.v[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0));
    }
    if constexpr (MX) {
      const auto rsc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(sp), (short)0, rows * (int)o.scale_stride, 0x00020000);
      // (past the last block the codes are zero; a byte there may be NaN's)
      const int blocks = g.blocks_k - 4 * u;
      const uint32_t mask = blocks >= 4 ? 0xFFFFFFFFu : blocks <= 0 ? 0u : (1u << 8 * blocks) - 1;
      const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(rsc, u < u_hi ? (uint32_t)(r * (int)o.scale_stride + 4 * u) : kPastEnd, 0, 0);
      f.scale = (int)((w & mask) >> 8 * half);
    }
  };
  auto frag = [&](const Unit<T>& f, auto S) __attribute__((always_inline)) -> auto {
    constexpr int s = decltype(S)::value;
    if constexpr (EXACT) return P::widen(Prod<MX8>::join(f.v[2 * s], f.v[2 * s + 1]), f.scale >> 16 * s & 255);
    else if constexpr (MX) return P::join(f.v[2 * s], f.v[2 * s + 1]);
    else return __builtin_bit_cast(typename P::Frag, f.v[s]);
  };

  f32x16 acc[MB];
#pragma unroll
  for (int j = 0; j < MB; ++j) acc[j] = f32x16{};
  const uint8_t* spa = MX ? g.a.scales + (int64_t)n0 * g.a.scale_stride : nullptr;
  for (int u0 = u_lo + wave; u0 < u_hi; u0 += DEEP * kFewWaves) {
    Unit<T> ua[DEEP], ub[DEEP][MB];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      load(ua[d], ra, at_a, l32, g.a, spa, min(32, g.n - n0), u0 + d * kFewWaves);
#pragma unroll
      for (int j = 0; j < MB; ++j) load(ub[d][j], rb, at_b[j], 32 * j + l32, g.b, g.b.scales, g.m, u0 + d * kFewWaves);
    }
    __builtin_amdgcn_sched_barrier(0);                  // (all on their way before the first is used)
#pragma unroll
    for (int d = 0; d < DEEP; ++d)
      static_for<P::STEPS>([&](auto S) __attribute__((always_inline)) -> void {
        const auto fa = frag(ua[d], S);
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          int sa = 0, sb = 0;
          if constexpr (MX) { sa = ua[d].scale; sb = ub[d][j].scale; }
          acc[j] = P::template mul<decltype(S)::value>(fa, frag(ub[d][j], S), acc[j], sa, sb);
        }
      });
  }
#pragma unroll
  for (int j = 0; j < MB; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) sums[wave][j][q][lane] = float4{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
  __syncthreads();
  if (wave >= MB) return;
  float v[16];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float4 t = sums[0][wave][q][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) {
      const float4 x = sums[w][wave][q][lane];
      t.x += x.x; t.y += x.y; t.z += x.z; t.w += x.w;
    }
    v[4 * q] = t.x; v[4 * q + 1] = t.y; v[4 * q + 2] = t.z; v[4 * q + 3] = t.w;
  }
  const int64_t m = 32 * wave + l32;
  if (!g.part) {
    Res t;
    add_bias(g.f, n0, lane, v);
    if (g.f.res.type >= 0) load_res(g.f.res, 32 * wave, n0, g.f.rows, g.f.cols, lane, t);
    finish_block<false>(g.f, 32 * wave, n0, lane, t, v);
  } else if (m < g.m) {
    float* p = g.part + ((int64_t)split * g.m + m) * g.ld + n0 + 4 * half;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<f32x4_t*>(p + 8 * q) = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
  }
#endif
}

// ------------------------------------------------------------------ host

int64_t part_ld(int64_t n) { return (n + 31) / 32 * 32; }

// a workgroup per tile, or as many as the compute units hold
int64_t gemm_grid(const GemmArgs& g, int per_cu) {
  return std::min<int64_t>((int64_t)g.tiles_a * g.tiles_b * g.splits, (int64_t)kCus * per_cu);
}

template <class T> st_status few_launch(const GemmArgs& g, hipStream_t st) {
  const unsigned grid = (unsigned)g.tiles_a * g.splits;
  if (g.m <= 32) few_rows<T, 1><<<grid, 64 * kFewWaves, 0, st>>>(g);
  else few_rows<T, 2><<<grid, 64 * kFewWaves, 0, st>>>(g);
  return launch_check("few_rows");
}

template <class T, bool AC, bool BC, bool PLAIN> st_status gemm_launch(const GemmArgs& g, int shape, hipStream_t st) {
  constexpr int type = std::is_same<T, F32>::value ? ST_F32 : std::is_same<T, BF16>::value ? ST_BF16 : ST_MX8;
  const unsigned grid = (unsigned)gemm_grid(g, shape_of(type, shape).per_cu);
  if constexpr (std::is_same<T, MX8X>::value) gemm<T, AC, BC, 128, 64, 2, 2, 2, PLAIN><<<grid, 256, 0, st>>>(g);
  else if (shape == 2) gemm<T, AC, BC, 64, 64, 2, 2, 4, PLAIN><<<grid, 256, 0, st>>>(g);
  else if (shape == 1) gemm<T, AC, BC, 128, 64, 2, 2, std::is_same<T, MX8>::value ? 2 : 3, PLAIN><<<grid, 256, 0, st>>>(g);
  else if constexpr (!std::is_same<T, F32>::value) gemm<T, AC, BC, 256, 256, 2, 4, 2, PLAIN><<<grid, 512, 0, st>>>(g);
  else if constexpr (PLAIN) gemm<T, AC, BC, 128, 128, 2, 2, 2, true><<<grid, 256, 0, st>>>(g);
  else return fail(ST_ERR_UNSUPPORTED, "matrix product: no such tile");   // (comes with split sums alone, which are plain)
  return launch_check("gemm");
}

st_status join_launch(const float* part, int splits, const Finish& f, hipStream_t st) {
  const int64_t blocks_n = part_ld(f.cols) / 32, blocks = ((int64_t)f.rows + 31) / 32 * blocks_n;
  if (blocks > max_blocks(64)) return fail(ST_ERR_UNSUPPORTED, "matrix product: too many blocks for one launch");
  gemm_join<<<(unsigned)blocks, 64, 0, st>>>(part, splits, part_ld(f.cols), f, (int)blocks_n);
  return launch_check("gemm_join");
}

}  // namespace

size_t product_bytes(int64_t m, int64_t n, int64_t k, int type, bool cols) {
  if (m <= 0 || n <= 0 || k <= 0) return 0;
  size_t most = 0;
  for (int exact = 0; exact <= (type == ST_MX8); ++exact) {
    const Choice c = choose(m, n, k, type, exact, cols);
    if (c.splits > 1) most = std::max(most, (size_t)c.splits * (size_t)m * (size_t)part_ld(n) * 4);
  }
  return most;
}

st_status product_launch(const Product& p, void* workspace, hipStream_t st) {
  if (p.k == 0) return join_launch(nullptr, 0, p.f, st);       // an empty sum: the epilogue of zeros
  // (an 8-bit output too: a cut sum lands on a code's other side now and then, 6% off,
  // 0.001 of the norm where the exact sums' codes are those of the 64-bit values)
  const bool exact = p.type == ST_MX8 && (p.f.y.type != ST_BF16 || (p.f.pre.type >= 0 && p.f.pre.type != ST_BF16));
  const Choice c = choose(p.m, p.n, p.k, p.type, exact, p.a_col);
  const bool few = c.shape == kFewShape;
  const Shape h = few ? Shape{32, kFewRows, 1} : shape_of(p.type, c.shape);
  const int es = type_size(p.type), kt = 128 / es;
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
  if (ta * tb * c.splits >= (1ll << 31)) return fail(ST_ERR_UNSUPPORTED, "matrix product: too many tiles");
  g.tiles_a = (int32_t)ta;
  g.tiles_b = (int32_t)tb;
  const bool plain = g.part || (p.f.act == kActNone && p.f.pre.type < 0 && p.f.res.type < 0 && p.f.y.type != ST_MX8);
  st_status s;
  if (few)
    s = exact ? few_launch<MX8X>(g, st) : p.type == ST_MX8 ? few_launch<MX8>(g, st)
        : p.type == ST_BF16 ? few_launch<BF16>(g, st) : few_launch<F32>(g, st);
  else if (p.type == ST_MX8)
    s = exact ? (plain ? gemm_launch<MX8X, false, false, true>(g, c.shape, st) : gemm_launch<MX8X, false, false, false>(g, c.shape, st))
              : (plain ? gemm_launch<MX8, false, false, true>(g, c.shape, st) : gemm_launch<MX8, false, false, false>(g, c.shape, st));
  else if (p.type == ST_BF16)                           // (gradients' products are plain)
    s = p.b_col ? gemm_launch<BF16, true, true, true>(g, c.shape, st) : p.a_col ? gemm_launch<BF16, true, false, true>(g, c.shape, st)
        : plain ? gemm_launch<BF16, false, false, true>(g, c.shape, st) : gemm_launch<BF16, false, false, false>(g, c.shape, st);
  else
    s = p.b_col ? gemm_launch<F32, true, true, true>(g, c.shape, st) : p.a_col ? gemm_launch<F32, true, false, true>(g, c.shape, st)
        : plain ? gemm_launch<F32, false, false, true>(g, c.shape, st) : gemm_launch<F32, false, false, false>(g, c.shape, st);
  if (s != ST_OK || c.splits == 1) return s;
  return join_launch(g.part, c.splits, p.f, st);
}

}  // namespace st
