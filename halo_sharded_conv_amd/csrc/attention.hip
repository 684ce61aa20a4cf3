// Attention over packed sequences: forward.
//
//   out = softmax(scale * q k^T) v,   lse = log sum exp(scale * q k^T)
// per sequence and head, in one pass over the keys: with the running maximum m
// and denominator l of a row, a tile of scores s adds p = exp(s - m), and where
// m grows, l and the output so far are scaled by exp(m_old - m_new).
//
// The products run transposed: S^T = K Q^T, then O^T += V^T P^T.  A lane then
// holds one row (query) of the scores and of the output for its whole life, so
// the maximum and the sum of a row need one exchange between the wave's
// halves per tile and none inside a product, and the scores go from the first
// product to the second in registers.  See attention.h for the LDS tiles.
//
// Rows are (token, head of the group) pairs, so heads that share keys share
// the tiles of K and V, and a single query token of a grouped head still fills
// the rows of a tile.
//
// Bound: the matrix cores, with the exponentials beside them (64 channels: as
// long as the products).  Tile: 4 waves of 32 rows share 64 keys of K and V, two
// stages; K Q^T reads a tile once per 32 rows, which leaves the LDS a quarter
// busy.  Three waves per SIMD up to 128 bytes a row (64 channels: 912 -> 971
// TFLOP/s), two above.  Measured: 4 x 4096 tokens, 16 heads of 128: 520 us, 1050
// TFLOP/s (76% of a large bf16 product); causal 16001 tokens, 16 / 4 heads of
// 128: 1.0 ms, 1030; 2 x 8192, 16 heads of 64: 575 us, 950; fp32, 4096 tokens, 8
// heads of 128: 580 us, 118 (77% of a large fp32 product).  One wave with 32 keys
// a step serves sequences of up to 64 rows: single tokens of 16 / 4 heads of 64
// over 79000 keys 24 us, 5.0 TB/s.
#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "attention.h"

namespace st {
namespace {

// m grows only where a tile exceeds it by more than this (in powers of two):
// p stays below 2^8, and most tiles then scale nothing
constexpr float kSlack = 8.f;

// What a matrix product must not see next to a zero weight: 0 * inf and 0 * NaN
// are NaN, but a masked key has no weight at all.
template <class T> struct Special;
template <> struct Special<BF16> {
  typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ bool any(bf16x8 v) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const u32x4_t w = __builtin_bit_cast(u32x4_t, v) & 0x7FFF7FFFu;
    u16x2 m = u16x2{0, 0};                              // largest magnitude of the even and odd values
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t word = w[i];                       // (a bit cast of a vector's element reads element 0)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, word));
    }
    return (m.x >= 0x7F80) | (m.y >= 0x7F80);
  }
  static __device__ __forceinline__ bf16x8 finite(bf16x8 v) {
    u16x8 w = __builtin_bit_cast(u16x8, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (w[i] & 0x7F80) == 0x7F80 ? 0 : w[i];
    return __builtin_bit_cast(bf16x8, w);
  }
};
template <> struct Special<F32> {
  static __device__ __forceinline__ bool any(f32x8 v) {
    bool f = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) f |= (__float_as_uint(v[i]) & 0x7F800000u) == 0x7F800000u;
    return f;
  }
  static __device__ __forceinline__ f32x8 finite(f32x8 v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (__float_as_uint(v[i]) & 0x7F800000u) == 0x7F800000u ? 0.f : v[i];
    return v;
  }
};

// The NaN and infinities of four channels of V over the keys [j, end) that a
// row sees (those below `limit`).  Every seen key has a weight above zero, so
// they enter the row's sum as they are.
template <class T>
__device__ __attribute__((noinline)) f32x4_t special_keys(const char* v, int64_t stride, int j, int end, int limit, int c) {
  f32x4_t x = f32x4_t{};
  for (; j < end; ++j) {
    float y[4];
    load_vec<T, 4>(v + (int64_t)j * stride + c * T::kSize, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] += j < limit && (__float_as_uint(y[i]) & 0x7F800000u) == 0x7F800000u ? y[i] : 0.f;
  }
  return x;
}
template <class T>
__device__ __forceinline__ void special_sum(const char* v, int64_t stride, int j, int end, int limit, int c, int dim, float (&x)[4]) {
  f32x4_t y = f32x4_t{};
  if (c < dim) y = special_keys<T>(v, stride, j, end, limit, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = y[i];
}

// waves per SIMD that the registers allow
template <class T, int DP> constexpr int fwd_waves() { return DP * T::kSize > 256 ? 1 : DP * T::kSize > 128 ? 2 : 3; }

template <class T, int DP, int KT, int NW>
__global__ __launch_bounds__(64 * NW, (fwd_waves<T, DP>())) void attn_forward(const AttnArgs a) {
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

  const int row0 = it.at + wave * 32;                   // the wave's first row
  const int row = row0 + l32;
  const int token = (int)quo(row, a.by_group), head = kvh * a.group + row - token * a.group;
  const bool live = token < it.lq;
  const int off = it.lk - it.lq;                        // causal: token i sees keys <= i + off
  // keys below `limit` are seen by this lane's row
  const int limit = a.causal ? min(it.lk, token + off + 1) : it.lk;
  // every row of the workgroup sees the keys below `all`; no row of this wave
  // sees one at or past `wave_last`
  const int all = min(it.hi, a.causal ? (int)quo(it.at, a.by_group) + off + 1 : it.lk);
  const int wave_last = a.causal ? min(it.lk, (int)quo(row0 + 31, a.by_group) + off + 1) : it.lk;

  typename M::Row qf[SR];
  {
    const char* p = a.q.p + (int64_t)(it.q0 + token) * a.q.t + (int64_t)head * a.q.h;
#pragma unroll
    for (int s = 0; s < SR; ++s) {
      const int byte = (2 * s + half) * 16;
      qf[s] = live && byte < a.dim * T::kSize ? *reinterpret_cast<const typename M::Row*>(p + byte) : typename M::Row{};
    }
  }
  // this lane's transfers: byte offsets within a tile of K and of V
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

  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x16{};
  float m = -INFINITY, l = 0.f;
  bool sp = false;                                      // this lane met a NaN or an infinity there

  auto fetch = [&](char* ks, char* vs, int j0) __attribute__((always_inline)) {
    const int64_t left = min(KT, it.hi - j0);            // rows past the range read zeros
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

  // one tile: MASKED where some row may not see some key of it
  auto step = [&](auto MASKED, const char* ks, const char* vs, char* kn, char* vn, int j0) __attribute__((always_inline)) {
    constexpr bool masked = decltype(MASKED)::value;
    __builtin_amdgcn_s_waitcnt(0x0F70);                 // vmcnt(0): this tile is in LDS
    __syncthreads();                                    // ... for every wave; the other tile is free
    if (j0 + KT < it.hi) fetch(kn, vn, j0 + KT);
    if (masked && j0 >= wave_last) return;              // (uniform) nothing here is seen by these rows
    f32x16 s[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      s[b] = f32x16{};
#pragma unroll
      for (int c = 0; c < SR; ++c) s[b] = M::rows(Tl::row(ks, b, c, lane), qf[c], s[b]);
    }
    if constexpr (masked) {
      const int lim = limit - j0 - 4 * half;
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * b + 8 * (r / 4) + r % 4 >= lim) s[b][r] = -INFINITY;
    }
    float mx = s[0][0];
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[b][r]);
    mx = half_max(mx) * a.scale_log2;
    if (__any(mx > m + kSlack)) {
      const float mn = mx > m + kSlack ? mx : m;        // row by row: a row's bits are its own
      const float f = mn == m ? 1.f : exp2_hw(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= f;
    }
    const float ms = m == -INFINITY ? 0.f : m;          // no key seen so far: p = 0
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[b][r] = exp2_hw(fmaf(s[b][r], a.scale_log2, -ms));
        l += s[b][r];
      }
    // a hidden key's NaN or infinity has no part in a row: a masked tile's product
    // takes the finite values, what is left is added to the rows that see it at
    // the end (special_sum)
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const typename M::Col p = M::regs(s[b], t);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          typename M::Col w = Tl::col(vs, b, t, d, lane);
          if constexpr (masked) {
            const bool bad = Special<T>::any(w);
            sp |= bad;
            if (__any(bad)) w = Special<T>::finite(w);
          }
          o[d] = M::cols(w, p, o[d]);
        }
        if constexpr (masked) __builtin_amdgcn_sched_barrier(0);
      }
  };

  // whole tiles that every row sees, in pairs, then the rest with the mask
  const int first_masked = it.lo + max(0, (all - it.lo) / (2 * KT)) * (2 * KT);
  if (it.lo < it.hi) {
    fetch(k0s, v0s, it.lo);
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

  l = half_sum(l);
  const float inv = l == 0.f ? 0.f : 1.f / l;           // a row that sees no key: zeros
  const bool split = it.part >= 0;
  const int64_t slot = split ? ((int64_t)it.part * a.kv_heads + kvh) * (32 * NW) + wave * 32 + l32 : 0;
  const int64_t stat = (int64_t)(it.q0 + token) * a.heads + head;
  if (half == 0) {
    const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
    if (split) a.part2[slot] = lse2;
    else if (live && a.lse) a.lse[stat] = lse2 * kLn2;
  }
  char* po = split ? reinterpret_cast<char*>(a.part + slot * DP)
                   : a.out.p + (int64_t)(it.q0 + token) * a.out.t + (int64_t)head * a.out.h;
  if (__any(sp)) {
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int c = reg_channel(d, r4, lane);
        float x[4];
        special_sum<T>(vb, a.v.t, first_masked, min(it.hi, wave_last), limit, c, a.dim, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][4 * r4 + i] += x[i];
      }
  }
  if (split) {
#pragma unroll
    for (int d = 0; d < DB; ++d) store_block<F32>(po, o[d], inv, d, DP, lane);
  } else if (live) {
#pragma unroll
    for (int d = 0; d < DB; ++d) store_block<T>(po, o[d], inv, d, a.dim, lane);
  }
}

// Joins the parts of a tile whose keys were split: each part is a softmax of its
// own with log2 of its denominator, so the whole is their sum weighted by
// 2^(part - max).  A workgroup takes one row: DP / 4 threads hold four channels
// each, 1024 / DP of them add every so-many-th part, then their sums in order.
template <class T, int DP>
__global__ __launch_bounds__(256) void attn_join(const AttnArgs a, int tile) {
  constexpr int CT = DP / 4, LANES = 256 / CT;
  __shared__ f32x4_t acc[LANES][CT];
  __shared__ float red[4], den[LANES];
  const int r = blockIdx.x % tile, unit = blockIdx.x / tile;
  const int kvh = unit % a.kv_heads;
  const AttnJoin j = a.joins[unit / a.kv_heads];
  const int row = j.at + r, token = (int)quo(row, a.by_group), head = kvh * a.group + row - token * a.group;
  if (token >= j.lq) return;
  const int64_t first = ((int64_t)j.first * a.kv_heads + kvh) * tile + r, pitch = (int64_t)a.kv_heads * tile;
  float m = -INFINITY;
  for (int p = threadIdx.x; p < j.count; p += 256) m = fmaxf(m, a.part2[first + p * pitch]);
  for (int i = 1; i < 64; i <<= 1) m = fmaxf(m, __shfl_xor(m, i));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float ms = m == -INFINITY ? 0.f : m;
  const int ct = threadIdx.x % CT, g = threadIdx.x / CT;
  float l = 0.f;
  f32x4_t o = f32x4_t{};
  if (g < LANES) {
#pragma unroll 4
    for (int p = g; p < j.count; p += LANES) {
      const int64_t slot = first + p * pitch;
      const float w = exp2_hw(a.part2[slot] - ms);
      const f32x4_t x = *reinterpret_cast<const f32x4_t*>(a.part + slot * DP + 4 * ct);
      l += w;
#pragma unroll
      for (int e = 0; e < 4; ++e)                       // a weight is above zero, underflow or not
        o[e] += (__float_as_uint(x[e]) & 0x7F800000u) == 0x7F800000u ? x[e] : w * x[e];
    }
    acc[g][ct] = o;
    if (ct == 0) den[g] = l;
  }
  __syncthreads();
  if (threadIdx.x >= CT) return;
  l = 0.f;
  o = f32x4_t{};
  const int n = min(LANES, j.count);
  for (int i = 0; i < n; ++i) {
    l += den[i];
    o += acc[i][ct];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t tok = j.q0 + token;
  if (threadIdx.x == 0 && a.lse) a.lse[tok * a.heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  const float x[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  if (4 * ct < a.dim) store_vec<T, 4>(a.out.p + tok * a.out.t + (int64_t)head * a.out.h + 4 * ct * T::kSize, x);
}

template <class T, int DP> st_status forward_dim(st_seqs* s, AttnArgs a, hipStream_t st) {
  constexpr int KT = T::kSize == 2 ? 64 : 32;
  const AttnList& l = s->list[kListForward];
  float* part = a.part;
  for (int w = 0; w < 2; ++w) {
    if (l.item[w].empty()) continue;
    const int tile = l.tile[w];
    a.joins = l.d_join[w];
    a.part = part;
    a.part2 = part + l.parts[w] * s->kv_heads * tile * (int64_t)DP;
    part = a.part2 + (l.parts[w] * s->kv_heads * tile + 63) / 64 * 64;
    st_status r = attn_launches(l.item[w].size(), s->kv_heads, w == 0 ? 256 : 64, [&](size_t first, int grid) {
      a.items = l.d_item[w] + first;
      if (w == 0) attn_forward<T, DP, KT, 4><<<grid, 256, 0, st>>>(a);
      else attn_forward<T, DP, 32, 1><<<grid, 64, 0, st>>>(a);
      return launch_check("attn_forward");
    });
    if (r != ST_OK) return r;
    if (l.join[w].empty()) continue;
    attn_join<T, DP><<<(int)(l.join[w].size() * s->kv_heads * tile), 256, 0, st>>>(a, tile);
    r = launch_check("attn_join");
    if (r != ST_OK) return r;
  }
  return ST_OK;
}

}  // namespace

size_t attn_forward_bytes(const st_seqs* s) {
  size_t n = 0;
  for (int w = 0; w < 2; ++w) {
    const AttnList& l = s->list[kListForward];
    const size_t rows = (size_t)(l.parts[w] * s->kv_heads * l.tile[w]);
    n += rows * s->dp * sizeof(float) + (rows + 63) / 64 * 64 * sizeof(float);
  }
  return n;
}

// Checks and converts a tensor's view.  `span` tokens of one head's group must
// lie within 31-bit byte offsets of each other (a tile's transfers).
st_status attn_tensor(AttnTensor& out, const st_tokens* v, int64_t tokens, int heads, int dim, int esize, int span,
                      const char* name) {
  const std::string who(name);
  if (!v) return fail(ST_ERR_INVALID_ARG, who + ": NULL argument");
  if (tokens == 0) {
    out = AttnTensor{nullptr, 0, 0};
    return ST_OK;
  }
  if (!v->data) return fail(ST_ERR_INVALID_ARG, who + ": NULL data");
  if (!aligned16(v->data)) return fail(ST_ERR_ALIGNMENT, who + ": data not 16-byte aligned");
  // one token or one head has no stride: any value stands for it
  const int64_t t = tokens == 1 ? (int64_t)dim * heads : v->token_stride;
  const int64_t h = heads == 1 ? dim : v->head_stride;
  if (t < 0 || h < 0) return fail(ST_ERR_INVALID_ARG, who + ": negative stride");
  if (t > (1ll << 30) / ((int64_t)span * esize) || h > (1ll << 40))
    return fail(ST_ERR_UNSUPPORTED, who + ": stride too large");
  if ((t * esize) % 16 || (h * esize) % 16)
    return fail(ST_ERR_ALIGNMENT, who + ": strides must be multiples of 16 bytes");
  const bool by_token = tokens == 1 ? h >= dim : h >= dim && t >= (heads - 1) * h + dim;
  const bool by_head = t >= dim && (heads == 1 || h >= (tokens - 1) * t + dim);
  if (!by_token && !by_head) return fail(ST_ERR_BAD_SHAPE, who + ": rows overlap");
  out = AttnTensor{static_cast<char*>(v->data), t * esize, h * esize};
  return ST_OK;
}

}  // namespace st

using namespace st;

extern "C" {

size_t st_attention_workspace_bytes(const st_seqs* seqs, int32_t backward) {
  if (!seqs) return 0;
  const size_t f = attn_forward_bytes(seqs);
  return backward ? std::max(f, attn_backward_bytes(seqs)) : f;
}

st_status st_attention_packed(st_seqs* seqs, const st_tokens* q, const st_tokens* k, const st_tokens* v, float scale,
                              const st_tokens* out, float* lse_or_null, void* workspace, size_t workspace_bytes,
                              void* stream) {
  auto err = [](st_status s, const std::string& m) { return fail(s, "st_attention_packed: " + m); };
  if (!seqs || !q || !k || !v || !out) return err(ST_ERR_INVALID_ARG, "NULL argument");
  if (!(scale > 0.f) || !std::isfinite(scale)) return err(ST_ERR_INVALID_ARG, "scale must be positive and finite");
  const int es = seqs->dtype == ST_F32 ? 4 : 2;
  AttnArgs a{};
  st_status s;
  if ((s = attn_tensor(a.q, q, seqs->total_q, seqs->heads, seqs->dim, es, 1, "st_attention_packed: q")) != ST_OK ||
      (s = attn_tensor(a.k, k, seqs->total_k, seqs->kv_heads, seqs->dim, es, 64, "st_attention_packed: k")) != ST_OK ||
      (s = attn_tensor(a.v, v, seqs->total_k, seqs->kv_heads, seqs->dim, es, 64, "st_attention_packed: v")) != ST_OK ||
      (s = attn_tensor(a.out, out, seqs->total_q, seqs->heads, seqs->dim, es, 1, "st_attention_packed: out")) != ST_OK)
    return s;
  if (!aligned16(lse_or_null) || !aligned16(workspace)) return err(ST_ERR_ALIGNMENT, "lse or workspace not 16-byte aligned");
  const size_t need = attn_forward_bytes(seqs);
  if (need && (!workspace || workspace_bytes < need)) return err(ST_ERR_WORKSPACE, "workspace missing or too small");
  if (seqs->total_q == 0) return ok();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  s = seqs_device_table(seqs, st);
  if (s != ST_OK) return s;
  a.lse = lse_or_null;
  a.part = static_cast<float*>(workspace);
  a.group = seqs->group;
  a.by_group = div31((uint32_t)seqs->group);
  a.kv_heads = seqs->kv_heads;
  a.heads = seqs->heads;
  a.dim = seqs->dim;
  a.causal = seqs->causal;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  if (seqs->dtype == ST_BF16) switch (seqs->dp) {
      case 32: return forward_dim<BF16, 32>(seqs, a, st);
      case 64: return forward_dim<BF16, 64>(seqs, a, st);
      case 96: return forward_dim<BF16, 96>(seqs, a, st);
      default: return forward_dim<BF16, 128>(seqs, a, st);
    }
  switch (seqs->dp) {
    case 32: return forward_dim<F32, 32>(seqs, a, st);
    case 64: return forward_dim<F32, 64>(seqs, a, st);
    case 96: return forward_dim<F32, 96>(seqs, a, st);
    default: return forward_dim<F32, 128>(seqs, a, st);
  }
}

}  // extern "C"
