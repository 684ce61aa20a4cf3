// Rotary positions with several axes (time, height, width), and the cell
// positions of a sharded volume that they take.
//
// A head of D channels is cut into one section per axis (axis a has d_a
// channels, the rest is left alone).  Pair i of section a turns by
//   angle = position_a * base^(-2 i / d_a)
//   (u, v) -> (u cos - v sin, u sin + v cos)
// where the pair is (i, i + d_a / 2) of the section ("halves") or
// (2 i, 2 i + 1) ("adjacent").  The inverse turns by -angle: it is also the
// gradient, since a rotation's transpose is its inverse.
//
// Bound: HBM, every value read once and written once.  A workgroup takes a few
// whole tokens: it first puts cos and sin of their pairs into LDS (each angle
// once per token, shared by all heads), then its threads walk the tokens'
// vectors of pairs.  The angle is formed in turns in 64 bits (position times
// base^(..) / 2 pi, less its nearest whole number), so its error stays below
// 2^-23 turns at any 32-bit position; the rotation itself is fp32.  Measured:
// 114688 tokens of 36 heads of 64 (24 turning), fp32 in and bf16 out: 276 us, 5.8
// TB/s.
#include <algorithm>
#include <cmath>
#include <string>

#include "tokens.h"

namespace st {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 256;
constexpr int kRopePairs = kRopeMaxDim / 2;
constexpr int kRopeUnroll = 4;
constexpr int kRopeTable = 4096;          // (cos, sin) entries in LDS

struct RopeArgs {
  const char* x;
  char* out;
  const int32_t* positions;
  int64_t xt, xh, ot, oh;                 // strides in bytes
  int32_t tokens, heads, rotated, naxes;
  int32_t pairs;                          // D / 2: pairs of a head, the untouched rest included
  int32_t turned;                         // the first `turned` pairs rotate
  int32_t vecs;                           // pair vectors of a head: pairs / VEC
  int32_t tb;                             // tokens of a workgroup
  int32_t block0;                         // this launch's first workgroup
  Div31 by_vecs, by_heads, by_turned;
  float sign;
  double turn[kRopePairs];                // turns per position
  uint8_t axis[kRopePairs];
  uint16_t a[kRopePairs], b[kRopePairs];  // channels of pair vector j (VEC of each)
};
static_assert(sizeof(RopeArgs) <= kMaxKernargBytes, "kernel argument struct too large");

// VEC pairs (u[i], v[i]); adjacent pairs lie interleaved at one place
template <class T, int VEC, bool ADJ>
__device__ __forceinline__ void load_pairs(const char* p, int a, int b, float (&u)[VEC], float (&v)[VEC]) {
  if constexpr (ADJ) {
    float t[2 * VEC];
    load_vec<T, 2 * VEC>(p + a * T::kSize, t);
#pragma unroll
    for (int i = 0; i < VEC; ++i) { u[i] = t[2 * i]; v[i] = t[2 * i + 1]; }
  } else {
    load_vec<T, VEC>(p + a * T::kSize, u);
    load_vec<T, VEC>(p + b * T::kSize, v);
  }
}
template <class T, int VEC, bool ADJ>
__device__ __forceinline__ void store_pairs(char* p, int a, int b, const float (&u)[VEC], const float (&v)[VEC]) {
  if constexpr (ADJ) {
    float t[2 * VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) { t[2 * i] = u[i]; t[2 * i + 1] = v[i]; }
    store_vec<T, 2 * VEC>(p + a * T::kSize, t);
  } else {
    store_vec<T, VEC>(p + a * T::kSize, u);
    store_vec<T, VEC>(p + b * T::kSize, v);
  }
}

template <class TX, class TO, int VEC, bool ADJ>
__global__ __launch_bounds__(kRopeThreads) void rope_axes(const RopeArgs a) {
  __shared__ float2 table[kRopeTable];
  const int t0 = (a.block0 + (int)blockIdx.x) * a.tb;
  const int nt = min(a.tb, a.tokens - t0);
  for (int i = threadIdx.x; i < nt * a.turned; i += kRopeThreads) {
    const int t = quo(i, a.by_turned), p = i - t * a.turned;
    const double w = (double)a.positions[(int64_t)(t0 + t) * a.naxes + a.axis[p]] * a.turn[p];
    float c, s;
    sincospif(2.f * (float)(w - rint(w)), &s, &c);
    table[i] = make_float2(c, a.sign * s);
  }
  __syncthreads();
  const int items = nt * a.heads * a.vecs;
  for (int i0 = threadIdx.x; i0 < items; i0 += kRopeThreads * kRopeUnroll) {
    float u[kRopeUnroll][VEC], v[kRopeUnroll][VEC];
    int jv[kRopeUnroll], hd[kRopeUnroll], tk[kRopeUnroll];
#pragma unroll
    for (int k = 0; k < kRopeUnroll; ++k) {
      const int i = min(i0 + k * kRopeThreads, items - 1);
      const int q = quo(i, a.by_vecs);
      jv[k] = i - q * a.vecs;
      tk[k] = quo(q, a.by_heads);
      hd[k] = q - tk[k] * a.heads;
      load_pairs<TX, VEC, ADJ>(a.x + (int64_t)(t0 + tk[k]) * a.xt + (int64_t)hd[k] * a.xh, a.a[jv[k]], a.b[jv[k]], u[k],
                               v[k]);
    }
#pragma unroll
    for (int k = 0; k < kRopeUnroll; ++k) {
      if (i0 + k * kRopeThreads >= items) break;
      const int p = jv[k] * VEC;
      if (hd[k] < a.rotated && p < a.turned) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float2 cs = table[tk[k] * a.turned + p + e];
          const float nu = u[k][e] * cs.x - v[k][e] * cs.y;
          v[k][e] = u[k][e] * cs.y + v[k][e] * cs.x;
          u[k][e] = nu;
        }
      }
      store_pairs<TO, VEC, ADJ>(a.out + (int64_t)(t0 + tk[k]) * a.ot + (int64_t)hd[k] * a.oh, a.a[jv[k]], a.b[jv[k]],
                                u[k], v[k]);
    }
  }
}

template <class TX, class TO, int VEC>
st_status rope_launch(RopeArgs& a, bool adj, hipStream_t st) {
  const int64_t blocks = ((int64_t)a.tokens + a.tb - 1) / a.tb;
  for (int64_t b = 0; b < blocks; b += max_blocks(kRopeThreads)) {
    a.block0 = (int32_t)b;
    const dim3 grid((uint32_t)std::min<int64_t>(blocks - b, max_blocks(kRopeThreads)));
    if (adj) rope_axes<TX, TO, VEC, true><<<grid, kRopeThreads, 0, st>>>(a);
    else rope_axes<TX, TO, VEC, false><<<grid, kRopeThreads, 0, st>>>(a);
    const st_status s = launch_check("rope_axes");
    if (s != ST_OK) return s;
  }
  return ST_OK;
}

template <class TX, class TO> st_status rope_vec(RopeArgs& a, int vec, bool adj, hipStream_t st) {
  switch (vec) {
    case 4: return rope_launch<TX, TO, 4>(a, adj, st);
    case 2: return rope_launch<TX, TO, 2>(a, adj, st);
    default: return rope_launch<TX, TO, 1>(a, adj, st);
  }
}

// ------------------------------------------------------------ positions

struct PosShard {
  int32_t* out;
  Div31 w, h, d;
  int32_t rows, off[3];
  int32_t block_begin;
};
struct PosArgs {
  int32_t nshards, ndim;
  int32_t block0;                         // this launch's first block
  PosShard sh[ST_MAX_SHARDS];
};
static_assert(sizeof(PosArgs) <= kMaxKernargBytes, "kernel argument struct too large");

__global__ __launch_bounds__(256) void cell_positions(const PosArgs a) {
  const int blk = a.block0 + (int)blockIdx.x;
  int i = 0;
  while (i + 1 < a.nshards && a.sh[i + 1].block_begin <= blk) ++i;
  const PosShard& s = a.sh[i];
  const int64_t r = (int64_t)(blk - s.block_begin) * 256 + threadIdx.x;
  if (r >= s.rows) return;
  const uint32_t q = quo((uint32_t)r, s.w), w = (uint32_t)r - q * s.w.d;
  const uint32_t q2 = quo(q, s.h), h = q - q2 * s.h.d;
  const uint32_t n = quo(q2, s.d), d = q2 - n * s.d.d;
  int32_t* o = s.out + r * a.ndim;
  int k = 0;
  if (a.ndim == 3) o[k++] = s.off[0] + (int)d;
  o[k++] = s.off[1] + (int)h;
  o[k] = s.off[2] + (int)w;
}

}  // namespace
}  // namespace st

using namespace st;

extern "C" {

st_status st_plan_positions(const st_plan* plan, int32_t* const* pos_bufs, void* stream) {
  auto err = [](st_status s, const std::string& m) { return fail(s, "st_plan_positions: " + m); };
  if (!plan || !pos_bufs) return err(ST_ERR_INVALID_ARG, "NULL argument");
  PosArgs a{};
  a.nshards = (int32_t)plan->shards.size();
  a.ndim = plan->ndim;
  int64_t blocks = 0;
  for (int i = 0; i < a.nshards; ++i) {
    const Shard& s = plan->shards[i];
    if (!pos_bufs[i]) return err(ST_ERR_INVALID_ARG, "NULL shard buffer");
    if (!aligned16(pos_bufs[i])) return err(ST_ERR_ALIGNMENT, "shard buffer not 16-byte aligned");
    const int64_t rows = plan->batch * s.ext[0] * s.ext[1] * s.ext[2];
    if (rows >= (1ll << 31)) return err(ST_ERR_UNSUPPORTED, "a shard of 2^31 cells or more");
    PosShard& v = a.sh[i];
    v.out = pos_bufs[i];
    v.w = div31((uint32_t)s.ext[2]);
    v.h = div31((uint32_t)s.ext[1]);
    v.d = div31((uint32_t)s.ext[0]);
    v.rows = (int32_t)rows;
    for (int ax = 0; ax < kAxes; ++ax) {
      if (s.off[ax] + s.ext[ax] > INT32_MAX) return err(ST_ERR_UNSUPPORTED, "positions past 2^31");
      v.off[ax] = (int32_t)s.off[ax];
    }
    v.block_begin = (int32_t)blocks;
    blocks += (rows + 255) / 256;
  }
  if (blocks >= (1ll << 31)) return err(ST_ERR_UNSUPPORTED, "too many cells");
  for (int64_t b = 0; b < blocks; b += max_blocks(256)) {
    a.block0 = (int32_t)b;
    const int n = (int)std::min<int64_t>(blocks - b, max_blocks(256));
    cell_positions<<<n, 256, 0, static_cast<hipStream_t>(stream)>>>(a);
    const st_status s = launch_check("cell_positions");
    if (s != ST_OK) return s;
  }
  return ST_OK;
}

st_status st_rope_axes(const void* x, st_dtype x_dtype, int64_t x_token_stride, int64_t x_head_stride, int64_t tokens,
                       int32_t heads, int32_t rotated_heads, int32_t head_dim, const int32_t* positions, int32_t naxes,
                       const int32_t* axis_dims, double base, int32_t pairs, int32_t inverse, void* out,
                       st_dtype out_dtype, int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  auto err = [](st_status s, const std::string& m) { return fail(s, "st_rope_axes: " + m); };
  if (!axis_dims) return err(ST_ERR_INVALID_ARG, "NULL argument");
  if ((x_dtype != ST_F32 && x_dtype != ST_BF16) || (out_dtype != ST_F32 && out_dtype != ST_BF16))
    return err(ST_ERR_INVALID_ARG, "dtype must be ST_F32 or ST_BF16");
  if (tokens < 0 || heads < 1 || rotated_heads < 0 || rotated_heads > heads)
    return err(ST_ERR_INVALID_ARG, "tokens >= 0, heads >= 1 and 0 <= rotated_heads <= heads");
  if (naxes < 1 || naxes > 3) return err(ST_ERR_UNSUPPORTED, "1 to 3 axes");
  if (head_dim < 2 || head_dim % 2 || head_dim > kRopeMaxDim)
    return err(ST_ERR_UNSUPPORTED, "head_dim must be even and at most 256");
  if (pairs != ST_ROPE_HALVES && pairs != ST_ROPE_ADJACENT) return err(ST_ERR_INVALID_ARG, "unknown pairing");
  if (!(base > 1.0) || !(base < 1e30)) return err(ST_ERR_INVALID_ARG, "base must be above 1 and finite");
  int64_t sum = 0;
  for (int i = 0; i < naxes; ++i) {
    if (axis_dims[i] < 0 || axis_dims[i] % 2) return err(ST_ERR_BAD_SHAPE, "axis widths must be even and >= 0");
    sum += axis_dims[i];
  }
  if (sum > head_dim) return err(ST_ERR_BAD_SHAPE, "axis widths add up to more than head_dim");
  // one token or one head has no stride: any value stands for it
  if (tokens == 1) x_token_stride = out_token_stride = 0;
  if (heads == 1) x_head_stride = out_head_stride = 0;
  if (x_token_stride < 0 || x_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0)
    return err(ST_ERR_INVALID_ARG, "negative stride");
  if (heads > 65536 || tokens >= (1ll << 31)) return err(ST_ERR_UNSUPPORTED, "too many heads or tokens");
  if (tokens == 0) return ok();
  if (!x || !out || !positions) return err(ST_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(x) || !aligned16(out) || !aligned16(positions))
    return err(ST_ERR_ALIGNMENT, "x, out or positions not 16-byte aligned");
  // rows of the output must not overlap: tokens outermost or heads outermost
  const bool by_token = (heads == 1 || out_head_stride >= head_dim) &&
                        (tokens == 1 || out_token_stride >= (heads - 1) * out_head_stride + head_dim);
  const bool by_head = (tokens == 1 || out_token_stride >= head_dim) &&
                       (heads == 1 || out_head_stride >= (tokens - 1) * out_token_stride + head_dim);
  if (!by_token && !by_head) return err(ST_ERR_BAD_SHAPE, "rows of out overlap");
  if (x == out && (x_dtype != out_dtype || x_token_stride != out_token_stride || x_head_stride != out_head_stride))
    return err(ST_ERR_INVALID_ARG, "in place needs the same dtype and strides on both sides");
  RopeArgs a{};
  a.x = static_cast<const char*>(x);
  a.out = static_cast<char*>(out);
  a.positions = positions;
  const int ex = x_dtype == ST_F32 ? 4 : 2, eo = out_dtype == ST_F32 ? 4 : 2;
  a.xt = x_token_stride * ex;
  a.xh = x_head_stride * ex;
  a.ot = out_token_stride * eo;
  a.oh = out_head_stride * eo;
  a.tokens = (int32_t)tokens;
  a.heads = heads;
  a.rotated = rotated_heads;
  a.naxes = naxes;
  a.pairs = head_dim / 2;
  a.turned = (int32_t)sum / 2;
  a.sign = inverse ? -1.f : 1.f;
  const bool adj = pairs == ST_ROPE_ADJACENT;
  // widest vector of pairs: every section start and half width a multiple of
  // it, every row start and stride aligned for it
  int vec = 4;
  auto fits = [&](int v) {
    int64_t g = 0;
    int lo = 0;
    for (int i = 0; i <= naxes; ++i) {
      const int d = i < naxes ? axis_dims[i] : head_dim - (int)sum;
      if ((d / 2) % v || (!adj && lo % v)) return false;
      lo += d;
    }
    const int w = adj ? 2 * v : v;
    g = x_token_stride | x_head_stride | out_token_stride | out_head_stride;
    return g % w == 0;
  };
  while (vec > 1 && !fits(vec)) vec >>= 1;
  if (adj && vec == 1 && ((x_token_stride | x_head_stride | out_token_stride | out_head_stride) & 1))
    return err(ST_ERR_ALIGNMENT, "adjacent pairs need even strides");
  a.vecs = a.pairs / vec;
  int lo = 0, p = 0;
  for (int i = 0; i <= naxes; ++i) {
    const int d = i < naxes ? axis_dims[i] : head_dim - (int)sum;
    for (int k = 0; k < d / 2; ++k, ++p) {
      if (i < naxes) {
        a.turn[p] = std::pow(base, -2.0 * k / d) / (2.0 * M_PI);
        a.axis[p] = (uint8_t)i;
      }
      if (p % vec == 0) {
        a.a[p / vec] = (uint16_t)(adj ? lo + 2 * k : lo + k);
        a.b[p / vec] = (uint16_t)(adj ? lo + 2 * k + 1 : lo + d / 2 + k);
      }
    }
    lo += d;
  }
  // tokens of a workgroup: about 2048 vectors of work, within the table, and
  // at least 512 workgroups where the tokens allow it
  int64_t tb = std::max<int64_t>(1, 2048 / ((int64_t)heads * a.vecs));
  tb = std::min<int64_t>(tb, std::max<int64_t>(1, (tokens + 511) / 512));
  if (a.turned) tb = std::min<int64_t>(tb, kRopeTable / a.turned);
  a.tb = (int32_t)tb;
  a.by_vecs = div31((uint32_t)a.vecs);
  a.by_heads = div31((uint32_t)heads);
  a.by_turned = div31((uint32_t)std::max(1, a.turned));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (x_dtype == ST_F32)
    return out_dtype == ST_F32 ? rope_vec<F32, F32>(a, vec, adj, st) : rope_vec<F32, BF16>(a, vec, adj, st);
  return out_dtype == ST_F32 ? rope_vec<BF16, F32>(a, vec, adj, st) : rope_vec<BF16, BF16>(a, vec, adj, st);
}

}  // extern "C"
