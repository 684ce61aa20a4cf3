// st_linear and st_linear_backward: checks, the rows that have to be padded, the
// pass over the gradient at the output, and the products.
//
// The pass over dy (bound: HBM) forms p = dy * act'(pre), rounded to the products'
// type, and sums p's columns for dbias in fp32 before the rounding: every thread
// keeps the sums of its own 8 columns over the rows it visits, a workgroup adds
// its threads in a fixed order and writes one partial row, and a second kernel
// adds those in order.  With no activation p is dy itself.
//
// p in bf16 is what the bf16 matrix cores take: half of 2^-8 of every term, independent
// from term to term.  dx and dw of 16384 x 2048 x 8192 with GELU are 0.0023 of the norm off,
// 0.0017 of it by their own rounding (an fp32 p: that alone, at a tenth of the rate).
#include "linear.h"

namespace st {
namespace {

// ---------------------------------------------------------------- padding

// Rows whose length is no multiple of 16 bytes, copied to rows that are: the
// products' transfers are 16 bytes wide, and a NaN behind a row's end must not meet
// the other operand's zeros.
struct PadArgs {
  const char* src;
  char* dst;
  int64_t src_stride, dst_stride, rows;
  Div31 by_chunks;
  int32_t bytes;                      // of a row
  uint32_t units;
};
__global__ __launch_bounds__(256) void pad_rows(const PadArgs a) {
  const uint32_t u = blockIdx.x * 256u + threadIdx.x;
  if (u >= a.units) return;
  const uint32_t row = quo(u, a.by_chunks), chunk = u - row * a.by_chunks.d;
  const char* p = a.src + (int64_t)row * a.src_stride + chunk * 16;
  const int left = a.bytes - (int)chunk * 16;
  u32x4_t w = {0, 0, 0, 0};
  if (left >= 16) {
    w = *reinterpret_cast<const u32x4_any*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) w[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
  }
  *reinterpret_cast<u32x4_t*>(a.dst + (int64_t)row * a.dst_stride + chunk * 16) = w;
}

int64_t padded_bytes(int64_t channels, int es) { return (channels * es + 15) / 16 * 16; }
size_t align_up(size_t n) { return (n + 255) / 256 * 256; }

// x's rows at `at` with padding; scales stay where they are
st_status pad_launch(Rows& x, int64_t rows, int64_t channels, char* at, hipStream_t st) {
  const int es = type_size(x.type);
  PadArgs a{};
  a.src_stride = x.stride;
  a.dst_stride = padded_bytes(channels, es);
  a.bytes = (int32_t)(channels * es);
  const int64_t chunks = a.dst_stride / 16, most = std::max<int64_t>(1, ((1ll << 30) - 1) / chunks);
  a.by_chunks = div31((uint32_t)chunks);
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = std::min(most, rows - r);
    a.src = x.p + r * x.stride;
    a.dst = at + r * a.dst_stride;
    a.units = (uint32_t)(n * chunks);
    pad_rows<<<(a.units + 255) / 256, 256, 0, st>>>(a);
    const st_status s = launch_check("pad_rows");
    if (s != ST_OK) return s;
  }
  x.p = at;
  x.stride = a.dst_stride;
  return ST_OK;
}

// ----------------------------------------------------- gradient at the output

constexpr int kGradThreads = 256;
constexpr int kGradUnroll = 4;
constexpr int kGradGroups = 1024;     // workgroups: four a CU

struct GradArgs {
  Rows dy, pre, p;                    // pre, p: type -1 where absent
  float* partial;                     // [parts][cols], or NULL
  int64_t rows;
  int32_t cols, p_cols, act, lpr_log2, strips, parts;
};

// One group of 8 columns over its rows.  FULL: all 8 exist.
template <int ACT, class TP, class TD, bool FULL> __device__ __forceinline__ void grad_rows(const GradArgs& a, int c, int n, int64_t first, int64_t step, float (&sum)[8]) {
  const int p_n = a.p_cols - c;                         // (the padding past the columns gets zeros)
  auto rows = [&](auto U, int64_t r0) __attribute__((always_inline)) -> void {
    constexpr int kRows = decltype(U)::value;
    float g[kRows][8], z[kRows][8];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t r = r0 + u * step;
      load_some<TD, 8>(a.dy.p + r * a.dy.stride + (int64_t)c * TD::kSize, FULL ? 8 : n, g[u]);
      if constexpr (ACT != kActNone) {
        if constexpr (std::is_same<TP, MX8>::value) load_values<8>(a.pre, r, c, FULL ? 8 : n, z[u]);
        else load_some<TP, 8>(a.pre.p + r * a.pre.stride + (int64_t)c * TP::kSize, FULL ? 8 : n, z[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t r = r0 + u * step;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (ACT != kActNone) g[u][i] *= slope_of<ACT>(z[u][i]);   // (columns that are not there: 0)
        sum[i] += g[u][i];
      }
      if (a.p.type >= 0) store_some<8>(a.p.type, a.p.p + r * a.p.stride + (int64_t)c * (a.p.type == ST_F32 ? 4 : 2), FULL ? 8 : p_n, g[u]);
    }
  };
  int64_t r = first;
  for (; r + (kGradUnroll - 1) * step < a.rows; r += kGradUnroll * step) rows(std::integral_constant<int, kGradUnroll>{}, r);
  for (; r < a.rows; r += step) rows(std::integral_constant<int, 1>{}, r);
}

template <int ACT, class TP, class TD> __global__ __launch_bounds__(kGradThreads) void grad_pass(const GradArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ float acc[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lpr = 1 << a.lpr_log2, sub = lane & (lpr - 1), per = 4 * (64 >> a.lpr_log2);
  const int strip = blockIdx.x % a.strips, part = blockIdx.x / a.strips;
  const int c = (strip * lpr + sub) * 8, n = a.cols - c;
  const int64_t first = (int64_t)part * per + wave * (64 >> a.lpr_log2) + (lane >> a.lpr_log2), step = (int64_t)a.parts * per;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  if (n >= 8) grad_rows<ACT, TP, TD, true>(a, c, n, first, step, sum);
  else if (n > 0) grad_rows<ACT, TP, TD, false>(a, c, n, first, step, sum);
  if (!a.partial) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    for (int m = lpr; m < 64; m <<= 1) sum[i] += __shfl_xor(sum[i], m);
    if (lane < lpr) acc[wave][sub * 8 + i] = sum[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < lpr * 8; i += kGradThreads) {
    const int col = strip * lpr * 8 + i;
    if (col < a.cols) a.partial[(int64_t)part * a.cols + col] = (acc[0][i] + acc[1][i]) + (acc[2][i] + acc[3][i]);
  }
#endif
}

template <int ACT> st_status grad_launch(const GradArgs& g, unsigned grid, hipStream_t st) {
#define GRAD_CASE(TP, TD) grad_pass<ACT, TP, TD><<<grid, kGradThreads, 0, st>>>(g)
  const bool f = g.dy.type == ST_F32;
  if constexpr (ACT == kActNone) {
    if (f) GRAD_CASE(F32, F32); else GRAD_CASE(F32, BF16);
  } else if (g.pre.type == ST_MX8) {
    if (f) GRAD_CASE(MX8, F32); else GRAD_CASE(MX8, BF16);
  } else if (g.pre.type == ST_BF16) {
    if (f) GRAD_CASE(BF16, F32); else GRAD_CASE(BF16, BF16);
  } else {
    if (f) GRAD_CASE(F32, F32); else GRAD_CASE(F32, BF16);
  }
#undef GRAD_CASE
  return launch_check("grad_pass");
}

struct GradShape {
  int lpr_log2, strips, parts;
};
GradShape grad_shape(int64_t rows, int64_t cols) {
  GradShape g{};
  while ((8 << g.lpr_log2) < cols && g.lpr_log2 < 6) ++g.lpr_log2;
  const int64_t wide = 8ll << g.lpr_log2, per = 4 * (64 >> g.lpr_log2);
  g.strips = (int)((cols + wide - 1) / wide);
  g.parts = (int)std::max<int64_t>(1, std::min<int64_t>(kGradGroups / g.strips, (rows + per - 1) / per));
  return g;
}

// ---------------------------------------------------------------- workspace

struct Layout {                       // byte offsets of the regions
  size_t x, w, p, sums, parts, total;
};
Layout layout_of(int64_t rows, int64_t in, int64_t out, int type, bool backward) {
  const int es = type_size(type);
  const bool pad = in * es % 16 != 0;
  const size_t ldk = (size_t)padded_bytes(in, es), ldn = (size_t)padded_bytes(out, es);
  Layout l{};
  size_t at = 0;
  auto take = [&](size_t n) { const size_t o = at; at += align_up(n); return o; };
  // (backward: x may come in 8 bits, p may be formed: both regions always)
  l.x = take(pad || backward ? (size_t)rows * ldk : 0);
  l.w = take(pad ? (size_t)out * ldk : 0);
  l.p = take(backward ? (size_t)rows * ldn : 0);
  l.sums = take(backward ? (size_t)grad_shape(rows, out).parts * (size_t)out * 4 : 0);
  size_t part = backward ? 0 : product_bytes(rows, out, in, type, false);
  if (backward) part = std::max(product_bytes(rows, in, out, type, true), product_bytes(out, in, rows, type, true));
  l.parts = take(part);
  l.total = at;
  return l;
}

st_status linear_sizes(int64_t rows, int64_t in, int64_t out, const char* me) {
  if (rows < 0 || in < 1 || out < 1) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": negative rows, or no channels");
  if (rows >= (1ll << 30) || in >= (1ll << 24) || out >= (1ll << 24))
    return fail(ST_ERR_UNSUPPORTED, std::string(me) + ": 2^30 rows or 2^24 channels");
  return ST_OK;
}
// Tiles address 256 rows from one base by 32 bits
st_status linear_stride(const Rows& r, const char* what) {
  if (r.type >= 0 && (r.stride >= (1 << 22) || r.scale_stride >= (1 << 22)))
    return fail(ST_ERR_UNSUPPORTED, std::string(what) + ": rows of 4 MiB or more apart");
  return ST_OK;
}

}  // namespace
}  // namespace st

using namespace st;

extern "C" {

size_t st_linear_workspace_bytes(int64_t rows, int64_t in, int64_t out, int32_t type, int32_t backward) {
  if (rows < 0 || in < 1 || out < 1 || rows >= (1ll << 30) || in >= (1ll << 24) || out >= (1ll << 24)) return 0;
  if (type < 0 || type > ST_MX8 || (backward && type == ST_MX8)) return 0;
  return layout_of(rows, in, out, type, backward != 0).total;
}

st_status st_linear(int64_t rows, int64_t in, int64_t out, const st_rows* x, const st_rows* w, const float* bias_or_null,
                    int32_t act, const st_rows* residual_or_null, const st_rows* y, const st_rows* pre_or_null,
                    void* workspace, size_t workspace_bytes, void* stream) {
  const char* const me = "st_linear";
  st_status s = linear_sizes(rows, in, out, me);
  if (s != ST_OK) return s;
  if (act < ST_ACT_NONE || act > ST_ACT_SILU) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": unknown activation");
  if (!aligned16(bias_or_null) || !aligned16(workspace)) return fail(ST_ERR_ALIGNMENT, std::string(me) + ": bias or workspace not 16-byte aligned");
  Product p{};
  p.f.pre = p.f.res = no_rows();
  if ((s = rows_of(p.b, x, rows, in, kTakesAll, me, "x")) != ST_OK) return s;
  if ((s = rows_of(p.a, w, out, in, kTakesAll, me, "w")) != ST_OK) return s;
  if (p.a.type != p.b.type) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": x and w differ in type");
  if ((s = rows_of(p.f.y, y, rows, out, kTakesAll, me, "y")) != ST_OK) return s;
  if (pre_or_null && (s = rows_of(p.f.pre, pre_or_null, rows, out, kTakesAll, me, "pre")) != ST_OK) return s;
  if (residual_or_null && (s = rows_of(p.f.res, residual_or_null, rows, out, kTakesFloat, me, "residual")) != ST_OK) return s;
  if ((s = linear_stride(p.b, me)) != ST_OK || (s = linear_stride(p.a, me)) != ST_OK) return s;
  if (rows > 0 && (meet(p.f.y, rows, out, p.b, rows, in) || meet(p.f.y, rows, out, p.a, out, in) ||
                   meet(p.f.pre, rows, out, p.b, rows, in) || meet(p.f.pre, rows, out, p.a, out, in) ||
                   meet(p.f.y, rows, out, p.f.pre, rows, out) || meet(p.f.pre, rows, out, p.f.res, rows, out) ||
                   (meet(p.f.y, rows, out, p.f.res, rows, out) && !same_rows(p.f.y, p.f.res))))
    return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": an output overlaps an input or the other output");
  const Rows bv = floats_of(bias_or_null, out);
  if (meet(p.f.y, rows, out, bv, 1, out) || meet(p.f.pre, rows, out, bv, 1, out))
    return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": an output overlaps the bias");
  p.type = p.a.type;
  const Layout l = layout_of(rows, in, out, p.type, false);
  if (rows > 0 && l.total > 0 && (!workspace || workspace_bytes < l.total))
    return fail(ST_ERR_WORKSPACE, std::string(me) + ": workspace missing or too small");
  if (rows == 0) return ok();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (in * type_size(p.type) % 16 != 0) {
    if ((s = pad_launch(p.b, rows, in, ws + l.x, st)) != ST_OK) return s;
    if ((s = pad_launch(p.a, out, in, ws + l.w, st)) != ST_OK) return s;
  }
  p.m = rows;
  p.n = out;
  p.k = in;
  p.f.bias = bias_or_null;
  p.f.act = act;
  p.f.rows = (int32_t)rows;
  p.f.cols = (int32_t)out;
  return product_launch(p, ws + l.parts, st);
}

st_status st_linear_backward(int64_t rows, int64_t in, int64_t out, const st_rows* x, const st_rows* w, int32_t act,
                             const st_rows* pre_or_null, const st_rows* dy, const st_rows* dx_or_null,
                             const st_rows* dw_or_null, float* dbias_or_null, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const char* const me = "st_linear_backward";
  st_status s = linear_sizes(rows, in, out, me);
  if (s != ST_OK) return s;
  if (act < ST_ACT_NONE || act > ST_ACT_SILU) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": unknown activation");
  if (act != ST_ACT_NONE && !pre_or_null) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": an activation's gradient needs pre");
  if (!aligned16(dbias_or_null) || !aligned16(workspace)) return fail(ST_ERR_ALIGNMENT, std::string(me) + ": dbias or workspace not 16-byte aligned");
  Rows rx, rw, rdy, pre = no_rows(), dx = no_rows(), dw = no_rows();
  if ((s = rows_of(rx, x, rows, in, kTakesAll, me, "x")) != ST_OK) return s;
  if ((s = rows_of(rw, w, out, in, kTakesFloat, me, "w")) != ST_OK) return s;
  if (rx.type != rw.type && rx.type != ST_MX8) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": x is neither in w's type nor in 8 bits");
  if ((s = rows_of(rdy, dy, rows, out, kTakesFloat, me, "dy")) != ST_OK) return s;
  if (pre_or_null && (s = rows_of(pre, pre_or_null, rows, out, kTakesAll, me, "pre")) != ST_OK) return s;
  if (dx_or_null && (s = rows_of(dx, dx_or_null, rows, in, kTakesFloat, me, "dx")) != ST_OK) return s;
  if (dw_or_null && (s = rows_of(dw, dw_or_null, out, in, kTakesFloat, me, "dw")) != ST_OK) return s;
  for (const Rows* r : {&rx, &rw, &rdy, &pre})
    if ((s = linear_stride(*r, me)) != ST_OK) return s;
  struct Side { const Rows* r; int64_t rows, cols; };
  const Side ins[4] = {{&rx, rows, in}, {&rw, out, in}, {&rdy, rows, out}, {&pre, rows, out}};
  const Side outs[2] = {{&dx, rows, in}, {&dw, out, in}};
  for (const Side& o : outs)
    for (const Side& i : ins)
      if (meet(*o.r, o.rows, o.cols, *i.r, i.rows, i.cols)) return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": an output overlaps an input");
  const Rows db = floats_of(dbias_or_null, out);
  for (const Side& i : ins)
    if (meet(db, 1, out, *i.r, i.rows, i.cols)) return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": dbias overlaps an input");
  if (meet(dx, rows, in, dw, out, in) || meet(db, 1, out, dx, rows, in) || meet(db, 1, out, dw, out, in))
    return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": two outputs overlap");
  const int type = rw.type, es = type_size(type);
  const Layout l = layout_of(rows, in, out, type, true);
  if (rows > 0 && (!workspace || workspace_bytes < l.total)) return fail(ST_ERR_WORKSPACE, std::string(me) + ": workspace missing or too small");
  const hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);

  // p: dy itself where it can be read as it is
  const bool form = rows > 0 && (dx_or_null || dw_or_null) && (act != ST_ACT_NONE || rdy.type != type || out * es % 16 != 0);
  Rows p = rdy;
  if (rows > 0 && (form || dbias_or_null)) {
    const GradShape gs = grad_shape(rows, out);
    GradArgs g{};
    g.dy = rdy;
    g.pre = act != ST_ACT_NONE ? pre : no_rows();
    g.p = no_rows();
    g.rows = rows;
    g.cols = (int32_t)out;
    g.act = act;
    g.lpr_log2 = gs.lpr_log2;
    g.strips = gs.strips;
    g.parts = gs.parts;
    if (form) {
      p = Rows{ws + l.p, nullptr, padded_bytes(out, es), 0, type};
      g.p = p;
      g.p_cols = (int32_t)(p.stride / es);
    }
    if (dbias_or_null) g.partial = reinterpret_cast<float*>(ws + l.sums);
    const unsigned grid = (unsigned)(gs.strips * gs.parts);
    s = act == kActGelu ? grad_launch<kActGelu>(g, grid, st) : act == kActSilu ? grad_launch<kActSilu>(g, grid, st)
        : act == kActRelu ? grad_launch<kActRelu>(g, grid, st) : grad_launch<kActNone>(g, grid, st);
    if (s != ST_OK) return s;
    if (dbias_or_null && (s = add_rows_launch(g.partial, gs.parts, (int)out, dbias_or_null, st)) != ST_OK) return s;
  } else if (dbias_or_null) {
    if ((s = add_rows_launch(nullptr, 0, (int)out, dbias_or_null, st)) != ST_OK) return s;
  }
  const bool pad = in * es % 16 != 0;
  if (dx_or_null && rows > 0) {
    Product q{};
    q.f.pre = q.f.res = no_rows();
    q.a = rw;
    if (pad && (s = pad_launch(q.a, out, in, ws + l.w, st)) != ST_OK) return s;
    q.b = p;
    q.type = type;
    q.a_col = true;
    q.m = rows;
    q.n = in;
    q.k = out;
    q.f.y = dx;
    q.f.rows = (int32_t)rows;
    q.f.cols = (int32_t)in;
    if ((s = product_launch(q, ws + l.parts, st)) != ST_OK) return s;
  }
  if (dw_or_null) {
    Product q{};
    q.f.pre = q.f.res = no_rows();
    q.a = rx;
    if (rows > 0 && rx.type == ST_MX8) {
      // the 8-bit form's values are bf16 (and fp32) numbers: nothing is rounded here
      q.a = Rows{ws + l.x, nullptr, padded_bytes(in, es), 0, type};
      if ((s = mx8_load_rows(rows, in, rx, kActNone, q.a, st)) != ST_OK) return s;
    } else if (rows > 0 && pad) {
      if ((s = pad_launch(q.a, rows, in, ws + l.x, st)) != ST_OK) return s;
    }
    q.b = p;
    q.type = type;
    q.a_col = q.b_col = true;
    q.m = out;
    q.n = in;
    q.k = rows;
    q.f.y = dw;
    q.f.rows = (int32_t)out;
    q.f.cols = (int32_t)in;
    if ((s = product_launch(q, ws + l.parts, st)) != ST_OK) return s;
  }
  return ok();
}

}  // extern "C"
