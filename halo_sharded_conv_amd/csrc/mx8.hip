// Activations and weights in the 8-bit form: rows of e4m3 codes with one power of
// two per 32 channels, stored and read back.
//
// Bound: HBM; a pass reads every value once and writes it once (1 + 1/32 bytes
// for the 8-bit side).  A lane holds 8 channels, so that four lanes hold a block
// and its largest magnitude crosses them by two DPP steps; a code row is written
// 8 bytes a lane, a block's scale by its first lane.  Both write past the caches:
// 16384 x 8192 in bf16 stored in 63 us in place of 76 (6.4 TB/s), read back in 58 in
// place of 80 (7.0), and a product of 16384 x 2048 x 8192 that writes into what has just been
// read back does not wait for it (the two 698 -> 605 us); reading back codes just
// stored (134 MB, which the last cache holds) takes 10 us longer.  2048^2 x 64 in bf16:
// 147 us (5.5 TB/s) and 157.
#include <algorithm>
#include <string>

#include "rows.h"

namespace st {
namespace {

constexpr int kMxThreads = 256;
constexpr int kMxUnroll = 4;          // 8-channel groups of one lane in flight

struct MxArgs {
  Rows x, out;
  Div31 by_groups;                    // groups of 8 channels in a row, blocks made whole
  int32_t channels, act;
  uint32_t units;                     // groups of this launch
};

// one group of 8 channels: its row and first channel
struct MxAt {
  uint32_t row;
  int c, n;                           // n: channels of the group that exist (<= 0: none)
};
__device__ __forceinline__ MxAt mx_at(const MxArgs& a, uint32_t u) {
  MxAt g;
  g.row = quo(u, a.by_groups);
  g.c = (int)(u - g.row * a.by_groups.d) * 8;
  g.n = u < a.units ? min(8, a.channels - g.c) : 0;
  return g;
}

template <class T> __global__ __launch_bounds__(kMxThreads) void mx8_store(const MxArgs a) {
  const uint32_t u0 = blockIdx.x * (kMxThreads * kMxUnroll) + threadIdx.x;
  float v[kMxUnroll][8];
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i) {
    const MxAt g = mx_at(a, u0 + i * kMxThreads);
    load_some<T, 8>(a.x.p + (int64_t)g.row * a.x.stride + (int64_t)g.c * T::kSize, g.n, v[i]);
  }
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i) {
    const MxAt g = mx_at(a, u0 + i * kMxThreads);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, mx_bits(v[i][j]));
    const int s = mx_scale(block_max<8>(top));
    store_codes<8, true>(a.out, g.row, g.c, g.n, v[i], s);
  }
}

template <bool ACT> __global__ __launch_bounds__(kMxThreads) void mx8_load(const MxArgs a) {
  const uint32_t u0 = blockIdx.x * (kMxThreads * kMxUnroll) + threadIdx.x;
  uint32_t w[kMxUnroll][2];
  int s[kMxUnroll];
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i) {
    const MxAt g = mx_at(a, u0 + i * kMxThreads);
    s[i] = load_codes<8>(a.x, g.row, g.c, g.n, w[i]);
  }
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i) {
    const MxAt g = mx_at(a, u0 + i * kMxThreads);
    float v[8];
    mx_values(w[i][0], s[i], v);
    mx_values(w[i][1], s[i], v + 4);
    if constexpr (ACT) activate(a.act, v);
    if (g.n > 0) store_some<8, true>(a.out.type, a.out.p + (int64_t)g.row * a.out.stride + (int64_t)g.c * (a.out.type == ST_F32 ? 4 : 2), g.n, v);
  }
}

// Launches of fewer than 2^31 groups each
template <class F> st_status mx_launches(MxArgs a, int64_t rows, int64_t channels, F launch) {
  const int64_t groups = (channels + kMxBlock - 1) / kMxBlock * (kMxBlock / 8);
  a.channels = (int32_t)channels;
  a.by_groups = div31((uint32_t)groups);
  const int64_t most = std::max<int64_t>(1, ((1ll << 30) - 1) / groups);
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = std::min(most, rows - r);
    a.units = (uint32_t)(n * groups);
    const st_status s = launch(a, (int)((a.units + kMxThreads * kMxUnroll - 1) / (kMxThreads * kMxUnroll)));
    if (s != ST_OK) return s;
    a.x.p += n * a.x.stride;
    a.out.p += n * a.out.stride;
    if (a.x.scales) a.x.scales += n * a.x.scale_stride;
    if (a.out.scales) a.out.scales += n * a.out.scale_stride;
  }
  return ST_OK;
}

st_status mx_sizes(int64_t rows, int64_t channels, const char* what) {
  if (rows < 0 || channels < 1) return fail(ST_ERR_INVALID_ARG, std::string(what) + ": negative rows or no channels");
  if (rows >= (1ll << 31) || channels >= (1ll << 31) - 64) return fail(ST_ERR_UNSUPPORTED, std::string(what) + ": 2^31 rows or channels");
  return ST_OK;
}

}  // namespace

st_status mx8_store_rows(int64_t rows, int64_t channels, const Rows& x, const Rows& out, hipStream_t st) {
  MxArgs a{};
  a.x = x;
  a.out = out;
  return mx_launches(a, rows, channels, [&](const MxArgs& b, int blocks) {
    if (x.type == ST_F32) mx8_store<F32><<<blocks, kMxThreads, 0, st>>>(b);
    else mx8_store<BF16><<<blocks, kMxThreads, 0, st>>>(b);
    return launch_check("mx8_store");
  });
}

st_status mx8_load_rows(int64_t rows, int64_t channels, const Rows& x, int act, const Rows& out, hipStream_t st) {
  MxArgs a{};
  a.x = x;
  a.out = out;
  a.act = act;
  return mx_launches(a, rows, channels, [&](const MxArgs& b, int blocks) {
    if (act == kActNone) mx8_load<false><<<blocks, kMxThreads, 0, st>>>(b);
    else mx8_load<true><<<blocks, kMxThreads, 0, st>>>(b);
    return launch_check("mx8_load");
  });
}

}  // namespace st

using namespace st;

extern "C" {

st_status st_mx8_store(int64_t rows, int64_t channels, const st_rows* x, const st_rows* out, void* stream) {
  const char* const me = "st_mx8_store";
  st_status s = mx_sizes(rows, channels, me);
  if (s != ST_OK) return s;
  Rows rx, ro;
  if ((s = rows_of(rx, x, rows, channels, kTakesFloat, me, "x")) != ST_OK) return s;
  if ((s = rows_of(ro, out, rows, channels, 1u << ST_MX8, me, "out")) != ST_OK) return s;
  if (rows_meet(rx, ro, rows, channels)) return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": x and out overlap");
  if (rows == 0) return ok();
  return mx8_store_rows(rows, channels, rx, ro, static_cast<hipStream_t>(stream));
}

st_status st_mx8_load(int64_t rows, int64_t channels, const st_rows* x, int32_t act, const st_rows* out, void* stream) {
  const char* const me = "st_mx8_load";
  st_status s = mx_sizes(rows, channels, me);
  if (s != ST_OK) return s;
  if (act < ST_ACT_NONE || act > ST_ACT_SILU) return fail(ST_ERR_INVALID_ARG, std::string(me) + ": unknown activation");
  Rows rx, ro;
  if ((s = rows_of(rx, x, rows, channels, 1u << ST_MX8, me, "x")) != ST_OK) return s;
  if ((s = rows_of(ro, out, rows, channels, kTakesFloat, me, "out")) != ST_OK) return s;
  if (rows_meet(rx, ro, rows, channels)) return fail(ST_ERR_BAD_SHAPE, std::string(me) + ": x and out overlap");
  if (rows == 0) return ok();
  return mx8_load_rows(rows, channels, rx, act, ro, static_cast<hipStream_t>(stream));
}

}  // extern "C"
