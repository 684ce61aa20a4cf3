// Planner of packed-sequence attention: cuts every sequence into tiles of rows
// (forward, dq) or keys (dk, dv), splits a tile's long loop over several
// workgroups where there are too few tiles to fill the GPU, and orders the work
// longest first.  Host only, except the upload of the tables and its release.
#include <algorithm>
#include <cstring>
#include <new>
#include <string>

#include "sequences.h"

namespace st {

// Four-wave tiles serve long sequences; a sequence with at most two waves'
// worth of rows (keys) goes to one-wave workgroups, so a single token or a small
// window does not leave three waves idle.
AttnShape attn_shape(st_dtype dtype) {
  AttnShape s{};
  const bool f32 = dtype == ST_F32;
  s.tile[kListForward][0] = 128;
  s.tile[kListDq][0] = 128;
  s.tile[kListDkv][0] = 128;
  for (int l = 0; l < kLists; ++l) s.tile[l][1] = 32;
  s.step[kListForward] = f32 ? 32 : 64;
  s.step[kListDq] = f32 ? 32 : 64;
  s.step[kListDkv] = f32 ? 32 : 64;
  // Two four-wave or four one-wave workgroups per CU.  Also where a CU holds one
  // (wide dk, dv; fp32): half as many, longer pieces leave the GPU uneven (a
  // causal 8192-token step's dk and dv 690 -> 935 us), more pay for more partial
  // results (mixed images forward 59 -> 98 us at 1024).
  for (int l = 0; l < kLists; ++l) {
    s.fill[l][0] = 512;
    s.fill[l][1] = 1024;
  }
  return s;
}

namespace {

constexpr int kMinSteps = 4;                     // shortest split: 4 steps of the loop

struct Seq {
  int32_t q0, lq, k0, lk;
};

// keys [0, n) that the rows below `row_end` of the sequence see
int64_t keys_seen(const Seq& s, int64_t row_end, int group, bool causal) {
  if (!causal) return s.lk;
  const int64_t last = std::min<int64_t>(s.lq, (row_end + group - 1) / group) - 1;   // last token of the tile
  return std::max<int64_t>(0, std::min<int64_t>(s.lk, last + 1 + s.lk - s.lq));
}
// first row that sees key j
int64_t first_row(const Seq& s, int64_t j, int group, bool causal) {
  if (!causal) return 0;
  return std::max<int64_t>(0, j - (s.lk - (int64_t)s.lq)) * group;
}

void build(st_seqs* p, const std::vector<Seq>& seqs, int which) {
  AttnList& l = p->list[which];
  const int step = p->shape.step[which];
  const bool rows = which != kListDkv;
  int64_t steps[2] = {0, 0};
  for (int w = 0; w < 2; ++w) l.tile[w] = p->shape.tile[which][w];
  for (const Seq& s : seqs) {
    const int64_t extent = rows ? (int64_t)s.lq * p->group : s.lk;
    const int w = extent <= 2 * p->shape.tile[which][1] ? 1 : 0;
    for (int64_t at = 0; at < extent; at += l.tile[w]) {
      AttnItem it{s.q0, s.lq, s.k0, s.lk, (int32_t)at, 0, 0, -1};
      if (rows) {
        it.hi = (int32_t)keys_seen(s, std::min(extent, at + l.tile[w]), p->group, p->causal);
      } else {
        it.lo = (int32_t)std::min<int64_t>(first_row(s, at, p->group, p->causal), (int64_t)s.lq * p->group);
        it.hi = s.lq * p->group;
      }
      steps[w] += (it.hi - it.lo + step - 1) / step;
      l.item[w].push_back(it);
    }
  }
  for (int w = 0; w < 2; ++w) {
    const int64_t fill = p->shape.fill[which][w];
    const int64_t per = std::max<int64_t>(kMinSteps, (steps[w] * p->kv_heads + fill - 1) / fill);
    std::vector<AttnItem> out;
    out.reserve(l.item[w].size());
    for (const AttnItem& it : l.item[w]) {
      const int64_t n = (it.hi - it.lo + step - 1) / step;
      if (n < 2 * per) {
        out.push_back(it);
        continue;
      }
      const int64_t cuts = (n + per - 1) / per;
      AttnJoin j{it.q0, it.lq, it.k0, it.lk, it.at, (int32_t)l.parts[w], (int32_t)cuts, 0};
      l.join[w].push_back(j);
      for (int64_t c = 0; c < cuts; ++c) {
        AttnItem piece = it;
        piece.lo = (int32_t)(it.lo + n * c / cuts * step);
        piece.hi = c + 1 == cuts ? it.hi : (int32_t)(it.lo + n * (c + 1) / cuts * step);
        piece.part = (int32_t)l.parts[w]++;
        out.push_back(piece);
      }
    }
    std::stable_sort(out.begin(), out.end(),
                     [](const AttnItem& a, const AttnItem& b) { return a.hi - a.lo > b.hi - b.lo; });
    l.item[w].swap(out);
  }
}

}  // namespace

st_status seqs_device_table(st_seqs* p, hipStream_t stream) {
  std::lock_guard<std::mutex> lock(p->dev_mu);
  int dev = -1;
  st_status s = hip_check(hipGetDevice(&dev), "hipGetDevice");
  if (s != ST_OK) return s;
  if (p->d_table) {
    if (dev != p->dev_id) return fail(ST_ERR_INVALID_ARG, "the sequences' work tables live on another device");
    return ST_OK;
  }
  size_t bytes = 0;
  for (AttnList& l : p->list)
    for (int w = 0; w < 2; ++w) bytes += l.item[w].size() * sizeof(AttnItem) + l.join[w].size() * sizeof(AttnJoin);
  if (bytes == 0) return ST_OK;
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  s = hip_check(hipStreamIsCapturing(stream, &cap), "hipStreamIsCapturing");
  if (s != ST_OK) return s;
  if (cap != hipStreamCaptureStatusNone)
    return fail(ST_ERR_UNSUPPORTED,
                "the sequences' work tables are not on the device yet: call st_seqs_upload before capturing");
  std::vector<char> host(bytes);
  s = hip_check(hipMalloc(reinterpret_cast<void**>(&p->d_table), bytes), "sequence tables: hipMalloc");
  if (s != ST_OK) { p->d_table = nullptr; return s; }
  size_t at = 0;
  for (AttnList& l : p->list)
    for (int w = 0; w < 2; ++w) {
      l.d_item[w] = reinterpret_cast<const AttnItem*>(p->d_table + at);
      std::memcpy(host.data() + at, l.item[w].data(), l.item[w].size() * sizeof(AttnItem));
      at += l.item[w].size() * sizeof(AttnItem);
      l.d_join[w] = reinterpret_cast<const AttnJoin*>(p->d_table + at);
      std::memcpy(host.data() + at, l.join[w].data(), l.join[w].size() * sizeof(AttnJoin));
      at += l.join[w].size() * sizeof(AttnJoin);
    }
  s = hip_check(hipMemcpy(p->d_table, host.data(), bytes, hipMemcpyHostToDevice), "sequence tables: hipMemcpy");
  if (s != ST_OK) { (void)hipFree(p->d_table); p->d_table = nullptr; return s; }
  p->dev_id = dev;
  return ST_OK;
}

}  // namespace st

using namespace st;

extern "C" {

st_status st_plan_sequences(int32_t nseq, const int32_t* q_lens, const int32_t* k_lens_or_null, int32_t heads,
                            int32_t kv_heads, int32_t head_dim, st_dtype dtype, int32_t causal, st_seqs** out) {
  auto err = [](st_status s, const std::string& m) { return fail(s, "st_plan_sequences: " + m); };
  if (!out) return err(ST_ERR_INVALID_ARG, "NULL argument");
  *out = nullptr;
  if (nseq < 1 || !q_lens) return err(ST_ERR_INVALID_ARG, "at least one sequence and its lengths are needed");
  if (dtype != ST_F32 && dtype != ST_BF16) return err(ST_ERR_INVALID_ARG, "dtype must be ST_F32 or ST_BF16");
  if (heads < 1 || kv_heads < 1) return err(ST_ERR_INVALID_ARG, "heads and kv_heads must be >= 1");
  if (heads % kv_heads) return err(ST_ERR_BAD_SHAPE, "kv_heads must divide heads");
  if (head_dim < 8 || head_dim % 8 || head_dim > ST_MAX_HEAD_DIM)
    return err(ST_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 and at most 128");
  if (heads > 65536) return err(ST_ERR_UNSUPPORTED, "more than 65536 heads");
  const int32_t* k_lens = k_lens_or_null ? k_lens_or_null : q_lens;
  const int group = heads / kv_heads;
  int64_t tq = 0, tk = 0;
  std::vector<Seq> seqs;
  try {
    seqs.reserve(nseq);
    for (int i = 0; i < nseq; ++i) {
      if (q_lens[i] < 0 || k_lens[i] < 0) return err(ST_ERR_INVALID_ARG, "negative length");
      if ((int64_t)q_lens[i] * group >= (1ll << 30) || k_lens[i] >= (1 << 30))
        return err(ST_ERR_UNSUPPORTED, "a sequence of 2^30 rows or keys or more");
      seqs.push_back(Seq{(int32_t)tq, q_lens[i], (int32_t)tk, k_lens[i]});
      tq += q_lens[i];
      tk += k_lens[i];
      if (tq >= (1ll << 31) - 1 || tk >= (1ll << 31) - 1) return err(ST_ERR_UNSUPPORTED, "2^31 tokens or more");
    }
    st_seqs* p = new st_seqs;
    p->nseq = nseq;
    p->heads = heads;
    p->kv_heads = kv_heads;
    p->group = group;
    p->dim = head_dim;
    p->dp = attn_padded_dim(head_dim);
    p->causal = causal != 0;
    p->dtype = dtype;
    p->total_q = tq;
    p->total_k = tk;
    p->shape = attn_shape(dtype);
    try {
      for (int l = 0; l < kLists; ++l) build(p, seqs, l);
    } catch (...) {
      delete p;
      throw;
    }
    for (const AttnList& l : p->list)
      for (int w = 0; w < 2; ++w)
        if ((int64_t)l.item[w].size() * kv_heads >= (1ll << 31) || l.parts[w] * kv_heads >= (1ll << 31)) {
          delete p;
          return err(ST_ERR_UNSUPPORTED, "too many tiles");
        }
    *out = p;
  } catch (const std::bad_alloc&) {
    return err(ST_ERR_INVALID_ARG, "out of host memory");
  }
  return ST_OK;
}

st_status st_seqs_destroy(st_seqs* seqs) {
  if (!seqs) return fail(ST_ERR_INVALID_ARG, "st_seqs_destroy: NULL plan");
  st_status s = ST_OK;
  if (seqs->d_table) {
    int cur = -1;
    (void)hipGetDevice(&cur);
    if (cur != seqs->dev_id) (void)hipSetDevice(seqs->dev_id);
    s = hip_check(hipFree(seqs->d_table), "st_seqs_destroy: hipFree");
    if (cur >= 0 && cur != seqs->dev_id) (void)hipSetDevice(cur);
  }
  delete seqs;
  return s;
}

st_status st_seqs_upload(st_seqs* seqs, void* stream) {
  if (!seqs) return fail(ST_ERR_INVALID_ARG, "st_seqs_upload: NULL plan");
  st_status s = seqs_device_table(seqs, static_cast<hipStream_t>(stream));
  if (s != ST_OK) return s;
  return hip_check(hipStreamSynchronize(static_cast<hipStream_t>(stream)), "st_seqs_upload: hipStreamSynchronize");
}

}  // extern "C"
