// C ABI of libfcp (see include/fcp.h): argument validation, TMA descriptor
// encoding and kernel launches. Every check runs on the host before any
// launch; nothing here allocates device memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "kernels.h"
#include "plan.h"

namespace {

using fcp::Plan;

int64_t g_wait_ns = 2000000000LL;  // bounded device waits give up after 2 s

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

int num_sms() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && cache[dev]) return cache[dev];
  int n = 0;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (dev < 64) cache[dev] = n;
  return n;
}

// Token-major [rows][heads][d] 16-bit tensor, boxes of 64 x 1 x box_rows with the
// 128-byte swizzle (one swizzle panel of a 128-row tile, or of a part of one).
bool make_map(CUtensorMap* m, const void* ptr, int d, int heads, int64_t rows, bool f16 = false, int box_rows = 128) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// fp32 [rows][heads][d] tensor, boxes of 32 x 1 x box_rows with the 128-byte
// swizzle: the target of the backward's reduce-adds.
bool make_map_f32(CUtensorMap* m, void* ptr, int d, int heads, int64_t rows, int box_rows = 128) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)d * 4, (cuuint64_t)heads * d * 4};
  cuuint32_t box[3] = {32, 1, (cuuint32_t)box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, ptr, dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// e4m3 [rows][heads][d] tensor (one byte per element), boxes of d x 1 x 128
// (d = 128: one 128-byte swizzled row per key or query).
bool make_map_u8(CUtensorMap* m, void* ptr, int d, int heads, int64_t rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)heads * d};
  cuuint32_t box[3] = {(cuuint32_t)d, 1, 128};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, ptr, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

const int32_t* table(const fcp_dev_plan* dp, int tb) { return dp->base + dp->tables[tb]; }

// Host copy of a table entry (the serialized tables live in the plan).
int32_t host_at(const Plan* p, int tb, int64_t i) { return p->dev[p->tab_off[tb] + i]; }

int check_dims(const fcp_dims& d, const Plan* p) {
  if (d.T <= 0 || d.hq <= 0 || d.hkv <= 0) return FCP_ERR_INVALID_ARG;
  if (d.d != 64 && d.d != 128) return FCP_ERR_UNSUPPORTED;
  if (d.hq % d.hkv != 0) return FCP_ERR_UNSUPPORTED;
  if (p && d.T != p->T) return FCP_ERR_INVALID_ARG;
  return FCP_OK;
}

float softmax_scale(const fcp_dims& d) { return d.scale > 0.f ? d.scale : 1.0f / std::sqrt((float)d.d); }

int64_t remote_rows_of(const Plan* p, int32_t shard) {
  return shard < 0 ? p->total_remote : p->shards[shard].remote_rows;
}

}  // namespace

namespace fcp {
int64_t wait_limit_ns() { return g_wait_ns; }

// A device-plan handle must describe its host plan exactly: the kernels index
// the device tables with these offsets and counts, so a handle that was
// corrupted, hand-edited or bound to another plan is rejected before anything
// is launched.
int check_dev_plan(const fcp_dev_plan* dp, int32_t shard) {
  if (!dp || !dp->host || !dp->base) return FCP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dp->base) & 15) != 0) return FCP_ERR_INVALID_ARG;
  const Plan* p = dp->host;
  if (dp->n_shards != p->N || (int64_t)dp->T != p->T || dp->total_remote_rows != p->total_remote ||
      dp->bytes != (int64_t)p->dev.size() * 4)
    return FCP_ERR_INVALID_ARG;
  for (int t = 0; t < fcp::TB_COUNT; ++t)
    if (dp->tables[t] != p->tab_off[t] || dp->counts[t] != p->tab_cnt[t]) return FCP_ERR_INVALID_ARG;
  for (int t = fcp::TB_COUNT; t < 16; ++t)
    if (dp->tables[t] != 0 || dp->counts[t] != 0) return FCP_ERR_INVALID_ARG;
  if (shard < -1 || shard >= dp->n_shards) return FCP_ERR_INVALID_ARG;
  return FCP_OK;
}
}  // namespace fcp

using fcp::check_dev_plan;

extern "C" {

const char* fcp_strerror(int s) {
  switch (s) {
    case FCP_OK: return "ok";
    case FCP_ERR_INVALID_ARG: return "invalid argument";
    case FCP_ERR_UNSUPPORTED: return "unsupported shape";
    case FCP_ERR_CUDA: return "CUDA error";
    case FCP_ERR_TIMEOUT: return "bounded device wait expired";
    case FCP_ERR_INFEASIBLE: return "policy infeasible for this input";
    case FCP_ERR_CAPACITY: return "buffer too small";
    case FCP_ERR_MISSING_PART: return "partial result missing or duplicated";
    default: return "unknown status";
  }
}

int fcp_plan(const int32_t* doclens, int32_t n_docs, int32_t cp, int32_t policy,
             double target_imbalance, fcp_plan_t** out) {
  if (!out) return FCP_ERR_INVALID_ARG;
  *out = nullptr;
  return fcp::make_plan(doclens, n_docs, cp, policy, target_imbalance, out);
}

int fcp_plan_window(const fcp_plan_t* plan, int32_t window, int32_t sinks, fcp_plan_t** out) {
  if (!out) return FCP_ERR_INVALID_ARG;
  *out = nullptr;
  if (!plan) return FCP_ERR_INVALID_ARG;
  try {
    return fcp::make_window_plan(*plan, window, sinks, out);
  } catch (const std::bad_alloc&) {  // no host memory for the tables
    return FCP_ERR_CAPACITY;
  }
}

void fcp_plan_free(fcp_plan_t* plan) { delete plan; }

int fcp_plan_shard(const fcp_plan_t* plan, int32_t shard, fcp_shard_view* out) {
  if (!plan || !out || shard < 0 || shard >= plan->N) return FCP_ERR_INVALID_ARG;
  const fcp::Shard& s = plan->shards[shard];
  static_assert(sizeof(fcp::Piece) == sizeof(fcp_range), "piece layout");
  out->n_pieces = (int32_t)s.pieces.size();
  out->pieces = reinterpret_cast<const fcp_range*>(s.pieces.data());
  out->n_need = (int32_t)s.kv_need.size();
  out->kv_need = s.kv_need.data();
  out->n_remote = (int32_t)s.kv_remote.size();
  out->kv_remote = s.kv_remote.data();
  out->tokens = s.tokens;
  out->useful_pairs = s.W;
  out->remote_rows = s.remote_rows;
  out->kbuf_base = s.kbuf_base;
  out->fwd_tiles = s.fwd_tiles;
  out->fwd_qtiles = s.fwd_qtiles;
  out->fwd_masked = s.fwd_masked;
  out->bwd_tiles = s.bwd_tiles;
  out->bwd_ktiles = s.bwd_ktiles;
  return FCP_OK;
}

int fcp_plan_query_indices(const fcp_plan_t* plan, int32_t shard, int32_t* idx, int64_t cap,
                           int64_t* n) {
  if (!plan || !n || shard < 0 || shard >= plan->N || cap < 0) return FCP_ERR_INVALID_ARG;
  const fcp::Shard& s = plan->shards[shard];
  *n = s.tokens;
  if (cap < s.tokens) return FCP_ERR_CAPACITY;
  if (!idx && s.tokens > 0) return FCP_ERR_INVALID_ARG;
  int64_t k = 0;
  for (const fcp::Piece& p : s.pieces)
    for (int32_t t = p.start; t < p.end; ++t) idx[k++] = t;
  return FCP_OK;
}

int fcp_plan_stats(const fcp_plan_t* plan, fcp_plan_stats_t* out) {
  if (!plan || !out) return FCP_ERR_INVALID_ARG;
  std::memset(out, 0, sizeof(*out));
  out->cp = plan->N;
  out->n_docs = (int32_t)plan->D.size();
  out->T = plan->T;
  out->imbalance = plan->imbalance;
  for (const fcp::Shard& s : plan->shards) {
    out->max_pairs = std::max(out->max_pairs, s.W);
    out->total_pairs += s.W;
    out->remote_rows_total += s.remote_rows;
    out->remote_rows_max = std::max(out->remote_rows_max, s.remote_rows);
  }
  out->eq4_tokens = plan->eq4;
  out->eq5_tokens = plan->eq5;
  out->eq2_max_dev = plan->eq2dev;
  out->iterations = plan->iterations;
  for (uint8_t f : plan->per_doc) out->n_per_doc += f;
  return FCP_OK;
}

int fcp_plan_per_doc_flags(const fcp_plan_t* plan, int32_t* out, int32_t n_docs) {
  if (!plan || !out || n_docs != (int32_t)plan->D.size()) return FCP_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n_docs; ++i) out[i] = plan->per_doc[i];
  return FCP_OK;
}

int64_t fcp_plan_device_bytes(const fcp_plan_t* plan) {
  return plan ? (int64_t)plan->dev.size() * 4 : 0;
}

int fcp_plan_device_image(const fcp_plan_t* plan, void* dst, int64_t bytes) {
  if (!plan || !dst) return FCP_ERR_INVALID_ARG;
  const int64_t need = fcp_plan_device_bytes(plan);
  if (bytes < need) return FCP_ERR_CAPACITY;
  std::memcpy(dst, plan->dev.data(), (size_t)need);
  return FCP_OK;
}

int fcp_plan_bind(const fcp_plan_t* plan, const void* dev_buf, int64_t bytes, fcp_dev_plan* out) {
  if (!plan || !dev_buf || !out) return FCP_ERR_INVALID_ARG;
  if (!aligned16(dev_buf)) return FCP_ERR_INVALID_ARG;
  const int64_t need = fcp_plan_device_bytes(plan);
  if (bytes < need) return FCP_ERR_CAPACITY;
  std::memset(out, 0, sizeof(*out));
  out->host = plan;
  out->base = static_cast<const int32_t*>(dev_buf);
  out->bytes = need;
  out->n_shards = plan->N;
  out->T = (int32_t)plan->T;
  out->total_remote_rows = plan->total_remote;
  for (int t = 0; t < fcp::TB_COUNT; ++t) {
    out->tables[t] = plan->tab_off[t];
    out->counts[t] = plan->tab_cnt[t];
  }
  return FCP_OK;
}

int fcp_plan_upload(const fcp_plan_t* plan, void* dev_buf, int64_t bytes, void* stream,
                    fcp_dev_plan* out) {
  const int st = fcp_plan_bind(plan, dev_buf, bytes, out);
  if (st != FCP_OK) return st;
  if (cudaMemcpyAsync(dev_buf, plan->dev.data(), (size_t)out->bytes, cudaMemcpyHostToDevice,
                      static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return FCP_ERR_CUDA;
  return FCP_OK;
}

// Workspace layout (each region 256-byte aligned): [0, 256) error word (byte
// 0) and the persistent kernels' work counter (byte kWorkCounterOff); the
// backward's row statistics D_i and LSE (fp32 [Hq][T] each); fp16 copies of Q and dO ([T][Hq][d] each, backward); fp16
// copies of V ([T][Hkv][d]) and of the received V rows ([R][Hkv][d], R = all
// shards' remote rows of the plan), the forward's P*V operands; e4m3 copies
// of Q, K and the received K rows; partial sums of the norm weights' gradients;
// the biased backward's sums of dS by distance. Only the header holds what a
// call leaves for the next one (the zeros of its counters): the rest moves with
// the sizes, and one workspace may serve several.
constexpr int64_t kWorkCounterOff = 64;

struct WsLayout {
  int64_t delta, lse2, q16, do16, v16, vb16, q8, k8, kb8, partial, by_distance, total;
};

// Header words of the e4m3 Q K^T forward: amax bits of Q and K, then their
// scales 2^kq and 2^kk.
constexpr int64_t kQkAmaxOff = 128;
constexpr int64_t kQkScaleOff = 136;
// Range of the backward's operands (zero between calls).
constexpr int64_t kRangeOff = 144;
// Diagnostic counter of the forward: online-softmax rescales of O after a
// query tile's first key tile (one count per warp and event).
constexpr int64_t kRescaleCountOff = 192;
// Tickets of the norm weights' gradients (zero between calls).
constexpr int64_t kTicketsOff = 68;
static_assert(kRangeOff + (int64_t)sizeof(fcp::BwdRange) <= kRescaleCountOff, "range inside the header");
static_assert(kTicketsOff + (1 + fcp::kNormRopeGroups) * 4 <= kQkAmaxOff, "tickets inside the header");

static int64_t ws_align(int64_t x) { return (x + 255) / 256 * 256; }

static WsLayout ws_layout(const fcp_dims& d, int64_t remote_rows) {
  const int64_t T = std::max(d.T, 0), hq = std::max(d.hq, 0), hkv = std::max(d.hkv, 0),
                dd = std::max(d.d, 0);
  WsLayout w;
  w.delta = 256;
  w.lse2 = w.delta + ws_align(hq * T * 4);
  w.q16 = w.lse2 + ws_align(hq * T * 4);
  w.do16 = w.q16 + ws_align(T * hq * dd * 2);
  w.v16 = w.do16 + ws_align(T * hq * dd * 2);
  w.vb16 = w.v16 + ws_align(T * hkv * dd * 2);
  const int64_t R = std::max<int64_t>(remote_rows, 0);
  w.q8 = w.vb16 + ws_align(R * hkv * dd * 2);
  w.k8 = w.q8 + ws_align(T * hq * dd);
  w.kb8 = w.k8 + ws_align(T * hkv * dd);
  w.partial = w.kb8 + ws_align(R * hkv * dd);
  w.by_distance = w.partial + ws_align((fcp::kNormRopeMaxCtas + fcp::kNormRopeGroups) * 2 * dd * 4);
  w.total = w.by_distance + ws_align(hq * fcp::kTableDistances * 4);
  return w;
}

int64_t fcp_workspace_bytes(fcp_dims dims, const fcp_plan_t* plan) {
  return ws_layout(dims, plan ? plan->total_remote : 0).total;
}

int fcp_gather_kv(const void* k, const void* v, const fcp_dev_plan* plan, int32_t shard,
                  int32_t hkv, int32_t d, void* kbuf, void* vbuf, void* stream) {
  int st = check_dev_plan(plan, shard);
  if (st) return st;
  if (hkv <= 0 || (d != 64 && d != 128)) return FCP_ERR_UNSUPPORTED;
  const Plan* p = plan->host;
  const int64_t rows = remote_rows_of(p, shard);
  if (rows == 0) return FCP_OK;
  if (!k || !v || !kbuf || !vbuf) return FCP_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(kbuf) || !aligned16(vbuf)) return FCP_ERR_INVALID_ARG;
  int32_t t0 = 0, t1 = plan->counts[fcp::TB_COPY], shift = 0;
  if (shard >= 0) {
    t0 = host_at(p, fcp::TB_CSHARD, shard);
    t1 = host_at(p, fcp::TB_CSHARD, shard + 1);
    shift = (int32_t)p->shards[shard].kbuf_base;
  }
  return fcp::launch_gather(k, v, table(plan, fcp::TB_COPY) + 4 * t0, t1 - t0, shift,
                            (int64_t)hkv * d * 2, kbuf, vbuf, plan->T, (int32_t)rows, num_sms(),
                            static_cast<cudaStream_t>(stream));
}

// Whether two arrays of n floats share a byte.
static bool ranges_meet(const float* a, const float* b, int64_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b), len = 4 * (uintptr_t)n;
  return x < y + len && y < x + len;
}

// The table's pointer and the bucket starts (host): the first distance of the
// first bucket is 0 and none is below the one before.
static int check_bias(const fcp_rel_bias* b, const fcp_dims& dims) {
  if (softmax_scale(dims) < 1e-30f) return FCP_ERR_UNSUPPORTED;  // the kernels add biases over the scale
  if (!b || !b->bias || !b->starts || (reinterpret_cast<uintptr_t>(b->bias) & 3)) return FCP_ERR_INVALID_ARG;
  if (b->n_buckets < 1 || (b->zero_grads != 0 && b->zero_grads != 1)) return FCP_ERR_INVALID_ARG;
  if (b->n_buckets > FCP_MAX_BUCKETS) return FCP_ERR_UNSUPPORTED;
  if (b->starts[0] != 0) return FCP_ERR_INVALID_ARG;
  for (int32_t u = 1; u < b->n_buckets; ++u)
    if (b->starts[u] < b->starts[u - 1]) return FCP_ERR_INVALID_ARG;
  return FCP_OK;
}

static void set_bias(fcp::BiasParams* p, const fcp_rel_bias* b, float* dbias, float* by_distance) {
  static_assert(FCP_MAX_BUCKETS == fcp::kMaxBuckets, "bucket count");
  p->bias = b->bias;
  p->dbias = dbias;
  p->by_distance = by_distance;
  // Tiles of several buckets reach 254 distances past the last one's first.
  p->n_distances = std::min(std::min(b->starts[b->n_buckets - 1], fcp::kTableDistances) + 256, fcp::kTableDistances);
  p->n = b->n_buckets;
  std::copy(b->starts, b->starts + b->n_buckets, p->starts);
}

// How the biased backward cuts a KV head's query heads into units of their own
// (dK and dV are added up over the units). One unit for all of them reads K and
// V once, but where a long document's first key tiles are a large share of the
// work the other CTAs wait for them. Estimated as the longer of the longest unit
// and the mean a CTA, a unit's beginning and end counted as three steps. 7001
// tokens in documents of up to 4096, groups of three heads: 224 us in one unit,
// 198 in two, 136 in three. With eight units a CTA and more there is nothing to
// even out: one document of 16K, groups of eight, 10.5 a CTA, 2.91 ms whole,
// four heads a unit 2.94, two 3.05, one 3.36; the 32K workload, groups of four,
// 4.83 whole, two heads a unit 5.13, one 5.78.
static void cut_groups(fcp::BiasParams* b, const Plan* p, int32_t shard, int32_t n_items, const fcp_dims& dims, int sms) {
  const int G = dims.hq / dims.hkv;
  b->parts = 1;
  b->part_heads = G;
  if (G == 1 || (int64_t)n_items * dims.hkv >= 8 * (int64_t)sms) return;  // units enough to even out
  constexpr double kEnds = 3;
  const int32_t t0 = shard < 0 ? 0 : host_at(p, fcp::TB_BSHARD, shard);
  int64_t sum = 0, longest = 0;
  for (int32_t i = 0; i < n_items; ++i) {
    const int64_t t = (int64_t)(t0 + i) * fcp::kBwdTileInts;
    const int64_t nq = (int64_t)host_at(p, fcp::TB_BTILES, t + 6) + host_at(p, fcp::TB_BTILES, t + 9);
    sum += nq;
    longest = std::max(longest, nq);
  }
  double best = INFINITY;
  for (int heads = G; heads >= 1; --heads) {
    const int parts = (G + heads - 1) / heads;
    if ((G + parts - 1) / parts != heads) continue;  // as many parts with fewer heads
    const double mean = ((double)sum * G + kEnds * n_items * parts) * dims.hkv / sms;
    const double cost = std::max(longest * heads + kEnds, mean);
    if (cost < best) {
      best = cost;
      b->parts = parts;
      b->part_heads = heads;
    }
  }
}

// The window of a plan and the maps of tiles that hold sinks: k, v and the
// received kb, vb as the launch's own maps name them (v's as fp16 copies in the
// forward), dk and dv for a backward.
static bool set_window(fcp::WindowParams* w, const Plan* p, const fcp_dims& dims, const void* k, const void* v,
                       const void* kb, const void* vb, int64_t kb_rows, bool v_f16, float* dk, float* dv) {
  w->window = p->window;
  w->sinks = p->sinks;
  w->slots = fcp::sink_slots(p->sinks);
  if (w->slots == 0) return true;
  const int rest = fcp::kTileN - w->slots;
  auto both = [&](CUtensorMap* sinks, CUtensorMap* others, const void* at, int64_t rows, bool f16) {
    return make_map(sinks, at, dims.d, dims.hkv, rows, f16, w->slots) &&
           make_map(others, at, dims.d, dims.hkv, rows, f16, rest);
  };
  bool ok = both(&w->k_sinks, &w->k_rest, k, dims.T, false) && both(&w->v_sinks, &w->v_rest, v, dims.T, v_f16) &&
            both(&w->kb_sinks, &w->kb_rest, kb, kb_rows, false) && both(&w->vb_sinks, &w->vb_rest, vb, kb_rows, v_f16);
  if (dk)
    ok = ok && make_map_f32(&w->dk_sinks, dk, dims.d, dims.hkv, dims.T, w->slots) &&
         make_map_f32(&w->dk_rest, dk, dims.d, dims.hkv, dims.T, rest) &&
         make_map_f32(&w->dv_sinks, dv, dims.d, dims.hkv, dims.T, w->slots) &&
         make_map_f32(&w->dv_rest, dv, dims.d, dims.hkv, dims.T, rest);
  return ok;
}

// Forward over the plan's gathered key layout (ring < -1: own rows from K/V,
// received rows from kbuf/vbuf) or in ring order (ring >= -1: every needed key
// from its owner's rows of K/V, owners visited by ring distance; ring = -1 all
// of them in one pass, ring = s only the keys of owner (shard - s) mod N).
static int attn_fwd_impl(const void* q, const void* k, const void* v, const void* kbuf, const void* vbuf,
                         const fcp_dev_plan* plan, int32_t shard, int32_t kv_lo, int32_t kv_hi,
                         fcp_dims dims, int32_t out_dtype, void* out, float* lse, void* ws,
                         int64_t ws_bytes, void* stream, int32_t ring, bool qk8 = false,
                         const fcp_rel_bias* bias = nullptr) {
  const bool ring_order = ring >= -1;
  int st = check_dev_plan(plan, shard);
  if (st) return st;
  const Plan* p = plan->host;
  if ((st = check_dims(dims, p))) return st;
  if (p->window > 0 && (ring_order || qk8 || bias)) return FCP_ERR_UNSUPPORTED;
  if (!q || !k || !v || !out || !lse || !ws) return FCP_ERR_INVALID_ARG;
  if (out_dtype != FCP_OUT_BF16 && out_dtype != FCP_OUT_F32) return FCP_ERR_INVALID_ARG;
  if (kv_lo < 0 || kv_hi > dims.T || kv_lo > kv_hi) return FCP_ERR_INVALID_ARG;
  const WsLayout wl = ws_layout(dims, p->total_remote);
  if (ws_bytes < wl.total) return FCP_ERR_CAPACITY;
  if (ring_order && ring >= plan->n_shards) return FCP_ERR_INVALID_ARG;
  const int64_t rrows = ring_order ? 0 : remote_rows_of(p, shard);
  if (rrows > 0 && (!kbuf || !vbuf)) return FCP_ERR_INVALID_ARG;
  for (const void* ptr : {q, k, v, (const void*)out, (const void*)lse, (const void*)ws})
    if (!aligned16(ptr)) return FCP_ERR_INVALID_ARG;
  if (rrows > 0 && (!aligned16(kbuf) || !aligned16(vbuf))) return FCP_ERR_INVALID_ARG;

  // fp16 copies of V and of the received V rows: the P*V operands.
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  char* wsb = static_cast<char*>(ws);
  void* v16 = wsb + wl.v16;
  void* vb16 = wsb + wl.vb16;
  int* counter = reinterpret_cast<int*>(wsb + kWorkCounterOff);
  if (qk8) {
    // e4m3 copies of Q, K and the received K rows (with K's scale: they are
    // copies of K rows), each tensor with its own power-of-two scale.
    if (dims.d != 128) return FCP_ERR_UNSUPPORTED;
    unsigned* amax = reinterpret_cast<unsigned*>(wsb + kQkAmaxOff);
    float* scales = reinterpret_cast<float*>(wsb + kQkScaleOff);
    if (cudaMemsetAsync(amax, 0, 2 * sizeof(unsigned), cs) != cudaSuccess) return FCP_ERR_CUDA;
    int sq = fcp::launch_quant_e4m3(q, wsb + wl.q8, (int64_t)dims.T * dims.hq * dims.d, amax, scales,
                                    num_sms(), cs);
    if (sq == FCP_OK)
      sq = fcp::launch_quant_e4m3(k, wsb + wl.k8, (int64_t)dims.T * dims.hkv * dims.d, amax + 1, scales + 1,
                                  num_sms(), cs);
    if (sq == FCP_OK && rrows > 0)
      sq = fcp::launch_quant_e4m3_with(kbuf, wsb + wl.kb8, rrows * dims.hkv * dims.d, amax + 1, num_sms(), cs);
    if (sq) return sq;
  }
  if (int st2 = fcp::launch_convert_f16(v, v16, (int64_t)dims.T * dims.hkv * dims.d, vbuf, vb16,
                                        rrows * dims.hkv * dims.d, static_cast<int*>(ws), counter, num_sms(), cs))
    return st2;

  fcp::FwdLaunch a;
  std::memset(&a, 0, sizeof(a));
  bool ok = make_map(&a.tm_v, v16, dims.d, dims.hkv, dims.T, true);
  if (qk8) {
    ok = ok && make_map_u8(&a.tm_q, wsb + wl.q8, dims.d, dims.hq, dims.T) &&
         make_map_u8(&a.tm_k, wsb + wl.k8, dims.d, dims.hkv, dims.T) &&
         make_map_u8(&a.tm_kb, rrows > 0 ? wsb + wl.kb8 : wsb + wl.k8, dims.d, dims.hkv, rrows > 0 ? rrows : dims.T);
  } else {
    ok = ok && make_map(&a.tm_q, q, dims.d, dims.hq, dims.T) && make_map(&a.tm_k, k, dims.d, dims.hkv, dims.T) &&
         make_map(&a.tm_kb, rrows > 0 ? kbuf : k, dims.d, dims.hkv, rrows > 0 ? rrows : dims.T);
  }
  ok = ok && make_map(&a.tm_vb, rrows > 0 ? vb16 : v16, dims.d, dims.hkv, rrows > 0 ? rrows : dims.T, true);
  if (!ok) return FCP_ERR_CUDA;
  a.qk8 = qk8;
  fcp::FwdParams& fp = a.p;
  fp.pieces = table(plan, ring_order ? fcp::TB_RPIECES : fcp::TB_PIECES);
  fp.segs = table(plan, ring_order ? fcp::TB_RSEGS : fcp::TB_SEGS);
  fp.seg_filter = ring_order ? ring : -1;
  fp.tiles = table(plan, fcp::TB_FTILES);
  if (shard < 0) {
    fp.order = table(plan, fcp::TB_FORDER);
    fp.n_items = plan->counts[fcp::TB_FTILES];
    fp.kbuf_shift = 0;
  } else {
    const int32_t t0 = host_at(p, fcp::TB_FSHARD, shard), t1 = host_at(p, fcp::TB_FSHARD, shard + 1);
    fp.order = table(plan, fcp::TB_IDENT) + t0;
    fp.n_items = t1 - t0;
    fp.kbuf_shift = ring_order ? 0 : (int32_t)p->shards[shard].kbuf_base;
  }
  fp.kv_lo = kv_lo;
  fp.kv_hi = kv_hi;
  fp.T = dims.T;
  fp.hq = dims.hq;
  fp.hkv = dims.hkv;
  fp.scale_log2 = softmax_scale(dims) * 1.4426950408889634f;
  fp.out_f32 = out_dtype == FCP_OUT_F32;
  fp.out = out;
  fp.lse = lse;
  fp.err = static_cast<int*>(ws);
  fp.work_counter = counter;
  fp.qk_scale = qk8 ? reinterpret_cast<const float*>(wsb + kQkScaleOff) : nullptr;
  fp.rescale_count = reinterpret_cast<int*>(wsb + kRescaleCountOff);
  fp.n_tiles = plan->counts[fcp::TB_FTILES];
  fp.n_pieces = plan->counts[ring_order ? fcp::TB_RPIECES : fcp::TB_PIECES];
  fp.n_segs = plan->counts[ring_order ? fcp::TB_RSEGS : fcp::TB_SEGS];
  fp.kb_rows = rrows > 0 ? (int32_t)rrows : dims.T;
  fp.wait_ns = g_wait_ns;
  a.d = dims.d;
  a.num_sms = num_sms();
  if ((a.has_bias = bias != nullptr)) set_bias(&a.bias, bias, nullptr, nullptr);
  if ((a.has_window = p->window > 0) &&
      !set_window(&a.window, p, dims, k, v16, rrows > 0 ? kbuf : k, rrows > 0 ? vb16 : v16, rrows > 0 ? rrows : dims.T, true,
                  nullptr, nullptr))
    return FCP_ERR_CUDA;
  if (a.has_window) {
    const int32_t d0 = shard < 0 ? 0 : host_at(p, fcp::TB_RSEGS, shard);
    a.window.doubles = table(plan, fcp::TB_RPIECES) + 4 * (int64_t)d0;
    a.window.n_doubles = (shard < 0 ? plan->counts[fcp::TB_RPIECES] : host_at(p, fcp::TB_RSEGS, shard + 1)) - d0;
  }
  return fcp::launch_attn_fwd(a, cs);
}

int fcp_attn_fwd(const void* q, const void* k, const void* v, const void* kbuf, const void* vbuf,
                 const fcp_dev_plan* plan, int32_t shard, int32_t kv_lo, int32_t kv_hi,
                 fcp_dims dims, int32_t out_dtype, void* out, float* lse, void* ws,
                 int64_t ws_bytes, void* stream) {
  return attn_fwd_impl(q, k, v, kbuf, vbuf, plan, shard, kv_lo, kv_hi, dims, out_dtype, out, lse, ws,
                       ws_bytes, stream, -2);
}

int fcp_attn_fwd_qk8(const void* q, const void* k, const void* v, const void* kbuf, const void* vbuf,
                     const fcp_dev_plan* plan, int32_t shard, int32_t kv_lo, int32_t kv_hi, fcp_dims dims,
                     int32_t out_dtype, void* out, float* lse, void* ws, int64_t ws_bytes, void* stream) {
  return attn_fwd_impl(q, k, v, kbuf, vbuf, plan, shard, kv_lo, kv_hi, dims, out_dtype, out, lse, ws,
                       ws_bytes, stream, -2, true);
}

int fcp_attn_fwd_bias(const void* q, const void* k, const void* v, const void* kbuf, const void* vbuf,
                      const fcp_rel_bias* bias, const fcp_dev_plan* plan, int32_t shard, int32_t kv_lo, int32_t kv_hi,
                      fcp_dims dims, int32_t out_dtype, void* out, float* lse, void* ws, int64_t ws_bytes,
                      void* stream) {
  const int st = check_bias(bias, dims);
  if (st) return st;
  return attn_fwd_impl(q, k, v, kbuf, vbuf, plan, shard, kv_lo, kv_hi, dims, out_dtype, out, lse, ws, ws_bytes, stream,
                       -2, false, bias);
}

int fcp_rel_buckets(int32_t n_buckets, int32_t max_distance, int32_t* starts) {
  if (!starts || n_buckets < 2) return FCP_ERR_INVALID_ARG;
  if (n_buckets > FCP_MAX_BUCKETS) return FCP_ERR_UNSUPPORTED;
  const int32_t exact = n_buckets / 2, far = n_buckets - exact;
  if (max_distance <= exact) return FCP_ERR_INVALID_ARG;
  for (int32_t u = 0; u < n_buckets; ++u) {
    // The smallest distance x with floor(far ln(x / exact) / ln(max / exact)) >= u - exact.
    const double x = u <= exact ? u : exact * std::pow((double)max_distance / exact, (double)(u - exact) / far);
    const double near = std::nearbyint(x);  // a distance that the power meets but for its rounding
    starts[u] = (int32_t)(std::fabs(x - near) <= 1e-9 * x ? near : std::ceil(x));
    if (u > 0) starts[u] = std::max(starts[u], starts[u - 1]);
  }
  return FCP_OK;
}

int fcp_quant_e4m3(const void* x, int64_t n, void* out, float* scale_out, void* scratch, void* stream) {
  if (n < 0 || n % 8 != 0) return FCP_ERR_INVALID_ARG;
  if (n == 0) return FCP_OK;
  if (!x || !out || !scale_out || !scratch) return FCP_ERR_INVALID_ARG;
  if (!aligned16(x) || (reinterpret_cast<uintptr_t>(out) & 7) || (reinterpret_cast<uintptr_t>(scratch) & 3))
    return FCP_ERR_INVALID_ARG;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(scratch, 0, sizeof(unsigned), cs) != cudaSuccess) return FCP_ERR_CUDA;
  return fcp::launch_quant_e4m3(x, out, n, static_cast<unsigned*>(scratch), scale_out, num_sms(), cs);
}

int fcp_round_bf16(const float* x, int64_t n, void* out, void* stream) {
  if (n < 0 || n % 8 != 0) return FCP_ERR_INVALID_ARG;
  if (n == 0) return FCP_OK;
  if (!x || !out || !aligned16(x) || !aligned16(out)) return FCP_ERR_INVALID_ARG;
  return fcp::launch_round_bf16(x, out, n, num_sms(), static_cast<cudaStream_t>(stream));
}

int fcp_attn_fwd_ring(const void* q, const void* k, const void* v, const fcp_dev_plan* plan,
                      int32_t shard, int32_t ring_step, fcp_dims dims, int32_t out_dtype, void* out,
                      float* lse, void* ws, int64_t ws_bytes, void* stream) {
  if (ring_step < -1) return FCP_ERR_INVALID_ARG;
  return attn_fwd_impl(q, k, v, nullptr, nullptr, plan, shard, 0, dims.T, dims, out_dtype, out, lse, ws,
                       ws_bytes, stream, ring_step);
}

int fcp_merge(const float* o_parts, const float* lse_parts, int32_t B, int64_t rows, int32_t hq,
              int32_t d, void* out, float* lse_out, void* stream) {
  if (B < 1 || rows < 0 || hq < 1) return FCP_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FCP_ERR_UNSUPPORTED;
  if (B > d / 4 || rows * hq >= (int64_t(1) << 30)) return FCP_ERR_UNSUPPORTED;
  if (rows == 0) return FCP_OK;
  if (!o_parts || !lse_parts || !out || !lse_out) return FCP_ERR_INVALID_ARG;
  if (!aligned16(o_parts) || !aligned16(out)) return FCP_ERR_INVALID_ARG;
  return fcp::launch_merge(o_parts, lse_parts, B, rows, hq, d, out, lse_out, num_sms(),
                           static_cast<cudaStream_t>(stream));
}

int fcp_merge_ring(const fcp_dev_plan* plan, const float* o_parts, const float* lse_parts,
                   const int32_t* part_step, int32_t B, int32_t hq, int32_t d, void* out, float* lse_out,
                   void* stream) {
  int st = check_dev_plan(plan, -1);
  if (st) return st;
  if (!part_step && B > 0) return FCP_ERR_INVALID_ARG;
  const int32_t N = plan->n_shards;
  if (B != N) return FCP_ERR_MISSING_PART;
  std::vector<uint8_t> seen(N, 0);
  for (int32_t b = 0; b < B; ++b) {
    const int32_t s = part_step[b];
    if (s < 0 || s >= N || seen[s]) return FCP_ERR_MISSING_PART;
    seen[s] = 1;
  }
  return fcp_merge(o_parts, lse_parts, B, plan->T, hq, d, out, lse_out, stream);
}

static int attn_bwd_impl(const void* q, const void* k, const void* v, const void* kbuf, const void* vbuf,
                         const void* out, int32_t out_dtype, const float* lse, const void* dout,
                         const fcp_dev_plan* plan, int32_t shard, fcp_dims dims, float* dq, float* dk,
                         float* dv, void* ws, int64_t ws_bytes, void* stream, const fcp_rel_bias* bias,
                         float* dbias) {
  int st = check_dev_plan(plan, shard);
  if (st) return st;
  const Plan* p = plan->host;
  if ((st = check_dims(dims, p))) return st;
  if (p->window > 0 && bias) return FCP_ERR_UNSUPPORTED;
  if (!q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv || !ws) return FCP_ERR_INVALID_ARG;
  if (out_dtype != FCP_OUT_BF16 && out_dtype != FCP_OUT_F32) return FCP_ERR_INVALID_ARG;
  const WsLayout wl = ws_layout(dims, p->total_remote);
  if (ws_bytes < wl.total) return FCP_ERR_CAPACITY;
  const int64_t rrows = remote_rows_of(p, shard);
  if (rrows > 0 && (!kbuf || !vbuf)) return FCP_ERR_INVALID_ARG;
  for (const void* ptr : {q, k, v, out, (const void*)lse, dout, (const void*)dq, (const void*)dk,
                          (const void*)dv, (const void*)ws})
    if (!aligned16(ptr)) return FCP_ERR_INVALID_ARG;
  if (rrows > 0 && (!aligned16(kbuf) || !aligned16(vbuf))) return FCP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* wsb = static_cast<char*>(ws);
  float* delta = reinterpret_cast<float*>(wsb + wl.delta);
  float* lse2 = reinterpret_cast<float*>(wsb + wl.lse2);
  fcp::BwdRange* range = reinterpret_cast<fcp::BwdRange*>(wsb + kRangeOff);
  void* q16 = wsb + wl.q16;
  void* do16 = wsb + wl.do16;

  if (bias && bias->zero_grads) {
    const int64_t n = (int64_t)dims.T * dims.hkv * dims.d * sizeof(float);
    if (cudaMemsetAsync(dk, 0, n, s) != cudaSuccess || cudaMemsetAsync(dv, 0, n, s) != cudaSuccess ||
        cudaMemsetAsync(dbias, 0, sizeof(float) * dims.hq * bias->n_buckets, s) != cudaSuccess)
      return FCP_ERR_CUDA;
  }
  // Row statistics and dQ = 0 for the shard's query rows, and the operands' range.
  int32_t r0 = 0, r1 = plan->counts[fcp::TB_ROWS];
  if (shard >= 0) {
    r0 = host_at(p, fcp::TB_RSHARD, shard);
    r1 = host_at(p, fcp::TB_RSHARD, shard + 1);
  }
  int32_t piece0 = 0, n_pieces = 0;  // this shard's pieces in the table
  for (int32_t j = 0; j <= shard; ++j) {
    piece0 += n_pieces;
    n_pieces = (int32_t)p->shards[j].pieces.size();
  }
  fcp::PreLaunch pre;
  std::memset(&pre, 0, sizeof(pre));
  pre.out = out;
  pre.out_f32 = out_dtype == FCP_OUT_F32;
  pre.lse = lse;
  pre.dout = static_cast<const __nv_bfloat16*>(dout);
  pre.q = static_cast<const __nv_bfloat16*>(q);
  pre.v = static_cast<const __nv_bfloat16*>(v);
  pre.vbuf = static_cast<const __nv_bfloat16*>(vbuf);
  pre.v_rows = shard < 0 ? 0 : rrows;  // over all shards they are copies of V's own rows
  pre.rows = table(plan, fcp::TB_ROWS);
  pre.order = table(plan, fcp::TB_IDENT) + r0;
  pre.n_chunks = r1 - r0;
  pre.n_rows_table = plan->counts[fcp::TB_ROWS];
  pre.T = dims.T;
  pre.hq = dims.hq;
  pre.hkv = dims.hkv;
  pre.delta = delta;
  pre.lse2 = lse2;
  pre.dq = dq;
  pre.q16 = static_cast<__half*>(q16);
  pre.do16 = static_cast<__half*>(do16);
  pre.range = range;
  pre.pieces = table(plan, fcp::TB_PIECES) + 8 * (int64_t)piece0;
  pre.n_pieces = n_pieces;
  pre.any_tiles = p->window > 0;
  pre.num_sms = num_sms();
  pre.err = static_cast<int*>(ws);
  pre.zero_word = reinterpret_cast<int*>(wsb + kWorkCounterOff);
  st = fcp::launch_bwd_preprocess(pre, dims.d, s);
  if (st) return st;

  fcp::BwdLaunch a;
  std::memset(&a, 0, sizeof(a));
  bool ok = make_map(&a.tm_q, q16, dims.d, dims.hq, dims.T, true) &&
            make_map(&a.tm_do, do16, dims.d, dims.hq, dims.T, true) &&
            make_map(&a.tm_k, k, dims.d, dims.hkv, dims.T) && make_map(&a.tm_v, v, dims.d, dims.hkv, dims.T) &&
            make_map_f32(&a.tm_dq, dq, dims.d, dims.hq, dims.T) &&
            make_map_f32(&a.tm_dk, dk, dims.d, dims.hkv, dims.T) &&
            make_map_f32(&a.tm_dv, dv, dims.d, dims.hkv, dims.T);
  if (rrows > 0)
    ok = ok && make_map(&a.tm_kb, kbuf, dims.d, dims.hkv, rrows) &&
         make_map(&a.tm_vb, vbuf, dims.d, dims.hkv, rrows);
  else
    ok = ok && make_map(&a.tm_kb, k, dims.d, dims.hkv, dims.T) && make_map(&a.tm_vb, v, dims.d, dims.hkv, dims.T);
  if (!ok) return FCP_ERR_CUDA;
  fcp::BwdParams& bp = a.p;
  bp.pieces = table(plan, fcp::TB_PIECES);
  bp.tiles = table(plan, fcp::TB_BTILES);
  if (shard < 0) {
    bp.order = table(plan, fcp::TB_BORDER);
    bp.n_items = plan->counts[fcp::TB_BTILES];
    bp.kbuf_shift = 0;
  } else {
    const int32_t t0 = host_at(p, fcp::TB_BSHARD, shard), t1 = host_at(p, fcp::TB_BSHARD, shard + 1);
    bp.order = table(plan, fcp::TB_IDENT) + t0;
    bp.n_items = t1 - t0;
    bp.kbuf_shift = (int32_t)p->shards[shard].kbuf_base;
  }
  bp.T = dims.T;
  bp.hq = dims.hq;
  bp.hkv = dims.hkv;
  bp.scale = softmax_scale(dims);
  bp.scale_log2 = bp.scale * 1.4426950408889634f;
  bp.lse2 = lse2;
  bp.delta = delta;
  bp.dq = dq;
  bp.dk = dk;
  bp.dv = dv;
  bp.range = range;
  bp.err = static_cast<int*>(ws);
  bp.work_counter = reinterpret_cast<int*>(wsb + kWorkCounterOff);
  bp.n_tiles = plan->counts[fcp::TB_BTILES];
  bp.kb_rows = rrows > 0 ? (int32_t)rrows : dims.T;
  bp.wait_ns = g_wait_ns;
  a.d = dims.d;
  a.num_sms = num_sms();
  if ((a.has_bias = bias != nullptr)) {
    set_bias(&a.bias, bias, dbias, reinterpret_cast<float*>(wsb + wl.by_distance));
    cut_groups(&a.bias, p, shard, bp.n_items, dims, a.num_sms);
  }
  if ((a.has_window = p->window > 0) &&
      !set_window(&a.window, p, dims, k, v, rrows > 0 ? kbuf : k, rrows > 0 ? vbuf : v, rrows > 0 ? rrows : dims.T, false, dk,
                  dv))
    return FCP_ERR_CUDA;
  return fcp::launch_attn_bwd(a, s);
}

int fcp_attn_bwd(const void* q, const void* k, const void* v, const void* kbuf, const void* vbuf,
                 const void* out, int32_t out_dtype, const float* lse, const void* dout,
                 const fcp_dev_plan* plan, int32_t shard, fcp_dims dims, float* dq, float* dk,
                 float* dv, void* ws, int64_t ws_bytes, void* stream) {
  return attn_bwd_impl(q, k, v, kbuf, vbuf, out, out_dtype, lse, dout, plan, shard, dims, dq, dk, dv, ws, ws_bytes, stream,
                       nullptr, nullptr);
}

int fcp_attn_bwd_bias(const void* q, const void* k, const void* v, const void* kbuf, const void* vbuf,
                      const fcp_rel_bias* bias, const void* out, int32_t out_dtype, const float* lse, const void* dout,
                      const fcp_dev_plan* plan, int32_t shard, fcp_dims dims, float* dq, float* dk, float* dv,
                      float* dbias, void* ws, int64_t ws_bytes, void* stream) {
  const int st = check_bias(bias, dims);
  if (st) return st;
  if (!dbias || (reinterpret_cast<uintptr_t>(dbias) & 3)) return FCP_ERR_INVALID_ARG;
  // Added to while the biases are read.
  if (dims.hq > 0 && ranges_meet(bias->bias, dbias, (int64_t)dims.hq * bias->n_buckets)) return FCP_ERR_INVALID_ARG;
  return attn_bwd_impl(q, k, v, kbuf, vbuf, out, out_dtype, lse, dout, plan, shard, dims, dq, dk, dv, ws, ws_bytes, stream,
                       bias, dbias);
}

// Rows of a strided operand: T rows of `len` bytes, `stride` bytes apart.
struct RowSpan {
  uintptr_t at;
  int64_t stride, len;
};

// Whether a byte lies in a row of both. Spans with one stride are compared
// row by row (slices of one fused tensor interleave without sharing a byte);
// others by their whole extent.
static bool spans_meet(const RowSpan& a, const RowSpan& b, int64_t rows) {
  const int64_t ext_a = (rows - 1) * a.stride + a.len, ext_b = (rows - 1) * b.stride + b.len;
  if (a.at + (uintptr_t)ext_a <= b.at || b.at + (uintptr_t)ext_b <= a.at) return false;
  if (a.stride != b.stride) return true;
  const int64_t off = ((int64_t)(b.at - a.at) % a.stride + a.stride) % a.stride;  // b's start inside a row of a
  return off < a.len || off + b.len > a.stride;
}

static int check_norm_rope(const fcp_norm_rope* nr, const void* wq, const void* wk, const float* inv_freq,
                           const fcp_dims& dims) {
  if (!nr || (nr->norm != 0 && nr->norm != 1) || (nr->interleaved != 0 && nr->interleaved != 1) ||
      (nr->w_dtype != FCP_OUT_BF16 && nr->w_dtype != FCP_OUT_F32) || (nr->add_dw != 0 && nr->add_dw != 1))
    return FCP_ERR_INVALID_ARG;
  if (nr->norm && !(nr->eps >= 0.f && nr->eps <= 3.4e38f)) return FCP_ERR_INVALID_ARG;
  if (!nr->norm && (wq || wk)) return FCP_ERR_INVALID_ARG;
  if (nr->rot_dim < 0 || nr->rot_dim > dims.d) return FCP_ERR_INVALID_ARG;
  if (nr->rot_dim % 16) return FCP_ERR_UNSUPPORTED;
  if (nr->rot_dim > 0 && (!inv_freq || (reinterpret_cast<uintptr_t>(inv_freq) & 3))) return FCP_ERR_INVALID_ARG;
  const uintptr_t wmask = nr->w_dtype == FCP_OUT_F32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(wq) & wmask) || (reinterpret_cast<uintptr_t>(wk) & wmask))
    return FCP_ERR_INVALID_ARG;
  return FCP_OK;
}

// The launch's tiles, weights and options; the operands are set by the callers.
static fcp::NormRopeLaunch norm_rope_launch(const fcp_norm_rope* nr, const void* wq, const void* wk,
                                            const float* inv_freq, const fcp_dev_plan* plan, int32_t shard,
                                            const fcp_dims& dims) {
  const Plan* p = plan->host;
  fcp::NormRopeLaunch a;
  std::memset(&a, 0, sizeof(a));
  int32_t t0 = 0, t1 = plan->counts[fcp::TB_FTILES];
  a.rows = p->T;
  if (shard >= 0) {
    t0 = host_at(p, fcp::TB_FSHARD, shard);
    t1 = host_at(p, fcp::TB_FSHARD, shard + 1);
    a.rows = p->shards[shard].tokens;
  }
  a.n_tiles = t1 - t0;
  a.d = dims.d;
  a.interleaved = nr->interleaved != 0;
  a.num_sms = num_sms();
  a.p.pieces = table(plan, fcp::TB_PIECES);
  a.p.tiles = table(plan, fcp::TB_FTILES) + 4 * (int64_t)t0;
  a.p.n_pieces = plan->counts[fcp::TB_PIECES];
  a.p.T = dims.T;
  a.p.hq = dims.hq;
  a.p.hkv = dims.hkv;
  a.p.norm = nr->norm;
  a.p.eps = nr->eps;
  a.p.rot_dim = nr->rot_dim;
  a.p.w_f32 = nr->w_dtype == FCP_OUT_F32;
  a.p.add_dw = nr->add_dw;
  a.p.inv_freq = inv_freq;
  a.p.wq = wq;
  a.p.wk = wk;
  return a;
}

// A strided operand of `heads` heads: 16-byte aligned rows that hold them.
static bool strided_ok(const void* ptr, int64_t stride, int64_t heads, const fcp_dims& dims) {
  return ptr && aligned16(ptr) && stride % 8 == 0 && stride >= heads * dims.d &&
         stride <= INT64_MAX / 4 / std::max(dims.T, 1);
}

int fcp_qk_norm_rope(const void* q_in, int64_t q_stride, const void* k_in, int64_t k_stride, const void* v_in,
                     int64_t v_stride, const void* wq, const void* wk, const float* inv_freq,
                     const fcp_norm_rope* nr, const fcp_dev_plan* plan, int32_t shard, fcp_dims dims, void* q, void* k,
                     void* v, void* stream) {
  int st = check_dev_plan(plan, shard);
  if (st) return st;
  if ((st = check_dims(dims, plan->host))) return st;
  if ((st = check_norm_rope(nr, wq, wk, inv_freq, dims))) return st;
  if (!strided_ok(q_in, q_stride, dims.hq, dims) || !strided_ok(k_in, k_stride, dims.hkv, dims)) return FCP_ERR_INVALID_ARG;
  if (!v != !v_in || (v && !strided_ok(v_in, v_stride, dims.hkv, dims))) return FCP_ERR_INVALID_ARG;
  if (!q || !k || !aligned16(q) || !aligned16(k) || !aligned16(v)) return FCP_ERR_INVALID_ARG;
  const int64_t lq = (int64_t)dims.hq * dims.d * 2, lk = (int64_t)dims.hkv * dims.d * 2;
  const RowSpan in[3] = {{(uintptr_t)q_in, q_stride * 2, lq}, {(uintptr_t)k_in, k_stride * 2, lk}, {(uintptr_t)v_in, v_stride * 2, lk}};
  const RowSpan out[3] = {{(uintptr_t)q, lq, lq}, {(uintptr_t)k, lk, lk}, {(uintptr_t)v, lk, lk}};
  const int n = v ? 3 : 2;
  for (int o = 0; o < n; ++o) {
    for (int i = 0; i < n; ++i) {
      const bool in_place = i == o && in[i].at == out[o].at && in[i].stride == out[o].stride;
      if (!in_place && spans_meet(out[o], in[i], dims.T)) return FCP_ERR_INVALID_ARG;
      if (i < o && spans_meet(out[o], out[i], dims.T)) return FCP_ERR_INVALID_ARG;
    }
  }
  fcp::NormRopeLaunch a = norm_rope_launch(nr, wq, wk, inv_freq, plan, shard, dims);
  a.p.q_in = static_cast<const __nv_bfloat16*>(q_in);
  a.p.k_in = static_cast<const __nv_bfloat16*>(k_in);
  a.p.v_in = static_cast<const __nv_bfloat16*>(v_in);
  a.p.q_in_stride = q_stride;
  a.p.k_in_stride = k_stride;
  a.p.v_in_stride = v_stride;
  a.p.q = static_cast<__nv_bfloat16*>(q);
  a.p.k = static_cast<__nv_bfloat16*>(k);
  a.p.v = static_cast<__nv_bfloat16*>(v);
  return fcp::launch_norm_rope(a, static_cast<cudaStream_t>(stream));
}

int fcp_qk_norm_rope_bwd(const float* dq, const float* dk, const float* dv, const void* q_in, int64_t q_stride,
                         const void* k_in, int64_t k_stride, const void* wq, const void* wk, const float* inv_freq,
                         const fcp_norm_rope* nr, const fcp_dev_plan* plan, int32_t shard, fcp_dims dims, void* dq_in,
                         int64_t dq_stride, void* dk_in, int64_t dk_stride, void* dv_in, int64_t dv_stride, float* dwq,
                         float* dwk, void* ws, int64_t ws_bytes, void* stream) {
  int st = check_dev_plan(plan, shard);
  if (st) return st;
  if ((st = check_dims(dims, plan->host))) return st;
  if ((st = check_norm_rope(nr, wq, wk, inv_freq, dims))) return st;
  if (!dq || !dk || !aligned16(dq) || !aligned16(dk) || !aligned16(dv)) return FCP_ERR_INVALID_ARG;
  if (nr->norm && (!strided_ok(q_in, q_stride, dims.hq, dims) || !strided_ok(k_in, k_stride, dims.hkv, dims)))
    return FCP_ERR_INVALID_ARG;
  if (!strided_ok(dq_in, dq_stride, dims.hq, dims) || !strided_ok(dk_in, dk_stride, dims.hkv, dims))
    return FCP_ERR_INVALID_ARG;
  if (!dv != !dv_in || (dv && !strided_ok(dv_in, dv_stride, dims.hkv, dims))) return FCP_ERR_INVALID_ARG;
  if (!nr->norm && (dwq || dwk)) return FCP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dwq) & 3) || (reinterpret_cast<uintptr_t>(dwk) & 3)) return FCP_ERR_INVALID_ARG;
  if (dwq && dwk && ranges_meet(dwq, dwk, dims.d)) return FCP_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws)) return FCP_ERR_INVALID_ARG;
  const WsLayout wl = ws_layout(dims, plan->host->total_remote);
  if (ws_bytes < wl.total) return FCP_ERR_CAPACITY;
  const int64_t lq = (int64_t)dims.hq * dims.d, lk = (int64_t)dims.hkv * dims.d;
  const RowSpan out[3] = {{(uintptr_t)dq_in, dq_stride * 2, lq * 2}, {(uintptr_t)dk_in, dk_stride * 2, lk * 2}, {(uintptr_t)dv_in, dv_stride * 2, lk * 2}};
  const RowSpan grad[3] = {{(uintptr_t)dq, lq * 4, lq * 4}, {(uintptr_t)dk, lk * 4, lk * 4}, {(uintptr_t)dv, lk * 4, lk * 4}};
  const RowSpan x[2] = {{(uintptr_t)q_in, q_stride * 2, lq * 2}, {(uintptr_t)k_in, k_stride * 2, lk * 2}};
  const int n = dv ? 3 : 2;
  for (int o = 0; o < n; ++o) {
    for (int i = 0; i < n; ++i) {
      if (spans_meet(out[o], grad[i], dims.T)) return FCP_ERR_INVALID_ARG;
      if (i < o && spans_meet(out[o], out[i], dims.T)) return FCP_ERR_INVALID_ARG;
    }
    for (int i = 0; i < 2 && nr->norm; ++i) {
      const bool in_place = i == o && x[i].at == out[o].at && x[i].stride == out[o].stride;
      if (!in_place && spans_meet(out[o], x[i], dims.T)) return FCP_ERR_INVALID_ARG;
    }
  }
  fcp::NormRopeLaunch a = norm_rope_launch(nr, wq, wk, inv_freq, plan, shard, dims);
  a.backward = true;
  a.p.q_in = static_cast<const __nv_bfloat16*>(q_in);
  a.p.k_in = static_cast<const __nv_bfloat16*>(k_in);
  a.p.q_in_stride = q_stride;
  a.p.k_in_stride = k_stride;
  a.p.dq = dq;
  a.p.dk = dk;
  a.p.dv = dv;
  a.p.dq_in = static_cast<__nv_bfloat16*>(dq_in);
  a.p.dk_in = static_cast<__nv_bfloat16*>(dk_in);
  a.p.dv_in = static_cast<__nv_bfloat16*>(dv_in);
  a.p.dq_in_stride = dq_stride;
  a.p.dk_in_stride = dk_stride;
  a.p.dv_in_stride = dv_stride;
  a.p.dwq = dwq;
  a.p.dwk = dwk;
  char* wsb = static_cast<char*>(ws);
  a.p.partial = reinterpret_cast<float*>(wsb + wl.partial);
  a.p.tickets = reinterpret_cast<int*>(wsb + kTicketsOff);
  a.p.err = static_cast<int*>(ws);
  return fcp::launch_norm_rope(a, static_cast<cudaStream_t>(stream));
}

// The options and weights of a residual norm, and the launch's rows.
static int res_norm_params(fcp::ResNormParams* p, const fcp_res_norm* rn, const void* y, const void* gate, const void* w_post,
                           const void* w_pre, const fcp_dev_plan* plan, int32_t shard, int32_t n) {
  if (int st = check_dev_plan(plan, shard)) return st;
  if (n < 8 || n > 16384 || n % 8) return FCP_ERR_UNSUPPORTED;
  if (!rn) return FCP_ERR_INVALID_ARG;
  auto flag = [](int32_t v) { return v == 0 || v == 1; };
  auto finite = [](float v) { return std::fabs(v) <= 3.4e38f; };
  if (!flag(rn->post_norm) || !flag(rn->pre_norm) || !flag(rn->add_dw) || !flag(rn->gate_fn) || !flag(rn->res_dtype) ||
      !flag(rn->w_dtype))
    return FCP_ERR_INVALID_ARG;
  if (!(rn->eps >= 0.f) || !finite(rn->eps) || !finite(rn->res_scale) || !finite(rn->branch_scale)) return FCP_ERR_INVALID_ARG;
  if (!y && (gate || w_post)) return FCP_ERR_INVALID_ARG;
  if (!rn->pre_norm && w_pre) return FCP_ERR_INVALID_ARG;
  if (!aligned16(w_post) || !aligned16(w_pre)) return FCP_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  const Plan* host = plan->host;
  p->T = plan->T;
  p->n = n;
  p->num_sms = num_sms();
  p->units = plan->T;
  p->unit_rows = 1;
  if (shard >= 0) {
    const int32_t r0 = host_at(host, fcp::TB_RSHARD, shard), r1 = host_at(host, fcp::TB_RSHARD, shard + 1);
    static_assert(fcp::kResNormChunk >= fcp::kRowChunk, "a chunk's rows");
    p->chunks = table(plan, fcp::TB_ROWS) + 2 * (int64_t)r0;
    // By chunks where they are short and many. 32768 tokens of 2048 values, forward and gradient, by chunks and by
    // rows: documents of one token 120 and 204 us, 4277 and 5705; of 20 tokens 132 and 208, 249 and 331; of 63 159 and
    // 216, 128 and 215; one document (chunks of 128) 263 and 302, 120 and 203.
    if (host->shards[shard].tokens < 48 * (int64_t)(r1 - r0) && r1 - r0 >= 4 * p->num_sms) p->unit_rows = fcp::kResNormChunk;
    p->units = (int64_t)(r1 - r0) * (fcp::kResNormChunk / p->unit_rows);
  }
  p->post_norm = rn->post_norm;
  p->gate_fn = rn->gate_fn;
  p->res_f32 = rn->res_dtype == FCP_OUT_F32;
  p->w_f32 = rn->w_dtype == FCP_OUT_F32;
  p->add_dw = rn->add_dw;
  p->eps = rn->eps;
  p->res_scale = rn->res_scale;
  p->branch_scale = rn->branch_scale;
  p->y = y;
  p->gate = gate;
  p->w_post = w_post;
  p->w_pre = w_pre;
  return FCP_OK;
}

// One operand's rows of n values of `size` bytes.
struct Rows {
  const void* at;
  int64_t stride, size;
  bool ok(const fcp::ResNormParams& p) const {
    return at && aligned16(at) && stride % 8 == 0 && stride >= p.n && stride <= INT64_MAX / 16 / p.T;
  }
  RowSpan span(const fcp::ResNormParams& p) const { return {(uintptr_t)at, stride * size, p.n * size}; }
  bool same(const Rows& o) const { return at == o.at && stride * size == o.stride * o.size; }
};

// An operand that is one run of bytes: a weight, its gradient, the workspace.
struct Flat {
  const void* at;
  int64_t bytes;
  bool meets(const Flat& o) const {
    const uintptr_t a = (uintptr_t)at, b = (uintptr_t)o.at;
    return at && o.at && a < b + (uintptr_t)o.bytes && b < a + (uintptr_t)bytes;
  }
  // Of the rows that end behind its start, whether the first begins before its end.
  bool meets(const Rows& o, const fcp::ResNormParams& p) const {
    if (!at || !o.at) return false;
    const RowSpan r = o.span(p);
    const int64_t before = (int64_t)((uintptr_t)at - r.at) - r.len;  // rows that begin here or earlier end too soon
    const int64_t t = before < 0 ? 0 : before / r.stride + 1;
    return t < p.T && r.at + (uintptr_t)(t * r.stride) < (uintptr_t)at + (uintptr_t)bytes;
  }
};

// No output's rows meet a flat operand, and no flat output (the first n_out of
// them) an input's rows or another flat operand.
static bool flats_apart(const fcp::ResNormParams& p, const Flat* f, int n_f, int n_flat_out, const Rows* out, int n_out,
                        const Rows* in, int n_in) {
  for (int a = 0; a < n_f; ++a) {
    for (int o = 0; o < n_out; ++o)
      if (f[a].meets(out[o], p)) return false;
    for (int i = 0; a < n_flat_out && i < n_in; ++i)
      if (f[a].meets(in[i], p)) return false;
    for (int b = 0; a < n_flat_out && b < n_f; ++b)
      if (b != a && f[a].meets(f[b])) return false;
  }
  return true;
}

// No output meets another operand, but for out[i] on in[i] itself.
static bool rows_apart(const fcp::ResNormParams& p, const Rows* out, int n_out, const Rows* in, int n_in) {
  for (int o = 0; o < n_out; ++o) {
    if (!out[o].at) continue;
    for (int i = 0; i < n_in; ++i)
      if (in[i].at && !(i == o && out[o].same(in[i])) && spans_meet(out[o].span(p), in[i].span(p), p.T)) return false;
    for (int i = 0; i < o; ++i)
      if (out[i].at && spans_meet(out[o].span(p), out[i].span(p), p.T)) return false;
  }
  return true;
}

int fcp_residual_norm(const void* x, int64_t x_stride, const void* y, int64_t y_stride, const void* gate,
                      int64_t gate_stride, const void* w_post, const void* w_pre, const fcp_res_norm* rn,
                      const fcp_dev_plan* plan, int32_t shard, int32_t n, void* x_out, int64_t x_out_stride, void* h,
                      int64_t h_stride, void* stream) {
  fcp::ResNormParams p;
  if (int st = res_norm_params(&p, rn, y, gate, w_post, w_pre, plan, shard, n)) return st;
  const int64_t res = p.res_f32 ? 4 : 2;
  const Rows in[4] = {{x, x_stride, res}, {nullptr, 0, 0}, {y, y_stride, 2}, {gate, gate_stride, 2}};  // h is in no one's place
  const Rows out[2] = {{x_out, x_out_stride, res}, {h, h_stride, 2}};
  if (!in[0].ok(p) || (y && !in[2].ok(p)) || (gate && !in[3].ok(p))) return FCP_ERR_INVALID_ARG;
  if (!x_out && (y || rn->res_scale != 1.f || !h)) return FCP_ERR_INVALID_ARG;
  if ((x_out && !out[0].ok(p)) || !h != !rn->pre_norm || (h && !out[1].ok(p))) return FCP_ERR_INVALID_ARG;
  if (!rows_apart(p, out, 2, in, 4)) return FCP_ERR_INVALID_ARG;
  const int64_t w_bytes = (int64_t)n * (p.w_f32 ? 4 : 2);
  const Flat flat[2] = {{w_post, w_bytes}, {w_pre, w_bytes}};
  if (!flats_apart(p, flat, 2, 0, out, 2, in, 4)) return FCP_ERR_INVALID_ARG;
  p.x = x;
  p.x_row = x_stride * res;
  p.y_row = y_stride * 2;
  p.gate_row = gate_stride * 2;
  p.x_out = x_out;
  p.x_out_row = x_out_stride * res;
  p.h = h;
  p.h_row = h_stride * 2;
  return fcp::launch_res_norm(p, static_cast<cudaStream_t>(stream));
}

int64_t fcp_residual_norm_ws_bytes(int32_t n) { return n < 8 || n > 16384 || n % 8 ? 0 : fcp::res_norm_ws_bytes(n); }

int fcp_residual_norm_bwd(const void* dh, int64_t dh_stride, const void* dx_out, int64_t dx_out_stride, const void* x_out,
                          int64_t x_out_stride, const void* y, int64_t y_stride, const void* gate, int64_t gate_stride,
                          const void* w_post, const void* w_pre, const fcp_res_norm* rn, const fcp_dev_plan* plan,
                          int32_t shard, int32_t n, void* dx, int64_t dx_stride, void* dy, int64_t dy_stride, void* dgate,
                          int64_t dgate_stride, float* dw_post, float* dw_pre, void* ws, int64_t ws_bytes, void* stream) {
  fcp::ResNormParams p;
  if (int st = res_norm_params(&p, rn, y, gate, w_post, w_pre, plan, shard, n)) return st;
  const int64_t res = p.res_f32 ? 4 : 2;
  const Rows in[5] = {{dx_out, dx_out_stride, res}, {y, y_stride, 2}, {gate, gate_stride, 2}, {dh, dh_stride, 2}, {x_out, x_out_stride, res}};
  const Rows out[3] = {{dx, dx_stride, res}, {dy, dy_stride, 2}, {dgate, dgate_stride, 2}};
  if (!dh != !rn->pre_norm || (dh && (!in[3].ok(p) || !in[4].ok(p)))) return FCP_ERR_INVALID_ARG;
  if ((!dh && !dx_out) || (dx_out && !in[0].ok(p))) return FCP_ERR_INVALID_ARG;
  if ((y && !in[1].ok(p)) || (gate && !in[2].ok(p))) return FCP_ERR_INVALID_ARG;
  if (!out[0].ok(p) || !dy != !y || (dy && !out[1].ok(p)) || !dgate != !gate || (dgate && !out[2].ok(p)))
    return FCP_ERR_INVALID_ARG;
  if ((dw_post && !y) || (dw_pre && !dh)) return FCP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dw_post) & 3) || (reinterpret_cast<uintptr_t>(dw_pre) & 3)) return FCP_ERR_INVALID_ARG;
  if (!rows_apart(p, out, 3, in, dh ? 5 : 3)) return FCP_ERR_INVALID_ARG;
  const int64_t w_bytes = (int64_t)n * (p.w_f32 ? 4 : 2);
  const Flat flat[5] = {{dw_post, (int64_t)n * 4}, {dw_pre, (int64_t)n * 4},
                        {dw_post || dw_pre ? ws : nullptr, fcp::res_norm_ws_bytes(n)}, {w_post, w_bytes}, {w_pre, w_bytes}};
  if (!flats_apart(p, flat, 5, 3, out, 3, in, dh ? 5 : 3)) return FCP_ERR_INVALID_ARG;
  if (dw_post || dw_pre) {
    if (!ws || !aligned16(ws)) return FCP_ERR_INVALID_ARG;
    if (ws_bytes < fcp::res_norm_ws_bytes(n)) return FCP_ERR_CAPACITY;
  }
  p.x = x_out;
  p.x_row = x_out_stride * res;
  p.y_row = y_stride * 2;
  p.gate_row = gate_stride * 2;
  p.dh = dh;
  p.dh_row = dh_stride * 2;
  p.dx_out = dx_out;
  p.dx_out_row = dx_out_stride * res;
  p.dx = dx;
  p.dx_row = dx_stride * res;
  p.dy = dy;
  p.dy_row = dy_stride * 2;
  p.dgate = dgate;
  p.dgate_row = dgate_stride * 2;
  p.dw_post = dw_post;
  p.dw_pre = dw_pre;
  p.partial = static_cast<float*>(ws);
  return fcp::launch_res_norm(p, static_cast<cudaStream_t>(stream));
}

int fcp_get_device_status(void* ws, void* stream) {
  if (!ws) return FCP_ERR_INVALID_ARG;
  int word = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(&word, ws, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return FCP_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return FCP_ERR_CUDA;
  if (word == 0) return FCP_OK;
  if (cudaMemsetAsync(ws, 0, sizeof(int), s) != cudaSuccess) return FCP_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return FCP_ERR_CUDA;
  if (word & 1) return FCP_ERR_TIMEOUT;
  if (word & 4) return FCP_ERR_UNSUPPORTED;  // an input exceeds the fp16 operand range
  if (word & fcp::kErrBadTable) return FCP_ERR_INVALID_ARG;  // checked build: a table index out of range
  return FCP_ERR_CUDA;
}

void fcp_debug_set_wait_limit(int64_t ns) { g_wait_ns = ns == 0 ? 2000000000LL : ns; }

int fcp_debug_rescale_events(void* ws, void* stream, int64_t* count) {
  if (!ws || !count) return FCP_ERR_INVALID_ARG;
  int word = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* counter = static_cast<char*>(ws) + kRescaleCountOff;
  if (cudaMemcpyAsync(&word, counter, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return FCP_ERR_CUDA;
  if (cudaMemsetAsync(counter, 0, sizeof(int), s) != cudaSuccess) return FCP_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return FCP_ERR_CUDA;
  *count = word;
  return FCP_OK;
}

}  // extern "C"
