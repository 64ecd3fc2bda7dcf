// Document-masked attention backward on sm_103a (tcgen05 + TMA + TMEM).
//
// The exact gradient of the forward in attn_fwd.cu, for an upstream dO:
//   P = exp(S - LSE), dV = P^T dO, dP = dO V^T, D_i = <dO_i, O_i>,
//   dS = P (dP - D), dQ = scale dS K, dK = scale dS^T Q.
// "FlashCP" Fig. 6 names this "Attention BWD" and pairs it with a
// ReduceScatter of the KV gradients; on one GPU that reduction is the
// scatter-add of every key tile's dK/dV into the keys' global rows.
//
// Work unit: one key tile (<= 128 keys of one key segment) for one KV head.
// The CTA loops over the query heads of that GQA group and the query tiles
// that can see the keys -- those of the piece, and of the shard's earlier
// piece of the same document when the tile lies before that piece's end -- so
// dK and dV accumulate in TMEM over the whole group and reach global memory
// once per unit.
//
// Per step (one query head, one 128-row query tile), with keys as rows:
//   S^T = K Q^T, dP^T = V dO^T                (TMEM)
//   P^T = exp2(S^T scale log2e - LSE log2e)   (masked; fp16, back into TMEM)
//   dS^T = P^T (dP^T - D)                     (fp16, shared memory)
//   dV += P^T dO  (A operand from TMEM),  dK += dS^T Q,  dQ = dS K
// and dQ leaves TMEM through shared memory with TMA bulk reduce-adds
// (32-column chunks), one instruction per 16 KB.
//
// Tensor-core operands are fp16 (11 significant bits against bf16's 8): Q and
// dO arrive as fp16 copies made by the preprocess pass, K and V tiles are
// converted from bf16 in shared memory once per work unit, and P and dS are
// rounded to fp16. fp16 keeps its 11 bits from 2^-14 up and a call's gradients
// may be of any size, so dO, V, P and dS are scaled by powers of two. With e_i
// the exponent that the preprocess took out of row i of dO (its norm is then in
// [1, 2)), E the largest of them and 2^v above every |V_j| of the call,
//   P_ij 2^(10 + e_i - E) <= 2^10,  |dP_ij - D_i| 2^(-e_i - v) < 2^2,
// and their product, dS 2^(10 - E - v), is below 2^12: there is room for
// probabilities of up to 8 (an LSE of another precision's scores), and P keeps
// all its bits down to 2^-24. Results are scaled back where they leave the
// kernel. The factors ride on operations that were there: the exponent of P,
// V's conversion, the epilogues' products. Q and K are as they are: exact from
// 2^-17 up, below that off by 2^-25 at most.
//
// CTA roles (512 threads, persistent):
//   warp 0       loads (TMA for K, V, Q, dO; plain loads for LSE and D)
//   warp 1       issues MMAs and owns TMEM
//   warps 2-3    convert each unit's K/V tiles to fp16
//   warps 4-7    P and dS for query columns 0-63 (one key row per thread);
//                dV to global at the end of a unit
//   warps 8-11   P and dS for query columns 64-127; dK to global
//   warps 12-15  dQ: TMEM -> shared memory -> TMA reduce-add into global
// MMA order per step j, so that the exp work of step j+1 overlaps the dK/dQ
// products of step j:  dV_j, S_{j+1}, dQ_j, dK_j, dP_{j+1}. Q tiles are
// double-buffered; the dO tile is single-buffered (its last reader, dV_j,
// runs first in the step).
//
// With a bias (a separate instantiation), S gains b[h][bucket(i - j)] and
//   db[h][u] = sum of dS over the pairs with bucket u.
// Warps 2-3 are idle between conversions: they bring each step's LSE and D, the
// one bias of a tile of one bucket folded into LSE, and for a tile of several
// its 255 biases by distance (BiasSteps); and they sum the stored dS of tiles
// of one bucket (TileSums). The compute warps are the critical path, so they
// have only the window's adds and, in tiles of several buckets, the sums along
// the diagonals (add_block). One document of 16K (16 query and 2 KV heads of
// 128, 64 buckets): 2.90 ms against 2.57 without; the 32K workload 4.84
// against 4.62; 4096 tokens of 12 heads of 64, most of whose tiles hold several
// buckets: 94 us against 74. The steps' code of all roles together does not
// fit the instruction cache, so what a step executes counts by its length (on
// the 32K workload masks and MMAs written out took 0.2 ms more each, a loop or a call
// in BiasSteps::load another 0.4 to 0.8). Slower: the sums
// in the compute warps, by matrix instructions (no faster, for their set-up),
// in a table for each CTA.
#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "bias.cuh"
#include "kernels.h"
#include "sm103.cuh"

namespace fcp {

using namespace dev;

namespace {

constexpr int kThreads = 512;

// The call's scaling (see above), made by one thread of each CTA.
constexpr int kProbExp = 10;
struct Scaling {
  float lse_add;   // 10 - E
  float v;         // 2^-v
  float dv;        // 2^(E - 10)
  float ds;        // 2^(E - 10 + v)
  float dqk;       // that times the softmax scale
  __device__ __forceinline__ void init(const BwdRange* r, float scale) {
    const int e_max = (int)__ldcg(&r->e_max);
    const int field = (int)(__ldcg(&r->v2) >> 23);  // exponent of |V|^2
    const int E = e_max ? e_max - kRowExpBias : 0;
    const int ve = ((field - 127) >> 1) + 1;
    lse_add = (float)(kProbExp - E);
    v = scalbnf(1.f, -ve);
    dv = scalbnf(1.f, E - kProbExp);
    ds = scalbnf(1.f, E - kProbExp + ve);
    dqk = scale * ds;
  }
};

template <int D>
struct BwdCfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kK = 0;
  static constexpr int kV = kTile;
  static constexpr int kQ = 2 * kTile;           // 2 stages
  static constexpr int kDO = 4 * kTile;          // 1 stage
  static constexpr int kStage = 5 * kTile;       // 2 x [128 rows][32 fp32] dQ chunks
  static constexpr int kDS = kStage + 2 * 16384; // 128 x 128 fp16 (two 64-column panels)
  // [stage][lse2 | delta][128] fp32; with a bias one stage, and the 256 entries
  // of the step's bias window in the place of the other.
  static constexpr int kStat = kDS + 128 * 128 * 2;
  static constexpr int kSmem = kStat + 2 * 2 * 128 * 4;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0;           // S^T; P^T (fp16) in cols [0,32) and [64,96)
  static constexpr uint32_t kColDP = 128;        // dP^T, then dQ
  static constexpr uint32_t kColDV = 256;
  static constexpr uint32_t kColDK = 256 + D;
};

struct BwdItem {
  int key0, n, src, src_row, qa0, qa_end, na, qb0, qb_end, nb, nq, g;
  bool bad;  // checked build: the unit's table entries are out of range (skip it)
  int h0, heads;  // the unit's query heads
};

// Query tiles q0, q0 + 128, ... (n of them) lie inside [0, q_end] and q_end <= T.
__device__ __forceinline__ bool qrange_ok(int q0, int q_end, int n, int T) {
  return n == 0 || (n > 0 && q0 >= 0 && q_end <= T && (int64_t)q0 + (int64_t)(n - 1) * 128 < q_end);
}

// Parts that the query heads of a KV head are cut into, a unit each: with a bias
// as many as the launch says (the form without one adds up dK and dV over the
// heads of a group in TMEM, in one order).
__host__ __device__ __forceinline__ int group_parts(const NoBias&) { return 1; }
__host__ __device__ __forceinline__ int group_parts(const BiasParams& bp) { return bp.parts; }

template <class Bias>
__device__ __forceinline__ BwdItem decode(const BwdParams& p, const Bias& bias, int G, int w) {
  const WorkSlot ws = work_slot(w, p.n_items, p.hkv * group_parts(bias), p.order_block);
  const int item = __ldg(p.order + ws.pos);
  BwdItem it;
  it.bad = false;
  if constexpr (kDeviceChecks) {
    if (item < 0 || item >= p.n_tiles) {
      it = BwdItem{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, true};
      return it;
    }
  }
  const int* t = p.tiles + kBwdTileInts * item;
  it.key0 = __ldg(t + 0);
  it.n = __ldg(t + 1);
  it.src = __ldg(t + 2);
  it.src_row = __ldg(t + 3) - (it.src ? p.kbuf_shift : 0);
  it.qa0 = __ldg(t + 4);
  it.qa_end = __ldg(t + 5);
  it.na = __ldg(t + 6);
  it.qb0 = __ldg(t + 7);
  it.qb_end = __ldg(t + 8);
  it.nb = __ldg(t + 9);
  it.nq = it.na + it.nb;
  it.g = ws.head;
  it.h0 = ws.head * G;
  it.heads = G;
  if constexpr (std::is_same_v<Bias, BiasParams>) {
    it.g = ws.head / bias.parts;
    const int first = (ws.head - it.g * bias.parts) * bias.part_heads;
    it.h0 = it.g * G + first;
    it.heads = min(bias.part_heads, G - first);
  }
  if constexpr (kDeviceChecks) {
    const int rows = it.src ? p.kb_rows : p.T;
    it.bad = it.n < 1 || it.n > 128 || it.key0 < 0 || it.key0 > p.T - it.n || (it.src != 0 && it.src != 1) ||
             it.src_row < 0 || it.src_row > rows - it.n || !qrange_ok(it.qa0, it.qa_end, it.na, p.T) ||
             !qrange_ok(it.qb0, it.qb_end, it.nb, p.T);
  }
  return it;
}

// The query tiles of a unit's steps: for every head of the group the first
// range's tiles, then the second range's.
struct StepRows {
  int h, q0, q_end;
};
struct Steps {
  int h, idx;
  __device__ __forceinline__ explicit Steps(const BwdItem& it) : h(it.h0), idx(0) {}
  __device__ __forceinline__ StepRows rows(const BwdItem& it) const {
    return idx < it.na ? StepRows{h, it.qa0 + 128 * idx, it.qa_end} : StepRows{h, it.qb0 + 128 * (idx - it.na), it.qb_end};
  }
  __device__ __forceinline__ void next(const BwdItem& it) {
    if (++idx == it.nq) {
      idx = 0;
      ++h;
    }
  }
};

// With a bias: the statistics and the bias window of each step, which warps
// 2-3 (64 threads t) bring into shared memory.
struct BiasSteps {
  // The next step's, as they lie in memory: nothing waits for them until they
  // are stored.
  float lse[2], delta[2], one, win[4];
  bool windowed;                   // its tile holds several buckets
  float* one_bucket = nullptr;     // else its bucket's place in dbias
  BucketRun seen{0, 0, 0};

  __device__ __forceinline__ void load(const BwdParams& p, const BiasParams& bp, const Buckets& bk, const BwdItem& it,
                                       const Steps& steps, int t) {
    const StepRows sr = steps.rows(it);
    const float* bias_row = bp.bias + (size_t)sr.h * bp.n;
    const int first = sr.q0 - it.key0 - 127;  // distance of window entry 0
    const int near = max(first, 0);
    if (near < seen.lo || near >= seen.hi) bucket_run(seen, bk, bp.n, near);
    windowed = first + 254 >= seen.hi;
    one_bucket = windowed ? nullptr : bp.dbias + (size_t)sr.h * bp.n + seen.bucket;
    one = windowed ? 0.f : __ldg(bias_row + seen.bucket);
    const size_t row = (size_t)sr.h * p.T + sr.q0 + t;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool valid = t + 64 * u < sr.q_end - sr.q0;
      lse[u] = valid ? __ldg(p.lse2 + row + 64 * u) : -INFINITY;
      delta[u] = valid ? __ldg(p.delta + row + 64 * u) : 0.f;
    }
    if (windowed) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int dist = max(first + t + 64 * u, 0);
        win[u] = __ldg(bias_row + (dist < seen.hi && dist >= kNear ? seen.bucket : bk.of(bp.n, dist)));
      }
    }
  }
  __device__ __forceinline__ void store_lse(float* stat, int* windowed_sh, float inv_scale, float lse_add, int t) const {
    const float add = (one <= kMaskBelow ? -INFINITY : one * kLog2e) + lse_add;
    // Negated, as without a bias. A row whose buckets are all masked (-inf)
    // gets P = 0, as the rows past the piece do.
#pragma unroll
    for (int u = 0; u < 2; ++u) stat[t + 64 * u] = add + lse[u];
    if (windowed) {
#pragma unroll
      for (int u = 0; u < 4; ++u) stat[256 + t + 64 * u] = win[u] <= kMaskBelow ? -INFINITY : win[u] * inv_scale;
    }
    if (t == 0) *reinterpret_cast<volatile int*>(windowed_sh) = windowed;
  }
  __device__ __forceinline__ void store_delta(float* stat, float v_scale, int t) const {
#pragma unroll
    for (int u = 0; u < 2; ++u) stat[128 + t + 64 * u] = -delta[u] * v_scale;
  }
};

// With a bias: dS summed by buckets (fp32 sums of the stored fp16 values). A
// tile of one bucket, as most far from the diagonal are, is summed whole by
// warps 2-3, who keep the sum while the bucket and the head stay. In the others
// each compute warp takes its own block, 32 key rows x 64 query columns, and
// adds its diagonals to a table by distance (a lane's sums to neighbouring
// words), which a kernel after this one sums by buckets. Distances that the
// table does not hold are added by buckets at once. These atomics' order is not
// fixed, so neither are the last bits of db (nor are those of dQ, dK and dV).
struct TileSums {
  float sum = 0.f;
  float* at = nullptr;  // the bucket's place in dbias

  __device__ __forceinline__ void add(uint32_t panel, float* to, const Buckets& bk, int lane) {
    if (to != at) {
      flush(bk, lane);
      at = to;
    }
    sum += panel_sum(panel, lane);
  }
  __device__ __forceinline__ void flush(const Buckets& bk, int lane) {
    if (at) add_run(at, sum, bk.ds_scale, lane);
  }
};
// block: the stored dS; base: distance of its diagonal 0 (column 0, row 31).
// Out of line, for its registers are the ones that the P and dS loops lack.
static __device__ __noinline__ void add_block(uint32_t block, int h, const Buckets& bk, const BiasParams& bp, int base,
                                              int lane) {
  if (base + 94 < 0) return;
  __syncwarp();  // the warp's rows are stored
  float d[3];
  diagonal_sums(block, lane, d);
#pragma unroll
  for (int w = 0; w < 3; ++w) d[w] *= bk.ds_scale;
#pragma unroll 1
  for (int w = 0; w < 3; ++w, base += 32) {
    const int dist = base + lane;
    if (base + 31 < bp.n_distances) {
      if (dist >= 0) red_add(bp.by_distance + (size_t)h * bp.n_distances + dist, d[0]);
    } else {
      add_by_bucket(bp.dbias + (size_t)h * bp.n, bk.of(bp.n, dist), d[0], lane);
    }
    d[0] = d[1];
    d[1] = d[2];
  }
  __syncwarp();  // and read, before the next step's are
}

// TMA bulk reduce-add of a shared-memory tile into global memory.
__device__ __forceinline__ void tma_reduce_add_3d(const void* tmap, const void* src, int c0, int c1,
                                                  int c2) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
      " [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(tmap)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read_all() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void drain_group_sync() {  // the 128 threads of the dQ warpgroup
  asm volatile("bar.sync 1, 128;" ::: "memory");
}
// AND of `ok` over the 128 threads of the dQ warpgroup, so that its four warps
// leave (or stay in) the loop together and never strand one at bar.sync.
__device__ __forceinline__ bool drain_group_all(bool ok) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.and.pred po, 1, 128, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(out)
      : "r"((uint32_t)ok)
      : "memory");
  return out != 0;
}

template <int D, class Bias>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_kb, const __grid_constant__ CUtensorMap tm_vb,
                    const __grid_constant__ CUtensorMap tm_dq, const __grid_constant__ CUtensorMap tm_dk,
                    const __grid_constant__ CUtensorMap tm_dv, const BwdParams p,
                    const __grid_constant__ Bias bp) {
  using C = BwdCfg<D>;
  constexpr bool kBias = std::is_same_v<Bias, BiasParams>;
  // The bias's code does not leave the room in the instruction cache that all
  // MMAs of a step written out would take (0.19 ms more at d = 128 on the 32K
  // workload, two at a time 0.09; 4 us at d = 64 on 4096 tokens of 12 heads).
  // Without a bias they measured as fast or faster written out.
  constexpr int kMmaUnroll = kBias ? D / 32 : 8;
  // For the same reason masks have a place of their own there, off the way of
  // tiles that need none (one document of 16K 3.44 -> 3.13 ms), and for d = 64
  // (4096 tokens of 12 heads, without a bias 84 -> 77 us); at d = 128 without a
  // bias they are as well beside the values (512K workload 1.475 s, apart 1.485).
  constexpr bool kMaskApart = kBias || D == 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar_kv_full, bar_kv_conv, bar_kv_empty, bar_drain;
  __shared__ __align__(8) uint64_t bar_q_full[2], bar_q_empty[2], bar_do_full, bar_do_empty;
  __shared__ __align__(8) uint64_t bar_s_full, bar_dp_full, bar_p_ready, bar_ds_ready, bar_ds_free;
  __shared__ __align__(8) uint64_t bar_dq_full, bar_dq_free, bar_dkdv_full, bar_dkdv_free;
  __shared__ __align__(8) uint64_t bar_stg_full[2], bar_stg_free[2];  // dV / dK staging, per half
  __shared__ WorkRing<4> ring;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ Scaling scaling;
  __shared__ std::conditional_t<kBias, Buckets, NoBias> buckets;
  __shared__ int windowed_sh;  // bias: the step's tile spans several buckets

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if constexpr (kBias) buckets.init(bp, tid, kThreads);
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled layouts need 1024-byte alignment
    if (tid == 0) atomicOr(p.err, 2);
    return;
  }
  if (tid == 0) {
    mbar_init(&bar_kv_full, 1);
    mbar_init(&bar_kv_conv, 64);
    mbar_init(&bar_kv_empty, 1);
    mbar_init(&bar_drain, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar_q_full[s], kBias ? 1 : 2);
      mbar_init(&bar_q_empty[s], 1);
    }
    mbar_init(&bar_do_full, 1);
    mbar_init(&bar_do_empty, 1);
    mbar_init(&bar_s_full, kBias ? 3 : 1);   // with a bias LSE and the window, and D, by warps 2-3
    mbar_init(&bar_dp_full, kBias ? 3 : 1);
    mbar_init(&bar_p_ready, 256);
    mbar_init(&bar_ds_ready, 256);
    mbar_init(&bar_ds_free, kBias ? 3 : 1);
    mbar_init(&bar_dq_full, 1);
    mbar_init(&bar_dq_free, 128);
    mbar_init(&bar_dkdv_full, 1);
    mbar_init(&bar_dkdv_free, 256);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bar_stg_full[h], 128);
      mbar_init(&bar_stg_free[h], 1);
    }
    ring.init(1 + 2 + 8 + 4);  // MMA thread, conversion, compute and dQ warps
    abort_sh = 0;
    scaling.init(p.range, p.scale);
    if constexpr (kBias) buckets.ds_scale = scaling.ds;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_do);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_kb);
    prefetch_tmap(&tm_vb);
    prefetch_tmap(&tm_dq);
    prefetch_tmap(&tm_dk);
    prefetch_tmap(&tm_dv);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const WaitCtl wc{&abort_sh, p.err, p.wait_ns};
  const int n_work = p.n_items * p.hkv * group_parts(bp);
  const int G = p.hq / p.hkv;
  float* stat = reinterpret_cast<float*>(smem + C::kStat);

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    uint32_t kv_items = 0, qc = 0, dc = 0;
    uint32_t issued_q[2] = {0, 0};
    const float lse_add = scaling.lse_add, v_scale = scaling.v;
    bool ok = true;
    uint32_t k = 0;
    for (int w = blockIdx.x; ok;) {
      if (lane == 0) ok = ring.put(k, w, wc);
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      ++k;
      if (!ok || w >= n_work) break;
      // The next unit is claimed now (measured a little ahead of claiming it
      // after this unit's loads).
      int w_next = 0;
      if (lane == 0) w_next = next_work(p.work_counter);
      w_next = __shfl_sync(0xffffffffu, w_next, 0);
      const BwdItem it = decode(p, bp, G, w);
      if (it.bad) {  // checked build: skipped by every role
        if (lane == 0) atomicOr(p.err, kErrBadTable);
        w = w_next;
        continue;
      }
      if (kv_items > 0) {
        ok = mbar_wait(&bar_kv_empty, (kv_items - 1) & 1, wc);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar_kv_full, 2 * C::kTile);
        const CUtensorMap* tk = it.src ? &tm_kb : &tm_k;
        const CUtensorMap* tv = it.src ? &tm_vb : &tm_v;
        for (int pn = 0; pn < C::kPanels; ++pn) {
          tma_load_3d(smem + C::kK + pn * 16384, tk, &bar_kv_full, pn * 64, it.g, it.src_row);
          tma_load_3d(smem + C::kV + pn * 16384, tv, &bar_kv_full, pn * 64, it.g, it.src_row);
        }
      }
      ++kv_items;
      const int nsteps = it.heads * it.nq;
      // No L2 prefetches: issued through the tensor-memory accelerator, which
      // also carries this CTA's loads and dQ reduce-adds, they cost more in its
      // queue than they saved.
      Steps steps(it);
      for (int j = 0; j < nsteps; ++j, steps.next(it)) {
        const StepRows sr = steps.rows(it);
        const int h = sr.h, q0 = sr.q0;
        const int q_rows = min(128, sr.q_end - q0);
        // Q tile and the rows' LSE / D into Q stage s.
        const int s = qc & 1;
        if (qc >= 2) {
          ok = mbar_wait(&bar_q_empty[s], ((qc >> 1) - 1) & 1, wc);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_q_full[s], C::kTile);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_3d(smem + C::kQ + s * C::kTile + pn * 16384, &tm_q, &bar_q_full[s], pn * 64, h, q0);
          ++issued_q[s];
        }
        if constexpr (!kBias) {  // with a bias warps 2-3 write them
          float* st = stat + s * 256;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = lane + 32 * u;
            const bool valid = r < q_rows;
            // Stored negated (-LSE log2 e, -D): the compute warps add them with
            // packed f32x2 arithmetic. Rows past the piece get P = 0.
            st[r] = valid ? __ldg(p.lse2 + (size_t)h * p.T + q0 + r) + lse_add : -INFINITY;
            st[128 + r] = valid ? -__ldg(p.delta + (size_t)h * p.T + q0 + r) * v_scale : 0.f;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_q_full[s]);
        }
        ++qc;
        // dO tile into the single dO buffer once dV of the previous step is done.
        if (dc >= 1) {
          ok = mbar_wait(&bar_do_empty, (dc - 1) & 1, wc);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_do_full, C::kTile);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_3d(smem + C::kDO + pn * 16384, &tm_do, &bar_do_full, pn * 64, h, q0);
        }
        ++dc;
      }
      w = w_next;
    }
    if (lane == 0) {  // every copy this warp started has landed before the CTA exits
      if (kv_items) mbar_drain(&bar_kv_full, (kv_items - 1) & 1);
      for (int s = 0; s < 2; ++s)
        if (issued_q[s]) mbar_drain(&bar_q_full[s], (issued_q[s] - 1) & 1);
      if (dc) mbar_drain(&bar_do_full, (dc - 1) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_sq = idesc_f16kind(128, 128, false, false, false);  // S^T, dP^T
      constexpr uint32_t id_kd = idesc_f16kind(128, D, false, true, false);     // dV, dK
      constexpr uint32_t id_dq = idesc_f16kind(128, D, true, true, false);      // dQ = dS K
      const uint32_t sK = smem_u32(smem + C::kK), sV = smem_u32(smem + C::kV);
      const uint32_t sDO = smem_u32(smem + C::kDO), sDS = smem_u32(smem + C::kDS);
      uint32_t kv_items = 0, qc = 0, dc = 0, gstep = 0, items = 0;
      bool ok = true;
      auto qaddr = [&](uint32_t c) { return smem_u32(smem + C::kQ + (c & 1) * C::kTile); };
      auto issue_s = [&](uint32_t c) {
        const uint32_t sQ = qaddr(c);
#pragma unroll(kMmaUnroll)
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_bf16_ss(tmem + C::kColS, smem_desc_sw128(sK + off, 0, 1024),
                      smem_desc_sw128(sQ + off, 0, 1024), id_sq, kk > 0);
        }
        mma_commit(&bar_s_full);
      };
      auto issue_dp = [&]() {
#pragma unroll(kMmaUnroll)
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_bf16_ss(tmem + C::kColDP, smem_desc_sw128(sV + off, 0, 1024),
                      smem_desc_sw128(sDO + off, 0, 1024), id_sq, kk > 0);
        }
        mma_commit(&bar_dp_full);
      };
      for (uint32_t k = 0; ok; ++k) {
        int w;
        if (!(ok = ring.get(k, w, wc))) break;
        ring.release(k);
        if (w >= n_work) break;
        const BwdItem it = decode(p, bp, G, w);
        if (it.bad) continue;
        const int nsteps = it.heads * it.nq;
        if (!(ok = mbar_wait(&bar_kv_conv, kv_items & 1, wc))) break;
        tc_fence_after();
        // Prologue of the unit: S_0 and dP_0.
        if (!(ok = mbar_wait(&bar_q_full[qc & 1], (qc >> 1) & 1, wc))) break;
        tc_fence_after();
        issue_s(qc);
        if (gstep > 0 && !(ok = mbar_wait(&bar_dq_free, (gstep - 1) & 1, wc))) break;
        if (!(ok = mbar_wait(&bar_do_full, dc & 1, wc))) break;
        tc_fence_after();
        issue_dp();
        for (int j = 0; j < nsteps; ++j, ++gstep) {
          const uint32_t c = qc + j;
          const uint32_t sQ = qaddr(c);
          if (!(ok = mbar_wait(&bar_p_ready, gstep & 1, wc))) break;
          if (j == 0 && items > 0 && !(ok = mbar_wait(&bar_dkdv_free, (items - 1) & 1, wc))) break;
          tc_fence_after();
          // dV += P^T dO, P^T from TMEM: q columns 0-63 in cols [0,32), 64-127 in [64,96).
#pragma unroll(kMmaUnroll)
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ts(tmem + C::kColDV, tmem + C::kColS + (kk < 4 ? kk * 8 : 64 + (kk - 4) * 8),
                       smem_desc_sw128(sDO + kk * 2048, 16384, 1024), id_kd, (j > 0 || kk > 0));
          mma_commit(&bar_do_empty);
          if (j + 1 < nsteps) {  // S region is free once dV (issued above) has read P^T
            if (!(ok = mbar_wait(&bar_q_full[(c + 1) & 1], ((c + 1) >> 1) & 1, wc))) break;
            tc_fence_after();
            issue_s(c + 1);
          }
          if (!(ok = mbar_wait(&bar_ds_ready, gstep & 1, wc))) break;
          tc_fence_after();
#pragma unroll(kMmaUnroll)
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ss(tmem + C::kColDP, smem_desc_sw128(sDS + kk * 2048, 16384, 1024),
                        smem_desc_sw128(sK + kk * 2048, 16384, 1024), id_dq, kk > 0);
          mma_commit(&bar_dq_full);
#pragma unroll(kMmaUnroll)
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t aoff = (kk >> 2) * 16384 + (kk & 3) * 32;
            mma_bf16_ss(tmem + C::kColDK, smem_desc_sw128(sDS + aoff, 0, 1024),
                        smem_desc_sw128(sQ + kk * 2048, 16384, 1024), id_kd, (j > 0 || kk > 0));
          }
          mma_commit(&bar_ds_free);
          mma_commit(&bar_q_empty[c & 1]);
          if (j + 1 < nsteps) {  // DP region is free once dQ_j has been read out
            if (!(ok = mbar_wait(&bar_dq_free, gstep & 1, wc))) break;
            if (!(ok = mbar_wait(&bar_do_full, (dc + j + 1) & 1, wc))) break;
            tc_fence_after();
            issue_dp();
          }
        }
        if (!ok) break;
        mma_commit(&bar_dkdv_full);
        mma_commit(&bar_kv_empty);
        qc += nsteps;
        dc += nsteps;
        ++kv_items;
        ++items;
      }
      // Every MMA this thread issued has finished before TMEM is released.
      mma_commit(&bar_drain);
      mbar_drain(&bar_drain, 0);
    }
  } else if (warp == 2 || warp == 3) {
    // ------------------------------------------------------------ K/V to fp16
    const int t = tid - 64;
    uint32_t items = 0, gstep = 0;
    bool ok = true, ovf = false;
    uint4* kv = reinterpret_cast<uint4*>(smem + C::kK);  // K and V tiles are contiguous
    const float v_scale = scaling.v;
    BiasSteps bias;
    TileSums sums;
    const uint32_t ds_panel = smem_u32(smem + C::kDS) + (warp - 2) * 16384;
    for (uint32_t k = 0; ok; ++k) {
      int w = 0;
      ok = ring.get(k, w, wc);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      __syncwarp();
      if (lane == 0) ring.release(k);
      if (w >= n_work) break;
      BwdItem it;
      if constexpr (kDeviceChecks || kBias) {
        it = decode(p, bp, G, w);
        if (it.bad) continue;
      }
      auto convert = [&]() {
        ok = mbar_wait(&bar_kv_full, items & 1, wc);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; return; }
        constexpr int kVecs = C::kTile / 16;
        auto one = [&](int i, float mul) {
          uint4 x = kv[i];
          x.x = bf16x2_to_f16x2(x.x, mul, ovf);
          x.y = bf16x2_to_f16x2(x.y, mul, ovf);
          x.z = bf16x2_to_f16x2(x.z, mul, ovf);
          x.w = bf16x2_to_f16x2(x.w, mul, ovf);
          kv[i] = x;
        };
        // K as it is, V scaled. With a bias the shorter code wins (the 32K
        // workload: 4.84 ms for 4.95), without one the longer (4.62 for 4.64).
        if constexpr (kBias) {
          float mul = 1.f;
#pragma unroll 1
          for (int of_v = 0; of_v < 2; ++of_v, mul = v_scale)
#pragma unroll 2
            for (int i = t + of_v * kVecs; i < (of_v + 1) * kVecs; i += 64) one(i, mul);
        } else {
#pragma unroll 4
          for (int i = t; i < 2 * kVecs; i += 64) one(i, i < kVecs ? 1.f : v_scale);
        }
        fence_proxy_async_smem();
        mbar_arrive(&bar_kv_conv);
        ++items;
      };
      if constexpr (!kBias) {
        convert();
        if (!ok) break;
      } else {
        // With a bias these warps also follow the unit's steps: LSE, D and the
        // bias window of a step go into shared memory as soon as the compute
        // warps are done with those of the step before (they arrive at the
        // barriers of S and of dP, so the compute warps wait no more often),
        // and the dS tile of a step of one bucket is summed beside its dK and
        // dQ products, half of the columns by each warp.
        const int nsteps = it.heads * it.nq;
        Steps steps(it);
        for (int j = -1; j < nsteps; ++j) {
          const bool more = j + 1 < nsteps;
          float* one_bucket = bias.one_bucket;  // of step j
          if (more) {
            bias.load(p, bp, buckets, it, steps, t);
            steps.next(it);
          }
          if (j < 0) {
            convert();
          } else {
            ok = mbar_wait(&bar_p_ready, gstep & 1, wc);
            ok = __all_sync(0xffffffffu, ok);
          }
          if (!ok) break;
          if (more) {
            bias.store_lse(stat, &windowed_sh, 1.f / p.scale, scaling.lse_add, t);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_s_full);
          }
          if (j >= 0) {
            ok = mbar_wait(&bar_ds_ready, gstep & 1, wc);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            ++gstep;
          }
          if (more) {
            bias.store_delta(stat, scaling.v, t);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_dp_full);
          }
          if (j >= 0) {
            if (one_bucket) sums.add(ds_panel, one_bucket, buckets, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_ds_free);
          }
        }
      }
    }
    if constexpr (kBias) sums.flush(buckets, lane);
    if (ovf) atomicOr(p.err, 4);
  } else if (warp < 12) {
    // ------------------------------------------------------------ P and dS
    const int half = (warp - 4) >> 2;       // query columns [64*half, 64*half + 64)
    const int kr = (warp & 3) * 32 + lane;  // key row == TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_cols = lane_base + C::kColS + 64 * half;
    const uint32_t dp_cols = lane_base + C::kColDP + 64 * half;
    const uint32_t ds_panel = smem_u32(smem + C::kDS) + half * 16384;
    uint32_t qc = 0, gstep = 0, items = 0, stg = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      int w = 0;
      ok = ring.get(k, w, wc);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      __syncwarp();
      if (lane == 0) ring.release(k);
      if (w >= n_work) break;
      const BwdItem it = decode(p, bp, G, w);
      if (it.bad) continue;
      const int nsteps = it.heads * it.nq;
      const bool key_valid = kr < it.n;
      const int key = it.key0 + kr;
      Steps steps(it);
      for (int j = 0; j < nsteps; ++j, ++gstep, steps.next(it)) {
        const uint32_t c = qc + j, s = c & 1;
        const int q0 = steps.rows(it).q0;
        const int lim = key - q0 - 64 * half;  // local columns below lim cannot see this key
        // Whole tile below the diagonal with 128 keys: no element needs a mask
        // (query rows past the piece end have LSE = +inf, hence P = 0).
        const bool unmasked = it.n == 128 && it.key0 + 127 <= q0;
        ok = mbar_wait(&bar_s_full, gstep & 1, wc) &&
             (kBias || mbar_wait(&bar_q_full[s], (c >> 1) & 1, wc));
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        const float4* st4 = reinterpret_cast<const float4*>(stat + (kBias ? 0 : s * 256) + 64 * half);
        bool windowed = false;  // bias: the tile holds several buckets
        uint32_t pk[32];
        {
          // Both 32-column halves of this group's S^T in flight together.
          float va[32], vb[32];
          tmem_ld32(s_cols, va);
          tmem_ld32(s_cols + 32, vb);
          tmem_ld_wait();
          if constexpr (kBias) {
            // A tile of one bucket has its bias in the LSE; the others add the
            // window (entry column + 127 - row) to the raw scores.
            windowed = *reinterpret_cast<volatile int*>(&windowed_sh) != 0;
            if (windowed) {
              const float* w = stat + 256 + 64 * half + 127 - kr;
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                f2_split(f2_add(f2(va[e], va[e + 1]), f2(w[e], w[e + 1])), va[e], va[e + 1]);
                f2_split(f2_add(f2(vb[e], vb[e + 1]), f2(w[32 + e], w[33 + e])), vb[e], vb[e + 1]);
              }
            }
          }
          const uint64_t c2 = f2(p.scale_log2, p.scale_log2);
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            const float* v = e < 32 ? va + e : vb + (e - 32);
            const float4 l4 = st4[e >> 2];  // -LSE log2 e of the four query columns
            float p0, p1, p2, p3;
            f2_split(f2_fma(f2(v[0], v[1]), c2, f2(l4.x, l4.y)), p0, p1);
            f2_split(f2_fma(f2(v[2], v[3]), c2, f2(l4.z, l4.w)), p2, p3);
            p0 = ex2(p0);
            p1 = ex2(p1);
            p2 = ex2(p2);
            p3 = ex2(p3);
            if (!kMaskApart && !unmasked) {
              if (!key_valid || e < lim) p0 = 0.f;
              if (!key_valid || e + 1 < lim) p1 = 0.f;
              if (!key_valid || e + 2 < lim) p2 = 0.f;
              if (!key_valid || e + 3 < lim) p3 = 0.f;
            }
            pk[e >> 1] = pack_f16(p0, p1);
            pk[(e >> 1) + 1] = pack_f16(p2, p3);
          }
          if (kMaskApart && !unmasked) {
            const int first = key_valid ? lim : 64;
#pragma unroll
            for (int e = 0; e < 64; e += 2)
              pk[e >> 1] &= (e >= first ? 0xFFFFu : 0u) | (e + 1 >= first ? 0xFFFF0000u : 0u);
          }
        }
        {
          float f[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(pk[e]);
          tmem_st32(s_cols, f);  // P^T over the S values just read (same rows, own columns)
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&bar_p_ready);
        ok = mbar_wait(&bar_dp_full, gstep & 1, wc);
        if (ok && gstep > 0) ok = mbar_wait(&bar_ds_free, (gstep - 1) & 1, wc);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        // dS = P (dP - D), scaled, in packed fp16: (dP - D) and the product are
        // each rounded to fp16, the operand type of the dK and dQ products.
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          float v[32];
          tmem_ld32(dp_cols + cc * 32, v);
          tmem_ld_wait();
          uint32_t o[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const int col = cc * 32 + e;
            const float4 d4 = st4[32 + (col >> 2)];  // -D of the four query columns
            float a0, a1, a2, a3;
            f2_split(f2_add(f2(v[e], v[e + 1]), f2(d4.x, d4.y)), a0, a1);
            f2_split(f2_add(f2(v[e + 2], v[e + 3]), f2(d4.z, d4.w)), a2, a3);
            // Saturated: rows of other keys in the tile may pass the range, and
            // their P = 0 is to give 0.
            const uint32_t x01 = pack_f16_sat(a0, a1), x23 = pack_f16_sat(a2, a3);
            const uint32_t p01 = pk[col >> 1], p23 = pk[(col >> 1) + 1];
            const __half2 r01 = __hmul2(*reinterpret_cast<const __half2*>(&p01), *reinterpret_cast<const __half2*>(&x01));
            const __half2 r23 = __hmul2(*reinterpret_cast<const __half2*>(&p23), *reinterpret_cast<const __half2*>(&x23));
            o[e >> 1] = *reinterpret_cast<const uint32_t*>(&r01);
            o[(e >> 1) + 1] = *reinterpret_cast<const uint32_t*>(&r23);
          }
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
            st_shared_v4(ds_panel + sw128_offset(kr, cc * 4 + q4), o[4 * q4], o[4 * q4 + 1],
                         o[4 * q4 + 2], o[4 * q4 + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bar_ds_ready);
        if constexpr (kBias) {
          if (windowed)
            add_block(ds_panel + 4096 * (warp & 3), steps.h, buckets, bp,
                      q0 + 64 * half - it.key0 - 32 * (warp & 3) - 31, lane);
        }
      }
      if (!ok) break;
      qc += nsteps;
      // dV (columns-0 group) or dK (columns-64 group) of this key tile ->
      // global rows: 32-column chunks staged in this group's half of the dS
      // buffer (free once the unit's MMAs are done; the 128-byte swizzled
      // layout of a [128 rows][32 fp32] TMA box) and reduce-added by one
      // thread with TMA. Rows of keys past the tile hold zeros.
      ok = mbar_wait(&bar_dkdv_full, items & 1, wc);
      if constexpr (kBias) ok = ok && mbar_wait(&bar_ds_free, (gstep - 1) & 1, wc);  // the last dS is summed too
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_after();
      const uint32_t src_col = lane_base + (half == 0 ? C::kColDV : C::kColDK);
      const float mul = half == 0 ? scaling.dv : scaling.dqk;
      const CUtensorMap* tm_out = half == 0 ? &tm_dv : &tm_dk;
      // Two chunks in registers: the TMEM read of chunk cc + 2 is issued once
      // chunk cc is staged and waited for two chunks later, so its latency
      // (a TMEM read waits behind the MMAs' own TMEM traffic) overlaps the
      // reduce-adds of the chunks between.
      constexpr int kChunks = D / 32;
      float vv[2][32];
      tmem_ld32(src_col, vv[0]);
      tmem_ld32(src_col + 32, vv[1]);
      tmem_ld_wait();
#pragma unroll
      for (int cc = 0; cc < kChunks; ++cc, ++stg) {
        if (!ok) break;
        float* v = vv[cc & 1];
        if (stg > 0) {  // the previous chunk's reduce has read the staging tile
          ok = mbar_wait(&bar_stg_free[half], (stg - 1) & 1, wc);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        }
        if (cc >= 2) tmem_ld_wait();  // this chunk was read after chunk cc - 2 was staged
#pragma unroll
        for (int q4 = 0; q4 < 8; ++q4) {
          const float a0 = key_valid ? v[4 * q4] * mul : 0.f, a1 = key_valid ? v[4 * q4 + 1] * mul : 0.f;
          const float a2 = key_valid ? v[4 * q4 + 2] * mul : 0.f, a3 = key_valid ? v[4 * q4 + 3] * mul : 0.f;
          st_shared_v4(ds_panel + sw128_offset(kr, q4), __float_as_uint(a0), __float_as_uint(a1),
                       __float_as_uint(a2), __float_as_uint(a3));
        }
        fence_proxy_async_smem();
        mbar_arrive(&bar_stg_full[half]);
        if (cc + 2 < kChunks) tmem_ld32(src_col + (cc + 2) * 32, vv[cc & 1]);
        if (kr == 0) {
          ok = mbar_wait(&bar_stg_full[half], stg & 1, wc);
          if (ok) {
            tma_reduce_add_3d(tm_out, smem + C::kDS + half * 16384, cc * 32, it.g, it.key0);
            bulk_commit();
            bulk_wait_read_all();
          }
          mbar_arrive(&bar_stg_free[half]);
        }
        ok = __all_sync(0xffffffffu, ok);  // the issuing lane's outcome, warp-wide
      }
      tmem_ld_wait();  // no TMEM read left in flight, also when the loop gave up early
      // The last chunk's tile is read before dS of the next unit lands there.
      if (ok) ok = mbar_wait(&bar_stg_free[half], (stg - 1) & 1, wc);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_before();
      mbar_arrive(&bar_dkdv_free);
      ++items;
    }
    if (kr == 0) bulk_wait_all();  // this thread's reduces are complete before the CTA exits
  } else {
    // ------------------------------------------------------------ dQ drain
    // Thread r holds query row q0 + r. Each 32-column chunk goes to one of two
    // shared-memory staging tiles (the 128-byte swizzled layout of a
    // [128 rows][32 fp32] TMA box) and one thread reduce-adds it into dQ.
    // Rows past the piece end hold exact zeros (their P and dS are zero).
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint8_t* stage = smem + C::kStage;
    const float mul = scaling.dqk;
    uint32_t gstep = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      int w = 0;
      ok = drain_group_all(ring.get(k, w, wc));
      if (!ok) break;
      __syncwarp();
      if (lane == 0) ring.release(k);
      if (w >= n_work) break;
      const BwdItem it = decode(p, bp, G, w);
      if (it.bad) continue;
      const int nsteps = it.heads * it.nq;
      Steps steps(it);
      for (int j = 0; j < nsteps; ++j, ++gstep, steps.next(it)) {
        const StepRows sr = steps.rows(it);
        const int h = sr.h, q0 = sr.q0;
        ok = drain_group_all(mbar_wait(&bar_dq_full, gstep & 1, wc));
        if (!ok) break;
        tc_fence_after();
        // Two 32-column chunks at a time: both loads in flight together, the
        // TMEM columns released as soon as every chunk has been read.
        constexpr int kPairs = D / 64;
        float a[32], b[32];
        tmem_ld32(lane_base + C::kColDP, a);
        tmem_ld32(lane_base + C::kColDP + 32, b);
        tmem_ld_wait();
        if (kPairs == 1) {
          tc_fence_before();
          mbar_arrive(&bar_dq_free);  // every dQ column of this step has been read
        }
#pragma unroll 1
        for (int pr = 0; pr < kPairs; ++pr) {
          if (r == 0) bulk_wait_read_all();  // earlier reduces are done reading the tiles
          drain_group_sync();
          const uint32_t b0 = smem_u32(stage), b1 = smem_u32(stage + 16384);
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4) {
            st_shared_v4(b0 + sw128_offset(r, q4), __float_as_uint(a[4 * q4] * mul),
                         __float_as_uint(a[4 * q4 + 1] * mul), __float_as_uint(a[4 * q4 + 2] * mul),
                         __float_as_uint(a[4 * q4 + 3] * mul));
            st_shared_v4(b1 + sw128_offset(r, q4), __float_as_uint(b[4 * q4] * mul),
                         __float_as_uint(b[4 * q4 + 1] * mul), __float_as_uint(b[4 * q4 + 2] * mul),
                         __float_as_uint(b[4 * q4 + 3] * mul));
          }
          if (pr + 1 < kPairs) {
            tmem_ld32(lane_base + C::kColDP + 64 * (pr + 1), a);
            tmem_ld32(lane_base + C::kColDP + 64 * (pr + 1) + 32, b);
            tmem_ld_wait();
            if (pr + 2 == kPairs) {
              tc_fence_before();
              mbar_arrive(&bar_dq_free);  // every dQ column of this step has been read
            }
          }
          fence_proxy_async_smem();
          drain_group_sync();
          if (r == 0) {
            tma_reduce_add_3d(&tm_dq, stage, 64 * pr, h, q0);
            tma_reduce_add_3d(&tm_dq, stage + 16384, 64 * pr + 32, h, q0);
            bulk_commit();
          }
        }
      }
    }
    if (r == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  // The last CTA leaves the range as the next call expects it (every CTA has
  // read it: its scaling is older than its share of `done`).
  if (tid == 0 && atomicAdd(&p.range->done, 1) == (int)gridDim.x - 1) *p.range = BwdRange{0, 0, 0};
}

}  // namespace

// dbias += the table's sums by distance: one block a head, a warp a bucket. By
// atomics, as the kernel before adds to it: another call (with a workspace of
// its own, on another stream) may add to the same gradients.
constexpr int kTableThreads = 512;
static __global__ void __launch_bounds__(kTableThreads) table_sums_kernel(const __grid_constant__ BiasParams bp) {
  const float* table = bp.by_distance + (size_t)blockIdx.x * bp.n_distances;
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x >> 5; b < bp.n; b += kTableThreads / 32) {
    // (Starts reach 2^31 - 1: cut to the table before anything is added to them.)
    const int begin = min(bp.starts[b], bp.n_distances);
    const int end = b + 1 < bp.n ? min(bp.starts[b + 1], bp.n_distances) : bp.n_distances;
    float v = 0.f;
#pragma unroll 4
    for (int x = begin + lane; x < end; x += 32) v += __ldcg(table + x);
    v = warp_sum(v);
    if (lane == 0 && v != 0.f) red_add(bp.dbias + (size_t)blockIdx.x * bp.n + b, v);
  }
}

template <int D, class Bias>
static int launch_bwd_impl(const BwdLaunch& a, const Bias& bias, cudaStream_t st) {
  using C = BwdCfg<D>;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    if (cudaFuncSetAttribute(attn_bwd_kernel<D, Bias>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem) != cudaSuccess)
      return FCP_ERR_CUDA;
    attr_set[dev] = true;
  }
  const int parts = group_parts(bias);
  const int n_work = a.p.n_items * a.p.hkv * parts;
  if (n_work == 0) return FCP_OK;
  const int grid = n_work < a.num_sms ? n_work : a.num_sms;
  // Blocks of key tiles that fill the grid with one KV head: the CTAs running
  // together stream the same query rows (Q, dO, dQ) of that head group.
  BwdParams p = a.p;
  // Few units go item by item instead, so that the longest come first (4096
  // tokens of 12 heads of 64, with a bias, 7.7 units a CTA: 93 us for 105; one
  // document of 16K, 16 heads, 10.5: 2.91 ms for 2.97). With many the rows that
  // are shared count for more (one of 16K, 32 heads, 42 units: 5.13 ms in blocks,
  // 5.15 item by item; of 64K 75.6 and 78.8).
  p.order_block = n_work < 16 * grid ? 1 : grid;
  if constexpr (std::is_same_v<Bias, BiasParams>) {
    if (cudaMemsetAsync(bias.by_distance, 0, sizeof(float) * p.hq * bias.n_distances, st) != cudaSuccess)
      return FCP_ERR_CUDA;
  }
  attn_bwd_kernel<D, Bias><<<grid, kThreads, C::kSmem, st>>>(a.tm_q, a.tm_do, a.tm_k, a.tm_v, a.tm_kb,
                                                      a.tm_vb, a.tm_dq, a.tm_dk, a.tm_dv, p, bias);
  if constexpr (std::is_same_v<Bias, BiasParams>) table_sums_kernel<<<p.hq, kTableThreads, 0, st>>>(bias);
  return cudaGetLastError() == cudaSuccess ? FCP_OK : FCP_ERR_CUDA;
}

int launch_attn_bwd(const BwdLaunch& a, cudaStream_t st) {
  if (a.d == 128) return a.has_bias ? launch_bwd_impl<128>(a, a.bias, st) : launch_bwd_impl<128>(a, NoBias{}, st);
  if (a.d == 64) return a.has_bias ? launch_bwd_impl<64>(a, a.bias, st) : launch_bwd_impl<64>(a, NoBias{}, st);
  return FCP_ERR_UNSUPPORTED;
}

}  // namespace fcp
