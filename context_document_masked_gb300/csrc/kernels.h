// Launch interfaces of the libfcp device kernels (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/fcp.h"

// FCP_DEVICE_CHECKS=1 builds the checked library: every index the kernels
// read from the plan's device tables is checked against the table sizes and
// the tensors' rows before use; a failed check sets bit kErrBadTable of the
// error word (fcp_get_device_status: FCP_ERR_INVALID_ARG) and the kernel
// skips that work unit. It never traps.
#ifndef FCP_DEVICE_CHECKS
#define FCP_DEVICE_CHECKS 0
#endif

namespace fcp {

constexpr bool kDeviceChecks = FCP_DEVICE_CHECKS != 0;
constexpr int kErrBadTable = 8;

// Ints per backward unit in the plan's TB_BTILES table.
constexpr int kBwdTileInts = 12;

struct FwdParams {
  const int32_t* pieces;   // plan piece table
  const int32_t* segs;     // key segments
  const int32_t* tiles;    // query tiles (piece, q_start, q_rows, cost)
  const int32_t* order;    // tile indices to run, longest first
  int32_t n_items;
  int32_t kbuf_shift;      // subtracted from received-key rows (one-shard launches)
  int32_t kv_lo, kv_hi;    // key block
  int32_t seg_filter;      // -1: every key segment; else only segments whose first field equals it
  int32_t T, hq, hkv;
  float scale_log2;        // softmax scale * log2(e)
  int32_t out_f32;
  void* out;
  float* lse;
  int* err;
  int* work_counter;       // zero at launch (set by the preceding kernel of the call)
  const float* qk_scale;   // e4m3 Q K^T variant: the scales 2^kq, 2^kk of Q and K (else unused)
  int* rescale_count;      // if not null: +1 per warp each time O is rescaled after a later key tile
  int32_t order_block;     // work decode: items per block (set by the launch, see work_slot)
  int32_t n_tiles, n_pieces, n_segs, kb_rows;  // table sizes, rows behind tm_kb (checked build)
  int64_t wait_ns;
};

// Learned bias of the attention by buckets of the distance i - j: bucket u
// holds the distances from starts[u] to starts[u + 1] - 1 (the last one all
// from starts[u] on).
constexpr int kMaxBuckets = 128;
constexpr int kTableDistances = 8192;  // at most
struct BiasParams {
  const float* bias;       // [hq][n]
  float* dbias;            // backward: [hq][n], accumulated
  float* by_distance;      // backward: [hq][n_distances] sums of dS (set to zero by the launch)
  int32_t n_distances;
  int32_t parts, part_heads;  // backward: units a KV head's query heads are cut into, heads of a unit
  int32_t n;
  int32_t starts[kMaxBuckets];
};
struct NoBias {};          // kernels without a bias or a window take this in its place

// The mask of a windowed plan (fcp_plan_window): kernels for one take this in
// the bias's place. The sinks that a tile's queries see outside their windows lie
// in the first `slots` rows of one key tile (`slots` a multiple of 8, 0 for a plan
// without sinks), the tile's window keys behind them: boxes of `slots` and of
// 128 - slots rows.
struct WindowParams {
  CUtensorMap k_sinks, v_sinks, kb_sinks, vb_sinks;  // as tm_k, tm_v, tm_kb, tm_vb
  CUtensorMap k_rest, v_rest, kb_rest, vb_rest;
  CUtensorMap dk_sinks, dv_sinks, dk_rest, dv_rest;  // backward: as tm_dk, tm_dv
  int32_t window, sinks, slots;
  const int32_t* doubles;  // forward, odd groups: double query tiles (plan.h, TB_RPIECES)
  int32_t n_doubles;
};

struct FwdLaunch {
  CUtensorMap tm_q, tm_k, tm_v, tm_kb, tm_vb;
  FwdParams p;
  int d;
  int num_sms;
  bool qk8;                // Q, K, received K as e4m3 (boxes of 128 bytes x 1 x 128)
  bool has_bias;
  BiasParams bias;
  bool has_window;         // the plan is windowed (without a bias or e4m3)
  WindowParams window;
};

// Sizes of a backward's operands, found by its preprocess: each row of dO is
// divided by a power of two 2^e, and the kernel scales by these, so that the
// fp16 operands keep their bits whatever the gradient's size. Zero between calls.
struct BwdRange {
  unsigned e_max;          // largest e of a row that sees a key, + kRowExpBias (0: no such row)
  unsigned v2;             // bits of the largest |V_j|^2 (fp32)
  int done;                // CTAs of the backward that have ended
};
constexpr int kRowExpBias = 256;

struct BwdParams {
  const int32_t* pieces;
  const int32_t* tiles;    // backward units, kBwdTileInts ints each (plan.h, TB_BTILES)
  const int32_t* order;
  int32_t n_items;
  int32_t kbuf_shift;
  int32_t T, hq, hkv;
  float scale;             // softmax scale
  float scale_log2;
  const float* lse2;       // [Hq][T] -LSE log2 e + e, e the exponent taken out of the row's dO (BwdRange)
  const float* delta;      // [Hq][T] rowsum(dO * O) 2^-e
  float* dq;               // [T][Hq][d] fp32, accumulated
  float* dk;               // [T][Hkv][d] fp32, accumulated
  float* dv;
  BwdRange* range;
  int* err;
  int* work_counter;       // zero at launch (set by the preprocess)
  int32_t order_block;     // work decode: items per block (set by the launch, see work_slot)
  int32_t n_tiles, kb_rows;  // TB_BTILES size, rows behind tm_kb/tm_vb (checked build)
  int64_t wait_ns;
};

struct BwdLaunch {
  CUtensorMap tm_q, tm_do, tm_k, tm_v, tm_kb, tm_vb;
  CUtensorMap tm_dq;  // dQ fp32 [T][Hq][d], boxes of 32 x 1 x 128 (reduce-add target)
  CUtensorMap tm_dk, tm_dv;  // dK, dV fp32 [T][Hkv][d], same boxes (reduce-add targets)
  BwdParams p;
  int d;
  int num_sms;
  bool has_bias;
  BiasParams bias;
  bool has_window;
  WindowParams window;
};

int launch_attn_fwd(const FwdLaunch& a, cudaStream_t st);
int launch_attn_bwd(const BwdLaunch& a, cudaStream_t st);

// Limit of every bounded device wait (fcp_debug_set_wait_limit), in ns.
int64_t wait_limit_ns();

// Row statistics D_i = <dO_i, O_i> and LSE for the rows of the given row chunks,
// dQ rows set to zero, fp16 copies of Q and dO for the backward's MMAs (dO,
// delta and lse2 with the rows' exponents taken out, see BwdRange), and the
// range: V's from its rows [T][hkv][d] of the chunks and `v_rows` received rows
// of vbuf.
// *zero_word (if not null) is set to 0: the work counter of the kernel that
// follows in the same stream.
// n_rows_table: entries of `rows` (the checked build bounds the chunk indices).
// pieces: the shard's n_pieces entries of the piece table, ascending, whose last
// tiles' rows past the pieces are set to zero in the copies (with `any_tiles`,
// where tiles begin anywhere, 127 rows); none (0) for a call over all shards,
// which writes every row.
struct PreLaunch {
  const void* out;
  bool out_f32;
  const float* lse;        // [Hq][T]
  const __nv_bfloat16 *dout, *q, *v, *vbuf;
  int64_t v_rows;
  const int32_t* rows;
  const int32_t* order;
  int32_t n_chunks, n_rows_table, T, hq, hkv;
  float *delta, *lse2, *dq;
  __half *q16, *do16;
  BwdRange* range;
  const int32_t* pieces;
  int32_t n_pieces;
  bool any_tiles;
  int num_sms;
  int* err;
  int* zero_word;
};
int launch_bwd_preprocess(const PreLaunch& a, int32_t d, cudaStream_t st);

// fp16 copies of a bf16 array of n_elems (a multiple of 8) elements and of a
// second one of n_elems2 (0: none); *zero_word (if not null) is set to 0, as above.
int launch_convert_f16(const void* src, void* dst, int64_t n_elems, const void* src2, void* dst2, int64_t n_elems2, int* err,
                       int* zero_word, int num_sms, cudaStream_t st);

// bf16 copy (round to nearest even) of an fp32 array of n_elems (a multiple
// of 8) elements.
int launch_round_bf16(const float* src, void* dst, int64_t n_elems, int num_sms, cudaStream_t st);

// e4m3 copy of a bf16 array of n_elems (a multiple of 8) elements, scaled by
// the power of two 2^k, the largest with max|x| * 2^k <= 448 (exact to undo).
// *amax_bits must be zero on entry (it receives the bits of max|x|); the
// scale goes to *scale_out.
int launch_quant_e4m3(const void* src, void* dst, int64_t n_elems, unsigned* amax_bits,
                      float* scale_out, int num_sms, cudaStream_t st);
// The same with a scale computed before (from *amax_bits of another tensor):
// rows copied from that tensor share its scale.
int launch_quant_e4m3_with(const void* src, void* dst, int64_t n_elems, const unsigned* amax_bits,
                           int num_sms, cudaStream_t st);

// Gather of received KV rows: tasks (src_row, dst_row, nrows, shard); K/V
// hold src_rows rows, kbuf/vbuf dst_rows (bounds of the checked build).
int launch_gather(const void* k, const void* v, const int32_t* tasks, int32_t n_tasks,
                  int32_t dst_shift, int64_t row_bytes, void* kbuf, void* vbuf, int32_t src_rows,
                  int32_t dst_rows, int num_sms, cudaStream_t st);

int launch_merge(const float* o_parts, const float* lse_parts, int32_t B, int64_t rows, int32_t hq,
                 int32_t d, void* out, float* lse_out, int num_sms, cudaStream_t st);

// Head norm and rotation, and their gradient (norm_rope.cu). At most
// kNormRopeMaxCtas CTAs write partial sums of the weight gradients, summed in
// groups of kNormRopeGroup (the tickets of 14 groups and one for the groups
// fit the workspace header).
constexpr int kNormRopeGroup = 32;
constexpr int kNormRopeGroups = 14;
constexpr int kNormRopeMaxCtas = kNormRopeGroup * kNormRopeGroups;

struct NormRopeParams {
  const int32_t* pieces;   // plan piece table
  const int32_t* tiles;    // query tiles of the launch (piece, q_start, q_rows, cost)
  int32_t n_pieces;        // table size (checked build)
  int32_t n_units, chunk, chunks;  // units of `chunk` rows, `chunks` of them a tile (set by the launch)
  int32_t T, hq, hkv;
  int32_t norm;            // 0: rotation alone
  float eps;
  int32_t rot_dim;
  int32_t w_f32;           // weights: 1 fp32, 0 bf16
  const float* inv_freq;   // [rot_dim / 2]
  const void* wq;          // [d] or null (all ones)
  const void* wk;
  const __nv_bfloat16* q_in;  // rows of heads x d values, strides in elements
  const __nv_bfloat16* k_in;
  const __nv_bfloat16* v_in;
  int64_t q_in_stride, k_in_stride, v_in_stride;
  __nv_bfloat16* q;        // forward: contiguous outputs
  __nv_bfloat16* k;
  __nv_bfloat16* v;        // null: no V rows
  const float* dq;         // backward: contiguous fp32 gradients
  const float* dk;
  const float* dv;         // null: no V rows
  __nv_bfloat16* dq_in;
  __nv_bfloat16* dk_in;
  __nv_bfloat16* dv_in;
  int64_t dq_in_stride, dk_in_stride, dv_in_stride;
  int32_t add_dw;          // 1: dwq and dwk are added to
  float* dwq;              // [d] or null
  float* dwk;
  float* partial;          // [kNormRopeMaxCtas + their groups][2][d]
  int* tickets;            // 1 + kNormRopeGroups, zero at launch and at its end
  int* err;                // error word (checked build) or null
};

struct NormRopeLaunch {
  NormRopeParams p;
  int32_t n_tiles;
  int64_t rows;            // rows of those tiles
  int d;
  bool interleaved, backward;
  int num_sms;
};

int launch_norm_rope(const NormRopeLaunch& a, cudaStream_t st);

// The residual stream between two blocks, and its gradient (residual_norm.cu).
// *_row: bytes between rows. Null pointers: no block output, no gate, ones for
// weights, no norm before the next block (h and dh), no gradient of the residual
// after the block (dx_out); dx is null in the forward.
constexpr int kResNormMaxCtas = 1216;
constexpr int kResNormChunk = 128;   // rows of a chunk at most (plan.h, TB_ROWS)
struct ResNormParams {
  const int32_t* chunks;   // TB_ROWS entries of a shard; null: all tokens
  int64_t units;           // tokens, or of a shard kResNormChunk / unit_rows for each chunk
  int32_t unit_rows;       // 1 or kResNormChunk
  int32_t T, n, groups;    // (groups: set by the launch)
  int32_t post_norm, gate_fn, res_f32, w_f32, add_dw;
  float eps, res_scale, branch_scale;
  const void *x, *y, *gate, *w_post, *w_pre;  // x: before the block; in the backward after it
  int64_t x_row, y_row, gate_row;
  void *x_out, *h;
  int64_t x_out_row, h_row;
  const void *dh, *dx_out;
  int64_t dh_row, dx_out_row;
  void *dx, *dy, *dgate;
  int64_t dx_row, dy_row, dgate_row;
  float *dw_post, *dw_pre;
  float* partial;          // [res_norm_ws_bytes(n)]
  int num_sms;
};
int64_t res_norm_ws_bytes(int n);
int launch_res_norm(const ResNormParams& p, cudaStream_t st);

}  // namespace fcp
