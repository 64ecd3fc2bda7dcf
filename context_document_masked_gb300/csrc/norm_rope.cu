// RMS norm and rotary rotation of the query and key heads of a packed
// sequence, and its gradient.
//
// For every token t of the selected shard(s) and every query or key head x of
// it (d values, the projection's output):
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w            (w per dimension)
//   y = R(p) n,  p = t - start of t's document
// R(p) turns each of the first rot_dim / 2 pairs of dimensions by the angle
// p inv_freq[i]; the other dimensions pass. Positions start again at every
// document, and a context-parallel shard holds pieces of documents, so p
// comes from the plan's tiles, not from the row number. V rows are copied to
// their contiguous place in the same pass.
// Gradient, with z = R(p)^T dy and g = z w:
//   dx = r (g - x r^2 mean(g x)),  dw = sum over tokens and heads of z x r.
//
// Angles. p inv_freq / (2 pi) is taken modulo 1 exactly in integers: each
// frequency becomes a 64-bit fixed-point fraction of a turn once per CTA (by
// every warp, the few fp64 units made it half of a small call's time),
// and the fraction after p positions is the low 64 bits of an integer
// product, so a position of 10^6 is turned as exactly as position 1 (a
// product in fp32 would be off by up to 0.03 rad there).
//
// Layout. D / 8 lanes hold one head, eight values each as two chunks of four
// chosen so that both values of every pair are in one lane, in either pair
// order; a warp holds 2 heads (d = 128) or 4 (d = 64) at a time, a pass, and
// walks the heads of one token, whose angles it computes once: lane i those of
// pairs 2i and 2i + 1, handed round by shuffles.
//
// Bound: device memory, one read of each input and one write of each output,
// and its latency: four passes are loaded before the first is worked on, and
// the arithmetic runs on pairs of values (f32x2) to keep the registers that
// this takes. 65536 tokens of 64 + 8 + 8 heads of 128: 420 us, 6.39 TB/s (0.96
// of the copy rate measured on this part); gradient of 32768 tokens of 32 + 8
// + 8: 266 us, 5.80 TB/s (0.87). Slower: sixteen values a lane (gradient 287
// us, two passes do not fit), asynchronous copies into shared memory (485 and
// 370 us, for their instructions), units looked up ahead by the CTA (the same).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "sm103.cuh"

namespace fcp {

using namespace dev;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kE = 8;  // values of a head in a lane
// Passes over the heads in flight, and CTAs an SM, for the registers that both
// take (a few spilled ones cost the gradient a quarter of its speed).
constexpr int kFwdPasses = 4, kFwdCtas = 4, kBwdPasses = 4, kBwdCtas = 2;

__device__ __forceinline__ float f2_sum(uint64_t a, uint64_t b) {
  float lo, hi;
  f2_split(f2_add(a, b), lo, hi);
  return lo + hi;
}
// Where a lane's two chunks of kE / 2 values lie inside a head. The lanes of
// the first rot_dim values hold chunk l of the first half of the rotated
// dimensions and chunk l of the second half (the pairs (i, i + rot / 2) and the
// pairs (2i, 2i + 1) are then both inside a lane); the others two neighbouring
// chunks of the rest.
struct Lane {
  int l, head, off_a, off_b;
  bool turns;
};
template <int D>
__device__ __forceinline__ Lane lane_of(int lane, int rot_dim) {
  Lane x;
  x.l = lane % (D / kE);
  x.head = lane / (D / kE);
  x.turns = kE * x.l < rot_dim;
  x.off_a = x.turns ? kE / 2 * x.l : kE * x.l;
  x.off_b = x.turns ? (rot_dim + kE * x.l) / 2 : kE * x.l + kE / 2;
  return x;
}

// A lane's pairs (chunk a's, then chunk b's): bf16 as stored, and fp32.
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* at, const Lane& ln, uint32_t (&v)[kE / 2]) {
  const uint2 a = *reinterpret_cast<const uint2*>(at + ln.off_a), b = *reinterpret_cast<const uint2*>(at + ln.off_b);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
__device__ __forceinline__ void store_bf16(__nv_bfloat16* at, const Lane& ln, const uint64_t (&x)[kE / 2]) {
  *reinterpret_cast<uint2*>(at + ln.off_a) = make_uint2(pack2(x[0]), pack2(x[1]));
  *reinterpret_cast<uint2*>(at + ln.off_b) = make_uint2(pack2(x[2]), pack2(x[3]));
}
__device__ __forceinline__ void load_f32(const float* at, const Lane& ln, uint64_t (&x)[kE / 2]) {
  const float4 a = *reinterpret_cast<const float4*>(at + ln.off_a), b = *reinterpret_cast<const float4*>(at + ln.off_b);
  x[0] = f2(a.x, a.y), x[1] = f2(a.z, a.w), x[2] = f2(b.x, b.y), x[3] = f2(b.z, b.w);
}

// inv_freq (radians a position) as a fraction of a turn, in units of 2^-64.
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
  const double t = (double)inv_freq * 0.15915494309189533577;  // / (2 pi)
  return (uint64_t)((t - floor(t)) * 18446744073709551616.0);
}

// Cosines and sines of this lane's pairs at position `pos` (1 and 0 where it turns none); f0 and f1 are the
// frequencies of pairs 2 * lane and 2 * lane + 1.
template <bool INTER>
__device__ __forceinline__ void row_angles(uint32_t pos, uint64_t f0, uint64_t f1, const Lane& ln, int rot_dim,
                                           float (&c)[kE / 2], float (&s)[kE / 2]) {
  const float h0 = (float)(int32_t)((f0 * pos) >> 32) * 0x1p-31f;  // half turns, in [-1, 1]
  const float h1 = (float)(int32_t)((f1 * pos) >> 32) * 0x1p-31f;
  float c0, s0, c1, s1;
  sincospif(h0, &s0, &c0);
  sincospif(h1, &s1, &c1);
#pragma unroll
  for (int u = 0; u < kE / 4; ++u) {
    const int src = !INTER ? kE / 4 * ln.l + u : u < kE / 8 ? kE / 8 * ln.l + u : rot_dim / 8 + kE / 8 * ln.l + u - kE / 8;
    const float ca = __shfl_sync(0xffffffffu, c0, src), cb = __shfl_sync(0xffffffffu, c1, src);
    const float sa = __shfl_sync(0xffffffffu, s0, src), sb = __shfl_sync(0xffffffffu, s1, src);
    c[2 * u] = ln.turns ? ca : 1.f;
    c[2 * u + 1] = ln.turns ? cb : 1.f;
    s[2 * u] = ln.turns ? sa : 0.f;
    s[2 * u + 1] = ln.turns ? sb : 0.f;
  }
}

// The kE values of chunk a (the first kE / 4 pairs of registers) and chunk b
// turned in place: forwards for kSign = 1, backwards for -1. Where a lane turns
// none, its products with the sine take 0 for the value (an infinity times 0
// would not pass).
__device__ __forceinline__ uint64_t value_if(bool turns, uint64_t x) { return turns ? x : 0; }
template <bool INTER, int kSign>
__device__ __forceinline__ void turn(uint64_t (&x)[kE / 2], const float (&c)[kE / 2], const float (&s)[kE / 2], bool turns) {
  if constexpr (INTER) {  // pairs (2i, 2i + 1)
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) {
      float a, b, sa, sb;
      f2_split(x[e], a, b);
      f2_split(value_if(turns, x[e]), sa, sb);
      const float sn = kSign * s[e];
      x[e] = f2(a * c[e] - sb * sn, sa * sn + b * c[e]);
    }
  } else {  // value i of chunk a with value i of chunk b
#pragma unroll
    for (int i = 0; i < kE / 4; ++i) {
      const uint64_t c2 = f2(c[2 * i], c[2 * i + 1]), s2 = f2(s[2 * i], s[2 * i + 1]);
      const uint64_t n2 = f2(-s[2 * i], -s[2 * i + 1]);
      const uint64_t a = x[i], b = x[kE / 4 + i];
      x[i] = f2_fma(value_if(turns, b), kSign > 0 ? n2 : s2, f2_mul(a, c2));
      x[kE / 4 + i] = f2_fma(value_if(turns, a), kSign > 0 ? s2 : n2, f2_mul(b, c2));
    }
  }
}

// Sum over the N lanes of a head.
template <int N>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int m = 1; m < N; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

__device__ __forceinline__ float load_w(const void* w, int w_f32, int i) {
  if (!w) return 1.f;
  return w_f32 ? static_cast<const float*>(w)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// A unit of work: `chunk` rows of one query tile. Tiles are at most 128 rows
// of one piece; n_rows is 0 past the tile's end. (Checked build: a tile out of
// range is skipped. The forward has no error word; the attention calls read the
// same tables and report it.)
struct Rows {
  int first, n, pos;  // first row, rows, position of the first row in its document
};
__device__ __forceinline__ Rows unit_rows(const NormRopeParams& p, int u) {
  const int* t = p.tiles + 4 * (u / p.chunks);
  const int sub = (u % p.chunks) * p.chunk;
  const int piece = __ldg(t + 0), q0 = __ldg(t + 1), n = __ldg(t + 2);
  Rows r{0, 0, 0};
  if constexpr (kDeviceChecks) {
    if (piece < 0 || piece >= p.n_pieces || n < 1 || n > 128 || q0 < 0 || q0 > p.T - n) {
      if (p.err) atomicOr(p.err, kErrBadTable);
      return r;
    }
  }
  r.first = q0 + sub;
  r.n = min(p.chunk, n - sub);
  r.pos = r.first - __ldg(p.pieces + 8 * piece + 4);
  return r;
}

// ---------------------------------------------------------------- forward
template <int D, bool INTER>
__device__ __forceinline__ void heads_forward(const __nv_bfloat16* in, __nv_bfloat16* out, int n_heads, const float* w,
                                              const Lane& ln, const float (&c)[kE / 2], const float (&s)[kE / 2],
                                              const NormRopeParams& p) {
  constexpr int kHeads = 32 * kE / D;  // heads a warp holds at a time
  for (int h0 = 0; h0 < n_heads; h0 += kFwdPasses * kHeads) {
    uint32_t v[kFwdPasses][kE / 2];
#pragma unroll
    for (int u = 0; u < kFwdPasses; ++u) {
      const int h = h0 + u * kHeads + ln.head;
#pragma unroll
      for (int i = 0; i < kE / 2; ++i) v[u][i] = 0;
      if (h < n_heads) load_bf16(in + (size_t)h * D, ln, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kFwdPasses; ++u) {
      if (u > 0 && h0 + u * kHeads >= n_heads) break;
      const int h = h0 + u * kHeads + ln.head;
      uint64_t x[kE / 2];
#pragma unroll
      for (int i = 0; i < kE / 2; ++i) x[i] = unpack2(v[u][i]);
      if (p.norm) {
        uint64_t sa = 0, sb = 0, wl[kE / 2];
        load_f32(w, ln, wl);
#pragma unroll
        for (int i = 0; i < kE / 4; ++i) {
          sa = f2_fma(x[i], x[i], sa);
          sb = f2_fma(x[kE / 4 + i], x[kE / 4 + i], sb);
        }
        const float r = rsqrtf(head_sum<D / kE>(f2_sum(sa, sb)) * (1.f / D) + p.eps);
        const uint64_t r2 = f2(r, r);
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) x[i] = f2_mul(f2_mul(x[i], r2), wl[i]);
      }
      turn<INTER, 1>(x, c, s, ln.turns);
      if (h < n_heads) store_bf16(out + (size_t)h * D, ln, x);
    }
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, kFwdCtas) norm_rope_kernel(const NormRopeParams p) {
  __shared__ __align__(16) float w[2][D];
  __shared__ uint64_t turns[D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) w[i / D][i % D] = load_w(i < D ? p.wq : p.wk, p.w_f32, i % D);
  if (threadIdx.x < D / 2)
    turns[threadIdx.x] = 2 * threadIdx.x < p.rot_dim ? turn_fraction(__ldg(p.inv_freq + threadIdx.x)) : 0;
  __syncthreads();
  const Lane ln = lane_of<D>(lane, p.rot_dim);
  const uint64_t f0 = 2 * lane < D / 2 ? turns[2 * lane] : 0, f1 = 2 * lane < D / 2 ? turns[2 * lane + 1] : 0;
  for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
    const Rows rows = unit_rows(p, u);
    for (int i = warp; i < rows.n; i += kWarps) {
      const size_t t = rows.first + i;
      float c[kE / 2], s[kE / 2];
      row_angles<INTER>(rows.pos + i, f0, f1, ln, p.rot_dim, c, s);
      heads_forward<D, INTER>(p.q_in + t * p.q_in_stride, p.q + t * p.hq * D, p.hq, w[0], ln, c, s, p);
      heads_forward<D, INTER>(p.k_in + t * p.k_in_stride, p.k + t * p.hkv * D, p.hkv, w[1], ln, c, s, p);
      if (p.v) {
        const uint4* src = reinterpret_cast<const uint4*>(p.v_in + t * p.v_in_stride);
        uint4* dst = reinterpret_cast<uint4*>(p.v + t * p.hkv * D);
        for (int e = lane; e < p.hkv * D / 8; e += 32) dst[e] = src[e];
      }
    }
  }
}

// --------------------------------------------------------------- backward
// One token's heads: dx written, z x r added to acc (this lane's dims).
template <int D, bool INTER>
__device__ __forceinline__ void heads_backward(const float* dy, const __nv_bfloat16* in, __nv_bfloat16* dx, int n_heads,
                                               const float* w, uint64_t (&acc)[kE / 2], const Lane& ln,
                                               const float (&c)[kE / 2], const float (&s)[kE / 2],
                                               const NormRopeParams& p) {
  constexpr int kHeads = 32 * kE / D;
  for (int h0 = 0; h0 < n_heads; h0 += kBwdPasses * kHeads) {
    uint64_t zz[kBwdPasses][kE / 2];
    uint32_t v[kBwdPasses][kE / 2];
#pragma unroll
    for (int u = 0; u < kBwdPasses; ++u) {
      const int h = h0 + u * kHeads + ln.head;
#pragma unroll
      for (int i = 0; i < kE / 2; ++i) zz[u][i] = v[u][i] = 0;
      if (h < n_heads) {
        load_f32(dy + (size_t)h * D, ln, zz[u]);
        if (p.norm) load_bf16(in + (size_t)h * D, ln, v[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kBwdPasses; ++u) {
      if (u > 0 && h0 + u * kHeads >= n_heads) break;
      const int h = h0 + u * kHeads + ln.head;
      uint64_t(&z)[kE / 2] = zz[u];
      turn<INTER, -1>(z, c, s, ln.turns);
      if (p.norm) {
        uint64_t x[kE / 2], wl[kE / 2];
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) x[i] = unpack2(v[u][i]);
        load_f32(w, ln, wl);
        uint64_t sq = 0, gx2 = 0;
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
          sq = f2_fma(x[i], x[i], sq);
          gx2 = f2_fma(f2_mul(z[i], wl[i]), x[i], gx2);
        }
        const float ss = head_sum<D / kE>(f2_sum(sq, 0)), gx = head_sum<D / kE>(f2_sum(gx2, 0));
        // No head past the last one: with eps = 0 its 0 x inf would reach acc.
        const float r = h < n_heads ? rsqrtf(ss * (1.f / D) + p.eps) : 0.f;
        const float m = -r * (r * r * (gx * (1.f / D)));
        const uint64_t r2 = f2(r, r), m2 = f2(m, m);
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
          acc[i] = f2_fma(f2_mul(z[i], x[i]), r2, acc[i]);
          z[i] = f2_fma(x[i], m2, f2_mul(f2_mul(z[i], wl[i]), r2));
        }
      }
      if (h < n_heads) store_bf16(dx + (size_t)h * D, ln, z);
    }
  }
}

// Sum over the CTAs of `n` rows of 2 * D floats, rows stride apart, into out
// (fixed order). All threads of the CTA; every row was written before the
// ticket that let this CTA in was drawn. Added by one atomic an element: another
// call (with a workspace of its own, on another stream) may add to the same
// gradient.
template <int D>
__device__ __forceinline__ void sum_rows(const float* rows, int n, float* out_q, float* out_k, bool add) {
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float v[kNormRopeGroup];
#pragma unroll
    for (int r = 0; r < kNormRopeGroup; ++r) v[r] = r < n ? __ldcg(rows + (size_t)r * 2 * D + i) : 0.f;
#pragma unroll
    for (int m = kNormRopeGroup / 2; m; m >>= 1)
#pragma unroll
      for (int r = 0; r < m; ++r) v[r] += v[r + m];
    float* o = i < D ? out_q + i : out_k + i - D;
    if (o && add) red_add(o, v[0]);
    if (o && !add) *o = v[0];
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, kBwdCtas) norm_rope_bwd_kernel(const NormRopeParams p) {
  __shared__ __align__(16) float w[2][D];
  __shared__ uint64_t turns[D / 2];
  // The warps' sums of both weights' gradients, after the last row.
  __shared__ float sums[kWarps][2][D];
  __shared__ int ticket;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) w[i / D][i % D] = load_w(i < D ? p.wq : p.wk, p.w_f32, i % D);
  if (threadIdx.x < D / 2)
    turns[threadIdx.x] = 2 * threadIdx.x < p.rot_dim ? turn_fraction(__ldg(p.inv_freq + threadIdx.x)) : 0;
  __syncthreads();
  const Lane ln = lane_of<D>(lane, p.rot_dim);
  uint64_t aq[kE / 2], ak[kE / 2];
#pragma unroll
  for (int e = 0; e < kE / 2; ++e) aq[e] = ak[e] = 0;
  const uint64_t f0 = 2 * lane < D / 2 ? turns[2 * lane] : 0, f1 = 2 * lane < D / 2 ? turns[2 * lane + 1] : 0;
  for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
    const Rows rows = unit_rows(p, u);
    for (int i = warp; i < rows.n; i += kWarps) {
      const size_t t = rows.first + i;
      float c[kE / 2], s[kE / 2];
      row_angles<INTER>(rows.pos + i, f0, f1, ln, p.rot_dim, c, s);
      heads_backward<D, INTER>(p.dq + t * p.hq * D, p.q_in + t * p.q_in_stride, p.dq_in + t * p.dq_in_stride, p.hq, w[0],
                               aq, ln, c, s, p);
      heads_backward<D, INTER>(p.dk + t * p.hkv * D, p.k_in + t * p.k_in_stride, p.dk_in + t * p.dk_in_stride, p.hkv,
                               w[1], ak, ln, c, s, p);
      if (p.dv) {
        const float4* src = reinterpret_cast<const float4*>(p.dv + t * p.hkv * D);
        uint4* dst = reinterpret_cast<uint4*>(p.dv_in + t * p.dv_in_stride);
        for (int e = lane; e < p.hkv * D / 8; e += 32) {
          const float4 a = src[2 * e], b = src[2 * e + 1];
          dst[e] = make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
        }
      }
    }
  }
  if (!p.dwq && !p.dwk) return;

  // Weight gradients, in a fixed order (the result does not depend on which
  // CTA finishes when): lanes of a warp, warps of the CTA, CTAs of a group of
  // kNormRopeGroup by the last of them to finish, groups by the last group.
#pragma unroll
  for (int e = 0; e < kE / 2; ++e) {
    const int dim = 2 * e < kE / 2 ? ln.off_a + 2 * e : ln.off_b + 2 * e - kE / 2;
#pragma unroll
    for (int qk = 0; qk < 2; ++qk) {
      float lo, hi;
      f2_split(qk ? ak[e] : aq[e], lo, hi);
#pragma unroll
      for (int m = D / kE; m < 32; m <<= 1) {
        lo += __shfl_xor_sync(0xffffffffu, lo, m);
        hi += __shfl_xor_sync(0xffffffffu, hi, m);
      }
      if (lane < D / kE) {
        sums[warp][qk][dim] = lo;
        sums[warp][qk][dim + 1] = hi;
      }
    }
  }
  __syncthreads();
  float* part = p.partial + (size_t)blockIdx.x * 2 * D;
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += sums[k][i / D][i % D];
    __stcg(part + i, v);
  }
  const int group = blockIdx.x / kNormRopeGroup, n_groups = ((int)gridDim.x + kNormRopeGroup - 1) / kNormRopeGroup;
  const int in_group = min(kNormRopeGroup, (int)gridDim.x - group * kNormRopeGroup);
  // Tickets count up to the group's size and are set back to zero by the CTA
  // that draws the last one.
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) ticket = atomicAdd(p.tickets + 1 + group, 1);
  __syncthreads();
  if (ticket != in_group - 1) return;
  __threadfence();
  if (threadIdx.x == 0) p.tickets[1 + group] = 0;
  const float* rows = p.partial + (size_t)group * kNormRopeGroup * 2 * D;
  if (n_groups == 1) {
    sum_rows<D>(rows, in_group, p.dwq, p.dwk, p.add_dw != 0);
    return;
  }
  float* gpart = p.partial + (size_t)(kNormRopeMaxCtas + group) * 2 * D;
  sum_rows<D>(rows, in_group, gpart, gpart + D, false);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) ticket = atomicAdd(p.tickets, 1);
  __syncthreads();
  if (ticket != n_groups - 1) return;
  __threadfence();
  if (threadIdx.x == 0) p.tickets[0] = 0;
  float* all = p.partial + (size_t)kNormRopeMaxCtas * 2 * D;
  sum_rows<D>(all, n_groups, p.dwq, p.dwk, p.add_dw != 0);
}

}  // namespace

int launch_norm_rope(const NormRopeLaunch& a, cudaStream_t st) {
  NormRopeParams p = a.p;
  if (a.n_tiles == 0) {  // a shard without tokens
    for (float* dw : {p.dwq, p.dwk})
      if (a.backward && !p.add_dw && dw && cudaMemsetAsync(dw, 0, sizeof(float) * a.d, st) != cudaSuccess)
        return FCP_ERR_CUDA;
    return FCP_OK;
  }
  // Rows a CTA takes at a time: 8, one a warp, as a small sequence has to
  // spread over all SMs; whole tiles where tiles are short (documents of a
  // few tokens), whose units would otherwise mostly be empty (32768 tokens of 32 +
  // 8 + 8 heads of 128, forward and gradient: documents of one token 505 us and
  // 1.14 ms, in units of 8 rows 7.49 and 17.2; of 12 157 and 284 us for 736 and
  // 1776; of 63, below the border of 64, 145 and 269 for 189 and 386).
  const bool short_tiles = (int64_t)a.rows < (int64_t)a.n_tiles * 64 && a.n_tiles >= 2 * a.num_sms;
  p.chunk = short_tiles ? 128 : kWarps;
  p.chunks = 128 / p.chunk;
  const int64_t units = (int64_t)a.n_tiles * p.chunks;
  if (units > INT32_MAX) return FCP_ERR_UNSUPPORTED;
  p.n_units = (int)units;
  const int most = a.num_sms * (a.backward ? kBwdCtas : kFwdCtas);
  int64_t grid = units < most ? units : most;
  if (a.backward && grid > kNormRopeMaxCtas) grid = kNormRopeMaxCtas;
  auto go = [&](auto kernel) {
    kernel<<<(int)grid, kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? FCP_OK : FCP_ERR_CUDA;
  };
  if (a.backward) {
    if (a.d == 128) return a.interleaved ? go(norm_rope_bwd_kernel<128, true>) : go(norm_rope_bwd_kernel<128, false>);
    return a.interleaved ? go(norm_rope_bwd_kernel<64, true>) : go(norm_rope_bwd_kernel<64, false>);
  }
  if (a.d == 128) return a.interleaved ? go(norm_rope_kernel<128, true>) : go(norm_rope_kernel<128, false>);
  return a.interleaved ? go(norm_rope_kernel<64, true>) : go(norm_rope_kernel<64, false>);
}

}  // namespace fcp
