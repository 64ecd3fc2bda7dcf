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
// frequency becomes a 64-bit fixed-point fraction of a turn once per warp,
// and the fraction after p positions is the low 64 bits of an integer
// product, so a position of 10^6 is turned as exactly as position 1 (a
// product in fp32 would be off by up to 0.03 rad there).
//
// Layout. D / 16 lanes hold one head, 16 values each as two 16-byte chunks
// chosen so that both values of every pair are in one lane, in either pair
// order; a warp holds 4 heads (d = 128) or 8 (d = 64) at a time and walks the
// heads of one token, whose angles it computes once: lane i those of pairs
// 2i and 2i + 1, handed round by shuffles.
//
// Bound: device memory, one read of each input and one write of each output.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"

namespace fcp {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float lo16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi16(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  x[0] = lo16(v.x), x[1] = hi16(v.x), x[2] = lo16(v.y), x[3] = hi16(v.y);
  x[4] = lo16(v.z), x[5] = hi16(v.z), x[6] = lo16(v.w), x[7] = hi16(v.w);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// Where a lane's two chunks lie inside a head. Lanes below n_rot hold chunk l
// of the first half of the rotated dimensions and chunk l of the second half
// (the pairs (i, i + rot / 2) and the pairs (2i, 2i + 1) are then both inside
// a lane); the others two neighbouring chunks of the rest.
struct Lane {
  int l, head, off_a, off_b;
  bool turns;
};
template <int D>
__device__ __forceinline__ Lane lane_of(int lane, int rot_dim) {
  constexpr int kPerHead = D / 16;
  const int n_rot = rot_dim / 16;
  Lane x;
  x.l = lane % kPerHead;
  x.head = lane / kPerHead;
  x.turns = x.l < n_rot;
  x.off_a = x.turns ? 8 * x.l : 16 * x.l;
  x.off_b = x.turns ? rot_dim / 2 + 8 * x.l : 16 * x.l + 8;
  return x;
}

// inv_freq (radians a position) as a fraction of a turn, in units of 2^-64.
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
  const double t = (double)inv_freq * 0.15915494309189533577;  // / (2 pi)
  return (uint64_t)((t - floor(t)) * 18446744073709551616.0);
}

// Cosines and sines of this lane's eight pairs at position `pos`; f0 and f1
// are the frequencies of pairs 2 * lane and 2 * lane + 1.
template <bool INTER>
__device__ __forceinline__ void row_angles(uint32_t pos, uint64_t f0, uint64_t f1, const Lane& ln, int n_rot,
                                           float (&c)[8], float (&s)[8]) {
  const float h0 = (float)(int32_t)((f0 * pos) >> 32) * 0x1p-31f;  // half turns, in [-1, 1]
  const float h1 = (float)(int32_t)((f1 * pos) >> 32) * 0x1p-31f;
  float c0, s0, c1, s1;
  sincospif(h0, &s0, &c0);
  sincospif(h1, &s1, &c1);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int src = INTER ? (u < 2 ? 2 * ln.l + u : 2 * n_rot + 2 * ln.l + u - 2) : 4 * ln.l + u;
    const float ca = __shfl_sync(0xffffffffu, c0, src), cb = __shfl_sync(0xffffffffu, c1, src);
    const float sa = __shfl_sync(0xffffffffu, s0, src), sb = __shfl_sync(0xffffffffu, s1, src);
    c[2 * u] = ln.turns ? ca : 1.f;
    c[2 * u + 1] = ln.turns ? cb : 1.f;
    s[2 * u] = ln.turns ? sa : 0.f;
    s[2 * u + 1] = ln.turns ? sb : 0.f;
  }
}

// The sixteen values x[0..7] (chunk a), x[8..15] (chunk b) turned in place:
// forwards for kSign = 1, backwards for -1.
template <bool INTER, int kSign>
__device__ __forceinline__ void turn16(float (&x)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = INTER ? 2 * e : e, k = INTER ? 2 * e + 1 : 8 + e;
    const float a = x[i], b = x[k], sn = kSign * s[e];
    x[i] = a * c[e] - b * sn;
    x[k] = a * sn + b * c[e];
  }
}

template <int D>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int m = 1; m < D / 16; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

__device__ __forceinline__ float load_w(const void* w, int w_f32, int i) {
  if (!w) return 1.f;
  return w_f32 ? static_cast<const float*>(w)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// A unit of work: `chunk` rows of one query tile. Tiles are at most 128 rows
// of one piece; n_rows is 0 past the tile's end.
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
                                              const Lane& ln, const float (&c)[8], const float (&s)[8],
                                              const NormRopeParams& p) {
  constexpr int kHeads = 512 / D;  // heads a warp holds at a time
  float wl[16];
#pragma unroll
  for (int e = 0; e < 8; ++e) wl[e] = w[ln.off_a + e], wl[8 + e] = w[ln.off_b + e];
  for (int h0 = 0; h0 < n_heads; h0 += 2 * kHeads) {
    uint4 a[2], b[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int h = h0 + u * kHeads + ln.head;
      a[u] = b[u] = make_uint4(0, 0, 0, 0);
      if (h < n_heads) {
        a[u] = *reinterpret_cast<const uint4*>(in + (size_t)h * D + ln.off_a);
        b[u] = *reinterpret_cast<const uint4*>(in + (size_t)h * D + ln.off_b);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int h = h0 + u * kHeads + ln.head;
      float x[16];
      unpack8(a[u], x);
      unpack8(b[u], x + 8);
      if (p.norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(head_sum<D>(ss) * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * r * wl[e];
      }
      turn16<INTER, 1>(x, c, s);
      if (h < n_heads) {
        *reinterpret_cast<uint4*>(out + (size_t)h * D + ln.off_a) = pack8(x);
        *reinterpret_cast<uint4*>(out + (size_t)h * D + ln.off_b) = pack8(x + 8);
      }
    }
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeParams p) {
  __shared__ float w[2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) w[i / D][i % D] = load_w(i < D ? p.wq : p.wk, p.w_f32, i % D);
  __syncthreads();
  const Lane ln = lane_of<D>(lane, p.rot_dim);
  const int n_rot = p.rot_dim / 16, n_pairs = p.rot_dim / 2;
  const uint64_t f0 = 2 * lane < n_pairs ? turn_fraction(__ldg(p.inv_freq + 2 * lane)) : 0;
  const uint64_t f1 = 2 * lane < n_pairs ? turn_fraction(__ldg(p.inv_freq + 2 * lane + 1)) : 0;
  for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
    const Rows rows = unit_rows(p, u);
    for (int i = warp; i < rows.n; i += kWarps) {
      const size_t t = rows.first + i;
      float c[8], s[8];
      row_angles<INTER>(rows.pos + i, f0, f1, ln, n_rot, c, s);
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
// One token's heads: dx written, z x r added to acc[16] (this lane's dims).
template <int D, bool INTER>
__device__ __forceinline__ void heads_backward(const float* dy, const __nv_bfloat16* in, __nv_bfloat16* dx, int n_heads,
                                               const float* w, float (&acc)[16], const Lane& ln, const float (&c)[8],
                                               const float (&s)[8], const NormRopeParams& p) {
  constexpr int kHeads = 512 / D;
  for (int h0 = 0; h0 < n_heads; h0 += kHeads) {
    const int h = h0 + ln.head;
    float z[16], x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) z[e] = x[e] = 0.f;
    if (h < n_heads) {
      const float4* ga = reinterpret_cast<const float4*>(dy + (size_t)h * D + ln.off_a);
      const float4* gb = reinterpret_cast<const float4*>(dy + (size_t)h * D + ln.off_b);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 va = ga[i], vb = gb[i];
        z[4 * i] = va.x, z[4 * i + 1] = va.y, z[4 * i + 2] = va.z, z[4 * i + 3] = va.w;
        z[8 + 4 * i] = vb.x, z[9 + 4 * i] = vb.y, z[10 + 4 * i] = vb.z, z[11 + 4 * i] = vb.w;
      }
      if (p.norm) {
        unpack8(*reinterpret_cast<const uint4*>(in + (size_t)h * D + ln.off_a), x);
        unpack8(*reinterpret_cast<const uint4*>(in + (size_t)h * D + ln.off_b), x + 8);
      }
    }
    turn16<INTER, -1>(z, c, s);
    if (p.norm) {
      float ss = 0.f, gx = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float g = z[e] * w[(e < 8 ? ln.off_a : ln.off_b - 8) + e];
        ss = fmaf(x[e], x[e], ss);
        gx = fmaf(g, x[e], gx);
      }
      ss = head_sum<D>(ss);
      gx = head_sum<D>(gx);
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      const float m = r * r * (gx * (1.f / D));
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float g = z[e] * w[(e < 8 ? ln.off_a : ln.off_b - 8) + e];
        acc[e] = fmaf(z[e], x[e] * r, acc[e]);
        z[e] = r * (g - x[e] * m);
      }
    }
    if (h < n_heads) {
      *reinterpret_cast<uint4*>(dx + (size_t)h * D + ln.off_a) = pack8(z);
      *reinterpret_cast<uint4*>(dx + (size_t)h * D + ln.off_b) = pack8(z + 8);
    }
  }
}

// Sum over the CTAs of `n` rows of 2 * D floats, rows stride apart, into out
// (fixed order). All threads of the CTA; every row was written before the
// ticket that let this CTA in was drawn.
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
    if (o) *o = add ? *o + v[0] : v[0];
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_bwd_kernel(const NormRopeParams p) {
  __shared__ float w[2][D];
  // Each lane's sixteen sums for the key weights, then (after the last row)
  // the warps' sums of both weights.
  __shared__ float4 acc_k[kWarps][4][32];
  __shared__ int ticket;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) w[i / D][i % D] = load_w(i < D ? p.wq : p.wk, p.w_f32, i % D);
#pragma unroll
  for (int e = 0; e < 4; ++e) acc_k[warp][e][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  const Lane ln = lane_of<D>(lane, p.rot_dim);
  const int n_rot = p.rot_dim / 16, n_pairs = p.rot_dim / 2;
  const uint64_t f0 = 2 * lane < n_pairs ? turn_fraction(__ldg(p.inv_freq + 2 * lane)) : 0;
  const uint64_t f1 = 2 * lane < n_pairs ? turn_fraction(__ldg(p.inv_freq + 2 * lane + 1)) : 0;
  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
    const Rows rows = unit_rows(p, u);
    for (int i = warp; i < rows.n; i += kWarps) {
      const size_t t = rows.first + i;
      float c[8], s[8];
      row_angles<INTER>(rows.pos + i, f0, f1, ln, n_rot, c, s);
      heads_backward<D, INTER>(p.dq + t * p.hq * D, p.q_in + t * p.q_in_stride, p.dq_in + t * p.dq_in_stride, p.hq, w[0],
                               acc, ln, c, s, p);
      float ak[16];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 v = acc_k[warp][e][lane];
        ak[4 * e] = v.x, ak[4 * e + 1] = v.y, ak[4 * e + 2] = v.z, ak[4 * e + 3] = v.w;
      }
      heads_backward<D, INTER>(p.dk + t * p.hkv * D, p.k_in + t * p.k_in_stride, p.dk_in + t * p.dk_in_stride, p.hkv,
                               w[1], ak, ln, c, s, p);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc_k[warp][e][lane] = make_float4(ak[4 * e], ak[4 * e + 1], ak[4 * e + 2], ak[4 * e + 3]);
      if (p.dv) {
        const float4* src = reinterpret_cast<const float4*>(p.dv + t * p.hkv * D);
        uint4* dst = reinterpret_cast<uint4*>(p.dv_in + t * p.dv_in_stride);
        for (int e = lane; e < p.hkv * D / 8; e += 32) {
          const float4 a = src[2 * e], b = src[2 * e + 1];
          dst[e] = make_uint4(pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w));
        }
      }
    }
  }
  if (!p.dwq && !p.dwk) return;

  // Weight gradients, in a fixed order (the result does not depend on which
  // CTA finishes when): lanes of a warp, warps of the CTA, CTAs of a group of
  // kNormRopeGroup by the last of them to finish, groups by the last group.
  float ak[16];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 v = acc_k[warp][e][lane];
    ak[4 * e] = v.x, ak[4 * e + 1] = v.y, ak[4 * e + 2] = v.z, ak[4 * e + 3] = v.w;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e)
#pragma unroll
    for (int m = D / 16; m < 32; m <<= 1) {
      acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], m);
      ak[e] += __shfl_xor_sync(0xffffffffu, ak[e], m);
    }
  __syncthreads();
  float* sums = reinterpret_cast<float*>(acc_k);  // [kWarps][2][D]
  if (lane < D / 16) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int dim = e < 8 ? ln.off_a + e : ln.off_b + e - 8;
      sums[(warp * 2 + 0) * D + dim] = acc[e];
      sums[(warp * 2 + 1) * D + dim] = ak[e];
    }
  }
  __syncthreads();
  float* part = p.partial + (size_t)blockIdx.x * 2 * D;
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += sums[k * 2 * D + i];
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
    sum_rows<D>(rows, in_group, p.dwq, p.dwk, true);
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
  for (int g = 0; g < n_groups; g += kNormRopeGroup)
    sum_rows<D>(all + (size_t)g * 2 * D, min(kNormRopeGroup, n_groups - g), p.dwq, p.dwk, true);
}

}  // namespace

int launch_norm_rope(const NormRopeLaunch& a, cudaStream_t st) {
  NormRopeParams p = a.p;
  if (a.n_tiles == 0) return FCP_OK;
  // Rows a CTA takes at a time: 8, one a warp, as a small sequence has to
  // spread over all SMs; whole tiles where tiles are short (documents of a
  // few tokens), whose units would otherwise mostly be empty.
  const bool short_tiles = (int64_t)a.rows < (int64_t)a.n_tiles * 64 && a.n_tiles >= 2 * a.num_sms;
  p.chunk = short_tiles ? 128 : kWarps;
  p.chunks = 128 / p.chunk;
  const int64_t units = (int64_t)a.n_tiles * p.chunks;
  if (units > INT32_MAX) return FCP_ERR_UNSUPPORTED;
  p.n_units = (int)units;
  const int most = a.num_sms * (a.backward ? 2 : 4);
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
