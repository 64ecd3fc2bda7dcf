// The stream between two blocks of a layer, and its gradient.
//
// For every token of the selected shard(s), with the block's output y, its gate
// z and the residual x before the block (rows of n values):
//   u = y r_y w_post,  r_y = 1 / sqrt(mean(y^2) + eps)   (r_y = 1 without post_norm)
//   X = a x + b g(z) u                                   (g: sigmoid or as it is)
//   h = X r w_pre,     r = 1 / sqrt(mean(X^2) + eps)
// X is stored as the residual after the block; h, the next block's input, comes
// from X before that rounding. Gradient, from dh and the stored X's dX':
//   dX = dX' + r (k - X r^2 mean(k X)),  k = dh w_pre
//   dx = a dX,  c = b dX,  dz = c u g'(z),  e = c g(z) w_post
//   dy = r_y (e - y r_y^2 mean(e y))  (e without post_norm)
//   dw_pre = sum dh X r,  dw_post = sum c g(z) y r_y   over the shard's tokens.
//
// One CTA holds a row at a time, one or two groups of eight values a thread, and
// takes rows grid by grid. Sums over a row are in fp32: lanes, then warps through
// shared memory. The weights' gradients stay in the thread that holds the
// columns; at the end each CTA writes them as one row, and a second kernel
// sums the rows in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "sm103.cuh"

namespace fcp {

using namespace dev;

namespace {

constexpr int kV = 8;  // values of a group: 16 bytes of bf16
constexpr int kMaxWarps = 32;

// Groups a thread holds, and threads a row: one group up to 2048 values, two
// above (16384 values: 1024 threads).
__host__ __device__ constexpr int groups_of(int n) { return n <= 2048 ? 1 : 2; }
__host__ __device__ constexpr int threads_of(int n) { return (n / kV + 32 * groups_of(n) - 1) / (32 * groups_of(n)) * 32; }
int most_ctas(int n) { return std::min(kResNormMaxCtas, 152 * 1024 / threads_of(n)); }

__device__ __forceinline__ void load8(const void* row, bool f32, int i, float (&v)[kV]) {
  if (f32) {
    const float4 a = reinterpret_cast<const float4*>(row)[2 * i], b = reinterpret_cast<const float4*>(row)[2 * i + 1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(row)[i];
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = __uint_as_float(w[j] << 16), v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8(void* row, bool f32, int i, const float (&v)[kV]) {
  if (f32) {
    reinterpret_cast<float4*>(row)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(row)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    reinterpret_cast<uint4*>(row)[i] =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
}
// Weights of group i; ones without.
__device__ __forceinline__ void load_w(const void* w, bool f32, int i, float (&v)[kV]) {
  if (w) {
    load8(w, f32, i, v);
  } else {
#pragma unroll
    for (int e = 0; e < kV; ++e) v[e] = 1.f;
  }
}

// Sums of K values over the CTA's threads (every thread gets them). `sh` is not
// read any more when the next call's values arrive in the other half.
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float (*sh)[kMaxWarps], int& half) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int m = 16; m; m >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  float(*s)[kMaxWarps] = sh + 4 * half;
  half ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) s[k][threadIdx.x >> 5] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float t = 0.f;
    for (int w = 0; w < warps; ++w) t += s[k][w];
    v[k] = t;
  }
}

// g(z) and g'(z); the sigmoid and its derivative without a loss of bits at
// either end (e = exp(-|z|) is at most 1).
__device__ __forceinline__ void gate_of(int fn, float z, float& g, float& dg) {
  if (fn == FCP_GATE_SIGMOID) {
    const float e = __expf(-fabsf(z)), d = __fdividef(1.f, 1.f + e);
    g = z >= 0.f ? d : e * d;
    dg = e * d * d;
  } else {
    g = z;
    dg = 1.f;
  }
}

// Row k of the launch: a token, or -1 for a place past a chunk's end. Chunks are
// runs of at most kResNormChunk rows of a shard; none for all tokens in order.
__device__ __forceinline__ int64_t row_at(const ResNormParams& p, int64_t k) {
  if (!p.chunks) return k;
  const int32_t* c = p.chunks + 2 * (k / kResNormChunk);
  const int r = (int)(k % kResNormChunk), first = __ldg(c), n = __ldg(c + 1);
  if constexpr (kDeviceChecks) {
    if (first < 0 || n < 0 || first > p.T - n) return -1;
  }
  return r < n ? first + r : -1;
}

__device__ __forceinline__ const char* at(const void* base, int64_t row_bytes, int64_t t) {
  return static_cast<const char*>(base) + row_bytes * t;
}
__device__ __forceinline__ char* at(void* base, int64_t row_bytes, int64_t t) {
  return static_cast<char*>(base) + row_bytes * t;
}

template <int G>
__global__ void __launch_bounds__(1024) res_norm_kernel(const ResNormParams p) {
  __shared__ float sh[8][kMaxWarps];
  int half = 0;
  const float inv_n = 1.f / p.n;
  for (int64_t k = blockIdx.x; k < p.places; k += gridDim.x) {
    const int64_t t = row_at(p, k);
    if (t < 0) continue;
    float x[G][kV], y[G][kV];
    float sum[1] = {0.f};
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
#pragma unroll
      for (int e = 0; e < kV; ++e) x[c][e] = y[c][e] = 0.f;
      if (i < p.groups) {
        load8(at(p.x, p.x_row, t), p.res_f32, i, x[c]);
        if (p.y) load8(at(p.y, p.y_row, t), false, i, y[c]);
      }
#pragma unroll
      for (int e = 0; e < kV; ++e) sum[0] += y[c][e] * y[c][e];
    }
    float ry = 1.f;
    if (p.y && p.post_norm) {
      row_sums(sum, sh, half);
      ry = rsqrtf(sum[0] * inv_n + p.eps);
    }
    sum[0] = 0.f;
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i >= p.groups) continue;
      float w[kV], z[kV];
      load_w(p.w_post, p.w_f32, i, w);
      if (p.gate) load8(at(p.gate, p.gate_row, t), false, i, z);
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        float g = 1.f, dg;
        if (p.gate) gate_of(p.gate_fn, z[e], g, dg);
        x[c][e] = p.res_scale * x[c][e] + (p.y ? p.branch_scale * g * (y[c][e] * ry * w[e]) : 0.f);
        sum[0] += x[c][e] * x[c][e];
      }
      if (p.x_out) store8(at(p.x_out, p.x_out_row, t), p.res_f32, i, x[c]);
    }
    if (!p.h) continue;
    row_sums(sum, sh, half);
    const float r = rsqrtf(sum[0] * inv_n + p.eps);
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i >= p.groups) continue;
      float w[kV];
      load_w(p.w_pre, p.w_f32, i, w);
#pragma unroll
      for (int e = 0; e < kV; ++e) w[e] *= x[c][e] * r;
      store8(at(p.h, p.h_row, t), false, i, w);
    }
  }
}

template <int G>
__global__ void __launch_bounds__(1024) res_norm_bwd_kernel(const ResNormParams p) {
  __shared__ float sh[8][kMaxWarps];
  int half = 0;
  const float inv_n = 1.f / p.n;
  float acc_pre[G][kV], acc_post[G][kV];
#pragma unroll
  for (int c = 0; c < G; ++c)
#pragma unroll
    for (int e = 0; e < kV; ++e) acc_pre[c][e] = acc_post[c][e] = 0.f;
  for (int64_t k = blockIdx.x; k < p.places; k += gridDim.x) {
    const int64_t t = row_at(p, k);
    if (t < 0) continue;
    float x[G][kV], dh[G][kV], y[G][kV];
    float sum[3] = {0.f, 0.f, 0.f};  // X^2, k X, y^2
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
#pragma unroll
      for (int e = 0; e < kV; ++e) x[c][e] = dh[c][e] = y[c][e] = 0.f;
      if (i < p.groups) {
        float w[kV];
        if (p.dh) {
          load8(at(p.x, p.x_row, t), p.res_f32, i, x[c]);
          load8(at(p.dh, p.dh_row, t), false, i, dh[c]);
          load_w(p.w_pre, p.w_f32, i, w);
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            sum[0] += x[c][e] * x[c][e];
            sum[1] += dh[c][e] * w[e] * x[c][e];
          }
        }
        if (p.y) load8(at(p.y, p.y_row, t), false, i, y[c]);
#pragma unroll
        for (int e = 0; e < kV; ++e) sum[2] += y[c][e] * y[c][e];
      }
    }
    row_sums(sum, sh, half);
    const float r = p.dh ? rsqrtf(sum[0] * inv_n + p.eps) : 0.f;
    const float m = r * (r * r * (sum[1] * inv_n));
    const float ry = p.post_norm && p.y ? rsqrtf(sum[2] * inv_n + p.eps) : 1.f;
    float ey[1] = {0.f};
    // dh becomes e.
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i >= p.groups) continue;
      float w[kV], d[kV], z[kV], dz[kV];
      load_w(p.w_pre, p.w_f32, i, w);
#pragma unroll
      for (int e = 0; e < kV; ++e) d[e] = 0.f;
      if (p.dx_out) load8(at(p.dx_out, p.dx_out_row, t), p.res_f32, i, d);
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        acc_pre[c][e] += dh[c][e] * x[c][e] * r;
        d[e] += r * (dh[c][e] * w[e]) - x[c][e] * m;
        z[e] = p.res_scale * d[e];
      }
      store8(at(p.dx, p.dx_row, t), p.res_f32, i, z);
      if (!p.y) continue;
      load_w(p.w_post, p.w_f32, i, w);
      if (p.gate) load8(at(p.gate, p.gate_row, t), false, i, z);
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        float g = 1.f, dg = 0.f;
        if (p.gate) gate_of(p.gate_fn, z[e], g, dg);
        const float cd = p.branch_scale * d[e], u = y[c][e] * ry;
        dz[e] = cd * (u * w[e]) * dg;
        acc_post[c][e] += cd * g * u;
        dh[c][e] = cd * g * w[e];
        ey[0] += dh[c][e] * y[c][e];
      }
      if (p.gate) store8(at(p.dgate, p.dgate_row, t), false, i, dz);
    }
    if (!p.y) continue;
    float my = 0.f;
    if (p.post_norm) {
      row_sums(ey, sh, half);
      my = ry * (ry * ry * (ey[0] * inv_n));
    }
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i >= p.groups) continue;
#pragma unroll
      for (int e = 0; e < kV; ++e) y[c][e] = ry * dh[c][e] - y[c][e] * my;
      store8(at(p.dy, p.dy_row, t), false, i, y[c]);
    }
  }
  float* part = p.partial + (size_t)blockIdx.x * 2 * p.n;
#pragma unroll
  for (int c = 0; c < G; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    if (i >= p.groups) continue;
    if (p.dw_post) store8(part, true, i, acc_post[c]);
    if (p.dw_pre) store8(part + p.n, true, i, acc_pre[c]);
  }
}

// Sums of the CTAs' rows: 32 columns a block, its warps every 32nd row, then the
// warps one after another. Added by one atomic an element (another call may
// add to the same gradient).
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) res_norm_dw_kernel(const float* partial, int rows, int n, float* dw_post,
                                                                     float* dw_pre, int add) {
  __shared__ float sh[kSumWarps][33];
  float* out = blockIdx.y ? dw_pre : dw_post;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = 32 * blockIdx.x + lane;
  float v = 0.f;
  if (col < n)
#pragma unroll 4
    for (int r = warp; r < rows; r += kSumWarps) v += __ldcg(partial + ((size_t)2 * r + blockIdx.y) * n + col);
  sh[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && col < n) {
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) v += sh[w][lane];
    if (add) red_add(out + col, v);
    else out[col] = v;
  }
}

}  // namespace

int64_t res_norm_ws_bytes(int n) { return (int64_t)most_ctas(n) * 2 * n * sizeof(float); }

int launch_res_norm(const ResNormParams& a, cudaStream_t st) {
  ResNormParams p = a;
  p.groups = p.n / kV;
  const int threads = threads_of(p.n), grid = (int)std::min<int64_t>(p.places, most_ctas(p.n));
  if (grid > 0) {
    const bool two = groups_of(p.n) == 2;
    if (p.dx) two ? res_norm_bwd_kernel<2><<<grid, threads, 0, st>>>(p) : res_norm_bwd_kernel<1><<<grid, threads, 0, st>>>(p);
    else two ? res_norm_kernel<2><<<grid, threads, 0, st>>>(p) : res_norm_kernel<1><<<grid, threads, 0, st>>>(p);
  }
  // (A shard without tokens: no rows, whose sum is written as zero.)
  if (p.dx && (p.dw_post || p.dw_pre))
    res_norm_dw_kernel<<<dim3((p.n + 31) / 32, 2), 32 * kSumWarps, 0, st>>>(p.partial, grid, p.n, p.dw_post, p.dw_pre,
                                                                          p.add_dw);
  return cudaGetLastError() == cudaSuccess ? FCP_OK : FCP_ERR_CUDA;
}

}  // namespace fcp
