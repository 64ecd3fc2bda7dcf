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
// takes rows grid by grid. The next row's operands are fetched into shared memory
// by asynchronous copies while one is worked on (a ring of two; its words are
// read by the warp that fetched them, so no barrier guards it). Sums over a row are in
// fp32: lanes, then warps through shared memory. The weights' gradients stay in
// the thread that holds the columns; at the end each CTA writes them as one row,
// and a second kernel sums the rows in a fixed order.
//
// Bound: device memory, each operand read once and each result written once; on the
// way there instructions and, in the gradient, registers (its sums take 32 of a
// thread's 128, which leaves 16 warps an SM). 65536 rows of 8192, bf16 residual,
// sigmoid gate: 874 us, 6.14 TB/s (0.91 of the measured copy rate); gradient of
// 32768 rows of 4096: 398 us, 5.39 TB/s (0.79). From 1264 and 887: registers that a launch
// bound of 1024 threads had cut to 64 (1103, 546), the ring (1058, 511), pairs of values an
// instruction and four sums in six shuffles (952, 504), the gate's form at compile
// time (898, 464), the operands' presence too, and zeros for groups past a row's end in
// place of branches (884, 401). Slower in the gradient: four groups a thread (581: eight
// warps an SM), one (1162: spills), fp32 pairs kept for raw bf16 (488).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "kernels.h"
#include "sm103.cuh"

namespace fcp {

using namespace dev;

namespace {

constexpr int kV = 8;  // values of a group: 16 bytes of bf16
constexpr int kMaxWarps = 32;

// Groups a thread holds. The forward: one up to 1024 values, two above (16384
// values: 1024 threads). The gradient, whose instructions a row and thread count
// for more: up to four.
__host__ __device__ constexpr int groups_of(int n, bool bwd) {
  return n <= 1024 ? 1 : bwd && n > 8192 ? 4 : 2;
}
__host__ __device__ constexpr int threads_of(int n, bool bwd) {
  return (n / kV + 32 * groups_of(n, bwd) - 1) / (32 * groups_of(n, bwd)) * 32;
}
// CTAs of the gradient at most (each writes a row of the weights' sums).
int most_ctas(int n) { return std::min(kResNormMaxCtas, 152 * 512 / threads_of(n, true)); }

// The arithmetic runs on pairs of values (f32x2): with one value an instruction
// its issue bound the kernels, not memory. A group is four pairs.
struct Pairs {
  uint64_t v[4];
};
__device__ __forceinline__ uint64_t both(float x) { return f2(x, x); }

// A group as it lies in memory: what a row's loads in flight take of the
// registers, and pairs of fp32 from there.
template <bool F32>
struct Raw {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* row, int i) {
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); ++j) v[j] = __ldcs(reinterpret_cast<const uint4*>(row) + (F32 ? 2 * i + j : i));
  }
  // The same by way of shared memory, `place` this thread's word among its
  // neighbours' (fp32: of two such runs of words). The two words of an fp32
  // group are fetched by two lanes of the warp, so that a warp's fetch covers whole
  // lines; i: the group, n: groups of a row.
  static __device__ __forceinline__ void fetch(uint4* place, const void* row, int i, int n) {
    const uint4* src = reinterpret_cast<const uint4*>(row) + i;
    if constexpr (F32) {
      const int lane = threadIdx.x & 31, block = (int)threadIdx.x - lane;
      src += i - lane;  // word 2 (i - lane) + lane
      place += block;   // words 2 block + lane and 32 on
      if (2 * i - lane < 2 * n) copy(place, src);
      if (2 * i - lane + 32 < 2 * n) copy(place + 32, src + 32);
    } else if (i < n) {
      copy(place, src);
    }
  }
  __device__ __forceinline__ void take(const uint4* place) {
    if constexpr (F32) {
      place += threadIdx.x;
      v[0] = place[0];
      v[1] = place[1];
    } else {
      v[0] = place[0];
    }
  }
  // Zeros in the place of a group past the row's end, which no fetch covers: such
  // threads compute with them and only do not store.
  static __device__ __forceinline__ void clear(uint4* place) {
    if constexpr (F32) {
      place += threadIdx.x;
      place[1] = make_uint4(0, 0, 0, 0);
    }
    place[0] = make_uint4(0, 0, 0, 0);
  }
  static __device__ __forceinline__ void copy(uint4* to, const uint4* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); ++j) v[j] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint64_t pair(int j) const {
    if constexpr (F32) {
      const uint4 q = v[j >> 1];
      return j & 1 ? f2(__uint_as_float(q.z), __uint_as_float(q.w)) : f2(__uint_as_float(q.x), __uint_as_float(q.y));
    } else {
      return unpack2(j == 0 ? v[0].x : j == 1 ? v[0].y : j == 2 ? v[0].z : v[0].w);
    }
  }
};
template <bool F32>
__device__ __forceinline__ void store8(void* row, int i, const Pairs& x) {
  if constexpr (F32) {
    float a[kV];
#pragma unroll
    for (int j = 0; j < 4; ++j) f2_split(x.v[j], a[2 * j], a[2 * j + 1]);
    __stcs(reinterpret_cast<float4*>(row) + 2 * i, make_float4(a[0], a[1], a[2], a[3]));
    __stcs(reinterpret_cast<float4*>(row) + 2 * i + 1, make_float4(a[4], a[5], a[6], a[7]));
  } else {
    __stcs(reinterpret_cast<uint4*>(row) + i, make_uint4(pack2(x.v[0]), pack2(x.v[1]), pack2(x.v[2]), pack2(x.v[3])));
  }
}
// Weights of group i (in L1 after a CTA's first row); ones without.
template <bool THERE = false>
__device__ __forceinline__ Pairs load_w(const void* w, bool f32, int i) {
  Pairs r;
  if (!THERE && !w) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = both(1.f);
  } else if (THERE || f32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w) + 2 * i), b = __ldg(reinterpret_cast<const float4*>(w) + 2 * i + 1);
    r.v[0] = f2(a.x, a.y), r.v[1] = f2(a.z, a.w), r.v[2] = f2(b.x, b.y), r.v[3] = f2(b.z, b.w);
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(w) + i);
    r.v[0] = unpack2(a.x), r.v[1] = unpack2(a.y), r.v[2] = unpack2(a.z), r.v[3] = unpack2(a.w);
  }
  return r;
}
__device__ __forceinline__ float sum_of(uint64_t a) {
  float lo, hi;
  f2_split(a, lo, hi);
  return lo + hi;
}

// Sums of one, or of four values at once, over the CTA's threads (every thread
// gets them). Four: after two exchanges a lane holds one of the values, so they
// take 6 shuffles, not 20. A half is not read any more when the call after the next
// one's values arrive there.
struct Sums {
  float4 four[2][kMaxWarps];
  float one[2][kMaxWarps];  // (zeros in the places of warps that there are not)
};
__device__ __forceinline__ void init(Sums& sh) {
  for (int i = threadIdx.x; i < 2 * kMaxWarps; i += blockDim.x) sh.one[i / kMaxWarps][i % kMaxWarps] = 0.f;
  __syncthreads();
}
__device__ __forceinline__ float shuffled(float v, int m) { return v + __shfl_xor_sync(0xffffffffu, v, m); }
__device__ __forceinline__ float row_sum(float v, Sums& sh, int& half) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v = shuffled(v, m);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  float* s = sh.one[half];
  half ^= 1;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < warps; w += 4) {
    const float4 a = *reinterpret_cast<const float4*>(s + w);
    v += (a.x + a.y) + (a.z + a.w);
  }
  return v;
}
__device__ __forceinline__ float4 row_sums(float4 v, Sums& sh, int& half) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1, second = lane & 2;
  // Even lanes keep the sums of x and y, odd ones those of z and w; then one each.
  const float a = (odd ? v.z : v.x) + __shfl_xor_sync(0xffffffffu, odd ? v.x : v.z, 1);
  const float b = (odd ? v.w : v.y) + __shfl_xor_sync(0xffffffffu, odd ? v.y : v.w, 1);
  float t = (second ? b : a) + __shfl_xor_sync(0xffffffffu, second ? a : b, 2);
#pragma unroll
  for (int m = 4; m < 32; m <<= 1) t = shuffled(t, m);
  const int warps = blockDim.x >> 5;
  if (warps == 1)  // lane 0 holds x's sum, 1 z's, 2 y's, 3 w's
    return make_float4(__shfl_sync(0xffffffffu, t, 0), __shfl_sync(0xffffffffu, t, 2), __shfl_sync(0xffffffffu, t, 1),
                       __shfl_sync(0xffffffffu, t, 3));
  float4* s = sh.four[half];
  half ^= 1;
  if (lane < 4) reinterpret_cast<float*>(s + (threadIdx.x >> 5))[(lane >> 1) | (lane & 1) << 1] = t;
  __syncthreads();
  float4 r = s[0];
  for (int w = 1; w < warps; ++w) {
    const float4 o = s[w];
    r = make_float4(r.x + o.x, r.y + o.y, r.z + o.z, r.w + o.w);
  }
  return r;
}

// g(z) and g'(z) = g (1 - g) for the sigmoid, as e g g, which keeps its bits where
// g is near 1; e is cut below infinity, where it would meet g = 0. (min.NaN: a
// NaN stays one.)
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
enum Gate { kNoGate, kPlainGate, kSigmoidGate };
template <Gate GATE>
__device__ __forceinline__ uint64_t gate_of(uint64_t z) {
  if constexpr (GATE != kSigmoidGate) return z;
  float a, b;
  f2_split(f2_mul(z, both(-1.4426950408889634f)), a, b);
  return f2(rcp(1.f + ex2(a)), rcp(1.f + ex2(b)));
}
template <Gate GATE>
__device__ __forceinline__ void gate_of(uint64_t z, uint64_t& g, uint64_t& dg) {
  if constexpr (GATE != kSigmoidGate) {
    g = z;
    dg = both(1.f);
  } else {
    float a, b;
    f2_split(f2_mul(z, both(-1.4426950408889634f)), a, b);
    asm("min.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(a));  // 126
    asm("min.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(b));
    const uint64_t e = f2(ex2(a), ex2(b));
    f2_split(f2_add(e, both(1.f)), a, b);
    g = f2(rcp(a), rcp(b));
    dg = f2_mul(f2_mul(e, g), g);
  }
}

__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The tokens of a CTA: units of the launch in steps of the grid. A unit is one
// token, or of a shard `unit_rows` rows of a chunk (a run of at most kResNormChunk
// rows): one, as rows have to spread over the SMs, or the whole chunk where chunks
// are short (documents of a few tokens), whose units would otherwise mostly be empty.
struct RowWalk {
  int64_t unit;
  int row, end;
  __device__ __forceinline__ RowWalk() : unit(blockIdx.x), row(0), end(0) {}
  // The next token, or -1.
  __device__ __forceinline__ int64_t next(const ResNormParams& p) {
    if (!p.chunks) {
      const int64_t t = unit;
      unit += gridDim.x;
      return t < p.units ? t : -1;
    }
    while (row >= end) {
      if (unit >= p.units) return -1;
      const int per = kResNormChunk / p.unit_rows, sub = (int)(unit % per) * p.unit_rows;
      const int32_t* c = p.chunks + 2 * (unit / per);
      const int first = __ldg(c), n = __ldg(c + 1);
      unit += gridDim.x;
      if constexpr (kDeviceChecks) {
        if (first < 0 || n < 0 || first > p.T - n) continue;
      }
      row = first + sub;
      end = first + min(n, sub + p.unit_rows);
    }
    return row++;
  }
};

__device__ __forceinline__ const char* at(const void* base, int64_t row_bytes, int64_t t) {
  return static_cast<const char*>(base) + row_bytes * t;
}
__device__ __forceinline__ char* at(void* base, int64_t row_bytes, int64_t t) {
  return static_cast<char*>(base) + row_bytes * t;
}

// A thread's groups of one row, c of them, `kWords` words of 16 bytes each, in a
// stage of the ring in shared memory; the words of neighbouring threads are
// neighbours. Only a warp's own lanes read what it fetched.
constexpr int kFwdWords[2] = {3, 4}, kBwdWords[2] = {5, 7};  // bf16, fp32 residual

template <int G, int THREADS, int CTAS, bool RING, bool F32, Gate GATE>
__global__ void __launch_bounds__(THREADS, CTAS) res_norm_kernel(const ResNormParams p) {
  extern __shared__ uint4 ring[];
  __shared__ __align__(16) Sums sh;
  init(sh);
  constexpr int kWords = kFwdWords[F32];
  const int step = blockDim.x;
  int half = 0, stage = 0;
  const float inv_n = 1.f / p.n;
  RowWalk walk;
  auto place = [&](int st, int c) { return ring + (st * G + c) * kWords * step + threadIdx.x; };
  auto fetch = [&](int st, int64_t t) {
    if constexpr (RING) {
#pragma unroll
      for (int c = 0; c < G; ++c) {
        const int i = threadIdx.x + c * step;
        if (t < 0) continue;
        uint4* at_c = place(st, c);
        if (p.y) Raw<false>::fetch(at_c, at(p.y, p.y_row, t), i, p.groups);
        if constexpr (GATE != kNoGate) Raw<false>::fetch(at_c + step, at(p.gate, p.gate_row, t), i, p.groups);
        Raw<F32>::fetch(at_c + 2 * step, at(p.x, p.x_row, t), i, p.groups);
      }
      async_commit();
    }
  };
  if constexpr (RING) {
    for (int c = 0; c < G; ++c)
      for (int st = 0; st < 2 && threadIdx.x + c * step >= p.groups; ++st) {
        Raw<false>::clear(place(st, c));
        Raw<false>::clear(place(st, c) + step);
        Raw<F32>::clear(place(st, c) + 2 * step);
      }
  }
  int64_t t = walk.next(p);
  fetch(0, t);
  for (int64_t next; t >= 0; t = next, stage ^= 1) {
    next = walk.next(p);
    if constexpr (RING && F32) __syncwarp();  // the lanes have read the last row
    fetch(stage ^ 1, next);
    Raw<F32> xr[G];
    Raw<false> yr[G], zr[G];
    if constexpr (RING) async_wait<1>();
    if constexpr (RING && F32) __syncwarp();
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * step;
      xr[c].zero(), yr[c].zero(), zr[c].zero();
      if (!RING && i >= p.groups) continue;
      if constexpr (RING) {
        const uint4* at_c = place(stage, c);
        if (p.y) yr[c].take(at_c);
        if constexpr (GATE != kNoGate) zr[c].take(at_c + step);
        xr[c].take(at_c + 2 * step);
      } else {
        if (p.y) yr[c].load(at(p.y, p.y_row, t), i);
        xr[c].load(at(p.x, p.x_row, t), i);
        if constexpr (GATE != kNoGate) zr[c].load(at(p.gate, p.gate_row, t), i);
      }
    }
    float ry = 1.f;
    if (p.y && p.post_norm) {
      uint64_t s2 = 0;
#pragma unroll
      for (int c = 0; c < G; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2 = f2_fma(yr[c].pair(j), yr[c].pair(j), s2);
      ry = rsqrtf(row_sum(sum_of(s2), sh, half) * inv_n + p.eps);
    }
    const uint64_t a2 = both(p.res_scale), b2 = both(p.branch_scale * ry);
    uint64_t s2 = 0;
    Pairs x[G];
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * step;
      const bool there = i < p.groups;
      if (p.y) {
        const Pairs w = load_w(p.w_post, p.w_f32, there ? i : 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint64_t u = f2_mul(f2_mul(yr[c].pair(j), b2), w.v[j]);
          if constexpr (GATE != kNoGate) u = f2_mul(u, gate_of<GATE>(zr[c].pair(j)));
          x[c].v[j] = f2_fma(xr[c].pair(j), a2, u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[c].v[j] = f2_mul(xr[c].pair(j), a2);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = f2_fma(x[c].v[j], x[c].v[j], s2);
      if (p.x_out && there) store8<F32>(at(p.x_out, p.x_out_row, t), i, x[c]);
    }
    if (!p.h) continue;
    const uint64_t r2 = both(rsqrtf(row_sum(sum_of(s2), sh, half) * inv_n + p.eps));
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * step;
      const bool there = i < p.groups;
      Pairs w = load_w(p.w_pre, p.w_f32, there ? i : 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) w.v[j] = f2_mul(f2_mul(x[c].v[j], r2), w.v[j]);
      if (there) store8<false>(at(p.h, p.h_row, t), i, w);
    }
  }
}

// FULL: every operand but the gate is there and the weights are fp32, as in nearly
// every call of a stack of layers: no branch for each group and operand.
template <int G, int THREADS, int CTAS, bool RING, bool F32, Gate GATE, bool FULL>
__global__ void __launch_bounds__(THREADS, CTAS) res_norm_bwd_kernel(const ResNormParams p) {
  extern __shared__ uint4 ring[];
  __shared__ __align__(16) Sums sh;
  init(sh);
  constexpr int kWords = kBwdWords[F32], kRes = F32 ? 2 : 1;
  const int step = blockDim.x;
  int half = 0, half4 = 0, stage = 0;
  const float inv_n = 1.f / p.n;
  Pairs acc_pre[G], acc_post[G];
#pragma unroll
  for (int c = 0; c < G; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc_pre[c].v[j] = acc_post[c].v[j] = 0;
  RowWalk walk;
  auto place = [&](int st, int c) { return ring + (st * G + c) * kWords * step + threadIdx.x; };
  auto fetch = [&](int st, int64_t t) {
    if constexpr (RING) {
#pragma unroll
      for (int c = 0; c < G; ++c) {
        const int i = threadIdx.x + c * step;
        if (t < 0) continue;
        uint4* at_c = place(st, c);
        if (FULL || p.dh) {
          Raw<false>::fetch(at_c, at(p.dh, p.dh_row, t), i, p.groups);
          Raw<F32>::fetch(at_c + 3 * step, at(p.x, p.x_row, t), i, p.groups);
        }
        if (FULL || p.y) Raw<false>::fetch(at_c + step, at(p.y, p.y_row, t), i, p.groups);
        if constexpr (GATE != kNoGate) Raw<false>::fetch(at_c + 2 * step, at(p.gate, p.gate_row, t), i, p.groups);
        if (FULL || p.dx_out) Raw<F32>::fetch(at_c + (3 + kRes) * step, at(p.dx_out, p.dx_out_row, t), i, p.groups);
      }
      async_commit();
    }
  };
  if constexpr (RING) {
    for (int c = 0; c < G; ++c)
      for (int st = 0; st < 2 && threadIdx.x + c * step >= p.groups; ++st) {
        for (int a = 0; a < 3; ++a) Raw<false>::clear(place(st, c) + a * step);
        for (int a = 0; a < 2; ++a) Raw<F32>::clear(place(st, c) + (3 + a * kRes) * step);
      }
  }
  int64_t t = walk.next(p);
  fetch(0, t);
  for (int64_t next; t >= 0; t = next, stage ^= 1) {
    next = walk.next(p);
    if constexpr (RING && F32) __syncwarp();  // the lanes have read the last row
    fetch(stage ^ 1, next);
    Raw<F32> xr[G], dr[G];
    Raw<false> hr[G], yr[G], zr[G];
    if constexpr (RING) async_wait<1>();
    if constexpr (RING && F32) __syncwarp();
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * step;
      xr[c].zero(), hr[c].zero(), yr[c].zero(), dr[c].zero(), zr[c].zero();
      if (!RING && i >= p.groups) continue;
      if constexpr (RING) {
        const uint4* at_c = place(stage, c);
        if (FULL || p.dh) {
          hr[c].take(at_c);
          xr[c].take(at_c + 3 * step);
        }
        if (FULL || p.y) yr[c].take(at_c + step);
      } else {
        if (FULL || p.dh) {
          xr[c].load(at(p.x, p.x_row, t), i);
          hr[c].load(at(p.dh, p.dh_row, t), i);
        }
        if (FULL || p.y) yr[c].load(at(p.y, p.y_row, t), i);
        if (FULL || p.dx_out) dr[c].load(at(p.dx_out, p.dx_out_row, t), i);
        if constexpr (GATE != kNoGate) zr[c].load(at(p.gate, p.gate_row, t), i);
      }
    }
    uint64_t xx = 0, kx = 0, yy = 0;
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * step;
      const Pairs w = load_w<FULL>(p.w_pre, p.w_f32, i < p.groups ? i : 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t x = xr[c].pair(j), y = yr[c].pair(j);
        xx = f2_fma(x, x, xx);
        kx = f2_fma(f2_mul(hr[c].pair(j), x), w.v[j], kx);
        yy = f2_fma(y, y, yy);
      }
    }
    const float4 sums = row_sums(make_float4(sum_of(xx), sum_of(kx), sum_of(yy), 0.f), sh, half4);
    const float r = FULL || p.dh ? rsqrtf(sums.x * inv_n + p.eps) : 0.f;
    const float ry = p.post_norm ? rsqrtf(sums.z * inv_n + p.eps) : 1.f;
    const uint64_t r2 = both(r), nm2 = both(-r * (r * r * (sums.y * inv_n))), ry2 = both(ry);
    uint64_t ey = 0;
    Pairs ee[G];  // e
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * step;
      const bool there = i < p.groups;
      Pairs w = load_w<FULL>(p.w_pre, p.w_f32, there ? i : 0), out;
      if constexpr (RING) {  // what the sums did not need stayed in shared memory till now
        const uint4* at_c = place(stage, c);
        if constexpr (GATE != kNoGate) zr[c].take(at_c + 2 * step);
        if (FULL || p.dx_out) dr[c].take(at_c + (3 + kRes) * step);
      }
      Pairs d;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t x = xr[c].pair(j), h = hr[c].pair(j);
        acc_pre[c].v[j] = f2_fma(f2_mul(h, x), r2, acc_pre[c].v[j]);
        d.v[j] = f2_fma(x, nm2, f2_fma(f2_mul(h, w.v[j]), r2, dr[c].pair(j)));
        out.v[j] = f2_mul(d.v[j], both(p.res_scale));
      }
      if (there) store8<F32>(at(p.dx, p.dx_row, t), i, out);
      if (!FULL && !p.y) continue;
      w = load_w<FULL>(p.w_post, p.w_f32, there ? i : 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint64_t g = both(1.f), dg = 0;
        if constexpr (GATE != kNoGate) gate_of<GATE>(zr[c].pair(j), g, dg);
        const uint64_t y = yr[c].pair(j), cd = f2_mul(d.v[j], both(p.branch_scale)), cu = f2_mul(cd, f2_mul(y, ry2));
        if constexpr (GATE != kNoGate) out.v[j] = f2_mul(f2_mul(cu, w.v[j]), dg);
        acc_post[c].v[j] = f2_fma(cu, g, acc_post[c].v[j]);
        ee[c].v[j] = f2_mul(f2_mul(cd, w.v[j]), g);
        ey = f2_fma(ee[c].v[j], y, ey);
      }
      if constexpr (GATE != kNoGate)
        if (there) store8<false>(at(p.dgate, p.dgate_row, t), i, out);
    }
    if (!FULL && !p.y) continue;
    const float my = p.post_norm ? ry * (ry * ry * (row_sum(sum_of(ey), sh, half) * inv_n)) : 0.f;
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = threadIdx.x + c * step;
#pragma unroll
      for (int j = 0; j < 4; ++j) ee[c].v[j] = f2_fma(yr[c].pair(j), both(-my), f2_mul(ee[c].v[j], ry2));
      if (i < p.groups) store8<false>(at(p.dy, p.dy_row, t), i, ee[c]);
    }
  }
  float* part = p.partial + (size_t)blockIdx.x * 2 * p.n;
#pragma unroll
  for (int c = 0; c < G; ++c) {
    const int i = threadIdx.x + c * step;
    if (i >= p.groups) continue;
    if (p.dw_post) store8<true>(part, i, acc_post[c]);
    if (p.dw_pre) store8<true>(part + p.n, i, acc_pre[c]);
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

// Starts the kernel; its CTAs, or 0 for an error.
template <class Kernel>
static int start(Kernel kernel, int bytes, int ctas, int most, int threads, const ResNormParams& p, cudaStream_t st) {
  if (bytes > 40 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return 0;
  // As many CTAs as are resident at once: by registers, by shared memory, and 32 an SM.
  const int fit = std::max(1, std::min({ctas, 227 * 1024 / (bytes + 2048), 32}));
  const int grid = (int)std::min({p.units, (int64_t)fit * p.num_sms, (int64_t)most});
  kernel<<<grid, threads, bytes, st>>>(p);
  return grid;
}
// Rows that do not fit the shared memory twice come straight from memory (RING
// false): more than 8192 values.
template <int G, int THREADS, int CTAS, bool RING, bool F32, Gate GATE, bool BWD>
static int start(const ResNormParams& p, cudaStream_t st) {
  const int threads = threads_of(p.n, BWD), ctas = CTAS * THREADS / threads;
  const int bytes = RING ? 2 * G * (BWD ? kBwdWords : kFwdWords)[F32] * threads * 16 : 0;
  if constexpr (BWD) {
    const bool full = p.dh && p.y && p.dx_out && p.w_pre && p.w_post && p.w_f32;
    if constexpr (!RING) return start(res_norm_bwd_kernel<G, THREADS, CTAS, RING, F32, GATE, false>, bytes, ctas, most_ctas(p.n), threads, p, st);
    else return full ? start(res_norm_bwd_kernel<G, THREADS, CTAS, RING, F32, GATE, true>, bytes, ctas, most_ctas(p.n), threads, p, st)
                : start(res_norm_bwd_kernel<G, THREADS, CTAS, RING, F32, GATE, false>, bytes, ctas, most_ctas(p.n), threads, p, st);
  }
  else return start(res_norm_kernel<G, THREADS, CTAS, RING, F32, GATE>, bytes, ctas, INT_MAX, threads, p, st);
}
template <int G, int THREADS, int CTAS, bool RING, bool BWD>
static int start(const ResNormParams& p, cudaStream_t st) {
  auto gated = [&](auto f32) {
    constexpr bool kF32 = decltype(f32)::value;
    if (!p.gate) return start<G, THREADS, CTAS, RING, kF32, kNoGate, BWD>(p, st);
    return p.gate_fn == FCP_GATE_SIGMOID ? start<G, THREADS, CTAS, RING, kF32, kSigmoidGate, BWD>(p, st)
                                         : start<G, THREADS, CTAS, RING, kF32, kPlainGate, BWD>(p, st);
  };
  return p.res_f32 ? gated(std::true_type()) : gated(std::false_type());
}

int launch_res_norm(const ResNormParams& a, cudaStream_t st) {
  ResNormParams p = a;
  p.groups = p.n / kV;
  int grid = 0;
  if (p.units > 0) {
    if (p.dx)
      grid = p.n <= 1024   ? start<1, 128, 5, true, true>(p, st)
             : p.n <= 2048 ? start<2, 128, 4, true, true>(p, st)
             : p.n <= 4096 ? start<2, 256, 2, true, true>(p, st)
             : p.n <= 8192 ? start<2, 512, 1, true, true>(p, st)
                           : start<4, 512, 1, false, true>(p, st);
    else
      grid = p.n <= 1024   ? start<1, 128, 8, true, false>(p, st)
             : p.n <= 4096 ? start<2, 256, 4, true, false>(p, st)
             : p.n <= 8192 ? start<2, 512, 2, true, false>(p, st)
                           : start<2, 1024, 1, false, false>(p, st);
    if (grid == 0) return FCP_ERR_CUDA;
  }
  // (A shard without tokens: no rows, whose sum is written as zero.)
  if (p.dx && (p.dw_post || p.dw_pre))
    res_norm_dw_kernel<<<dim3((p.n + 31) / 32, 2), 32 * kSumWarps, 0, st>>>(p.partial, grid, p.n, p.dw_post, p.dw_pre,
                                                                          p.add_dw);
  return cudaGetLastError() == cudaSuccess ? FCP_OK : FCP_ERR_CUDA;
}

}  // namespace fcp
