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
// sigmoid gate: 849 us, 6.32 TB/s (0.93 of the measured copy rate); gradient of
// 32768 rows of 4096: 385 us, 5.58 TB/s (0.82; with an fp32 residual 470 us, 6.28
// TB/s). From 1264 and 887: registers that a launch bound of 1024 threads had cut to
// 64 (1103, 546), the ring (1058, 511), pairs of values an instruction and four sums
// in six shuffles (952, 504), the gate's form at compile time (898, 464), the
// operands' presence too, and zeros for groups past a row's end in place of branches
// (884, 401), shared memory for a CTA's own number of warps (849, 385; fp32 585 to
// 470, two CTAs an SM). Slower in the gradient: four groups a thread (581: eight
// warps an SM), one (1162: spills), fp32 pairs kept for raw bf16 (488).
//
// Share of the copy rate by width (2^27 values, every operand, fp32 weights; residual bf16 / fp32):
//   n         64        128       256       768       1024      2048      4096      5120
//   forward   0.24/0.34 0.48/0.66 0.90/0.84 0.78/0.92 0.83/0.89 0.93/0.96 0.92/0.95 0.91/0.93
//   gradient  0.19/0.26 0.38/0.49 0.71/0.79 0.75/0.85 0.80/0.86 0.86/0.92 0.82/0.92 0.62/0.72
//   n         6144      7168      8192      8200      9216      12288     16384
//   forward   0.85/0.94 0.86/0.95 0.89/0.87 0.61/0.72 0.75/0.85 0.76/0.89 0.75/0.85
//   gradient  0.65/0.75 0.65/0.76 0.68/0.74 0.33/0.42 0.40/0.51 0.49/0.56 0.52/0.58
// Below 256 values a part of the one warp's lanes hold none. The gradient of 4097 to 8191 values
// has one CTA an SM, of 9 to 16 warps, which all wait at a row's two barriers (5120: ten
// warps, 35% of the issue slots used). A width just above a step of the CTA's size leaves
// lanes empty (2056: forward 0.72, gradient 0.65; 4104: 0.73, 0.50), and rows that are not
// whole lines of 128 bytes cost a tenth beside a neighbour with as many warps (5000 for 5120:
// gradient 0.53 for 0.62; 8200 for 8256: forward 0.61 for 0.69, gradient 0.33 for 0.35).
//
// Rows of more than 8192 values. Forward: the ring where it fits the shared memory,
// else the next row is fetched into L2 (16384 rows of 16384: bf16 566 to 510 us, fp32
// 820 to 624; of 9216 396 to 298, 448 to 364). Gradient: a row on two CTAs of a
// cluster, which exchange their sums by each other's shared memory, where one CTA
// had four groups a thread and no ring: 16384 rows of 16384 1392 to 1202 us, fp32 1806 to
// 1461; of 9216 929 to 898, 1066 to 966; 32768 rows of 8200 1795 to 1926, 2111 to 2054 (the
// pair loses 7% in bf16 there). A pair takes 4.5 us for a row of 8200, 4.2 of 9216 and
// 5.6 of 16384: the two cluster barriers of a row, whose release waits for the row's stores,
// not the bytes (of a warp's stalls the barriers have most: membar 1.9, barrier 0.7 an
// issue; DRAM reads are the algorithmic ones at 8200 too). Clusters of more and smaller
// CTAs, two an SM, were slower (1936 us).
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

// A thread holds one group up to 1024 values, two above (the forward's 16384:
// 1024 threads). The gradient takes a row of more than 8192 values by a cluster of
// two CTAs, half a row each: its registers do not suffice for 1024 threads.
constexpr bool paired(int n, bool bwd) { return bwd && n > 8192; }
constexpr int threads_of(int n, bool bwd) {
  const int groups = paired(n, bwd) ? (n / kV + 1) / 2 : n / kV, per = n <= 1024 ? 32 : 64;
  return (groups + per - 1) / per * 32;
}
// CTAs, or pairs of them, of the gradient at most (each writes a row of the weights' sums).
int most_sums(int n) { return std::min(kResNormMaxCtas, 152 * 512 / threads_of(n, true) / (paired(n, true) ? 2 : 1)); }

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
  // Into L2 by one lane a line.
  static __device__ __forceinline__ void ahead(const void* row, int i) {
    const char* line = static_cast<const char*>(row) + (F32 ? 32 : 16) * (int64_t)i;
    if (!(threadIdx.x & (F32 ? 3 : 7))) asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
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
// What is known at compile time of a call: nothing, or that every operand but the
// gate is there and which type the weights have.
enum Full { kAny, kFullF32, kFullBf16 };

// Weights of group i (in L1 after a CTA's first row); ones without.
template <Full FULL = kAny>
__device__ __forceinline__ Pairs load_w(const void* w, bool f32, int i) {
  Pairs r;
  if (FULL == kAny && !w) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = both(1.f);
  } else if (FULL == kFullF32 || (FULL == kAny && f32)) {
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

// Sums of one, or of four values at once, over the threads of the CTA or of the
// pair of CTAs (every thread gets them). Four: after two exchanges a lane holds
// one of the values, so they take 6 shuffles, not 20. A half is not read any more
// when the call after the next one's values arrive there. In whole lines of 128
// bytes, so that the ring behind them starts on one (else 4 to 6% slower), and for
// the CTA's own number of warps: only then two CTAs with rings of 4096 values and
// an fp32 residual fit an SM (585 to 470 us).
template <int WARPS>
struct alignas(128) Sums {
  float4 four[2][WARPS];
  float one[2][WARPS];  // (zeros in the places of warps that there are not)
};
template <int WARPS>
__device__ __forceinline__ void init(Sums<WARPS>& sh) {
  for (int i = threadIdx.x; i < 2 * WARPS; i += blockDim.x) sh.one[i / WARPS][i % WARPS] = 0.f;
  __syncthreads();
}
// A pair's warps write into both CTAs' shared memory, so each CTA reads its own.
__device__ __forceinline__ uint32_t pair_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
template <bool PAIR>
__device__ __forceinline__ void put(float* to, float v) {
  *to = v;
  if constexpr (PAIR) {
    uint32_t other;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(other) : "r"(smem_u32(to)), "r"(pair_rank() ^ 1));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(other), "f"(v) : "memory");
  }
}
template <bool PAIR>
__device__ __forceinline__ void sync_all() {
  if constexpr (PAIR)
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  else
    __syncthreads();
}
__device__ __forceinline__ float shuffled(float v, int m) { return v + __shfl_xor_sync(0xffffffffu, v, m); }
template <bool PAIR, int WARPS>
__device__ __forceinline__ float row_sum(float v, Sums<WARPS>& sh, int& half) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v = shuffled(v, m);
  int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  if (!PAIR && warps == 1) return v;
  if constexpr (PAIR) {
    if (pair_rank()) warp += warps;
    warps *= 2;
  }
  float* s = sh.one[half];
  half ^= 1;
  if ((threadIdx.x & 31) == 0) put<PAIR>(s + warp, v);
  sync_all<PAIR>();
  v = 0.f;
  for (int w = 0; w < warps; w += 4) {
    const float4 a = *reinterpret_cast<const float4*>(s + w);
    v += (a.x + a.y) + (a.z + a.w);
  }
  return v;
}
template <bool PAIR, int WARPS>
__device__ __forceinline__ float4 row_sums(float4 v, Sums<WARPS>& sh, int& half) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1, second = lane & 2;
  // Even lanes keep the sums of x and y, odd ones those of z and w; then one each.
  const float a = (odd ? v.z : v.x) + __shfl_xor_sync(0xffffffffu, odd ? v.x : v.z, 1);
  const float b = (odd ? v.w : v.y) + __shfl_xor_sync(0xffffffffu, odd ? v.y : v.w, 1);
  float t = (second ? b : a) + __shfl_xor_sync(0xffffffffu, second ? a : b, 2);
#pragma unroll
  for (int m = 4; m < 32; m <<= 1) t = shuffled(t, m);
  int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  if (!PAIR && warps == 1)  // lane 0 holds x's sum, 1 z's, 2 y's, 3 w's
    return make_float4(__shfl_sync(0xffffffffu, t, 0), __shfl_sync(0xffffffffu, t, 2), __shfl_sync(0xffffffffu, t, 1),
                       __shfl_sync(0xffffffffu, t, 3));
  if constexpr (PAIR) {
    if (pair_rank()) warp += warps;
    warps *= 2;
  }
  float4* s = sh.four[half];
  half ^= 1;
  if (lane < 4) put<PAIR>(reinterpret_cast<float*>(s + warp) + ((lane >> 1) | (lane & 1) << 1), t);
  sync_all<PAIR>();
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

// The tokens of a CTA (or pair): units of the launch in steps of the grid. A unit is one
// token, or of a shard `unit_rows` rows of a chunk (a run of at most kResNormChunk
// rows): one, as rows have to spread over the SMs, or the whole chunk where chunks
// are short (documents of a few tokens), whose units would otherwise mostly be empty.
template <int PER = 1>
struct RowWalk {
  int64_t unit;
  int row, end;
  __device__ __forceinline__ RowWalk() : unit(blockIdx.x / PER), row(0), end(0) {}
  // The next token, or -1.
  __device__ __forceinline__ int64_t next(const ResNormParams& p) {
    if (!p.chunks) {
      const int64_t t = unit;
      unit += gridDim.x / PER;
      return t < p.units ? t : -1;
    }
    while (row >= end) {
      if (unit >= p.units) return -1;
      const int per = kResNormChunk / p.unit_rows, sub = (int)(unit % per) * p.unit_rows;
      const int32_t* c = p.chunks + 2 * (unit / per);
      const int first = __ldg(c), n = __ldg(c + 1);
      unit += gridDim.x / PER;
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
  __shared__ Sums<THREADS / 32> sh;
  init(sh);
  constexpr int kWords = kFwdWords[F32];
  const int step = blockDim.x;
  int half = 0, stage = 0;
  const float inv_n = 1.f / p.n;
  RowWalk<> walk;
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
    } else if (t >= 0) {
#pragma unroll
      for (int c = 0; c < G; ++c) {
        const int i = threadIdx.x + c * step;
        if (i >= p.groups) continue;
        if (p.y) Raw<false>::ahead(at(p.y, p.y_row, t), i);
        if constexpr (GATE != kNoGate) Raw<false>::ahead(at(p.gate, p.gate_row, t), i);
        Raw<F32>::ahead(at(p.x, p.x_row, t), i);
      }
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
      ry = rsqrtf(row_sum<false>(sum_of(s2), sh, half) * inv_n + p.eps);
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
    const uint64_t r2 = both(rsqrtf(row_sum<false>(sum_of(s2), sh, half) * inv_n + p.eps));
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

// FULL, as in nearly every call of a stack of layers: no branch for each group and
// operand (32768 rows of 4096: 386 us for 429 with fp32 weights, 375 for 409 with bf16;
// one variant for both types of weights: 425 and 403).
// PAIR: a row's first groups on one CTA of a cluster, the rest on the other.
template <int G, int THREADS, int CTAS, bool PAIR, bool F32, Gate GATE, Full FULL>
__global__ void __launch_bounds__(THREADS, CTAS) res_norm_bwd_kernel(const ResNormParams p) {
  extern __shared__ uint4 ring[];
  __shared__ Sums<THREADS / 32 * (PAIR ? 2 : 1)> sh;
  init(sh);
  if constexpr (PAIR) sync_all<true>();  // the other CTA is there, its zeros too
  constexpr int kWords = kBwdWords[F32], kRes = F32 ? 2 : 1;
  const int step = blockDim.x, share = (p.groups + 1) / 2;
  const int first = PAIR ? (int)pair_rank() * share : 0, last = PAIR ? min(p.groups, first + share) : p.groups;  // this CTA's groups
  int half = 0, half4 = 0, stage = 0;
  const float inv_n = 1.f / p.n;
  Pairs acc_pre[G], acc_post[G];
#pragma unroll
  for (int c = 0; c < G; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc_pre[c].v[j] = acc_post[c].v[j] = 0;
  RowWalk<PAIR ? 2 : 1> walk;
  auto place = [&](int st, int c) { return ring + (st * G + c) * kWords * step + threadIdx.x; };
  auto fetch = [&](int st, int64_t t) {
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = first + threadIdx.x + c * step;
      if (t < 0) continue;
      uint4* at_c = place(st, c);
      if (FULL || p.dh) {
        Raw<false>::fetch(at_c, at(p.dh, p.dh_row, t), i, last);
        Raw<F32>::fetch(at_c + 3 * step, at(p.x, p.x_row, t), i, last);
      }
      if (FULL || p.y) Raw<false>::fetch(at_c + step, at(p.y, p.y_row, t), i, last);
      if constexpr (GATE != kNoGate) Raw<false>::fetch(at_c + 2 * step, at(p.gate, p.gate_row, t), i, last);
      if (FULL || p.dx_out) Raw<F32>::fetch(at_c + (3 + kRes) * step, at(p.dx_out, p.dx_out_row, t), i, last);
    }
    async_commit();
  };
  for (int c = 0; c < G; ++c)
    for (int st = 0; st < 2 && first + (int)threadIdx.x + c * step >= last; ++st) {
      for (int a = 0; a < 3; ++a) Raw<false>::clear(place(st, c) + a * step);
      for (int a = 0; a < 2; ++a) Raw<F32>::clear(place(st, c) + (3 + a * kRes) * step);
    }
  int64_t t = walk.next(p);
  fetch(0, t);
  for (int64_t next; t >= 0; t = next, stage ^= 1) {
    next = walk.next(p);
    if constexpr (F32) __syncwarp();  // the lanes have read the last row
    fetch(stage ^ 1, next);
    Raw<F32> xr[G], dr[G];
    Raw<false> hr[G], yr[G], zr[G];
    async_wait<1>();
    if constexpr (F32) __syncwarp();
#pragma unroll
    for (int c = 0; c < G; ++c) {
      xr[c].zero(), hr[c].zero(), yr[c].zero(), dr[c].zero(), zr[c].zero();
      const uint4* at_c = place(stage, c);
      if (FULL || p.dh) {
        hr[c].take(at_c);
        xr[c].take(at_c + 3 * step);
      }
      if (FULL || p.y) yr[c].take(at_c + step);
    }
    uint64_t xx = 0, kx = 0, yy = 0;
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = first + threadIdx.x + c * step;
      const Pairs w = load_w<FULL>(p.w_pre, p.w_f32, i < last ? i : 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t x = xr[c].pair(j), y = yr[c].pair(j);
        xx = f2_fma(x, x, xx);
        kx = f2_fma(f2_mul(hr[c].pair(j), x), w.v[j], kx);
        yy = f2_fma(y, y, yy);
      }
    }
    const float4 sums = row_sums<PAIR>(make_float4(sum_of(xx), sum_of(kx), sum_of(yy), 0.f), sh, half4);
    const float r = FULL || p.dh ? rsqrtf(sums.x * inv_n + p.eps) : 0.f;
    const float ry = p.post_norm ? rsqrtf(sums.z * inv_n + p.eps) : 1.f;
    const uint64_t r2 = both(r), nm2 = both(-r * (r * r * (sums.y * inv_n))), ry2 = both(ry);
    uint64_t ey = 0;
    Pairs ee[G];  // e
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = first + threadIdx.x + c * step;
      const bool there = i < last;
      Pairs w = load_w<FULL>(p.w_pre, p.w_f32, there ? i : 0), out;
      const uint4* at_c = place(stage, c);  // what the sums did not need stayed in shared memory till now
      if constexpr (GATE != kNoGate) zr[c].take(at_c + 2 * step);
      if (FULL || p.dx_out) dr[c].take(at_c + (3 + kRes) * step);
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
    const float my = p.post_norm ? ry * (ry * ry * (row_sum<PAIR>(sum_of(ey), sh, half) * inv_n)) : 0.f;
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int i = first + threadIdx.x + c * step;
#pragma unroll
      for (int j = 0; j < 4; ++j) ee[c].v[j] = f2_fma(yr[c].pair(j), both(-my), f2_mul(ee[c].v[j], ry2));
      if (i < last) store8<false>(at(p.dy, p.dy_row, t), i, ee[c]);
    }
  }
  float* part = p.partial + (size_t)(blockIdx.x / (PAIR ? 2 : 1)) * 2 * p.n;
#pragma unroll
  for (int c = 0; c < G; ++c) {
    const int i = first + threadIdx.x + c * step;
    if (i >= last) continue;
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

int64_t res_norm_ws_bytes(int n) { return (int64_t)most_sums(n) * 2 * n * sizeof(float); }

// Starts the kernel with CTAs, or clusters of `per`, up to `most`; their number, or 0
// for an error.
template <class Kernel>
static int start(Kernel kernel, int bytes, int sums, int ctas, int most, int threads, int per, const ResNormParams& p, cudaStream_t st) {
  if (bytes > 40 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return 0;
  // As many CTAs as are resident at once: by registers, by shared memory, and 32 an SM.
  const int fit = std::max(1, std::min({ctas, 228 * 1024 / (bytes + sums + 1024), 32}));
  const int grid = (int)std::min({p.units, std::max((int64_t)fit * p.num_sms / per, (int64_t)1), (int64_t)most});
  if (per == 1) {
    kernel<<<grid, threads, bytes, st>>>(p);
    return grid;
  }
  cudaLaunchConfig_t config = {};
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim = {(unsigned)per, 1, 1};
  config.gridDim = dim3(grid * per);
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = bytes;
  config.stream = st;
  config.attrs = &cluster;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, p) == cudaSuccess ? grid : 0;
}
template <int G, int THREADS, int CTAS, bool RING, bool F32, Gate GATE>
static int start_fwd(const ResNormParams& p, int ring, cudaStream_t st) {
  const int threads = threads_of(p.n, false), ctas = CTAS * THREADS / threads;
  return start(res_norm_kernel<G, THREADS, CTAS, RING, F32, GATE>, RING ? ring : 0, sizeof(Sums<THREADS / 32>), ctas, INT_MAX, threads, 1, p, st);
}
template <int G, int THREADS, int CTAS, bool F32, Gate GATE>
static int start_fwd(const ResNormParams& p, cudaStream_t st) {
  const int ring = 2 * G * kFwdWords[F32] * threads_of(p.n, false) * 16;
  // (Two stages of fp32 rows of more than 14336 values are too large; of bf16 ones none are.)
  static_assert(2 * G * kFwdWords[0] * THREADS * 16 <= 224 * 1024, "a ring that does not fit");
  if constexpr (THREADS == 1024 && F32)
    if (ring > 224 * 1024) return start_fwd<G, THREADS, CTAS, false, F32, GATE>(p, ring, st);
  return start_fwd<G, THREADS, CTAS, true, F32, GATE>(p, ring, st);
}
template <int G, int THREADS, int CTAS, bool PAIR, bool F32, Gate GATE>
static int start_bwd(const ResNormParams& p, cudaStream_t st) {
  const int threads = threads_of(p.n, true), ctas = CTAS * THREADS / threads, bytes = 2 * G * kBwdWords[F32] * threads * 16;
  auto go = [&](auto kernel) { return start(kernel, bytes, sizeof(Sums<THREADS / 32 * (PAIR ? 2 : 1)>), ctas, most_sums(p.n), threads, PAIR ? 2 : 1, p, st); };
  if (!(p.dh && p.y && p.dx_out && p.w_pre && p.w_post)) return go(res_norm_bwd_kernel<G, THREADS, CTAS, PAIR, F32, GATE, kAny>);
  return p.w_f32 ? go(res_norm_bwd_kernel<G, THREADS, CTAS, PAIR, F32, GATE, kFullF32>)
                 : go(res_norm_bwd_kernel<G, THREADS, CTAS, PAIR, F32, GATE, kFullBf16>);
}
// The variant for the residual's type and the gate.
template <int G, int THREADS, int CTAS, bool BWD, bool PAIR = false>
static int start(const ResNormParams& p, cudaStream_t st) {
  auto one = [&](auto f32, auto gate) {
    if constexpr (BWD) return start_bwd<G, THREADS, CTAS, PAIR, decltype(f32)::value, decltype(gate)::value>(p, st);
    else return start_fwd<G, THREADS, CTAS, decltype(f32)::value, decltype(gate)::value>(p, st);
  };
  auto gated = [&](auto f32) {
    if (!p.gate) return one(f32, std::integral_constant<Gate, kNoGate>());
    return p.gate_fn == FCP_GATE_SIGMOID ? one(f32, std::integral_constant<Gate, kSigmoidGate>())
                                         : one(f32, std::integral_constant<Gate, kPlainGate>());
  };
  return p.res_f32 ? gated(std::true_type()) : gated(std::false_type());
}

int launch_res_norm(const ResNormParams& a, cudaStream_t st) {
  ResNormParams p = a;
  p.groups = p.n / kV;
  int grid = 0;
  if (p.units > 0) {
    if (p.dx)
      grid = p.n <= 1024   ? start<1, 128, 5, true>(p, st)
             : p.n <= 2048 ? start<2, 128, 4, true>(p, st)
             : p.n <= 4096 ? start<2, 256, 2, true>(p, st)
             : p.n <= 8192 ? start<2, 512, 1, true>(p, st)
                           : start<2, 512, 1, true, true>(p, st);
    else
      grid = p.n <= 1024   ? start<1, 128, 8, false>(p, st)
             : p.n <= 4096 ? start<2, 256, 4, false>(p, st)
             : p.n <= 8192 ? start<2, 512, 2, false>(p, st)
                           : start<2, 1024, 1, false>(p, st);
    if (grid == 0) return FCP_ERR_CUDA;
  }
  // (A shard without tokens: no rows, whose sum is written as zero.)
  if (p.dx && (p.dw_post || p.dw_pre))
    res_norm_dw_kernel<<<dim3((p.n + 31) / 32, 2), 32 * kSumWarps, 0, st>>>(p.partial, grid, p.n, p.dw_post, p.dw_pre,
                                                                          p.add_dw);
  return cudaGetLastError() == cudaSuccess ? FCP_OK : FCP_ERR_CUDA;
}

}  // namespace fcp
