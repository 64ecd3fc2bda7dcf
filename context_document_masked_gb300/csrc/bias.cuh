// Device helpers of the bucketed distance bias, shared by the attention
// forward and backward.
//
// The scores of a tile are a Toeplitz matrix of biases: element (row, column)
// depends on the distance alone, so 32 rows x 128 columns have 159 distances.
// Far from the diagonal all of a warp's tile falls into one bucket and its
// bias is one number, added where the softmax subtracts its maximum. The
// others add a window of biases by distance, kept in shared memory. Window
// entries are the bias over the softmax scale, added to the raw scores.
//
// The straight-line code that a tile takes matters more here than its
// operations: shuffles from a window kept in registers (five instructions an
// element, 10 KB of code) left the warps waiting for instructions and took
// 2.05 ms against the plain forward's 1.48 ms on the 32K workload, and 1.6 ms
// against 0.8 ms on one document of 16K (16 query and 2 KV heads of 128, 64
// buckets). Through shared memory: 1.57 and 1.01 ms; the eight warps read
// a tile's windows in 1,024 cycles, half as many as its products take.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "kernels.h"
#include "sm103.cuh"

namespace fcp {
namespace dev {

constexpr float kLog2e = 1.4426950408889634f;
// A bias at or below this masks its bucket. Scores near it are 2^-4 apart in
// fp32: a row with no bucket above it would have no softmax to speak of.
constexpr float kMaskBelow = -1e6f;

// The buckets in shared memory: their first distances, and the bucket of each
// distance below kNear (near the diagonal every element needs its own).
constexpr int kNear = 128;
struct Buckets {
  int starts[kMaxBuckets];
  uint8_t near[kNear];
  float ds_scale;  // backward: what the stored dS are multiplied by

  __device__ __forceinline__ void init(const BiasParams& bp, int tid, int threads) {
    for (int i = tid; i < bp.n; i += threads) starts[i] = bp.starts[i];
    __syncthreads();
    for (int i = tid; i < kNear; i += threads) near[i] = (uint8_t)search(bp.n, i);
  }
  // Last bucket whose first distance is <= dist (dist >= 0, starts[0] = 0).
  __device__ __forceinline__ int search(int n, int dist) const {
    int b = 0;
#pragma unroll
    for (int step = kMaxBuckets / 2; step; step >>= 1)
      if (b + step < n && starts[b + step] <= dist) b += step;
    return b;
  }
  __device__ __forceinline__ int of(int n, int dist) const {
    if (dist < kNear) return near[dist];
    return dist >= starts[n - 1] ? n - 1 : search(n, dist);
  }
};

// The bias of a bucket in units of log 2.
__device__ __forceinline__ float bias_log2(const float* row, int bucket) {
  const float b = __ldg(row + bucket);
  return b <= kMaskBelow ? -INFINITY : b * kLog2e;
}

// The bucket that a run of tiles shares: distances [lo, hi).
struct BucketRun {
  int lo, hi, bucket;
};
__device__ __forceinline__ void bucket_run(BucketRun& r, const Buckets& bk, int n, int dist) {
  r.bucket = bk.of(n, dist);
  r.lo = bk.starts[r.bucket];
  r.hi = r.bucket + 1 < n ? bk.starts[r.bucket + 1] : INT32_MAX;
}

// The same over the softmax scale, to be added to raw scores.
__device__ __forceinline__ float bias_over_scale(const float* row, int bucket, float inv_scale) {
  const float b = __ldg(row + bucket);
  return b <= kMaskBelow ? -INFINITY : b * inv_scale;
}

// The forward's window of one warp: entry y (0 .. 158) is the bias of the
// distance far - y, and row `lane`, column c of the tile takes entry
// c + 31 - lane. A row's 128 entries are read as 32 float4: four copies of the
// window, copy k shifted by k entries, give every row an aligned start, and
// copies 168 floats apart put the eight rows of a quarter-warp into different
// banks. Distances fall from one entry to a lane's next, 32 below it, and far
// from the diagonal the bucket is most often the same: it is kept and only
// looked up again when it is not (16K as above: 1.09 ms with a search for every
// entry. All entries' loads before the first store: 1.02, but 1.61 for 1.57 on
// the 32K workload).
constexpr int kWindowCopy = 168;
constexpr int kWindowFloats = 4 * kWindowCopy;
__device__ __forceinline__ void fill_window(float* win, const Buckets& bk, int n, const float* row, int far,
                                            float inv_scale, int lane) {
  __syncwarp();  // every row of the tile before has been read
  int bucket = n - 1;
#pragma unroll 1
  for (int y = lane; y < 160; y += 32) {
    const int dist = max(far - y, 0);
    if (dist < kNear) bucket = bk.near[dist];
    else if (bk.starts[bucket] > dist) bucket = bk.search(n, dist);
    const float b = bias_over_scale(row, bucket, inv_scale);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (y >= k) win[k * kWindowCopy + y - k] = b;
  }
  __syncwarp();
}
__device__ __forceinline__ const float4* window_row(const float* win, int lane) {
  const int first = 31 - lane, k = first & 3;
  return reinterpret_cast<const float4*>(win + k * kWindowCopy + first - k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Adds the warp's sum of v, times mul, to *at and sets v back to zero.
__device__ __forceinline__ void add_run(float* at, float& v, float mul, int lane) {
  if (!__any_sync(0xffffffffu, v != 0.f)) return;
  const float sum = warp_sum(v);
  if (lane == 0 && sum != 0.f) red_add(at, sum * mul);
  v = 0.f;
}

// Adds each lane's v to row[bucket], the buckets not falling with the lane:
// one atomic for every bucket of the warp.
__device__ __forceinline__ void add_by_bucket(float* row, int bucket, float v, int lane) {
#pragma unroll 1
  for (int m = 1; m < 32; m <<= 1) {  // inclusive sums inside a run of equal buckets
    const float up = __shfl_up_sync(0xffffffffu, v, m);
    const int b = __shfl_up_sync(0xffffffffu, bucket, m);
    if (lane >= m && b == bucket) v += up;
  }
  const int next = __shfl_down_sync(0xffffffffu, bucket, 1);
  if ((lane == 31 || next != bucket) && v != 0.f) red_add(row + bucket, v);
}

// Blocks of dS: 32 rows (keys) x 64 columns (queries), fp16,
// rows of 128 bytes in the 128-byte swizzle. Diagonal y holds the elements
// with column - row = y - 31.
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
// sum += one of a pair of fp16 values (one instruction: the fp32 add takes the
// 16-bit operand).
__device__ __forceinline__ void add_lo(float& sum, uint32_t pair) {
  asm("add.f32.f16 %0, %1, %0;" : "+f"(sum) : "h"((uint16_t)pair));
}
__device__ __forceinline__ void add_hi(float& sum, uint32_t pair) {
  asm("add.f32.f16 %0, %1, %0;" : "+f"(sum) : "h"((uint16_t)(pair >> 16)));
}

// Sum of a 128 x 64 panel of dS, in shares of the lanes. A short loop: what it
// fetches counts for more than its operations.
__device__ __forceinline__ float panel_sum(uint32_t panel, int lane) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int c = 0; c < 32; ++c) {
    uint32_t v[4];
    ld_shared_v4(panel + 512 * c + 16 * lane, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      add_lo(sum[i], v[i]);
      add_hi(sum[i], v[i]);
    }
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// Sums along the diagonals: this lane's lane, lane + 32 and lane + 64. Every
// lane reads its row and hands each pair of columns to the lane that keeps its
// first element's diagonal; the second element's is the next one, kept apart
// (b) until the end.
__device__ __forceinline__ void diagonal_sums(uint32_t block, int lane, float (&sum)[3]) {
  float a_lo = 0.f, a_hi = 0.f, b_lo = 0.f, b_hi = 0.f, b_last = 0.f;
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
#pragma unroll 1
    for (int c8 = 0; c8 < 4; ++c8) {
      uint32_t v[4];
      ld_shared_v4(block + sw128_offset(lane, 4 * half + c8), v);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int c = 8 * c8 + 2 * m;
        const uint32_t got = __shfl_sync(0xffffffffu, v[m], c + 31 - lane);
        if (lane >= c) {
          add_lo(a_lo, got);
          add_hi(b_lo, got);
        } else {
          add_lo(a_hi, got);
          add_hi(b_hi, got);
        }
      }
    }
    // The low entries are complete; the high ones are the next half's low ones.
    sum[0] = sum[1];
    sum[1] = a_lo + __shfl_sync(0xffffffffu, lane == 31 ? b_last : b_lo, lane + 31);
    b_last = b_lo;
    a_lo = a_hi;
    b_lo = b_hi;
    a_hi = b_hi = 0.f;
  }
  sum[2] = a_lo + __shfl_sync(0xffffffffu, lane == 31 ? b_last : b_lo, lane + 31);
}

}  // namespace dev
}  // namespace fcp
