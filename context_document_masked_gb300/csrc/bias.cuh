// Device helpers of the bucketed distance bias, shared by the attention
// forward and backward.
//
// A warp works on 32 rows and a run of columns whose distances i - j are a
// Toeplitz window: element (l, c) has window index l - c or c - l plus a
// constant, so a tile of 32 x N elements has N + 31 distinct distances. Far
// from the diagonal they all fall into one bucket and the tile's bias is one
// number. Otherwise lane l keeps the window's entries l, l + 32, ... in
// registers and every column is served by one shuffle: lanes read entries
// that are a permutation of the lanes' numbers, each lane offering the one of
// its entries that its reader needs.
#pragma once

#include <cstdint>

#include "kernels.h"

namespace fcp {
namespace dev {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMaskBelow = -1e30f;  // a bias at or below this masks its bucket

// Last bucket whose first distance is <= dist (dist >= 0, starts[0] = 0).
__device__ __forceinline__ int bucket_of(const int* starts, int n, int dist) {
  int b = 0;
#pragma unroll
  for (int step = kMaxBuckets / 2; step; step >>= 1)
    if (b + step < n && starts[b + step] <= dist) b += step;
  return b;
}

// The bias of a bucket in units of log 2.
__device__ __forceinline__ float bias_log2(const float* row, int bucket) {
  const float b = __ldg(row + bucket);
  return b <= kMaskBelow ? -INFINITY : b * kLog2e;
}

// The bucket that a run of tiles shares: distances [lo, hi) have the value.
struct BucketRun {
  int lo, hi, bucket;
  float value;
};
__device__ __forceinline__ void bucket_run(BucketRun& r, const int* starts, int n, const float* row, int dist) {
  r.bucket = bucket_of(starts, n, dist);
  r.lo = starts[r.bucket];
  r.hi = r.bucket + 1 < n ? starts[r.bucket + 1] : INT32_MAX;
  r.value = bias_log2(row, r.bucket);
}

// Backward: element (lane, e) of a warp's 32 x 64 tile has window entry
// e + 31 - lane, held by lane (e + 31 - lane) mod 32.
__device__ __forceinline__ float window_at(const float (&win)[3], int e, int lane) {
  const float mine = lane >= (e & 31) ? win[e >> 5] : win[(e >> 5) + 1];
  return __shfl_sync(0xffffffffu, mine, e + 31 - lane);
}
// The reverse: x of element (lane, e) added to its window entry's sum.
__device__ __forceinline__ void window_add(float (&sum)[3], int e, int lane, float x) {
  const float got = __shfl_sync(0xffffffffu, x, e + 31 - lane);
  const bool low = lane >= (e & 31);
  sum[e >> 5] += low ? got : 0.f;
  sum[(e >> 5) + 1] += low ? 0.f : got;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Adds the warp's sum of v to *at and sets v back to zero.
__device__ __forceinline__ void add_run(float* at, float& v, int lane) {
  const float sum = warp_sum(v);
  if (lane == 0 && sum != 0.f) atomicAdd(at, sum);
  v = 0.f;
}

// Adds each lane's v to row[bucket], the buckets not falling with the lane:
// one atomic for every bucket of the warp.
__device__ __forceinline__ void add_by_bucket(float* row, int bucket, float v, int lane) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {  // inclusive sums inside a run of equal buckets
    const float up = __shfl_up_sync(0xffffffffu, v, m);
    const int b = __shfl_up_sync(0xffffffffu, bucket, m);
    if (lane >= m && b == bucket) v += up;
  }
  const int next = __shfl_down_sync(0xffffffffu, bucket, 1);
  if ((lane == 31 || next != bucket) && v != 0.f) atomicAdd(row + bucket, v);
}

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}

}  // namespace dev
}  // namespace fcp
