// rel_bias.cuh -- the learned relative position bias of the attention kernels: how a distance
// d = (key's position) - (query's position) finds its number in the table [num_buckets, H].
//
// Buckets are intervals of d: near distances have one each, farther ones share buckets that grow
// with the logarithm of the distance, and all from max_distance on share the last.  Read in the
// order of d they are `nseg` segments, segment s holding start[s] <= d < start[s + 1].  The host
// works the borders out once per call and hands them over as a kernel parameter, so a kernel
// neither takes logarithms nor reads a map: it copies the borders and its head's bias into shared
// memory, and a tile of scores whose corner distances fall into one segment (most tiles: beyond
// max_distance there is one segment on either side) adds a constant, which the exponential's
// multiply-add takes in for nothing.  Only tiles that a border crosses look distances up.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "rel_plan.h"

namespace mha {

// stands in for RelBias in kernels that add no bias
struct NoRel {};
template <class Rel>
struct IsRel {
  static constexpr bool value = true;
};
template <>
struct IsRel<NoRel> {
  static constexpr bool value = false;
};

// A CTA's copy in shared memory: borders (INT_MAX behind the last segment) and bias.
struct RelShared {
  int start[kRelMaxSeg + 1];
  float bias[kRelMaxSeg + 1];
};
static_assert(sizeof(RelShared) == 8 * (kRelMaxSeg + 1), "");

// Entry s of the copy, for head h, the bias times `mul` (log2 e where exponentials are powers of
// two).  A value below kRelOut (a mask's: -1e9, a type's lowest, -inf) leaves its bucket out: it becomes
// -inf.  At that size fp32 sums of a score and a bias have lost all but a few bits of the score, so a
// softmax among such keys alone says nothing; and (t - m) c of such a t could pass the exponent's range
// by its rounding.
constexpr float kRelOut = -1e6f;
__device__ __forceinline__ void rel_load(RelShared& sh, const RelBias& r, int h, int s, float mul) {
  if (s > kRelMaxSeg) return;
  int at = INT_MAX;
  float v = 0.f;
  if (s < r.nseg) {
    const int32_t seg = r.seg[s];
    at = s == 0 ? INT_MIN : rel_start(seg);
    const int64_t i = static_cast<int64_t>(rel_row(seg)) * r.H + h;
    v = r.table_f32 ? __ldg(static_cast<const float*>(r.table) + i)
                    : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(r.table) + i));
    v = v < kRelOut ? -INFINITY : v * mul;
  }
  sh.start[s] = at;
  sh.bias[s] = v;
}

// The segment of each of N distances: borders behind the last segment are INT_MAX, start[0] INT_MIN.
// `steps` (rel_steps) is the same for all threads; the N searches run side by side.
__device__ __forceinline__ int rel_steps(int nseg) { return nseg <= 32 ? 16 : kRelMaxSeg / 2; }
template <int N>
__device__ __forceinline__ void rel_segments(const RelShared& sh, int steps, const int (&d)[N],
                                             int (&s)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0;
#pragma unroll 1
  for (int step = steps; step > 0; step >>= 1) {
    int at[N];
#pragma unroll
    for (int i = 0; i < N; ++i) at[i] = sh.start[s[i] + step];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += at[i] <= d[i] ? step : 0;
  }
}
__device__ __forceinline__ int rel_segment(const RelShared& sh, int steps, int d) {
  const int one[1] = {d};
  int s[1];
  rel_segments<1>(sh, steps, one, s);
  return s[0];
}

// A sum of any number of terms, with the rounding errors carried along (Kahan's summation): off by 2^-23
// of the terms' sizes, however many there are.
struct LongSum {
  float sum = 0.f, over = 0.f;  // over: what sum holds too much
  __device__ __forceinline__ void add(float x) {
    const float y = x - over, next = sum + y;
    over = (next - sum) - y;
    sum = next;
  }
};

// The gradient of head h's column of the table, by a block of kRelGradThreads threads:
// dtable[bucket of s, h] = sum over batch elements and tiles of partial[b, h, tile, s], in a fixed
// order; buckets without a segment get 0.
constexpr int kRelGradThreads = 256;
__device__ __forceinline__ void rel_table_grad(const RelBias& rel, void* dtable, int B, int tiles,
                                               int h) {
  constexpr int kWarps = kRelGradThreads / 32;
  __shared__ float part[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto put = [&](int u, float v) {
    const int64_t i = static_cast<int64_t>(u) * rel.H + h;
    if (rel.table_f32)
      static_cast<float*>(dtable)[i] = v;
    else
      static_cast<__nv_bfloat16*>(dtable)[i] = __float2bfloat16_rn(v);
  };
  if (static_cast<int>(threadIdx.x) < rel.num_buckets) {
    bool held = false;
    for (int s = 0; s < rel.nseg; ++s)
      held |= rel_row(rel.seg[s]) == static_cast<int>(threadIdx.x);
    if (!held) put(threadIdx.x, 0.f);
  }
  for (int s0 = 0; s0 < rel.nseg; s0 += 32) {
    const int s = s0 + lane;
    LongSum v;
    if (s < rel.nseg) {
      const float* head = rel.partial + static_cast<int64_t>(h) * tiles * rel.nseg + s;
      const int64_t rows = static_cast<int64_t>(B) * tiles;
      const int64_t skip = static_cast<int64_t>(rel.H - 1) * tiles;  // rows of the other heads
      int64_t b = 0, tile = warp;  // row r = b * tiles + tile, every kWarps-th
      while (tile >= tiles) tile -= tiles, ++b;
#pragma unroll 4
      for (int64_t r = warp; r < rows; r += kWarps) {
        v.add(head[(r + b * skip) * rel.nseg]);
        tile += kWarps;
        while (tile >= tiles) tile -= tiles, ++b;
      }
    }
    part[warp][lane] = v.sum;
    __syncthreads();
    if (warp == 0 && s < rel.nseg) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) sum += part[i][lane];
      put(rel_row(rel.seg[s]), sum);
    }
    __syncthreads();
  }
}

}  // namespace mha
