// rel_plan.h -- host side of the learned relative position bias: the buckets of distances as
// intervals, and the arguments of the launches (device side: rel_bias.cuh).
#pragma once

#include <climits>
#include <cstdint>

namespace mha {

constexpr int kRelMaxSeg = 128;  // buckets a table may have

// The bias of one call, as the kernels take it.
struct RelBias {
  const void* table;            // [num_buckets, H], fp32 or bf16
  int table_f32;
  int H;
  int nseg;                     // segments in the order of the distance (see rel_bias.cuh)
  int num_buckets;
  float* partial;               // backward: the tiles' sums of dS per segment (device scratch)
  int32_t start[kRelMaxSeg];    // first distance of a segment; start[0] = INT_MIN
  uint8_t bucket[kRelMaxSeg];   // the segment's row of the table
};

// Fills start, bucket and nseg; false where the numbers describe no buckets:
// 2 <= num_buckets <= 128 (4 at least, and even, when bidirectional), max_distance above the
// distances that have a bucket of their own.
bool rel_plan(int num_buckets, int max_distance, bool bidirectional, RelBias* r);
// The bucket of distance d.
int rel_bucket_of(const RelBias& r, int d);

}  // namespace mha
