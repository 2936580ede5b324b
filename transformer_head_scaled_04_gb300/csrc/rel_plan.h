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
  // segment s: its first distance << 7 | its row of the table, one word, because lanes that read
  // different words of a parameter are served one after another (of the first segment, which has
  // no first distance, -kRelFar)
  int32_t seg[kRelMaxSeg];
};
constexpr int kRelFar = (1 << 24) - 1;  // positions are at most 2^24, distances less
constexpr int rel_start(int32_t seg) { return seg >> 7; }
constexpr int rel_row(int32_t seg) { return seg & 127; }

// Fills seg and nseg; false where the numbers describe no buckets:
// 2 <= num_buckets <= 128 (4 at least, and even, when bidirectional), max_distance above the
// distances that have a bucket of their own and at most kRelFar.
bool rel_plan(int num_buckets, int max_distance, bool bidirectional, RelBias* r);
// The bucket of distance d.
int rel_bucket_of(const RelBias& r, int d);

}  // namespace mha
