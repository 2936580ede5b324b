// rel_plan.cu -- the buckets of the learned relative position bias as intervals of the distance.
//
// Per side with n = |d| and `per` buckets (num_buckets / 2 on either side when bidirectional, else
// all of them for keys before the query, while keys at or after it count as n = 0), e = per / 2:
//   bucket = n                                                            for n < e
//   bucket = min(per - 1, e + floor((per - e) log(n / e) / log(max_distance / e)))   otherwise
// Keys after the query (d > 0) take the upper half of the table when bidirectional.  The last
// bucket of a side reaches to infinity.
#include "rel_plan.h"

#include <cmath>

namespace mha {
namespace {

// A whole number of up to 64 factors below 2^24.
struct Product {
  uint32_t w[48] = {1};
  int n = 1;
  void times(uint32_t f, int count) {
    for (; count > 0; --count) {
      uint64_t carry = 0;
      for (int i = 0; i < n; ++i) {
        carry += static_cast<uint64_t>(w[i]) * f;
        w[i] = static_cast<uint32_t>(carry);
        carry >>= 32;
      }
      if (carry != 0) w[n++] = static_cast<uint32_t>(carry);
    }
  }
  bool at_least(const Product& o) const {
    if (n != o.n) return n > o.n;
    for (int i = n - 1; i >= 0; --i)
      if (w[i] != o.w[i]) return w[i] > o.w[i];
    return true;
  }
};

// The first n of bucket e + t: the least whole n with n >= e (max_distance / e)^(t / (per - e)).  Where
// that border is a whole number (16 = 8 * 16^(2/8)) its double may come out on either side of it; others lie
// as close to one without being one (8 of per = 8, max_distance = 15688794: 3e-13 of it above 352539).
// 1e-12 covers the rounding of pow and lies far below the next whole number's distance: within that a
// comparison of whole numbers decides, n^(per - e) >= e^(per - e - t) max_distance^t.
int first_of(int t, int per, int e, int max_distance) {
  const double b = e * std::pow(static_cast<double>(max_distance) / e,
                                static_cast<double>(t) / (per - e));
  const int n = static_cast<int>(std::ceil(b * (1.0 - 1e-12)));
  if (n > b * (1.0 + 1e-12)) return n;
  Product left, right;
  left.times(n, per - e);
  right.times(e, per - e - t);
  right.times(max_distance, t);
  return left.at_least(right) ? n : n + 1;
}

}  // namespace

bool rel_plan(int num_buckets, int max_distance, bool bidirectional, RelBias* r) {
  if (num_buckets < 2 || num_buckets > kRelMaxSeg) return false;
  if (bidirectional && (num_buckets < 4 || num_buckets % 2 != 0)) return false;
  const int per = bidirectional ? num_buckets / 2 : num_buckets;
  const int e = per / 2;
  if (max_distance <= e || max_distance > kRelFar) return false;
  int first[kRelMaxSeg + 1];
  for (int u = 0; u < per; ++u) first[u] = u < e ? u : first_of(u - e, per, e, max_distance);
  int n = 0;
  auto add = [&](int start, int bucket) {
    r->seg[n] = (n == 0 ? -kRelFar : start) * 128 + bucket;
    ++n;
  };
  // keys before the query, farthest first; a bucket whose successor starts at the same n is empty
  for (int u = per - 1; u >= 0; --u) {
    if (u + 1 < per && first[u + 1] == first[u]) continue;
    // n in [first[u], first[u + 1]) is d in (-first[u + 1], -first[u]]
    add(u + 1 < per ? 1 - first[u + 1] : INT_MIN, u);
  }
  if (bidirectional)  // keys after the query; n = 0 belongs to the other side
    for (int u = 0; u < per; ++u) {
      if (u + 1 < per && (first[u + 1] == first[u] || first[u + 1] <= 1)) continue;
      add(first[u] < 1 ? 1 : first[u], per + u);
    }
  r->nseg = n;
  r->num_buckets = num_buckets;
  return true;
}

int rel_bucket_of(const RelBias& r, int d) {
  int s = 0;
  while (s + 1 < r.nseg && rel_start(r.seg[s + 1]) <= d) ++s;
  return rel_row(r.seg[s]);
}

}  // namespace mha
