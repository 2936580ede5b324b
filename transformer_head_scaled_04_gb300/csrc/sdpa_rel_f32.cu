// sdpa_rel_f32.cu -- fp32 attention with a learned relative position bias, forward and backward, on
// the tensor cores.
//
//   forward   x = scale q.k + t (t: rel_bias.cuh), O = softmax(x) V, lse = log sum exp x
//   backward  p = exp(x - lse), D = rowsum(dO O), dS = p (dO.v - D),
//             dQ = scale dS K, dK = scale dS^T Q, dV = p^T dO, dt(segment) = sum of its dS
//
// Operands are scaled by powers of two that bring their largest value to 2^13 .. 2^14 and split into
// two fp16 terms, a = hi + lo (mma_f16.cuh); a product is hi hi + hi lo + lo hi with fp32 sums.  Every row
// of Q, K, V and dO has a scale of its own, so no row costs another one its accuracy, whether a mask hides
// it or not.  Scores take the two rows' factors back after the product over d.  In a product over rows the
// right operand's factors go into the left one (p_ij with the factor of V's row j, dS_ij with K's) before
// that is split, row by row of a tile under a scale that follows from its largest value: what no query
// sees has a weight of 0 there.  What is left of a value is at most 2^-23 of it or 2^-38 of the largest in
// its row (half a step of fp16's least, 2^-25, beside 2^13), and the dropped lo lo is at most 2^-22 of the
// product: fp32's own accuracy for values that are not far below their row's largest.  (Two tf32 terms
// give the same at twice the time of the tensor cores: the first form with fp16 terms took the forward of
// 8 x 8 heads of 1001 from 322 us to 239.  One scale for a tile's 32 rows on the right, which a hidden row
// of 1e8 spoils, took 195 there where this takes 214, and 695 against 710 in the backward.)  The tensor
// cores cut sums off instead of rounding them, 2^-24 of the sum per step towards zero (9e-6 of a gradient
// over 900 keys in one chain), so the large products are kept apart from the small ones, a chain spans one
// tile at most, and tiles are added up with ordinary additions.
//
// A CTA owns 64 rows (16 per warp) and goes over the other operand in tiles of 32 rows: while one tile
// is computed the next one's fp32 values arrive (asynchronous copies); then its rows' largest values
// are found and it is split into one or both of
//   rows   [row][d] halves, for products over d: a lane (lane = 4 g + t) reads 16 bytes of a row, eight
//          neighbouring d, as the inner positions of two steps (any order of the inner dimension
//          gives the same sum); 16-byte units of odd rows are swapped by 4, which frees the reads of
//          bank conflicts
//   pairs  words of two neighbouring rows' halves, for products over rows: the inner positions of a
//          score fragment are the columns a lane holds, 2 t and 2 t + 1, and 2 t + 8 and + 9, whose two
//          words for a d lie side by side, so that 16 bytes are the fragments of two d; the output's
//          columns are d = 16 v + 2 g + e
// and the CTA's own rows once into fragments, 16 bytes per lane and step: a lane's registers are filled
// in the order in which the product takes them, with no moves between (8 x 8 heads of 1001, with a scale
// per tile: with moves and unpaired arithmetic 223 us forward and 768 backward, without 196 and 705),
// so that scores go into the next product without any exchange.  d is padded to 64 or 128 with zeros.
// The bias of a tile that lies within one segment is a constant; otherwise the CTA looks its distances
// up once into a table.  Bound by the products, three per multiply-add of the formulas, and in the
// backward S and dP twice (dQ by its own kernel: no atomics, reproducible), and by the latencies between
// the barriers of a tile: the forward reaches 272 of the 590 TFLOP/s that these products measured alone
// (2 x 16 heads of 4096 1514 us), with 12 warps on an SM that issue in 40% of the cycles.  Not taken
// (measured with a scale per tile, when that case took 1376 us): 32 rows per warp, which halves the reads of
// K and V (1257 us there, but 52 instead of 41 for 4 x 8 causal heads of 500 and nothing gained at 8 x 8 of
// 1001), two buffers for the terms (206 us instead of 195 at 8 x 8 heads of 1001); and, with a scale per
// row, weights' scales from their rows' maxima where a tile's rows of V are alike (218 us instead of 214).
#include <cmath>

#include "device_common.cuh"
#include "launchers.h"
#include "mma_f16.cuh"
#include "rel_bias.cuh"

namespace mha {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 64;   // rows that a CTA owns, 16 per warp
constexpr int kTile = 32;   // rows of the other operand's tile
constexpr int kNT = kTile / 8;
constexpr int kDist = kRows + kTile - 1;  // distances of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct RelF32 {
  const float *Q, *K, *V, *dO;
  float *out, *dQ, *dK, *dV;   // out: the forward's O
  float* lse;                  // forward: written if not null; backward: read
  const float* Dv;             // backward: [B, H, Nq] rowsum(dO O)
  int64_t st[8][3];            // strides b, h, n of Q, K, V, O, dO, dQ, dK, dV (d: 1)
  int B, H, Nq, Nk, d_k, d_v, mask;
  const int32_t* key_len;
  float scale;
};

template <bool kVec>
__device__ __forceinline__ void copy_async(uint32_t dst, const float* src, bool valid) {
  if (kVec)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// This thread's part of copying tiles of rows of a [N, d] matrix with row stride sn into raw
// [kTile][DP]: rows from `limit` on and columns from d on become zeros (nothing of them is read).
template <int DP, bool kVec>
struct TileCopy {
  static constexpr int kUnit = kVec ? 4 : 1, kPer = DP / kUnit;
  static constexpr int kStep = kThreads / kPer;  // rows between a thread's copies (kPer <= kThreads)
  static_assert(kThreads % kPer == 0 && kTile % kStep == 0, "");
  const float* src;  // the thread's column of row 0
  int64_t sn;
  int limit;         // 0 where the column lies past d
  __device__ __forceinline__ TileCopy(const float* m, int64_t sn_, int rows, int d) {
    const int c = static_cast<int>(threadIdx.x) % kPer * kUnit;
    src = m + c;
    sn = sn_;
    limit = c < d ? rows : 0;
  }
  __device__ __forceinline__ void operator()(float* raw, int n0) const {
    const int r0 = static_cast<int>(threadIdx.x) / kPer;
    const float* from = src + static_cast<int64_t>(n0 + r0) * sn;
    const uint32_t to = smem_u32(raw) + (r0 * DP + static_cast<int>(threadIdx.x) % kPer * kUnit) * 4;
#pragma unroll(kVec ? kTile / kStep : 4)
    for (int i = 0; i < kTile / kStep; ++i) {
      const bool ok = n0 + r0 + i * kStep < limit;
      copy_async<kVec>(to + i * kStep * DP * 4, ok ? from : src, ok);
      from += kStep * sn;
    }
  }
};

// ---- scales: powers of two, the largest value goes to 2^13 .. 2^14 (below 2^-112 to less)
struct Scale {
  float mul, inv;
};
__device__ __forceinline__ Scale scale_for(uint32_t top) {  // the bits of the largest |value|
  const int e = max(static_cast<int>(top >> 23), 15);       // its exponent, plus 127
  return {__uint_as_float(static_cast<uint32_t>(267 - e) << 23),
          __uint_as_float(static_cast<uint32_t>(e - 13) << 23)};
}

// ---- a tile of fp32 values -> two fp16 terms
// The halves of unit u (8 values) of row r, in [rows][DP]: units of odd rows are swapped by 4.
template <int DP>
__device__ __forceinline__ int unit_at(int r, int u) {
  return r * (DP / 8) + (u ^ ((r & 1) << 2));
}
template <int DP>
__host__ __device__ constexpr int pair_pitch() {
  return 2 * DP + 8;  // words of a group: row pairs 8 s + t and 8 s + t + 4, group 4 s + t
}
template <int DP>
__host__ __device__ constexpr int rows_bytes(int rows) {
  return 2 * rows * DP * 2;  // hi, then lo
}
template <int DP>
__host__ __device__ constexpr int pairs_bytes() {
  return 2 * kTile / 4 * pair_pitch<DP>() * 4;
}

// the halves of x, and what they leave, rounded to halves
__device__ __forceinline__ uint32_t halves(float2 x) { return pack_half(x.x, x.y); }
__device__ __forceinline__ uint32_t rest_of(float2 x, uint32_t hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return halves(ffma2(f, make_float2(-1.f, -1.f), x));
}

// This thread's share of a raw tile: per item four columns of the rows of two pairs, 8 s + t and
// 8 s + t + 4.
template <int DP>
struct Share {
  static constexpr int kItems = kTile / 4 * (DP / 4) / kThreads;
  float4 x[kItems][4];
  __device__ __forceinline__ static int group(int i) { return (i * kThreads + threadIdx.x) / (DP / 4); }
  __device__ __forceinline__ static int col(int i) {
    return (i * kThreads + threadIdx.x) % (DP / 4) * 4;
  }
  __device__ __forceinline__ static int row(int i, int k) {  // of x[i][k]
    return 16 * (group(i) >> 2) + 2 * (group(i) & 3) + (k & 1) + 8 * (k >> 1);
  }
  __device__ __forceinline__ static float top(const float4& v) {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
  }
  __device__ __forceinline__ void read(const float* raw) {
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[i][k] = *reinterpret_cast<const float4*>(raw + row(i, k) * DP + col(i));
  }
  // the scales of the four rows of x[i], from the largest |value| in each: its exponent is the top of
  // the upper 16 bits, two rows' of which meet in one word
  __device__ __forceinline__ void scales(int i, Scale (&f)[4]) const {
    uint32_t w[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      w[u] = __byte_perm(__float_as_uint(top(x[i][2 * u])), __float_as_uint(top(x[i][2 * u + 1])),
                         0x7632);
#pragma unroll
    for (int off = 1; off < DP / 4; off <<= 1)  // the DP / 4 lanes of a row
#pragma unroll
      for (int u = 0; u < 2; ++u)
        w[u] = __vmaxu2(w[u], __shfl_xor_sync(0xffffffffu, w[u], off));
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = scale_for(k & 1 ? w[k >> 1] : w[k >> 1] << 16);
  }
  // writes its terms as rows and as pairs, either may be null, every row under a scale of its own; the
  // factors that undo the scales go to inv
  __device__ __forceinline__ void write(uint8_t* to_rows, uint32_t* to_pairs, float* inv) const {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int c = col(i);
      Scale f[4];
      scales(i, f);
      if (c == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) inv[row(i, k)] = f[k].inv;
      }
      float2 v[4][2];  // row k, columns c + 2 u, + 1
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 mul2 = make_float2(f[k].mul, f[k].mul);
        v[k][0] = fmul2(make_float2(x[i][k].x, x[i][k].y), mul2);
        v[k][1] = fmul2(make_float2(x[i][k].z, x[i][k].w), mul2);
      }
      uint32_t h[4][2], l[4][2];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          h[k][u] = halves(v[k][u]);
          l[k][u] = rest_of(v[k][u], h[k][u]);
        }
      if (to_rows != nullptr) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint8_t* at = to_rows + unit_at<DP>(row(i, k), c >> 3) * 16 + (c & 4) * 2;
          *reinterpret_cast<uint2*>(at) = make_uint2(h[k][0], h[k][1]);
          *reinterpret_cast<uint2*>(at + kTile * DP * 2) = make_uint2(l[k][0], l[k][1]);
        }
      }
      if (to_pairs != nullptr) {
        uint32_t* at = to_pairs + group(i) * pair_pitch<DP>() + 2 * c;
        constexpr int kLo = kTile / 4 * pair_pitch<DP>();
        auto put = [&](uint32_t* to, const uint32_t (&w)[4][2], int u) {
          *reinterpret_cast<uint4*>(to + 4 * u) = make_uint4(
              __byte_perm(w[0][u], w[1][u], 0x5410), __byte_perm(w[2][u], w[3][u], 0x5410),
              __byte_perm(w[0][u], w[1][u], 0x7632), __byte_perm(w[2][u], w[3][u], 0x7632));
        };
        put(at, h, 0);
        put(at, h, 1);
        put(at + kLo, l, 0);
        put(at + kLo, l, 1);
      }
    }
  }
  // the same for rows row0 .. of the CTA's own, as fragments
  __device__ __forceinline__ void write_own(uint32_t* to, int row0, float* inv) const {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int c = col(i), unit = c >> 3, step = 2 * (unit >> 2) + ((c >> 2) & 1);
      Scale f[4];
      scales(i, f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 mul2 = make_float2(f[k].mul, f[k].mul);
        const int r = row0 + row(i, k), g = r & 7;
        uint32_t* at = to + (((r >> 4) * (DP / 16) + step) * 32 + 4 * g + (unit & 3)) * 4 +
                       ((r >> 3) & 1);
        const float2 v0 = fmul2(make_float2(x[i][k].x, x[i][k].y), mul2);
        const float2 v1 = fmul2(make_float2(x[i][k].z, x[i][k].w), mul2);
        const uint32_t h0 = halves(v0), h1 = halves(v1);
        at[0] = h0;
        at[2] = h1;
        at[kRows * DP / 2] = rest_of(v0, h0);
        at[kRows * DP / 2 + 2] = rest_of(v1, h1);
        if (c == 0) inv[r] = f[k].inv;
      }
    }
  }
};

// The CTA's own 64 rows, split into fragments, and the factors that undo their scales; raw is scratch.
template <int DP, bool kVec>
__device__ __forceinline__ void own_rows(uint32_t* to, float* inv, float* raw, const float* src,
                                         int64_t sn, int n0, int limit, int d) {
  static_assert(DP / 4 <= 32 && 32 % (DP / 4) == 0, "a row within a warp");
  const TileCopy<DP, kVec> copy(src, sn, limit, d);
#pragma unroll 1
  for (int i = 0; i < kRows; i += kTile) {
    copy(raw, n0 + i);
    copy_commit();
    copy_wait();
    __syncthreads();
    Share<DP> s;
    s.read(raw);
    s.write_own(to, i, inv);
    __syncthreads();
  }
}

// ---- products
template <int DP>
__device__ __forceinline__ uint4 unit16(const uint8_t* rows, int r, int u) {
  return *reinterpret_cast<const uint4*>(rows + unit_at<DP>(r, u) * 16);
}
__device__ __forceinline__ float2 pair_of(const float (&s)[4], int half) {
  return make_float2(s[2 * half], s[2 * half + 1]);
}
__device__ __forceinline__ void set_pair(float (&s)[4], int half, float2 v) {
  s[2 * half] = v.x;
  s[2 * half + 1] = v.y;
}

// s[n] = A B^T over d: A the warp's own 16 rows, B's rows 8 n + g of kTile
template <int DP>
__device__ __forceinline__ void product_d(float (&s)[kNT][4], const uint32_t* A, int warp, int lane,
                                          const uint8_t* B) {
  constexpr int kLoA = kRows * DP / 8, kLoB = kTile * DP * 2;
  const int g = lane >> 2, t = lane & 3;
  const uint4* a4 = reinterpret_cast<const uint4*>(A) + warp * (DP / 16) * 32 + lane;
  float hi[kNT][4], lo[kNT][4];
#pragma unroll
  for (int h = 0; h < DP / 32; ++h) {
    const uint4 x0 = a4[2 * h * 32], x1 = a4[(2 * h + 1) * 32];
    const uint4 y0 = a4[2 * h * 32 + kLoA], y1 = a4[(2 * h + 1) * 32 + kLoA];
    const uint32_t a0[4] = {x0.x, x0.y, x0.z, x0.w}, a1[4] = {x1.x, x1.y, x1.z, x1.w};
    const uint32_t l0[4] = {y0.x, y0.y, y0.z, y0.w}, l1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
    for (int n = 0; n < kNT; n += 2) {  // two columns' chains side by side
      uint4 b[2], bl[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        b[i] = unit16<DP>(B, 8 * (n + i) + g, t + 4 * h);
        bl[i] = unit16<DP>(B + kLoB, 8 * (n + i) + g, t + 4 * h);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (h == 0)
          mma16816_zero(lo[n + i], l0, b[i].x, b[i].y);
        else
          mma16816(lo[n + i], l0, b[i].x, b[i].y);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (h == 0)
          mma16816_zero(hi[n + i], a0, b[i].x, b[i].y);
        else
          mma16816(hi[n + i], a0, b[i].x, b[i].y);
#pragma unroll
      for (int i = 0; i < 2; ++i) mma16816(lo[n + i], l1, b[i].z, b[i].w);
#pragma unroll
      for (int i = 0; i < 2; ++i) mma16816(hi[n + i], a1, b[i].z, b[i].w);
#pragma unroll
      for (int i = 0; i < 2; ++i) mma16816(lo[n + i], a0, bl[i].x, bl[i].y);
#pragma unroll
      for (int i = 0; i < 2; ++i) mma16816(lo[n + i], a1, bl[i].z, bl[i].w);
    }
  }
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) set_pair(s[n], i, fadd2(pair_of(hi[n], i), pair_of(lo[n], i)));
}

// the fragments of 16 x 32 scores, rows g and g + 8 times mul0 and mul1, as the operand of a product
// over rows
struct ScoreFrags {
  uint32_t hi[kNT / 2][4], lo[kNT / 2][4];
  __device__ __forceinline__ ScoreFrags(const float (&p)[kNT][4], float mul0, float mul1) {
#pragma unroll
    for (int s = 0; s < kNT / 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // (g, 2 t), (g + 8, 2 t), then the next eight columns
        const float mul = i & 1 ? mul1 : mul0;
        const float2 x = fmul2(pair_of(p[2 * s + (i >> 1)], i & 1), make_float2(mul, mul));
        hi[s][i] = halves(x);
        lo[s][i] = rest_of(x, hi[s][i]);
      }
  }
};
// the scale for row g (half 0) or g + 8 (half 1) of a warp's scores
__device__ __forceinline__ Scale score_scale(const float (&p)[kNT][4], int half) {
  float m = 0.f;
#pragma unroll
  for (int n = 0; n < kNT; ++n) m = fmax3(m, fabsf(p[n][2 * half]), fabsf(p[n][2 * half + 1]));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return scale_for(__float_as_uint(m));
}

// the scores of columns 8 n + 2 t and + 1 times mul[column]
__device__ __forceinline__ void scale_columns(float (&p)[kNT][4], const float* mul, int t) {
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    const float2 f = *reinterpret_cast<const float2*>(mul + 8 * n + 2 * t);
#pragma unroll
    for (int i = 0; i < 2; ++i) set_pair(p[n], i, fmul2(pair_of(p[n], i), f));
  }
}

// o[2 v + e] (d = 16 v + 2 g + e) += P B over the tile's rows (B as pairs), rows g and g + 8 times inv0
// and inv1
template <int DP>
__device__ __forceinline__ void product_rows(float (&o)[DP / 8][4], const ScoreFrags& p,
                                             const uint32_t* B, float inv0, float inv1, int g,
                                             int t) {
  constexpr int kP = pair_pitch<DP>(), kLo = kTile / 4 * kP;
  const float2 inv[2] = {make_float2(inv0, inv0), make_float2(inv1, inv1)};
#pragma unroll
  for (int u = 0; u < DP / 32; ++u) {
    uint4 b[kNT / 2][2];
    float sum[4][4];  // the small terms first, then the large: a chain of two where cuts matter
#pragma unroll
    for (int s = 0; s < kNT / 2; ++s) {
      uint4 l[2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t* at = B + (4 * s + t) * kP + 2 * (32 * u + 16 * v + 2 * g);
        b[s][v] = *reinterpret_cast<const uint4*>(at);
        l[v] = *reinterpret_cast<const uint4*>(at + kLo);
      }
#pragma unroll
      for (int v = 0; v < 2; ++v)
        if (s == 0) {
          mma16816_zero(sum[2 * v], p.lo[s], b[s][v].x, b[s][v].y);
          mma16816_zero(sum[2 * v + 1], p.lo[s], b[s][v].z, b[s][v].w);
        } else {
          mma16816(sum[2 * v], p.lo[s], b[s][v].x, b[s][v].y);
          mma16816(sum[2 * v + 1], p.lo[s], b[s][v].z, b[s][v].w);
        }
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        mma16816(sum[2 * v], p.hi[s], l[v].x, l[v].y);
        mma16816(sum[2 * v + 1], p.hi[s], l[v].z, l[v].w);
      }
    }
#pragma unroll
    for (int s = 0; s < kNT / 2; ++s)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        mma16816(sum[2 * v], p.hi[s], b[s][v].x, b[s][v].y);
        mma16816(sum[2 * v + 1], p.hi[s], b[s][v].z, b[s][v].w);
      }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        set_pair(o[4 * u + n], i, ffma2(pair_of(sum[n], i), inv[i], pair_of(o[4 * u + n], i)));
  }
}

// rows g (half 0) or g + 8 (half 1) of product_rows' output, times mul, to dst
template <int DP, bool kVec>
__device__ __forceinline__ void store_row(float* dst, const float (&o)[DP / 8][4], int half, int t,
                                          int d, float mul) {
#pragma unroll
  for (int v = 0; v < DP / 16; ++v) {
    const int c = 16 * v + 4 * t;
    const float4 x = make_float4(o[2 * v][2 * half] * mul, o[2 * v + 1][2 * half] * mul,
                                 o[2 * v][2 * half + 1] * mul, o[2 * v + 1][2 * half + 1] * mul);
    if (kVec) {
      if (c < d) *reinterpret_cast<float4*>(dst + c) = x;
    } else {
      if (c < d) dst[c] = x.x;
      if (c + 1 < d) dst[c + 1] = x.y;
      if (c + 2 < d) dst[c + 2] = x.z;
      if (c + 3 < d) dst[c + 3] = x.w;
    }
  }
}

__device__ __forceinline__ int keys_of(const RelF32& p, int b) {
  return p.mask == 2 ? min(max(__ldg(p.key_len + b), 0), p.Nk) : p.Nk;
}

// x, at most 0 (NaN stays NaN): the exponent x - lse of a weight that the backward rebuilds.  Scores and
// lse may be so large that their difference is rounding, several hundred from 2^30 on; no weight passes 1.
__device__ __forceinline__ float at_most_0(float x) {
  float y;
  asm("min.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

// x = s f + t, f = f0 (row g) or f1 (g + 8) times col[column]; t the constant, or of the lane's columns
// 8 n + 2 t, + 1 and rows g, g + 8 from the table (at: its entry for column 2 t and row g; a row less is
// a distance more)
__device__ __forceinline__ void add_bias(float (&s)[kNT][4], float f0, float f1, const float* col,
                                         int t, bool near, float constant, const float* at) {
  const float2 f[2] = {make_float2(f0, f0), make_float2(f1, f1)};
  if (near) {
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      const float2 c = *reinterpret_cast<const float2*>(col + 8 * n + 2 * t);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        set_pair(s[n], i, ffma2(pair_of(s[n], i), fmul2(f[i], c),
                                make_float2(at[8 * n - 8 * i], at[8 * n + 1 - 8 * i])));
    }
  } else {
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      const float2 c = *reinterpret_cast<const float2*>(col + 8 * n + 2 * t);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        set_pair(s[n], i, ffma2(pair_of(s[n], i), fmul2(f[i], c), make_float2(constant, constant)));
    }
  }
}

// ============================================================================ forward
template <int DP>
struct FwdSmem {
  uint32_t Q[rows_bytes<DP>(kRows) / 4];
  uint8_t K[rows_bytes<DP>(kTile)];
  uint32_t V[pairs_bytes<DP>() / 4];
  float rawK[kTile * DP], rawV[kTile * DP];
  float table[kDist + 1], q_inv[kRows], k_inv[kTile], v_inv[kTile];
  RelShared rs;
};

// One CTA per 64 queries of a head.
template <int DP, bool kVec>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 3 : 2)
    sdpa_rel_f32_kernel(const RelF32 p, const __grid_constant__ RelBias rel) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  extern __shared__ __align__(16) uint8_t smem[];
  FwdSmem<DP>& sm = *reinterpret_cast<FwdSmem<DP>*>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z;
  const int q0 = (p.mask == 1 ? static_cast<int>(gridDim.x - 1 - blockIdx.x)  // longest first
                              : static_cast<int>(blockIdx.x)) * kRows;
  const int L = keys_of(p, b);
  const int last = min(q0 + kRows, p.Nq) - 1;
  const int nt = p.mask == 1 ? last / kTile + 1 : (L + kTile - 1) / kTile;
  const TileCopy<DP, kVec> copy_k(p.K + b * p.st[1][0] + h * p.st[1][1], p.st[1][2], L, p.d_k);
  const TileCopy<DP, kVec> copy_v(p.V + b * p.st[2][0] + h * p.st[2][1], p.st[2][2], L, p.d_v);
  auto load = [&](int j) {
    copy_k(sm.rawK, j * kTile);
    copy_v(sm.rawV, j * kTile);
    copy_commit();
  };
  for (int s = threadIdx.x; s <= kRelMaxSeg; s += kThreads) rel_load(sm.rs, rel, h, s, kLog2e);
  own_rows<DP, kVec>(sm.Q, sm.q_inv, sm.rawK, p.Q + b * p.st[0][0] + h * p.st[0][1], p.st[0][2], q0,
                     p.Nq, p.d_k);
  const float unit = p.scale * kLog2e;  // scores in powers of two
  const float q_inv[2] = {sm.q_inv[16 * warp + g] * unit, sm.q_inv[16 * warp + g + 8] * unit};
  const int row[2] = {q0 + 16 * warp + g, q0 + 16 * warp + g + 8};
  const int limit[2] = {p.mask == 1 ? row[0] : L - 1, p.mask == 1 ? row[1] : L - 1};
  float o[DP / 8][4] = {};
  float m[2] = {-INFINITY, -INFINITY};
  float2 l[2] = {};
  int seg_next = INT_MIN;
  float seg_bias = 0.f;
  if (nt > 0) load(0);
  for (int j = 0; j < nt; ++j) {
    const int d0 = j * kTile - (q0 + kRows - 1);  // the tile's smallest distance
    if (d0 >= seg_next) {
      const int seg = rel_segment(sm.rs, rel_steps(rel.nseg), d0);
      seg_next = sm.rs.start[seg + 1];
      seg_bias = sm.rs.bias[seg];
    }
    const bool near = d0 + kDist - 1 >= seg_next;
    copy_wait();
    __syncthreads();  // the tile is there, the previous one done with
    if (near && threadIdx.x < kDist)
      sm.table[threadIdx.x] =
          sm.rs.bias[rel_segment(sm.rs, rel_steps(rel.nseg), d0 + threadIdx.x)];
    {
      Share<DP> k, v;
      k.read(sm.rawK);
      v.read(sm.rawV);
      k.write(sm.K, nullptr, sm.k_inv);
      v.write(nullptr, sm.V, sm.v_inv);
    }
    __syncthreads();
    if (j + 1 < nt) load(j + 1);
    if (p.mask != 1 || j * kTile <= q0 + 16 * warp + 15) {
      float s[kNT][4];
      product_d<DP>(s, sm.Q, warp, lane, sm.K);
      float mx[2] = {-INFINITY, -INFINITY};
      add_bias(s, q_inv[0], q_inv[1], sm.k_inv, t, near, seg_bias,
               sm.table + 2 * t - (16 * warp + g) + kRows - 1);
      if (j * kTile + kTile - 1 > (p.mask == 1 ? q0 + 16 * warp : L - 1)) {
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j * kTile + 8 * n + 2 * t + (i & 1) > limit[i >> 1]) s[n][i] = -INFINITY;
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i >> 1] = fmaxf(mx[i >> 1], s[n][i]);
      float alpha[2], ref[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        const float m_new = fmaxf(m[i], mx[i]);
        ref[i] = m_new == -INFINITY ? 0.f : m_new;
        alpha[i] = ex2_approx(m[i] - ref[i]);
        m[i] = m_new;
        l[i] = fmul2(l[i], make_float2(alpha[i], alpha[i]));
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2 x = fadd2(pair_of(s[n], i), make_float2(-ref[i], -ref[i]));
          x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
          set_pair(s[n], i, x);
          l[i] = fadd2(l[i], x);
        }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int u = 0; u < DP / 8; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            set_pair(o[u], i, fmul2(pair_of(o[u], i), make_float2(alpha[i], alpha[i])));
      }
      scale_columns(s, sm.v_inv, t);
      const Scale f0 = score_scale(s, 0), f1 = score_scale(s, 1);
      product_rows<DP>(o, ScoreFrags(s, f0.mul, f1.mul), sm.V, f0.inv, f1.inv, g, t);
    }
  }
  float* ob = p.out + b * p.st[3][0] + h * p.st[3][1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float sum = l[i].x + l[i].y;
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (row[i] < p.Nq) {
      store_row<DP, kVec>(ob + static_cast<int64_t>(row[i]) * p.st[3][2], o, i, t, p.d_v,
                          sum > 0.f ? 1.f / sum : 0.f);
      if (t == 0 && p.lse != nullptr)
        p.lse[(static_cast<int64_t>(b) * p.H + h) * p.Nq + row[i]] =
            sum > 0.f ? fmaf(m[i], kLn2, logf(sum)) : INFINITY;
    }
  }
}

// ============================================================================ backward
template <int DP>
struct DqSmem {
  uint32_t Q[rows_bytes<DP>(kRows) / 4], G[rows_bytes<DP>(kRows) / 4];  // G: dO
  uint32_t Kp[pairs_bytes<DP>() / 4];
  union {
    struct {
      uint8_t K[rows_bytes<DP>(kTile)], V[rows_bytes<DP>(kTile)];
    };
    float S[kRows * (kTile + 1)];  // dS where segments meet, when K and V are done with
  };
  float rawK[kTile * DP], rawV[kTile * DP];
  float D[kRows], lse[kRows], q_inv[kRows], g_inv[kRows];
  float k_inv[kTile], v_inv[kTile];
  float table[kDist + 1];
  float far[kWarps];
  float part[kWarps][32];  // a warp's sums of the segments span[..][0] .. span[..][1]
  int span[kWarps][2];
  RelShared rs;
};

// 64 queries' dQ and their sums of dS per segment (thread s owns segment s)
template <int DP, bool kVec>
__device__ __forceinline__ void queries_part(const RelF32& p, const RelBias& rel, DqSmem<DP>& sm,
                                             int h, int b, int tile, int tiles) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int q0 = tile * kRows;
  const int L = keys_of(p, b);
  const int last = min(q0 + kRows, p.Nq) - 1;
  const int nt = p.mask == 1 ? last / kTile + 1 : (L + kTile - 1) / kTile;
  const int64_t bh = static_cast<int64_t>(b) * p.H + h;
  const TileCopy<DP, kVec> copy_k(p.K + b * p.st[1][0] + h * p.st[1][1], p.st[1][2], L, p.d_k);
  const TileCopy<DP, kVec> copy_v(p.V + b * p.st[2][0] + h * p.st[2][1], p.st[2][2], L, p.d_v);
  const float* gb = p.dO + b * p.st[4][0] + h * p.st[4][1];
  auto load = [&](int j) {
    copy_k(sm.rawK, j * kTile);
    copy_v(sm.rawV, j * kTile);
    copy_commit();
  };
  for (int s = tid; s <= kRelMaxSeg; s += kThreads) rel_load(sm.rs, rel, h, s, 1.f);
  if (tid < kRows) {
    const int64_t i = bh * p.Nq + q0 + tid;
    sm.D[tid] = q0 + tid < p.Nq ? p.Dv[i] : 0.f;
    sm.lse[tid] = q0 + tid < p.Nq ? p.lse[i] : INFINITY;
  }
  own_rows<DP, kVec>(sm.Q, sm.q_inv, sm.rawK, p.Q + b * p.st[0][0] + h * p.st[0][1], p.st[0][2], q0,
                     p.Nq, p.d_k);
  own_rows<DP, kVec>(sm.G, sm.g_inv, sm.rawK, gb, p.st[4][2], q0, p.Nq, p.d_v);
  const int r_loc[2] = {16 * warp + g, 16 * warp + g + 8};
  const int limit[2] = {p.mask == 1 ? q0 + r_loc[0] : L - 1, p.mask == 1 ? q0 + r_loc[1] : L - 1};
  const float lse[2] = {sm.lse[r_loc[0]], sm.lse[r_loc[1]]}, D[2] = {sm.D[r_loc[0]], sm.D[r_loc[1]]};
  const float q_inv[2] = {sm.q_inv[r_loc[0]] * p.scale, sm.q_inv[r_loc[1]] * p.scale};
  const float g_inv[2] = {sm.g_inv[r_loc[0]], sm.g_inv[r_loc[1]]};
  float dq[DP / 8][4] = {};
  LongSum far, own;
  int seg = 0, seg_next = INT_MIN;
  float seg_bias = 0.f;
  auto flush_far = [&]() {  // by all threads
    float v = far.sum;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == 0) sm.far[warp] = v;
    far = LongSum();
    __syncthreads();
    if (tid == seg) own.add((sm.far[0] + sm.far[1]) + (sm.far[2] + sm.far[3]));
    __syncthreads();
  };
  if (nt > 0) load(0);
  for (int j = 0; j < nt; ++j) {
    const int d0 = j * kTile - (q0 + kRows - 1);
    if (d0 >= seg_next) {
      if (j > 0) flush_far();
      seg = rel_segment(sm.rs, rel_steps(rel.nseg), d0);
      seg_next = sm.rs.start[seg + 1];
      seg_bias = sm.rs.bias[seg];
    }
    const bool near = d0 + kDist - 1 >= seg_next;
    copy_wait();
    __syncthreads();  // the tile is there, the previous one done with
    int dist_seg = 0;  // the segment of distance d0 + tid
    if (near) {
      dist_seg = rel_segment(sm.rs, rel_steps(rel.nseg), d0 + tid);
      if (tid < kDist) sm.table[tid] = sm.rs.bias[dist_seg];
    }
    {
      Share<DP> k, v;
      k.read(sm.rawK);
      v.read(sm.rawV);
      k.write(sm.K, sm.Kp, sm.k_inv);
      v.write(sm.V, nullptr, sm.v_inv);
    }
    __syncthreads();
    if (j + 1 < nt) load(j + 1);
    const bool skip = p.mask == 1 && j * kTile > q0 + 16 * warp + 15;
    float s[kNT][4] = {};
    if (!skip) {
      float dp[kNT][4];
      product_d<DP>(s, sm.Q, warp, lane, sm.K);
      product_d<DP>(dp, sm.G, warp, lane, sm.V);
      add_bias(s, q_inv[0], q_inv[1], sm.k_inv, t, near, seg_bias,
               sm.table + 2 * t - r_loc[0] + kRows - 1);
      if (j * kTile + kTile - 1 > (p.mask == 1 ? q0 + 16 * warp : L - 1)) {
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j * kTile + 8 * n + 2 * t + (i & 1) > limit[i >> 1]) s[n][i] = -INFINITY;
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const float2 c = *reinterpret_cast<const float2*>(sm.v_inv + 8 * n + 2 * t);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2 x = fadd2(pair_of(s[n], i), make_float2(-lse[i], -lse[i]));
          x = fmul2(x, make_float2(kLog2e, kLog2e));
          x = make_float2(ex2_approx(at_most_0(x.x)), ex2_approx(at_most_0(x.y)));
          const float2 fg = fmul2(make_float2(g_inv[i], g_inv[i]), c);
          set_pair(s[n], i, fmul2(x, ffma2(pair_of(dp[n], i), fg, make_float2(-D[i], -D[i]))));
        }
      }
    }
    if (near) {
      __syncthreads();  // K and V as rows are done with
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sm.S[r_loc[i >> 1] * (kTile + 1) + 8 * n + 2 * t + (i & 1)] = s[n][i];
    } else {
      float2 x = make_float2(0.f, 0.f);
#pragma unroll
      for (int n = 0; n < kNT; ++n) x = fadd2(x, fadd2(pair_of(s[n], 0), pair_of(s[n], 1)));
      far.add(x.x + x.y);
    }
    if (!skip) {
      scale_columns(s, sm.k_inv, t);
      const Scale f0 = score_scale(s, 0), f1 = score_scale(s, 1);
      product_rows<DP>(dq, ScoreFrags(s, f0.mul, f1.mul), sm.Kp, f0.inv, f1.inv, g, t);
    }
    if (near) {  // sums over the diagonals, one per thread, then over each warp's segments
      __syncthreads();
      float acc = 0.f;
#pragma unroll 8
      for (int r = 0; r < kRows; ++r) {
        const int c = r + tid - (kRows - 1);
        if (c >= 0 && c < kTile) acc += sm.S[r * (kTile + 1) + c];
      }
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const float up = __shfl_up_sync(0xffffffffu, acc, off);
        const int other = __shfl_up_sync(0xffffffffu, dist_seg, off);
        if (lane >= off && other == dist_seg) acc += up;
      }
      const int first = __shfl_sync(0xffffffffu, dist_seg, 0);
      const int next = __shfl_down_sync(0xffffffffu, dist_seg, 1);
      if (lane == 31 || next != dist_seg) sm.part[warp][dist_seg - first] = acc;
      if (lane == 0) sm.span[warp][0] = first;
      if (lane == 31) sm.span[warp][1] = dist_seg;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (tid >= sm.span[w][0] && tid <= sm.span[w][1])
          own.add(sm.part[w][tid - sm.span[w][0]]);
    }
  }
  if (nt > 0) {
    __syncthreads();
    flush_far();
  }
  if (tid < rel.nseg) rel.partial[(bh * tiles + tile) * rel.nseg + tid] = own.sum;
  float* out = p.dQ + b * p.st[5][0] + h * p.st[5][1];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (q0 + r_loc[i] < p.Nq)
      store_row<DP, kVec>(out + static_cast<int64_t>(q0 + r_loc[i]) * p.st[5][2], dq, i, t, p.d_k,
                          p.scale);
}

template <int DP>
struct DkdvSmem {
  uint32_t K[rows_bytes<DP>(kRows) / 4], V[rows_bytes<DP>(kRows) / 4];
  uint8_t Q[rows_bytes<DP>(kTile)], G[rows_bytes<DP>(kTile)];  // G: dO
  uint32_t Qp[pairs_bytes<DP>() / 4], Gp[pairs_bytes<DP>() / 4];
  float rawQ[kTile * DP], rawG[kTile * DP];
  float D[kTile], lse[kTile];  // both negated
  float q_inv[kTile], g_inv[kTile];
  float k_inv[kRows], v_inv[kRows];
  float table[kDist + 1];
  RelShared rs;
};

// 64 keys' dK and dV from tiles of 32 queries
template <int DP, bool kVec>
__device__ __forceinline__ void keys_part(const RelF32& p, const RelBias& rel, DkdvSmem<DP>& sm,
                                          int h, int b, int tile) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int k0 = tile * kRows;
  const int L = keys_of(p, b);
  const int64_t bh = static_cast<int64_t>(b) * p.H + h;
  const TileCopy<DP, kVec> copy_q(p.Q + b * p.st[0][0] + h * p.st[0][1], p.st[0][2], p.Nq, p.d_k);
  const TileCopy<DP, kVec> copy_g(p.dO + b * p.st[4][0] + h * p.st[4][1], p.st[4][2], p.Nq, p.d_v);
  const int i0 = p.mask == 1 ? k0 / kTile : 0;  // the first tile of queries that sees a key
  const int ni = k0 < L ? (p.Nq + kTile - 1) / kTile : 0;
  const int key[2] = {k0 + 16 * warp + g, k0 + 16 * warp + g + 8};
  float dk[DP / 8][4] = {}, dv[DP / 8][4] = {};
  if (i0 < ni) {
    auto load = [&](int i) {
      copy_q(sm.rawQ, i * kTile);
      copy_g(sm.rawG, i * kTile);
      copy_commit();
    };
    for (int s = tid; s <= kRelMaxSeg; s += kThreads) rel_load(sm.rs, rel, h, s, 1.f);
    own_rows<DP, kVec>(sm.K, sm.k_inv, sm.rawQ, p.K + b * p.st[1][0] + h * p.st[1][1], p.st[1][2],
                       k0, L, p.d_k);
    own_rows<DP, kVec>(sm.V, sm.v_inv, sm.rawQ, p.V + b * p.st[2][0] + h * p.st[2][1], p.st[2][2],
                       k0, L, p.d_v);
    const int r = 16 * warp + g;
    const float k_inv[2] = {sm.k_inv[r] * p.scale, sm.k_inv[r + 8] * p.scale};
    const float v_inv[2] = {sm.v_inv[r], sm.v_inv[r + 8]};
    int seg_start = INT_MAX;
    float seg_bias = 0.f;
    load(i0);
    for (int i = i0; i < ni; ++i) {
      const int q0 = i * kTile;
      const int d0 = k0 - (q0 + kTile - 1);  // distances d0 + e, e = key row + 31 - query
      if (d0 + kDist - 1 < seg_start) {
        const int seg = rel_segment(sm.rs, rel_steps(rel.nseg), d0 + kDist - 1);
        seg_start = sm.rs.start[seg];
        seg_bias = sm.rs.bias[seg];
      }
      const bool near = d0 < seg_start;
      copy_wait();
      __syncthreads();  // the tile is there, the previous one done with
      if (tid < kTile) {
        sm.D[tid] = q0 + tid < p.Nq ? -p.Dv[bh * p.Nq + q0 + tid] : 0.f;
        sm.lse[tid] = q0 + tid < p.Nq ? -p.lse[bh * p.Nq + q0 + tid] : -INFINITY;
      }
      if (near && tid < kDist)
        sm.table[tid] = sm.rs.bias[rel_segment(sm.rs, rel_steps(rel.nseg), d0 + tid)];
      {
        Share<DP> q, o;
        q.read(sm.rawQ);
        o.read(sm.rawG);
        q.write(sm.Q, sm.Qp, sm.q_inv);
        o.write(sm.G, sm.Gp, sm.g_inv);
      }
      __syncthreads();
      if (i + 1 < ni) load(i + 1);
      float s[kNT][4], ds[kNT][4];
      product_d<DP>(s, sm.K, warp, lane, sm.Q);
      product_d<DP>(ds, sm.V, warp, lane, sm.G);
      // the table by row (key) minus column (query): a row more is a distance more
      const float* at = sm.table + 16 * warp + g - 2 * t + kTile - 1;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const float2 c = *reinterpret_cast<const float2*>(sm.q_inv + 8 * n + 2 * t);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 bias = near ? make_float2(at[8 * e - 8 * n], at[8 * e - 8 * n - 1])
                                   : make_float2(seg_bias, seg_bias);
          set_pair(s[n], e, ffma2(pair_of(s[n], e), fmul2(make_float2(k_inv[e], k_inv[e]), c), bias));
        }
      }
      if (k0 + 16 * warp + 15 >= L || (p.mask == 1 && k0 + 16 * warp + 15 > q0)) {
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = key[e >> 1];
            if (j >= L || (p.mask == 1 && j > q0 + 8 * n + 2 * t + (e & 1))) s[n][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const float2 lse = *reinterpret_cast<const float2*>(sm.lse + 8 * n + 2 * t);
        const float2 D = *reinterpret_cast<const float2*>(sm.D + 8 * n + 2 * t);
        const float2 c = *reinterpret_cast<const float2*>(sm.g_inv + 8 * n + 2 * t);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2 x = fadd2(pair_of(s[n], e), lse);
          x = fmul2(x, make_float2(kLog2e, kLog2e));
          x = make_float2(ex2_approx(at_most_0(x.x)), ex2_approx(at_most_0(x.y)));
          set_pair(s[n], e, x);
          const float2 fg = fmul2(make_float2(v_inv[e], v_inv[e]), c);
          set_pair(ds[n], e, fmul2(x, ffma2(pair_of(ds[n], e), fg, D)));
        }
      }
      scale_columns(s, sm.g_inv, t);
      const Scale s0 = score_scale(s, 0), s1 = score_scale(s, 1);
      product_rows<DP>(dv, ScoreFrags(s, s0.mul, s1.mul), sm.Gp, s0.inv, s1.inv, g, t);
      scale_columns(ds, sm.q_inv, t);
      const Scale d0s = score_scale(ds, 0), d1s = score_scale(ds, 1);
      product_rows<DP>(dk, ScoreFrags(ds, d0s.mul, d1s.mul), sm.Qp, d0s.inv, d1s.inv, g, t);
    }
  }
  float* ok = p.dK + b * p.st[6][0] + h * p.st[6][1];
  float* ov = p.dV + b * p.st[7][0] + h * p.st[7][1];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (key[e] < p.Nk) {
      store_row<DP, kVec>(ok + static_cast<int64_t>(key[e]) * p.st[6][2], dk, e, t, p.d_k, p.scale);
      store_row<DP, kVec>(ov + static_cast<int64_t>(key[e]) * p.st[7][2], dv, e, t, p.d_v, 1.f);
    }
}

// A CTA takes 64 keys or 64 queries of a head, first the keys of all heads, then the queries: one launch
// keeps the GPU filled where one kind alone would leave it waiting for its longest CTAs (4 x 8 heads of
// 500, causal: 112 us in two launches, 77 in one, 72 now), and the two kinds' code meets on an SM only in
// between (keys and queries of a head side by side, 8 x 8 heads of 1001: 858 us).  A tile takes a
// CTA alone on its SM 4 us and two CTAs 2 us each: what bounds it is latency between barriers with
// eight warps on an SM; 248 registers leave no third CTA room.
template <int DP>
struct BwdSmem {
  union {
    DqSmem<DP> q;
    DkdvSmem<DP> k;
  };
};
template <int DP, bool kVec>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 2 : 1)
    sdpa_rel_bwd_f32_kernel(const RelF32 p, const __grid_constant__ RelBias rel) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output (D among it) is complete from here on
  extern __shared__ __align__(16) uint8_t smem[];
  BwdSmem<DP>& sm = *reinterpret_cast<BwdSmem<DP>*>(smem);
  const uint32_t nq = (p.Nq + kRows - 1) / kRows, nk = (p.Nk + kRows - 1) / kRows;
  const uint32_t heads = static_cast<uint32_t>(p.B) * p.H;
  const bool keys = blockIdx.x < heads * nk;
  const uint32_t x = keys ? blockIdx.x : blockIdx.x - heads * nk, tiles = keys ? nk : nq;
  uint32_t bh = x / tiles, tile = x % tiles;
  if (p.mask == 1) {  // the longest of all heads first
    bh = x % heads;
    tile = keys ? x / heads : tiles - 1 - x / heads;
  }
  const int h = static_cast<int>(bh % p.H), b = static_cast<int>(bh / p.H);
  if (keys)
    keys_part<DP, kVec>(p, rel, sm.k, h, b, static_cast<int>(tile));
  else
    queries_part<DP, kVec>(p, rel, sm.q, h, b, static_cast<int>(tile), static_cast<int>(tiles));
}

// the gradient of the table alone, one block per head
__global__ void __launch_bounds__(kRelGradThreads)
    rel_table_grad_kernel(const __grid_constant__ RelBias rel, void* dtable, int B, int tiles) {
  pdl_launch_dependents();
  pdl_wait();  // the partial sums are complete from here on
  rel_table_grad(rel, dtable, B, tiles, static_cast<int>(blockIdx.x));
}

template <class F>
cudaError_t go(F* kernel, dim3 grid, size_t smem, const RelF32& p, const RelBias& rel,
               cudaStream_t s) {
  cudaError_t e =
      prepare_kernel(reinterpret_cast<const void*>(kernel), static_cast<int>(smem), nullptr);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, grid, dim3(kThreads), smem, s, p, rel);
}

// 16-byte copies: whole quads of aligned rows
bool quads(const void* ptr, const int64_t* st, int d) {
  return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && d % 4 == 0 && st[0] % 4 == 0 &&
         st[1] % 4 == 0 && st[2] % 4 == 0;
}

}  // namespace

cudaError_t launch_sdpa_rel_f32(const SdpaArgs& a, const RelBias& rel, cudaStream_t s) {
  RelF32 p = {};
  p.Q = static_cast<const float*>(a.Q);
  p.K = static_cast<const float*>(a.K);
  p.V = static_cast<const float*>(a.V);
  p.out = static_cast<float*>(a.O);
  p.lse = a.lse;
  const int64_t* st[4] = {a.sq, a.sk, a.sv, a.so};
  for (int t = 0; t < 4; ++t)
    for (int i = 0; i < 3; ++i) p.st[t][i] = st[t][i];
  p.B = a.B; p.H = a.H; p.Nq = a.Nq; p.Nk = a.Nk; p.d_k = a.d_k; p.d_v = a.d_v;
  p.mask = a.mask;
  p.key_len = a.key_len;
  p.scale = a.scale;
  const bool vec = quads(a.Q, p.st[0], a.d_k) && quads(a.K, p.st[1], a.d_k) &&
                   quads(a.V, p.st[2], a.d_v) && quads(a.O, p.st[3], a.d_v);
  const dim3 grid((a.Nq + kRows - 1) / kRows, a.H, a.B);
  if (a.d_k <= 64 && a.d_v <= 64)
    return vec ? go(sdpa_rel_f32_kernel<64, true>, grid, sizeof(FwdSmem<64>), p, rel, s)
               : go(sdpa_rel_f32_kernel<64, false>, grid, sizeof(FwdSmem<64>), p, rel, s);
  return vec ? go(sdpa_rel_f32_kernel<128, true>, grid, sizeof(FwdSmem<128>), p, rel, s)
             : go(sdpa_rel_f32_kernel<128, false>, grid, sizeof(FwdSmem<128>), p, rel, s);
}

int rel_bwd_tiles(int Nq, int Nk, int dtype) {
  return dtype == 1 ? (Nk + 127) / 128 : (Nq + kRows - 1) / kRows;
}

cudaError_t launch_sdpa_rel_bwd_f32(const SdpaBwdArgs& a, const RelBias& rel, void* dtable,
                                    cudaStream_t s) {
  RelF32 p = {};
  p.Q = static_cast<const float*>(a.Q);
  p.K = static_cast<const float*>(a.K);
  p.V = static_cast<const float*>(a.V);
  p.dO = static_cast<const float*>(a.dO);
  p.dQ = static_cast<float*>(a.dQ);
  p.dK = static_cast<float*>(a.dK);
  p.dV = static_cast<float*>(a.dV);
  p.lse = const_cast<float*>(a.lse);
  p.Dv = a.Dv;
  const void* ptr[8] = {a.Q, a.K, a.V, a.O, a.dO, a.dQ, a.dK, a.dV};
  const int dims[8] = {a.d_k, a.d_k, a.d_v, a.d_v, a.d_v, a.d_k, a.d_k, a.d_v};
  bool vec = true;
  for (int t = 0; t < 8; ++t) {
    for (int i = 0; i < 3; ++i) p.st[t][i] = a.st[t][i];
    if (t != 3) vec = vec && quads(ptr[t], p.st[t], dims[t]);
  }
  p.B = a.B; p.H = a.H; p.Nq = a.Nq; p.Nk = a.Nk; p.d_k = a.d_k; p.d_v = a.d_v;
  p.mask = a.mask;
  p.key_len = a.key_len;
  p.scale = a.scale;
  cudaError_t e = launch_sdpa_bwd_rowdot(a, 0, s);  // D
  if (e != cudaSuccess) return e;
  const int64_t blocks = static_cast<int64_t>(a.B) * a.H *
                         ((a.Nq + kRows - 1) / kRows + (a.Nk + kRows - 1) / kRows);
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;  // 64 rows each: past any memory
  const dim3 grid(static_cast<unsigned>(blocks));
  if (a.d_k <= 64 && a.d_v <= 64)
    e = vec ? go(sdpa_rel_bwd_f32_kernel<64, true>, grid, sizeof(BwdSmem<64>), p, rel, s)
            : go(sdpa_rel_bwd_f32_kernel<64, false>, grid, sizeof(BwdSmem<64>), p, rel, s);
  else
    e = vec ? go(sdpa_rel_bwd_f32_kernel<128, true>, grid, sizeof(BwdSmem<128>), p, rel, s)
            : go(sdpa_rel_bwd_f32_kernel<128, false>, grid, sizeof(BwdSmem<128>), p, rel, s);
  return e == cudaSuccess ? launch_rel_table_grad(rel, dtable, a.B, rel_bwd_tiles(a.Nq, a.Nk, 0), s)
                          : e;
}

cudaError_t launch_rel_table_grad(const RelBias& rel, void* dtable, int B, int tiles,
                                  cudaStream_t s) {
  return launch_pdl(rel_table_grad_kernel, dim3(rel.H), dim3(kRelGradThreads), 0, s, rel, dtable, B,
                    tiles);
}

}  // namespace mha
