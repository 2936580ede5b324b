// sdpa_rel_f32.cu -- fp32 attention with a learned relative position bias, forward and backward,
// on the tensor cores (fp32 values as two tf32 terms, three products: mma_tf32.cuh).
//
//   forward   x = scale q.k + t (t: rel_bias.cuh), O = softmax(x) V, lse = log sum exp x
//   backward  p = exp(x - lse), D = rowsum(dO O), dS = p (dO.v - D),
//             dQ = scale dS K, dK = scale dS^T Q, dV = p^T dO, dt(segment) = sum of its dS
//
// Warp products of 16 x 8 x 8 have register fragments that need no exchange between a score and its
// use as the next product's operand, if the inner dimension is read in a fitting order (any order
// gives the same sum): with lane = 4 g + t,
//   products over d: inner positions t and t + 4 of a step are two neighbouring d, and a lane reads
//     four of them at once, d = 32 u + 8 t + 4 v .. + 3;
//   products over keys (or queries): positions t and t + 4 are rows 8 n + 2 t and 8 n + 2 t + 1, which
//     are the two columns of the score fragment that the lane holds; the output's columns are
//     d = 4 g + e + 32 u, so that a lane again reads four at once.
// Rows in shared memory are d + 4 floats apart: both kinds of 16-byte reads are free of conflicts.
// Tiles are 64 rows of the operand that a CTA owns (16 per warp) against 32 of the other, d
// padded to 64 or 128 with zeros.  The bias of a tile that lies within one segment is a constant;
// otherwise the CTA looks its distances up once into a table.  Bound by the products: three per
// multiply-add of the formulas.
#include <cmath>

#include "device_common.cuh"
#include "launchers.h"
#include "mma_tf32.cuh"
#include "rel_bias.cuh"

namespace mha {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 64;    // rows that a CTA owns, 16 per warp
constexpr int kBwdRows = 32;  // rows per step of the backward kernels
constexpr float kLog2e = 1.4426950408889634f;

__host__ __device__ constexpr int pitch_of(int dp) { return dp + 4; }
constexpr int kFwdKeys = 32;  // keys per step of the forward (two steps in shared memory)

struct RelF32 {
  const float *Q, *K, *V, *O, *dO;
  float *out, *dQ, *dK, *dV;   // out: the forward's O
  float* lse;                  // forward: written if not null; backward: read
  float* Dv;                   // backward: [B, H, Nq] rowsum(dO O)
  int64_t st[8][3];            // strides b, h, n of Q, K, V, O, dO, dQ, dK, dV (d: 1)
  int H, Nq, Nk, d_k, d_v, mask;
  const int32_t* key_len;
  float scale;
};

__device__ __forceinline__ void copy_async(uint32_t dst, const float* src, bool valid, int bytes16) {
  if (bytes16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// rows n0 .. n0 + kN - 1 of a [N, d] matrix with row stride sn into dst [kN][DP + 4]; rows from
// `limit` on and columns from d on become zeros (nothing of them is read)
template <int DP, bool kVec, int kN>
__device__ __forceinline__ void load_rows(float* dst, const float* src, int64_t sn, int n0,
                                          int limit, int d) {
  constexpr int kUnit = kVec ? 4 : 1;
  constexpr int kPer = DP / kUnit;
  static_assert(kN * kPer % kThreads == 0, "");
#pragma unroll 4
  for (int i = 0; i < kN * kPer / kThreads; ++i) {
    const int e = i * kThreads + threadIdx.x;
    const int r = e / kPer, c = e % kPer * kUnit;
    const bool ok = n0 + r < limit && c < d;
    const float* from = ok ? src + static_cast<int64_t>(n0 + r) * sn + c : src;
    copy_async(smem_u32(dst + r * pitch_of(DP) + c), from, ok, kVec);
  }
}

// the lane's four values of row r for chunk cc of a product over d
template <int DP>
__device__ __forceinline__ float4 row4(const float* m, int r, int cc, int t) {
  return *reinterpret_cast<const float4*>(m + r * pitch_of(DP) + 32 * (cc >> 1) + 8 * t +
                                          4 * (cc & 1));
}
// the lane's four values of row r for half u of a product over rows
template <int DP>
__device__ __forceinline__ float4 col4(const float* m, int r, int u, int g) {
  return *reinterpret_cast<const float4*>(m + r * pitch_of(DP) + 32 * u + 4 * g);
}

template <int N>
__device__ __forceinline__ void add_up(float (&d)[N][4], const float (&hi)[N][4],
                                       const float (&lo)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) d[n][i] = hi[n][i] + lo[n][i];
}

// s[n] = A B^T over d: A's rows a_row + g, + 8; B's rows 8 n + g
template <int DP, int NT>
__device__ __forceinline__ void product_d(float (&s)[NT][4], const float* A, int a_row,
                                          const float* B, int g, int t) {
  float hi[NT][4] = {}, lo[NT][4] = {};
#pragma unroll
  for (int cc = 0; cc < DP / 16; ++cc) {
    const float4 x = row4<DP>(A, a_row + g, cc, t), y = row4<DP>(A, a_row + g + 8, cc, t);
    const Tf32FragA a0 = frag_a(x.x, y.x, x.y, y.y), a1 = frag_a(x.z, y.z, x.w, y.w);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float4 b = row4<DP>(B, 8 * n + g, cc, t);
      mma_f32(hi[n], lo[n], a0, b.x, b.y);
      mma_f32(hi[n], lo[n], a1, b.z, b.w);
    }
  }
  add_up(s, hi, lo);
}

// o[4 u + e] += P B over rows: P the fragments of 16 x 8 NT scores, B's rows 8 n + 2 t, + 1
template <int DP, int NT>
__device__ __forceinline__ void product_rows(float (&o)[DP / 8][4], const float (&p)[NT][4],
                                             const float* B, int g, int t) {
#pragma unroll
  for (int u = 0; u < DP / 32; ++u) {
    float hi[4][4] = {}, lo[4][4] = {};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const Tf32FragA a = frag_a(p[n][0], p[n][2], p[n][1], p[n][3]);
      const float4 x = col4<DP>(B, 8 * n + 2 * t, u, g), y = col4<DP>(B, 8 * n + 2 * t + 1, u, g);
      mma_f32(hi[0], lo[0], a, x.x, y.x);
      mma_f32(hi[1], lo[1], a, x.y, y.y);
      mma_f32(hi[2], lo[2], a, x.z, y.z);
      mma_f32(hi[3], lo[3], a, x.w, y.w);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[4 * u + e][i] += hi[e][i] + lo[e][i];
  }
}

// rows g (half 0) or g + 8 (half 1) of product_rows' output, times mul, to dst
template <int DP, bool kVec>
__device__ __forceinline__ void store_row(float* dst, const float (&o)[DP / 8][4], int half, int t,
                                          int d, float mul) {
#pragma unroll
  for (int u = 0; u < DP / 32; ++u) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int c = 32 * u + 8 * t + 4 * v;
      const float4 x = make_float4(o[4 * u][2 * half + v] * mul, o[4 * u + 1][2 * half + v] * mul,
                                   o[4 * u + 2][2 * half + v] * mul,
                                   o[4 * u + 3][2 * half + v] * mul);
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
}

__device__ __forceinline__ int keys_of(const RelF32& p, int b) {
  return p.mask == 2 ? min(max(__ldg(p.key_len + b), 0), p.Nk) : p.Nk;
}

// ============================================================================ forward
template <int DP>
__host__ __device__ constexpr int fwd_smem() {
  return (4 * kFwdKeys * pitch_of(DP) + kRows + kFwdKeys) * 4 +
         static_cast<int>(sizeof(RelShared));
}

// One CTA per 64 queries of a head; K and V in steps of 32 keys, the next step's
// copies in flight while one is computed.
template <int DP, bool kVec>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 3 : 2)
    sdpa_rel_f32_kernel(const RelF32 p, const __grid_constant__ RelBias rel) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  constexpr int kK = kFwdKeys, kNT = kK / 8, kP = pitch_of(DP);
  extern __shared__ float smem[];
  float* sK = smem;                       // [2][kK][kP]
  float* sV = sK + 2 * kK * kP;           // [2][kK][kP]
  float* table = sV + 2 * kK * kP;        // bias of distance d0 + e at e
  RelShared& rs = *reinterpret_cast<RelShared*>(table + kRows + kK);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z;
  const int q0 = (p.mask == 1 ? static_cast<int>(gridDim.x - 1 - blockIdx.x)  // longest first
                              : static_cast<int>(blockIdx.x)) * kRows;
  const int L = keys_of(p, b);
  const int last = min(q0 + kRows, p.Nq) - 1;
  const int nt = p.mask == 1 ? last / kK + 1 : (L + kK - 1) / kK;
  const float* kb = p.K + b * p.st[1][0] + h * p.st[1][1];
  const float* vb = p.V + b * p.st[2][0] + h * p.st[2][1];
  auto load = [&](int j) {
    load_rows<DP, kVec, kK>(sK + (j & 1) * kK * kP, kb, p.st[1][2], j * kK, L, p.d_k);
    load_rows<DP, kVec, kK>(sV + (j & 1) * kK * kP, vb, p.st[2][2], j * kK, L, p.d_v);
    copy_commit();
  };
  for (int s = threadIdx.x; s <= kRelMaxSeg; s += kThreads) rel_load(rs, rel, h, s, 1.f);
  // Q through the K buffer into registers: the A fragments' values, not yet split
  float qa[DP / 16][4], qb[DP / 16][4];
  {
    const float* qs = p.Q + b * p.st[0][0] + h * p.st[0][1];
    static_assert(2 * kK >= kRows, "");
    load_rows<DP, kVec, kRows>(sK, qs, p.st[0][2], q0, p.Nq, p.d_k);
    copy_commit();
    copy_wait<0>();
    __syncthreads();
#pragma unroll
    for (int cc = 0; cc < DP / 16; ++cc) {
      const float4 x = row4<DP>(sK, 16 * warp + g, cc, t), y = row4<DP>(sK, 16 * warp + g + 8, cc, t);
      qa[cc][0] = x.x; qa[cc][1] = x.y; qa[cc][2] = x.z; qa[cc][3] = x.w;
      qb[cc][0] = y.x; qb[cc][1] = y.y; qb[cc][2] = y.z; qb[cc][3] = y.w;
    }
    __syncthreads();
  }
  const int row[2] = {q0 + 16 * warp + g, q0 + 16 * warp + g + 8};
  const int limit[2] = {p.mask == 1 ? row[0] : L - 1, p.mask == 1 ? row[1] : L - 1};
  float o[DP / 8][4] = {};
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int seg_next = INT_MIN;
  float seg_bias = 0.f;
  if (nt > 0) load(0);
  for (int j = 0; j < nt; ++j) {
    if (j + 1 < nt) load(j + 1);
    const int d0 = j * kK - (q0 + kRows - 1);  // the tile's smallest distance
    if (d0 >= seg_next) {
      const int seg = rel_segment(rs, rel_steps(rel.nseg), d0);
      seg_next = rs.start[seg + 1];
      seg_bias = rs.bias[seg];
    }
    const bool near = d0 + kRows + kK - 2 >= seg_next;
    if (near)
      for (int e = threadIdx.x; e < kRows + kK - 1; e += kThreads)
        table[e] = rs.bias[rel_segment(rs, rel_steps(rel.nseg), d0 + e)];
    if (j + 1 < nt)
      copy_wait<1>();
    else
      copy_wait<0>();
    __syncthreads();
    if (p.mask != 1 || j * kK <= q0 + 16 * warp + 15) {
      const float* k = sK + (j & 1) * kK * kP;
      const float* v = sV + (j & 1) * kK * kP;
      float s[kNT][4], hi[kNT][4] = {}, lo[kNT][4] = {};
#pragma unroll
      for (int cc = 0; cc < DP / 16; ++cc) {
        const Tf32FragA a0 = frag_a(qa[cc][0], qb[cc][0], qa[cc][1], qb[cc][1]);
        const Tf32FragA a1 = frag_a(qa[cc][2], qb[cc][2], qa[cc][3], qb[cc][3]);
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          const float4 x = row4<DP>(k, 8 * n + g, cc, t);
          mma_f32(hi[n], lo[n], a0, x.x, x.y);
          mma_f32(hi[n], lo[n], a1, x.z, x.w);
        }
      }
      add_up(s, hi, lo);
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 8 * n + 2 * t + (i & 1);  // the tile's key
          const float bias = near ? table[c - (16 * warp + g + 8 * (i >> 1)) + kRows - 1] : seg_bias;
          s[n][i] = j * kK + c <= limit[i >> 1] ? fmaf(s[n][i], p.scale, bias) : -INFINITY;
          mx[i >> 1] = fmaxf(mx[i >> 1], s[n][i]);
        }
      float alpha[2], ref[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        const float m_new = fmaxf(m[i], mx[i]);
        ref[i] = m_new == -INFINITY ? 0.f : m_new;
        alpha[i] = ex2_approx((m[i] - ref[i]) * kLog2e);
        m[i] = m_new;
        l[i] *= alpha[i];
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[n][i] = ex2_approx((s[n][i] - ref[i >> 1]) * kLog2e);
          l[i >> 1] += s[n][i];
        }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int u = 0; u < DP / 8; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[u][i] *= alpha[i >> 1];
      }
      product_rows<DP, kNT>(o, s, v, g, t);
    }
    __syncthreads();  // this step's buffers and table may be written again
  }
  float* ob = p.out + b * p.st[3][0] + h * p.st[3][1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (row[i] < p.Nq) {
      store_row<DP, kVec>(ob + static_cast<int64_t>(row[i]) * p.st[3][2], o, i, t, p.d_v,
                          l[i] > 0.f ? 1.f / l[i] : 0.f);
      if (t == 0 && p.lse != nullptr)
        p.lse[(static_cast<int64_t>(b) * p.H + h) * p.Nq + row[i]] =
            l[i] > 0.f ? m[i] + logf(l[i]) : INFINITY;
    }
  }
}

// ============================================================================ backward
// dS of one step's element: p = exp(s scale + bias - lse), 0 where the pair is not allowed
__device__ __forceinline__ float weight(float s, float scale, float bias, float lse, bool ok) {
  return ok ? ex2_approx(fmaf(s, scale, bias - lse) * kLog2e) : 0.f;
}

template <int DP>
__host__ __device__ constexpr int dq_smem() {
  return ((2 * kRows + 2 * kBwdRows) * pitch_of(DP) + kRows * (kBwdRows + 1) + 2 * kRows + 96 +
          96 + 4) * 4 + static_cast<int>(sizeof(RelShared));
}

// One CTA per 64 queries: D, dQ and the tile's sums of dS per segment (thread s owns segment s).
template <int DP, bool kVec>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 3 : 2)
    sdpa_rel_dq_f32_kernel(const RelF32 p, const __grid_constant__ RelBias rel) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  constexpr int kP = pitch_of(DP), kNT = kBwdRows / 8, kDist = kRows + kBwdRows - 1;
  extern __shared__ float smem[];
  float* sQ = smem;                              // [64][kP]
  float* sG = sQ + kRows * kP;                   // [64][kP]: dO
  float* sK = sG + kRows * kP;                   // [32][kP]
  float* sV = sK + kBwdRows * kP;                // [32][kP]
  float* sS = sV + kBwdRows * kP;                // [64][33]: dS where segments meet
  float* sD = sS + kRows * (kBwdRows + 1);       // [64]: D
  float* sL = sD + kRows;                        // [64]: lse
  float* table = sL + kRows;                     // [95]
  float* diag = table + 96;                      // [95]: sums over the diagonals
  float* red = diag + 96;                        // [4]
  RelShared& rs = *reinterpret_cast<RelShared*>(red + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z;
  const int q0 = (p.mask == 1 ? static_cast<int>(gridDim.x - 1 - blockIdx.x)
                              : static_cast<int>(blockIdx.x)) * kRows;
  const int L = keys_of(p, b);
  const int last = min(q0 + kRows, p.Nq) - 1;
  const int nt = p.mask == 1 ? last / kBwdRows + 1 : (L + kBwdRows - 1) / kBwdRows;
  const int64_t bh = static_cast<int64_t>(b) * p.H + h;
  const float* kb = p.K + b * p.st[1][0] + h * p.st[1][1];
  const float* vb = p.V + b * p.st[2][0] + h * p.st[2][1];
  load_rows<DP, kVec, kRows>(sQ, p.Q + b * p.st[0][0] + h * p.st[0][1], p.st[0][2], q0, p.Nq,
                             p.d_k);
  load_rows<DP, kVec, kRows>(sG, p.dO + b * p.st[4][0] + h * p.st[4][1], p.st[4][2], q0, p.Nq,
                             p.d_v);
  copy_commit();
  for (int s = tid; s <= kRelMaxSeg; s += kThreads) rel_load(rs, rel, h, s, 1.f);
  copy_wait<0>();
  __syncthreads();
  {  // two threads to a row
    const int r = tid >> 1;
    const float* orow = p.O + b * p.st[3][0] + h * p.st[3][1] +
                        static_cast<int64_t>(q0 + r) * p.st[3][2];
    float acc = 0.f;
    if (q0 + r < p.Nq)
      for (int d = tid & 1; d < p.d_v; d += 2) acc = fmaf(sG[r * kP + d], orow[d], acc);
    acc += __shfl_xor_sync(0xffffffffu, acc, 1);
    if ((tid & 1) == 0) {
      sD[r] = acc;
      sL[r] = q0 + r < p.Nq ? p.lse[bh * p.Nq + q0 + r] : INFINITY;
      if (q0 + r < p.Nq) p.Dv[bh * p.Nq + q0 + r] = acc;
    }
  }
  const int r_loc[2] = {16 * warp + g, 16 * warp + g + 8};
  const int limit[2] = {p.mask == 1 ? q0 + r_loc[0] : L - 1, p.mask == 1 ? q0 + r_loc[1] : L - 1};
  float dq[DP / 8][4] = {};
  float far = 0.f, own = 0.f;
  int seg = 0, seg_next = INT_MIN;
  float seg_bias = 0.f;
  auto flush_far = [&]() {  // by all threads
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) far += __shfl_xor_sync(0xffffffffu, far, off);
    if (lane == 0) red[warp] = far;
    far = 0.f;
    __syncthreads();
    if (tid == seg) own += (red[0] + red[1]) + (red[2] + red[3]);
    __syncthreads();
  };
  for (int j = 0; j < nt; ++j) {
    __syncthreads();  // the previous step is done with the buffers
    load_rows<DP, kVec, kBwdRows>(sK, kb, p.st[1][2], j * kBwdRows, L, p.d_k);
    load_rows<DP, kVec, kBwdRows>(sV, vb, p.st[2][2], j * kBwdRows, L, p.d_v);
    copy_commit();
    const int d0 = j * kBwdRows - (q0 + kRows - 1);
    if (d0 >= seg_next || (j & 63) == 0) {
      if (j > 0) flush_far();  // also every 64 steps, which bounds the length of a sum
      seg = rel_segment(rs, rel_steps(rel.nseg), d0);
      seg_next = rs.start[seg + 1];
      seg_bias = rs.bias[seg];
    }
    const bool near = d0 + kDist - 1 >= seg_next;
    if (near && tid < kDist) table[tid] = rs.bias[rel_segment(rs, rel_steps(rel.nseg), d0 + tid)];
    copy_wait<0>();
    __syncthreads();
    const bool skip = p.mask == 1 && j * kBwdRows > q0 + 16 * warp + 15;
    float s[kNT][4] = {};
    if (!skip) {
      float dp[kNT][4];
      product_d<DP, kNT>(s, sQ, 16 * warp, sK, g, t);
      product_d<DP, kNT>(dp, sG, 16 * warp, sV, g, t);
      const float lse[2] = {sL[r_loc[0]], sL[r_loc[1]]}, D[2] = {sD[r_loc[0]], sD[r_loc[1]]};
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 8 * n + 2 * t + (i & 1);
          const float bias = near ? table[c - r_loc[i >> 1] + kRows - 1] : seg_bias;
          const float w = weight(s[n][i], p.scale, bias, lse[i >> 1],
                                 j * kBwdRows + c <= limit[i >> 1]);
          s[n][i] = w * (dp[n][i] - D[i >> 1]);
        }
    }
    if (near) {
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sS[r_loc[i >> 1] * (kBwdRows + 1) + 8 * n + 2 * t + (i & 1)] = s[n][i];
    } else {
#pragma unroll
      for (int n = 0; n < kNT; ++n) far += (s[n][0] + s[n][1]) + (s[n][2] + s[n][3]);
    }
    if (!skip) product_rows<DP, kNT>(dq, s, sK, g, t);
    if (near) {  // sums over the diagonals, then over each segment's diagonals
      __syncthreads();
      if (tid < kDist) {
        float acc = 0.f;
#pragma unroll 8
        for (int r = 0; r < kRows; ++r) {
          const int c = r + tid - (kRows - 1);
          if (c >= 0 && c < kBwdRows) acc += sS[r * (kBwdRows + 1) + c];
        }
        diag[tid] = acc;
      }
      __syncthreads();
      if (tid < rel.nseg) {
        const int lo = rs.start[tid] <= d0 ? 0 : min(rs.start[tid] - d0, kDist);
        const int hi = rs.start[tid + 1] > d0 + kDist - 1 ? kDist - 1 : rs.start[tid + 1] - 1 - d0;
        for (int e = lo; e <= hi; ++e) own += diag[e];
      }
    }
  }
  if (nt > 0) {
    __syncthreads();
    flush_far();
  }
  if (tid < rel.nseg) rel.partial[(bh * gridDim.x + blockIdx.x) * rel.nseg + tid] = own;
  float* out = p.dQ + b * p.st[5][0] + h * p.st[5][1];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (q0 + r_loc[i] < p.Nq)
      store_row<DP, kVec>(out + static_cast<int64_t>(q0 + r_loc[i]) * p.st[5][2], dq, i, t, p.d_k,
                          p.scale);
}

template <int DP>
__host__ __device__ constexpr int dkdv_smem() {
  return ((2 * kRows + 2 * kBwdRows) * pitch_of(DP) + 2 * kBwdRows + 96) * 4 +
         static_cast<int>(sizeof(RelShared));
}

// One CTA per 64 keys: dK and dV from steps of 32 queries (after the dq kernel, which leaves D).
template <int DP, bool kVec>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 3 : 2)
    sdpa_rel_dkdv_f32_kernel(const RelF32 p, const __grid_constant__ RelBias rel) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  constexpr int kP = pitch_of(DP), kNT = kBwdRows / 8, kDist = kRows + kBwdRows - 1;
  extern __shared__ float smem[];
  float* sK = smem;                   // [64][kP]
  float* sV = sK + kRows * kP;        // [64][kP]
  float* sQ = sV + kRows * kP;        // [32][kP]
  float* sG = sQ + kBwdRows * kP;     // [32][kP]: dO
  float* sD = sG + kBwdRows * kP;     // [32]
  float* sL = sD + kBwdRows;          // [32]
  float* table = sL + kBwdRows;       // [95]
  RelShared& rs = *reinterpret_cast<RelShared*>(table + 96);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z, k0 = static_cast<int>(blockIdx.x) * kRows;
  const int L = keys_of(p, b);
  const int64_t bh = static_cast<int64_t>(b) * p.H + h;
  const float* qb = p.Q + b * p.st[0][0] + h * p.st[0][1];
  const float* gb = p.dO + b * p.st[4][0] + h * p.st[4][1];
  const int i0 = p.mask == 1 ? k0 / kBwdRows : 0;  // the first query step that sees a key
  const int ni = k0 < L ? (p.Nq + kBwdRows - 1) / kBwdRows : 0;
  load_rows<DP, kVec, kRows>(sK, p.K + b * p.st[1][0] + h * p.st[1][1], p.st[1][2], k0, L, p.d_k);
  load_rows<DP, kVec, kRows>(sV, p.V + b * p.st[2][0] + h * p.st[2][1], p.st[2][2], k0, L, p.d_v);
  copy_commit();
  for (int s = tid; s <= kRelMaxSeg; s += kThreads) rel_load(rs, rel, h, s, 1.f);
  const int key[2] = {k0 + 16 * warp + g, k0 + 16 * warp + g + 8};
  float dk[DP / 8][4] = {}, dv[DP / 8][4] = {};
  int seg_start = INT_MAX;
  float seg_bias = 0.f;
  for (int i = i0; i < ni; ++i) {
    __syncthreads();  // the previous step is done with the buffers (the first: rs is there)
    const int q0 = i * kBwdRows;
    load_rows<DP, kVec, kBwdRows>(sQ, qb, p.st[0][2], q0, p.Nq, p.d_k);
    load_rows<DP, kVec, kBwdRows>(sG, gb, p.st[4][2], q0, p.Nq, p.d_v);
    copy_commit();
    if (tid < kBwdRows) {
      sD[tid] = q0 + tid < p.Nq ? p.Dv[bh * p.Nq + q0 + tid] : 0.f;
      sL[tid] = q0 + tid < p.Nq ? p.lse[bh * p.Nq + q0 + tid] : INFINITY;
    }
    const int d0 = k0 - (q0 + kBwdRows - 1);  // distances d0 + e, e = key row + 31 - query
    if (d0 + kDist - 1 < seg_start) {
      const int seg = rel_segment(rs, rel_steps(rel.nseg), d0 + kDist - 1);
      seg_start = rs.start[seg];
      seg_bias = rs.bias[seg];
    }
    const bool near = d0 < seg_start;
    if (near && tid < kDist) table[tid] = rs.bias[rel_segment(rs, rel_steps(rel.nseg), d0 + tid)];
    copy_wait<0>();
    __syncthreads();
    float s[kNT][4], ds[kNT][4];
    product_d<DP, kNT>(s, sK, 16 * warp, sQ, g, t);
    product_d<DP, kNT>(ds, sV, 16 * warp, sG, g, t);
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 8 * n + 2 * t + (e & 1), j = key[e >> 1];
        const float bias = near ? table[j - k0 - c + kBwdRows - 1] : seg_bias;
        const bool ok = j < L && (p.mask != 1 || j <= q0 + c);
        s[n][e] = weight(s[n][e], p.scale, bias, sL[c], ok);
        ds[n][e] = s[n][e] * (ds[n][e] - sD[c]);
      }
    product_rows<DP, kNT>(dv, s, sG, g, t);
    product_rows<DP, kNT>(dk, ds, sQ, g, t);
  }
  copy_wait<0>();  // K and V, where no step waited for them
  float* ok = p.dK + b * p.st[6][0] + h * p.st[6][1];
  float* ov = p.dV + b * p.st[7][0] + h * p.st[7][1];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (key[e] < p.Nk) {
      store_row<DP, kVec>(ok + static_cast<int64_t>(key[e]) * p.st[6][2], dk, e, t, p.d_k, p.scale);
      store_row<DP, kVec>(ov + static_cast<int64_t>(key[e]) * p.st[7][2], dv, e, t, p.d_v, 1.f);
    }
}

// the gradient of the table alone, one block per head
__global__ void __launch_bounds__(kRelGradThreads)
    rel_table_grad_kernel(const __grid_constant__ RelBias rel, void* dtable, int B, int tiles) {
  pdl_launch_dependents();
  pdl_wait();  // the partial sums are complete from here on
  rel_table_grad(rel, dtable, B, tiles, static_cast<int>(blockIdx.x));
}

template <class F>
cudaError_t go(F* kernel, dim3 grid, int smem, const RelF32& p, const RelBias& rel,
               cudaStream_t s) {
  cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), smem, nullptr);
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
  p.H = a.H; p.Nq = a.Nq; p.Nk = a.Nk; p.d_k = a.d_k; p.d_v = a.d_v;
  p.mask = a.mask;
  p.key_len = a.key_len;
  p.scale = a.scale;
  const bool vec = quads(a.Q, p.st[0], a.d_k) && quads(a.K, p.st[1], a.d_k) &&
                   quads(a.V, p.st[2], a.d_v) && quads(a.O, p.st[3], a.d_v);
  const dim3 grid((a.Nq + kRows - 1) / kRows, a.H, a.B);
  if (a.d_k <= 64 && a.d_v <= 64)
    return vec ? go(sdpa_rel_f32_kernel<64, true>, grid, fwd_smem<64>(), p, rel, s)
               : go(sdpa_rel_f32_kernel<64, false>, grid, fwd_smem<64>(), p, rel, s);
  return vec ? go(sdpa_rel_f32_kernel<128, true>, grid, fwd_smem<128>(), p, rel, s)
             : go(sdpa_rel_f32_kernel<128, false>, grid, fwd_smem<128>(), p, rel, s);
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
  p.O = static_cast<const float*>(a.O);
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
  p.H = a.H; p.Nq = a.Nq; p.Nk = a.Nk; p.d_k = a.d_k; p.d_v = a.d_v;
  p.mask = a.mask;
  p.key_len = a.key_len;
  p.scale = a.scale;
  const bool small = a.d_k <= 64 && a.d_v <= 64;
  const dim3 gq((a.Nq + kRows - 1) / kRows, a.H, a.B), gk((a.Nk + kRows - 1) / kRows, a.H, a.B);
  cudaError_t e;
  if (small)
    e = vec ? go(sdpa_rel_dq_f32_kernel<64, true>, gq, dq_smem<64>(), p, rel, s)
            : go(sdpa_rel_dq_f32_kernel<64, false>, gq, dq_smem<64>(), p, rel, s);
  else
    e = vec ? go(sdpa_rel_dq_f32_kernel<128, true>, gq, dq_smem<128>(), p, rel, s)
            : go(sdpa_rel_dq_f32_kernel<128, false>, gq, dq_smem<128>(), p, rel, s);
  if (e != cudaSuccess) return e;
  if (small)
    e = vec ? go(sdpa_rel_dkdv_f32_kernel<64, true>, gk, dkdv_smem<64>(), p, rel, s)
            : go(sdpa_rel_dkdv_f32_kernel<64, false>, gk, dkdv_smem<64>(), p, rel, s);
  else
    e = vec ? go(sdpa_rel_dkdv_f32_kernel<128, true>, gk, dkdv_smem<128>(), p, rel, s)
            : go(sdpa_rel_dkdv_f32_kernel<128, false>, gk, dkdv_smem<128>(), p, rel, s);
  return e == cudaSuccess ? launch_rel_table_grad(rel, dtable, a.B, rel_bwd_tiles(a.Nq, a.Nk, 0), s)
                          : e;
}

cudaError_t launch_rel_table_grad(const RelBias& rel, void* dtable, int B, int tiles,
                                  cudaStream_t s) {
  return launch_pdl(rel_table_grad_kernel, dim3(rel.H), dim3(kRelGradThreads), 0, s, rel, dtable, B,
                    tiles);
}

}  // namespace mha
