// sdpa_rel_decode.cu -- one generation step against a key/value cache with a learned relative
// position bias:
//   O[b,h,r] = softmax_j(Q[b,h,r] . K[b,h,j] scale + t(j - (L_b - Nq + r)), allowed) V[b,h,j]
// for the Nq <= 16 newest of L_b cached positions (t: rel_bias.cuh; allowed as in sdpa_decode.cu).
//
// Bound by reading the cache once.  A CTA takes a run of positions of one head and its four warps
// take turns at tiles of it (16 positions in bf16, 8 in fp32), each with a running maximum and sum
// of its own.  All 16 rows of queries go through one warp product (bf16: m16n8k16; fp32: m16n8k8 in
// two tf32 terms, mma_tf32.cuh), whose operands come straight from the cache into registers: the
// order of the inner dimension is free, so a lane's fragments are 16-byte pieces of rows,
//   scores: lane (g, t) reads pieces t, t + 4, .. of position g (whole 32-byte sectors per row), and
//     takes neighbouring values as the fragment's inner positions;
//   values: lane (g, t) reads piece g (fp32: g, g + 8, ..) of the positions whose scores it holds
//     (columns 2 t and 2 t + 1 of the score fragments), so the weights need no exchange.
// The next tile's loads are in flight while one is computed; nothing goes through shared memory but
// the warps' results at the end.  A row's reference for the exponentials is raised (and its sums
// rescaled) only when a score passes it by 2^8.  A tile within one segment of distances adds a
// constant; only tiles that a border crosses look distances up, score by score.  Runs of one head
// meet in a second launch; one run writes O itself.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "device_common.cuh"
#include "launchers.h"
#include "mma_tf32.cuh"
#include "rel_bias.cuh"

namespace mha {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;  // a score may pass its row's reference by this (in powers of two)

struct Params {
  int H, Nq, Lmax, causal, d_k, d_v;
  int chunk, n_split;        // positions of a CTA, CTAs of a head
  const int32_t* cache_len;
  float scale;
  const void *Q, *K, *V;
  void* O;
  int64_t sq[3], sk[3], sv[3], so[3];
  float* part;               // [B, H, n_split, Nq, DP] sums, then [B, H, n_split, Nq] {m, l}
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the softmax state of a lane's two rows, g and g + 8, in powers of two
template <int NO>
struct Rows {
  float m[2], l[2];
  float o[NO][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < NO; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
  }
  // scores x (NS fragments, -inf where not allowed; `unit` of them make a power of two) -> weights
  template <int NS>
  __device__ __forceinline__ void weigh(float (&x)[NS][4], float unit) {
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[i >> 1] = fmaxf(mx[i >> 1], x[n][i]);
    const float slack = kSlack / unit;
    if (__any_sync(0xffffffffu, mx[0] > m[0] + slack || mx[1] > m[1] + slack)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        const float m_new = fmaxf(m[i], mx[i]);
        const float a = m_new == -INFINITY ? 1.f : ex2_approx((m[i] - m_new) * unit);
        m[i] = m_new;
        l[i] *= a;
#pragma unroll
        for (int n = 0; n < NO; ++n) {
          o[n][2 * i] *= a;
          o[n][2 * i + 1] *= a;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ref = m[i >> 1] == -INFINITY ? 0.f : m[i >> 1];
        x[n][i] = ex2_approx((x[n][i] - ref) * unit);
        l[i >> 1] += x[n][i];
      }
  }
};

// what is common to the tiles of a warp: allowed positions and the bias
struct Where {
  int L, Nq, limit[2];  // rows g, g + 8 see positions up to limit
  int row[2];
  int seg_next, steps;
  float seg_bias;
  __device__ __forceinline__ Where(const Params& p, const RelBias& rel, int L_, int end, int g) {
    L = L_;
    steps = rel_steps(rel.nseg);
    Nq = p.Nq;
    seg_next = INT_MIN;
    seg_bias = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      row[i] = g + 8 * i;
      limit[i] = row[i] < Nq ? min(p.causal ? L - Nq + row[i] : L - 1, end - 1) : -1;
    }
  }
  // scale, bias and mask of a tile of 8 NS positions from j0 on
  template <int NS>
  __device__ __forceinline__ void scores(float (&x)[NS][4], const RelShared& rs, int j0, int t,
                                         float c) {
    const int d0 = j0 - (L - 1);  // the tile's distances lie in d0 .. d0 + 8 NS - 1 + Nq - 1
    if (d0 >= seg_next) {
      const int seg = rel_segment(rs, steps, d0);
      seg_next = rs.start[seg + 1];
      seg_bias = rs.bias[seg];
    }
    const bool near = d0 + 8 * NS + Nq - 2 >= seg_next;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const int j = j0 + 8 * n + 2 * t;
      float bias[4] = {seg_bias, seg_bias, seg_bias, seg_bias};
      if (near) {
        const int d = j - (L - Nq + row[0]);
        const int at[4] = {d, d + 1, d - 8, d - 7};  // rows g and g + 8
        int seg[4];
        rel_segments<4>(rs, steps, at, seg);
#pragma unroll
        for (int i = 0; i < 4; ++i) bias[i] = rs.bias[seg[i]];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[n][i] = j + (i & 1) <= limit[i >> 1] ? fmaf(x[n][i], c, bias[i]) : -INFINITY;
    }
  }
};

// The warps' results in shared memory (so: [kWarps][Nq][DP], sml: [kWarps][Nq] {m, l}) leave as O, or
// as this run's part.
template <int DP, typename T>
__device__ __forceinline__ void join_warps(const Params& p, const float* so, const float* sml,
                                           float unit, int64_t bh, int split, T* O) {
  const int Nq = p.Nq;
  __syncthreads();
  for (int e = threadIdx.x; e < Nq * DP; e += kThreads) {  // (a sum of 0: no key; NaN stays NaN)
    const int row = e / DP, d = e % DP;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sml[(w * Nq + row) * 2]);
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = ex2_approx((sml[(w * Nq + row) * 2] - ref) * unit);
      l = fmaf(a, sml[(w * Nq + row) * 2 + 1], l);
      o = fmaf(a, so[(w * Nq + row) * DP + d], o);
    }
    if (p.n_split == 1) {
      if (d < p.d_v) O[row * p.so[2] + d] = static_cast<T>(l == 0.f ? 0.f : o / l);
    } else {
      const int64_t i = (bh * p.n_split + split) * Nq + row;
      p.part[i * DP + d] = o;
      if (d == 0) {
        float* ml = p.part + static_cast<int64_t>(gridDim.z) * p.H * p.n_split * Nq * DP + 2 * i;
        ml[0] = m;
        ml[1] = l;
      }
    }
  }
}

// The fragments of each warp go to shared memory; col(n, i): the column of o[n][i] in its row.
template <int DP, typename T, int NO, class Col>
__device__ __forceinline__ void finish(const Params& p, Rows<NO>& r, float* so, float* sml,
                                       float unit, int warp, int lane, int64_t bh, int split, T* O,
                                       Col col) {
  const int g = lane >> 2, t = lane & 3, Nq = p.Nq;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.l[i] += __shfl_xor_sync(0xffffffffu, r.l[i], 1);
    r.l[i] += __shfl_xor_sync(0xffffffffu, r.l[i], 2);
    const int row = g + 8 * i;
    if (row < Nq) {
      if (t == 0) {
        sml[(warp * Nq + row) * 2] = r.m[i];
        sml[(warp * Nq + row) * 2 + 1] = r.l[i];
      }
#pragma unroll
      for (int n = 0; n < NO; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) so[(warp * Nq + row) * DP + col(n, e)] = r.o[n][2 * i + e];
    }
  }
  join_warps<DP>(p, so, sml, unit, bh, split, O);
}

// a run that holds no cached position
template <int DP, typename T>
__device__ __forceinline__ void finish_empty(const Params& p, int64_t bh, int split, T* O) {
  if (p.n_split == 1) {
    for (int e = threadIdx.x; e < p.Nq * p.d_v; e += kThreads)
      O[e / p.d_v * p.so[2] + e % p.d_v] = static_cast<T>(0.f);
  } else if (static_cast<int>(threadIdx.x) < p.Nq) {  // its sums are not read
    const int64_t i = (bh * p.n_split + split) * p.Nq + threadIdx.x;
    float* ml =
        p.part + static_cast<int64_t>(gridDim.z) * p.H * p.n_split * p.Nq * DP + 2 * i;
    ml[0] = -INFINITY;
    ml[1] = 0.f;
  }
}

// ============================================================================ bf16, d = 64
struct TileBf16 {
  uint4 k[4], v[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* K, const __nv_bfloat16* V, int64_t sk,
                                       int64_t sv, int j0, int end, int g, int t) {
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = j0 + 8 * n + g;
      const uint4* r = reinterpret_cast<const uint4*>(K + j * sk);
      k[2 * n] = j < end ? __ldcs(r + t) : none;
      k[2 * n + 1] = j < end ? __ldcs(r + t + 4) : none;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + 8 * (i >> 1) + 2 * t + (i & 1);
      v[i] = j < end ? __ldcs(reinterpret_cast<const uint4*>(V + j * sv) + g) : none;
    }
  }
};

__global__ void __launch_bounds__(kThreads, 4)
    sdpa_rel_decode_bf16_kernel(const __grid_constant__ Params p,
                                const __grid_constant__ RelBias rel) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  __shared__ RelShared rs;
  __shared__ float sml[kWarps * kDecodeMaxQ * 2];
  __shared__ __align__(16) float so[kWarps * kDecodeMaxQ * 64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * p.H + h;
  const int L = min(max(__ldg(p.cache_len + b), 0), p.Lmax);
  const int begin = split * p.chunk, end = min(begin + p.chunk, L);
  __nv_bfloat16* O = static_cast<__nv_bfloat16*>(p.O) + b * p.so[0] + h * p.so[1];
  if (begin >= L) return finish_empty<64>(p, bh, split, O);
  const __nv_bfloat16* K = static_cast<const __nv_bfloat16*>(p.K) + b * p.sk[0] + h * p.sk[1];
  const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(p.V) + b * p.sv[0] + h * p.sv[1];
  TileBf16 tile;
  int j0 = begin + 16 * warp;
  tile.load(K, V, p.sk[2], p.sv[2], j0, end, g, t);
  for (int s = threadIdx.x; s <= kRelMaxSeg; s += kThreads) rel_load(rs, rel, h, s, kLog2e);
  uint32_t qf[4][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i;
    uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
    if (r < p.Nq) {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.Q) +
                                                      b * p.sq[0] + h * p.sq[1] + r * p.sq[2]);
      x = __ldg(q + t);
      y = __ldg(q + t + 4);
    }
    qf[0][i] = x.x; qf[0][2 + i] = x.y; qf[1][i] = x.z; qf[1][2 + i] = x.w;
    qf[2][i] = y.x; qf[2][2 + i] = y.y; qf[3][i] = y.z; qf[3][2 + i] = y.w;
  }
  __syncthreads();
  const float c = p.scale * kLog2e;
  Where where(p, rel, L, end, g);
  Rows<8> r;
  r.clear();
  for (; j0 < end; j0 += 16 * kWarps) {
    float x[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] = 0.f;
      const uint4 lo = tile.k[2 * n], hi = tile.k[2 * n + 1];
      mma_bf16(x[n], qf[0], lo.x, lo.y);
      mma_bf16(x[n], qf[1], lo.z, lo.w);
      mma_bf16(x[n], qf[2], hi.x, hi.y);
      mma_bf16(x[n], qf[3], hi.z, hi.w);
    }
    const uint4 v[4] = {tile.v[0], tile.v[1], tile.v[2], tile.v[3]};
    tile.load(K, V, p.sk[2], p.sv[2], j0 + 16 * kWarps, end, g, t);
    where.scores<2>(x, rs, j0, t, c);
    r.weigh<2>(x, 1.f);
    const uint32_t a[4] = {pack_bf16x2(x[0][0], x[0][1]), pack_bf16x2(x[0][2], x[0][3]),
                           pack_bf16x2(x[1][0], x[1][1]), pack_bf16x2(x[1][2], x[1][3])};
#pragma unroll
    for (int n = 0; n < 8; ++n) {  // column n of the lane's pieces: d = 8 g + n
      auto word = [n](const uint4& u) { return n < 2 ? u.x : n < 4 ? u.y : n < 6 ? u.z : u.w; };
      const uint32_t pick = n & 1 ? 0x7632u : 0x5410u;
      mma_bf16(r.o[n], a, __byte_perm(word(v[0]), word(v[1]), pick),
               __byte_perm(word(v[2]), word(v[3]), pick));
    }
  }
  finish<64>(p, r, so, sml, 1.f, warp, lane, bh, split, O,
             [t](int n, int e) { return 16 * t + 8 * e + n; });
}

// ============================================================================ fp32, d <= 128
template <int DP, bool kVec>
struct TileF32 {
  float4 k[DP / 16], v[2][DP / 32];
  __device__ __forceinline__ static float4 piece(const float* row, int c, int d, bool ok) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (kVec) {
      if (ok && c < d) x = __ldcs(reinterpret_cast<const float4*>(row + c));
    } else if (ok) {
      if (c < d) x.x = __ldcs(row + c);
      if (c + 1 < d) x.y = __ldcs(row + c + 1);
      if (c + 2 < d) x.z = __ldcs(row + c + 2);
      if (c + 3 < d) x.w = __ldcs(row + c + 3);
    }
    return x;
  }
  __device__ __forceinline__ void load(const float* K, const float* V, const Params& p, int j0,
                                       int end, int g, int t) {
    const int jk = j0 + g;
#pragma unroll
    for (int u = 0; u < DP / 16; ++u)
      k[u] = piece(K + jk * p.sk[2], 4 * (t + 4 * u), p.d_k, jk < end);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int jv = j0 + 2 * t + i;
#pragma unroll
      for (int u = 0; u < DP / 32; ++u)
        v[i][u] = piece(V + jv * p.sv[2], 4 * (g + 8 * u), p.d_v, jv < end);
    }
  }
};

template <int DP, bool kVec>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 4 : 2)
    sdpa_rel_decode_f32_kernel(const __grid_constant__ Params p,
                               const __grid_constant__ RelBias rel) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  __shared__ RelShared rs;
  __shared__ float sml[kWarps * kDecodeMaxQ * 2];
  // the queries' fragments in two terms, [DP / 8][32 lanes][hi 4, lo 4]; at the end the warps' sums
  constexpr int kShared = kWarps * kDecodeMaxQ * DP;
  static_assert(kShared >= DP / 8 * 32 * 8, "");
  __shared__ __align__(16) float so[kShared];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * p.H + h;
  const int L = min(max(__ldg(p.cache_len + b), 0), p.Lmax);
  const int begin = split * p.chunk, end = min(begin + p.chunk, L);
  float* O = static_cast<float*>(p.O) + b * p.so[0] + h * p.so[1];
  if (begin >= L) return finish_empty<DP>(p, bh, split, O);
  const float* K = static_cast<const float*>(p.K) + b * p.sk[0] + h * p.sk[1];
  const float* V = static_cast<const float*>(p.V) + b * p.sv[0] + h * p.sv[1];
  TileF32<DP, kVec> tile;
  int j0 = begin + 8 * warp;
  tile.load(K, V, p, j0, end, g, t);
  for (int s = threadIdx.x; s <= kRelMaxSeg; s += kThreads) rel_load(rs, rel, h, s, 1.f);
  const float* Q = static_cast<const float*>(p.Q) + b * p.sq[0] + h * p.sq[1];
  for (int u = warp; u < DP / 16; u += kWarps) {
    const float4 x = TileF32<DP, kVec>::piece(Q + g * p.sq[2], 4 * (t + 4 * u), p.d_k, g < p.Nq);
    const float4 y =
        TileF32<DP, kVec>::piece(Q + (g + 8) * p.sq[2], 4 * (t + 4 * u), p.d_k, g + 8 < p.Nq);
    const Tf32FragA f[2] = {frag_a(x.x, y.x, x.y, y.y), frag_a(x.z, y.z, x.w, y.w)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4* at = reinterpret_cast<uint4*>(so) + ((2 * u + i) * 32 + lane) * 2;
      at[0] = make_uint4(f[i].hi[0], f[i].hi[1], f[i].hi[2], f[i].hi[3]);
      at[1] = make_uint4(f[i].lo[0], f[i].lo[1], f[i].lo[2], f[i].lo[3]);
    }
  }
  __syncthreads();
  auto frag = [&](int step) {
    const uint4* at = reinterpret_cast<const uint4*>(so) + (step * 32 + lane) * 2;
    const uint4 x = at[0], y = at[1];
    return Tf32FragA{{x.x, x.y, x.z, x.w}, {y.x, y.y, y.z, y.w}};
  };
  Where where(p, rel, L, end, g);
  Rows<DP / 8> r;
  r.clear();
  for (; j0 < end; j0 += 8 * kWarps) {
    float x[1][4], hi[4] = {}, lo[4] = {};
#pragma unroll
    for (int u = 0; u < DP / 16; ++u) {
      mma_f32(hi, lo, frag(2 * u), tile.k[u].x, tile.k[u].y);
      mma_f32(hi, lo, frag(2 * u + 1), tile.k[u].z, tile.k[u].w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[0][i] = hi[i] + lo[i];
    float4 v[2][DP / 32];
#pragma unroll
    for (int u = 0; u < DP / 32; ++u) {
      v[0][u] = tile.v[0][u];
      v[1][u] = tile.v[1][u];
    }
    tile.load(K, V, p, j0 + 8 * kWarps, end, g, t);
    where.template scores<1>(x, rs, j0, t, p.scale);
    r.template weigh<1>(x, kLog2e);
    const Tf32FragA a = frag_a(x[0][0], x[0][2], x[0][1], x[0][3]);
#pragma unroll
    for (int u = 0; u < DP / 32; ++u) {
      const float b0[4] = {v[0][u].x, v[0][u].y, v[0][u].z, v[0][u].w};
      const float b1[4] = {v[1][u].x, v[1][u].y, v[1][u].z, v[1][u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // one product deep: the small terms first, then the large
        float sum[4] = {};
        mma_f32(sum, sum, a, b0[e], b1[e]);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.o[4 * u + e][i] += sum[i];
      }
    }
  }
  __syncthreads();  // the queries' fragments are done with
  finish<DP>(p, r, so, sml, kLog2e, warp, lane, bh, split, O,
             [t](int n, int e) { return 32 * (n >> 2) + 8 * t + 4 * e + (n & 3); });
}

// ---- few queries: fused multiply-adds instead of products of 16 rows.  Lane (g, t) sums a quarter of
// position g's score (the quarters meet in two shuffles) and has the values' pieces of positions 2 t
// and 2 t + 1, whose weights it takes from their lanes; the four partial outputs meet at the end.
// Multiply-adds instead of splits and products of 16 mostly empty rows: 8 heads of 131072 positions 124
// us -> 81 (0.98 of the measured bandwidth); with 4 queries the two take the same time (69 and 71 us for
// 8 x 16 heads of 4096), so the products take over from 3.
template <int DP, bool kVec, int NQ>
__global__ void __launch_bounds__(kThreads, DP * NQ <= 64 ? 4 : DP * NQ <= 128 ? 3 : 2)
    sdpa_rel_decode_few_f32_kernel(const __grid_constant__ Params p,
                                   const __grid_constant__ RelBias rel) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  using Tile = TileF32<DP, kVec>;
  __shared__ RelShared rs;
  __shared__ float sml[kWarps * NQ * 2];
  __shared__ __align__(16) float so[kWarps * NQ * DP];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * p.H + h;
  const int L = min(max(__ldg(p.cache_len + b), 0), p.Lmax);
  const int begin = split * p.chunk, end = min(begin + p.chunk, L);
  float* O = static_cast<float*>(p.O) + b * p.so[0] + h * p.so[1];
  if (begin >= L) return finish_empty<DP>(p, bh, split, O);
  const float* K = static_cast<const float*>(p.K) + b * p.sk[0] + h * p.sk[1];
  const float* V = static_cast<const float*>(p.V) + b * p.sv[0] + h * p.sv[1];
  Tile tile;
  int j0 = begin + 8 * warp;
  tile.load(K, V, p, j0, end, g, t);
  for (int s = threadIdx.x; s <= kRelMaxSeg; s += kThreads) rel_load(rs, rel, h, s, 1.f);
  const float* Q = static_cast<const float*>(p.Q) + b * p.sq[0] + h * p.sq[1];
  float4 q[NQ][DP / 16];
  int limit[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    limit[i] = i < p.Nq ? min(p.causal ? L - p.Nq + i : L - 1, end - 1) : -1;
#pragma unroll
    for (int u = 0; u < DP / 16; ++u)
      q[i][u] = Tile::piece(Q + i * p.sq[2], 4 * (t + 4 * u), p.d_k, i < p.Nq);
  }
  __syncthreads();
  float m[NQ], l[NQ], o[NQ][DP / 8];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) o[i][d] = 0.f;
  }
  const int steps = rel_steps(rel.nseg);
  int seg_next = INT_MIN;
  float seg_bias = 0.f;
  for (; j0 < end; j0 += 8 * kWarps) {
    float x[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float a = 0.f, c = 0.f;
#pragma unroll
      for (int u = 0; u < DP / 16; ++u) {
        a = fmaf(q[i][u].x, tile.k[u].x, a);
        c = fmaf(q[i][u].y, tile.k[u].y, c);
        a = fmaf(q[i][u].z, tile.k[u].z, a);
        c = fmaf(q[i][u].w, tile.k[u].w, c);
      }
      x[i] = a + c;
    }
    float4 v[2][DP / 32];
#pragma unroll
    for (int u = 0; u < DP / 32; ++u) {
      v[0][u] = tile.v[0][u];
      v[1][u] = tile.v[1][u];
    }
    tile.load(K, V, p, j0 + 8 * kWarps, end, g, t);
    const int d0 = j0 - (L - 1);  // the tile's distances lie in d0 .. d0 + 7 + Nq - 1
    if (d0 >= seg_next) {
      const int seg = rel_segment(rs, steps, d0);
      seg_next = rs.start[seg + 1];
      seg_bias = rs.bias[seg];
    }
    const bool near = d0 + 6 + p.Nq >= seg_next;
    const int j = j0 + g;
    bool raise = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      x[i] += __shfl_xor_sync(0xffffffffu, x[i], 1);
      x[i] += __shfl_xor_sync(0xffffffffu, x[i], 2);
      float bias = seg_bias;
      if (near) bias = rs.bias[rel_segment(rs, steps, j - (L - p.Nq + i))];
      x[i] = j <= limit[i] ? fmaf(x[i], p.scale, bias) : -INFINITY;
      raise |= x[i] > m[i] + kSlack / kLog2e;
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        float top = fmaxf(m[i], x[i]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float a = top == -INFINITY ? 1.f : ex2_approx((m[i] - top) * kLog2e);
        m[i] = top;
        l[i] *= a;
#pragma unroll
        for (int d = 0; d < DP / 8; ++d) o[i][d] *= a;
      }
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const float w = ex2_approx((x[i] - (m[i] == -INFINITY ? 0.f : m[i])) * kLog2e);
      l[i] += w;  // the same in the four lanes of a position
      const float w0 = __shfl_sync(0xffffffffu, w, 8 * t), w1 = __shfl_sync(0xffffffffu, w, 8 * t + 4);
#pragma unroll
      for (int u = 0; u < DP / 32; ++u) {
        o[i][4 * u + 0] = fmaf(w0, v[0][u].x, fmaf(w1, v[1][u].x, o[i][4 * u + 0]));
        o[i][4 * u + 1] = fmaf(w0, v[0][u].y, fmaf(w1, v[1][u].y, o[i][4 * u + 1]));
        o[i][4 * u + 2] = fmaf(w0, v[0][u].z, fmaf(w1, v[1][u].z, o[i][4 * u + 2]));
        o[i][4 * u + 3] = fmaf(w0, v[0][u].w, fmaf(w1, v[1][u].w, o[i][4 * u + 3]));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) {
      o[i][d] += __shfl_xor_sync(0xffffffffu, o[i][d], 1);
      o[i][d] += __shfl_xor_sync(0xffffffffu, o[i][d], 2);
    }
    if (i < p.Nq) {
      if (lane == 0) {
        sml[(warp * p.Nq + i) * 2] = m[i];
        sml[(warp * p.Nq + i) * 2 + 1] = l[i];
      }
      if (t == 0) {
#pragma unroll
        for (int u = 0; u < DP / 32; ++u)
          *reinterpret_cast<float4*>(so + (warp * p.Nq + i) * DP + 32 * u + 4 * g) =
              make_float4(o[i][4 * u], o[i][4 * u + 1], o[i][4 * u + 2], o[i][4 * u + 3]);
      }
    }
  }
  join_warps<DP>(p, so, sml, kLog2e, bh, split, O);
}

// ============================================================================ the runs' results
// one block per (query row, head, batch element): DP columns x kJoinThreads / DP groups of runs, 1024
// threads for more than 32 runs, else 256
constexpr int kMaxSplit = 1024;

template <int DP, typename T, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads)
    sdpa_rel_join_kernel(const __grid_constant__ Params p, float unit) {
  pdl_launch_dependents();
  pdl_wait();  // the runs' results are complete from here on
  constexpr int kGroups = kJoinThreads / DP;
  __shared__ float w[kMaxSplit], red[kJoinThreads / 32], sum[kJoinThreads], total[kJoinThreads / 32];
  const int row = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int64_t bh = static_cast<int64_t>(b) * p.H + h;
  const int n = p.n_split;
  const float* ml = p.part + static_cast<int64_t>(gridDim.z) * p.H * n * p.Nq * DP;
  auto at = [&](int s) { return (bh * n + s) * p.Nq + row; };
  float m = -INFINITY;
  for (int s = tid; s < n; s += kJoinThreads) {
    w[s] = ml[2 * at(s)];
    m = fmaxf(m, w[s]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (tid % 32 == 0) red[tid / 32] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int i = 1; i < kJoinThreads / 32; ++i) m = fmaxf(m, red[i]);
  if (m == -INFINITY) m = 0.f;
  float l = 0.f;
  for (int s = tid; s < n; s += kJoinThreads) {
    w[s] = ex2_approx((w[s] - m) * unit);
    l = fmaf(w[s], ml[2 * at(s) + 1], l);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  if (tid % 32 == 0) total[tid / 32] = l;
  __syncthreads();
  l = total[0];
#pragma unroll
  for (int i = 1; i < kJoinThreads / 32; ++i) l += total[i];
  float o = 0.f;
  const int d = tid % DP;
#pragma unroll 8
  for (int s = tid / DP; s < n; s += kGroups)
    if (w[s] > 0.f) o = fmaf(w[s], p.part[at(s) * DP + d], o);
  sum[tid] = o;
  __syncthreads();
  if (tid < p.d_v) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) o += sum[i * DP + tid];
    T* O = static_cast<T*>(p.O) + b * p.so[0] + h * p.so[1] + row * p.so[2];
    O[tid] = static_cast<T>(l == 0.f ? 0.f : o / l);
  }
}

// Runs of a head and positions of a run (a multiple of 64, 16 for each warp).  A round of CTAs that fit
// on the GPU at once takes about the time of a run's positions and 96 more (start and the warps' join),
// the second launch that of 150 and of some per run.  Of 1 to 8 full rounds the most whose time is within
// 8% of the least are taken: caches that are not full leave short runs better balanced.  Measured (us,
// full caches / lengths drawn evenly): 64 x 16 heads of 4096 in bf16 168 / 88 with the 4 runs taken,
// 176 / 92 with 2, 185 / 101 with 16; 8 x 16 heads of 16384 with 4 queries 88 / 55 with 19, 107 / 57
// with 6; 16 x 8 heads of 4096 31 / 18 with 8, 29 / 23 with 4.
void plan(int B, int H, int Nq, int Lmax, int dp, int dtype, int* chunk, int* n_split) {
  const int64_t heads = static_cast<int64_t>(B) * H;
  const int64_t fit = 152 * (dtype == 1 ? 4 : dp == 64 ? (Nq == 2 ? 3 : 4) : (Nq == 1 ? 3 : 2));
  constexpr int kRounds = 8;
  int64_t runs[kRounds], positions[kRounds], cost[kRounds], least = -1;
  for (int i = 0; i < kRounds; ++i) {
    int64_t n = std::max<int64_t>(1, (i + 1) * fit / heads);
    n = std::min<int64_t>({n, (Lmax + 63) / 64, kMaxSplit});
    const int64_t c = ((Lmax + n - 1) / n + 63) / 64 * 64;
    n = (Lmax + c - 1) / c;
    cost[i] = (heads * n + fit - 1) / fit * (c + 96) + (n > 1 ? 150 + n * (Nq + 3) / 10 : 0);
    runs[i] = n;
    positions[i] = c;
    if (least < 0 || cost[i] < least) least = cost[i];
  }
  int i = kRounds - 1;
  while (cost[i] * 100 > least * 108) --i;
  *chunk = static_cast<int>(positions[i]);
  *n_split = static_cast<int>(runs[i]);
}

int padded(int dtype, int d_k, int d_v) { return dtype == 1 || (d_k <= 64 && d_v <= 64) ? 64 : 128; }

}  // namespace

size_t rel_decode_workspace(int B, int H, int Nq, int Lmax, int d_k, int d_v, int dtype) {
  const int dp = padded(dtype, d_k, d_v);
  int chunk, n;
  plan(B, H, Nq, Lmax, dp, dtype, &chunk, &n);
  return n == 1 ? 0 : static_cast<size_t>(B) * H * n * Nq * (dp + 2) * sizeof(float);
}

cudaError_t launch_sdpa_rel_decode(const RelDecodeArgs& a, const RelBias& rel, int dtype,
                                   float* part, cudaStream_t s) {
  Params p = {};
  p.H = a.H; p.Nq = a.Nq; p.Lmax = a.Lmax; p.causal = a.causal; p.d_k = a.d_k; p.d_v = a.d_v;
  const int dp = padded(dtype, a.d_k, a.d_v);
  plan(a.B, a.H, a.Nq, a.Lmax, dp, dtype, &p.chunk, &p.n_split);
  p.cache_len = a.cache_len;
  p.scale = a.scale;
  p.Q = a.Q; p.K = a.K; p.V = a.V; p.O = a.O;
  for (int i = 0; i < 3; ++i) {
    p.sq[i] = a.st[0][i];
    p.sk[i] = a.st[1][i];
    p.sv[i] = a.st[2][i];
    p.so[i] = a.st[3][i];
  }
  p.part = part;
  const dim3 grid(p.n_split, a.H, a.B), rows(a.Nq, a.H, a.B);
  auto go = [&](auto kernel, auto join, auto join_many, float unit) {
    cudaError_t e = launch_pdl(kernel, grid, dim3(kThreads), 0, s, p, rel);
    if (e == cudaSuccess && p.n_split > 32)
      e = launch_pdl(join_many, rows, dim3(1024), 0, s, p, unit);
    else if (e == cudaSuccess && p.n_split > 1)
      e = launch_pdl(join, rows, dim3(256), 0, s, p, unit);
    return e;
  };
  if (dtype == 1)
    return go(sdpa_rel_decode_bf16_kernel, sdpa_rel_join_kernel<64, __nv_bfloat16, 256>,
              sdpa_rel_join_kernel<64, __nv_bfloat16, 1024>, 1.f);
  bool vec = a.d_k % 4 == 0 && a.d_v % 4 == 0;
  const void* ptr[3] = {a.Q, a.K, a.V};
  for (int t = 0; t < 3; ++t) {
    vec = vec && reinterpret_cast<uintptr_t>(ptr[t]) % 16 == 0;
    for (int i = 0; i < 3; ++i) vec = vec && a.st[t][i] % 4 == 0;
  }
  auto go_f32 = [&](auto dim, auto quads) {
    constexpr int DP = decltype(dim)::value;
    constexpr bool kVec = decltype(quads)::value;
    auto f = [&](auto kernel) {
      return go(kernel, sdpa_rel_join_kernel<DP, float, 256>, sdpa_rel_join_kernel<DP, float, 1024>,
                kLog2e);
    };
    if (a.Nq == 1) return f(sdpa_rel_decode_few_f32_kernel<DP, kVec, 1>);
    if (a.Nq == 2) return f(sdpa_rel_decode_few_f32_kernel<DP, kVec, 2>);
    return f(sdpa_rel_decode_f32_kernel<DP, kVec>);
  };
  using std::integral_constant;
  if (dp == 64)
    return vec ? go_f32(integral_constant<int, 64>{}, std::true_type{})
               : go_f32(integral_constant<int, 64>{}, std::false_type{});
  return vec ? go_f32(integral_constant<int, 128>{}, std::true_type{})
             : go_f32(integral_constant<int, 128>{}, std::false_type{});
}

}  // namespace mha
