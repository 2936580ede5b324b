// sdpa_decode_q8.cu -- attention of a few new queries against an 8-bit key/value cache (see
// q8_common.cuh for the codes and scales), optionally adding every cached position's attention
// weight to a running total:
//   O[b,h,i] = sum_j p_ij v_j,  p_i = softmax_j(q_i . k_j * scale, allowed),
//   weights[b,g,j] += sum over the heads h of group g and the queries i of p_ij
// with k_j, v_j = code * scale of the block; allowed: j < L_b and, causal, j <= L_b - Nq + i.
// Head h reads the cache of head h / (H / Hkv); the G * Nq query rows that share a cache head
// are the rows of one product.
//
// Bound by reading the codes from HBM: 128 bytes per position and head.  Hence
//   - one pass over the cache; the running maximum and sum of the softmax in fp32 registers;
//   - all (head, 32-position tile) pairs of the batch laid out in one line and cut into equal
//     runs, one per warp of a grid that just fills the GPU, so sequences of any mix of lengths
//     keep every SM busy to the end, and a run is long enough that partial results are few;
//   - every warp streams its tiles through a ring of its own (TMA, one mbarrier per slot): no
//     block-wide barrier in the loop, 12 KB in flight per warp;
//   - the products on the tensor cores (mma.sync m16n8k16, fp16 operands, fp32 sums), the cache
//     as the operand with 16 rows and the queries as the one with 8 columns: S^T = K Q^T and
//     O^T = V^T P^T, since there are often no more than 8 query rows.  tcgen05 would want 64
//     rows or more and the codes staged a second time as 16-bit operands.  Codes become fp16
//     exactly, in registers, straight into the operand layout: the order of a product's inner
//     dimension is free, so lane t of a quad takes the 16 consecutive values 16t.. of a key, and
//     of a value row the 8 columns 8g.. for its lane group g, and only P is transposed, 8 x 8
//     at a time (movmatrix);
//   - the scales stay out of the operands: a key's multiplies its score, a value's enters the
//     exponent (p_j = 2^(x_j + log2 s_j - m)) and the softmax sum takes p_j / s_j.  With m the
//     maximum of x_j + log2 s_j the weights p_j that meet the value codes lie in [0, 2^13],
//     within fp16 whatever the scales are.
// Precision: scores, statistics and sums are fp32.  Queries are scaled by a power of two (their
// row's largest value to [2^13, 2^14)) and rounded to fp16, which holds every bf16 significand;
// fp32 queries and weights are split into two fp16 terms (22 bits) and their products done
// twice, each inner step's part of a score and each tile's PV summed apart and added in fp32
// (the tensor cores' own accumulation truncates).
// Runs end at heads' ends: each piece leaves (O, m, l) in the workspace, and a second launch
// joins a row's pieces, and adds the weights 2^(x_ij - m_i) / l_i from the scores that the first
// one stored.  No atomics: one order of sums.
// Every wait is bounded.
#include <cuda_bf16.h>

#include <algorithm>

#include "launchers.h"
#include "q8_common.cuh"

namespace mha {
namespace {

constexpr int kD = 64;
constexpr int kTile = 32;                  // positions per tile
constexpr int kTileBytes = kTile * kD;     // 2 KB of K, 2 KB of V
constexpr int kStages = 3;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kSmemBytes = 1024 + kWarps * kStages * (2 * kTileBytes + 8);
constexpr int kErrTimeout = -6;
constexpr int kSiteDecodeQ8 = 33;
constexpr float kOffset = 13.f;            // weights that meet the codes: 2^13 at most

// How the rows of a cache head are cut: groups of 8 * NR rows, NR column tiles of the products
struct RowPlan {
  int R, NR, RG, RS;  // rows per cache head, column tiles and groups, rows stored per piece
};
RowPlan row_plan(int H, int Hkv, int Nq, int dtype) {
  RowPlan p;
  p.R = H / Hkv * Nq;
  // the column tiles of a group share each converted operand; fp32's second terms leave the
  // registers for two, bf16 for four
  p.NR = p.R <= 8 ? 1 : p.R <= 16 || dtype != 1 ? 2 : 4;
  p.RG = (p.R + 8 * p.NR - 1) / (8 * p.NR);
  p.RS = std::min(p.R, 8 * p.NR);
  return p;
}
// blocks of the first launch that share an SM: two at up to 128 registers a thread
constexpr int blocks_per_sm(int terms, int nr) { return terms * nr <= 2 ? 2 : 1; }
// warps of its grid at most, as far as the workspace goes (a GB300 has 152 SMs)
constexpr int max_workers(int terms, int nr) { return 160 * kWarps * blocks_per_sm(terms, nr); }

struct Params {
  DecodeQ8Args a;
  RowPlan rp;
  int workers;        // warps of the first launch's grid
  float* part;        // [slots][RS][64] unnormalised O
  float* stat;        // [slots][RS][2] m, l
  float* scores;      // [B][Hkv][R][Lpad] x in base-2 units (-inf: excluded); null: not kept
  int64_t Lpad;
  int* status;
  uint64_t timeout_ns;
};

__device__ __forceinline__ int cached(const DecodeQ8Args& a, int b) {
  return min(max(__ldg(a.cache_len + b), 0), a.Lmax);
}
__device__ __forceinline__ int tiles_of(int L) { return (L + kTile - 1) / kTile; }

// Sums over batch elements by a whole warp: tiles of all, and of those before `b`
__device__ __forceinline__ void tile_sums(const DecodeQ8Args& a, int b, int64_t* before,
                                          int64_t* total) {
  const int lane = threadIdx.x & 31;
  int64_t all = 0, pre = 0;
  for (int x = lane; x < a.B; x += 32) {
    const int t = tiles_of(cached(a, x));
    all += t;
    pre += x < b ? t : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    pre += __shfl_xor_sync(0xffffffffu, pre, o);
  }
  *before = pre;
  *total = all;
}
// batch element that holds tile x of the line (x < total * per), and the tiles before it
__device__ __forceinline__ int find_batch(const DecodeQ8Args& a, int64_t x, int64_t per,
                                          int64_t* before) {
  const int lane = threadIdx.x & 31;
  int64_t base = 0;
  for (int x0 = 0;; x0 += 32) {
    const int b = x0 + lane;
    const int64_t n = b < a.B ? tiles_of(cached(a, b)) * per : 0;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, base + incl > x);
    if (m != 0) {
      const int src = __ffs(m) - 1;
      *before = base + __shfl_sync(0xffffffffu, incl - n, src);
      return x0 + src;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    if (x0 + 32 >= a.B) {  // past the end: not reached for x < total
      *before = base;
      return a.B;
    }
  }
}
// run of worker w of W over T tiles, and the worker of tile x (W <= T: no run is empty)
__device__ __forceinline__ int64_t run_start(int64_t w, int64_t T, int64_t W) { return w * T / W; }
__device__ __forceinline__ int64_t worker_of(int64_t x, int64_t T, int64_t W) {
  return ((x + 1) * W - 1) / T;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// four codes to two fp16 pairs (exact)
template <int QT>
__device__ __forceinline__ void codes_to_half(uint32_t u, uint32_t& h0, uint32_t& h1) {
  if constexpr (QT == kE4m3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(u));
  } else {
    // code + 128 in the low bits of an fp16 between 1024 and 2048, minus 1152
    const uint32_t v = u ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t x = __byte_perm(v, 0x64646464u, 0x4140), y = __byte_perm(v, 0x64646464u, 0x4342);
    __half2 p = __hsub2(*reinterpret_cast<__half2*>(&x), off);
    __half2 q = __hsub2(*reinterpret_cast<__half2*>(&y), off);
    h0 = *reinterpret_cast<uint32_t*>(&p);
    h1 = *reinterpret_cast<uint32_t*>(&q);
  }
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// what fp16 rounding left of a and b, rounded to fp16
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return pack_half(a - f.x, b - f.y);
}

__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
      f[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void load16(const float* p, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 u = reinterpret_cast<const float4*>(p)[i];
    f[4 * i] = u.x;
    f[4 * i + 1] = u.y;
    f[4 * i + 2] = u.z;
    f[4 * i + 3] = u.w;
  }
}

// a place on the line of tiles: tile kt of nt of head-and-row-group hr of batch element b
struct Cursor {
  int b, hr, kt, nt, L;
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// T: float (two fp16 terms per operand) or bf16 (one).  NR: column tiles of 8 query rows
template <typename T, int QT, int NR>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(sizeof(T) / 2, NR))
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const Params p) {
  constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;
  const DecodeQ8Args& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * (kStages * 2 * kTileBytes);
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(smem + kWarps * kStages * 2 * kTileBytes) + warp * kStages;
  if (lane == 0) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(bars + s), 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on

  // this warp's run of tiles.  Consecutive workers sit in different blocks, so that few tiles
  // spread over the SMs
  const int per = a.Hkv * p.rp.RG;
  int64_t unused, T_all;
  tile_sums(a, 0, &unused, &T_all);
  T_all *= per;
  const int64_t W = min(static_cast<int64_t>(p.workers), T_all);
  const int64_t worker = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  if (worker >= W) return;
  const int64_t x0 = run_start(worker, T_all, W);
  const int count = static_cast<int>(run_start(worker + 1, T_all, W) - x0);

  Cursor c;
  {
    int64_t before;
    c.b = find_batch(a, x0, per, &before);
    c.L = cached(a, c.b);
    c.nt = tiles_of(c.L);
    c.hr = static_cast<int>((x0 - before) / c.nt);
    c.kt = static_cast<int>((x0 - before) % c.nt);
  }
  auto advance = [&](Cursor& k) {
    if (++k.kt < k.nt) return;
    k.kt = 0;
    if (++k.hr < per) return;
    k.hr = 0;
    do {
      k.L = ++k.b < a.B ? cached(a, k.b) : kTile;  // past the last: never used
      k.nt = tiles_of(k.L);
    } while (k.nt == 0);
  };
  Cursor ahead = c;  // the next tile to ask for
  int asked = 0;
  auto ask = [&]() {
    const int s = asked % kStages;
    if (lane == 0) {
      const uint32_t bar = smem_u32(bars + s);
      uint8_t* dst = ring + s * 2 * kTileBytes;
      mbar_arrive_expect_tx(bar, 2 * kTileBytes);
      tma_load_4d(smem_u32(dst), &tmK, bar, 0, ahead.kt * kTile, ahead.hr / p.rp.RG, ahead.b);
      tma_load_4d(smem_u32(dst + kTileBytes), &tmV, bar, 0, ahead.kt * kTile,
                  ahead.hr / p.rp.RG, ahead.b);
    }
    advance(ahead);
    ++asked;
  };
  while (asked < min(kStages, count)) ask();

  // scales of a tile: lanes 0, 1 those of its two 16-position groups' keys, 2, 3 values'.  A
  // group behind the last position counts as 1 (its scores are excluded below).
  auto load_scale = [&](const Cursor& k) -> float {
    const int pos = k.kt * kTile + (lane & 1) * 16;
    if (lane >= 4 || pos >= k.L) return 1.f;
    const int64_t at =
        (static_cast<int64_t>(k.b) * a.Hkv + k.hr / p.rp.RG) * a.n_blocks + pos / a.block;
    return __ldg((lane < 2 ? a.k_scale : a.v_scale) + at);
  };

  // In the products' results a lane holds positions g and g + 8 of each 16 for the two rows
  // 8 nr + 2t + {0, 1}: the row statistics below are those rows'.
  uint32_t qf[kTerms][NR][4][2];  // queries, row 8 nr + g: operand fragments of four inner steps
  float qs[NR][2];                // what a score is to be multiplied by for its row
  int lim[NR][2];                 // last position that the row may see
  float o[NR][4][4], l[NR][2], m[NR][2];
  const float c2 = a.scale * 1.4426950408889634f;

  auto start_segment = [&]() {
    const int hk = c.hr / p.rp.RG, r0 = c.hr % p.rp.RG * (8 * NR);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int r = r0 + nr * 8 + g;
      float f[16];
      if (r < p.rp.R) {
        const int h = hk * (a.H / a.Hkv) + r / a.Nq;
        load16(static_cast<const T*>(a.Q) + c.b * a.sq[0] + h * a.sq[1] + (r % a.Nq) * a.sq[2] +
                   t * 16,
               f);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = 0.f;
      }
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int ex = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
      const float up = pow2i(13 - ex), down = pow2i(ex - 13) * c2;
      // inner step k: lane t supplies dims 16t + 4k + {0, 1} and {2, 3}
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float u = f[4 * k + 2 * x] * up, v = f[4 * k + 2 * x + 1] * up;
          const uint32_t hi = pack_half(u, v);
          qf[0][nr][k][x] = hi;
          if constexpr (kTerms == 2) qf[kTerms - 1][nr][k][x] = pack_rest(u, v, hi);
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qs[nr][e] = __shfl_sync(0xffffffffu, down, (2 * t + e) * 4);
        lim[nr][e] = a.causal ? c.L - a.Nq + (r0 + nr * 8 + 2 * t + e) % a.Nq : c.L - 1;
        l[nr][e] = 0.f;
        m[nr][e] = -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nr][j][i] = 0.f;
    }
  };

  auto end_segment = [&]() {
    const int64_t slot = worker + static_cast<int64_t>(c.b) * per + c.hr;
    const int r0 = c.hr % p.rp.RG * (8 * NR);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rl = nr * 8 + 2 * t + e;
        float s = l[nr][e];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        if (r0 + rl < p.rp.R) {
          // columns 8g + 2j and 8g + 2j + 1
          float4* dst = reinterpret_cast<float4*>(p.part + (slot * p.rp.RS + rl) * kD + g * 8);
          dst[0] = make_float4(o[nr][0][e], o[nr][0][2 + e], o[nr][1][e], o[nr][1][2 + e]);
          dst[1] = make_float4(o[nr][2][e], o[nr][2][2 + e], o[nr][3][e], o[nr][3][2 + e]);
          if (g == 0)
            *reinterpret_cast<float2*>(p.stat + (slot * p.rp.RS + rl) * 2) =
                make_float2(m[nr][e], s);
        }
      }
  };

  bool fresh = true;
  float sc_next = load_scale(c);
  for (int it = 0; it < count; ++it) {
    if (fresh) start_segment();
    const float sc = sc_next;
    Cursor nx = c;
    advance(nx);
    if (it + 1 < count) sc_next = load_scale(nx);  // a tile ahead of its use
    const float sc_log = log2f(sc), sc_inv = 1.f / sc;
    const int s = it % kStages;
    if (!__all_sync(0xffffffffu,
                    mbar_wait(smem_u32(bars + s), (it / kStages) & 1, p.timeout_ns))) {
      if (lane == 0) record_error(p.status, kErrTimeout, kSiteDecodeQ8);
      for (int x = it; x < asked; ++x)  // copies in flight land (bounded) before the block ends
        (void)mbar_wait(smem_u32(bars + x % kStages), (x / kStages) & 1, p.timeout_ns);
      return;
    }
    const uint8_t* sK = ring + s * 2 * kTileBytes;
    const uint8_t* sV = sK + kTileBytes;
    const int pos = c.kt * kTile;
    // some row may not see the whole tile
    const bool edge = pos + kTile - 1 > c.L - (a.causal ? a.Nq : 1);

    // ---- scores of two groups of 16 positions
    float x[2][NR][4], ev[2], inv[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t h[2][8];  // positions g and g + 8: 16-byte chunk t of a row, 64-byte swizzle
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int row = q * 16 + z * 8 + g;
        const uint4 u = *reinterpret_cast<const uint4*>(
            sK + row * kD + ((t ^ ((row >> 1) & 3)) << 4));
        codes_to_half<QT>(u.x, h[z][0], h[z][1]);
        codes_to_half<QT>(u.y, h[z][2], h[z][3]);
        codes_to_half<QT>(u.z, h[z][4], h[z][5]);
        codes_to_half<QT>(u.w, h[z][6], h[z][7]);
      }
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        float part[kTerms == 2 ? 4 : 1][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t fa[4] = {h[0][2 * k], h[1][2 * k], h[0][2 * k + 1], h[1][2 * k + 1]};
          float (&d)[4] = part[kTerms == 2 ? k : 0];
          if (kTerms == 2 || k == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = 0.f;
          }
          if constexpr (kTerms == 2)
            mma16816(d, fa, qf[kTerms - 1][nr][k][0], qf[kTerms - 1][nr][k][1]);
          mma16816(d, fa, qf[0][nr][k][0], qf[0][nr][k][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[q][nr][i] = kTerms == 2 ? (part[0][i] + part[kTerms - 1][i]) +
                                          (part[kTerms == 2 ? 2 : 0][i] + part[kTerms == 2 ? 3 : 0][i])
                                    : part[0][i];
      }
    }
    // ---- scaled scores, kept for the weights; + log2 of the value's scale; running maximum
    float top[NR][2];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) top[nr][0] = top[nr][1] = -INFINITY;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float ks = __shfl_sync(0xffffffffu, sc, q);
      ev[q] = __shfl_sync(0xffffffffu, sc_log, 2 + q);
      inv[q] = __shfl_sync(0xffffffffu, sc_inv, 2 + q);
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[q][nr][i] *= ks * qs[nr][i & 1];
          if (edge && pos + q * 16 + (i >> 1) * 8 + g > lim[nr][i & 1]) x[q][nr][i] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          top[nr][e] = fmaxf(top[nr][e], fmaxf(x[q][nr][e], x[q][nr][2 + e]) + ev[q]);
      }
    }
    if (p.scores != nullptr) {
      const int64_t row0 =
          (static_cast<int64_t>(c.b) * a.Hkv + c.hr / p.rp.RG) * p.rp.R +
          c.hr % p.rp.RG * (8 * NR);
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rl = nr * 8 + 2 * t + e;
          if (c.hr % p.rp.RG * (8 * NR) + rl < p.rp.R) {
            float* dst = p.scores + (row0 + rl) * p.Lpad + pos + g;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              dst[q * 16] = x[q][nr][e];
              dst[q * 16 + 8] = x[q][nr][2 + e];
            }
          }
        }
    }
    bool grew = false;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = top[nr][e];
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        top[nr][e] = fmaxf(m[nr][e], v);
        grew |= top[nr][e] > m[nr][e];
      }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // a first maximum (m = -inf) finds O = l = 0
          const float f = top[nr][e] == m[nr][e] ? 1.f : ex2_approx(m[nr][e] - top[nr][e]);
          m[nr][e] = top[nr][e];
          l[nr][e] *= f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[nr][j][e] *= f;
            o[nr][j][2 + e] *= f;
          }
        }
    }
    // ---- weights, 16 positions at a time, and their product with the value codes
    float po[kTerms == 2 ? NR : 1][4][4];
    if constexpr (kTerms == 2) {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) po[nr][j][i] = 0.f;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t pf[kTerms][NR][2];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mm = m[nr][e] == -INFINITY ? 0.f : m[nr][e];
          // the fp32 path keeps the offset out of the exponent, whose rounding it would coarsen
          const float shift = ev[q] - mm + (kTerms == 2 ? 0.f : kOffset);
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            float v = ex2_approx(x[q][nr][2 * z + e] + shift);
            if constexpr (kTerms == 2) v *= 8192.f;  // 2^kOffset
            w[2 * z + e] = v;
            l[nr][e] = fmaf(v, inv[q], l[nr][e]);
          }
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint32_t hi = pack_half(w[2 * z], w[2 * z + 1]);
          pf[0][nr][z] = transpose8x8(hi);
          if constexpr (kTerms == 2)
            pf[kTerms - 1][nr][z] = transpose8x8(pack_rest(w[2 * z], w[2 * z + 1], hi));
        }
      }
      // value rows 2t, 2t+1, 2t+8, 2t+9 of the 16, columns 8g .. 8g+7
      uint2 v[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int row = q * 16 + 2 * t + (z >> 1) * 8 + (z & 1);
        v[z] = *reinterpret_cast<const uint2*>(
            sV + row * kD + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
        if (edge) {
          // rows behind the last position hold anything: 0.  A NaN among the rows that some
          // query may not see must reach only those that do: taken out of the product here,
          // put into O below
          if (pos + row >= c.L) v[z] = make_uint2(0u, 0u);
          if constexpr (QT == kE4m3) {
            v[z].x &= ~__vcmpeq4(v[z].x & 0x7f7f7f7fu, 0x7f7f7f7fu);
            v[z].y &= ~__vcmpeq4(v[z].y & 0x7f7f7f7fu, 0x7f7f7f7fu);
          }
        }
      }
      uint32_t b0[8], b1[8];  // column 8g + j: rows 2t, 2t+1, and 2t+8, 2t+9
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t a0 = z ? v[0].y : v[0].x, a1 = z ? v[1].y : v[1].x;
        const uint32_t a2 = z ? v[2].y : v[2].x, a3 = z ? v[3].y : v[3].x;
        codes_to_half<QT>(__byte_perm(a0, a1, 0x5140), b0[4 * z], b0[4 * z + 1]);
        codes_to_half<QT>(__byte_perm(a0, a1, 0x7362), b0[4 * z + 2], b0[4 * z + 3]);
        codes_to_half<QT>(__byte_perm(a2, a3, 0x5140), b1[4 * z], b1[4 * z + 1]);
        codes_to_half<QT>(__byte_perm(a2, a3, 0x7362), b1[4 * z + 2], b1[4 * z + 3]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t fa[4] = {b0[2 * j], b0[2 * j + 1], b1[2 * j], b1[2 * j + 1]};
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          if constexpr (kTerms == 2) {
            mma16816(po[nr][j], fa, pf[kTerms - 1][nr][0], pf[kTerms - 1][nr][1]);
            mma16816(po[nr][j], fa, pf[0][nr][0], pf[0][nr][1]);
          } else {
            mma16816(o[nr][j], fa, pf[0][nr][0], pf[0][nr][1]);
          }
        }
      }
    }
    if constexpr (kTerms == 2) {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nr][j][i] += po[nr][j][i];
    }
    if (QT == kE4m3 && edge) {
      // columns 8g .. 8g+7 of each position: NaN into the rows that see it
      for (int row = 0; row < kTile && pos + row < c.L; ++row) {
        const uint2 u = *reinterpret_cast<const uint2*>(
            sV + row * kD + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
        if ((__vcmpeq4(u.x & 0x7f7f7f7fu, 0x7f7f7f7fu) |
             __vcmpeq4(u.y & 0x7f7f7f7fu, 0x7f7f7f7fu)) == 0)
          continue;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((((i < 4 ? u.x : u.y) >> (8 * (i & 3))) & 127u) == 127u)
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (pos + row <= lim[nr][e])
                  o[nr][i >> 1][2 * (i & 1) + e] = __int_as_float(0x7fffffff);
      }
    }
    __syncwarp();  // every lane has read the slot
    if (asked < count) ask();
    fresh = nx.hr != c.hr || nx.b != c.b;
    if (fresh || it + 1 == count) end_segment();
    c = nx;
  }
}

// ---- joining the pieces
// the workers that hold pieces of segment hr of batch element b (whole warp); false: none
__device__ __forceinline__ bool pieces_of(const Params& p, int b, int hr, int64_t* first,
                                          int64_t* last) {
  const int per = p.a.Hkv * p.rp.RG;
  int64_t before, total;
  tile_sums(p.a, b, &before, &total);
  const int nt = tiles_of(cached(p.a, b));
  if (nt == 0) return false;
  const int64_t T = total * per, W = min(static_cast<int64_t>(p.workers), T);
  const int64_t x = before * per + static_cast<int64_t>(hr) * nt;
  *first = worker_of(x, T, W);
  *last = worker_of(x + nt - 1, T, W);
  return true;
}

__device__ __forceinline__ void put2(__nv_bfloat16* q, float a, float b) {
  *reinterpret_cast<uint32_t*>(q) = pack_bf16x2(a, b);
}
__device__ __forceinline__ void put2(float* q, float a, float b) {
  *reinterpret_cast<float2*>(q) = make_float2(a, b);
}

constexpr int kWeightKeys = 4096;  // positions per block of the weights' part

// Blocks 0 .. row_blocks-1: O.  kWide: the eight warps of a block split the pieces of one row;
// otherwise each takes a row of its own.  The blocks behind: weights, 4096 positions each.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads) decode_q8_join_kernel(const Params p, int row_blocks,
                                                                  int weight_blocks) {
  const DecodeQ8Args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = a.Hkv * p.rp.RG, G = a.H / a.Hkv;
  const int group = 8 * p.rp.NR;
  pdl_launch_dependents();
  pdl_wait();  // the pieces are complete from here on
  if (static_cast<int>(blockIdx.x) < row_blocks) {
    __shared__ float so[kWarps][kD], sm[kWarps], sl[kWarps];
    const int64_t row = kWide ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv * p.rp.R;
    if (row >= rows) return;  // a whole warp (kWide: no warp)
    const int r = static_cast<int>(row % p.rp.R);
    const int hk = static_cast<int>(row / p.rp.R % a.Hkv);
    const int b = static_cast<int>(row / p.rp.R / a.Hkv);
    const int hr = hk * p.rp.RG + r / group;
    int64_t first = 0, last = -1;
    if (!pieces_of(p, b, hr, &first, &last)) last = first - 1;
    const int64_t seg = static_cast<int64_t>(b) * per + hr;
    float m = -INFINITY, l = 0.f;
    float2 o = make_float2(0.f, 0.f);
    for (int64_t w = first + (kWide ? warp : 0); w <= last; w += kWide ? kWarps : 1) {
      const int64_t at = (w + seg) * p.rp.RS + r % group;
      const float2 st = *reinterpret_cast<const float2*>(p.stat + at * 2);
      const float2 v = *reinterpret_cast<const float2*>(p.part + at * kD + 2 * lane);
      // -inf: no position of the piece is allowed.  (A NaN sum must not be lost here.)
      const float top = fmaxf(m, st.x);
      const float f = m == top ? 1.f : ex2_approx(m - top);
      const float h = st.x == top ? 1.f : ex2_approx(st.x - top);
      m = top;
      l = l * f + st.y * h;
      o.x = o.x * f + v.x * h;
      o.y = o.y * f + v.y * h;
    }
    if constexpr (kWide) {
      so[warp][2 * lane] = o.x;
      so[warp][2 * lane + 1] = o.y;
      if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
      }
      __syncthreads();
      if (warp != 0) return;
      m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w]);
      l = 0.f;
      o = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float h = sm[w] == m ? 1.f : ex2_approx(sm[w] - m);
        l += sl[w] * h;
        o.x += so[w][2 * lane] * h;
        o.y += so[w][2 * lane + 1] * h;
      }
    }
    const float y = l == 0.f ? 0.f : 1.f / l;  // no allowed position: zeros
    const int h = hk * G + r / a.Nq;
    put2(static_cast<T*>(a.O) + b * a.so[0] + h * a.so[1] + (r % a.Nq) * a.so[2] + 2 * lane,
         o.x * y, o.y * y);
    return;
  }
  // ---- weights: m and 1 / l of every row of the cache head, then its positions
  const int64_t x = static_cast<int64_t>(blockIdx.x) - row_blocks;
  const int64_t bh = x / weight_blocks;
  const int hk = static_cast<int>(bh % a.Hkv), b = static_cast<int>(bh / a.Hkv);
  const int L = cached(a, b);
  const int j0 = static_cast<int>(x % weight_blocks) * kWeightKeys;
  if (j0 >= L) return;
  extern __shared__ float rowstat[];  // [R][2]
  // the first row's scores and the totals are asked for before the statistics are known
  constexpr int kQuads = kWeightKeys / 4 / kThreads;
  const float* sc = p.scores + bh * p.rp.R * p.Lpad;
  float* out = a.weights + bh * a.Lmax;
  float4 x0[kQuads];
  float w[kQuads][4];
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int j = j0 + (k * kThreads + static_cast<int>(threadIdx.x)) * 4;
    if (j < L) x0[k] = *reinterpret_cast<const float4*>(sc + j);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[k][i] = j + i < L ? out[j + i] : 0.f;
  }
  for (int r = warp; r < p.rp.R; r += kWarps) {
    int64_t first, last;
    const int hr = hk * p.rp.RG + r / group;
    pieces_of(p, b, hr, &first, &last);  // L > 0: there are some
    const int64_t seg = static_cast<int64_t>(b) * per + hr;
    float m = -INFINITY, l = 0.f;
    for (int64_t s = first + lane; s <= last; s += 32) {
      const float2 st =
          *reinterpret_cast<const float2*>(p.stat + ((s + seg) * p.rp.RS + r % group) * 2);
      const float top = fmaxf(m, st.x);
      l = l * (m == top ? 1.f : ex2_approx(m - top)) +
          st.y * (st.x == top ? 1.f : ex2_approx(st.x - top));
      m = top;
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, s);
      const float l2 = __shfl_xor_sync(0xffffffffu, l, s);
      const float top = fmaxf(m, m2);
      l = l * (m == top ? 1.f : ex2_approx(m - top)) + l2 * (m2 == top ? 1.f : ex2_approx(m2 - top));
      m = top;
    }
    if (lane == 0) {  // weight = 2^(x + offset - m) / l (the pieces' own reference)
      rowstat[2 * r] = m == -INFINITY ? 0.f : kOffset - m;
      rowstat[2 * r + 1] = l == 0.f ? 0.f : 1.f / l;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int j = j0 + (k * kThreads + static_cast<int>(threadIdx.x)) * 4;
    if (j >= L) break;
    float4 x = x0[k];
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r = 0;;) {
      const float shift = rowstat[2 * r], inv = rowstat[2 * r + 1];
      const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)  // an excluded position takes nothing of a NaN row
        if (xs[i] != -INFINITY) s[i] = fmaf(ex2_approx(xs[i] + shift), inv, s[i]);
      if (++r == p.rp.R) break;
      x = *reinterpret_cast<const float4*>(sc + r * p.Lpad + j);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j + i < L) out[j + i] = w[k][i] + s[i];
  }
}

struct Workspace {
  size_t stat, scores, total;  // byte offsets; part is at 0
  int64_t Lpad;
};
Workspace plan(int B, int H, int Hkv, int Nq, int Lmax, int dtype, bool weights) {
  const RowPlan rp = row_plan(H, Hkv, Nq, dtype);
  const size_t slots =
      max_workers(dtype == 1 ? 1 : 2, rp.NR) + static_cast<size_t>(B) * Hkv * rp.RG;
  Workspace w;
  w.Lpad = (static_cast<int64_t>(Lmax) + kTile - 1) / kTile * kTile;
  w.stat = slots * rp.RS * kD * sizeof(float);
  w.scores = w.stat + (slots * rp.RS * 2 * sizeof(float) + 255) / 256 * 256;
  w.total = w.scores;
  if (weights) w.total += static_cast<size_t>(B) * Hkv * rp.R * w.Lpad * sizeof(float);
  return w;
}

template <typename T, int QT, int NR>
cudaError_t launch_main(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, int blocks,
                        cudaStream_t s) {
  auto kern = decode_q8_kernel<T, QT, NR>;
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kern), kSmemBytes, nullptr);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(blocks), dim3(kThreads), kSmemBytes, s, tk, tv, p);
}
template <typename T>
cudaError_t launch_all(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, int qtype,
                       int blocks, cudaStream_t s) {
  constexpr int kMost = sizeof(T) == 4 ? 2 : 4;  // row_plan's
  cudaError_t e;
  if (p.rp.NR == 1)
    e = qtype == kE4m3 ? launch_main<T, kE4m3, 1>(tk, tv, p, blocks, s)
                       : launch_main<T, kInt8, 1>(tk, tv, p, blocks, s);
  else if (p.rp.NR == 2)
    e = qtype == kE4m3 ? launch_main<T, kE4m3, 2>(tk, tv, p, blocks, s)
                       : launch_main<T, kInt8, 2>(tk, tv, p, blocks, s);
  else
    e = qtype == kE4m3 ? launch_main<T, kE4m3, kMost>(tk, tv, p, blocks, s)
                       : launch_main<T, kInt8, kMost>(tk, tv, p, blocks, s);
  if (e != cudaSuccess) return e;
  // a row's pieces where all sequences are alike: workers / segments, and the ends
  const int64_t heads = static_cast<int64_t>(p.a.B) * p.a.Hkv, rows = heads * p.rp.R;
  const bool wide = p.workers / (heads * p.rp.RG) > 8;
  const int row_blocks = static_cast<int>(wide ? rows : (rows + kWarps - 1) / kWarps);
  const int weight_blocks =
      p.scores != nullptr ? (p.a.Lmax + kWeightKeys - 1) / kWeightKeys : 0;
  const dim3 grid(static_cast<unsigned>(row_blocks + heads * weight_blocks));
  const size_t smem = p.scores != nullptr ? p.rp.R * 2 * sizeof(float) : 0;
  return wide ? launch_pdl(decode_q8_join_kernel<T, true>, grid, dim3(kThreads), smem, s, p,
                           row_blocks, weight_blocks)
              : launch_pdl(decode_q8_join_kernel<T, false>, grid, dim3(kThreads), smem, s, p,
                           row_blocks, weight_blocks);
}

}  // namespace

size_t decode_q8_workspace(int B, int H, int Hkv, int Nq, int Lmax, bool weights) {
  return std::max(plan(B, H, Hkv, Nq, Lmax, 0, weights).total,
                  plan(B, H, Hkv, Nq, Lmax, 1, weights).total);
}

cudaError_t launch_sdpa_decode_q8(const DecodeQ8Args& a, int dtype, int qtype, void* ws,
                                  const DevCtx& ctx, cudaStream_t s) {
  CUtensorMap tk, tv;
  if (!encode_map_u8(&tk, a.Kc, a.B, a.Hkv, a.Lmax, a.sk, kTile) ||
      !encode_map_u8(&tv, a.Vc, a.B, a.Hkv, a.Lmax, a.sv, kTile))
    return cudaErrorInvalidValue;
  const Workspace w = plan(a.B, a.H, a.Hkv, a.Nq, a.Lmax, dtype, a.weights != nullptr);
  Params p;
  p.a = a;
  p.rp = row_plan(a.H, a.Hkv, a.Nq, dtype);
  const int terms = dtype == 1 ? 1 : 2;
  const int blocks = std::min(ctx.num_sms * blocks_per_sm(terms, p.rp.NR),
                              max_workers(terms, p.rp.NR) / kWarps);
  p.workers = blocks * kWarps;
  p.part = static_cast<float*>(ws);
  p.stat = reinterpret_cast<float*>(static_cast<char*>(ws) + w.stat);
  p.scores = a.weights != nullptr
                 ? reinterpret_cast<float*>(static_cast<char*>(ws) + w.scores) : nullptr;
  p.Lpad = w.Lpad;
  p.status = ctx.status;
  p.timeout_ns = ctx.timeout_ns;
  return dtype == 1 ? launch_all<__nv_bfloat16>(tk, tv, p, qtype, blocks, s)
                    : launch_all<float>(tk, tv, p, qtype, blocks, s);
}

}  // namespace mha
