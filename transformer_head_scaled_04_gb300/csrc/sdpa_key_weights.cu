// sdpa_key_weights.cu -- the attention weight every key of a prompt received:
//   weights[b,g,j] += sum over the heads h of group g and the queries i of exp(s_ij - lse_i),
//   s_ij = q_i . k_j * scale, lse_i the forward's log-sum-exp of row i (mha_sdpa_fwd_lse)
// the column sums of the attention matrix, which is never stored.  A key belongs to one CTA, so
// the sums have one order and need no atomics.
//
// bf16 (key_weights_bf16_kernel): bound by the exponentials, one per (query, key) pair; the
// product itself is a quarter of the attention forward's tensor work.  One CTA per 128 keys:
// S^T = K Q^T (tcgen05.mma 128x128x16 into one of two TMEM buffers) for every 128-query tile of
// the group's heads that sees the keys, so a key's row lies in one thread and its sum needs no
// other: x = s * scale log2 e - lse log2 e, sum += 2^x, in paired fp32 operations.  Eight warps
// sum, a key's 128 columns in two halves, and two CTAs share an SM (320 threads, 99 KB, 256 TMEM
// columns each): four summing warps per scheduler.  Where the key tiles alone leave SMs idle the
// query tiles are split over several CTAs, their sums added by a second launch in a fixed order.
// 8 x 16 heads x 4096 372 us (60% of the exponential unit's rate), causal 217; 32 x 8 x 256 12.
//
// fp32 (key_weights_f32_kernel): the same sums with mma.sync m16n8k16.  Rows of Q and K are scaled
// by a power of two (largest value to [2^13, 2^14)) and split into two fp16 terms, 22 bits; three
// products (hi hi, hi lo, lo hi) give S = K Q^T, the four inner steps apart and added in fp32, as
// the tensor cores' own accumulation truncates.  One CTA per 128 keys, 16 to a warp with their
// terms in registers; chunks of 32 queries are split into terms once per CTA, in shared memory,
// the next chunk on its way from global memory meanwhile.  The (head, chunk) pairs are split over
// CTAs as above.  8 heads x 8 padded prompts of up to 1000 take 59 us, a causal prompt of 1024 23
// us; with one fp32 multiply-add per term and lane = key, whose operands came from shared memory
// at a quarter of the units' rate, 156 and 58 us.  The price of 22 bits: a weight is off by 7e-8 to
// 9e-8 (rms, padded prompts of 333), with products in fp32 4e-8 to 5e-8.  Bound by waits inside a
// warp: of 3.5 warps per scheduler 2.9 wait for the product before theirs in a chain of three or
// for its sums (47% of issue slots used, 37% of the mma.sync pipe).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "device_common.cuh"
#include "launchers.h"
#include "mma_f16.cuh"

namespace mha {
namespace {

constexpr int kD = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMissing = -1.f;  // for a sum that a time-out left out (sums are not negative)
struct KwParams {
  KeyWeightsArgs a;
  int split;      // CTAs that share a key tile's queries
  float* part;    // [split][B * Hkv][Nk] (split > 1)
  int* status;
  uint64_t timeout_ns;
};

// ============================================================================ fp32
constexpr int kKeys = 128;    // keys per CTA
constexpr int kQueries = 32;  // queries per chunk
constexpr int kWarps = 8;
static_assert(kKeys == 16 * kWarps && kWarps * 32 == 8 * kQueries,
              "a key tile per warp, eight threads to a query");

// the power of two that brings a row's largest magnitude to [2^13, 2^14), and its inverse.  2^-113
// keeps both normal numbers; rows below that are multiples of 2^-149, which 2^126 makes exact in
// fp16's two terms
__device__ __forceinline__ float2 row_scale(float amax) {
  const int ex = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -113);
  return make_float2(__uint_as_float((140 - ex) << 23), __uint_as_float((114 + ex) << 23));
}

__global__ void __launch_bounds__(kWarps * 32, 2) key_weights_f32_kernel(const KwParams p) {
  const KeyWeightsArgs& a = p.a;
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  const int g = blockIdx.y, b = blockIdx.z;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, t = lane & 3;  // fragment row (or column) and place in it
  const int z = static_cast<int>(blockIdx.x) % p.split;
  const int k0 = static_cast<int>(blockIdx.x) / p.split * kKeys;
  const int nk = a.mask == 2 ? min(max(__ldg(a.key_len + b), 0), a.Nk) : a.Nk;
  const int nq = a.query_len != nullptr ? min(max(__ldg(a.query_len + b), 0), a.Nq) : a.Nq;
  if (k0 >= nk) return;
  const int G = a.H / a.Hkv;
  const int first = a.mask == 1 ? k0 : 0;  // queries before the first key see none of these
  const int per_head = nq > first ? (nq - first + kQueries - 1) / kQueries : 0;
  const int64_t all = static_cast<int64_t>(G) * per_head;
  const int u0 = static_cast<int>(all * z / p.split);
  const int u1 = static_cast<int>(all * (z + 1) / p.split);

  // queries of a chunk, two terms, 16-byte piece i of row q stored at i ^ (q & 7); their scales
  // and lse log2 e
  __shared__ uint4 s_hi[2][kQueries][8], s_lo[2][kQueries][8];
  __shared__ float s_scale[2][kQueries], s_lse[2][kQueries];

  // this warp's keys: rows r and r + 8 of 16; lane t holds values 16t.. of a row, inner step k the
  // four from 16t + 4k on
  uint32_t khi[4][4], klo[4][4];
  float kscale[2];
  const float c = a.scale * kLog2e;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int j = min(k0 + warp * 16 + e * 8 + r, nk - 1);
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.K) +
                                                        b * a.sk[0] + g * a.sk[1] + j * a.sk[2]) +
                        t * 4;
    float f[16], amax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = src[i];
      f[4 * i] = v.x;
      f[4 * i + 1] = v.y;
      f[4 * i + 2] = v.z;
      f[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float2 sc = row_scale(amax);
    kscale[e] = sc.y * c;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float u = f[4 * k + 2 * x] * sc.x, v = f[4 * k + 2 * x + 1] * sc.x;
        khi[k][2 * x + e] = pack_half(u, v);
        klo[k][2 * x + e] = pack_rest(u, v, khi[k][2 * x + e]);
      }
  }

  // a thread's part of a chunk: values 8 (tid % 8).. of query tid / 8
  float4 next[2];
  float next_lse = 0.f;
  auto load = [&](int u) {
    const int h = g * G + u / per_head, i = first + u % per_head * kQueries + (tid >> 3);
    next[0] = next[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    next_lse = INFINITY;  // a row that does not count
    if (i < nq) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(a.Q) +
                                                        b * a.sq[0] + h * a.sq[1] + i * a.sq[2]);
      next[0] = q[(tid & 7) * 2];
      next[1] = q[(tid & 7) * 2 + 1];
      next_lse = a.lse[(static_cast<int64_t>(b) * a.H + h) * a.Nq + i];
    }
  };
  auto store = [&](int buf) {
    const float f[8] = {next[0].x, next[0].y, next[0].z, next[0].w,
                        next[1].x, next[1].y, next[1].z, next[1].w};
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float2 sc = row_scale(amax);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = f[2 * i] * sc.x, v = f[2 * i + 1] * sc.x;
      hi[i] = pack_half(u, v);
      lo[i] = pack_rest(u, v, hi[i]);
    }
    const int q = tid >> 3, at = (tid & 7) ^ (q & 7);
    s_hi[buf][q][at] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    s_lo[buf][q][at] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if ((tid & 7) == 0) {
      s_scale[buf][q] = sc.y;
      s_lse[buf][q] = next_lse * kLog2e;
    }
  };
  if (u0 < u1) {
    load(u0);
    store(0);
  }
  __syncthreads();
  float sum[2] = {0.f, 0.f};
  for (int u = u0, buf = 0; u < u1; ++u, buf ^= 1) {
    const int i0 = first + u % per_head * kQueries;
    if (u + 1 < u1) load(u + 1);
#pragma unroll
    for (int n = 0; n < kQueries / 8; ++n) {  // queries 8n + r as the product's columns
      uint32_t qh[8], ql[8];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint4 v = s_hi[buf][8 * n + r][(2 * t + x) ^ r];
        const uint4 w = s_lo[buf][8 * n + r][(2 * t + x) ^ r];
        qh[4 * x] = v.x, qh[4 * x + 1] = v.y, qh[4 * x + 2] = v.z, qh[4 * x + 3] = v.w;
        ql[4 * x] = w.x, ql[4 * x + 1] = w.y, ql[4 * x + 2] = w.z, ql[4 * x + 3] = w.w;
      }
      float part[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mma16816_zero(part[k], klo[k], qh[2 * k], qh[2 * k + 1]);
        mma16816(part[k], khi[k], ql[2 * k], ql[2 * k + 1]);
        mma16816(part[k], khi[k], qh[2 * k], qh[2 * k + 1]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // queries 8n + 2t + e, keys r and r + 8
        const int q = 8 * n + 2 * t + e;
        const float l2 = s_lse[buf][q], qs = s_scale[buf][q];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int i = 2 * x + e;
          const float s = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
          const bool counts =
              l2 != INFINITY && (a.mask != 1 || k0 + warp * 16 + x * 8 + r <= i0 + q);
          if (counts) sum[x] += exp2f(fmaf(s, qs * kscale[x], -l2));
        }
      }
    }
    if (u + 1 < u1) store(buf ^ 1);
    __syncthreads();
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {  // over the lanes that had other queries of the key
    sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
    sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
  }
  if (t == 0) {
    const int64_t bg = static_cast<int64_t>(b) * a.Hkv + g;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = k0 + warp * 16 + x * 8 + r;
      if (j >= nk) continue;
      if (p.split == 1)
        a.weights[bg * a.ld + j] += sum[x];
      else
        p.part[(static_cast<int64_t>(z) * a.B * a.Hkv + bg) * a.Nk + j] = sum[x];
    }
  }
}

// ============================================================================ bf16
constexpr int kT = 128;                   // keys and queries per tile
constexpr int kTileBytes = kT * kD * 2;   // 16 KB
constexpr int kStages = 5;                // query tiles in flight
constexpr int kSumWarps = 8;              // warp w: TMEM lanes 32 (w % 4).., columns 64 (w / 4)..
constexpr int kWarpTma = kSumWarps, kWarpMma = kSumWarps + 1;
constexpr int kTcThreads = (kSumWarps + 2) * 32;
constexpr uint32_t kTmemCols = 256;       // two S^T buffers
constexpr int kErrTimeout = -6;
enum : int { kSiteKwProducer = 34, kSiteKwMma = 35, kSiteKwMath = 36 };
constexpr int kOffQ = kTileBytes;
constexpr int kOffLse = kOffQ + kStages * kTileBytes;  // [stages][128] -lse log2 e
constexpr int kOffBar = kOffLse + kStages * kT * 4;
constexpr int kBarK = 0, kBarQ = 1, kBarQFree = kBarQ + kStages, kBarS = kBarQFree + kStages,
              kBarSFree = kBarS + 2, kBarDrain = kBarSFree + 2, kNumBars = kBarDrain + 1;
constexpr int kTcSmem = 1024 + kOffBar + kNumBars * 8 + 16;

__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

// 32 queries of one key: acc += 2^(s c + nl)
__device__ __forceinline__ void add_chunk(const uint32_t (&s)[32], const float* nl, float2 c2,
                                          float2 (&acc)[4]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 n = *reinterpret_cast<const float4*>(nl + 4 * i);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 4 * i + 2 * h;
      float2 x = ffma2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), c2,
                       h ? make_float2(n.z, n.w) : make_float2(n.x, n.y));
      x.x = ex2_approx(x.x);
      x.y = ex2_approx(x.y);
      acc[k / 2 % 4] = fadd2(acc[k / 2 % 4], x);
    }
  }
}
// the scores of columns outside first <= i < last, which may be anything: -inf
__device__ __forceinline__ void exclude(uint32_t (&s)[32], int first, int last) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i < first || i >= last) s[i] = 0xff800000u;
}

__global__ void __launch_bounds__(kTcThreads, 2)
    key_weights_bf16_kernel(const __grid_constant__ CUtensorMap tmQ,
                            const __grid_constant__ CUtensorMap tmK, const KwParams p) {
  const KeyWeightsArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // key tile, cache head, batch element and share of the query tiles.  Causal: the tiles with the
  // most queries first over all heads; otherwise a head's tiles next to one another (its queries
  // stay in L2)
  const int tiles = (a.Nk + kT - 1) / kT, heads = a.B * a.Hkv;
  int unit = static_cast<int>(blockIdx.x);
  const int z = unit % p.split;
  unit /= p.split;
  const int kt = a.mask == 1 ? unit / heads : unit % tiles;
  const int bg = a.mask == 1 ? unit % heads : unit / tiles;
  const int g = bg % a.Hkv, b = bg / a.Hkv;
  const int k0 = kt * kT;

  pdl_wait();  // the previous kernel's output is complete from here on
  const int nk = a.mask == 2 ? min(max(__ldg(a.key_len + b), 0), a.Nk) : a.Nk;
  const int nq = a.query_len != nullptr ? min(max(__ldg(a.query_len + b), 0), a.Nq) : a.Nq;
  if (k0 >= nk) return;
  // (head, query tile) pairs: tiles first_q .. of each head of the group
  const int G = a.H / a.Hkv;
  const int first_q = a.mask == 1 ? kt : 0;
  const int per_head = max((nq + kT - 1) / kT - first_q, 0);
  const int64_t all = static_cast<int64_t>(G) * per_head;
  const int u0 = static_cast<int>(all * z / p.split);
  const int n = static_cast<int>(all * (z + 1) / p.split) - u0;
  float* out = p.split == 1 ? a.weights + static_cast<int64_t>(bg) * a.ld
                            : p.part + (static_cast<int64_t>(z) * heads + bg) * a.Nk;
  if (n == 0) {
    if (p.split > 1)
      for (int j = k0 + static_cast<int>(threadIdx.x); j < min(k0 + kT, nk); j += kTcThreads)
        out[j] = 0.f;
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(bar(kBarK), 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(kBarQ + i), 1);
      mbar_init(bar(kBarQFree + i), 1 + kSumWarps);  // the products, and the warps' use of lse
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarS + i), 2);  // the products, and their issuer (see there)
      mbar_init(bar(kBarSFree + i), kSumWarps);
    }
    mbar_init(bar(kBarDrain), 1);
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (not before: a following kernel that takes its TMEM ahead of its own wait must not get there
  // first, since it gives it back only after this one has ended)
  pdl_launch_dependents();

  float* lse_s = reinterpret_cast<float*>(smem + kOffLse);
  if (warp == kWarpTma) {
    // ------------------------------------------------------------------ queries and their lse
    const float* lse = a.lse + (static_cast<int64_t>(b) * a.H + g * G) * a.Nq;
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      mbar_arrive_expect_tx(bar(kBarK), kTileBytes);
      tma_load_4d(smem_u32(smem), &tmK, bar(kBarK), 0, k0, g, b);
    }
    bool ok = true;
    int asked = 0, s = 0, tile = u0 % per_head, h = u0 / per_head;
    uint32_t phase = 1;
    // lse entries are loaded four tiles ahead of their use; rows that do not count: 2^-inf = 0
    constexpr int kAhead = 4;
    float l[kAhead][kT / 32];
    int l_tile = tile, l_h = h, l_left = n;
    auto load_lse = [&](float (&v)[kT / 32]) {
      if (l_left-- <= 0) return;
#pragma unroll
      for (int i = 0; i < kT / 32; ++i) {
        const int row = (first_q + l_tile) * kT + 32 * i + lane;
        v[i] = row < nq ? __ldg(lse + static_cast<int64_t>(l_h) * a.Nq + row) : INFINITY;
      }
      if (++l_tile == per_head) l_tile = 0, ++l_h;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load_lse(l[k]);
    for (int j0 = 0; ok && j0 < n; j0 += kAhead) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (!ok || j0 + k >= n) break;
        if (!warp_all(mbar_wait_backoff(bar(kBarQFree + s), phase, p.timeout_ns))) {
          ok = false;
          break;
        }
#pragma unroll
        for (int i = 0; i < kT / 32; ++i) lse_s[s * kT + 32 * i + lane] = -l[k][i] * kLog2e;
        load_lse(l[k]);
        __syncwarp();
        if (lane == 0) {  // the arrival releases the entries too
          mbar_arrive_expect_tx(bar(kBarQ + s), kTileBytes);
          tma_load_4d(smem_u32(smem + kOffQ + s * kTileBytes), &tmQ, bar(kBarQ + s), 0,
                      (first_q + tile) * kT, g * G + h, b);
        }
        ++asked;
        if (++s == kStages) s = 0, phase ^= 1;
        if (++tile == per_head) tile = 0, ++h;
      }
    }
    if (lane == 0) {
      if (!ok) record_error(p.status, kErrTimeout, kSiteKwProducer);
      // every copy started here lands before the CTA can exit
      (void)mbar_wait(bar(kBarK), 0, p.timeout_ns);
      for (int j = max(asked - kStages, 0); j < asked; ++j)
        (void)mbar_wait(bar(kBarQ + j % kStages), (j / kStages) & 1, p.timeout_ns);
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16_f32(kT, kT, false, false);
      const uint64_t dK = smem_desc_sw128(smem_u32(smem), 1024, 1024);
      const uint64_t dQ = smem_desc_sw128(smem_u32(smem + kOffQ), 1024, 1024);
      bool ok = mbar_wait(bar(kBarK), 0, p.timeout_ns);
      for (int j = 0; ok && j < n; ++j) {
        const int s = j % kStages, buf = j & 1;
        if (!mbar_wait(bar(kBarQ + s), (j / kStages) & 1, p.timeout_ns) ||
            (j > 1 && !mbar_wait(bar(kBarSFree + buf), ((j >> 1) - 1) & 1, p.timeout_ns))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t bq = dQ + static_cast<uint64_t>((s * kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk)
          mma_bf16_ss(tmem + buf * kT, dK + kk * 2, bq + kk * 2, idS, kk > 0 ? 1u : 0u);
        mma_commit(bar(kBarQFree + s));
        mma_commit(bar(kBarS + buf));
        // releases to the summing warps what this thread acquired with the tile: its lse entries
        mbar_arrive(bar(kBarS + buf));
      }
      if (!ok) record_error(p.status, kErrTimeout, kSiteKwMma);
      mma_commit(bar(kBarDrain));
      (void)mbar_wait(bar(kBarDrain), 0, p.timeout_ns);  // no MMA in flight past this point
    }
  } else {
    // ------------------------------------------------------------------ sums
    const int quarter = warp & 3, col0 = (warp >> 2) * 64;
    const int key = k0 + quarter * 32 + lane;
    const float c = fmaxf(a.scale * kLog2e, 1.2e-38f);  // -inf * c stays -inf
    const float2 c2 = make_float2(c, c);
    const uint32_t t_s = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + col0;
    float2 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
    int slot = 0, tile = u0 % per_head;  // of the ring; of the head, from first_q
    uint32_t phase = 0;                  // bit `buf` that of S buffer buf
    auto wait_s = [&](int buf) -> bool {
      const bool got = warp_all(mbar_wait(bar(kBarS + buf), (phase >> buf) & 1, p.timeout_ns));
      if (!got && lane == 0) record_error(p.status, kErrTimeout, kSiteKwMath);
      phase ^= 1u << buf;
      tc_fence_after();
      return got;
    };
    // 32 columns are worked on while the next 32 are on their way from TMEM
    uint32_t r0[32], r1[32];
    bool ok = wait_s(0);
    tmem_ld32(t_s, r0);
    int j = 0;
    auto add_tile = [&](auto mask_type) {
      constexpr bool kMask = decltype(mask_type)::value;
      const int buf = j & 1, q0 = (first_q + tile) * kT;
      const float* nl = lse_s + slot * kT + col0;
      // columns that count: from the diagonal on, before the last query
      const int first = (a.mask == 1 ? key - q0 : 0) - col0, last = nq - q0 - col0;
      tmem_wait_ld();
      reg_fence(r0);
      tmem_ld32(t_s + buf * kT + 32, r1);
      if constexpr (kMask) exclude(r0, first, last);
      add_chunk(r0, nl, c2, acc);
      tmem_wait_ld();
      reg_fence(r1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarSFree + buf));  // the buffer may be overwritten
      if (j + 1 < n) ok = wait_s(buf ^ 1);
      tmem_ld32(t_s + (buf ^ 1) * kT, r0);  // behind the last tile: unused
      if constexpr (kMask) exclude(r1, first - 32, last - 32);
      add_chunk(r1, nl + 32, c2, acc);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarQFree + slot));
      if (++slot == kStages) slot = 0;
      if (++tile == per_head) tile = 0;
      ++j;
    };
    // Tiles some of whose columns do not count for some key, a head's first (causal) and last, have
    // code of their own, and the others a loop of their own: in one loop with a branch those took
    // 410 instead of 366 us (8 x 16 heads x 4096)
    const int full = nq / kT - first_q;  // tiles of a head before one that the queries end in
    while (ok && j < n) {
      if (tile >= full || (a.mask == 1 && tile == 0)) {
        add_tile(std::true_type{});
      } else {
        const int end = min(n, j + min(full, per_head) - tile);
        while (ok && j < end) add_tile(std::false_type{});
      }
    }
    tmem_wait_ld();
    // the two column halves of a key through the (now unused) key tile's memory.  After a time-out
    // the key's weight stays as it was: nothing is added here, nor where the shares are added up
    float* half = reinterpret_cast<float*>(smem);
    const float2 t = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
    if (col0 > 0) half[quarter * 32 + lane] = ok ? t.x + t.y : kMissing;
    named_bar_sync(1, kSumWarps * 32);
    if (col0 == 0 && key < nk) {
      const float other = half[quarter * 32 + lane], sum = t.x + t.y + other;
      const bool whole = ok && other != kMissing;
      if (p.split > 1)
        out[key] = whole ? sum : kMissing;
      else if (whole)
        out[key] += sum;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// weights += the shares' sums, in order; keys with a share missing keep what they have
__global__ void __launch_bounds__(256) key_weights_add_kernel(const KwParams p) {
  const KeyWeightsArgs& a = p.a;
  pdl_launch_dependents();
  pdl_wait();  // the shares are complete from here on
  const int bg = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  const int nk = a.mask == 2 ? min(max(__ldg(a.key_len + bg / a.Hkv), 0), a.Nk) : a.Nk;
  if (j >= nk) return;
  float s = 0.f;
  bool missing = false;
  for (int z = 0; z < p.split; ++z) {
    const float share = p.part[(static_cast<int64_t>(z) * gridDim.y + bg) * a.Nk + j];
    missing |= share == kMissing;  // (no branch: the loads of all shares go out together)
    s += share;
  }
  if (!missing) a.weights[static_cast<int64_t>(bg) * a.ld + j] += s;
}

// CTAs per key tile: enough for two on each of 152 SMs (fp32: twice that, for shorter CTAs), no
// more than there are query tiles or chunks.  Against one CTA per key tile: a bf16 head of 4096
// 9.9 and 22.3 us, four 20.1 and 22.3; three fp32 prompts of 333 12.5 and 43.9
int key_weights_split(int B, int H, int Hkv, int Nq, int Nk, int dtype) {
  const int keys = dtype == 1 ? kT : kKeys, rows = dtype == 1 ? kT : kQueries;
  const int64_t units = static_cast<int64_t>(B) * Hkv * ((Nk + keys - 1) / keys);
  const int64_t queries = static_cast<int64_t>(H / Hkv) * ((Nq + rows - 1) / rows);
  const int64_t want = dtype == 1 ? 304 : 608;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(queries, want / units)));
}

}  // namespace

size_t key_weights_workspace(int B, int H, int Hkv, int Nq, int Nk, int dtype) {
  const int split = key_weights_split(B, H, Hkv, Nq, Nk, dtype);
  return split == 1 ? 0 : static_cast<size_t>(split) * B * Hkv * Nk * sizeof(float);
}

cudaError_t launch_key_weights(const KeyWeightsArgs& a, int dtype, void* ws, const DevCtx& ctx,
                               cudaStream_t s) {
  KwParams p;
  p.a = a;
  p.split = key_weights_split(a.B, a.H, a.Hkv, a.Nq, a.Nk, dtype);
  p.part = static_cast<float*>(ws);
  p.status = ctx.status;
  p.timeout_ns = ctx.timeout_ns;
  cudaError_t e;
  if (dtype != 1) {
    e = launch_pdl(key_weights_f32_kernel,
                   dim3((a.Nk + kKeys - 1) / kKeys * p.split, a.Hkv, a.B), dim3(kWarps * 32), 0, s,
                   p);
  } else {
    CUtensorMap tq, tk;
    if (!encode_map_bf16(&tq, a.Q, a.B, a.H, a.Nq, a.sq, kT) ||
        !encode_map_bf16(&tk, a.K, a.B, a.Hkv, a.Nk, a.sk, kT))
      return cudaErrorInvalidValue;
    e = prepare_kernel(reinterpret_cast<const void*>(key_weights_bf16_kernel), kTcSmem, nullptr);
    if (e != cudaSuccess) return e;
    const int units = a.B * a.Hkv * ((a.Nk + kT - 1) / kT);
    e = launch_pdl(key_weights_bf16_kernel, dim3(units * p.split), dim3(kTcThreads), kTcSmem, s,
                   tq, tk, p);
  }
  if (e != cudaSuccess || p.split == 1) return e;
  return launch_pdl(key_weights_add_kernel, dim3((a.Nk + 255) / 256, a.B * a.Hkv), dim3(256), 0, s,
                    p);
}

}  // namespace mha
