// kv_evict_q8.cu -- drop the cached positions with the least accumulated attention weight and
// move the rest into another 8-bit cache (see q8_common.cuh for the codes and scales).
//
// Two launches.  select: per (batch element, head) the kept positions, ascending: the newest
// `recent` and, of the others, those with the largest weights (equal weights: the lower
// position).  A cluster of up to eight CTAs holds a head's weights in registers, 16 neighbours to
// a thread, so they are read from memory once (heads longer than that are read again for every
// step).  The k-th largest weight is found by a radix descent over the weights' bits, eight at a
// time, with the counts of one digit in shared memory and added up over the cluster; then one
// prefix sum over threads and CTAs gives every kept position its place.  No sorting, no order that
// depends on timing: the counts are sums of integers.
// gather: one CTA per (block of the new cache, head, batch element) copies the block's rows; the
// block takes the largest scale of the tokens it receives, and codes that came under a smaller
// one are written under it.  Bound by HBM: 64 bytes read and written per row of K and of V.
// 64 x 16 heads 4096 -> 1024: 65 us, 17 of them the select; 8 heads 131072 -> 8001 20 us.
#include "launchers.h"
#include "q8_common.cuh"

namespace mha {
namespace {

constexpr int kEach = 16;  // weights per thread

// fp32 to an unsigned integer of the same order; -0 equals +0 and NaN the lowest value
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  const uint32_t key = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return w == w ? key : 0x007fffffu;  // that of -inf
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// kThreads a power of two.  The grid's x is B * H clusters of `ctas` CTAs.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) kv_evict_select_kernel(const KvEvictArgs a, int ctas) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  constexpr int kWarps = kThreads / 32;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x) % ctas;  // CTA of the cluster
  const int64_t bh = blockIdx.x / ctas;
  const int b = static_cast<int>(bh / a.H);
  const int L = min(max(__ldg(a.cache_len + b), 0), a.Lmax);
  int32_t* kept = a.kept + bh * a.keep;
  const int n_out = min(L, a.keep);
  if (bh % a.H == 0 && rank == 0 && tid == 0) a.len_out[b] = n_out;
  for (int i = n_out + rank * kThreads + tid; i < a.keep; i += ctas * kThreads) kept[i] = -1;
  if (L <= a.keep) {  // nothing to drop (the same for the whole cluster)
    for (int i = rank * kThreads + tid; i < L; i += ctas * kThreads) kept[i] = i;
    return;
  }
  const float* w = a.weights + bh * a.Lmax;
  const int recent = min(a.recent, a.keep);
  const int m = L - recent;      // candidates: positions 0..m-1
  const int k = a.keep - recent;  // of which the k largest stay, 0 <= k < m
  // position of a thread's first weight in step c of `steps`
  const int per_step = ctas * kThreads * kEach;
  const int steps = (L + per_step - 1) / per_step;
  auto first = [&](int c) { return ((c * ctas + rank) * kThreads + tid) * kEach; };
  uint32_t key[kEach];  // 0, below any weight's, for a position that is no candidate
  const bool vector = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
  auto load = [&](int c) {
    const int j0 = first(c);
    if (vector && j0 + kEach <= m) {
#pragma unroll
      for (int i = 0; i < kEach / 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(w + j0 + 4 * i);
        key[4 * i] = order_key(v.x);
        key[4 * i + 1] = order_key(v.y);
        key[4 * i + 2] = order_key(v.z);
        key[4 * i + 3] = order_key(v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i) key[i] = j0 + i < m ? order_key(w[j0 + i]) : 0u;
    }
  };
  __shared__ int hist[2][256];  // of the digit: this CTA's; two, so that one round can be read
                                // by the cluster while the next is cleared
  __shared__ int s_count[256], s_warp[kWarps], s_pick[2], s_total[2][2];
  auto sync_all = [&]() {
    if (ctas == 1)
      __syncthreads();
    else
      cluster_sync_all();
  };

  // ---- the k-th largest key
  uint32_t prefix = 0;  // its high bits
  int above = 0;        // candidates above the prefix
  load(0);
  for (int shift = 24, round = 0; k > 0 && shift >= 0; shift -= 8, round ^= 1) {
    int* h = hist[round];
    for (int i = tid; i < 256; i += kThreads) h[i] = 0;
    __syncthreads();
    for (int c = 0; c < steps; ++c) {
      if (steps > 1) load(c);
      // (k < m: what is no candidate cannot become the k-th largest)
      const uint32_t want = prefix >> ((shift + 8) & 31);
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (shift == 24 || (key[i] >> ((shift + 8) & 31)) == want)
          atomicAdd(&h[(key[i] >> shift) & 255u], 1);
    }
    sync_all();
    if (ctas > 1) {  // a thread per digit adds up the cluster's
      if (tid < 256) {
        const uint32_t at = smem_u32(h + tid);
        int n = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < ctas) n += ld_cluster(mapa_shared(at, r));
        s_count[tid] = n;
      }
      __syncthreads();
      h = s_count;
    }
    if (warp == 0) {  // lane l: digits 255 - 8l downwards, eight of them
      int n[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] = h[255 - 8 * lane - i];
        sum += n[i];
      }
      int before = sum;  // exclusive sum over the lanes, then digit by digit
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      before += above - sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (before < k && before + n[i] >= k) {  // one lane's one digit
          s_pick[0] = 255 - 8 * lane - i;
          s_pick[1] = before;
        }
        before += n[i];
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_pick[0]) << shift;
    above = s_pick[1];
  }
  const int ties = k - above;  // candidates equal to the k-th largest that stay, lowest first

  // ---- places: behind all kept weights above it, and those ties before it that stay
  int gt0 = 0, eq0 = 0;  // of the steps before
  for (int c = 0; c < steps; ++c) {
    if (steps > 1) load(c);
    const int j0 = first(c);
    // bit i: weight i stays whatever the ties; is one
    auto below = [&](int end) { return (1u << min(max(end - j0, 0), kEach)) - 1u; };
    uint32_t gt = below(L) & ~below(m), eq = 0;
    if (k > 0) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        gt |= (key[i] > prefix ? 1u : 0u) << i;
        eq |= (key[i] == prefix ? 1u : 0u) << i;
      }
    }
    // both counts in one scan: at most 16384 each
    const int mine = (__popc(gt) << 16) | __popc(eq);
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) s_warp[warp] = scan;
    __syncthreads();
    if (warp == 0) {
      const int v = lane < kWarps ? s_warp[lane] : 0;
      int t = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += u;
      }
      if (lane < kWarps) s_warp[lane] = t - v;
      if (lane == 31) {
        s_total[c & 1][0] = static_cast<int>(static_cast<uint32_t>(t) >> 16);
        s_total[c & 1][1] = t & 0xffff;
      }
    }
    sync_all();
    int g = gt0, e = eq0;  // of the CTAs before, and (gt0, eq0) of all up to this step
    for (int r = 0; r < ctas; ++r) {
      int rg = s_total[c & 1][0], re = s_total[c & 1][1];
      if (ctas > 1) {
        rg = ld_cluster(mapa_shared(smem_u32(&s_total[c & 1][0]), r));
        re = ld_cluster(mapa_shared(smem_u32(&s_total[c & 1][1]), r));
      }
      if (r < rank) g += rg, e += re;
      gt0 += rg;
      eq0 += re;
    }
    const uint32_t before = static_cast<uint32_t>(s_warp[warp] + scan - mine);
    g += static_cast<int>(before >> 16);
    e += static_cast<int>(before & 0xffffu);
    int32_t* to = kept + g + min(e, ties);
    while (eq != 0) {  // the ties that stay join the others: seldom more than one
      if (e++ < ties) gt |= eq & (0u - eq);
      eq &= eq - 1u;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if ((gt >> i) & 1u) *to++ = j0 + i;
    __syncthreads();  // s_warp is written again
  }
  if (ctas > 1) cluster_sync_all();  // no CTA leaves while others may read its counts
}

constexpr int kGatherThreads = 128;

// 16 bytes of a row.  Rows are 64 bytes and their neighbours often stay behind: with plain loads
// 64 x 16 heads 4096 -> 1024 read 247 MB from HBM, 128 bytes at a time, so 156 MB (58 -> 52 us)
__device__ __forceinline__ uint4 load_row(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// BLOCK: tokens per scale.  Four threads to a row, of K and of V; a row is asked for as soon as
// its position is known (-1: there is none), together with its scale.  Twelve CTAs to an SM where
// a thread has two rows at most (64 x 16 heads 4096 -> 1024 67.7 -> 65 us over the ten that its
// registers would leave; four rows spill: 8 heads 131072 -> 8001 20.5 -> 25.7 us).
template <int QT, int BLOCK>
__global__ void __launch_bounds__(kGatherThreads, BLOCK <= 64 ? 12 : 7)
    kv_evict_gather_kernel(const KvEvictArgs a) {
  pdl_launch_dependents();
  pdl_wait();  // the select kernel's positions are complete from here on
  constexpr int kRows = (BLOCK + 31) / 32;  // of a thread
  const int h = blockIdx.y, b = blockIdx.z, tid = static_cast<int>(threadIdx.x);
  const int64_t bh = static_cast<int64_t>(b) * a.H + h;
  const int lo = static_cast<int>(blockIdx.x) * BLOCK, chunk = (tid & 3) * 16;
  const int32_t* kept = a.kept + bh * a.keep + lo;
  int j[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = (tid >> 2) + 32 * k;
    j[k] = r < BLOCK && lo + r < a.keep ? kept[r] : -1;
  }
  const uint8_t* ki = static_cast<const uint8_t*>(a.Kc) + b * a.sk[0] + h * a.sk[1] + chunk;
  const uint8_t* vi = static_cast<const uint8_t*>(a.Vc) + b * a.sv[0] + h * a.sv[1] + chunk;
  uint4 u[2][kRows];
  float sc[2][kRows], w[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k)
    if (j[k] >= 0) {
      u[0][k] = load_row(ki + j[k] * a.sk[2]);
      u[1][k] = load_row(vi + j[k] * a.sv[2]);
      sc[0][k] = a.k_scale[bh * a.n_blocks + j[k] / BLOCK];
      sc[1][k] = a.v_scale[bh * a.n_blocks + j[k] / BLOCK];
      if (chunk == 0) w[k] = a.weights[bh * a.Lmax + j[k]];
    }
  float most[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kRows; ++k)
    if (j[k] >= 0) {
      most[0] = fmaxf(most[0], sc[0][k]);
      most[1] = fmaxf(most[1], sc[1][k]);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    most[0] = fmaxf(most[0], __shfl_xor_sync(0xffffffffu, most[0], o));
    most[1] = fmaxf(most[1], __shfl_xor_sync(0xffffffffu, most[1], o));
  }
  __shared__ float smax[2][4];
  if ((tid & 31) == 0) {
    smax[0][tid >> 5] = most[0];
    smax[1][tid >> 5] = most[1];
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const float now =
        fmaxf(fmaxf(smax[x][0], smax[x][1]), fmaxf(smax[x][2], smax[x][3]));
    // (a block without rows keeps its scale: the first row belongs to thread 0)
    if (tid == 0 && j[0] >= 0)
      (x ? a.v_scale_out : a.k_scale_out)[bh * a.n_blocks_out + blockIdx.x] = now;
    const int64_t* so = x ? a.svo : a.sko;
    uint8_t* out = static_cast<uint8_t*>(x ? a.Vo : a.Ko) + b * so[0] + h * so[1] +
                   static_cast<int64_t>(lo) * so[2] + chunk;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (j[k] < 0) continue;
      uint4 v = u[x][k];
      if (sc[x][k] < now) {
        const float ratio = sc[x][k] / now;  // exact for powers of two
        v = make_uint4(q8_rescale4<QT>(v.x, ratio), q8_rescale4<QT>(v.y, ratio),
                       q8_rescale4<QT>(v.z, ratio), q8_rescale4<QT>(v.w, ratio));
      }
      *reinterpret_cast<uint4*>(out + ((tid >> 2) + 32 * k) * so[2]) = v;
    }
  }
  if (a.weights_out != nullptr && chunk == 0) {
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (j[k] >= 0) a.weights_out[bh * a.Lmax_out + lo + (tid >> 2) + 32 * k] = w[k];
  }
}

template <int kThreads>
cudaError_t launch_select(const KvEvictArgs& a, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.H * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ctas;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kv_evict_select_kernel<kThreads>, a, ctas);
}

template <int QT>
cudaError_t launch_gather(const KvEvictArgs& a, cudaStream_t s) {
  const dim3 grid((a.keep + a.block - 1) / a.block, a.H, a.B);
  auto kern = a.block == 16   ? kv_evict_gather_kernel<QT, 16>
              : a.block == 32 ? kv_evict_gather_kernel<QT, 32>
              : a.block == 64 ? kv_evict_gather_kernel<QT, 64>
                              : kv_evict_gather_kernel<QT, 128>;
  return launch_pdl(kern, grid, dim3(kGatherThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kv_evict_q8(const KvEvictArgs& a, int qtype, cudaStream_t s) {
  // Threads that hold a head's weights at once: 256 for up to 4096 positions, then 512 in one to
  // eight CTAs, then 1024 in eight.  Small CTAs share an SM: 64 x 16 heads of 4096 65 us with 256
  // threads and 111 with 1024; 512 x 8192 46 us with 512 threads, 48 with two CTAs of 256, 64 with
  // 1024 (53 where 256 threads read the weights twice); 16 x 32768 12.7, 13.3 and 15.4 us; 64 x
  // 65536 36 us with eight CTAs of 512, 34 with four of 1024.
  auto ctas_for = [&](int threads) {
    int n = 1;
    while (n < 8 && a.Lmax > n * threads * kEach) n *= 2;
    return n;
  };
  const cudaError_t e = a.Lmax <= 256 * kEach       ? launch_select<256>(a, 1, s)
                        : a.Lmax <= 8 * 512 * kEach ? launch_select<512>(a, ctas_for(512), s)
                                                    : launch_select<1024>(a, 8, s);
  if (e != cudaSuccess) return e;
  return qtype == kE4m3 ? launch_gather<kE4m3>(a, s) : launch_gather<kInt8>(a, s);
}

}  // namespace mha
