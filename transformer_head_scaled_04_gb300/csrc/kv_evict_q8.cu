// kv_evict_q8.cu -- drop the cached positions with the least accumulated attention weight and
// move the rest into another 8-bit cache (see q8_common.cuh for the codes and scales).
//
// Two launches.  select: per (batch element, head) the kept positions, ascending: the newest
// `recent` and, of the others, those with the largest weights (equal weights: the lower
// position).  The k-th largest weight is found by a radix descent over the weights' bits, eight
// at a time (the counts of one digit in shared memory), which reads the weights from L2 four
// times instead of sorting them; one more pass writes the positions in order.
// gather: one CTA per (block of the new cache, head, batch element) copies the block's rows; the
// block takes the largest scale of the tokens it receives, and codes that came under a smaller
// one are written under it.  Bound by HBM: 64 bytes read and written per row of K and of V.
#include <climits>

#include "launchers.h"
#include "q8_common.cuh"

namespace mha {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

// fp32 to an unsigned integer of the same order; -0 equals +0 and NaN the lowest value
__device__ __forceinline__ uint32_t order_key(float w) {
  if (!(w == w)) return 0x007fffffu;  // that of -inf
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) kv_evict_select_kernel(const KvEvictArgs a) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int64_t bh = static_cast<int64_t>(b) * a.H + h;
  const int L = min(max(__ldg(a.cache_len + b), 0), a.Lmax);
  int32_t* kept = a.kept + bh * a.keep;
  const int n_out = min(L, a.keep);
  if (h == 0 && tid == 0) a.len_out[b] = n_out;
  for (int i = n_out + tid; i < a.keep; i += kSelThreads) kept[i] = -1;
  if (L <= a.keep) {  // nothing to drop
    for (int i = tid; i < L; i += kSelThreads) kept[i] = i;
    return;
  }
  const float* w = a.weights + bh * a.Lmax;
  const int recent = min(a.recent, a.keep);
  const int m = L - recent;       // candidates: positions 0..m-1
  int k = a.keep - recent;        // of which the k largest stay, 0 <= k < m
  __shared__ int hist[256];
  __shared__ int s_digit, s_above;
  __shared__ int s_sum[2][kSelWarps];
  uint32_t prefix = 0;            // the high bits of the k-th largest key
  int above = 0;                  // candidates above the prefix so far
  for (int shift = 24; k > 0 && shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int j = tid; j < m; j += kSelThreads) {
      const uint32_t key = order_key(w[j]);
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(key >> shift) & 255u], 1);  // integers: any order gives the same count
    }
    __syncthreads();
    if (tid == 0) {
      int c = above, d = 255;
      while (d > 0 && c + hist[d] < k) c += hist[d--];
      s_digit = d;
      s_above = c;
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    above = s_above;
  }
  const int ties = k - above;  // candidates equal to the k-th largest that stay, lowest first
  // kept positions in order: running counts of the kept and of the ties
  int base = 0, tie_base = 0;
  for (int j0 = 0; j0 < L; j0 += kSelThreads) {
    const int j = j0 + tid;
    const uint32_t key = j < m ? order_key(w[j]) : 0u;
    const bool eq = k > 0 && j < m && key == prefix;
    const bool gt = (k > 0 && j < m && key > prefix) || (j >= m && j < L);
    const uint32_t be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_sum[0][warp] = __popc(be);
    __syncthreads();
    int tie = tie_base + __popc(be & ((1u << lane) - 1u)), ties_here = 0;
    for (int x = 0; x < kSelWarps; ++x) {
      if (x < warp) tie += s_sum[0][x];
      ties_here += s_sum[0][x];
    }
    const bool keep = gt || (eq && tie < ties);
    const uint32_t bk = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) s_sum[1][warp] = __popc(bk);
    __syncthreads();
    int at = base + __popc(bk & ((1u << lane) - 1u)), here = 0;
    for (int x = 0; x < kSelWarps; ++x) {
      if (x < warp) at += s_sum[1][x];
      here += s_sum[1][x];
    }
    if (keep) kept[at] = j;
    base += here;
    tie_base += ties_here;
    __syncthreads();
  }
}

constexpr int kGatherThreads = 256;  // 128 for K, 128 for V

template <int QT>
__global__ void __launch_bounds__(kGatherThreads) kv_evict_gather_kernel(const KvEvictArgs a) {
  pdl_launch_dependents();
  pdl_wait();  // the select kernel's positions are complete from here on
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * a.H + h;
  const int n_out = min(min(max(__ldg(a.cache_len + b), 0), a.Lmax), a.keep);
  const int lo = static_cast<int>(blockIdx.x) * a.block;
  const int rows = min(a.block, n_out - lo);
  if (rows <= 0) return;
  __shared__ int src[128];
  __shared__ float ssc[2][128];
  __shared__ float smax[8];
  const int part = threadIdx.x >> 7, tid = threadIdx.x & 127;
  const float* scale = (part ? a.v_scale : a.k_scale) + bh * a.n_blocks;
  float sc = 0.f;
  if (tid < rows) {
    const int j = a.kept[bh * a.keep + lo + tid];
    sc = scale[j / a.block];
    ssc[part][tid] = sc;
    if (part == 0) {
      src[tid] = j;
      if (a.weights_out != nullptr)
        a.weights_out[bh * a.Lmax_out + lo + tid] = a.weights[bh * a.Lmax + j];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sc = fmaxf(sc, __shfl_xor_sync(0xffffffffu, sc, o));
  if ((threadIdx.x & 31) == 0) smax[threadIdx.x >> 5] = sc;
  __syncthreads();
  const float now = fmaxf(fmaxf(smax[part * 4], smax[part * 4 + 1]),
                          fmaxf(smax[part * 4 + 2], smax[part * 4 + 3]));
  if (tid == 0) (part ? a.v_scale_out : a.k_scale_out)[bh * a.n_blocks_out + blockIdx.x] = now;
  const int64_t* si = part ? a.sv : a.sk;
  const int64_t* so = part ? a.svo : a.sko;
  const uint8_t* in = static_cast<const uint8_t*>(part ? a.Vc : a.Kc) + b * si[0] + h * si[1] +
                      (tid & 3) * 16;
  uint8_t* out = static_cast<uint8_t*>(part ? a.Vo : a.Ko) + b * so[0] + h * so[1] + lo * so[2] +
                 (tid & 3) * 16;
  for (int r = tid >> 2; r < rows; r += 32) {
    uint4 u = *reinterpret_cast<const uint4*>(in + src[r] * si[2]);
    const float was = ssc[part][r];
    if (was < now) {
      const float ratio = was / now;  // exact: powers of two
      u = make_uint4(q8_rescale4<QT>(u.x, ratio), q8_rescale4<QT>(u.y, ratio),
                     q8_rescale4<QT>(u.z, ratio), q8_rescale4<QT>(u.w, ratio));
    }
    *reinterpret_cast<uint4*>(out + r * so[2]) = u;
  }
}

}  // namespace

cudaError_t launch_kv_evict_q8(const KvEvictArgs& a, int qtype, cudaStream_t s) {
  cudaError_t e =
      launch_pdl(kv_evict_select_kernel, dim3(a.H, a.B), dim3(kSelThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.keep + a.block - 1) / a.block, a.H, a.B);
  return qtype == kE4m3
             ? launch_pdl(kv_evict_gather_kernel<kE4m3>, grid, dim3(kGatherThreads), 0, s, a)
             : launch_pdl(kv_evict_gather_kernel<kInt8>, grid, dim3(kGatherThreads), 0, s, a);
}

}  // namespace mha
