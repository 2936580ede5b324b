// kv_append_q8.cu -- new keys and values into an 8-bit key/value cache (see q8_common.cuh for
// the codes and scales).
//
// One CTA per (block of tokens, head, batch element) that new tokens touch, 128 threads for the
// keys and 128 for the values, so a block's scale has one writer and needs no atomics.  Bound by
// HBM for prompts (2 or 4 bytes read and 1 written per value); for single tokens by the launch.
// Each thread holds 16 values of a row: four threads read a row's 64 values, so a warp's loads
// cover whole rows.  Prompts of 4096 tokens to 8 x 16 heads, bf16: 34 us in integers, 33 in e4m3,
// 6.0 TB/s (integers took 49 us instead of 44 when values were widened to fp32 as they arrived:
// fewer loads in flight); one token to 64 x 16 heads 4.2 us.
#include <cuda_bf16.h>

#include "launchers.h"
#include "q8_common.cuh"

namespace mha {
namespace {

constexpr int kD = 64;
constexpr int kThreads = 256;  // 128 for K, 128 for V

// 16 values as they are stored, and as fp32
__device__ __forceinline__ void widen(const uint4 (&u)[2], float (&f)[16]) {  // bf16
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
      f[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void widen(const uint4 (&u)[4], float (&f)[16]) {  // fp32
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[4 * i] = __uint_as_float(u[i].x);
    f[4 * i + 1] = __uint_as_float(u[i].y);
    f[4 * i + 2] = __uint_as_float(u[i].z);
    f[4 * i + 3] = __uint_as_float(u[i].w);
  }
}

// largest finite magnitude
template <int N>
__device__ __forceinline__ float largest_fp32(const uint4 (&u)[N]) {
  float f[16], amax = 0.f;
  widen(u, f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float m = fabsf(f[i]);
    amax = m <= 3.402823466e38f ? fmaxf(amax, m) : amax;  // false for inf and NaN
  }
  return amax;
}
__device__ __forceinline__ float largest(const uint4 (&u)[4]) { return largest_fp32(u); }
__device__ __forceinline__ float largest(const uint4 (&u)[2]) {
  // magnitudes compare as integers, two at a time; inf and NaN are the largest, and seldom there
  // (prompts as above 36.4 -> 34.2 us)
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) m = __vmaxu2(m, w[k] & 0x7fff7fffu);
  }
  m = max(m >> 16, m & 0xffffu);
  return m < 0x7f80u ? __uint_as_float(m << 16) : largest_fp32(u);
}

// BLOCK: tokens per scale
template <typename T, int QT, int BLOCK>
__global__ void __launch_bounds__(kThreads) kv_append_q8_kernel(const KvAppendArgs a) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  constexpr int kRows = (BLOCK + 31) / 32;  // rows of a block that one thread takes a part of
  const int h = blockIdx.y, b = blockIdx.z;
  const int L = min(max(__ldg(a.cache_len + b), 0), a.Lmax);
  const int n = a.new_len == nullptr ? a.N : min(max(__ldg(a.new_len + b), 0), a.N);
  const int blk = L / BLOCK + static_cast<int>(blockIdx.x);
  // positions first..end-1 of this block are new, lo..first-1 are there already
  const int64_t lo = static_cast<int64_t>(blk) * BLOCK;
  const int64_t end64 = min(min(static_cast<int64_t>(L) + n, static_cast<int64_t>(a.Lmax)),
                            lo + BLOCK);
  const int64_t first64 = max(lo, static_cast<int64_t>(L));
  if (first64 >= end64) return;  // uniform over the block
  const int first = static_cast<int>(first64 - lo), end = static_cast<int>(end64 - lo);

  const int part = threadIdx.x >> 7, tid = threadIdx.x & 127;
  const int row0 = tid >> 2, chunk = tid & 3;
  const T* x = static_cast<const T*>(part ? a.V : a.K);
  const int64_t* sx = part ? a.sv : a.sk;
  uint8_t* cache = static_cast<uint8_t*>(part ? a.Vc : a.Kc);
  const int64_t* sc = part ? a.svc : a.skc;
  float* scale = (part ? a.v_scale : a.k_scale) +
                 (static_cast<int64_t>(b) * a.H + h) * a.n_blocks + blk;
  x += b * sx[0] + h * sx[1] + (lo - L) * sx[2] + chunk * 16;
  cache += b * sc[0] + h * sc[1] + lo * sc[2] + chunk * 16;

  // largest finite magnitude of the block's new tokens
  constexpr int kQuads = sizeof(T);  // 16-byte loads of 16 values
  uint4 raw[kRows][kQuads];          // as stored: half the registers of fp32 for bf16
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = row0 + 32 * k;
    if (r >= first && r < end)
#pragma unroll
      for (int i = 0; i < kQuads; ++i)
        raw[k][i] = reinterpret_cast<const uint4*>(x + r * sx[2])[i];
  }
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = row0 + 32 * k;
    if (r >= first && r < end) amax = fmaxf(amax, largest(raw[k]));
  }
  __shared__ float smax[8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) smax[threadIdx.x >> 5] = amax;
  const float was = first > 0 ? *scale : 0.f;
  __syncthreads();  // also: every thread has read the old scale
  amax = fmaxf(fmaxf(smax[part * 4], smax[part * 4 + 1]),
               fmaxf(smax[part * 4 + 2], smax[part * 4 + 3]));
  const float fresh = pow2i(q8_exponent<QT>(amax));
  const float now = fmaxf(was, fresh);
  if (tid == 0) *scale = now;
  // (exact for the library's own scales, powers of two; under another that was there x * inv is
  // what is rounded to the code)
  const float inv = 1.f / now;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = row0 + 32 * k;
    uint4* dst = reinterpret_cast<uint4*>(cache + r * sc[2]);
    if (r >= first && r < end) {
      float f[16];
      widen(raw[k], f);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = q8_encode4<QT>(f[4 * i] * inv, f[4 * i + 1] * inv, f[4 * i + 2] * inv,
                              f[4 * i + 3] * inv);
      *dst = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (r < first && now > was) {  // tokens that were there, under the larger scale
      const float ratio = was * inv;
      const uint4 u = *dst;
      *dst = make_uint4(q8_rescale4<QT>(u.x, ratio), q8_rescale4<QT>(u.y, ratio),
                        q8_rescale4<QT>(u.z, ratio), q8_rescale4<QT>(u.w, ratio));
    }
  }
  if (a.weights != nullptr)
    for (int r = first + static_cast<int>(threadIdx.x); r < end; r += kThreads)
      a.weights[(static_cast<int64_t>(b) * a.H + h) * a.Lmax + lo + r] = 0.f;
}

template <typename T, int QT>
cudaError_t launch_block(const KvAppendArgs& a, dim3 grid, cudaStream_t s) {
  switch (a.block) {
    case 16: return launch_pdl(kv_append_q8_kernel<T, QT, 16>, grid, dim3(kThreads), 0, s, a);
    case 32: return launch_pdl(kv_append_q8_kernel<T, QT, 32>, grid, dim3(kThreads), 0, s, a);
    case 64: return launch_pdl(kv_append_q8_kernel<T, QT, 64>, grid, dim3(kThreads), 0, s, a);
    default: return launch_pdl(kv_append_q8_kernel<T, QT, 128>, grid, dim3(kThreads), 0, s, a);
  }
}

}  // namespace

cudaError_t launch_kv_append_q8(const KvAppendArgs& a, int dtype, int qtype, cudaStream_t s) {
  // N tokens that begin inside a block touch one block more than their number asks for
  const dim3 grid((a.N + 2 * a.block - 2) / a.block, a.H, a.B);
  if (dtype == 1)
    return qtype == kE4m3 ? launch_block<__nv_bfloat16, kE4m3>(a, grid, s)
                          : launch_block<__nv_bfloat16, kInt8>(a, grid, s);
  return qtype == kE4m3 ? launch_block<float, kE4m3>(a, grid, s)
                        : launch_block<float, kInt8>(a, grid, s);
}

}  // namespace mha
