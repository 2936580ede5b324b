// sdpa_decode_q8.cu -- attention of a few new queries against an 8-bit key/value cache (see
// q8_common.cuh for the codes and scales), optionally adding every cached position's attention
// weight to a running total:
//   O[b,h,i] = sum_j p_ij v_j,  p_i = softmax_j(q_i . k_j * scale, allowed),
//   weights[b,g,j] += sum over the heads h of group g and the queries i of p_ij
// with k_j, v_j = code * scale of the block; allowed: j < L_b and, causal, j <= L_b - Nq + i.
// Head h reads the cache of head h / (H / Hkv).
//
// One CTA per (query, head, batch element): scores to the workspace, their max and sum, then O;
// a second launch adds the weights, one thread per cached position.
#include <cuda_bf16.h>

#include "launchers.h"
#include "q8_common.cuh"

namespace mha {
namespace {

constexpr int kD = 64;
constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

// keys that query i of the Nq newest may see
__device__ __forceinline__ int visible(const DecodeQ8Args& a, int L, int i) {
  return a.causal ? max(L - a.Nq + 1 + i, 0) : L;
}

template <typename T, int QT>
__global__ void __launch_bounds__(kThreads) decode_q8_kernel(const DecodeQ8Args a, float* ws) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int hk = h / (a.H / a.Hkv);
  const int L = min(max(__ldg(a.cache_len + b), 0), a.Lmax);
  const int n = visible(a, L, i);
  const int64_t row = (static_cast<int64_t>(b) * a.H + h) * a.Nq + i;
  float* x = ws + row * a.Lmax;
  float* stat = ws + static_cast<int64_t>(a.B) * a.H * a.Nq * a.Lmax + row * 2;
  __shared__ float sq[kD], red[kThreads], so[kThreads * 4];
  const T* q = static_cast<const T*>(a.Q) + b * a.sq[0] + h * a.sq[1] + i * a.sq[2];
  if (tid < kD) sq[tid] = to_f32(q[tid]);
  __syncthreads();
  const uint8_t* kc = static_cast<const uint8_t*>(a.Kc) + b * a.sk[0] + hk * a.sk[1];
  const uint8_t* vc = static_cast<const uint8_t*>(a.Vc) + b * a.sv[0] + hk * a.sv[1];
  const int64_t sb = (static_cast<int64_t>(b) * a.Hkv + hk) * a.n_blocks;
  float m = -INFINITY;
  for (int j = tid; j < n; j += kThreads) {
    const uint32_t* r = reinterpret_cast<const uint32_t*>(kc + j * a.sk[2]);
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      float f[4];
      q8_decode4<QT>(r[c], f);
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fmaf(sq[4 * c + e], f[e], s);
    }
    s *= a.k_scale[sb + j / a.block] * a.scale * 1.4426950408889634f;
    x[j] = s;
    m = fmaxf(m, s);
  }
  red[tid] = m;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (tid < o) red[tid] = fmaxf(red[tid], red[tid + o]);
    __syncthreads();
  }
  m = red[0] == -INFINITY ? 0.f : red[0];
  __syncthreads();
  float l = 0.f;
  for (int j = tid; j < n; j += kThreads) l += exp2f(x[j] - m);
  red[tid] = l;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (tid < o) red[tid] += red[tid + o];
    __syncthreads();
  }
  l = red[0];
  if (tid == 0) {
    stat[0] = m;
    stat[1] = l;
  }
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = tid >> 4; j < n; j += kThreads / 16) {
    float f[4];
    q8_decode4<QT>(reinterpret_cast<const uint32_t*>(vc + j * a.sv[2])[tid & 15], f);
    const float p = exp2f(x[j] - m) * a.v_scale[sb + j / a.block];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = fmaf(p, f[e], o[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) so[tid * 4 + e] = o[e];
  __syncthreads();
  if (tid < kD) {
    float y = 0.f;
    for (int g = 0; g < kThreads / 16; ++g) y += so[(g * 16 + tid / 4) * 4 + tid % 4];
    put(static_cast<T*>(a.O) + b * a.so[0] + h * a.so[1] + i * a.so[2] + tid,
        n > 0 ? y / l : 0.f);
  }
}

__global__ void __launch_bounds__(kThreads)
    decode_q8_weights_kernel(const DecodeQ8Args a, const float* ws) {
  pdl_launch_dependents();
  pdl_wait();  // scores and statistics are complete from here on
  const int hk = blockIdx.y, b = blockIdx.z;
  const int j = blockIdx.x * kThreads + threadIdx.x;
  const int L = min(max(__ldg(a.cache_len + b), 0), a.Lmax);
  if (j >= L) return;
  const int G = a.H / a.Hkv;
  const int64_t row0 = (static_cast<int64_t>(b) * a.H + hk * G) * a.Nq;
  const float* stat = ws + static_cast<int64_t>(a.B) * a.H * a.Nq * a.Lmax;
  float s = 0.f;
  for (int r = 0; r < G * a.Nq; ++r)
    if (j < visible(a, L, r % a.Nq))
      s += exp2f(ws[(row0 + r) * a.Lmax + j] - stat[(row0 + r) * 2]) / stat[(row0 + r) * 2 + 1];
  a.weights[(static_cast<int64_t>(b) * a.Hkv + hk) * a.Lmax + j] += s;
}

}  // namespace

size_t decode_q8_workspace(int B, int H, int Hkv, int Nq, int Lmax, bool weights) {
  (void)Hkv;
  (void)weights;
  return static_cast<size_t>(B) * H * Nq * (static_cast<size_t>(Lmax) + 2) * sizeof(float);
}

cudaError_t launch_sdpa_decode_q8(const DecodeQ8Args& a, int dtype, int qtype, void* ws,
                                  const DevCtx& ctx, cudaStream_t s) {
  (void)ctx;
  float* w = static_cast<float*>(ws);
  const dim3 grid(a.Nq, a.H, a.B);
  cudaError_t e;
  if (dtype == 1)
    e = qtype == kE4m3
            ? launch_pdl(decode_q8_kernel<__nv_bfloat16, kE4m3>, grid, dim3(kThreads), 0, s, a, w)
            : launch_pdl(decode_q8_kernel<__nv_bfloat16, kInt8>, grid, dim3(kThreads), 0, s, a, w);
  else
    e = qtype == kE4m3 ? launch_pdl(decode_q8_kernel<float, kE4m3>, grid, dim3(kThreads), 0, s, a, w)
                       : launch_pdl(decode_q8_kernel<float, kInt8>, grid, dim3(kThreads), 0, s, a, w);
  if (e != cudaSuccess || a.weights == nullptr) return e;
  return launch_pdl(decode_q8_weights_kernel, dim3((a.Lmax + kThreads - 1) / kThreads, a.Hkv, a.B),
                    dim3(kThreads), 0, s, a, static_cast<const float*>(w));
}

}  // namespace mha
