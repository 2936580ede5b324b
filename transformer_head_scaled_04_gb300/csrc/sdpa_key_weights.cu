// sdpa_key_weights.cu -- the attention weight every key of a prompt received:
//   weights[b,g,j] += sum over the heads h of group g and the queries i of exp(s_ij - lse_i),
//   s_ij = q_i . k_j * scale, lse_i the forward's log-sum-exp of row i (mha_sdpa_fwd_lse)
// the column sums of the attention matrix, which is never stored.  A key belongs to one CTA, so
// the sums have one order and need no atomics.
//
// key_weights_simt_kernel: 32 keys per CTA, each warp taking every eighth query of the group's
// heads; lane = key, its row in registers, the queries broadcast from shared memory.
#include <cuda_bf16.h>

#include "launchers.h"
#include "device_common.cuh"

namespace mha {
namespace {

constexpr int kD = 64;
constexpr int kKeys = 32;     // keys per CTA
constexpr int kQueries = 32;  // queries staged at a time
constexpr int kWarps = 8;

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) key_weights_simt_kernel(const KeyWeightsArgs a) {
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's output is complete from here on
  const int g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int k0 = blockIdx.x * kKeys, j = k0 + lane;
  const int nk = a.mask == 2 ? min(max(__ldg(a.key_len + b), 0), a.Nk) : a.Nk;
  const int nq = a.query_len != nullptr ? min(max(__ldg(a.query_len + b), 0), a.Nq) : a.Nq;
  if (k0 >= nk) return;
  __shared__ float4 sq[kQueries][kD / 4];
  __shared__ float slse[kQueries];
  __shared__ float part[kWarps][kKeys];
  float k[kD];
  const T* kr = static_cast<const T*>(a.K) + b * a.sk[0] + g * a.sk[1] + min(j, nk - 1) * a.sk[2];
#pragma unroll
  for (int d = 0; d < kD; ++d) k[d] = to_f32(kr[d]);
  const int G = a.H / a.Hkv;
  const float c = a.scale * 1.4426950408889634f;
  const int first = a.mask == 1 ? k0 : 0;  // queries before the first key see none of these
  float sum = 0.f;
  for (int h = g * G; h < (g + 1) * G; ++h) {
    const T* q = static_cast<const T*>(a.Q) + b * a.sq[0] + h * a.sq[1];
    const float* lse = a.lse + (static_cast<int64_t>(b) * a.H + h) * a.Nq;
    for (int i0 = first; i0 < nq; i0 += kQueries) {
      __syncthreads();
      for (int t = tid; t < kQueries * kD; t += kWarps * 32) {
        const int i = i0 + t / kD;
        reinterpret_cast<float*>(sq)[t] = i < nq ? to_f32(q[i * a.sq[2] + t % kD]) : 0.f;
      }
      if (tid < kQueries)  // +inf (a row without keys, or none at all): every weight 0
        slse[tid] = i0 + tid < nq ? lse[i0 + tid] * 1.4426950408889634f : INFINITY;
      __syncthreads();
      for (int t = warp; t < kQueries && i0 + t < nq; t += kWarps) {
        float s = 0.f;
#pragma unroll
        for (int d = 0; d < kD / 4; ++d) {
          const float4 v = sq[t][d];
          s = fmaf(v.x, k[4 * d], s);
          s = fmaf(v.y, k[4 * d + 1], s);
          s = fmaf(v.z, k[4 * d + 2], s);
          s = fmaf(v.w, k[4 * d + 3], s);
        }
        const float l2 = slse[t];
        if (l2 != INFINITY && (a.mask != 1 || j <= i0 + t)) sum += exp2f(fmaf(s, c, -l2));
      }
    }
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && j < nk) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w][lane];
    a.weights[(static_cast<int64_t>(b) * a.Hkv + g) * a.ld + j] += s;
  }
}

}  // namespace

size_t key_weights_workspace(int B, int H, int Hkv, int Nq, int Nk, int dtype) {
  (void)B, (void)H, (void)Hkv, (void)Nq, (void)Nk, (void)dtype;
  return 0;
}

cudaError_t launch_key_weights_simt(const KeyWeightsArgs& a, int dtype, cudaStream_t s) {
  const dim3 grid((a.Nk + kKeys - 1) / kKeys, a.Hkv, a.B);
  return dtype == 1
             ? launch_pdl(key_weights_simt_kernel<__nv_bfloat16>, grid, dim3(kWarps * 32), 0, s, a)
             : launch_pdl(key_weights_simt_kernel<float>, grid, dim3(kWarps * 32), 0, s, a);
}

}  // namespace mha
