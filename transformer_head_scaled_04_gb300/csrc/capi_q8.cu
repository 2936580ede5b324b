// capi_q8.cu -- the C ABI of the 8-bit key/value cache (declared in include/mha.h): argument
// validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mha.h"
#include "launchers.h"
#include "nvtx_range.h"

namespace {

using mha::DevCtx;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool valid_dtype(int dt) { return dt == MHA_F32 || dt == MHA_BF16; }
bool valid_qtype(int qt) { return qt == MHA_Q8_E4M3 || qt == MHA_Q8_I8; }
bool valid_block(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }
int blocks_of(int Lmax, int block) { return (Lmax - 1) / block + 1; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// element strides {b, h, n, d} of tensor t: the caller's, or those of a contiguous
// [B, H, N, 64]; `unit` is what 16 bytes hold
int take_strides(const int64_t* strides, int t, int64_t H, int64_t N, int64_t unit,
                 int64_t (&out)[4]) {
  const int64_t cont[4] = {H * N * 64, N * 64, 64, 1};
  for (int i = 0; i < 4; ++i) {
    out[i] = strides ? strides[4 * t + i] : cont[i];
    if (out[i] < 0) return MHA_ERR_INVALID;
  }
  if (out[3] != 1) return MHA_ERR_UNSUPPORTED;
  for (int i = 0; i < 3; ++i)
    if (out[i] == 0 || out[i] % unit != 0) return MHA_ERR_ALIGN;
  return MHA_OK;
}

int64_t unit_of(int dtype) { return dtype == MHA_BF16 ? 8 : 4; }
int done(cudaError_t e) { return e == cudaSuccess ? MHA_OK : MHA_ERR_CUDA; }

// scale <= 0 means 1/sqrt(64)
float scale_of(float scale) { return scale > 0.f ? scale : 0.125f; }

}  // namespace

extern "C" {

int mha_kv_append_q8(int B, int H, int N, int Lmax, int d_k, int d_v, int dtype, int qtype,
                     int block, const int32_t* new_len, const int32_t* cache_len, const void* K,
                     const void* V, void* K_cache, void* V_cache, float* k_scale, float* v_scale,
                     float* weights, const int64_t* strides, cudaStream_t stream) {
  MHA_NVTX_RANGE("mha_kv_append_q8");
  if (B < 1 || H < 1 || N < 1 || Lmax < 1 || d_k < 1 || d_v < 1 || !valid_dtype(dtype) ||
      !valid_qtype(qtype))
    return MHA_ERR_INVALID;
  if (cache_len == nullptr || K == nullptr || V == nullptr || K_cache == nullptr ||
      V_cache == nullptr || k_scale == nullptr || v_scale == nullptr)
    return MHA_ERR_INVALID;
  if (K_cache == V_cache || k_scale == v_scale) return MHA_ERR_INVALID;
  if (d_k != 64 || d_v != 64 || !valid_block(block) || B > 65535 || H > 65535 ||
      N > (1 << 30) || Lmax > (1 << 30))
    return MHA_ERR_UNSUPPORTED;
  mha::KvAppendArgs a;
  int st = take_strides(strides, 0, H, N, unit_of(dtype), a.sk);
  if (st == MHA_OK) st = take_strides(strides, 1, H, N, unit_of(dtype), a.sv);
  if (st == MHA_OK) st = take_strides(strides, 2, H, Lmax, 16, a.skc);
  if (st == MHA_OK) st = take_strides(strides, 3, H, Lmax, 16, a.svc);
  if (st != MHA_OK) return st;
  for (const void* q : {K, V, static_cast<const void*>(K_cache), static_cast<const void*>(V_cache)})
    if (!aligned(q, 16)) return MHA_ERR_ALIGN;
  if (!aligned(cache_len, 4) || !aligned(new_len, 4) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(weights, 4))
    return MHA_ERR_ALIGN;
  DevCtx ctx;
  st = mha::current_device_ctx(&ctx);
  if (st != MHA_OK) return st;
  a.B = B; a.H = H; a.N = N; a.Lmax = Lmax; a.block = block; a.n_blocks = blocks_of(Lmax, block);
  a.new_len = new_len; a.cache_len = cache_len;
  a.K = K; a.V = V; a.Kc = K_cache; a.Vc = V_cache;
  a.k_scale = k_scale; a.v_scale = v_scale; a.weights = weights;
  return done(mha::launch_kv_append_q8(a, dtype, qtype, stream));
}

int mha_decode_q8_workspace_size(int B, int H, int Hkv, int Nq, int Lmax, int with_weights,
                                 size_t* bytes) {
  if (bytes == nullptr || B < 1 || H < 1 || Hkv < 1 || Nq < 1 || Lmax < 1 || H % Hkv != 0 ||
      (with_weights != 0 && with_weights != 1))
    return MHA_ERR_INVALID;
  // rows of a cache head in the join's shared memory, blocks of its grid, tiles of all heads
  const int64_t rows = static_cast<int64_t>(H / Hkv) * Nq, heads = static_cast<int64_t>(B) * Hkv;
  if (Nq > mha::kDecodeMaxQ || Lmax > (1 << 30) || rows > 4096 || heads * rows > (1 << 28) ||
      heads * ((rows + 7) / 8) * ((Lmax + 31) / 32) >= (1LL << 31))
    return MHA_ERR_UNSUPPORTED;
  *bytes = round_up(mha::decode_q8_workspace(B, H, Hkv, Nq, Lmax, with_weights != 0), 256);
  return MHA_OK;
}

int mha_sdpa_decode_q8_fwd(int B, int H, int Hkv, int Nq, int Lmax, int d_k, int d_v, int dtype,
                           int qtype, int block, int causal, const int32_t* cache_len,
                           float scale, const void* Q, const void* K_cache, const void* V_cache,
                           const float* k_scale, const float* v_scale, void* O,
                           const int64_t* strides, float* weights, void* workspace,
                           size_t ws_bytes, cudaStream_t stream) {
  MHA_NVTX_RANGE("mha_sdpa_decode_q8_fwd");
  if (B < 1 || H < 1 || Hkv < 1 || Nq < 1 || Lmax < 1 || d_k < 1 || d_v < 1 ||
      !valid_dtype(dtype) || !valid_qtype(qtype) || H % Hkv != 0)
    return MHA_ERR_INVALID;
  if ((causal != 0 && causal != 1) || Nq > Lmax) return MHA_ERR_INVALID;
  if (cache_len == nullptr || Q == nullptr || K_cache == nullptr || V_cache == nullptr ||
      k_scale == nullptr || v_scale == nullptr || O == nullptr)
    return MHA_ERR_INVALID;
  if (std::isnan(scale) || std::isinf(scale)) return MHA_ERR_INVALID;
  if (d_k != 64 || d_v != 64 || !valid_block(block) || B > 65535 || H > 65535)
    return MHA_ERR_UNSUPPORTED;
  mha::DecodeQ8Args a;
  int st = take_strides(strides, 0, H, Nq, unit_of(dtype), a.sq);
  if (st == MHA_OK) st = take_strides(strides, 1, Hkv, Lmax, 16, a.sk);
  if (st == MHA_OK) st = take_strides(strides, 2, Hkv, Lmax, 16, a.sv);
  if (st == MHA_OK) st = take_strides(strides, 3, H, Nq, unit_of(dtype), a.so);
  if (st != MHA_OK) return st;
  for (const void* q : {Q, K_cache, V_cache, static_cast<const void*>(O)})
    if (!aligned(q, 16)) return MHA_ERR_ALIGN;
  if (!aligned(cache_len, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(weights, 4))
    return MHA_ERR_ALIGN;
  size_t need = 0;
  st = mha_decode_q8_workspace_size(B, H, Hkv, Nq, Lmax, weights != nullptr ? 1 : 0, &need);
  if (st != MHA_OK) return st;
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return MHA_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return MHA_ERR_ALIGN;
  DevCtx ctx;
  st = mha::current_device_ctx(&ctx);
  if (st != MHA_OK) return st;
  a.B = B; a.H = H; a.Hkv = Hkv; a.Nq = Nq; a.Lmax = Lmax; a.block = block;
  a.n_blocks = blocks_of(Lmax, block);
  a.causal = causal; a.cache_len = cache_len; a.scale = scale_of(scale);
  a.Q = Q; a.Kc = K_cache; a.Vc = V_cache; a.k_scale = k_scale; a.v_scale = v_scale; a.O = O;
  a.weights = weights;
  return done(mha::launch_sdpa_decode_q8(a, dtype, qtype, workspace, ctx, stream));
}

int mha_key_weights_workspace_size(int B, int H, int Hkv, int Nq, int Nk, int dtype,
                                   size_t* bytes) {
  if (bytes == nullptr || B < 1 || H < 1 || Hkv < 1 || Nq < 1 || Nk < 1 || H % Hkv != 0 ||
      !valid_dtype(dtype))
    return MHA_ERR_INVALID;
  // blocks of the launch's grids (queries are split, and heads a grid's y, only where key tiles
  // are few)
  const int64_t heads = static_cast<int64_t>(B) * Hkv;
  if (B > 65535 || H > 65535 || heads * ((Nk + 127) / 128) > (1 << 30) || Nq > (1 << 30) ||
      static_cast<int64_t>(H / Hkv) * ((Nq + 31) / 32) > (1 << 30))
    return MHA_ERR_UNSUPPORTED;
  *bytes = round_up(mha::key_weights_workspace(B, H, Hkv, Nq, Nk, dtype), 256);
  return MHA_OK;
}

int mha_sdpa_key_weights(int B, int H, int Hkv, int Nq, int Nk, int d_k, int dtype, int mask,
                         const int32_t* key_len, const int32_t* query_len, float scale,
                         const void* Q, const void* K, const float* lse, const int64_t* strides,
                         float* weights, int64_t weights_ld, void* workspace, size_t ws_bytes,
                         cudaStream_t stream) {
  MHA_NVTX_RANGE("mha_sdpa_key_weights");
  if (B < 1 || H < 1 || Hkv < 1 || Nq < 1 || Nk < 1 || d_k < 1 || !valid_dtype(dtype) ||
      H % Hkv != 0 || mask < MHA_MASK_NONE || mask > MHA_MASK_KEY_PADDING)
    return MHA_ERR_INVALID;
  if ((mask == MHA_MASK_CAUSAL && Nq != Nk) ||
      (mask == MHA_MASK_KEY_PADDING && key_len == nullptr))
    return MHA_ERR_INVALID;
  if (Q == nullptr || K == nullptr || lse == nullptr || weights == nullptr || weights_ld < Nk)
    return MHA_ERR_INVALID;
  if (std::isnan(scale) || std::isinf(scale)) return MHA_ERR_INVALID;
  if (d_k != 64 || B > 65535 || H > 65535 || Nq > (1 << 30) || Nk > (1 << 30))
    return MHA_ERR_UNSUPPORTED;
  mha::KeyWeightsArgs a;
  int st = take_strides(strides, 0, H, Nq, unit_of(dtype), a.sq);
  if (st == MHA_OK) st = take_strides(strides, 1, Hkv, Nk, unit_of(dtype), a.sk);
  if (st != MHA_OK) return st;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(lse, 4) || !aligned(weights, 4) ||
      !aligned(key_len, 4) || !aligned(query_len, 4))
    return MHA_ERR_ALIGN;
  size_t need = 0;
  st = mha_key_weights_workspace_size(B, H, Hkv, Nq, Nk, dtype, &need);
  if (st != MHA_OK) return st;
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return MHA_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return MHA_ERR_ALIGN;
  DevCtx ctx;
  st = mha::current_device_ctx(&ctx);
  if (st != MHA_OK) return st;
  a.B = B; a.H = H; a.Hkv = Hkv; a.Nq = Nq; a.Nk = Nk; a.mask = mask;
  a.key_len = mask == MHA_MASK_KEY_PADDING ? key_len : nullptr;
  a.query_len = query_len;
  a.scale = scale_of(scale);
  a.Q = Q; a.K = K; a.lse = lse; a.weights = weights; a.ld = weights_ld;
  return done(mha::launch_key_weights(a, dtype, workspace, ctx, stream));
}

int mha_kv_evict_q8(int B, int H, int Lmax, int Lmax_out, int d_k, int d_v, int qtype, int block,
                    int keep, int recent, const int32_t* cache_len, const void* K_cache,
                    const void* V_cache, const float* k_scale, const float* v_scale,
                    const float* weights, void* K_out, void* V_out, float* k_scale_out,
                    float* v_scale_out, float* weights_out, int32_t* len_out, int32_t* kept,
                    const int64_t* strides, cudaStream_t stream) {
  MHA_NVTX_RANGE("mha_kv_evict_q8");
  if (B < 1 || H < 1 || Lmax < 1 || Lmax_out < 1 || d_k < 1 || d_v < 1 || !valid_qtype(qtype) ||
      keep < 1 || keep > Lmax_out || recent < 0)
    return MHA_ERR_INVALID;
  const void* req[12] = {cache_len, K_cache, V_cache, k_scale,     v_scale, weights,
                         K_out,     V_out,   k_scale_out, v_scale_out, len_out, kept};
  for (const void* q : req)
    if (q == nullptr) return MHA_ERR_INVALID;
  // every output its own memory: none of them an input, nor one another
  const void* in[6] = {cache_len, K_cache, V_cache, k_scale, v_scale, weights};
  const void* out[7] = {K_out, V_out, k_scale_out, v_scale_out, weights_out, len_out, kept};
  for (int i = 0; i < 7; ++i) {
    if (out[i] == nullptr) continue;
    for (const void* q : in)
      if (out[i] == q) return MHA_ERR_INVALID;
    for (int k = 0; k < i; ++k)
      if (out[i] == out[k]) return MHA_ERR_INVALID;
  }
  if (d_k != 64 || d_v != 64 || !valid_block(block) || B > 65535 || H > 65535 ||
      static_cast<int64_t>(B) * H > (1 << 27) || Lmax > (1 << 30) || Lmax_out > (1 << 30))
    return MHA_ERR_UNSUPPORTED;
  mha::KvEvictArgs a;
  int st = take_strides(strides, 0, H, Lmax, 16, a.sk);
  if (st == MHA_OK) st = take_strides(strides, 1, H, Lmax, 16, a.sv);
  if (st == MHA_OK) st = take_strides(strides, 2, H, Lmax_out, 16, a.sko);
  if (st == MHA_OK) st = take_strides(strides, 3, H, Lmax_out, 16, a.svo);
  if (st != MHA_OK) return st;
  for (const void* q : {K_cache, V_cache, static_cast<const void*>(K_out),
                        static_cast<const void*>(V_out)})
    if (!aligned(q, 16)) return MHA_ERR_ALIGN;
  const void* words[9] = {cache_len,   k_scale,     v_scale, weights, k_scale_out,
                          v_scale_out, weights_out, len_out, kept};
  for (const void* q : words)
    if (!aligned(q, 4)) return MHA_ERR_ALIGN;
  DevCtx ctx;
  st = mha::current_device_ctx(&ctx);
  if (st != MHA_OK) return st;
  a.B = B; a.H = H; a.Lmax = Lmax; a.Lmax_out = Lmax_out; a.block = block;
  a.n_blocks = blocks_of(Lmax, block); a.n_blocks_out = blocks_of(Lmax_out, block);
  a.keep = keep; a.recent = recent; a.cache_len = cache_len;
  a.Kc = K_cache; a.Vc = V_cache; a.k_scale = k_scale; a.v_scale = v_scale; a.weights = weights;
  a.Ko = K_out; a.Vo = V_out; a.k_scale_out = k_scale_out; a.v_scale_out = v_scale_out;
  a.weights_out = weights_out; a.len_out = len_out; a.kept = kept;
  return done(mha::launch_kv_evict_q8(a, qtype, stream));
}

}  // extern "C"
