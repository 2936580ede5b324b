// capi_rel.cu -- the C ABI of attention with a learned relative position bias (declared in
// include/mha.h): argument validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mha.h"
#include "launchers.h"
#include "nvtx_range.h"

namespace {

using mha::DevCtx;

constexpr int kMaxRows = 1 << 24;  // positions of a sequence: distances and tile counts fit easily

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool valid_dtype(int dt) { return dt == MHA_F32 || dt == MHA_BF16; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int done(cudaError_t e) { return e == cudaSuccess ? MHA_OK : MHA_ERR_CUDA; }
float scale_of(float scale, int d_k) {
  return scale > 0.f ? scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(d_k)));
}

// the table and its buckets
int take_bias(const void* bias, int bias_dtype, int H, int num_buckets, int max_distance,
              int bidirectional, mha::RelBias* r) {
  if (bias == nullptr || !valid_dtype(bias_dtype) || (bidirectional != 0 && bidirectional != 1))
    return MHA_ERR_INVALID;
  if (num_buckets > mha::kRelMaxSeg || max_distance > mha::kRelFar) return MHA_ERR_UNSUPPORTED;
  if (!mha::rel_plan(num_buckets, max_distance, bidirectional != 0, r)) return MHA_ERR_INVALID;
  if (!aligned(bias, bias_dtype == MHA_F32 ? 4 : 2)) return MHA_ERR_ALIGN;
  r->table = bias;
  r->table_f32 = bias_dtype == MHA_F32;
  r->H = H;
  r->partial = nullptr;
  return MHA_OK;
}

// Element strides of `count` tensors [B, H, rows[t], dims[t]], the caller's or contiguous ones, and
// what the kernels ask of them and of the pointers.  written: bit t set for outputs.
int take_strides(const int64_t* strides, int count, int H, const int* rows, const int* dims,
                 const void* const* ptrs, unsigned written, int dtype, int64_t (*st)[4]) {
  for (int t = 0; t < count; ++t) {
    const int64_t cont[4] = {static_cast<int64_t>(H) * rows[t] * dims[t],
                             static_cast<int64_t>(rows[t]) * dims[t], dims[t], 1};
    for (int i = 0; i < 4; ++i) {
      st[t][i] = strides ? strides[4 * t + i] : cont[i];
      if (st[t][i] < 0) return MHA_ERR_INVALID;
    }
    if (st[t][3] != 1) return MHA_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
      if ((dtype == MHA_BF16 && (st[t][i] == 0 || st[t][i] % 8 != 0)) ||
          ((written >> t & 1) != 0 && st[t][i] == 0))
        return MHA_ERR_ALIGN;
    if (!aligned(ptrs[t], dtype == MHA_BF16 ? 16 : 4)) return MHA_ERR_ALIGN;
  }
  return MHA_OK;
}

// checks that all three calls share; rows: the longer of the sequences' lengths
int check_sizes(int B, int H, int rows, int d_k, int d_v, int dtype, float scale) {
  if (std::isnan(scale) || std::isinf(scale)) return MHA_ERR_INVALID;
  // the bf16 kernel adds bias / scale
  if (scale > 0.f && (scale < 0x1p-64f || scale > 0x1p64f)) return MHA_ERR_UNSUPPORTED;
  if (B > 65535 || H > 65535 || rows > kMaxRows) return MHA_ERR_UNSUPPORTED;
  if (dtype == MHA_BF16 ? d_k != 64 || d_v != 64 : d_k > 128 || d_v > 128)
    return MHA_ERR_UNSUPPORTED;
  return MHA_OK;
}

int check_mask(int mask, const int32_t* key_len, int Nq, int Nk) {
  if (mask < MHA_MASK_NONE || mask > MHA_MASK_KEY_PADDING) return MHA_ERR_INVALID;
  if (mask == MHA_MASK_CAUSAL && Nq != Nk) return MHA_ERR_INVALID;
  if (mask == MHA_MASK_KEY_PADDING && key_len == nullptr) return MHA_ERR_INVALID;
  return aligned(key_len, 4) ? MHA_OK : MHA_ERR_ALIGN;
}

#define REL_TRY(expr)                 \
  do {                                \
    const int st_ = (expr);           \
    if (st_ != MHA_OK) return st_;    \
  } while (0)

}  // namespace

extern "C" {

int mha_rel_bucket(int distance, int num_buckets, int max_distance, int bidirectional) {
  mha::RelBias r;
  if (num_buckets > mha::kRelMaxSeg || max_distance > mha::kRelFar) return MHA_ERR_UNSUPPORTED;
  if ((bidirectional != 0 && bidirectional != 1) ||
      !mha::rel_plan(num_buckets, max_distance, bidirectional != 0, &r))
    return MHA_ERR_INVALID;
  return mha::rel_bucket_of(r, distance);
}

int mha_sdpa_rel_fwd(int B, int H, int Nq, int Nk, int d_k, int d_v, int dtype, int mask,
                     const int32_t* key_len, float scale, const void* Q, const void* K,
                     const void* V, const void* bias, int bias_dtype, int num_buckets,
                     int max_distance, int bidirectional, void* O, const int64_t* strides,
                     float* lse, cudaStream_t stream) {
  MHA_NVTX_RANGE("mha_sdpa_rel_fwd");
  if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || d_k < 1 || d_v < 1 || !valid_dtype(dtype))
    return MHA_ERR_INVALID;
  if (Q == nullptr || K == nullptr || V == nullptr || O == nullptr) return MHA_ERR_INVALID;
  REL_TRY(check_mask(mask, key_len, Nq, Nk));
  REL_TRY(check_sizes(B, H, Nq > Nk ? Nq : Nk, d_k, d_v, dtype, scale));
  mha::RelBias rel;
  REL_TRY(take_bias(bias, bias_dtype, H, num_buckets, max_distance, bidirectional, &rel));
  const int rows[4] = {Nq, Nk, Nk, Nq}, dims[4] = {d_k, d_k, d_v, d_v};
  const void* ptrs[4] = {Q, K, V, O};
  int64_t st[4][4];
  REL_TRY(take_strides(strides, 4, H, rows, dims, ptrs, 8u, dtype, st));
  if (!aligned(lse, 4)) return MHA_ERR_ALIGN;
  DevCtx ctx;
  REL_TRY(mha::current_device_ctx(&ctx));
  mha::SdpaArgs a;
  a.B = B; a.H = H; a.Nq = Nq; a.Nk = Nk; a.d_k = d_k; a.d_v = d_v;
  a.mask = mask;
  a.key_len = mask == MHA_MASK_KEY_PADDING ? key_len : nullptr;
  a.scale = scale_of(scale, d_k);
  a.Q = Q; a.K = K; a.V = V; a.O = O;
  a.lse = lse;
  a.status = ctx.status;
  for (int i = 0; i < 4; ++i) {
    a.sq[i] = st[0][i];
    a.sk[i] = st[1][i];
    a.sv[i] = st[2][i];
    a.so[i] = st[3][i];
  }
  if (dtype == MHA_F32) return done(mha::launch_sdpa_rel_f32(a, rel, stream));
  CUtensorMap tq, tk, tv, to;
  if (!mha::encode_map_bf16(&tq, Q, B, H, Nq, st[0], 128) ||
      !mha::encode_map_bf16(&tk, K, B, H, Nk, st[1], 128) ||
      !mha::encode_map_bf16(&tv, V, B, H, Nk, st[2], 128) ||
      !mha::encode_map_bf16(&to, O, B, H, Nq, st[3], 32))
    return MHA_ERR_CUDA;
  return done(mha::launch_sdpa_rel_bf16(tq, tk, tv, to, a, rel, ctx, stream));
}

// the scratch of the backward without bias, then the tiles' sums of dS
static size_t bwd_partial_offset(int B, int H, int Nq, int dtype) {
  return round_up(mha::sdpa_bwd_scratch_bytes(B, H, Nq, dtype), 256);
}

int mha_sdpa_rel_bwd_workspace_size(int B, int H, int Nq, int Nk, int dtype, int num_buckets,
                                    size_t* bytes) {
  if (bytes == nullptr || B < 1 || H < 1 || Nq < 1 || Nk < 1 || !valid_dtype(dtype) ||
      num_buckets < 2)
    return MHA_ERR_INVALID;
  if (num_buckets > mha::kRelMaxSeg || B > 65535 || H > 65535 || Nq > kMaxRows || Nk > kMaxRows)
    return MHA_ERR_UNSUPPORTED;
  const size_t sums = static_cast<size_t>(B) * H * mha::rel_bwd_tiles(Nq, Nk, dtype) * num_buckets;
  *bytes = bwd_partial_offset(B, H, Nq, dtype) + round_up(sums * sizeof(float), 256);
  return MHA_OK;
}

int mha_sdpa_rel_bwd(int B, int H, int Nq, int Nk, int d_k, int d_v, int dtype, int mask,
                     const int32_t* key_len, float scale, const void* Q, const void* K,
                     const void* V, const void* bias, int bias_dtype, int num_buckets,
                     int max_distance, int bidirectional, const void* O, const void* dO,
                     const float* lse, void* dQ, void* dK, void* dV, void* dbias,
                     const int64_t* strides, void* workspace, size_t ws_bytes,
                     cudaStream_t stream) {
  MHA_NVTX_RANGE("mha_sdpa_rel_bwd");
  if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || d_k < 1 || d_v < 1 || !valid_dtype(dtype))
    return MHA_ERR_INVALID;
  const void* ptrs[8] = {Q, K, V, O, dO, dQ, dK, dV};
  for (const void* q : ptrs)
    if (q == nullptr) return MHA_ERR_INVALID;
  if (lse == nullptr || dbias == nullptr) return MHA_ERR_INVALID;
  REL_TRY(check_mask(mask, key_len, Nq, Nk));
  REL_TRY(check_sizes(B, H, Nq > Nk ? Nq : Nk, d_k, d_v, dtype, scale));
  mha::RelBias rel;
  REL_TRY(take_bias(bias, bias_dtype, H, num_buckets, max_distance, bidirectional, &rel));
  if (!aligned(lse, 4) || !aligned(dbias, bias_dtype == MHA_F32 ? 4 : 2)) return MHA_ERR_ALIGN;
  mha::SdpaBwdArgs a;
  const int rows[8] = {Nq, Nk, Nk, Nq, Nq, Nq, Nk, Nk};
  const int dims[8] = {d_k, d_k, d_v, d_v, d_v, d_k, d_k, d_v};
  REL_TRY(take_strides(strides, 8, H, rows, dims, ptrs, 0xe0u, dtype, a.st));
  size_t need = 0;
  REL_TRY(mha_sdpa_rel_bwd_workspace_size(B, H, Nq, Nk, dtype, num_buckets, &need));
  if (workspace == nullptr || ws_bytes < need) return MHA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MHA_ERR_ALIGN;
  DevCtx ctx;
  REL_TRY(mha::current_device_ctx(&ctx));
  a.B = B; a.H = H; a.Nq = Nq; a.Nk = Nk; a.d_k = d_k; a.d_v = d_v;
  a.mask = mask;
  a.window = 0;
  a.key_len = mask == MHA_MASK_KEY_PADDING ? key_len : nullptr;
  a.scale = scale_of(scale, d_k);
  a.Q = Q; a.K = K; a.V = V; a.O = O; a.dO = dO;
  a.lse = lse;
  a.Dv = static_cast<float*>(workspace);
  a.deterministic = mha_get_deterministic() != 0;
  a.dQ = dQ; a.dK = dK; a.dV = dV;
  rel.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                         bwd_partial_offset(B, H, Nq, dtype));
  cudaError_t e;
  if (dtype == MHA_BF16) {
    CUtensorMap tq, tk, tv, tg, tdq;
    const void* acc = reinterpret_cast<const char*>(a.Dv) + mha::sdpa_bwd_dq_acc_offset(B, H, Nq);
    if (!mha::encode_map_bf16(&tq, Q, B, H, Nq, a.st[0], 128) ||
        !mha::encode_map_bf16(&tk, K, B, H, Nk, a.st[1], 128) ||
        !mha::encode_map_bf16(&tv, V, B, H, Nk, a.st[2], 128) ||
        !mha::encode_map_bf16(&tg, dO, B, H, Nq, a.st[4], 128) ||
        !mha::encode_map_dq_acc(&tdq, acc, B, H, (Nq + 127) / 128 * 128))
      return MHA_ERR_CUDA;
    e = mha::launch_sdpa_bwd_rowdot(a, dtype, stream);
    if (e == cudaSuccess)
      e = mha::launch_sdpa_rel_bwd_bf16(tq, tk, tv, tg, tdq, a, rel, dbias, ctx, stream);
  } else {
    e = mha::launch_sdpa_rel_bwd_f32(a, rel, dbias, stream);
  }
  return done(e);
}

int mha_sdpa_rel_decode_workspace_size(int B, int H, int Nq, int Lmax, int d_k, int d_v, int dtype,
                                       size_t* bytes) {
  if (bytes == nullptr || B < 1 || H < 1 || Nq < 1 || Lmax < 1 || d_k < 1 || d_v < 1 ||
      !valid_dtype(dtype))
    return MHA_ERR_INVALID;
  if (Nq > mha::kDecodeMaxQ) return MHA_ERR_UNSUPPORTED;
  REL_TRY(check_sizes(B, H, Lmax, d_k, d_v, dtype, 0.f));
  *bytes = round_up(mha::rel_decode_workspace(B, H, Nq, Lmax, d_k, d_v, dtype), 256);
  return MHA_OK;
}

int mha_sdpa_rel_decode_fwd(int B, int H, int Nq, int Lmax, int d_k, int d_v, int dtype, int causal,
                            const int32_t* cache_len, float scale, const void* Q, const void* K,
                            const void* V, const void* bias, int bias_dtype, int num_buckets,
                            int max_distance, int bidirectional, void* O, const int64_t* strides,
                            void* workspace, size_t ws_bytes, cudaStream_t stream) {
  MHA_NVTX_RANGE("mha_sdpa_rel_decode_fwd");
  if (B < 1 || H < 1 || Nq < 1 || Lmax < 1 || d_k < 1 || d_v < 1 || !valid_dtype(dtype) ||
      (causal != 0 && causal != 1) || Nq > Lmax)
    return MHA_ERR_INVALID;
  if (cache_len == nullptr || Q == nullptr || K == nullptr || V == nullptr || O == nullptr)
    return MHA_ERR_INVALID;
  if (!aligned(cache_len, 4)) return MHA_ERR_ALIGN;
  REL_TRY(check_sizes(B, H, Lmax, d_k, d_v, dtype, scale));
  size_t need = 0;
  REL_TRY(mha_sdpa_rel_decode_workspace_size(B, H, Nq, Lmax, d_k, d_v, dtype, &need));
  mha::RelBias rel;
  REL_TRY(take_bias(bias, bias_dtype, H, num_buckets, max_distance, bidirectional, &rel));
  mha::RelDecodeArgs a;
  const int rows[4] = {Nq, Lmax, Lmax, Nq}, dims[4] = {d_k, d_k, d_v, d_v};
  const void* ptrs[4] = {Q, K, V, O};
  REL_TRY(take_strides(strides, 4, H, rows, dims, ptrs, 8u, dtype, a.st));
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return MHA_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return MHA_ERR_ALIGN;
  DevCtx ctx;
  REL_TRY(mha::current_device_ctx(&ctx));
  a.B = B; a.H = H; a.Nq = Nq; a.Lmax = Lmax; a.d_k = d_k; a.d_v = d_v;
  a.causal = causal;
  a.cache_len = cache_len;
  a.scale = scale_of(scale, d_k);
  a.Q = Q; a.K = K; a.V = V; a.O = O;
  return done(mha::launch_sdpa_rel_decode(a, rel, dtype, static_cast<float*>(workspace), stream));
}

}  // extern "C"
