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
//   - every warp streams its tiles through a ring of its own, 12 KB of 16-byte asynchronous
//     copies in flight, without a barrier between warps.  (Bulk copies issued by one lane and
//     waited for on mbarriers cost that warp 1200 of a tile's 3400 cycles.)
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
//     maximum of x_j + log2 s_j the weights p_j that meet the value codes lie in [0, 2^13].
//     Blocks whose scales are more than 2^10 apart are summed under references of their own
//     (careful_tile), since fp16 holds nothing below 2^-25.
// Precision: scores, statistics and sums are fp32.  Queries are scaled by a power of two (their
// row's largest value to [2^13, 2^14)) and rounded to fp16, which holds every bf16 significand;
// fp32 queries and weights are split into two fp16 terms (22 bits) and their products done
// twice, each inner step's part of a score and each tile's PV summed apart and added in fp32
// (the tensor cores' own accumulation truncates).  With bf16 queries the four inner steps and the
// tiles' PV are summed by the tensor cores and a weight is one fp16 term, 2^-11 off at most: an
// eighth of the output's own rounding to bf16 even if all of a row's weights erred alike.  Beyond
// references of 4096 exponents are differences of two scores, rounded as the stored ones.
// Runs end at heads' ends: each piece leaves (O, m, l) in the workspace, and a second launch
// joins a row's pieces, and adds the weights 2^(x_ij - m_i) / l_i from the scores that the first
// one stored.  Short caches of few heads take one launch, a block to a head, whose warps' pieces
// and scores meet in shared memory.  No atomics: one order of sums.
// 64 x 16 heads x 4096 positions 85 us (6.3 TB/s), with weights 101; 8 x 8 heads of 16 rows and up
// to 16384 positions, with weights, 31; 8 heads x 131072, fp32, 29; 8 heads x 37 4.1.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "launchers.h"
#include "mma_f16.cuh"
#include "q8_common.cuh"

namespace mha {
namespace {

constexpr int kD = 64;
constexpr int kTile = 32;                  // positions per tile
constexpr int kTileBytes = kTile * kD;     // 2 KB of K, 2 KB of V
constexpr int kStages = 3;
constexpr int kAloneMax = 768, kAloneFewer = 512, kAloneSegments = 152;  // see alone()
constexpr int kAlonePad = 4;               // floats between rows of scores: other banks
constexpr int kSlotBytes = 2 * kTileBytes;
constexpr int kWarps = 8;                  // of the join
constexpr int kThreads = kWarps * 32;
constexpr float kOffset = 13.f;            // weights that meet the codes: 2^13 at most
constexpr float kLift = 8192.f;            // 2^kOffset
constexpr float kHuge = 4096.f;            // references beyond it: careful_tile()
constexpr float kApart = 10.f;             // log2 of value scales' ratio: careful_tile()
constexpr float kNone = -3.402823466e38f;  // maximum of no position (finite: -inf - it is -inf)

// How the rows of a cache head are cut: groups of 8 * NR rows, NR column tiles of the products
struct RowPlan {
  int R, NR, RG, RS;  // rows per cache head, column tiles and groups, rows stored per piece
};
RowPlan row_plan(int H, int Hkv, int Nq, int dtype) {
  RowPlan p;
  p.R = H / Hkv * Nq;
  // The column tiles of a group share each converted operand; fp32's second terms leave the
  // registers for two, bf16's for four, but then for eight warps instead of twelve.  Four against
  // two: 8 x 8 heads x 16384 positions with 128 rows each 143 and 163 us (with weights 294 and
  // 379), 64 rows 80 and 83, lengths up to that 52.4 and 52.5, up to 2048 19.5 and 16.1; 32 rows
  // up to 16384 35.9 and 34.3
  p.NR = p.R <= 8 ? 1 : p.R <= 64 || dtype != 1 ? 2 : 4;
  p.RG = (p.R + 8 * p.NR - 1) / (8 * p.NR);
  p.RS = std::min(p.R, 8 * p.NR);
  return p;
}
// Warps of the first launch's one block per SM, by the registers that its operands take.  Twelve
// where 168 registers a thread do.  Sixteen at 128 spill (16 rows, 8 x 8 x 65536 positions 89.5 ->
// 97.7 us) or keep more requests in flight than HBM takes well (64 x 16 heads x 4096 positions 86.7
// -> 90.2 us); eight leave the tensor cores waiting (92.5 and 125 us).
constexpr int main_warps(int terms, int nr) { return terms * nr <= 2 ? 12 : 8; }
// Threads that the registers are shared out for.  bf16 queries of one column tile take 128 each at
// most, as for 16 warps, which leaves room for a block of the join to wait on the SM (one sequence
// of 131072, 8 heads: 27.1 us; with the 137 they would take 28.6)
constexpr int register_threads(int terms, int nr, bool alone) {
  return terms * nr == 1 && !alone ? 512 : main_warps(terms, nr) * 32;
}
// workers at most, as far as the workspace goes (a GB300 has 152 SMs)
constexpr int max_workers(int terms, int nr) { return 160 * main_warps(terms, nr); }

struct Params {
  DecodeQ8Args a;
  RowPlan rp;
  int workers;        // warps of the first launch's grid
  int block_shift;    // log2 of the positions per scale
  float* part;        // [slots][RS][64] unnormalised O
  float* stat;        // [slots][RS][2] m, l
  float* scores;      // [B][Hkv][R][Lpad] x in base-2 units (-inf: excluded); null: not kept
  int64_t Lpad;
};

__device__ __forceinline__ int cached(const DecodeQ8Args& a, int b) {
  return min(max(__ldg(a.cache_len + b), 0), a.Lmax);
}
__device__ __forceinline__ int tiles_of(int L) { return (L + kTile - 1) / kTile; }

// The line of tiles, seen by a whole warp: `per` segments (cache heads times row groups) of each
// batch element in turn, cut into runs of `run` tiles, one per worker (the last may be shorter).
// 32-bit numbers: the entry point refuses lines of 2^31 tiles.
struct Line {
  uint32_t total, run;
  int here;  // lane i: inclusive sum of the tiles of batch elements 0..i (i < 32)
};
__device__ __forceinline__ int scan_add(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}
// tiles of batch elements x0 + lane, summed over the lanes up to this one
__device__ __forceinline__ int scan_batch(const DecodeQ8Args& a, int x0, int per) {
  const int b = x0 + static_cast<int>(threadIdx.x & 31);
  return scan_add(b < a.B ? tiles_of(cached(a, b)) * per : 0);
}
__device__ __forceinline__ Line line_of(const DecodeQ8Args& a, int per, int workers) {
  Line n;
  n.here = scan_batch(a, 0, per);
  n.total = __shfl_sync(0xffffffffu, n.here, 31);
  for (int x0 = 32; x0 < a.B; x0 += 32)
    n.total += __shfl_sync(0xffffffffu, scan_batch(a, x0, per), 31);
  n.run = (n.total + workers - 1) / workers;
  return n;
}
// batch element that holds tile x (x < total), and the tiles before it
__device__ __forceinline__ int find_batch(const Line& n, const DecodeQ8Args& a, int per, uint32_t x,
                                          uint32_t* before) {
  uint32_t base = 0;
  for (int x0 = 0;; x0 += 32) {
    const uint32_t incl = x0 == 0 ? n.here : scan_batch(a, x0, per);
    const uint32_t m = __ballot_sync(0xffffffffu, base + incl > x);
    if (m != 0 || x0 + 32 >= a.B) {  // the second: not reached for x < total
      const int src = max(__ffs(m) - 1, 0);
      const uint32_t up = __shfl_sync(0xffffffffu, incl, max(src - 1, 0));
      *before = base + (src == 0 ? 0 : up);
      return min(x0 + src, a.B - 1);
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
}
// tiles before batch element b
__device__ __forceinline__ uint32_t tiles_before(const Line& n, const DecodeQ8Args& a, int per,
                                                 int b) {
  uint32_t base = 0;
  int x0 = 0;
  for (; x0 + 32 <= b; x0 += 32)
    base += __shfl_sync(0xffffffffu, x0 == 0 ? n.here : scan_batch(a, x0, per), 31);
  const int incl = x0 == 0 ? n.here : scan_batch(a, x0, per);
  const int up = __shfl_sync(0xffffffffu, incl, max(b - x0 - 1, 0));
  return base + (b == x0 ? 0 : up);
}

// 16 bytes from global to shared memory, past L1; a lane's copies complete in groups.  `policy`:
// the cache streams through L2 and is the first to leave it, so that the scores and pieces that
// the join reads stay there (64 x 16 heads x 4096 positions 87.3 -> 84.8 us, with weights 106.8
// -> 102.5).
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::256B [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// a place on the line of tiles: tile kt of nt of row group rg of head hk of batch element b
struct Cursor {
  int b, hk, rg, kt, nt, L;
};
// the first tile of the next row group, head or batch element that has any
__device__ __forceinline__ void next_segment(const Params& p, Cursor& k) {
  k.kt = 0;
  if (++k.rg < p.rp.RG) return;
  k.rg = 0;
  if (++k.hk < p.a.Hkv) return;
  k.hk = 0;
  do {
    k.L = ++k.b < p.a.B ? cached(p.a, k.b) : kTile;  // past the last: never used
    k.nt = tiles_of(k.L);
  } while (k.nt == 0);
}
// log2 of a positive normal number, exact for powers of two
__device__ __forceinline__ float log2_approx(float x) {
  const uint32_t u = __float_as_uint(x);
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__uint_as_float((u & 0x7fffffu) | 0x3f800000u)));
  return y + (__uint_as_float((u >> 23) | 0x4b000000u) - 8388735.f);  // + the exponent
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ void put2(__nv_bfloat16* q, float a, float b) {
  *reinterpret_cast<uint32_t*>(q) = pack_bf16x2(a, b);
}
__device__ __forceinline__ void put2(float* q, float a, float b) {
  *reinterpret_cast<float2*>(q) = make_float2(a, b);
}

// Joins (m, l) with the maxima and sums st of 2 kHalf lanes (kNone, 0: none), the same for all of
// them.  Returns the factor of the lane's own; `old`: that of what was in (m, l)
template <int kHalf>
__device__ __forceinline__ float join_lanes(float& m, float& l, float2 st, float& old) {
  float top = st.x;
#pragma unroll
  for (int s = kHalf; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  top = fmaxf(top, m);
  const float f = st.x == top ? 1.f : ex2_approx(st.x - top);
  old = m == top ? 1.f : ex2_approx(m - top);
  float sum = st.y * f;
#pragma unroll
  for (int s = kHalf; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  l = l * old + sum;
  m = top;
  return f;
}

// T: float (two fp16 terms per operand) or bf16 (one).  NR: column tiles of 8 query rows.
// kAlone: a block per cache head (of one row group), whose tiles its warps share; pieces and scores
// meet in shared memory, and no second launch is needed.
template <typename T, int QT, int NR, bool kAlone>
__global__ void __launch_bounds__(register_threads(sizeof(T) / 2, NR, kAlone), 1)
    decode_q8_kernel(const Params p) {
  constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;
  const DecodeQ8Args& a = p.a;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * (kStages * kSlotBytes);
  pdl_wait();  // the previous kernel's output is complete from here on
  pdl_launch_dependents();  // after the wait: the join reads cache_len before its own

  // this warp's run of tiles.  Consecutive workers sit in different blocks, so that few tiles
  // spread over the SMs
  constexpr int kMainWarps = main_warps(sizeof(T) / 2, NR);
  // kAlone: [rows][2] of the statistics, then [rows][Lpad] of the scores, behind the rings
  float* const alone_stat = reinterpret_cast<float*>(smem + kMainWarps * (kStages * kSlotBytes));
  float* const alone_scores = alone_stat + 8 * NR * 2;
  const int per = a.Hkv * p.rp.RG;
  const uint32_t worker = warp * gridDim.x + blockIdx.x;
  int count, live = 0;  // tiles; kAlone: warps that have any
  Cursor c;
  if constexpr (kAlone) {
    c.b = static_cast<int>(blockIdx.x) / a.Hkv;
    c.hk = static_cast<int>(blockIdx.x) % a.Hkv;
    c.rg = 0;
    c.L = cached(a, c.b);
    c.nt = tiles_of(c.L);
    const int each = max((c.nt + kMainWarps - 1) / kMainWarps, 1);
    live = (c.nt + each - 1) / each;
    c.kt = warp * each;
    count = max(min(each, c.nt - c.kt), 0);
  } else {
    const Line line = line_of(a, per, p.workers);
    const uint32_t x0 = worker * line.run;
    if (x0 >= line.total) return;
    count = static_cast<int>(min(line.run, line.total - x0));
    uint32_t before;
    c.b = find_batch(line, a, per, x0, &before);
    c.L = cached(a, c.b);
    c.nt = tiles_of(c.L);
    const int hr = static_cast<int>((x0 - before) / c.nt);
    c.kt = static_cast<int>((x0 - before) % c.nt);
    c.hk = hr / p.rp.RG;
    c.rg = hr % p.rp.RG;
  }
  // The next tile to ask for.  A lane copies chunk t of rows g, g + 8, g + 16 and g + 24 of K and
  // of V; chunk i of row r is stored at i ^ ((r >> 1) & 3), so that eight rows' chunks read
  // together, or a row's pairs, meet different banks.
  Cursor ahead = c;
  const uint8_t *k_next = nullptr, *v_next = nullptr;
  auto place = [&]() {
    const int64_t row = static_cast<int64_t>(ahead.kt) * kTile + g;
    k_next = static_cast<const uint8_t*>(a.Kc) + ahead.b * a.sk[0] + ahead.hk * a.sk[1] +
             row * a.sk[2] + t * 16;
    v_next = static_cast<const uint8_t*>(a.Vc) + ahead.b * a.sv[0] + ahead.hk * a.sv[1] +
             row * a.sv[2] + t * 16;
  };
  place();
  int asked = 0;
  const uint64_t policy = evict_first_policy();
  const int64_t k_step = 8 * a.sk[2], v_step = 8 * a.sv[2];
  const int k_at = (t ^ ((g >> 1) & 3)) << 4;  // chunk t of a row 8i + g
  const uint32_t dst0 = smem_u32(ring) + g * kD + k_at;
  auto ask = [&](int slot) {
    if (asked < count) {
      const uint32_t dst = dst0 + slot * kSlotBytes;
      if ((ahead.kt + 1) * kTile <= a.Lmax) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          copy16_async(dst + i * 8 * kD, k_next + i * k_step, policy);
          copy16_async(dst + kTileBytes + i * 8 * kD, v_next + i * v_step, policy);
        }
      } else {  // rows behind the cache: the slot keeps what it held, unused
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (ahead.kt * kTile + i * 8 + g < a.Lmax) {
            copy16_async(dst + i * 8 * kD, k_next + i * k_step, policy);
            copy16_async(dst + kTileBytes + i * 8 * kD, v_next + i * v_step, policy);
          }
      }
      ++asked;
      k_next += 4 * k_step;
      v_next += 4 * v_step;
      if (++ahead.kt == ahead.nt && asked < count) {
        next_segment(p, ahead);
        place();
      }
    }
    copy_async_commit();  // a group per tile, also an empty one
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) ask(s);

  const int v_at = (((g >> 1) ^ t) << 4) + (g & 1) * 8;  // columns 8g.. of a row 8i + 2t + {0, 1}

  // In the products' results a lane holds positions g and g + 8 of each 16 for the two rows
  // 8 nr + 2t + {0, 1}: the row statistics below are those rows'.
  uint32_t qf[kTerms][NR][4][2];  // queries, row 8 nr + g: operand fragments of four inner steps
  float2 qs[NR];                  // what a score is to be multiplied by for its row
  int lim[NR][2];                 // last position that the row may see
  float o[NR][4][4], m[NR][2];
  float2 l[NR];  // of the lane's own positions
  const float c2 = a.scale * 1.4426950408889634f;

  auto start_segment = [&]() {
    const int hk = c.hk, r0 = c.rg * (8 * NR);
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
      // (2^-113 keeps both powers normal numbers.  Rows below that are multiples of 2^-149, which
      // 2^126 makes exact in fp16's two terms)
      const int ex = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -113);
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
        (e ? qs[nr].y : qs[nr].x) = __shfl_sync(0xffffffffu, down, (2 * t + e) * 4);
        lim[nr][e] = a.causal ? c.L - a.Nq + (r0 + nr * 8 + 2 * t + e) % a.Nq : c.L - 1;
        m[nr][e] = kNone;
      }
      l[nr] = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nr][j][i] = 0.f;
    }
  };

  auto end_segment = [&]() {
    const int64_t slot =
        kAlone ? 0 : worker + static_cast<int64_t>(c.b) * per + c.hk * p.rp.RG + c.rg;
    // (kAlone: the warp's ring, whose copies have all landed and been read)
    float* part = kAlone ? reinterpret_cast<float*>(ring) : p.part;
    float* stat = kAlone ? part + 8 * NR * kD : p.stat;
    const int r0 = c.rg * (8 * NR);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rl = nr * 8 + 2 * t + e;
        float s = e ? l[nr].y : l[nr].x;
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        if (r0 + rl < p.rp.R) {
          // columns 8g + 2j and 8g + 2j + 1
          float4* dst = reinterpret_cast<float4*>(part + (slot * p.rp.RS + rl) * kD + g * 8);
          dst[0] = make_float4(o[nr][0][e], o[nr][0][2 + e], o[nr][1][e], o[nr][1][2 + e]);
          dst[1] = make_float4(o[nr][2][e], o[nr][2][2 + e], o[nr][3][e], o[nr][3][2 + e]);
          if (g == 0)
            *reinterpret_cast<float2*>(stat + (slot * p.rp.RS + rl) * 2) = make_float2(m[nr][e], s);
        }
      }
  };

  int slot = 0, done = 0;
  while (done < count) {
    // tiles kt .. of one row group and head
    start_segment();
    const int64_t head = static_cast<int64_t>(c.b) * a.Hkv + c.hk;
    // scales of a tile: lanes 0, 1 those of its two 16-position groups' keys, 2, 3 values'.  A
    // group behind the last position counts as 1 (its scores are excluded below).
    const float* scale_row = (lane < 2 ? a.k_scale : a.v_scale) + head * a.n_blocks;
    auto load_scale = [&](int kt) -> float {
      const int at = kt * kTile + (lane & 1) * 16;
      return lane < 4 && at < c.L ? __ldg(scale_row + (at >> p.block_shift)) : 1.f;
    };
    float* score_row = nullptr;  // of row 2t of the group
    const int rows_here = p.rp.R - c.rg * (8 * NR) - 2 * t;  // live rows from there on
    if (kAlone && a.weights != nullptr)
      score_row = alone_scores + 2 * t * p.Lpad + g;
    if (!kAlone && p.scores != nullptr)
      score_row = p.scores + (head * p.rp.R + c.rg * (8 * NR) + 2 * t) * p.Lpad + g;
    // Beyond kHuge a reference is too coarse for exponents in which the offset and the value's
    // scale are rounded together with it (from 2^24 on they would be lost)
    bool huge = false;
    // A tile with a value scale 2^kApart or more below the largest so far has weights that fp16
    // would round away under the row's reference (what is below 2^-38 of its largest), and they may
    // be all that a column has: it is taken under references of its own as well (64 x 16 heads x
    // 4096 with every other block 2^15 smaller 99 us instead of 84, scores of 1e5 102)
    float most_log = -INFINITY, value_log[2] = {0.f, 0.f};
    bool apart = false;
    float sc_next = load_scale(c.kt), sc = 1.f, sc_log = 0.f, sc_inv = 1.f;
    const int last = min(c.nt, c.kt + count - done);
    done += last - c.kt;
    const uint8_t *sK = nullptr, *sV = nullptr;
    int pos = 0;
    // tile c.kt once it has landed, and the next one to ask for into its slot
    auto begin_tile = [&]() {
      sc = sc_next;
      if (c.kt + 1 < last) sc_next = load_scale(c.kt + 1);  // a tile ahead of its use
      sc_log = log2_approx(sc);
      sc_inv = rcp_approx(sc);
      value_log[0] = __shfl_sync(0xffffffffu, sc_log, 2);
      value_log[1] = __shfl_sync(0xffffffffu, sc_log, 3);
      most_log = fmaxf(most_log, fmaxf(value_log[0], value_log[1]));
      apart = fminf(value_log[0], value_log[1]) < most_log - kApart;
      copy_async_wait<kStages - 1>();  // this lane's copies of the tile have landed
      __syncwarp();                    // and every lane's
      sK = ring + slot * kSlotBytes;
      sV = sK + kTileBytes;
      pos = c.kt * kTile;
    };
    auto end_tile = [&]() {
      __syncwarp();  // every lane has read the slot
      ask(slot);
      if (++slot == kStages) slot = 0;
    };
    // ---- what both forms of a tile do with a group q of 16 positions
    // products of its keys and the queries: positions g, g + 8 (rows 2t, 2t + 1 of row group nr)
    auto scores = [&](int q, float (&x)[NR][4]) {
      uint32_t h[2][8];  // positions g and g + 8: 16-byte chunk t of a row
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int row = q * 16 + z * 8 + g;
        const uint4 u = *reinterpret_cast<const uint4*>(sK + row * kD + k_at);
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
          if constexpr (kTerms == 2)
            mma16816_zero(d, fa, qf[kTerms - 1][nr][k][0], qf[kTerms - 1][nr][k][1]);
          if (kTerms == 1 && k == 0)
            mma16816_zero(d, fa, qf[0][nr][k][0], qf[0][nr][k][1]);
          else
            mma16816(d, fa, qf[0][nr][k][0], qf[0][nr][k][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[nr][i] = part[0][i];
          if constexpr (kTerms == 2)
            x[nr][i] = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
        }
      }
    };
    // its value rows 2t, 2t+1, 2t+8, 2t+9, columns 8g .. 8g+7
    auto value_codes = [&](int q, uint2 (&v)[4]) {
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int row = q * 16 + 2 * t + (z >> 1) * 8 + (z & 1);
        v[z] = *reinterpret_cast<const uint2*>(sV + row * kD + v_at);
      }
    };
    // the same as product operands: column 8g + j, rows 2t, 2t+1 in b0[j], 2t+8, 2t+9 in b1[j]
    auto value_halves = [&](const uint2 (&v)[4], uint32_t (&b0)[8], uint32_t (&b1)[8]) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t a0 = z ? v[0].y : v[0].x, a1 = z ? v[1].y : v[1].x;
        const uint32_t a2 = z ? v[2].y : v[2].x, a3 = z ? v[3].y : v[3].x;
        codes_to_half<QT>(__byte_perm(a0, a1, 0x5140), b0[4 * z], b0[4 * z + 1]);
        codes_to_half<QT>(__byte_perm(a0, a1, 0x7362), b0[4 * z + 2], b0[4 * z + 3]);
        codes_to_half<QT>(__byte_perm(a2, a3, 0x5140), b1[4 * z], b1[4 * z + 1]);
        codes_to_half<QT>(__byte_perm(a2, a3, 0x7362), b1[4 * z + 2], b1[4 * z + 3]);
      }
    };
    // the largest value of a row's 16 positions
    auto row_max = [](float v) -> float {
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
      return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
    };
    // the rows' references rise to `top`, and O and l with them
    auto rise = [&](const float (&top)[NR][2]) {
      bool far = false;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float v = fmaxf(m[nr][e], top[nr][e]);
          // a first maximum finds O = l = 0
          const float u = v == m[nr][e] ? 1.f : ex2_approx(m[nr][e] - v);
          m[nr][e] = v;
          far |= fabsf(v) > kHuge && v != kNone;
          (e ? l[nr].y : l[nr].x) *= u;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[nr][j][e] *= u;
            o[nr][j][2 + e] *= u;
          }
        }
      huge = __any_sync(0xffffffffu, far);
    };
    // A tile that every row sees, under references that are not huge.  False: one became so.  The
    // tile is to be taken again then, by the other form: nothing but the references, O and l under
    // them has changed
    auto tile = [&]() -> bool {
      float x[2][NR][4];
#pragma unroll
      for (int q = 0; q < 2; ++q) scores(q, x[q]);
      // ---- the scales: a score is x * f, its exponent x * f + log2 of the value's scale
      float2 f[2][NR];
      float inv[2];
      const float (&ev)[2] = value_log;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float ks = __shfl_sync(0xffffffffu, sc, q);
        inv[q] = __shfl_sync(0xffffffffu, sc_inv, 2 + q);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
          f[q][nr] = fmul2(make_float2(ks, ks), qs[nr]);
      }
      if (score_row != nullptr) {  // kept for the weights
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (nr * 8 + e < rows_here) {
              float* dst = score_row + (nr * 8 + e) * p.Lpad + pos;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const float fe = e ? f[q][nr].y : f[q][nr].x;
                dst[q * 16] = x[q][nr][e] * fe;
                dst[q * 16 + 8] = x[q][nr][2 + e] * fe;
              }
            }
      }
      // ---- running maximum
      float top[NR][2];
      bool grew = false;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[nr][e] = fmaxf(
              fmaf(fmaxf(x[0][nr][e], x[0][nr][2 + e]), e ? f[0][nr].y : f[0][nr].x, ev[0]),
              fmaf(fmaxf(x[1][nr][e], x[1][nr][2 + e]), e ? f[1][nr].y : f[1][nr].x, ev[1]));
          grew |= top[nr][e] > m[nr][e];
        }
      if (__any_sync(0xffffffffu, grew)) {  // seldom, once a row has seen many positions
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) top[nr][e] = row_max(top[nr][e]);
        rise(top);
        if (huge) return false;
      }
      // ---- weights, 16 positions at a time, and their product with the value codes
      [[maybe_unused]] float po[kTerms == 2 ? NR : 1][4][4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t pf[kTerms][NR][2];
        // the fp32 path keeps the offset out of the exponent, whose rounding it would coarsen
        const float up = ev[q] + (kTerms == 2 ? 0.f : kOffset);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          const float2 shift = make_float2(up - m[nr][0], up - m[nr][1]);
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            float2 w = make_float2(x[q][nr][2 * z], x[q][nr][2 * z + 1]);
            w = ffma2(w, f[q][nr], shift);
            w.x = ex2_approx(w.x);
            w.y = ex2_approx(w.y);
            if constexpr (kTerms == 2) w = fmul2(w, make_float2(kLift, kLift));
            l[nr] = ffma2(w, make_float2(inv[q], inv[q]), l[nr]);
            const uint32_t hi = pack_half(w.x, w.y);
            pf[0][nr][z] = transpose8x8(hi);
            if constexpr (kTerms == 2)
              pf[kTerms - 1][nr][z] = transpose8x8(pack_rest(w.x, w.y, hi));
          }
        }
        uint2 v[4];
        uint32_t b0[8], b1[8];
        value_codes(q, v);
        value_halves(v, b0, b1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t fa[4] = {b0[2 * j], b0[2 * j + 1], b1[2 * j], b1[2 * j + 1]};
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            if constexpr (kTerms == 2) {
              if (q == 0)
                mma16816_zero(po[nr][j], fa, pf[kTerms - 1][nr][0], pf[kTerms - 1][nr][1]);
              else
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
      return true;
    };
    // Any tile, its two groups one after the other, for half the code and registers.  (In one body
    // with the above, masks cost the other tiles 78 of 562 instructions and 14% of the time: 16
    // rows, 8 x 8 x 16384 positions.  Both groups at once: 128 rows to a head 153 us, not 143; 8
    // heads x 37 4.1 either way.)  Weights are 2^(x - ref) under the largest score of the row's 16
    // positions: the difference of two scores is exact where it counts, whatever their size.
    // 2^(ref - m) brings their sum under the row's reference and, with the values' scale, their
    // product.
    auto careful_tile = [&]() {
#pragma unroll 1
      for (int q = 0; q < 2; ++q) {
        float x[NR][4], ref[NR][2], top[NR][2];
        bool grew = false;
        scores(q, x);
        const float ks = __shfl_sync(0xffffffffu, sc, q);
        const float vs = __shfl_sync(0xffffffffu, sc, 2 + q);
        const float ev = __shfl_sync(0xffffffffu, sc_log, 2 + q);
        const int at = pos + q * 16;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = ks * (e ? qs[nr].y : qs[nr].x);
            float &x0 = x[nr][e], &x1 = x[nr][2 + e];
            x0 = at + g > lim[nr][e] ? -INFINITY : __fmul_rn(x0, f);
            x1 = at + g + 8 > lim[nr][e] ? -INFINITY : __fmul_rn(x1, f);
            if (score_row != nullptr && nr * 8 + e < rows_here) {
              float* dst = score_row + (nr * 8 + e) * p.Lpad + at;
              dst[0] = x0;
              dst[8] = x1;
            }
            ref[nr][e] = row_max(fmaxf(x0, x1));
            top[nr][e] = ref[nr][e] + ev;
            grew |= top[nr][e] > m[nr][e];
          }
        if (__any_sync(0xffffffffu, grew)) rise(top);
        uint2 v[4];
        uint32_t b0[8], b1[8];
        [[maybe_unused]] uint32_t nan = 0;
        value_codes(q, v);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          // rows behind the last position hold anything: 0.  A NaN among the rows that some query
          // may not see must reach only those that do: taken out of the product here, put into O
          // below
          if (at + 2 * t + (z >> 1) * 8 + (z & 1) >= c.L) v[z] = make_uint2(0u, 0u);
          if constexpr (QT == kE4m3) {
            const uint32_t nx = __vcmpeq4(v[z].x & 0x7f7f7f7fu, 0x7f7f7f7fu);
            const uint32_t ny = __vcmpeq4(v[z].y & 0x7f7f7f7fu, 0x7f7f7f7fu);
            v[z].x &= ~nx;
            v[z].y &= ~ny;
            nan |= nx | ny;
          }
        }
        value_halves(v, b0, b1);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          uint32_t pf[kTerms][2];
          float into_l[2], into_o[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            into_l[e] = ex2_approx(ref[nr][e] - m[nr][e]);
            into_o[e] = into_l[e] * vs;
            if (ref[nr][e] == -INFINITY) ref[nr][e] = 0.f;  // none allowed: weights of 0
          }
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float w0 = ex2_approx(x[nr][2 * z] - ref[nr][0]) * kLift;
            const float w1 = ex2_approx(x[nr][2 * z + 1] - ref[nr][1]) * kLift;
            l[nr].x = fmaf(w0, into_l[0], l[nr].x);
            l[nr].y = fmaf(w1, into_l[1], l[nr].y);
            const uint32_t hi = pack_half(w0, w1);
            pf[0][z] = transpose8x8(hi);
            if constexpr (kTerms == 2) pf[kTerms - 1][z] = transpose8x8(pack_rest(w0, w1, hi));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t fa[4] = {b0[2 * j], b0[2 * j + 1], b1[2 * j], b1[2 * j + 1]};
            float d[4];
            mma16816_zero(d, fa, pf[kTerms - 1][0], pf[kTerms - 1][1]);
            if constexpr (kTerms == 2) mma16816(d, fa, pf[0][0], pf[0][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nr][j][i] = fmaf(d[i], into_o[i & 1], o[nr][j][i]);
          }
        }
        if (QT == kE4m3 && __any_sync(0xffffffffu, nan != 0)) {
          // columns 8g .. 8g+7 of each position: NaN into the rows that see it (looked for in every
          // last tile, row by row: 16 rows of 8 x 8 heads x up to 16384 28.4 us instead of 26.8)
          const int end = min(q * 16 + 16, c.L - pos);
          for (int row = q * 16; row < end; ++row) {
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
      }
    };
    // tiles that every row sees, then, from the first one that is not for `tile` on, the others; a
    // tile that `tile` did not finish is begun already
    const int seen = min(last, max((c.L - (a.causal ? a.Nq : 1) + 1) / kTile, 0));
    bool begun = false;
    for (; c.kt < seen; ++c.kt) {
      begin_tile();
      if (apart || !tile()) {
        begun = true;
        break;
      }
      end_tile();
    }
    for (; c.kt < last; ++c.kt) {
      if (!begun) begin_tile();
      begun = false;
      careful_tile();
      end_tile();
    }
    end_segment();
    if (!kAlone && c.kt == c.nt) next_segment(p, c);
  }
  if constexpr (kAlone) {
    __syncthreads();
    for (int r = warp; r < p.rp.R; r += kMainWarps) {
      auto piece = [&](int w) {
        return reinterpret_cast<const float*>(smem + w * (kStages * kSlotBytes));
      };
      float2 st = make_float2(kNone, 0.f), o2 = make_float2(0.f, 0.f);
      if (lane < live) st = *reinterpret_cast<const float2*>(piece(lane) + 8 * NR * kD + 2 * r);
      float top = kNone, sum = 0.f, old;
      const float f = join_lanes<16>(top, sum, st, old);
      for (int w = 0; w < live; ++w) {
        const float fw = __shfl_sync(0xffffffffu, f, w);
        const float2 v = *reinterpret_cast<const float2*>(piece(w) + r * kD + 2 * lane);
        o2.x = fmaf(v.x, fw, o2.x);
        o2.y = fmaf(v.y, fw, o2.y);
      }
      const float y = sum == 0.f ? 0.f : 1.f / sum;  // no allowed position: zeros
      const int h = c.hk * (a.H / a.Hkv) + r / a.Nq;
      put2(static_cast<T*>(a.O) + c.b * a.so[0] + h * a.so[1] + (r % a.Nq) * a.so[2] + 2 * lane,
           o2.x * y, o2.y * y);
      // weight = 2^(x - top) 2^kOffset / sum: the difference of two scores first, as above
      if (lane == 0) *reinterpret_cast<float2*>(alone_stat + 2 * r) = make_float2(top, y * kLift);
    }
    if (a.weights == nullptr) return;
    __syncthreads();
    float* out = a.weights + (static_cast<int64_t>(c.b) * a.Hkv + c.hk) * a.Lmax;
    for (int j = threadIdx.x; j < c.L; j += kMainWarps * 32) {
      float w = 0.f;
      for (int r = 0; r < p.rp.R; ++r) {
        const float2 st = *reinterpret_cast<const float2*>(alone_stat + 2 * r);
        const float x = alone_scores[r * p.Lpad + j];
        if (x != -INFINITY) w = fmaf(ex2_approx(x - st.x), st.y, w);
      }
      out[j] += w;
    }
  }
}

// ---- joining the pieces
// the workers that hold pieces of segment hr of batch element b (which has tiles)
struct Pieces {
  uint32_t start, run;  // tiles before b's first segment, tiles of a run
  int nt;               // tiles of one of b's segments
  __device__ __forceinline__ Pieces(const Params& p, int b) {
    const int per = p.a.Hkv * p.rp.RG;
    const Line line = line_of(p.a, per, p.workers);
    start = tiles_before(line, p.a, per, b);
    run = line.run;
    nt = tiles_of(cached(p.a, b));
  }
  __device__ __forceinline__ int first(int hr) const { return (start + hr * nt) / run; }
  __device__ __forceinline__ int last(int hr) const { return (start + hr * nt + nt - 1) / run; }
};

// Merges (m2, l2) into (m, l): sums l under the larger maximum (kNone: nothing there; a NaN sum
// must not be lost).  Returns the two factors.
__device__ __forceinline__ float2 merge(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2);
  const float2 f = make_float2(m == top ? 1.f : ex2_approx(m - top),
                               m2 == top ? 1.f : ex2_approx(m2 - top));
  m = top;
  l = l * f.x + l2 * f.y;
  return f;
}

// Blocks 0 .. row_blocks-1: O.  kWide: the warps of a block split the pieces of one row;
// otherwise each takes a row of its own.  The blocks behind (kQuads > 0): weights, 1024 kQuads
// positions each.  What depends on the lengths alone is done before the pieces are waited for.
// At most 64 registers, for all of a step's blocks to be resident at once: with the 95 that four
// quads want, grouped heads' 1024 rows took four rounds.
template <typename T, bool kWide, int kQuads>
__global__ void __launch_bounds__(kThreads, 4) decode_q8_join_kernel(const Params p, int row_blocks,
                                                                     int weight_blocks) {
  const DecodeQ8Args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = a.Hkv * p.rp.RG, G = a.H / a.Hkv;
  const int group = 8 * p.rp.NR;
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) < row_blocks) {
    __shared__ float so[kWarps][kD], sm[kWarps], sl[kWarps];
    const int row = kWide ? blockIdx.x : blockIdx.x * kWarps + warp;
    const int rows = a.B * a.Hkv * p.rp.R;
    if (row >= rows) return;  // a whole warp (kWide: no warp)
    const int r = row % p.rp.R;
    const int hk = row / p.rp.R % a.Hkv;
    const int b = row / p.rp.R / a.Hkv;
    const int hr = hk * p.rp.RG + r / group;
    const Pieces pieces(p, b);
    const int first = pieces.nt > 0 ? pieces.first(hr) : 0;
    const int last = pieces.nt > 0 ? pieces.last(hr) : -1;
    const int64_t at0 = (static_cast<int64_t>(b) * per + hr) * p.rp.RS + r % group;
    pdl_wait();  // the pieces are complete from here on
    // 32 pieces at a time: a lane has the maximum and sum of one, so that the largest maximum, each
    // piece's factor and the sum take one exponential; then the pieces' O under their factors
    float m = kNone, l = 0.f;
    float2 o = make_float2(0.f, 0.f);
    constexpr int kStep = kWide ? kWarps : 1, kBatch = 8;  // pieces asked for at once
    for (int w = first + (kWide ? warp : 0); w <= last; w += 32 * kStep) {
      const int n = min(32, (last - w) / kStep + 1);
      const int64_t at = static_cast<int64_t>(w) * p.rp.RS + at0;
      float2 st = make_float2(kNone, 0.f), v[kBatch];
      if (lane < n)
        st = *reinterpret_cast<const float2*>(
            p.stat + (at + static_cast<int64_t>(lane) * kStep * p.rp.RS) * 2);
      auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          v[k] = make_float2(0.f, 0.f);
          if (k0 + k < n)
            v[k] = *reinterpret_cast<const float2*>(
                p.part + (at + static_cast<int64_t>(k0 + k) * kStep * p.rp.RS) * kD + 2 * lane);
        }
      };
      load(0);
      float old;
      const float f = join_lanes<16>(m, l, st, old);
      o.x *= old;
      o.y *= old;
      for (int k0 = 0; k0 < n; k0 += kBatch) {
        if (k0 > 0) load(k0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const float fk = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
          o.x = fmaf(v[k].x, fk, o.x);
          o.y = fmaf(v[k].y, fk, o.y);
        }
      }
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
      m = kNone;
      l = 0.f;
      o = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 f = merge(m, l, sm[w], sl[w]);
        o.x = o.x * f.x + so[w][2 * lane] * f.y;
        o.y = o.y * f.x + so[w][2 * lane + 1] * f.y;
      }
    }
    const float y = l == 0.f ? 0.f : 1.f / l;  // no allowed position: zeros
    const int h = hk * G + r / a.Nq;
    put2(static_cast<T*>(a.O) + b * a.so[0] + h * a.so[1] + (r % a.Nq) * a.so[2] + 2 * lane,
         o.x * y, o.y * y);
    return;
  }
  if constexpr (kQuads > 0) {
    // ---- weights: m and 1 / l of every row of the cache head, then its positions
    const int x = static_cast<int>(blockIdx.x) - row_blocks;
    const int bh = x / weight_blocks;
    const int hk = bh % a.Hkv, b = bh / a.Hkv;
    const int L = cached(a, b);
    const int j0 = x % weight_blocks * (4 * kThreads * kQuads);
    if (j0 >= L) return;
    extern __shared__ float rowstat[];  // [R][2]
    const Pieces pieces(p, b);          // L > 0: there are some
    const int R = p.rp.R;
    const float* sc = p.scores + static_cast<int64_t>(bh) * R * p.Lpad;
    float* out = a.weights + static_cast<int64_t>(bh) * a.Lmax;
    // position of the thread's quad k; what its weights were is asked for before the pieces are
    // waited for
    auto quad = [&](int k) { return j0 + (k * kThreads + static_cast<int>(threadIdx.x)) * 4; };
    const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    float was[kQuads][4];
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const int j = quad(k);
      if (vec && j + 4 <= L) {
        const float4 v = *reinterpret_cast<const float4*>(out + j);
        was[k][0] = v.x, was[k][1] = v.y, was[k][2] = v.z, was[k][3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < L) was[k][i] = out[j + i];
      }
    }
    pdl_wait();  // pieces and scores are complete from here on
    // scores of up to four rows and quads at a time, the next ones on their way meanwhile; the
    // first are asked for before the statistics are known
    constexpr int kRows = 4 / kQuads, kBufs = kQuads == 4 ? 1 : 2;
    float4 xs[kBufs][kRows][kQuads];
    auto load = [&](int r, float4 (&x)[kRows][kQuads]) {
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        const int j = quad(k);
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          if (j < L && r + u < R)
            x[u][k] = *reinterpret_cast<const float4*>(sc + (r + u) * p.Lpad + j);
      }
    };
    load(0, xs[0]);
    for (int r0 = 2 * warp; r0 < R; r0 += 2 * kWarps) {  // a row to each half of the warp
      const int r = min(r0 + (lane >> 4), R - 1);
      const int hr = hk * p.rp.RG + r / group;
      const int last = pieces.last(hr);
      const int64_t at0 = (static_cast<int64_t>(b) * per + hr) * p.rp.RS + r % group;
      float m = kNone, l = 0.f;
      for (int w = pieces.first(hr) + (lane & 15); w <= last; w += 16) {
        const float2 st = *reinterpret_cast<const float2*>(
            p.stat + (static_cast<int64_t>(w) * p.rp.RS + at0) * 2);
        merge(m, l, st.x, st.y);
      }
      const float2 mine = make_float2(m, l);
      float old;
      m = kNone;
      l = 0.f;
      join_lanes<8>(m, l, mine, old);
      if ((lane & 15) == 0) {  // weight = 2^(x - m) 2^kOffset / l, x - m first as in the pieces
        rowstat[2 * r] = m;
        rowstat[2 * r + 1] = l == 0.f ? 0.f : kLift / l;
      }
    }
    __syncthreads();
    float w[kQuads][4];
#pragma unroll
    for (int k = 0; k < kQuads; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[k][i] = 0.f;
    auto add = [&](int r, float4 (&x)[kRows][kQuads]) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (r + u >= R) break;
        const float2 st = *reinterpret_cast<const float2*>(rowstat + 2 * (r + u));
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
          const float v[4] = {x[u][k].x, x[u][k].y, x[u][k].z, x[u][k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)  // an excluded position takes nothing of a NaN row
            if (v[i] != -INFINITY) w[k][i] = fmaf(ex2_approx(v[i] - st.x), st.y, w[k][i]);
        }
      }
    };
    for (int r = 0; r < R; r += kBufs * kRows) {
      if constexpr (kBufs == 1) {
        if (r > 0) load(r, xs[0]);
        add(r, xs[0]);
      } else {
        load(r + kRows, xs[1]);
        add(r, xs[0]);
        load(r + 2 * kRows, xs[0]);
        add(r + kRows, xs[1]);
      }
    }
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const int j = quad(k);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[k][i] += was[k][i];
      if (vec && j + 4 <= L) {
        *reinterpret_cast<float4*>(out + j) = make_float4(w[k][0], w[k][1], w[k][2], w[k][3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < L) out[j + i] = w[k][i];
      }
    }
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

template <typename T, int QT, int NR, bool kAlone = false>
cudaError_t launch_main(const Params& p, int blocks, cudaStream_t s) {
  auto kern = decode_q8_kernel<T, QT, NR, kAlone>;
  constexpr int kMainWarps = main_warps(sizeof(T) / 2, NR);
  static_assert(!kAlone || 8 * NR * (kD + 2) * 4 <= kStages * kSlotBytes, "a piece in a ring");
  constexpr int kRing = kMainWarps * kStages * kSlotBytes, kRows = 8 * NR;
  constexpr int kSmem = kRing + (kAlone ? kRows * (2 + kAloneMax + kAlonePad) * 4 : 0);
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kern), kSmem, nullptr);
  if (e != cudaSuccess) return e;
  const size_t smem =
      kAlone && p.a.weights != nullptr ? kRing + (kRows * 2 + p.rp.R * p.Lpad) * 4
                                       : kRing + (kAlone ? kRows * 2 * 4 : 0);
  return launch_pdl(kern, dim3(blocks), dim3(kMainWarps * 32), smem, s, p);
}
// Whether one launch does it all: short caches of few heads (a block each, one per SM), whose rows
// are one group.  One and two launches in us, bf16 and fp32 without weights, the same with:
//   8 heads of 128, 1 row     3.7 4.9, 3.8 4.8;  4.2 5.1, 4.2 5.2
//   8 heads of 768, 1 row     5.1 5.4, 5.6 5.7;  5.9 5.9, 6.5 6.2
//   8 heads of 768, 8 rows    5.4 5.6, 6.2 6.4;  6.4 6.5, 7.0 6.8
//   144 heads of 768, 8 rows  5.9 7.9, 6.6 10.3; 7.2 9.2, 7.8 10.3
//   8 heads of 512, 16 rows   7.0 7.4, 7.8 8.0;  8.2 8.7, 9.1 9.1
//   8 heads of 768, 16 rows   8.0 7.4, 9.0 8.2;  9.3 9.0, 10.8 9.3
//   32 heads of 768, 16 rows  8.4 9.0, 9.4 10.3; 9.7 9.7, 11.1 11.0
// One row of 16 heads of 1000 6.5 and 5.8; 304 heads, a second round of blocks, of 384 8.9 and 7.9.
bool alone(int B, int H, int Hkv, int Nq, int Lmax) {
  const int rows = H / Hkv * Nq;
  const int64_t heads = static_cast<int64_t>(B) * Hkv;
  return rows <= 16 && heads <= kAloneSegments &&
         Lmax <= (rows > 8 && heads < 32 ? kAloneFewer : kAloneMax);
}
template <typename T>
cudaError_t launch_alone(Params p, int qtype, cudaStream_t s) {
  p.Lpad += kAlonePad;
  const int blocks = p.a.B * p.a.Hkv;
  if (p.rp.NR == 1)
    return qtype == kE4m3 ? launch_main<T, kE4m3, 1, true>(p, blocks, s)
                          : launch_main<T, kInt8, 1, true>(p, blocks, s);
  return qtype == kE4m3 ? launch_main<T, kE4m3, 2, true>(p, blocks, s)
                        : launch_main<T, kInt8, 2, true>(p, blocks, s);
}
template <typename T>
cudaError_t launch_all(const Params& p, int qtype, int blocks, cudaStream_t s) {
  constexpr int kMost = sizeof(T) == 4 ? 2 : 4;  // row_plan's
  cudaError_t e;
  if (p.rp.NR == 1)
    e = qtype == kE4m3 ? launch_main<T, kE4m3, 1>(p, blocks, s)
                       : launch_main<T, kInt8, 1>(p, blocks, s);
  else if (p.rp.NR == 2)
    e = qtype == kE4m3 ? launch_main<T, kE4m3, 2>(p, blocks, s)
                       : launch_main<T, kInt8, 2>(p, blocks, s);
  else
    e = qtype == kE4m3 ? launch_main<T, kE4m3, kMost>(p, blocks, s)
                       : launch_main<T, kInt8, kMost>(p, blocks, s);
  if (e != cudaSuccess) return e;
  // A block per row where a row has many pieces (if all sequences are alike: workers / segments,
  // and no more than tiles) and rows are few, else a warp.  Pieces and rows, block and warp: 228
  // and 8 29.4 and 39.3 us, 57 and 512 27.2 and 29.1, 28 and 256 21.6 and 22.3, 28 and 512 25.8
  // and 23.6, 28 and 1024 36.9 and 32.8, 16 and 16 5.5 and 5.9, 14 and 128 30.6 and 28.7
  const int64_t heads = static_cast<int64_t>(p.a.B) * p.a.Hkv, rows = heads * p.rp.R;
  const int64_t pieces =
      std::min<int64_t>(p.workers / (heads * p.rp.RG), (p.a.Lmax + kTile - 1) / kTile);
  const bool wide = pieces >= 16 && rows <= 16 * pieces;
  const int row_blocks = static_cast<int>(wide ? rows : (rows + kWarps - 1) / kWarps);
  // more positions to a thread where that still fills the GPU: the blocks' fixed cost (statistics
  // of the rows) is paid less often (one row, 64 x 16 heads x 4096 positions: four quads 102 us,
  // one 113 us; three rows: two 116, one 123)
  auto fills = [&](int n) { return heads * ((p.a.Lmax + 1024 * n - 1) / (1024 * n)) >= 2 * 152; };
  const int quads = p.rp.R <= 2 && fills(4) ? 4 : fills(2) ? 2 : 1;
  const int chunk = 4 * kThreads * quads;
  const int weight_blocks = p.scores != nullptr ? (p.a.Lmax + chunk - 1) / chunk : 0;
  const dim3 grid(static_cast<unsigned>(row_blocks + heads * weight_blocks));
  const size_t smem = p.scores != nullptr ? p.rp.R * 2 * sizeof(float) : 0;
  auto pick = [&](auto w) -> void (*)(Params, int, int) {
    constexpr bool kWide = decltype(w)::value;
    if (p.scores == nullptr) return decode_q8_join_kernel<T, kWide, 0>;
    return quads == 4   ? decode_q8_join_kernel<T, kWide, 4>
           : quads == 2 ? decode_q8_join_kernel<T, kWide, 2>
                        : decode_q8_join_kernel<T, kWide, 1>;
  };
  return launch_pdl(wide ? pick(std::true_type{}) : pick(std::false_type{}), grid, dim3(kThreads),
                    smem, s, p, row_blocks, weight_blocks);
}

}  // namespace

size_t decode_q8_workspace(int B, int H, int Hkv, int Nq, int Lmax, bool weights) {
  if (alone(B, H, Hkv, Nq, Lmax)) return 0;
  return std::max(plan(B, H, Hkv, Nq, Lmax, 0, weights).total,
                  plan(B, H, Hkv, Nq, Lmax, 1, weights).total);
}

cudaError_t launch_sdpa_decode_q8(const DecodeQ8Args& a, int dtype, int qtype, void* ws,
                                  const DevCtx& ctx, cudaStream_t s) {
  const Workspace w = plan(a.B, a.H, a.Hkv, a.Nq, a.Lmax, dtype, a.weights != nullptr);
  Params p;
  p.a = a;
  p.rp = row_plan(a.H, a.Hkv, a.Nq, dtype);
  const int blocks = std::min(ctx.num_sms, 160);
  p.workers = blocks * main_warps(dtype == 1 ? 1 : 2, p.rp.NR);
  p.block_shift = 0;
  while ((1 << p.block_shift) < a.block) ++p.block_shift;
  p.part = static_cast<float*>(ws);
  p.stat = reinterpret_cast<float*>(static_cast<char*>(ws) + w.stat);
  p.scores = a.weights != nullptr
                 ? reinterpret_cast<float*>(static_cast<char*>(ws) + w.scores) : nullptr;
  p.Lpad = w.Lpad;
  if (alone(a.B, a.H, a.Hkv, a.Nq, a.Lmax))
    return dtype == 1 ? launch_alone<__nv_bfloat16>(p, qtype, s) : launch_alone<float>(p, qtype, s);
  return dtype == 1 ? launch_all<__nv_bfloat16>(p, qtype, blocks, s)
                    : launch_all<float>(p, qtype, blocks, s);
}

}  // namespace mha
