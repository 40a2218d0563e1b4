// The attention of one new token per sequence over a paged key-value cache.
//
//   out[h] = sum_t softmax_t(scale * q[h] . k[t]) v[t],  lse[h] = log sum_t exp(...)
//
// What bounds it: every key and value is read once from HBM; 4 flops per
// element and query head, which the matrix cores have in plenty for up to 16
// query heads on one kv head.  More are taken 16 at a time, and each 16 read the
// cache again (4 x 32768 tokens of one kv head: 26 us for 16 query heads, 46 for
// 64).
//
// One wave takes a chunk of 32 tokens (64 of an int8 cache) of one kv head at
// a time.  Scores are K x Q^T tiles: the 16 rows are tokens, the 16 columns
// the query heads of the kv head, so a lane ends up with 4 tokens' scores of
// one head.  Which token a tile's row stands for is free: row 4a+i of tile t
// is token 8a+4t+i (16a+4t+i for int8), and then the probabilities that a
// lane holds are exactly the 8 (16) consecutive tokens that it has to feed to
// V^T x P^T, whose other operand is one 16-byte load from the [dim][token]
// value page.  Nothing moves between lanes except the running maximum, and
// that only when a score exceeds it by 2^8 or more: a factor common to sum
// and output cancels, so the maximum need not be exact.
//
// Precision: scores, maxima, sums and outputs are fp32.  A probability goes
// to the matrix cores as numbers of the operand type that add up to it: three
// of bfloat16 (also for int8 values), which hold all its 24 bits, or two of
// float16 with sums of their own, which hold 22 of those that are at least 2^-20
// of the maximum and end at 2^-42 of it.  The cores are far from bound: 64
// sequences of up to 8192 tokens, int8, take 106 us with two bfloat16 parts and
// 107 with three, a bfloat16 cache the same with either.  Of the outputs 0.44%
// (131071 tokens, bfloat16) and 2.3% (the int8 ones) were not the exact result's
// rounding with two, 0.05% and 0.3% with three.  int8 codes are exact operands;
// the key's scale multiplies the fp32 score, the value's the fp32 probability.
//
// The batch's tokens, one sequence after the other, are dealt out evenly to 512
// workgroups (two on every CU), which find their sequences from the lengths;
// a workgroup's 4 waves take its chunks in turn.  So very different lengths
// cost nothing (64 sequences of 1..8192 tokens, int8: 150 us with pieces of
// one length, 105 to 109 so, 5.2 TB/s), and one long sequence is split as well
// (131071 tokens: 62 us; 384 workgroups take 73, 768 take 66).  Waves join in
// LDS, cut sequences in a second kernel, each in a fixed order.  Where no
// sequence can be longer than 256 tokens each is one workgroup's, and there is
// no second kernel (one of 200: 11 us, 16 with one, most of it the launches).
#include "kv_attention.h"

namespace i8mm {

namespace {

constexpr int kJoinThreads = 256;
constexpr int kMaxParts = 512;  // workgroups that share a batch: two on every CU
constexpr int kWhole = 256;     // tokens up to which a sequence is one workgroup's

template <int CT, bool QBF, int NK, bool EXACT>
__global__ __launch_bounds__(64 * kWaves, NK <= 4 ? 2 : 1) void k_kv_attention(KvAttentionArgs a, Pages pg) {
  attend_own<CT, QBF, NK, EXACT>(a, pg, blockIdx.x, blockIdx.y);
}

// Joins the pieces of one (sequence, query head); a lane holds 4 dims.
template <bool QBF>
__global__ __launch_bounds__(kJoinThreads) void k_kv_join(KvAttentionArgs a, int D) {
  __shared__ float f[kMaxParts];
  __shared__ float dens[kJoinThreads / 64];
  __shared__ v4f part[kJoinThreads];
  const int64_t bh = blockIdx.x;
  const int b = (int)(bh / a.q_heads), hq = (int)(bh % a.q_heads);
  const int lane = threadIdx.x & 63;
  const int2 cut = a.cuts[b];
  const int n = cut.y;
  if (n == 1) return;  // one workgroup had it all
  const int tiles_h = (a.group + kKvHeadTile - 1) / kKvHeadTile;
  const int gy = hq / a.group * tiles_h + hq % a.group / kKvHeadTile;
  const int h = hq % a.group % kKvHeadTile;
  // piece i: of part cut.x / 2 + i; the first may be that part's second place
  auto piece = [&](int i) {
    const int64_t at = ((int64_t)gy * a.parts + (cut.x >> 1) + i) * 2 + (i == 0 ? cut.x & 1 : 0);
    return at * a.tile_heads + h;
  };
  // the outputs' first loads, before the factors are known
  const int quads = D / 4, groups = kJoinThreads / quads;
  const int g = threadIdx.x / quads, d = threadIdx.x % quads * 4;
  constexpr int kU = 4;  // loads in flight
  v4f v[kU];
  auto load = [&](int i) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
      v[u] = *reinterpret_cast<const v4f*>(a.part_o + piece(min(i + u * groups, n - 1)) * D + d);
  };
  if (n > 0) load(g);
  // every wave forms the maximum over all pieces; the factors are shared
  float mx = -INFINITY, den = 0.0f;
  for (int i = lane; i < n; i += 64) mx = fmaxf(mx, a.part_ml[2 * piece(i)]);
  mx = wave_max(mx);
  for (int i = threadIdx.x; i < n; i += kJoinThreads) {
    const float* ml = a.part_ml + 2 * piece(i);
    // no visible score: the sums are 0 (or NaN, which stays)
    f[i] = ml[0] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(ml[0] - mx);
    den += f[i] * ml[1];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) den += __shfl_xor(den, o, 64);
  if (lane == 0) dens[threadIdx.x >> 6] = den;
  __syncthreads();

  v4f sum = {0, 0, 0, 0};
  if (g < groups) {
    for (int i = g; i < n; i += groups * kU) {
      if (i != g) load(i);
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (i + u * groups < n) sum += f[i + u * groups] * v[u];
    }
  }
  part[threadIdx.x] = sum;
  __syncthreads();
  if (g == 0) {
    den = 0.0f;
    for (int w = 0; w < kJoinThreads / 64; ++w) den += dens[w];
    for (int w = 1; w < groups && w < n; ++w) sum += part[w * quads + threadIdx.x];
    const float inv = 1.0f / den;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float y = den == 0.0f ? 0.0f : sum[e] * inv;
      a.out[bh * D + d + e] = QBF ? __builtin_bit_cast(uint16_t, (__bf16)y) : f2h(y);
    }
    if (threadIdx.x == 0 && a.lse != nullptr)
      a.lse[bh] = den == 0.0f ? -INFINITY : (mx + __builtin_log2f(den)) * kLn2;
  }
}

template <int CT, bool QBF, int NK, bool EXACT>
hipError_t run(const KvAttentionArgs& a, const Pages& pg, hipStream_t s) {
  const dim3 grid((unsigned)(a.parts > 0 ? a.parts : a.B),
                  (unsigned)(pg.kv_heads * ((a.group + kKvHeadTile - 1) / kKvHeadTile)));
  hipLaunchKernelGGL((k_kv_attention<CT, QBF, NK, EXACT>), grid, dim3(64 * kWaves), 0, s, a, pg);
  return hipGetLastError();
}

// Head sizes that are whole 32-dim steps (int8: 64) have instances without
// idle registers and tiles: an int8 cache of 8 x 8192 tokens, 8 kv heads of
// 192 / 256 dims, is read at 3.8 / 4.1 TB/s so, 3.2 / 3.8 with the general
// one; 17 sequences of up to 1000 tokens of 6 x 96 dims take 19.1 us, 20.2 with
// the general one.  Other sizes, and 32 and 160 dims, lose up to the same.
template <int CT, bool QBF>
hipError_t pick(const KvAttentionArgs& a, const Pages& pg, hipStream_t s) {
  switch (pg.D) {
    case 64: return run<CT, QBF, 2, true>(a, pg, s);
    case 96: if constexpr (CT != kI8) return run<CT, QBF, 3, true>(a, pg, s); break;
    case 128: return run<CT, QBF, 4, true>(a, pg, s);
    case 192: return run<CT, QBF, 6, true>(a, pg, s);
    case 256: return run<CT, QBF, 8, true>(a, pg, s);
  }
  return pg.D < 128 ? run<CT, QBF, 4, false>(a, pg, s) : run<CT, QBF, 8, false>(a, pg, s);
}

}  // namespace

int kv_attention_parts(int64_t B, int64_t head_groups, int64_t max_len, int64_t window) {
  // a window begins anywhere in the 64 tokens that a sequence's first unit is aligned to
  if (window > 0 && window + kAlign - 1 < max_len) max_len = window + kAlign - 1;
  if (max_len <= kWhole) return 0;
  const int64_t most = B * ((max_len + 127) / 128);
  int64_t parts = (kMaxParts + head_groups - 1) / head_groups;
  if (parts > most) parts = most;
  return (int)parts;
}

hipError_t launch_kv_attention(const KvAttentionArgs& a, bool bf16, const int8mm_kv& kv,
                               hipStream_t s) {
  const Pages pg = pages_of(kv);
  hipError_t e;
  if (kv.dtype == INT8MM_F16)
    e = pick<kF16, false>(a, pg, s);
  else if (kv.dtype == INT8MM_BF16)
    e = pick<kBF16, true>(a, pg, s);
  else
    e = bf16 ? pick<kI8, true>(a, pg, s) : pick<kI8, false>(a, pg, s);
  if (e != hipSuccess || a.parts == 0 || a.whole_o != nullptr) return e;
  const dim3 grid((unsigned)((int64_t)a.B * a.q_heads)), block(kJoinThreads);
  if (bf16)
    hipLaunchKernelGGL(k_kv_join<true>, grid, block, 0, s, a, pg.D);
  else
    hipLaunchKernelGGL(k_kv_join<false>, grid, block, 0, s, a, pg.D);
  return hipGetLastError();
}

}  // namespace i8mm
