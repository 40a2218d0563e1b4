// Products of a few rows with 4-bit weights and group scales, and the
// one-time packing of those weights.
//
//   Y[m][n] = sum_g s[n][g] * sum_{k in g} X[m][k] * (q[n][k] - z[n][g]) + bias[n]
//
// What bounds it: the weight's N*K/2 bytes from HBM, read once per call (64
// rows a pass); a row of X adds 2*N*K flops, so up to 64 rows the matrix
// cores have room.
//
// Codes become MFMA operands without a table or a convert: a nibble or-ed
// into the mantissa of a fixed exponent is an exact number.  float16 rows:
// 1024 + q (or 1024 + 16 q), of which one packed add (fma) makes q - 8, exact.
// bfloat16 rows: 128 + q, and the constant comes off the group's sum with z:
// sum x (128 + q) - (128 + z) sum x, with sum x from one more MFMA against ones.
// Products of the codes are exact, sums are fp32 and the group's scale
// multiplies the fp32 sum: the one rounding to fewer bits is Y's.  The offset
// costs a sum about 4 of fp32's 24 bits, since its terms x (128 + q) are up to
// 18 times (143 / 8) those of the result, whose rounding keeps 8; and it ends
// the range where 128 terms of 143 |x| pass fp32's, above |x| = 2^113.
#include <type_traits>

#include "device_common.h"
#include "serving_launch.h"

namespace i8mm {

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float bf2f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f2bf(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

template <bool BF16>
__device__ __forceinline__ v4f mfma32(const v4u& a, const v4u& b, const v4f& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a),
                                                   __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Constants of the nibble extraction, held in registers: v_and_or_b32 takes
// no literals, and with literals each nibble pair costs an and plus an or.
struct Nibbles {
  uint32_t lo, hi, one;
};
template <bool BF16>
__device__ __forceinline__ Nibbles nibbles() {
  Nibbles n;
  asm("v_mov_b32 %0, 0x000f000f" : "=v"(n.lo));
  asm("v_mov_b32 %0, 0x00f000f0" : "=v"(n.hi));
  if constexpr (BF16)
    asm("v_mov_b32 %0, 0x43004300" : "=v"(n.one));
  else
    asm("v_mov_b32 %0, 0x64006400" : "=v"(n.one));
  return n;
}

// The 8 codes of one dword as an MFMA operand: float16 q - z, bfloat16
// 128 + q.  bias (float16): 1024 + z twice.
template <bool BF16>
__device__ __forceinline__ v4u codes8(uint32_t u, uint32_t bias, const Nibbles& n) {
  if constexpr (BF16) {
    return v4u{(u & n.lo) | n.one, ((u >> 4) & n.lo) | n.one, ((u >> 8) & n.lo) | n.one,
               ((u >> 12) & n.lo) | n.one};
  } else {
    const uint32_t w = u >> 8;
    const v2h z = __builtin_bit_cast(v2h, bias);
    const v2h sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    const v2h c = {(_Float16)960.0f, (_Float16)960.0f};
    const v2h y = c - z;  // -(64 + z)
    auto plain = [&](uint32_t x) { return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, x) - z); };
    auto wide = [&](uint32_t x) {
      return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(v2h, x), sixteenth, y));
    };
    return v4u{plain((u & n.lo) | n.one), wide((u & n.hi) | n.one), plain((w & n.lo) | n.one),
               wide((w & n.hi) | n.one)};
  }
}

constexpr int kCus = 256;  // compute units of the MI355X

// What both kernels do with one parameter entry and one dword of codes.
template <bool BF16, bool ZEROS, int GS>
struct Group {
  static constexpr int NG = 4 / GS;                    // entries per tile and channel
  static constexpr int PB = NG * (ZEROS ? 4 : 2);      // their bytes
  using Par = typename std::conditional<PB == 16, v4u, typename std::conditional<PB == 8, v2u,
              typename std::conditional<PB == 4, uint32_t, uint16_t>::type>::type>::type;
  // 16-bit word i of the entries, twice
  static __device__ __forceinline__ uint32_t word2(const Par& e, int i) {
    uint32_t u;
    if constexpr (PB <= 4)
      u = e;
    else
      u = e[i >> 1];
    return __builtin_amdgcn_perm(u, u, (i & 1) ? 0x03020302u : 0x01000100u);
  }
  // entry g's scale; 1024 + z twice (float16 operands); 128 + z (bfloat16 sums)
  static __device__ __forceinline__ float scale(const Par& e, int g) {
    return h2f((uint16_t)word2(e, ZEROS ? 2 * g : g));
  }
  static __device__ __forceinline__ uint32_t bias(const Par& e, int g) {
    return ZEROS && !BF16 ? word2(e, 2 * g + 1) : 0x64086408u;
  }
  static __device__ __forceinline__ float offset(const Par& e, int g) {
    return ZEROS ? h2f((uint16_t)word2(e, 2 * g + 1)) - 896.0f : 136.0f;
  }
};
constexpr uint32_t kOnesBf16 = 0x3f803f80u;

// ------------------------------------------------------ up to 16 rows
//
// One workgroup: P tiles of 16 channels, its waves splitting K tile by tile.
// GS: 32-k steps per parameter entry.  Rows 16-byte aligned, K a multiple of 8.
//
// X is the A operand and W the B operand, so that a lane's codes and its sums
// belong to the same channel (lane % 16) and one parameter entry serves both.
constexpr int max_waves(int P) { return P == 1 ? 16 : 8; }

template <bool BF16, bool ZEROS, int GS, int P>
__global__ __launch_bounds__(64 * max_waves(P)) void k_int4_few(
    const uint16_t* __restrict__ X, int M, int K, int64_t ldx, const uint8_t* __restrict__ Wq,
    const uint8_t* __restrict__ params, int N, const uint16_t* __restrict__ bias,
    uint16_t* __restrict__ Y) {
  using G = Group<BF16, ZEROS, GS>;
  extern __shared__ float red[];  // [waves][P][4][64]

  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, qd = lane >> 4;
  const int nt = (K + kInt4TileK - 1) / kInt4TileK;
  const int panel0 = blockIdx.x * P;
  const int64_t xl = (int64_t)min(r, M - 1) * ldx + qd * 8;

  // the last workgroup may have fewer than P tiles of channels: it takes the
  // last one again, and does not store it
  const int panels = (N + 15) / 16;
  int64_t first[P];
#pragma unroll
  for (int p = 0; p < P; ++p) first[p] = (int64_t)min(panel0 + p, panels - 1) * nt;
  const Nibbles nib = nibbles<BF16>();

  v4u w[2][P], x[4];
  typename G::Par par[2][P];
  auto load_w = [&](int st, int t) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t tile = first[p] + t;
      w[st][p] = __builtin_nontemporal_load(
          reinterpret_cast<const v4u*>(Wq + tile * kInt4TileBytes) + lane);
      par[st][p] = reinterpret_cast<const typename G::Par*>(params + tile * (16 * G::PB))[r];
    }
  };
  auto load_x = [&](int t, int s) __attribute__((always_inline)) {
    x[s] = *reinterpret_cast<const v4u*>(X + t * kInt4TileK + s * 32 + xl);
  };

  const int whole = K / kInt4TileK, last = whole - 1;

  v4f tot[P];
#pragma unroll
  for (int p = 0; p < P; ++p) tot[p] = v4f{0, 0, 0, 0};

  // tile t of stage st; a step's X registers take tile tn's as soon as the step
  // is done (tn < 0: none)
  auto compute = [&](int st, int tn) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < G::NG; ++g) {
      __builtin_amdgcn_sched_barrier(0);
      v4f acc[P], sx = {0, 0, 0, 0};
#pragma unroll
      for (int p = 0; p < P; ++p) acc[p] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int s = g * GS; s < (g + 1) * GS; ++s) {
        if constexpr (BF16) sx = mfma32<true>(x[s], v4u{kOnesBf16, kOnesBf16, kOnesBf16, kOnesBf16}, sx);
#pragma unroll
        for (int p = 0; p < P; ++p)
          acc[p] = mfma32<BF16>(x[s], codes8<BF16>(w[st][p][s], G::bias(par[st][p], g), nib), acc[p]);
        if (tn >= 0) load_x(tn, s);
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float sc = G::scale(par[st][p], g), off = G::offset(par[st][p], g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = acc[p][i];
          if constexpr (BF16) v = __builtin_fmaf(-off, sx[i], v);
          tot[p][i] = __builtin_fmaf(sc, v, tot[p][i]);
        }
      }
    }
  };

  // whole tiles: while one is multiplied, the next one's loads are in flight
  if (wave < whole) {
    load_w(0, wave);
    load_w(1, min(wave + waves, last));
#pragma unroll
    for (int s = 0; s < 4; ++s) load_x(wave, s);
    for (int t = wave; t < whole; t += 2 * waves) {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        if (st > 0 && t + waves >= whole) break;
        // a wave at its end reads the last tile again: with a branch around
        // the loads their registers spill
        compute(st, min(t + (st + 1) * waves, last));
        load_w(st, min(t + (st + 2) * waves, last));
      }
    }
  }
  // the last tile of a K that is not a multiple of 128
  if (whole < nt && wave == whole % waves) {
    load_w(0, whole);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      x[s] = v4u{0, 0, 0, 0};
      if (whole * kInt4TileK + s * 32 + qd * 8 < K) load_x(whole, s);
    }
    compute(0, -1);
  }

  // the waves' partial sums, added in wave order
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[((wave * P + p) * 4 + i) * 64 + lane] = tot[p][i];
  __syncthreads();
  for (int o = threadIdx.x; o < M * 16 * P; o += blockDim.x) {
    const int nl = o % (16 * P), m = o / (16 * P);
    const int n = panel0 * 16 + nl;
    if (n >= N) continue;
    const int at = ((nl >> 4) * 4 + (m & 3)) * 64 + (m >> 2) * 16 + (nl & 15);
    float y = 0.0f;
    for (int w = 0; w < waves; ++w) y += red[w * P * 256 + at];
    if (bias != nullptr) y += BF16 ? bf2f(bias[n]) : h2f(bias[n]);
    Y[(int64_t)m * N + n] = BF16 ? f2bf(y) : f2h(y);
  }
}

// ------------------------------------------- more rows, or any alignment
//
// 4 * KS waves share X: 4 groups of P channel tiles times the KS tiles of K of
// a step.  A step's X, up to 64 rows of KS * 256 contiguous bytes, goes through
// registers into LDS in operand order, the next step's while this one is
// multiplied; a chunk's place is exclusive-ored with its k so that neither side
// has bank conflicts.  Rows past M and k past K are zeros there, so every shape
// and alignment takes this one path.  Where few channels leave CUs idle K is
// split over workgroups too (blockIdx.z), and a second kernel adds their sums.
//
// 64 x 8192 x 28672 takes 50.5 us, of which 28 are the matrix instructions and
// the groups' scales alone (1.1 of the 1.2 PFLOP/s that a large library product
// reaches here), 10 the codes and LDS, the rest the loads; 48 x 5120 x 13811 in
// groups of 32 takes 22 to 23 us, 64 x 4096 x 11008 18.3.  Every wave forms
// bfloat16's sums of X for itself, one matrix instruction for each useful one
// with one channel tile: 64 x 8192 x 28672 takes 58 us in bfloat16, and 95 in
// groups of 32 (58 in float16).
template <bool BF16, bool ZEROS, int GS, int MT, int P, int KS>
__global__ __launch_bounds__(256 * KS) void k_int4_many(
    const uint16_t* __restrict__ X, int M, int K, int64_t ldx, int vec,
    const uint8_t* __restrict__ Wq, const uint8_t* __restrict__ params, int N,
    const uint16_t* __restrict__ bias, uint16_t* __restrict__ Y, float* __restrict__ part) {
  using G = Group<BF16, ZEROS, GS>;
  // X is requested two steps ahead and the weight three, where the registers
  // allow (64 x 8192 x 28672, groups of 128: 52.7 -> 50 us, 32 rows 38.5 -> 35;
  // with two channel tiles and narrow groups, or 16 waves, they would spill:
  // one and two)
  constexpr bool kDeep = KS == 2 && (P == 1 || GS == 4);
  constexpr int kStages = kDeep ? 4 : 3, kAhead = kDeep ? 2 : 1;
  constexpr int kManyWaves = 4 * KS;
  constexpr int kChunk = MT * KS * 4 * 64;  // 16-byte units of one step's X
  constexpr int kSums = kManyWaves * P * MT * 256 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kChunk * 16 > kSums ? 2 * kChunk * 16 : kSums];
  v4u* xs = reinterpret_cast<v4u*>(lds);        // [2][tile][MT][step][64]
  float* red = reinterpret_cast<float*>(lds);   // [wave][P][MT][4][64]

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, qd = lane >> 4;
  const int pg = wave & 3, ks = wave >> 2;
  const int nt = (K + kInt4TileK - 1) / kInt4TileK, steps = (nt + KS - 1) / KS;
  // this workgroup's steps
  const int step0 = (int)((int64_t)blockIdx.z * steps / gridDim.z);
  const int step1 = (int)((int64_t)(blockIdx.z + 1) * steps / gridDim.z);
  const int m0 = blockIdx.y * (16 * MT);
  const int panels = (N + 15) / 16, panel0 = blockIdx.x * (4 * P) + pg * P;
  int64_t first[P];
#pragma unroll
  for (int p = 0; p < P; ++p) first[p] = (int64_t)min(panel0 + p, panels - 1) * nt;
  const Nibbles nib = nibbles<BF16>();

  // staging: this thread's chunk of 8 k in rows row0 + 16 i
  const int c = threadIdx.x % (16 * KS), row0 = threadIdx.x / (16 * KS);
  v4u hold[kAhead][MT];
  auto fetch = [&](int h, int step) __attribute__((always_inline)) {
    const int k = step * (KS * kInt4TileK) + c * 8;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int m = m0 + row0 + 16 * i;
      hold[h][i] = v4u{0, 0, 0, 0};
      if (m >= M || k >= K) continue;
      const uint16_t* p = X + (int64_t)m * ldx + k;
      if (vec) {
        hold[h][i] = *reinterpret_cast<const v4u*>(p);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a = k + 2 * e < K ? p[2 * e] : 0u;
          const uint32_t b = k + 2 * e + 1 < K ? p[2 * e + 1] : 0u;
          hold[h][i][e] = a | (b << 16);
        }
      }
    }
  };
  auto stage = [&](int h, int buf) __attribute__((always_inline)) {
    const int t = c >> 4, sq = c & 15;  // tile of the step, (32-k step, quarter)
#pragma unroll
    for (int i = 0; i < MT; ++i)
      xs[buf * kChunk + ((t * MT + i) * 4 + (sq >> 2)) * 64 + (sq & 3) * 16 + (row0 ^ sq)] = hold[h][i];
  };

  v4u w[kStages][P];
  typename G::Par par[kStages][P];
  auto load_w = [&](int st, int step) __attribute__((always_inline)) {
    const int t = min(step * KS + ks, nt - 1);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t tile = first[p] + t;
      w[st][p] = __builtin_nontemporal_load(
          reinterpret_cast<const v4u*>(Wq + tile * kInt4TileBytes) + lane);
      par[st][p] = reinterpret_cast<const typename G::Par*>(params + tile * (16 * G::PB))[r];
    }
  };

  v4f tot[P][MT];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int m = 0; m < MT; ++m) tot[p][m] = v4f{0, 0, 0, 0};

  auto compute = [&](int st, int buf) __attribute__((always_inline)) {
    const v4u* xb = xs + buf * kChunk + ks * MT * 256;
#pragma unroll
    for (int g = 0; g < G::NG; ++g) {
      __builtin_amdgcn_sched_barrier(0);
      v4f acc[P][MT], sx[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        sx[m] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < P; ++p) acc[p][m] = v4f{0, 0, 0, 0};
      }
#pragma unroll
      for (int s = g * GS; s < (g + 1) * GS; ++s) {
        v4u x[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = xb[(m * 4 + s) * 64 + qd * 16 + (r ^ (s * 4 + qd))];
        if constexpr (BF16)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            sx[m] = mfma32<true>(x[m], v4u{kOnesBf16, kOnesBf16, kOnesBf16, kOnesBf16}, sx[m]);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const v4u b = codes8<BF16>(w[st][p][s], G::bias(par[st][p], g), nib);
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[p][m] = mfma32<BF16>(x[m], b, acc[p][m]);
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float sc = G::scale(par[st][p], g), off = G::offset(par[st][p], g);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = acc[p][m][i];
            if constexpr (BF16) v = __builtin_fmaf(-off, sx[m][i], v);
            tot[p][m][i] = __builtin_fmaf(sc, v, tot[p][m][i]);
          }
      }
    }
  };
  // LDS of this workgroup is written and read; loads into registers stay in flight
  auto sync = [&]() __attribute__((always_inline)) {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };

  // The later tiles of the last step may lie past K: their X is zero, and the
  // weight read in their place is finite.
  const int last = step1 - 1;
  if (step0 < step1) {
    fetch(0, step0);
    load_w(0, step0);
    if (kDeep) fetch(kAhead - 1, min(step0 + 1, last));
#pragma unroll
    for (int st = 1; st < kStages - 1; ++st) load_w(st, min(step0 + st, last));
    stage(0, 0);
    sync();
    for (int t = step0; t < step1; t += kStages) {
#pragma unroll
      for (int st = 0; st < kStages; ++st) {
        if (st > 0 && t + st > last) break;
        const int now = t + st, buf = (now - step0) & 1;
        // X first: loads return in order, and waiting for X must not wait for
        // the weight of steps further on
        fetch(st % kAhead, min(now + kAhead, last));
        load_w((st + kStages - 1) % kStages, min(now + kStages - 1, last));
        compute(st, buf);
        stage((st + 1) % kAhead, buf ^ 1);  // (read last a step ago, before the barrier there)
        sync();
      }
    }
  }

  // the waves' partial sums: the KS shares of K, in order
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[(((wave * P + p) * MT + m) * 4 + i) * 64 + lane] = tot[p][m][i];
  __syncthreads();
  const int rows = min(M - m0, 16 * MT);
  constexpr int kCols = 4 * P * 16;
  for (int o = threadIdx.x; o < rows * kCols; o += 64 * kManyWaves) {
    const int nl = o % kCols, m = o / kCols;
    const int n = blockIdx.x * kCols + nl;
    if (n >= N) continue;
    const int wv = nl / (16 * P), p = nl / 16 % P;
    const int at = (((wv * P + p) * MT + (m >> 4)) * 4 + (m & 3)) * 64 + ((m & 15) >> 2) * 16 + (nl & 15);
    float y = red[at];
#pragma unroll
    for (int h = 1; h < KS; ++h) y += red[at + h * 4 * P * MT * 256];
    if (part != nullptr) {
      part[((int64_t)blockIdx.z * M + m0 + m) * N + n] = y;
    } else {
      if (bias != nullptr) y += BF16 ? bf2f(bias[n]) : h2f(bias[n]);
      Y[(int64_t)(m0 + m) * N + n] = BF16 ? f2bf(y) : f2h(y);
    }
  }
}

// Adds the parts of K, in order.
template <bool BF16>
__global__ __launch_bounds__(256) void k_int4_sum(const float* __restrict__ part, int parts,
                                                  int64_t total, int N,
                                                  const uint16_t* __restrict__ bias,
                                                  uint16_t* __restrict__ Y) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    float y = 0.0f;
    for (int z = 0; z < parts; ++z) y += part[z * total + i];
    if (bias != nullptr) {
      const uint16_t b = bias[i % N];
      y += BF16 ? bf2f(b) : h2f(b);
    }
    Y[i] = BF16 ? f2bf(y) : f2h(y);
  }
}

// K == 0
__global__ void k_int4_bias(const uint16_t* __restrict__ bias, int64_t total, int N,
                            uint16_t* __restrict__ Y) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x)
    Y[i] = bias != nullptr ? bias[i % N] : 0;
}

// ---------------------------------------------------------------- packing

// Where the 8 codes of channel n, k .. k+7 (k a multiple of 8) are stored.
__device__ __forceinline__ int64_t code_dword(int64_t n, int64_t k, int64_t nt) {
  const int64_t tile = (n >> 4) * nt + (k >> 7);
  const int l = (int)(n & 15) + 16 * (int)((k >> 3) & 3);
  return tile * (kInt4TileBytes / 4) + l * 4 + (int)((k >> 5) & 3);
}
__device__ __forceinline__ uint32_t pack8_u4(const uint8_t (&c)[8]) {
  constexpr int at[8] = {0, 4, 1, 5, 2, 6, 3, 7};
  uint32_t u = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) u |= (uint32_t)(c[e] & 15) << (4 * at[e]);
  return u;
}

__global__ void k_int4_pack(const uint8_t* __restrict__ codes, int64_t N, int64_t K, int64_t Np,
                            int64_t nt, uint32_t* __restrict__ Wq) {
  const int64_t oct = nt * 16, total = Np * oct;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t n = i / oct, k = (i % oct) * 8;
    uint8_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = n < N && k + e < K ? codes[n * K + k + e] : 8;
    Wq[code_dword(n, k, nt)] = pack8_u4(c);
  }
}

// Parameter entries; i counts them in stored order [panel][tile][channel][sub-group].
__global__ void k_int4_params(const uint16_t* __restrict__ scales, const uint8_t* __restrict__ zeros,
                              int64_t N, int64_t K, int64_t group, int gs, int64_t nt,
                              int64_t total, uint16_t* __restrict__ params) {
  const int ng = kInt4TileK / gs;
  const int64_t groups = (K + group - 1) / group;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t e = i / ng, tile = e >> 4;
    const int64_t n = (tile / nt) * 16 + (e & 15);
    const int64_t k = (tile % nt) * kInt4TileK + (i % ng) * gs;
    const bool in = n < N && k < K;
    const int64_t at = in ? n * groups + k / group : 0;
    const uint16_t sc = in ? scales[at] : (uint16_t)0;
    if (zeros != nullptr) {
      params[2 * i] = sc;
      params[2 * i + 1] = f2h(1024.0f + (in ? (float)(zeros[at] & 15) : 8.0f));
    } else {
      params[i] = sc;
    }
  }
}

// One wave quantizes one group of one channel (channels past N: padding).
template <bool BF16>
__global__ __launch_bounds__(256) void k_int4_prepare(const uint16_t* __restrict__ W, int64_t N,
                                                      int64_t K, int64_t Np, int64_t group,
                                                      int gs, int64_t nt, bool zeros,
                                                      uint32_t* __restrict__ Wq,
                                                      uint16_t* __restrict__ params) {
  const int lane = threadIdx.x & 63;
  const int64_t groups = (K + group - 1) / group;
  for (int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); id < Np * groups;
       id += (int64_t)gridDim.x * 4) {
  const int64_t n = id / groups, g = id % groups;
  const int64_t k0 = g * group, k1 = min(K, k0 + group);
  // the last group also fills the padding of its tile
  const int64_t kend = g == groups - 1 ? nt * kInt4TileK : k0 + group;
  const uint16_t* row = W + n * K;
  auto value = [&](int64_t k) { return BF16 ? bf2f(row[k]) : h2f(row[k]); };
  float lo = 0.0f, hi = 0.0f;
  if (n < N)
    for (int64_t k = k0 + lane; k < k1; k += 64) {
      const float x = value(k);
      lo = fminf(lo, x);
      hi = fmaxf(hi, x);
    }
  hi = wave_max(hi);
  lo = -wave_max(-lo);
  const float span = zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f;
  const uint16_t sc = f2h(fminf(span, 65504.0f));
  const float s = h2f(sc);
  const float d = s > 0.0f ? s : 1.0f;
  const float z = zeros ? (s > 0.0f ? fminf(fmaxf(rintf(-lo / d), 0.0f), 15.0f) : 0.0f) : 8.0f;
  for (int64_t k = k0 + lane * 8; k < kend; k += 512) {
    uint8_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float q = z;
      if (n < N && k + e < k1 && s > 0.0f) q = fminf(fmaxf(rintf(value(k + e) / d) + z, 0.0f), 15.0f);
      c[e] = n < N && k + e < k1 ? (uint8_t)q : 8;
    }
    Wq[code_dword(n, k, nt)] = pack8_u4(c);
  }
  const int ng = kInt4TileK / gs;
  for (int64_t k = k0 + lane * gs; k < kend; k += 64 * gs) {
    const int64_t tile = (n >> 4) * nt + (k >> 7);
    const int64_t e = (tile * 16 + (n & 15)) * ng + (k & 127) / gs;
    const bool in = n < N && k < K;
    if (zeros) {
      params[2 * e] = in ? sc : (uint16_t)0;
      params[2 * e + 1] = f2h(1024.0f + (in ? z : 8.0f));
    } else {
      params[e] = in ? sc : (uint16_t)0;
    }
  }
  }
}

unsigned grid_for(int64_t total, int block) {
  const int64_t b = (total + block - 1) / block;
  return (unsigned)(b < 16384 ? b : 16384);
}

}  // namespace

hipError_t launch_int4_pack(const uint8_t* codes, int64_t N, int64_t K, int64_t group,
                            const uint16_t* scales, const uint8_t* zeros, uint32_t* Wq,
                            uint16_t* params, hipStream_t s) {
  const int64_t Np = int4_padded_rows(N), nt = int4_tiles_k(K);
  const int gs = 32 * int4_group_steps(group);
  hipLaunchKernelGGL(k_int4_pack, dim3(grid_for(Np * nt * 16, 256)), dim3(256), 0, s, codes, N, K,
                     Np, nt, Wq);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t entries = Np * nt * (kInt4TileK / gs);
  hipLaunchKernelGGL(k_int4_params, dim3(grid_for(entries, 256)), dim3(256), 0, s, scales, zeros, N,
                     K, group, gs, nt, entries, params);
  return hipGetLastError();
}

hipError_t launch_int4_prepare(const uint16_t* W, bool bf16, int64_t N, int64_t K, int64_t group,
                               bool zeros, uint32_t* Wq, uint16_t* params, hipStream_t s) {
  const int64_t Np = int4_padded_rows(N), nt = int4_tiles_k(K);
  const int gs = 32 * int4_group_steps(group);
  const int64_t waves = Np * ((K + group - 1) / group);
  // at most 2^20 workgroups: a launch holds fewer than 2^32 threads
  const dim3 grid((unsigned)(waves < (1 << 22) ? (waves + 3) / 4 : 1 << 20));
  if (bf16)
    hipLaunchKernelGGL(k_int4_prepare<true>, grid, dim3(256), 0, s, W, N, K, Np, group, gs, nt,
                       zeros, Wq, params);
  else
    hipLaunchKernelGGL(k_int4_prepare<false>, grid, dim3(256), 0, s, W, N, K, Np, group, gs, nt,
                       zeros, Wq, params);
  return hipGetLastError();
}

namespace {

template <bool BF16, bool ZEROS, int GS, int P>
hipError_t run_few(const Int4Args& a, hipStream_t s) {
  const int nt = (int)int4_tiles_k(a.K);
  int waves = max_waves(P);
  while (waves > nt) waves /= 2;
  hipLaunchKernelGGL((k_int4_few<BF16, ZEROS, GS, P>), dim3((a.N + 16 * P - 1) / (16 * P)),
                     dim3(64 * waves), (size_t)waves * P * 1024, s, a.X, a.M, a.K, a.ldx, a.Wq,
                     a.params, a.N, a.bias, a.Y);
  return hipGetLastError();
}

// P tiles of channels per wave, so that one round of workgroups covers N with
// one on every CU: X is read once per workgroup, from the L2, and that is what
// small P costs; large P leaves CUs idle (1 x 8192 x 28672: 24.5 us with 7 and
// 256 workgroups, 26.9 with 4, 34.3 with 1, 16 rows 26.4 and 70.2 with 1; 1 x
// 11008 x 4096: 8.1 us with 1, 15.1 with 4).  Where that would be 6, 7 are taken:
// an instance with 6 would take 20.2 us for 1 x 8192 x 22000, this one 21.3.
template <bool BF16, bool ZEROS, int GS>
hipError_t pick_few(const Int4Args& a, hipStream_t s) {
  const int P = ((a.N + 15) / 16 + kCus - 1) / kCus;
  if (P <= 1) return run_few<BF16, ZEROS, GS, 1>(a, s);
  if (P == 2) return run_few<BF16, ZEROS, GS, 2>(a, s);
  if (P == 3) return run_few<BF16, ZEROS, GS, 3>(a, s);
  if constexpr (GS > 1) {  // 32-wide groups: no registers for more than 4
    if (P == 5) return run_few<BF16, ZEROS, GS, 5>(a, s);
    if (P > 5) return run_few<BF16, ZEROS, GS, 7>(a, s);
  }
  return run_few<BF16, ZEROS, GS, 4>(a, s);
}

template <bool BF16, bool ZEROS, int GS, int MT, int P, int KS>
hipError_t run_many(const Int4Args& a, hipStream_t s) {
  const int z = int4_k_parts(a.M, a.K, a.N);
  const dim3 grid((a.N + 64 * P - 1) / (64 * P), (a.M + 16 * MT - 1) / (16 * MT), z);
  const int vec = a.K % 8 == 0 && (a.ldx % 8 == 0 || a.M == 1) && (reinterpret_cast<uintptr_t>(a.X) & 15) == 0;
  hipLaunchKernelGGL((k_int4_many<BF16, ZEROS, GS, MT, P, KS>), grid, dim3(256 * KS), 0, s, a.X,
                     a.M, a.K, a.ldx, vec, a.Wq, a.params, a.N, a.bias, a.Y,
                     z > 1 ? a.part : nullptr);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || z == 1) return e;
  const int64_t total = (int64_t)a.M * a.N;
  hipLaunchKernelGGL((k_int4_sum<BF16>), dim3(grid_for(total, 256)), dim3(256), 0, s, a.part, z,
                     total, a.N, a.bias, a.Y);
  return hipGetLastError();
}

// One channel tile a wave as long as one round of workgroups covers Y (64 x
// 4096 x 11008: 18.5 us, 25.5 with two; 48 x 5120 x 13811 in groups of 32: 22.3
// and 33), else two, which also halve the reads of X (64 x 4096 x 20000: 27.7
// us, 35 with one; 64 x 8192 x 28672: 51 and 63; 1000 x 4096 x 11008: 155 and
// 186).  bfloat16's 64 rows in groups of 32 have no registers for it (64 x 8192
// x 28672: 186 us spilling, 95 with one).
//
// Four tiles of K a step, 16 waves, where their 128 registers do (with two and 8
// waves, whose LDS reads, codes and matrix instructions hide one another less,
// 48 x 5120 x 13811 in groups of 32 takes 25.5 us instead of 23.2, 64 x 4096 x
// 16000 21 instead of 20, 20 x 3333 x 5000 32.2 instead of 24.7; up to K = 1024
// the two are within 2%), otherwise two and 8 waves (64 x 4096 x 11008 bfloat16
// in groups of 32: 27 us, 121 spilling with 16).
template <bool BF16, bool ZEROS, int GS, int MT>
hipError_t pick_many(const Int4Args& a, hipStream_t s) {
  if constexpr (MT > 1 && !(BF16 && GS == 1 && MT == 4))
    if ((int64_t)((a.N + 63) / 64) * ((a.M + 63) / 64) > kCus)
      return run_many<BF16, ZEROS, GS, MT, 2, 2>(a, s);
  constexpr bool wide = BF16 ? MT <= 2 || (MT == 3 && GS == 4) : MT <= 3 || GS > 1;
  return run_many<BF16, ZEROS, GS, MT, 1, wide ? 4 : 2>(a, s);
}

template <bool BF16, bool ZEROS, int GS>
hipError_t pick(const Int4Args& a, bool few, hipStream_t s) {
  if (few) return pick_few<BF16, ZEROS, GS>(a, s);
  if (a.M <= 16) return pick_many<BF16, ZEROS, GS, 1>(a, s);
  if (a.M <= 32) return pick_many<BF16, ZEROS, GS, 2>(a, s);
  if (a.M <= 48) return pick_many<BF16, ZEROS, GS, 3>(a, s);
  return pick_many<BF16, ZEROS, GS, 4>(a, s);
}

template <bool BF16, bool ZEROS>
hipError_t pick_group(const Int4Args& a, int steps, bool few, hipStream_t s) {
  switch (steps) {
    case 1: return pick<BF16, ZEROS, 1>(a, few, s);
    case 2: return pick<BF16, ZEROS, 2>(a, few, s);
    default: return pick<BF16, ZEROS, 4>(a, few, s);
  }
}

}  // namespace

bool int4_few_rows(const uint16_t* X, int64_t M, int64_t K, int64_t ldx) {
  return M <= 16 && K % 8 == 0 && (ldx % 8 == 0 || M == 1) && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
}

// Parts of K of the kernel for many rows: up to one round of workgroups, of at
// least 20 tiles for up to 32 rows, 14 for 48 and 10 for 64, whose tiles take
// longer.  Microseconds, the part count that this gives first:
//   24 x 4096 x 4096   1: 10.8, 3: 12.2     24 x 11008 x 4096  4: 14, 2: 17.6, 1: 25.3
//   48 x 2048 x 4096   1: 8.4, 2: 11.6      48 x 4096 x 4096   2: 12.2, 1: 14.4, 4: 12
//   48 x 8192 x 1024   4: 12, 2: 16.4, 1: 23.9, 9: 11.7
//   64 x 2048 x 2048   1: 9.7, 3: 11.7      60 x 8192 x 1024   6: 13, 3: 16.2, 1: 28.3, 12: 13.9
//   60 x 4096 x 4096 in groups of 32        3: 14.7, 1: 21, 4: 13.4
int int4_k_parts(int64_t M, int64_t K, int64_t N) {
  const int64_t groups = ((N + 63) / 64) * ((M + 63) / 64);
  const int64_t row_tiles = M <= 32 ? 2 : M <= 48 ? 3 : 4;
  const int64_t most = int4_tiles_k(K) * row_tiles / 40;
  int64_t z = groups > 0 ? kCus / groups : 1;
  if (z > most) z = most;
  return (int)(z < 1 ? 1 : z);
}

hipError_t launch_int4_linear(const Int4Args& a, bool bf16, int64_t group, bool zeros,
                              hipStream_t s) {
  if (a.K == 0) {
    const int64_t total = (int64_t)a.M * a.N;
    hipLaunchKernelGGL(k_int4_bias, dim3(grid_for(total, 256)), dim3(256), 0, s, a.bias, total, a.N,
                       a.Y);
    return hipGetLastError();
  }
  const int steps = int4_group_steps(group);
  const bool few = int4_few_rows(a.X, a.M, a.K, a.ldx);
  if (bf16)
    return zeros ? pick_group<true, true>(a, steps, few, s) : pick_group<true, false>(a, steps, few, s);
  return zeros ? pick_group<false, true>(a, steps, few, s) : pick_group<false, false>(a, steps, few, s);
}

}  // namespace i8mm
