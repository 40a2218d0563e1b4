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
// bfloat16 rows: 128 + q, and the constant comes off the group's sum, as z
// does in both types: sum x (c + q) - (c + z) sum x, with sum x from one more
// MFMA against ones.  Products of the codes are exact and sums are fp32; the
// group's scale multiplies the fp32 sum, so nothing is rounded before Y.
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

// Waves that share one group of tiles: as many as the registers and 64 KiB
// for their sums allow.
constexpr int max_waves(int P, int MT) { return P * MT == 1 ? 16 : P * MT <= 8 ? 8 : 4; }

// One workgroup: P tiles of 16 channels, up to 16*MT rows, its waves splitting
// K tile by tile.  GS: 32-k steps per parameter entry.
// ARR: X is in operand order (see k_int4_arrange); otherwise rows of X, 16-byte
// aligned and K a multiple of 8 (one tile of rows only).
//
// X is the A operand and W the B operand, so that a lane's codes and its sums
// belong to the same channel (lane % 16) and one parameter entry serves both.
template <bool BF16, bool ZEROS, int GS, int P, int MT, bool ARR>
__global__ __launch_bounds__(64 * max_waves(P, MT)) void k_int4_linear(
    const uint16_t* __restrict__ X, int M, int K, int64_t ldx, const uint8_t* __restrict__ Wq,
    const uint16_t* __restrict__ params, int N, const uint16_t* __restrict__ bias,
    uint16_t* __restrict__ Y) {
  constexpr int NG = 4 / GS;  // parameter entries per tile and channel
  constexpr int PB = NG * (ZEROS ? 4 : 2);  // their bytes
  using Par = typename std::conditional<PB == 16, v4u, typename std::conditional<PB == 8, v2u,
              typename std::conditional<PB == 4, uint32_t, uint16_t>::type>::type>::type;
  extern __shared__ float red[];  // [waves][P][MT][4][64]

  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, qd = lane >> 4;
  const int nt = (K + kInt4TileK - 1) / kInt4TileK;
  const int panel0 = blockIdx.x * P;
  const int m0 = blockIdx.y * (16 * MT);
  const int rows = min(M - m0, 16 * MT);

  const uint16_t* xp = ARR ? X + (int64_t)blockIdx.y * nt * (MT * 4 * 512)
                           : X;
  const int64_t xl = ARR ? lane * 8 : (int64_t)min(r, rows - 1) * ldx + qd * 8;
  // the last workgroup may have fewer than P tiles of channels: it takes the
  // last one again, and does not store it
  const int panels = (N + 15) / 16;
  int64_t first[P];
#pragma unroll
  for (int p = 0; p < P; ++p) first[p] = (int64_t)min(panel0 + p, panels - 1) * nt;
  const uint8_t* pp = reinterpret_cast<const uint8_t*>(params);

  const Nibbles nib = nibbles<BF16>();

  v4u w[2][P], x[MT][4];
  Par par[2][P];
  auto load_w = [&](int st, int t) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t tile = first[p] + t;
      w[st][p] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(Wq + tile * kInt4TileBytes) + lane);
      par[st][p] = reinterpret_cast<const Par*>(pp + tile * (16 * PB))[r];
    }
  };
  auto load_x = [&](int t, int m, int s) __attribute__((always_inline)) {
    x[m][s] = *reinterpret_cast<const v4u*>(
        xp + (ARR ? (((int64_t)t * MT + m) * 4 + s) * 512 : (int64_t)t * kInt4TileK + s * 32) + xl);
  };
  // 16-bit word i of the entries (a scale, and with zero points 1024 + z), twice
  auto word2 = [](const Par& e, int i) __attribute__((always_inline)) {
    uint32_t u;
    if constexpr (PB <= 4)
      u = e;
    else
      u = e[i >> 1];
    return __builtin_amdgcn_perm(u, u, (i & 1) ? 0x03020302u : 0x01000100u);
  };

  v4f tot[P][MT];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int m = 0; m < MT; ++m) tot[p][m] = v4f{0, 0, 0, 0};

  // tile of stage st; a step's X registers take tile tn's as soon as the step
  // is done (tn < 0: none)
  auto compute = [&](int st, int tn) __attribute__((always_inline)) {
    constexpr uint32_t one = 0x3f803f80u;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
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
        if constexpr (BF16)
#pragma unroll
          for (int m = 0; m < MT; ++m) sx[m] = mfma32<true>(x[m][s], v4u{one, one, one, one}, sx[m]);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const uint32_t z = ZEROS && !BF16 ? word2(par[st][p], 2 * g + 1) : 0x64086408u;
          const v4u b = codes8<BF16>(w[st][p][s], z, nib);
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[p][m] = mfma32<BF16>(x[m][s], b, acc[p][m]);
        }
        if (tn >= 0)
#pragma unroll
          for (int m = 0; m < MT; ++m) load_x(tn, m, s);
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float sc = h2f((uint16_t)word2(par[st][p], ZEROS ? 2 * g : g));
        const float off = ZEROS ? h2f((uint16_t)word2(par[st][p], 2 * g + 1)) - 896.0f : 136.0f;  // 128 + z
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

  // whole tiles: while one is multiplied, the next one's loads are in flight
  const int whole = ARR ? nt : K / kInt4TileK;
  const int last = whole - 1;
  if (wave < whole) {
    load_w(0, wave);
    load_w(1, min(wave + waves, last));
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 0; s < 4; ++s) load_x(wave, m, s);
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
  if (!ARR && whole < nt && wave == whole % waves) {
    load_w(0, whole);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      x[0][s] = v4u{0, 0, 0, 0};
      if (whole * kInt4TileK + s * 32 + qd * 8 < K) load_x(whole, 0, s);
    }
    compute(0, -1);
  }

  // the waves' partial sums, added in wave order
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[(((wave * P + p) * MT + m) * 4 + i) * 64 + lane] = tot[p][m][i];
  __syncthreads();
  for (int o = threadIdx.x; o < rows * 16 * P; o += blockDim.x) {
    const int nl = o % (16 * P), m = o / (16 * P);
    const int n = panel0 * 16 + nl;
    if (n >= N) continue;
    const int at = (((nl >> 4) * MT + (m >> 4)) * 4 + (m & 3)) * 64 + ((m & 15) >> 2) * 16 + (nl & 15);
    float y = 0.0f;
    for (int w = 0; w < waves; ++w) y += red[w * P * MT * 256 + at];
    if (bias != nullptr) y += BF16 ? bf2f(bias[n]) : h2f(bias[n]);
    Y[(int64_t)(m0 + m) * N + n] = BF16 ? f2bf(y) : f2h(y);
  }
}

// X in operand order: per 64 rows (16 * MT), k tile, 16 rows and 32 k the 64
// lanes' 8 elements (lane l: row l % 16, k 8 * (l / 16) ..), zeros past M and K.
// One KiB a load then comes from one place.  Rows of a usual X lie a power of
// two apart, 16 of them in one channel of the L2, and every workgroup reads
// them: 64 x 8192 x 13824 took 50.7 us from the rows, 26.4 us in this order.
__global__ __launch_bounds__(256) void k_int4_arrange(const uint16_t* __restrict__ X, int M, int K,
                                                      int64_t ldx, int MT, int64_t nt, int vec,
                                                      int64_t total, uint16_t* __restrict__ A) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int l = (int)(i & 63), s = (int)(i >> 6) & 3;
    const int64_t f = i >> 8;  // (chunk, tile, 16 rows)
    const int m = (int)(f % MT);
    const int64_t t = f / MT % nt, chunk = f / MT / nt;
    const int64_t row = chunk * 16 * MT + m * 16 + (l & 15);
    const int64_t k = t * kInt4TileK + s * 32 + (l >> 4) * 8;
    v4u x = {0, 0, 0, 0};
    if (row < M) {
      const uint16_t* p = X + row * ldx + k;
      if (vec && k + 8 <= K) {
        x = *reinterpret_cast<const v4u*>(p);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a = k + 2 * e < K ? p[2 * e] : 0u;
          const uint32_t b = k + 2 * e + 1 < K ? p[2 * e + 1] : 0u;
          x[e] = a | (b << 16);
        }
      }
    }
    *reinterpret_cast<v4u*>(A + i * 8) = x;
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
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= Np * groups) return;
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
  const dim3 grid((unsigned)((waves + 3) / 4));
  if (bf16)
    hipLaunchKernelGGL(k_int4_prepare<true>, grid, dim3(256), 0, s, W, N, K, Np, group, gs, nt,
                       zeros, Wq, params);
  else
    hipLaunchKernelGGL(k_int4_prepare<false>, grid, dim3(256), 0, s, W, N, K, Np, group, gs, nt,
                       zeros, Wq, params);
  return hipGetLastError();
}

namespace {

template <bool BF16, bool ZEROS, int GS, int P, int MT, bool ARR>
hipError_t run(const uint16_t* X, int M, int K, int64_t ldx, const void* Wq, const void* params,
               int N, const uint16_t* bias, uint16_t* Y, hipStream_t s) {
  const int nt = (int)int4_tiles_k(K);
  int waves = max_waves(P, MT);
  while (waves > nt) waves /= 2;
  const dim3 grid((unsigned)((N + 16 * P - 1) / (16 * P)), (unsigned)((M + 16 * MT - 1) / (16 * MT)));
  const size_t lds = (size_t)waves * P * MT * 1024;
  hipLaunchKernelGGL((k_int4_linear<BF16, ZEROS, GS, P, MT, ARR>), grid, dim3(64 * waves), lds, s, X, M,
                     K, ldx, static_cast<const uint8_t*>(Wq), static_cast<const uint16_t*>(params),
                     N, bias, Y);
  return hipGetLastError();
}

// P tiles of channels per wave, so that one round of workgroups covers N with
// one on every CU: X is read once per workgroup, from the L2, and that is what
// small P costs; large P leaves CUs idle (1 x 8192 x 28672: 23.5 us with 7 and
// 256 workgroups, 27.3 with 4, 32 with 1; 1 x 11008 x 4096: 9.7 us with 1, 17.1
// with 4).
template <bool BF16, bool ZEROS, int GS>
hipError_t pick_tile(const uint16_t* X, bool arranged, int M, int K, int64_t ldx, const void* Wq,
                     const void* params, int N, const uint16_t* bias, uint16_t* Y, hipStream_t s) {
#define INT4_RUN(p, m, a) return run<BF16, ZEROS, GS, p, m, a>(X, M, K, ldx, Wq, params, N, bias, Y, s)
  const int panels = (N + 15) / 16;
  const int P = (panels + kCus - 1) / kCus;
  if (!arranged) {
    if (P <= 1) INT4_RUN(1, 1, false);
    if (P == 2) INT4_RUN(2, 1, false);
    if (P == 3) INT4_RUN(3, 1, false);
    if constexpr (GS > 1) {  // 32-wide groups: no registers for more than 4
      if (P == 5) INT4_RUN(5, 1, false);
      if (P > 5) INT4_RUN(7, 1, false);
    }
    INT4_RUN(4, 1, false);
  }
  const int mt = int4_row_tiles(M);
  if (mt == 1 && P <= 2) INT4_RUN(1, 1, true);
  if (mt == 1) INT4_RUN(4, 1, true);
  if (P <= 1 && mt == 2) INT4_RUN(1, 2, true);
  if (P <= 1 && mt == 3) INT4_RUN(1, 3, true);
  if (P <= 1) INT4_RUN(1, 4, true);
  if (P == 2 || GS == 1) {
    if (mt == 2) INT4_RUN(2, 2, true);
    if (mt == 3) INT4_RUN(2, 3, true);
    INT4_RUN(2, 4, true);
  }
  if constexpr (GS > 1) {
    if (mt == 2) INT4_RUN(4, 2, true);
    if (mt == 3) INT4_RUN(4, 3, true);
    INT4_RUN(4, 4, true);
  }
  return hipErrorInvalidValue;  // not reached
#undef INT4_RUN
}

template <bool BF16, bool ZEROS>
hipError_t pick_group(const uint16_t* X, bool arranged, int M, int K, int64_t ldx, const void* Wq,
                      const void* params, int N, int steps, const uint16_t* bias, uint16_t* Y,
                      hipStream_t s) {
  switch (steps) {
    case 1: return pick_tile<BF16, ZEROS, 1>(X, arranged, M, K, ldx, Wq, params, N, bias, Y, s);
    case 2: return pick_tile<BF16, ZEROS, 2>(X, arranged, M, K, ldx, Wq, params, N, bias, Y, s);
    default: return pick_tile<BF16, ZEROS, 4>(X, arranged, M, K, ldx, Wq, params, N, bias, Y, s);
  }
}

}  // namespace

bool int4_x_direct(const uint16_t* X, int64_t M, int64_t K, int64_t ldx) {
  return M <= 16 && K % 8 == 0 && (ldx % 8 == 0 || M == 1) && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
}

size_t int4_arranged_bytes(int64_t M, int64_t K) {
  const int64_t per = 16 * int4_row_tiles(M);
  return (size_t)((M + per - 1) / per * per) * int4_tiles_k(K) * kInt4TileK * 2;
}

hipError_t launch_int4_linear(const uint16_t* X, bool bf16, int64_t M, int64_t K, int64_t ldx,
                              const void* Wq, const void* params, int64_t N, int64_t group,
                              bool zeros, const uint16_t* bias, uint16_t* Y, uint16_t* ws,
                              hipStream_t s) {
  if (K == 0) {
    hipLaunchKernelGGL(k_int4_bias, dim3(grid_for(M * N, 256)), dim3(256), 0, s, bias, M * N,
                       (int)N, Y);
    return hipGetLastError();
  }
  const bool arr = !int4_x_direct(X, M, K, ldx);
  if (arr) {
    const int64_t total = (int64_t)int4_arranged_bytes(M, K) / 16;
    const int vec = (ldx % 8 == 0 || M == 1) && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
    hipLaunchKernelGGL(k_int4_arrange, dim3(grid_for(total, 256)), dim3(256), 0, s, X, (int)M,
                       (int)K, ldx, int4_row_tiles(M), int4_tiles_k(K), vec, total, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    X = ws;
  }
  const int steps = int4_group_steps(group), m = (int)M, k = (int)K, n = (int)N;
  if (bf16)
    return zeros ? pick_group<true, true>(X, arr, m, k, ldx, Wq, params, n, steps, bias, Y, s)
                 : pick_group<true, false>(X, arr, m, k, ldx, Wq, params, n, steps, bias, Y, s);
  return zeros ? pick_group<false, true>(X, arr, m, k, ldx, Wq, params, n, steps, bias, Y, s)
               : pick_group<false, false>(X, arr, m, k, ldx, Wq, params, n, steps, bias, Y, s);
}

}  // namespace i8mm
