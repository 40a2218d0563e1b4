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

// The 8 codes of one dword as an MFMA operand: float16 q - 8, bfloat16 128 + q.
template <bool BF16>
__device__ __forceinline__ v4u codes8(uint32_t u) {
  if constexpr (BF16) {
    constexpr uint32_t m = 0x000f000fu, o = 0x43004300u;
    return v4u{(u & m) | o, ((u >> 4) & m) | o, ((u >> 8) & m) | o, ((u >> 12) & m) | o};
  } else {
    constexpr uint32_t lo = 0x000f000fu, hi = 0x00f000f0u, o = 0x64006400u;
    const uint32_t w = u >> 8;
    const v2h c1 = {(_Float16)1032.0f, (_Float16)1032.0f};
    const v2h c2 = {(_Float16)0.0625f, (_Float16)0.0625f};
    const v2h c3 = {(_Float16)-72.0f, (_Float16)-72.0f};
    auto plain = [&](uint32_t x) { return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, x) - c1); };
    auto wide = [&](uint32_t x) {
      return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(v2h, x), c2, c3));
    };
    return v4u{plain((u & lo) | o), wide((u & hi) | o), plain((w & lo) | o), wide((w & hi) | o)};
  }
}

// Waves that share one group of tiles: as many as its registers allow.
constexpr int max_waves(int P, int MT) { return P * MT == 1 ? 16 : MT <= 2 ? 8 : 4; }

// One workgroup: P tiles of 16 channels, up to 16*MT rows, its waves splitting
// K tile by tile.  GS: 32-k steps per parameter entry.
// X: rows 16-byte aligned, K a multiple of 8 (see k_int4_pad_x).
template <bool BF16, bool ZEROS, int GS, int P, int MT>
__global__ __launch_bounds__(64 * max_waves(P, MT)) void k_int4_linear(
    const uint16_t* __restrict__ X, int M, int K, int64_t ldx, const uint8_t* __restrict__ Wq,
    const uint16_t* __restrict__ params, int N, const uint16_t* __restrict__ bias,
    uint16_t* __restrict__ Y) {
  constexpr int NG = 4 / GS;             // parameter entries per tile and channel
  constexpr int EB = ZEROS ? 2 : 1;      // 16-bit words per entry
  constexpr bool CORR = BF16 || ZEROS;   // a constant comes off the sums
  constexpr float kOff = BF16 ? (ZEROS ? 128.0f : 136.0f) : -8.0f;
  extern __shared__ float red[];  // [waves][P][MT][4][64]

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int r = lane & 15, qd = lane >> 4;
  const int nt = (K + kInt4TileK - 1) / kInt4TileK;
  const int panel0 = blockIdx.x * P;
  const int m0 = blockIdx.y * (16 * MT);
  const int rows = min(M - m0, 16 * MT);

  const uint16_t* xrow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
    xrow[t] = X + (int64_t)(m0 + min(t * 16 + r, rows - 1)) * ldx;

  // this lane's 4 channels' entries: scales, or (scale, z) pairs
  using Par = typename std::conditional<ZEROS, v4u, v2u>::type;
  struct Tile {
    v4u w[P];
    v4u x[MT][4];
    Par par[P][NG];
  };
  auto load = [&](Tile& d, int t) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t tile = (int64_t)(panel0 + p) * nt + t;
      d.w[p] = __builtin_nontemporal_load(
          reinterpret_cast<const v4u*>(Wq + tile * kInt4TileBytes + lane * 16));
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        d.par[p][g] = *reinterpret_cast<const Par*>(params + ((tile * NG + g) * 16 + 4 * qd) * EB);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int k = t * kInt4TileK + s * 32 + qd * 8;
        d.x[m][s] = v4u{0, 0, 0, 0};
        if (k < K) d.x[m][s] = *reinterpret_cast<const v4u*>(xrow[m] + k);
      }
  };

  v4f tot[P][MT];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int m = 0; m < MT; ++m) tot[p][m] = v4f{0, 0, 0, 0};

  auto compute = [&](const Tile& d) __attribute__((always_inline)) {
    constexpr uint32_t one = BF16 ? 0x3f803f80u : 0x3c003c00u;
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
        if constexpr (CORR)
#pragma unroll
          for (int m = 0; m < MT; ++m) sx[m] = mfma32<BF16>(v4u{one, one, one, one}, d.x[m][s], sx[m]);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const v4u a = codes8<BF16>(d.w[p][s]);
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[p][m] = mfma32<BF16>(a, d.x[m][s], acc[p][m]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Par& e = d.par[p][g];
          const uint32_t u = ZEROS ? e[i] : e[i / 2] >> (16 * (i & 1));
          const float sc = h2f((uint16_t)u);
          float off = kOff;
          if constexpr (ZEROS) off += h2f((uint16_t)(u >> 16));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float a = acc[p][m][i];
            if constexpr (CORR) a = __builtin_fmaf(-off, sx[m][i], a);
            tot[p][m][i] = __builtin_fmaf(sc, a, tot[p][m][i]);
          }
        }
    }
  };

  // the next tile's loads are in flight while one is multiplied
  if (wave < nt) {
    Tile d[2];
    load(d[0], wave);
    int t = wave;
    for (; t + waves < nt; t += 2 * waves) {
      load(d[1], t + waves);
      compute(d[0]);
      if (t + 2 * waves < nt) load(d[0], t + 2 * waves);
      compute(d[1]);
    }
    if (t < nt) compute(d[0]);
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
    const int at = (((nl >> 4) * MT + (m >> 4)) * 4 + (nl & 3)) * 64 + ((nl & 15) >> 2) * 16 + (m & 15);
    float y = 0.0f;
    for (int w = 0; w < waves; ++w) y += red[w * P * MT * 256 + at];
    if (bias != nullptr) y += BF16 ? bf2f(bias[n]) : h2f(bias[n]);
    Y[(int64_t)(m0 + m) * N + n] = BF16 ? f2bf(y) : f2h(y);
  }
}

// Rows of X that are not 16-byte aligned or not a multiple of 8 long, copied
// to rows of K rounded up to 8 with zeros behind.
__global__ __launch_bounds__(256) void k_int4_pad_x(const uint16_t* __restrict__ X, int M, int K,
                                                    int64_t ldx, int Kp, uint16_t* __restrict__ P) {
  const int oct = Kp / 8;
  const int64_t total = (int64_t)M * oct;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t m = i / oct;
    const int k = (int)(i % oct) * 8;
    const uint16_t* row = X + m * ldx;
    v4u x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t a = k + 2 * e < K ? row[k + 2 * e] : 0u;
      const uint32_t b = k + 2 * e + 1 < K ? row[k + 2 * e + 1] : 0u;
      x[e] = a | (b << 16);
    }
    *reinterpret_cast<v4u*>(P + i * 8) = x;
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

// Parameter entries; i counts them in stored order [panel][tile][sub-group][channel].
__global__ void k_int4_params(const uint16_t* __restrict__ scales, const uint8_t* __restrict__ zeros,
                              int64_t N, int64_t K, int64_t group, int gs, int64_t nt,
                              int64_t total, uint16_t* __restrict__ params) {
  const int ng = kInt4TileK / gs;
  const int64_t groups = (K + group - 1) / group;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t e = i >> 4, tile = e / ng;
    const int64_t n = (tile / nt) * 16 + (i & 15);
    const int64_t k = (tile % nt) * kInt4TileK + (e % ng) * gs;
    const bool in = n < N && k < K;
    const int64_t at = in ? n * groups + k / group : 0;
    const uint16_t sc = in ? scales[at] : (uint16_t)0;
    if (zeros != nullptr) {
      params[2 * i] = sc;
      params[2 * i + 1] = f2h(in ? (float)(zeros[at] & 15) : 8.0f);
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
    const int64_t e = (tile * ng + (k & 127) / gs) * 16 + (n & 15);
    const bool in = n < N && k < K;
    if (zeros) {
      params[2 * e] = in ? sc : (uint16_t)0;
      params[2 * e + 1] = f2h(in ? z : 8.0f);
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

template <bool BF16, bool ZEROS, int GS, int P, int MT>
hipError_t run(const uint16_t* X, int M, int K, int64_t ldx, const void* Wq, const void* params,
               int N, const uint16_t* bias, uint16_t* Y, hipStream_t s) {
  const int nt = (int)int4_tiles_k(K);
  int waves = max_waves(P, MT);
  while (waves > nt) waves /= 2;
  const dim3 grid((unsigned)((N + 16 * P - 1) / (16 * P)), (unsigned)((M + 16 * MT - 1) / (16 * MT)));
  const size_t lds = (size_t)waves * P * MT * 1024;
  hipLaunchKernelGGL((k_int4_linear<BF16, ZEROS, GS, P, MT>), grid, dim3(64 * waves), lds, s, X, M,
                     K, ldx, static_cast<const uint8_t*>(Wq), static_cast<const uint16_t*>(params),
                     N, bias, Y);
  return hipGetLastError();
}

template <bool BF16, bool ZEROS, int GS>
hipError_t pick_tile(const uint16_t* X, int M, int K, int64_t ldx, const void* Wq,
                     const void* params, int N, const uint16_t* bias, uint16_t* Y, hipStream_t s) {
  constexpr int kWide = GS == 1 ? 2 : 4;  // tiles of channels a wave takes at once
  constexpr int kRows = GS == 1 ? 1 : 2;
  if (M <= 16 && N < 16384) return run<BF16, ZEROS, GS, 1, 1>(X, M, K, ldx, Wq, params, N, bias, Y, s);
  if (M <= 16) return run<BF16, ZEROS, GS, kWide, 1>(X, M, K, ldx, Wq, params, N, bias, Y, s);
  if (M <= 32) return run<BF16, ZEROS, GS, kRows, 2>(X, M, K, ldx, Wq, params, N, bias, Y, s);
  return run<BF16, ZEROS, GS, kRows, 4>(X, M, K, ldx, Wq, params, N, bias, Y, s);
}

template <bool BF16, bool ZEROS>
hipError_t pick_group(const uint16_t* X, int M, int K, int64_t ldx, const void* Wq,
                      const void* params, int N, int steps, const uint16_t* bias, uint16_t* Y,
                      hipStream_t s) {
  switch (steps) {
    case 1: return pick_tile<BF16, ZEROS, 1>(X, M, K, ldx, Wq, params, N, bias, Y, s);
    case 2: return pick_tile<BF16, ZEROS, 2>(X, M, K, ldx, Wq, params, N, bias, Y, s);
    default: return pick_tile<BF16, ZEROS, 4>(X, M, K, ldx, Wq, params, N, bias, Y, s);
  }
}

}  // namespace

bool int4_x_aligned(const uint16_t* X, int64_t M, int64_t K, int64_t ldx) {
  return K % 8 == 0 && (ldx % 8 == 0 || M == 1) && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
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
  if (!int4_x_aligned(X, M, K, ldx)) {
    const int Kp = (int)((K + 7) / 8 * 8);
    hipLaunchKernelGGL(k_int4_pad_x, dim3(grid_for(M * (Kp / 8), 256)), dim3(256), 0, s, X, (int)M,
                       (int)K, ldx, Kp, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    X = ws;
    K = ldx = Kp;
  }
  const int steps = int4_group_steps(group), m = (int)M, k = (int)K, n = (int)N;
  if (bf16)
    return zeros ? pick_group<true, true>(X, m, k, ldx, Wq, params, n, steps, bias, Y, s)
                 : pick_group<true, false>(X, m, k, ldx, Wq, params, n, steps, bias, Y, s);
  return zeros ? pick_group<false, true>(X, m, k, ldx, Wq, params, n, steps, bias, Y, s)
               : pick_group<false, false>(X, m, k, ldx, Wq, params, n, steps, bias, Y, s);
}

}  // namespace i8mm
