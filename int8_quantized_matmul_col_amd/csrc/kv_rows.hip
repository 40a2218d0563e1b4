// Writing tokens' keys and values into the pages of a key-value cache, and
// reading them back as rows.
//
// Bound by HBM for a prompt (each element read and written once; 16000 tokens
// of 8 x 128 dims to an int8 cache and back 51 us, 3.9 TB/s) and by the launch
// for the tokens of one decode step (4.2 us on the GPU for 64, 5.8 into an int8
// cache).  A workgroup takes up to 32 tokens of one kv head.  Keys are rows on
// both sides.  Values are rows on one side and [dim][token] in the page, so they
// turn in LDS; wherever 8 tokens of the workgroup lie side by side in a page (a
// prompt) they are one 16-byte (int8: 8-byte) access, otherwise (a decode step)
// each token's element is its own.
//
// An int8 cache: a = max |x| over the token's dims of the head, code =
// clamp(rne(127 x / a), -127, 127), the quantizer of the int8 matmul.
#include "device_common.h"
#include "serving_launch.h"

namespace i8mm {

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kTok = kKvRowsTokens;  // per workgroup
// Threads where a row has LN lanes: one pass up to 128 dims, two beyond (with
// 256 threads 4000 int8 tokens of 8 x 256 dims take 32.7 us both ways, 30.2 so).
constexpr int threads_of(int LN) { return kTok * LN < kKvRowsThreads ? kTok * LN : kKvRowsThreads; }
constexpr int kMaxD = INT8MM_KV_MAX_HEAD_DIM;

struct Rows {
  int8mm_kv kv;
  const int32_t* table;
  const int32_t* rows;
  const int32_t* positions;
  int table_rows, table_width, T, lps;
};

// Page and slot of token i as page * page_size + slot; -1 where there is none.
__device__ __forceinline__ int64_t place(const Rows& a, int i) {
  if (i >= a.T) return -1;
  const int row = a.rows[i], pos = a.positions[i];
  if ((unsigned)row >= (unsigned)a.table_rows || pos < 0) return -1;
  const int at = pos >> a.lps;
  if (at >= a.table_width) return -1;
  const int page = a.table[(int64_t)row * a.table_width + at];
  if ((unsigned)page >= (unsigned)a.kv.num_pages) return -1;
  return ((int64_t)page << a.lps) + (pos & (a.kv.page_size - 1));
}

// Bit j: the places 8j .. 8j+7 of the workgroup's kTok are consecutive slots of
// one page, the first at a multiple of 8 (and so an aligned access).  Called
// by every thread, with the places in LDS; each wave finds it for itself.
__device__ __forceinline__ uint32_t runs_of_8(const int64_t* p) {
  const int lane = threadIdx.x & 63, i = lane % kTok;
  const int64_t base = p[i & ~7];
  const bool ok = p[i] == base + (i & 7) && base >= 0 && (base & 7) == 0;
  const uint64_t all = __ballot(ok);
  uint32_t runs = 0;
#pragma unroll
  for (int j = 0; j < kTok / 8; ++j) runs |= ((all >> (8 * j)) & 0xff) == 0xff ? 1u << j : 0u;
  return runs;
}

// A store that leaves the L2 at once instead of at the kernel's end (a prompt's
// pages: 12.6 -> 11.8 us for 4000 tokens of 8 heads; the gathered rows, which
// are read next, are better left there).
template <typename V, typename T>
__device__ __forceinline__ void store(T* p, V x) {
  __builtin_nontemporal_store(x, reinterpret_cast<V*>(p));
}

template <bool BF16>
__device__ __forceinline__ float value(uint32_t bits) {
  return BF16 ? __uint_as_float(bits << 16) : h2f((uint16_t)bits);
}
template <bool BF16>
__device__ __forceinline__ uint32_t bits_of(float f) {
  return BF16 ? __builtin_bit_cast(uint16_t, (__bf16)f) : f2h(f);
}
__device__ __forceinline__ uint32_t half_of(const v4u& x, int e) {
  return (x[e >> 1] >> (16 * (e & 1))) & 0xffffu;
}

// Largest magnitude of a group of LN lanes' 8-element chunks, as fp32.  The
// bit patterns of magnitudes order like the values, NaN above all.
template <bool BF16, int LN>
__device__ __forceinline__ float group_absmax(const v4u& x) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t a = half_of(x, e) & 0x7fffu;
    m = a > m ? a : m;
  }
#pragma unroll
  for (int o = LN / 2; o > 0; o >>= 1) {
    const uint32_t w = __shfl_xor(m, o, 64);
    m = w > m ? w : m;
  }
  return value<BF16>(m);
}

// Codes of 8 values of scale a: r = 127/a and one fma a value where the result
// is provably the same (see quant8_fast, whose bound holds for any two
// floats), the division where a value lies near a tie or 127/a is no finite
// number (a below 2^-121, infinite or NaN).  The division forms 127 x, which
// passes fp32's range for large bfloat16 numbers: there x and a are both taken
// 2^-8 smaller, which leaves the quotient as it is (a branch of its own: 4000
// tokens of 8 x 128 dims 12.45 us, 12.65 with the factor in every division,
// 12.2 without).
template <bool BF16>
__device__ __forceinline__ v2u quantize(const v4u& x, float a) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23
  const float r = a > 0.0f ? 127.0f / a : 0.0f;
  int q[8];
  float dev = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float v = value<BF16>(half_of(x, e));
    const float s = __builtin_fmaf(v, r, kRound);
    dev = fmaxf(dev, fabsf(__builtin_fmaf(v, r, -(s - kRound))));
    q[e] = (int)__float_as_uint(s);  // low byte: the code
  }
  // (asked of the wave: the compiler would otherwise divide always and select)
  if (__any(dev > kTieGuard || !(r <= 3.0e38f) || (r == 0.0f && a > 0.0f))) {
    if (BF16 && __any(a > 0x1p120f)) {
      const float f = a > 0x1p120f ? 0x1p-8f : 1.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = quant_code(f * value<BF16>(half_of(x, e)), f * a);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = quant_code(value<BF16>(half_of(x, e)), a);
    }
  }
  const uint2 p = pack8_i8(q);
  return v2u{p.x, p.y};
}

// LN lanes hold one token's row, 8 elements each.
template <bool BF16, bool I8, int LN>
__global__ __launch_bounds__(threads_of(LN)) void k_kv_append(
    const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int64_t kts, int64_t khs,
    int64_t vts, int64_t vhs, int vec, Rows a) {
  constexpr int kThreads = threads_of(LN);
  constexpr int EB = I8 ? 1 : 2;
  constexpr int kLd = kMaxD * EB + 4;  // bytes of an LDS row: odd in dwords
  __shared__ int64_t at[kTok];
  __shared__ __attribute__((aligned(16))) uint8_t turn[kTok * kLd];
  constexpr int kPass = kTok * LN / kThreads;
  const int h = blockIdx.y, i0 = blockIdx.x * kTok;
  const int D = a.kv.head_dim, ps = a.kv.page_size;
  const int c = threadIdx.x % LN;  // chunk of 8 dims
  // the rows are requested before their places are looked up
  v4u xks[kPass], xvs[kPass];
#pragma unroll
  for (int w = 0; w < kPass; ++w) {
    const int i = threadIdx.x / LN + w * (kThreads / LN);
    v4u xk = {0, 0, 0, 0}, xv = {0, 0, 0, 0};
    if (i0 + i < a.T && c * 8 < D) {
      const uint16_t* sk = k + (int64_t)(i0 + i) * kts + h * khs + c * 8;
      const uint16_t* sv = v + (int64_t)(i0 + i) * vts + h * vhs + c * 8;
      if (vec) {
        xk = *reinterpret_cast<const v4u*>(sk);
        xv = *reinterpret_cast<const v4u*>(sv);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xk[e] = sk[2 * e] | ((uint32_t)sk[2 * e + 1] << 16);
          xv[e] = sv[2 * e] | ((uint32_t)sv[2 * e + 1] << 16);
        }
      }
    }
    xks[w] = xk;
    xvs[w] = xv;
  }
  if (threadIdx.x < kTok) at[threadIdx.x] = place(a, i0 + threadIdx.x);
  __syncthreads();

#pragma unroll
  for (int w = 0; w < kPass; ++w) {
    const int i = threadIdx.x / LN + w * (kThreads / LN);
    const int64_t p = at[i];
    const bool on = p >= 0 && c * 8 < D;  // the same for a token's lanes, but for idle ones
    const v4u xk = xks[w], xv = xvs[w];
    const int64_t page = p >> a.lps;
    const int slot = (int)(p & (ps - 1));
    uint32_t* lv = reinterpret_cast<uint32_t*>(turn + i * kLd + c * 8 * EB);
    if constexpr (I8) {
      const float ak = group_absmax<BF16, LN>(xk), av = group_absmax<BF16, LN>(xv);
      if (!on) continue;
      store(static_cast<int8_t*>(a.kv.k) + page * a.kv.k_page_stride +
            ((int64_t)h * ps + slot) * D + c * 8, quantize<BF16>(xk, ak));
      const v2u q = quantize<BF16>(xv, av);
      lv[0] = q[0];
      lv[1] = q[1];
      if (c == 0) {
        a.kv.k_scale[page * a.kv.ks_page_stride + h * ps + slot] = ak;
        a.kv.v_scale[page * a.kv.vs_page_stride + h * ps + slot] = av;
      }
    } else {
      if (!on) continue;
      store(static_cast<uint16_t*>(a.kv.k) + page * a.kv.k_page_stride +
            ((int64_t)h * ps + slot) * D + c * 8, xk);
#pragma unroll
      for (int e = 0; e < 4; ++e) lv[e] = xv[e];
    }
  }
  __syncthreads();

  // values: 8 tokens of one dim per thread
  const uint32_t runs = runs_of_8(at);
  for (int w = threadIdx.x; w < D * (kTok / 8); w += kThreads) {
    const int o = w % (kTok / 8) * 8, d = w / (kTok / 8);
    uint32_t x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t* src = turn + (o + e) * kLd + d * EB;
      x[e] = I8 ? *src : *reinterpret_cast<const uint16_t*>(src);
    }
    const int64_t base = (int64_t)h * D * ps + (int64_t)d * ps;
    uint8_t* pool = static_cast<uint8_t*>(a.kv.v);
    if ((runs >> (o / 8)) & 1) {
      uint8_t* dst = pool + ((at[o] >> a.lps) * a.kv.v_page_stride + base + (at[o] & (ps - 1))) * EB;
      if constexpr (I8)
        store(dst, v2u{x[0] | x[1] << 8 | x[2] << 16 | x[3] << 24,
                       x[4] | x[5] << 8 | x[6] << 16 | x[7] << 24});
      else
        store(dst, v4u{x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16,
                       x[6] | x[7] << 16});
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t p = at[o + e];
        if (p < 0) continue;
        uint8_t* dst = pool + ((p >> a.lps) * a.kv.v_page_stride + base + (p & (ps - 1))) * EB;
        if constexpr (I8)
          *dst = (uint8_t)x[e];
        else
          *reinterpret_cast<uint16_t*>(dst) = (uint16_t)x[e];
      }
    }
  }
}

// code c of scale a as a rounded 16-bit number
template <bool BF16>
__device__ __forceinline__ uint32_t dequant(uint32_t byte, float a) {
  return bits_of<BF16>((float)(int8_t)byte * (a / 127.0f));
}

template <bool BF16, bool I8, int LN>
__global__ __launch_bounds__(threads_of(LN)) void k_kv_gather(uint16_t* __restrict__ k,
                                                              uint16_t* __restrict__ v, Rows a) {
  constexpr int kThreads = threads_of(LN);
  constexpr int EB = I8 ? 1 : 2;
  constexpr int kLd = kMaxD * EB + 4;
  __shared__ int64_t at[kTok];
  __shared__ __attribute__((aligned(16))) uint8_t turn[kTok * kLd];
  const int h = blockIdx.y, i0 = blockIdx.x * kTok, H = a.kv.kv_heads;
  const int D = a.kv.head_dim, ps = a.kv.page_size;
  if (threadIdx.x < kTok) at[threadIdx.x] = place(a, i0 + threadIdx.x);
  __syncthreads();

  // keys (and scales), requested before the values' turn
  constexpr int kPass = kTok * LN / kThreads;
  const int c = threadIdx.x % LN;
  v4u xks[kPass];
  float aks[kPass], avs[kPass];
#pragma unroll
  for (int w = 0; w < kPass; ++w) {
    const int64_t p = at[threadIdx.x / LN + w * (kThreads / LN)];
    xks[w] = v4u{0, 0, 0, 0};
    aks[w] = avs[w] = 0.0f;
    if (p < 0 || c * 8 >= D) continue;
    const int64_t page = p >> a.lps;
    const int slot = (int)(p & (ps - 1));
    const int64_t row = page * a.kv.k_page_stride + ((int64_t)h * ps + slot) * D + c * 8;
    if constexpr (I8) {
      aks[w] = a.kv.k_scale[page * a.kv.ks_page_stride + h * ps + slot];
      avs[w] = a.kv.v_scale[page * a.kv.vs_page_stride + h * ps + slot];
      const v2u q = *reinterpret_cast<const v2u*>(static_cast<const int8_t*>(a.kv.k) + row);
      xks[w][0] = q[0];
      xks[w][1] = q[1];
    } else {
      xks[w] = *reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(a.kv.k) + row);
    }
  }

  const uint32_t runs = runs_of_8(at);
  for (int w = threadIdx.x; w < D * (kTok / 8); w += kThreads) {
    const int o = w % (kTok / 8) * 8, d = w / (kTok / 8);
    const int64_t base = (int64_t)h * D * ps + (int64_t)d * ps;
    const uint8_t* pool = static_cast<const uint8_t*>(a.kv.v);
    uint32_t x[8];
    if ((runs >> (o / 8)) & 1) {
      const uint8_t* src = pool + ((at[o] >> a.lps) * a.kv.v_page_stride + base + (at[o] & (ps - 1))) * EB;
      if constexpr (I8) {
        const v2u y = *reinterpret_cast<const v2u*>(src);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (y[e >> 2] >> (8 * (e & 3))) & 0xffu;
      } else {
        const v4u y = *reinterpret_cast<const v4u*>(src);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = half_of(y, e);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t p = at[o + e];
        x[e] = 0;
        if (p < 0) continue;
        const uint8_t* src = pool + ((p >> a.lps) * a.kv.v_page_stride + base + (p & (ps - 1))) * EB;
        x[e] = I8 ? *src : *reinterpret_cast<const uint16_t*>(src);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint8_t* dst = turn + (o + e) * kLd + d * EB;
      if constexpr (I8)
        *dst = (uint8_t)x[e];
      else
        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)x[e];
    }
  }
  __syncthreads();

#pragma unroll
  for (int w = 0; w < kPass; ++w) {
    const int i = threadIdx.x / LN + w * (kThreads / LN);
    if (i0 + i >= a.T || c * 8 >= D) continue;
    v4u xk = xks[w], xv = {0, 0, 0, 0};
    if (at[i] >= 0) {
      const uint32_t* lv = reinterpret_cast<const uint32_t*>(turn + i * kLd + c * 8 * EB);
      if constexpr (I8) {
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          const int s = 16 * (e & 1);
          const uint32_t uk = xks[w][e >> 1] >> s, uv = lv[e >> 1] >> s;
          xk[e] = dequant<BF16>(uk, aks[w]) | dequant<BF16>(uk >> 8, aks[w]) << 16;
          xv[e] = dequant<BF16>(uv, avs[w]) | dequant<BF16>(uv >> 8, avs[w]) << 16;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) xv[e] = lv[e];
      }
    }
    const int64_t out = ((int64_t)(i0 + i) * H + h) * D + c * 8;
    *reinterpret_cast<v4u*>(k + out) = xk;
    *reinterpret_cast<v4u*>(v + out) = xv;
  }
}

Rows rows_of(const int8mm_kv& kv, const int32_t* table, int table_rows, int table_width,
             const int32_t* rows, const int32_t* positions, int T) {
  return Rows{kv, table, rows, positions, table_rows, table_width, T, __builtin_ctz(kv.page_size)};
}

// The row's lanes: the power of two that holds head_dim / 8 chunks.
template <template <int> class F, typename... A>
hipError_t by_lanes(int D, A... a) {
  if (D <= 64) return F<8>::go(a...);
  if (D <= 128) return F<16>::go(a...);
  return F<32>::go(a...);
}

template <bool BF16, bool I8>
struct Append {
  template <int LN>
  struct At {
    static hipError_t go(const uint16_t* k, const uint16_t* v, int64_t kts, int64_t khs,
                         int64_t vts, int64_t vhs, int vec, Rows a, hipStream_t s) {
      const dim3 grid((unsigned)((a.T + kTok - 1) / kTok), (unsigned)a.kv.kv_heads);
      hipLaunchKernelGGL((k_kv_append<BF16, I8, LN>), grid, dim3(threads_of(LN)), 0, s, k, v, kts, khs,
                         vts, vhs, vec, a);
      return hipGetLastError();
    }
  };
};

template <bool BF16, bool I8>
struct Gather {
  template <int LN>
  struct At {
    static hipError_t go(uint16_t* k, uint16_t* v, Rows a, hipStream_t s) {
      const dim3 grid((unsigned)((a.T + kTok - 1) / kTok), (unsigned)a.kv.kv_heads);
      hipLaunchKernelGGL((k_kv_gather<BF16, I8, LN>), grid, dim3(threads_of(LN)), 0, s, k, v, a);
      return hipGetLastError();
    }
  };
};

}  // namespace

hipError_t launch_kv_append(const uint16_t* k, const uint16_t* v, bool bf16, int T, int64_t kts,
                            int64_t khs, int64_t vts, int64_t vhs, const int8mm_kv& kv,
                            const int32_t* table, int table_rows, int table_width,
                            const int32_t* rows, const int32_t* positions, hipStream_t s) {
  const Rows a = rows_of(kv, table, table_rows, table_width, rows, positions, T);
  const int vec = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) == 0 &&
                  ((kts | khs | vts | vhs) & 7) == 0;
  const int D = kv.head_dim;
  if (kv.dtype == INT8MM_I8)
    return bf16 ? by_lanes<Append<true, true>::template At>(D, k, v, kts, khs, vts, vhs, vec, a, s)
                : by_lanes<Append<false, true>::template At>(D, k, v, kts, khs, vts, vhs, vec, a, s);
  // 16-bit rows are moved as they are
  return by_lanes<Append<false, false>::template At>(D, k, v, kts, khs, vts, vhs, vec, a, s);
}

hipError_t launch_kv_gather(uint16_t* k, uint16_t* v, bool bf16, int T, const int8mm_kv& kv,
                            const int32_t* table, int table_rows, int table_width,
                            const int32_t* rows, const int32_t* positions, hipStream_t s) {
  const Rows a = rows_of(kv, table, table_rows, table_width, rows, positions, T);
  const int D = kv.head_dim;
  if (kv.dtype == INT8MM_I8)
    return bf16 ? by_lanes<Gather<true, true>::template At>(D, k, v, a, s)
                : by_lanes<Gather<false, true>::template At>(D, k, v, a, s);
  return by_lanes<Gather<false, false>::template At>(D, k, v, a, s);
}

}  // namespace i8mm
