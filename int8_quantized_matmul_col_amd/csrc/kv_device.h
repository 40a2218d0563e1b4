// What the attention kernels over key-value pages share: matrix operands from
// the caches' types, probabilities in parts, and the pages' addresses.
#pragma once

#include "device_common.h"
#include "serving_launch.h"

namespace i8mm {

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

enum { kF16 = 0, kBF16 = 1, kI8 = 2 };

template <bool BF16>
__device__ __forceinline__ v4f mfma32(const v4u& a, const v4u& b, const v4f& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a),
                                                   __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Two probabilities as pairs of the operand type, each from below and then the
// next of what is left: three of bfloat16 hold fp32's 24 bits.  float16's
// second part is held times kRest: float16 ends at 2^-24, and so a probability
// of 2^-15 or less of the maximum would keep fewer than 16 bits, one of 2^-30
// next to none, where another token has the maximum and no value.  All parts of
// a positive number are positive (float16: down to 2^-30 of the maximum), so
// that an infinite value stays one: its product with a part of 0, or with one
// of the other sign, would be NaN.  float16's first part is rounded from 2^-12
// lower, for a remainder of 2^-12 or more.
constexpr float kRest = 4096.0f;  // probabilities reach 2^14, their rest 2^3.6
__device__ __forceinline__ uint32_t bf16_below(float& a, float& b) {
  const uint32_t ua = __builtin_elementwise_sub_sat(__float_as_uint(a), 1u);
  const uint32_t ub = __builtin_elementwise_sub_sat(__float_as_uint(b), 1u);
  a -= __uint_as_float(ua & 0xffff0000u);
  b -= __uint_as_float(ub & 0xffff0000u);
  return __builtin_amdgcn_perm(ub, ua, 0x07060302u);
}
template <bool BF16, int PARTS>
__device__ __forceinline__ void split(float a, float b, uint32_t (&part)[PARTS]) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < PARTS - 1; ++i) part[i] = bf16_below(a, b);
    part[PARTS - 1] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2b));
  } else {
    const uint32_t ua = __builtin_elementwise_sub_sat(__float_as_uint(a), 4096u);
    const uint32_t ub = __builtin_elementwise_sub_sat(__float_as_uint(b), 4096u);
    const v2h h = __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_pkrtz(__uint_as_float(ua), __uint_as_float(ub)));
    part[0] = __builtin_bit_cast(uint32_t, h);
    part[1] = f2h2((a - (float)h[0]) * kRest, (b - (float)h[1]) * kRest);
  }
}

// 4 int8 codes -> two dwords of exact bfloat16 / float16 numbers.
__device__ __forceinline__ void codes_bf16(uint32_t u, uint32_t& a, uint32_t& b) {
  const float f0 = (float)(int8_t)u, f1 = (float)(int8_t)(u >> 8);
  const float f2 = (float)(int8_t)(u >> 16), f3 = (float)(int8_t)(u >> 24);
  a = __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
  b = __builtin_amdgcn_perm(__float_as_uint(f3), __float_as_uint(f2), 0x07060302u);
}
__device__ __forceinline__ void codes_f16(uint32_t u, uint32_t& a, uint32_t& b) {
  const uint32_t x = u ^ 0x80808080u;  // code + 128; 0x6400 | that = 1152 + code
  const v2h c = {(_Float16)1152.0f, (_Float16)1152.0f};
  a = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, x, 0x04010400u)) - c);
  b = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, x, 0x04030402u)) - c);
}
template <bool BF16>
__device__ __forceinline__ v4u codes8(uint32_t u0, uint32_t u1) {
  uint32_t a, b, c, d;
  if constexpr (BF16) {
    codes_bf16(u0, a, b);
    codes_bf16(u1, c, d);
  } else {
    codes_f16(u0, a, b);
    codes_f16(u1, c, d);
  }
  return v4u{a, b, c, d};
}

// x of lane N of this lane's row of 16 lanes.
template <int N>
__device__ __forceinline__ float row_lane(float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x150 + N, 0xf, 0xf, true));
}

// Scores (probabilities) times their tokens' factors: lane N of a row of 16
// lanes holds the factor of the row's token N.
template <int N, int NT>
__device__ __forceinline__ void scale_tokens(v4f (&s)[NT], float x) {
  s[N / 4][N % 4] *= row_lane<N>(x);
  if constexpr (N + 1 < 4 * NT) scale_tokens<N + 1>(s, x);
}

struct Pages {
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  int64_t k_page, v_page;    // bytes
  int64_t ks_page, vs_page;  // floats
  int num_pages, kv_heads, ps, lps, D;
};

inline Pages pages_of(const int8mm_kv& kv) {
  Pages pg;
  const int eb = kv.dtype == INT8MM_I8 ? 1 : 2;
  pg.k = static_cast<const uint8_t*>(kv.k);
  pg.v = static_cast<const uint8_t*>(kv.v);
  pg.ks = kv.k_scale;
  pg.vs = kv.v_scale;
  pg.k_page = kv.k_page_stride * eb;
  pg.v_page = kv.v_page_stride * eb;
  pg.ks_page = kv.ks_page_stride;
  pg.vs_page = kv.vs_page_stride;
  pg.num_pages = kv.num_pages;
  pg.kv_heads = kv.kv_heads;
  pg.ps = kv.page_size;
  pg.lps = __builtin_ctz(kv.page_size);
  pg.D = kv.head_dim;
  return pg;
}

}  // namespace

}  // namespace i8mm
