// Draws one token of each row of logits from a given uniform number, with
// temperature, top-k, top-p and min-p.
//
//   z = logit / T,  w = exp(z - max z);  order: by z downwards, then by index
//   top-k keeps the first k; top-p of those the ones with less than p of their
//   mass before them (the first always); min-p those with w >= min_p
//   token = the first index, in the vocabulary's order, whose running mass of
//   what is kept exceeds u times all of it
//
// Which token it is hangs on sums over a whole row, so they are exact: z is
// formed in 64 bits, bins of 1/8 in z split the line, and a weight is a whole
// number, round(2^36 exp(z - middle of its bin)).  Sums of them within a bin do
// not depend on the order or on how a row is cut, and 513 bins (all that lies
// within e^-64 of the maximum) times their powers of e^-1/8 are added in 64 bits.
//
// Bound by reading the logits: once, by S workgroups a row (k_sample_bins, 8192
// logits each), which leave per bin a count and a mass in one 64-bit word.  The
// second kernel, a workgroup a row, finds from the joined bins the one in which
// each filter cuts, reads the row again (from L2) only for that bin's tokens,
// sorts them, and so knows the cut itself; then the chunk that the given number
// falls into, and reads that.  Nothing is sorted but one bin.
#include "device_common.h"
#include "serving_launch.h"

namespace i8mm {

namespace {

enum { kF16 = 0, kBF16 = 1, kF32 = 2 };

constexpr int kBinThreads = 512;
constexpr int kPickThreads = 1024;
constexpr int kCopies = 8;       // of a workgroup's bins in LDS: lanes of equal bins collide less
constexpr int kLastBin = 512;    // 64 below the maximum
constexpr int kPitch = kSampleBins;
constexpr int kList = 2048;      // tokens of one bin that are sorted
constexpr int kDigits = 2048;
constexpr int kCountShift = 50;  // a word: a chunk's count (14 bits), its mass
constexpr uint64_t kMass = ((uint64_t)1 << kCountShift) - 1;
static_assert(kSampleChunk == kPickThreads * 8, "a thread takes 8 logits of a chunk");
static_assert(kSampleChunk < (1 << (64 - kCountShift)), "");
static_assert(kPitch > kLastBin, "");

// 8 logits from place v0 of the row, whose places mis .. mis + V - 1 exist and
// whose place 0 is on 16 bytes; -inf elsewhere.
template <int T>
__device__ __forceinline__ void load8(const void* base, int v0, int mis, int end, float (&x)[8]) {
  if (v0 >= mis && v0 + 8 <= end) {
    if constexpr (T == kF32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + v0);
      const float4 a = p[0], b = p[1];
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + v0);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (T == kBF16)
          x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        else
          x[i] = h2f((uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = -INFINITY;
      if (v0 + i >= mis && v0 + i < end) {
        if constexpr (T == kF32)
          x[i] = static_cast<const float*>(base)[v0 + i];
        else if constexpr (T == kBF16)
          x[i] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(base)[v0 + i] << 16);
        else
          x[i] = h2f(static_cast<const uint16_t*>(base)[v0 + i]);
      }
    }
  }
}

struct Row {
  const void* base;  // place 0, on 16 bytes
  int mis, end;      // places of the row
  double per8;       // 8 / T
  bool greedy;
};
template <int T>
__device__ __forceinline__ Row row_of(const SampleArgs& a, int b) {
  constexpr int eb = T == kF32 ? 4 : 2;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) + (int64_t)b * a.row_stride * eb;
  Row r;
  r.base = reinterpret_cast<const void*>(at & ~(uintptr_t)15);
  r.mis = (int)(at & 15) / eb;
  r.end = r.mis + a.V;
  const float t = a.temperature != nullptr ? a.temperature[b] : a.temperature_all;
  r.greedy = !(t > 0.0f);
  r.per8 = r.greedy ? 8.0 : 8.0 / (double)t;
  return r;
}

// z in eighths, and the weight of what it exceeds its bin's lower end by.
__device__ __forceinline__ double eighths(float x, double per8) {
#pragma clang fp contract(off)
  return (double)x * per8;
}
__device__ __forceinline__ uint64_t weight(double z8, double bin) {
#pragma clang fp contract(off)
  const double x = __builtin_fma(z8 - bin, 0.125, -0.0625);  // +- 1/16
  // the series of exp; what follows is below 2^-47
  double p = 1.0 / 5040;
  p = __builtin_fma(p, x, 1.0 / 720);
  p = __builtin_fma(p, x, 1.0 / 120);
  p = __builtin_fma(p, x, 1.0 / 24);
  p = __builtin_fma(p, x, 1.0 / 6);
  p = __builtin_fma(p, x, 0.5);
  p = __builtin_fma(p, x, 1.0);
  p = __builtin_fma(p, x, 1.0);
  // rounded to a whole number by the addition; its bits are the mantissa's
  const double y = __builtin_fma(p, 0x1p36, 0x1p52);
  return (uint64_t)__double_as_longlong(y) & (((uint64_t)1 << 52) - 1);
}

// Ascending keys for descending logits (-0 and 0 are equal).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u >> 31 ? u : ~u & 0x7fffffffu;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k >> 31 ? k : ~k & 0x7fffffffu);
}

__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

// ------------------------------------------------------ the bins of a chunk

template <int T>
__global__ __launch_bounds__(kBinThreads) void k_sample_bins(SampleArgs a) {
  constexpr int kPieces = kSampleChunk / 8 / kBinThreads;
  __shared__ uint64_t bins[kCopies][kPitch];
  __shared__ float tops[kBinThreads / 64];
  __shared__ int first, last, bad;
  const int c = blockIdx.x, b = blockIdx.y;
  const Row r = row_of<T>(a, b);
  float x[kPieces][8];
  int at[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    at[i] = c * kSampleChunk + (i * kBinThreads + (int)threadIdx.x) * 8;
    load8<T>(r.base, at[i], r.mis, r.end, x[i]);
  }
  for (int i = threadIdx.x; i < kCopies * kPitch; i += kBinThreads) (&bins[0][0])[i] = 0;
  if (threadIdx.x == 0) first = 0x7fffffff, last = 0, bad = 0;
  float top = -INFINITY;
  bool wrong = false;
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      top = fmaxf(top, x[i][e]);
      wrong |= !(x[i][e] < INFINITY);
    }
  top = wave_max_f(top);
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  if (__any(wrong) && (threadIdx.x & 63) == 0) bad = 1;
#pragma unroll
  for (int w = 0; w < kBinThreads / 64; ++w) top = fmaxf(top, tops[w]);

  if (r.greedy) {
    int mine = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (x[i][e] == top) mine = min(mine, at[i] + e - r.mis);
    if (mine != 0x7fffffff) atomicMin(&first, mine);
  } else if (top > -INFINITY) {
    uint64_t* own = bins[threadIdx.x & (kCopies - 1)];
    const double upper = floor(eighths(top, r.per8));
    int low = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double z8 = eighths(x[i][e], r.per8);
        const double bin = floor(z8);
        const double below = upper - bin;
        if (below <= (double)kLastBin) {  // (not where z is -inf or NaN)
          const int rel = (int)below;
          low = max(low, rel);
          atomicAdd(reinterpret_cast<unsigned long long*>(own + rel),
                    (unsigned long long)(weight(z8, bin) + ((uint64_t)1 << kCountShift)));
        }
      }
    atomicMax(&last, low);
  }
  __syncthreads();
  const int64_t place = (int64_t)b * a.S + c;
  if (threadIdx.x == 0) {
    SampleHead h;
    h.top = top;
    h.first = first;
    h.last = r.greedy || !(top > -INFINITY) ? -1 : last;
    h.bad = bad;
    a.heads[place] = h;
  }
  if (r.greedy) return;
  uint64_t* out = a.bins + place * kPitch;
  for (int i = threadIdx.x; i <= last; i += kBinThreads) {
    uint64_t n = 0;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) n += bins[k][i];
    out[i] = n;
  }
}

// ----------------------------------------------------------- the row's token

__device__ __forceinline__ double shfl_up_d(double v, int o) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = __shfl_up((uint32_t)u, o, 64), hi = __shfl_up((uint32_t)(u >> 32), o, 64);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ uint64_t shfl_up_u(uint64_t u, int o) {
  const uint32_t lo = __shfl_up((uint32_t)u, o, 64), hi = __shfl_up((uint32_t)(u >> 32), o, 64);
  return (uint64_t)hi << 32 | lo;
}

// Inclusive sums over the workgroup's threads, in a fixed order.
template <typename V, typename F>
__device__ __forceinline__ V block_scan(V x, V* part, F up) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const V y = up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) part[wave] = x;
  __syncthreads();
  V before = 0;
  for (int w = 0; w < wave; ++w) before += part[w];
  return before + x;
}

struct Pick {
  double scale[kPitch];   // e^(-bin / 8)
  double mass[kPitch];    // before a bin, in bin order (largest z first)
  uint64_t in[kPitch];    // in a bin
  uint32_t count[kPitch];   // before a bin
  uint32_t own[kPitch];     // in a bin
  union {
    uint64_t list[kList];
    struct {
      uint64_t mass[kDigits];
      uint32_t count[kDigits];
    } digit;
  };
  uint64_t extra[kSampleMaxChunks];  // of the bin that is kept in part
  double chunk[kSampleMaxChunks];    // kept mass of a chunk
  int off[kSampleMaxChunks], last[kSampleMaxChunks];
  uint8_t has[kSampleMaxChunks];
  uint64_t part_u[kPickThreads / 64];
  double part_d[kPickThreads / 64];
  float tops[kPickThreads / 64];
  int found, n;
  uint64_t answer_comp, answer_mass;
};

template <int T>
struct Picker {
  const SampleArgs& a;
  Pick& s;
  Row r;
  int b;
  double upper;     // the maximum's bin
  int listed = -1;  // the bin that s.list holds, sorted

  __device__ Picker(const SampleArgs& a_, Pick& s_, int b_) : a(a_), s(s_), b(b_) { r = row_of<T>(a, b); }

  __device__ __forceinline__ uint64_t word(int c, int bin) const {
    const int j = bin - s.off[c];
    return j >= 0 && j <= s.last[c] ? a.bins[((int64_t)b * a.S + c) * kPitch + j] : 0;
  }
  __device__ __forceinline__ uint64_t comp(float x, int v) const {
    return (uint64_t)key_of(x) << 32 | (uint32_t)(v - r.mis);
  }

  // f(x, place, z8) for the tokens of a bin.
  template <typename F>
  __device__ __forceinline__ void each(int bin, F f) {
    __syncthreads();
    if ((int)threadIdx.x < a.S) s.has[threadIdx.x] = (word(threadIdx.x, bin) >> kCountShift) != 0;
    __syncthreads();
    const double at = upper - (double)bin;
    // logits of the bin, generously, in 32 bits
    const double lo = at / r.per8, hi = (at + 1.0) / r.per8;
    float flo = (float)(lo - (fabs(lo) * 1e-6 + 1e-40)), fhi = (float)(hi + (fabs(hi) * 1e-6 + 1e-40));
    if (!(r.per8 > 0.0)) flo = -INFINITY, fhi = INFINITY;  // an infinite temperature
    for (int c = 0; c < a.S; ++c) {
      if (!s.has[c]) continue;
      const int v0 = c * kSampleChunk + (int)threadIdx.x * 8;
      float x[8];
      load8<T>(r.base, v0, r.mis, r.end, x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (x[e] >= flo && x[e] <= fhi) {
          const double z8 = eighths(x[e], r.per8);
          if (floor(z8) == at) f(x[e], v0 + e, z8);
        }
    }
  }

  // Where the tokens of `bin` stop being kept: those whose rank in the bin is
  // below `most` and that have less than `limit` before them, `before` of it
  // ahead of the bin.  Returns the last one that is kept, and the kept mass.
  __device__ void resolve(int bin, double before, uint32_t most, double limit, uint64_t* last,
                          uint64_t* mass) {
    const double scale = s.scale[bin];
    auto keeps = [&](uint32_t rank, uint64_t m) {
      return rank < most && (before + (double)m * scale < limit || (before == 0.0 && m == 0));
    };
    uint32_t n = s.own[bin], rank0 = 0;
    uint64_t mass0 = 0, want = 0, mask = 0;  // keys (key & mask) == want are left
    if (n > kList) {
      const int shifts[3] = {21, 10, 0};
      for (int d = 0; d < 3 && n > kList; ++d) {
        listed = -1;
        __syncthreads();
        for (int i = threadIdx.x; i < kDigits; i += kPickThreads) s.digit.mass[i] = 0, s.digit.count[i] = 0;
        const int shift = shifts[d];
        each(bin, [&](float x, int, double z8) {
          const uint32_t k = key_of(x);
          if ((k & mask) != want) return;
          const uint32_t i = (k >> shift) & (d == 2 ? 1023u : 2047u);
          atomicAdd(s.digit.count + i, 1u);
          atomicAdd(reinterpret_cast<unsigned long long*>(s.digit.mass + i),
                    (unsigned long long)weight(z8, upper - (double)bin));
        });
        if (threadIdx.x == 0) s.found = kDigits;
        __syncthreads();
        // two digits a thread
        const int i0 = threadIdx.x * 2;
        const uint64_t m0 = s.digit.mass[i0], m1 = s.digit.mass[i0 + 1];
        const uint32_t c0 = s.digit.count[i0], c1 = s.digit.count[i0 + 1];
        const uint64_t mi = block_scan<uint64_t>(m0 + m1, s.part_u, shfl_up_u) + mass0;
        const uint64_t ci = block_scan<uint64_t>((uint64_t)c0 + c1, s.part_u, shfl_up_u) + rank0;
        // the last digit whose first token is kept
        const uint64_t ma = mi - m0 - m1, mb = mi - m1;
        const uint32_t ca = (uint32_t)ci - c0 - c1, cb = (uint32_t)ci - c1;
        int mine = -1;
        if (c0 > 0 && keeps(ca, ma)) mine = i0;
        if (c1 > 0 && keeps(cb, mb)) mine = i0 + 1;
        __syncthreads();
        if (threadIdx.x == 0) s.found = -1;
        __syncthreads();
        if (mine >= 0) atomicMax(&s.found, mine);
        __syncthreads();
        const int digit = s.found;
        if (mine == digit) {
          s.answer_comp = digit & 1 ? cb : ca;
          s.answer_mass = digit & 1 ? mb : ma;
          s.n = (int)(digit & 1 ? c1 : c0);
        }
        __syncthreads();
        rank0 = (uint32_t)s.answer_comp;
        mass0 = s.answer_mass;
        n = (uint32_t)s.n;
        want |= (uint64_t)digit << shift;
        mask |= (uint64_t)(d == 2 ? 1023u : 2047u) << shift;
        __syncthreads();
      }
      if (n > kList) {
        // one key, many tokens: a number of them, in index order
        const uint32_t key = (uint32_t)want;
        const double z8 = eighths(of_key(key), r.per8);
        const uint64_t w = weight(z8, upper - (double)bin);
        uint32_t lo = 1, hi = n;
        while (lo < hi) {
          const uint32_t mid = lo + (hi - lo + 1) / 2;
          if (keeps(rank0 + mid - 1, mass0 + (uint64_t)(mid - 1) * w)) lo = mid; else hi = mid - 1;
        }
        *mass = mass0 + (uint64_t)lo * w;
        // the lo-th of them: threads take runs that follow one another
        const int per = (r.end + 8 * kPickThreads - 1) / (8 * kPickThreads) * 8;
        uint32_t mine = 0;
        for (int v = (int)threadIdx.x * per; v < (int)threadIdx.x * per + per; v += 8) {
          float x[8];
          load8<T>(r.base, v, r.mis, r.end, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) mine += v + e >= r.mis && v + e < r.end && key_of(x[e]) == key;
        }
        const uint64_t upto = block_scan<uint64_t>(mine, s.part_u, shfl_up_u);
        if (upto >= lo && upto - mine < lo) {
          uint32_t left = lo - (uint32_t)(upto - mine);
          for (int v = (int)threadIdx.x * per; left > 0; v += 8) {
            float x[8];
            load8<T>(r.base, v, r.mis, r.end, x);
            for (int e = 0; e < 8 && left > 0; ++e)
              if (v + e >= r.mis && v + e < r.end && key_of(x[e]) == key && --left == 0) s.found = v + e - r.mis;
          }
        }
        __syncthreads();
        *last = (uint64_t)key << 32 | (uint32_t)s.found;
        __syncthreads();
        return;
      }
    }
    if (listed != bin || mask != 0) {
      __syncthreads();
      if (threadIdx.x == 0) s.n = 0;
      for (int i = threadIdx.x; i < kList; i += kPickThreads) s.list[i] = ~(uint64_t)0;
      each(bin, [&](float x, int v, double) {
        if ((key_of(x) & mask) != want) return;
        const int i = atomicAdd(&s.n, 1);
        if (i < kList) s.list[i] = comp(x, v);
      });
      int size = 2;
      while (size < (int)n) size *= 2;
      // bitonic
      for (int k = 2; k <= size; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
          __syncthreads();
          for (int t = threadIdx.x; t < size / 2; t += kPickThreads) {
            const int i = 2 * t - (t & (j - 1));
            const uint64_t x = s.list[i], y = s.list[i + j];
            if ((x > y) == ((i & k) == 0)) s.list[i] = y, s.list[i + j] = x;
          }
        }
      listed = mask == 0 ? bin : -1;
    }
    __syncthreads();
    const uint32_t i0 = threadIdx.x * 2;
    uint64_t c[2], w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i] = s.list[i0 + i];
      w[i] = i0 + i < n ? weight(eighths(of_key((uint32_t)(c[i] >> 32)), r.per8), upper - (double)bin) : 0;
    }
    const uint64_t upto = block_scan<uint64_t>(w[0] + w[1], s.part_u, shfl_up_u) + mass0;
    __syncthreads();
    if (threadIdx.x == 0) s.found = -1;
    __syncthreads();
    int mine = -1;
    if (i0 < n && keeps(rank0 + i0, upto - w[0] - w[1])) mine = (int)i0;
    if (i0 + 1 < n && keeps(rank0 + i0 + 1, upto - w[1])) mine = (int)i0 + 1;
    if (mine >= 0) atomicMax(&s.found, mine);
    __syncthreads();
    if (mine == s.found) {
      s.answer_comp = c[mine & 1];
      s.answer_mass = mine & 1 ? upto : upto - w[1];
    }
    __syncthreads();
    *last = s.answer_comp;
    *mass = s.answer_mass;
    __syncthreads();
  }

  __device__ void run() {
    const int tid = threadIdx.x;
    // the chunks' heads
    float top = -INFINITY;
    int first = 0x7fffffff, bad = 0;
    SampleHead h{-INFINITY, 0, -1, 0};
    if (tid < a.S) h = a.heads[(int64_t)b * a.S + tid];
    if (tid == 0) s.n = 0, s.found = 0x7fffffff;
    top = wave_max_f(h.top);
    if ((tid & 63) == 0) s.tops[tid >> 6] = top;
    __syncthreads();
    for (int w = 0; w < kPickThreads / 64; ++w) top = fmaxf(top, s.tops[w]);
    if (h.bad) s.n = 1;
    if (r.greedy && tid < a.S && h.top == top) atomicMin(&s.found, h.first);
    __syncthreads();
    bad = s.n;
    first = s.found;
    const float t = a.temperature != nullptr ? a.temperature[b] : a.temperature_all;
    if (bad || !(top > -INFINITY) || t != t || r.greedy) {
      if (tid == 0) a.tokens[b] = bad || !(top > -INFINITY) || t != t ? -1 : first;
      return;
    }
    const double top8 = eighths(top, r.per8);
    upper = floor(top8);
    if (tid < kSampleMaxChunks) {
      int off = 1 << 20;
      if (tid < a.S && h.last >= 0) {
        const double d = upper - floor(eighths(h.top, r.per8));
        if (d <= (double)kLastBin) off = (int)d;
      }
      s.off[tid] = off;
      s.last[tid] = h.last;
      s.extra[tid] = 0;
    }
    __syncthreads();

    // all chunks' bins, and what lies before each
    uint64_t m = 0;
    uint32_t n = 0;
    double scale = 0.0;
    if (tid <= kLastBin) {
      for (int c = 0; c < a.S; ++c) {
        const uint64_t x = word(c, tid);
        m += x & kMass;
        n += (uint32_t)(x >> kCountShift);
      }
      scale = exp(-0.125 * tid);
      s.scale[tid] = scale;
      s.in[tid] = m;
      s.own[tid] = n;
    }
    const double own = (double)m * scale;
    const double upto = block_scan<double>(own, s.part_d, shfl_up_d);
    const uint64_t nupto = block_scan<uint64_t>(n, s.part_u, shfl_up_u);
    if (tid <= kLastBin) {
      s.mass[tid] = upto - own;
      s.count[tid] = (uint32_t)nupto - n;
    }
    __syncthreads();
    if (tid == kLastBin) s.answer_mass = (uint64_t)__double_as_longlong(upto), s.answer_comp = nupto;
    if (tid == 0) s.mass[0] = 0.0;
    __syncthreads();
    double total = __longlong_as_double((long long)s.answer_mass);
    const uint32_t all = (uint32_t)s.answer_comp;

    // the cut: bins before `bin` are kept, of it the tokens up to `comp`
    int bin = kLastBin + 1;
    uint64_t cut = ~(uint64_t)0;
    uint32_t most = 0xffffffffu;
    const int k = a.top_k != nullptr ? a.top_k[b] : a.top_k_all;
    if (k > 0 && (uint32_t)k < all) {
      __syncthreads();
      if (tid <= kLastBin && s.own[tid] > 0 && s.count[tid] < (uint32_t)k && s.count[tid] + s.own[tid] >= (uint32_t)k)
        s.found = tid;
      __syncthreads();
      bin = s.found;
      most = (uint32_t)k - s.count[bin];
      uint64_t kept = s.in[bin];
      if (most < s.own[bin])
        resolve(bin, s.mass[bin], most, INFINITY, &cut, &kept);
      else
        most = 0xffffffffu;
      total = s.mass[bin] + (double)kept * s.scale[bin];
    }
    const float p = a.top_p != nullptr ? a.top_p[b] : a.top_p_all;
    if (p < 1.0f) {
      const double limit = (double)p * total;
      __syncthreads();
      if (tid == 0) s.found = 0;
      __syncthreads();
      // the last bin whose first token is kept
      const bool starts = tid <= kLastBin && tid <= bin && s.own[tid] > 0 && s.mass[tid] < limit;
      if (starts) atomicMax(&s.found, tid);
      __syncthreads();
      const int at = s.found;
      uint64_t kept = 0;
      resolve(at, s.mass[at], at == bin ? most : 0xffffffffu, limit, &cut, &kept);
      bin = at;
    }
    const float mp = a.min_p != nullptr ? a.min_p[b] : a.min_p_all;
    double least = -INFINITY;  // z8 of min-p, where it cuts in `bin`
    if (mp > 0.0f) {
      const double z8 = top8 + 8.0 * log((double)fminf(mp, 1.0f));
      const double below = upper - floor(z8);
      if (below < (double)bin) bin = (int)below, cut = ~(uint64_t)0, least = z8;
      else if (below == (double)bin) least = z8;
    }

    // the kept mass of each chunk
    auto kept_in = [&](float x, int v, double z8) { return comp(x, v) <= cut && z8 >= least; };
    if (bin <= kLastBin) {
      const double at = upper - (double)bin;
      each(bin, [&](float x, int v, double z8) {
        if (kept_in(x, v, z8))
          atomicAdd(reinterpret_cast<unsigned long long*>(s.extra + v / kSampleChunk),
                    (unsigned long long)weight(z8, at));
      });
    }
    __syncthreads();
    for (int c = tid >> 6; c < a.S; c += kPickThreads / 64) {
      double x = 0.0;
      if (s.off[c] <= kLastBin) {
        const uint64_t* w = a.bins + ((int64_t)b * a.S + c) * kPitch;
        const int end = min(s.last[c], min(bin - 1, kLastBin) - s.off[c]);
        for (int j = tid & 63; j <= end; j += 64) x += (double)(w[j] & kMass) * s.scale[j + s.off[c]];
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double y = shfl_up_d(x, o);
        if ((tid & 63) >= o) x += y;
      }
      if ((tid & 63) == 63) s.chunk[c] = x + (bin <= kLastBin ? (double)s.extra[c] * s.scale[bin] : 0.0);
    }
    __syncthreads();
    double sum = 0.0;
    for (int c = 0; c < a.S; ++c) sum += s.chunk[c];
    float u = a.u[b];
    u = u > 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;
    const double target = (double)u * sum;
    double begin = 0.0;
    int c = 0;
    while (c < a.S && !(begin + s.chunk[c] > target)) begin += s.chunk[c++];
    // (rounding may leave nothing in the chunk: then the next one's first, or
    // the last that is kept)
    for (bool over = false;;) {
      if (c >= a.S) {
        over = true;
        c = a.S - 1;
        while (c > 0 && !(s.chunk[c] > 0.0)) --c;
      }
      const int v0 = c * kSampleChunk + tid * 8;
      float x[8];
      double w[8], mine = 0.0;
      load8<T>(r.base, v0, r.mis, r.end, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double z8 = eighths(x[e], r.per8);
        const double f = floor(z8);
        const double below = upper - f;
        w[e] = 0.0;
        if (top8 - z8 < 512.0 && below <= (double)bin && (below < (double)bin || kept_in(x[e], v0 + e, z8)))
          w[e] = (double)weight(z8, f) * s.scale[(int)below];
        mine += w[e];
      }
      const double last = block_scan<double>(mine, s.part_d, shfl_up_d);
      __syncthreads();
      if (tid == 0) s.found = over ? -1 : 0x7fffffff;
      __syncthreads();
      double at = begin + (last - mine);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        at += w[e];
        if (w[e] > 0.0) {
          if (over)
            atomicMax(&s.found, v0 + e);
          else if (at > target)
            atomicMin(&s.found, v0 + e);
        }
      }
      __syncthreads();
      const int found = s.found;
      if (found != 0x7fffffff) {
        if (tid == 0) a.tokens[b] = found < 0 ? -1 : found - r.mis;
        return;
      }
      begin += s.chunk[c];
      ++c;
      __syncthreads();
    }
  }
};

template <int T>
__global__ __launch_bounds__(kPickThreads) void k_sample_pick(SampleArgs a) {
  __shared__ Pick s;
  Picker<T> p(a, s, blockIdx.x);
  p.run();
}

template <int T>
hipError_t run(const SampleArgs& a, hipStream_t s) {
  if (a.S > 0) {
    hipLaunchKernelGGL(k_sample_bins<T>, dim3(a.S, a.B), dim3(kBinThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_sample_pick<T>, dim3(a.B), dim3(kPickThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t s) {
  if (dtype == INT8MM_F32) return run<kF32>(a, s);
  return dtype == INT8MM_BF16 ? run<kBF16>(a, s) : run<kF16>(a, s);
}

}  // namespace i8mm
