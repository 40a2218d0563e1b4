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
#include "kv_device.h"

namespace i8mm {

namespace {

constexpr int kWaves = 4;
constexpr int kJoinThreads = 256;
constexpr int kAlign = 64;  // of a sequence's first token, a multiple of both chunk sizes
constexpr int kMaxParts = 512;  // workgroups that share a batch: two on every CU
constexpr int kWhole = 256;     // tokens up to which a sequence is one workgroup's
constexpr float kSlack = 8.0f;  // how far (log2) a score may exceed the running maximum

struct Range {
  int row, lo, len;  // visible tokens [lo, len)
};
__device__ __forceinline__ Range visible(const KvAttentionArgs& a, int b, int num_pages, int ps) {
  Range v{0, 0, 0};
  v.row = a.rows != nullptr ? a.rows[b] : b;
  if ((unsigned)v.row >= (unsigned)a.table_rows || num_pages == 0) return v;
  int64_t top = (int64_t)a.table_width * ps;
  if (top > a.max_len) top = a.max_len;
  const int n = a.lengths[v.row];
  v.len = n < 0 ? 0 : n > top ? (int)top : n;
  v.lo = a.window > 0 && a.window < v.len ? v.len - (int)a.window : 0;
  if (v.lo < a.first) v.lo = min(a.first, v.len);
  return v;
}

// Work is counted in units of kWaves chunks.  units(): of a sequence.
__device__ __forceinline__ int units(const Range& v, int unit) {
  return v.len > v.lo ? (v.len - (v.lo & ~(kAlign - 1)) + unit - 1) / unit : 0;
}
// `total` units dealt out to `parts` workgroups: the first `more` get one more
// than the others.
struct Deal {
  uint32_t each, more;
  __device__ __forceinline__ Deal(uint32_t total, uint32_t parts)
      : each(total / parts), more(total - total / parts * parts) {}
  // where part x begins
  __device__ __forceinline__ uint32_t begin(uint32_t x) const { return x * each + min(x, more); }
  // the part that has unit u
  __device__ __forceinline__ uint32_t of(uint32_t u) const {
    const uint32_t big = more * (each + 1);
    return u < big ? u / (each + 1) : more + (u - big) / each;
  }
};
__device__ __forceinline__ int wave_scan(int n) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(n, o, 64);
    if (lane >= o) n += y;
  }
  return n;
}

// CT: the cache's type; QBF: bfloat16 queries and results; NK: 32-dim steps
// (EXACT: head_dim is NK * 32, otherwise at most that).
template <int CT, bool QBF, int NK, bool EXACT>
__global__ __launch_bounds__(64 * kWaves, NK <= 4 ? 2 : 1) void k_kv_attention(KvAttentionArgs a, Pages pg) {
  constexpr bool I8 = CT == kI8;
  constexpr bool PBF = CT != kF16;      // type of the P x V operands
  constexpr int kParts = PBF ? 3 : 2;   // that hold a probability
  constexpr int CH = I8 ? 64 : 32;      // tokens per chunk
  constexpr int SUB = CH / 4;           // consecutive tokens a lane feeds to P x V
  constexpr int NT = CH / 16;           // score tiles
  constexpr int NKL = I8 ? NK / 2 : NK;  // 16-byte key loads per token row and lane
  constexpr int DT = NK * 2;            // output tiles of 16 dims
  constexpr int DR = PBF ? 1 : DT;      // output tiles of float16's second part
  constexpr int EB = I8 ? 1 : 2;
  // float16 probabilities are held times 2^6, at most 2^14 (kSlack): with kRest
  // their bits end at 2^-42 of the maximum, and those from 2^-20 on keep 22
  constexpr float kBias = CT == kF16 ? 6.0f : 0.0f;
  const int D = EXACT ? NK * 32 : pg.D;

  __shared__ float so[kWaves * DT * 256];  // outputs, [wave][tile][4][lane]
  __shared__ float sm[kWaves * 16], sl[kWaves * 16];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, qd = lane >> 4;
  const int group = a.group;
  const int tiles_h = (group + kKvHeadTile - 1) / kKvHeadTile;
  const int kvh = blockIdx.y / tiles_h, ht = blockIdx.y % tiles_h;
  const int heads = min(group - ht * kKvHeadTile, kKvHeadTile);  // query heads of this tile
  const int head0 = kvh * group + ht * kKvHeadTile;
  constexpr int kUnit = kWaves * CH;

  // This workgroup's units.  One workgroup per sequence: all of them.
  // Otherwise the batch's units, one sequence after the other, are dealt out
  // evenly, and the workgroup finds its sequences from the lengths.
  int b = blockIdx.x, first = 0;      // lane i holds sequence first + i below
  uint32_t u0 = 0, u1 = 0, before = 0;  // units of sequences before `first`
  Range mine{0, 0, 0};
  int own = 0, upto = 0;               // this lane's sequence: units, and with the lanes before
  auto lanes = [&](int at) __attribute__((always_inline)) {
    first = at;
    mine = Range{0, 0, 0};
    if (at + lane < a.B) mine = visible(a, at + lane, pg.num_pages, pg.ps);
    own = units(mine, kUnit);
    upto = wave_scan(own);
  };
  int idx = 0;  // of the current sequence among the lanes
  int next_tab = -1;
  bool looked = false;  // next_tab holds the next sequence's entries
  if (a.parts > 0) {
    uint32_t total = 0;
    for (int at = 0; at < a.B; at += 64) {
      lanes(at);
      total += __builtin_amdgcn_readlane(upto, 63);
    }
    const Deal deal(total, a.parts);
    u0 = deal.begin(blockIdx.x);
    u1 = deal.begin(blockIdx.x + 1);
    if (first > 0) lanes(0);
    if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) {
      // for the join: the first part that has units of a sequence, whether
      // another sequence comes before in it, and how many parts have some
      uint32_t base = 0;
      for (int at = 0;;) {
        const uint32_t begin = base + upto - own;
        int2 c = {0, 0};
        if (own > 0) {
          const uint32_t x = deal.of(begin);
          c.x = (int)(x * 2 + (deal.begin(x) < begin ? 1 : 0));
          c.y = (int)(deal.of(begin + own - 1) - x + 1);
        }
        if (at + lane < a.B) a.cuts[at + lane] = c;
        base += __builtin_amdgcn_readlane(upto, 63);
        if ((at += 64) >= a.B) break;
        lanes(at);
      }
      if (first > 0) lanes(0);
    }
    if (u0 >= u1) return;
    while (before + __builtin_amdgcn_readlane(upto, 63) <= u0) {
      before += __builtin_amdgcn_readlane(upto, 63);
      lanes(first + 64);
    }
    idx = __builtin_ctzll(__ballot(before + upto > u0));
  }

  for (bool again = true, fresh = true; again; fresh = false) {
  int row, lo, len, ua, ub, n;
  if (a.parts > 0) {
    b = first + idx;
    row = __builtin_amdgcn_readlane(mine.row, idx);
    lo = __builtin_amdgcn_readlane(mine.lo, idx);
    len = __builtin_amdgcn_readlane(mine.len, idx);
    n = __builtin_amdgcn_readlane(own, idx);
    const uint32_t begin = before + __builtin_amdgcn_readlane(upto, idx) - n;
    ua = u0 > begin ? (int)(u0 - begin) : 0;
    ub = u1 - begin < (uint32_t)n ? (int)(u1 - begin) : n;
    again = u1 > begin + n;
  } else {
    const Range v = visible(a, b, pg.num_pages, pg.ps);
    row = v.row, lo = v.lo, len = v.len;
    n = units(v, kUnit);
    ua = 0, ub = n;
    again = false;
  }
  const int s0 = (lo & ~(kAlign - 1)) + ua * kUnit;
  const int s1 = min(len, (lo & ~(kAlign - 1)) + ub * kUnit);
  const int chunks = s1 > s0 ? (s1 - s0 + CH - 1) / CH : 0;  // taken by the waves in turn

  // Q^T operand: head r, dims as the key loads order them
  v4u q[NK];
  {
    const uint16_t* qp = a.q + (int64_t)b * a.q_batch_stride + (int64_t)(head0 + min(r, heads - 1)) * a.q_head_stride;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const int d = I8 ? (j / 2) * 64 + qd * 16 + (j & 1) * 8 : j * 32 + qd * 8;
      q[j] = v4u{0, 0, 0, 0};
      if (d < D) q[j] = *reinterpret_cast<const v4u*>(qp + d);
    }
  }
  const int32_t* trow = a.table + (int64_t)row * a.table_width;
  auto entries = [&](int at) __attribute__((always_inline)) {
    return at + lane < a.table_width ? trow[at + lane] : -1;
  };
  int pbase = s0 >> pg.lps;
  int tab;  // lane's page id: table entry pbase + lane
  if (!looked)
    tab = chunks > 0 ? entries(pbase) : -1;
  else
    tab = next_tab;
  if (again) {
    // the next sequence's first table entries, long before they are needed
    int i = idx;
    do ++i; while (i < 64 && __builtin_amdgcn_readlane(own, i) == 0);
    looked = i < 64;
    if (looked) {
      const int at = (__builtin_amdgcn_readlane(mine.lo, i) & ~(kAlign - 1)) >> pg.lps;
      const int32_t* t = a.table + (int64_t)__builtin_amdgcn_readlane(mine.row, i) * a.table_width;
      next_tab = at + lane < a.table_width ? t[at + lane] : -1;
    }
  }

  v4f o[DT], rest[DR];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = v4f{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < DR; ++i) rest[i] = v4f{0, 0, 0, 0};
  float m = -INFINITY, l = 0.0f;

  if (wave < chunks) {
    v4u kr[NT][NKL], vr[DT];
    float ksc = 0.0f, vsc = 0.0f;
    bool kvalid = false, vvalid = false;  // of the chunk last addressed: this lane's page exists
    const uint8_t* vptr = nullptr;

    // pages of chunk c; loads its keys (and scales)
    auto load_k = [&](int c) __attribute__((always_inline)) {
      const int t0 = s0 + c * CH;
      if (((t0 + CH - 1) >> pg.lps) >= pbase + 64) {
        pbase = t0 >> pg.lps;
        tab = entries(pbase);
      }
      const int kt = t0 + SUB * (r >> 2) + (r & 3);
      const int vt = t0 + SUB * qd;
      int pk = __shfl(tab, (kt >> pg.lps) - pbase);
      int pv = __shfl(tab, (vt >> pg.lps) - pbase);
      vvalid = (unsigned)pv < (unsigned)pg.num_pages;
      kvalid = (unsigned)pk < (unsigned)pg.num_pages;
      pk = kvalid ? pk : 0;
      pv = vvalid ? pv : 0;
      const int kslot = kt & (pg.ps - 1), vslot = vt & (pg.ps - 1);
      const uint8_t* kp = pg.k + pk * pg.k_page + ((int64_t)kvh * pg.ps + kslot) * (D * EB) + qd * 16;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < NKL; ++j) {
          const int at = j * 64 + qd * 16;  // byte in the row
          if (EXACT || at < D * EB)
            kr[t][j] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(kp + t * 4 * D * EB + j * 64));
          else
            kr[t][j] = v4u{0, 0, 0, 0};
        }
      vptr = pg.v + pv * pg.v_page + ((int64_t)kvh * D * pg.ps + vslot) * EB;
      if constexpr (I8) {
        ksc = pg.ks[pv * pg.ks_page + kvh * pg.ps + vslot + r];
        vsc = pg.vs[pv * pg.vs_page + kvh * pg.ps + vslot + r];
      }
    };
    const uint32_t vrow = r * pg.ps * EB;
    auto load_v = [&]() __attribute__((always_inline)) {
      // tiles as scalar offsets, formed anew each time: as lanes' offsets kept
      // over the loop they take 24 registers, which 256 dims of float16 lack
      uint32_t tile = 16 * pg.ps * EB;
      asm volatile("" : "+s"(tile));
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        // (tiles past head_dim, which are not stored, read its last one)
        const uint32_t at = (EXACT ? i : min(i, D / 16 - 1)) * tile;
        vr[i] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(vptr + at + vrow));
      }
    };

    const float scale2 = a.softcap > 0.0f ? a.scale / a.softcap : a.scale * kLog2e;
    load_k(wave);
    load_v();
    for (int c = wave; c < chunks; c += kWaves) {
      const int t0 = s0 + c * CH;
      const bool page_ok = vvalid;
      const bool whole = t0 >= lo && t0 + CH <= s1 && __all(page_ok);

      // scores
      v4f s[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        s[t] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NKL; ++j) {
          if constexpr (I8) {
            s[t] = mfma32<QBF>(codes8<QBF>(kr[t][j][0], kr[t][j][1]), q[2 * j], s[t]);
            s[t] = mfma32<QBF>(codes8<QBF>(kr[t][j][2], kr[t][j][3]), q[2 * j + 1], s[t]);
          } else {
            s[t] = mfma32<QBF>(kr[t][j], q[j], s[t]);
          }
        }
      }
      float ks16 = 0.0f, vs16 = 0.0f;
      if constexpr (I8) {
        ks16 = ksc * (1.0f / 127.0f);
        vs16 = vsc * (1.0f / 127.0f);
      }
      if (c + kWaves < chunks) load_k(c + kWaves);

      if constexpr (I8) {
        scale_tokens<0>(s, ks16);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[t][i] * scale2;
          if (a.softcap > 0.0f) x = a.softcap * kLog2e * tanhf(x);
          if (!whole) {
            const int tok = t0 + SUB * qd + 4 * t + i;
            x = page_ok && tok >= lo && tok < s1 ? x : -INFINITY;
          }
          s[t][i] = x;
        }

      // running maximum, per head (lane r), equal in the four lanes qd
      float top = s[0][0];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[t][i]);
      if (__any(top > m + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m, top);
        const float f = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i) o[i] *= f;
        if constexpr (!PBF)
#pragma unroll
          for (int i = 0; i < DT; ++i) rest[i] *= f;
      }
      const float base = m == -INFINITY ? 0.0f : m - kBias;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[t][i] = __builtin_amdgcn_exp2f(s[t][i] - base);
          l += s[t][i];
        }
      if constexpr (I8) {
        const float vs_ok = page_ok ? vs16 : 0.0f;
        const int tok = t0 + SUB * qd + r;  // whose scale this lane holds
        const float vs = whole || (tok >= lo && tok < s1) ? vs_ok : 0.0f;
        scale_tokens<0>(s, vs);
      } else if (!whole) {
        // values of tokens that are not visible may be anything: 0, not 0 * NaN
        v4u keep;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = t0 + SUB * qd + 2 * e;
          const uint32_t a0 = page_ok && tok >= lo && tok < s1 ? 0x0000ffffu : 0u;
          const uint32_t a1 = page_ok && tok + 1 >= lo && tok + 1 < s1 ? 0xffff0000u : 0u;
          keep[e] = a0 | a1;
        }
#pragma unroll
        for (int i = 0; i < DT; ++i) vr[i] &= keep;
      }

      // P^T operand, in parts
      v4u p[NT / 2][kParts];
#pragma unroll
      for (int u = 0; u < NT / 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t x[kParts];
          split<PBF>(s[2 * u + e / 2][2 * (e & 1)], s[2 * u + e / 2][2 * (e & 1) + 1], x);
#pragma unroll
          for (int i = 0; i < kParts; ++i) p[u][i][e] = x[i];
        }
      // (two output tiles at a time: an instruction does not wait for the one
      // before it; int8, 256 dims: 66 -> 63.8 us for 8 x 8192 tokens of 8 heads)
#pragma unroll
      for (int i = 0; i < DT; i += 2) {
        if constexpr (I8) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const v4u x = codes8<true>(vr[i][2 * u], vr[i][2 * u + 1]);
            const v4u y = codes8<true>(vr[i + 1][2 * u], vr[i + 1][2 * u + 1]);
#pragma unroll
            for (int e = 0; e < kParts; ++e) {
              o[i] = mfma32<true>(x, p[u][e], o[i]);
              o[i + 1] = mfma32<true>(y, p[u][e], o[i + 1]);
            }
          }
        } else if constexpr (PBF) {
#pragma unroll
          for (int e = 0; e < kParts; ++e) {
            o[i] = mfma32<true>(vr[i], p[0][e], o[i]);
            o[i + 1] = mfma32<true>(vr[i + 1], p[0][e], o[i + 1]);
          }
        } else {
#pragma unroll
          for (int j = i; j < i + 2; ++j) {
            o[j] = mfma32<false>(vr[j], p[0][0], o[j]);
            rest[j] = mfma32<false>(vr[j], p[0][1], rest[j]);
          }
        }
      }
      if (c + kWaves < chunks) load_v();
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
  }

  // join the waves
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x = o[i][e];
      if constexpr (!PBF) x += rest[i][e] * (1.0f / kRest);
      so[((wave * DT + i) * 4 + e) * 64 + lane] = x;
    }
  if (qd == 0) {
    sm[wave * 16 + r] = m;
    sl[wave * 16 + r] = l;
  }
  __syncthreads();
  for (int at = threadIdx.x; at < heads * D; at += blockDim.x) {
    const int h = at / D, d = at % D;
    float mx = sm[h];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mx = fmaxf(mx, sm[w * 16 + h]);
    float sum = 0.0f, den = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float mw = sm[w * 16 + h];
      // a wave without a visible token has l = 0 and o = 0
      const float f = mw == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(mw - mx);
      den += f * sl[w * 16 + h];
      sum += f * so[((w * DT + (d >> 4)) * 4 + (d & 3)) * 64 + ((d & 15) >> 2) * 16 + h];
    }
    if (ua == 0 && ub == n && a.whole_o != nullptr) {  // the whole sequence, to be joined with others
      const int64_t bh = (int64_t)b * a.q_heads + head0 + h;
      a.whole_o[bh * D + d] = sum;
      if (d == 0) {
        a.whole_ml[2 * bh] = mx - kBias;
        a.whole_ml[2 * bh + 1] = den;
      }
    } else if (ua == 0 && ub == n) {  // the whole sequence
      const int64_t bh = (int64_t)b * a.q_heads + head0 + h;
      const float y = den == 0.0f ? 0.0f : sum * (1.0f / den);
      a.out[bh * D + d] = QBF ? __builtin_bit_cast(uint16_t, (__bf16)y) : f2h(y);
      if (d == 0 && a.lse != nullptr)
        a.lse[bh] = den == 0.0f ? -INFINITY : (mx - kBias + __builtin_log2f(den)) * kLn2;
    } else {
      // only a workgroup's first and last sequence can be cut: two places
      const int64_t piece = ((int64_t)blockIdx.y * a.parts + blockIdx.x) * 2 + (fresh ? 0 : 1);
      const int64_t at_h = piece * a.tile_heads + h;
      a.part_o[at_h * D + d] = sum;
      if (d == 0) {
        a.part_ml[2 * at_h] = mx - kBias;
        a.part_ml[2 * at_h + 1] = den;
      }
    }
  }
  if (again) {
    __syncthreads();  // the next sequence's sums take the same place
    do {
      if (++idx == 64) {
        before += __builtin_amdgcn_readlane(upto, 63);
        lanes(first + 64);
        idx = 0;
        looked = false;
      }
    } while (__builtin_amdgcn_readlane(own, idx) == 0);
  }
  }
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
