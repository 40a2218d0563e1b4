// The attention of one new token per sequence over its pages, as the body of a
// kernel (kv_attention.hip says how it works): on its own, and beside the work on
// a prefix that all sequences share.
#pragma once

#include "kv_device.h"

namespace i8mm {

namespace {

constexpr int kWaves = 4;
constexpr int kAlign = 64;  // of a sequence's first token, a multiple of both chunk sizes
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
// bx: the workgroup among those that share a head group's tokens, by: the group.
template <int CT, bool QBF, int NK, bool EXACT>
__device__ __forceinline__ void attend_own(const KvAttentionArgs& a, const Pages& pg, int bx, int by) {
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
  const int kvh = by / tiles_h, ht = by % tiles_h;
  const int heads = min(group - ht * kKvHeadTile, kKvHeadTile);  // query heads of this tile
  const int head0 = kvh * group + ht * kKvHeadTile;
  constexpr int kUnit = kWaves * CH;

  // This workgroup's units.  One workgroup per sequence: all of them.
  // Otherwise the batch's units, one sequence after the other, are dealt out
  // evenly, and the workgroup finds its sequences from the lengths.
  int b = bx, first = 0;      // lane i holds sequence first + i below
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
    u0 = deal.begin(bx);
    u1 = deal.begin(bx + 1);
    if (first > 0) lanes(0);
    if (bx == 0 && by == 0 && wave == 0) {
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
  for (int at = threadIdx.x; at < heads * D; at += 64 * kWaves) {
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
      const int64_t piece = ((int64_t)by * a.parts + bx) * 2 + (fresh ? 0 : 1);
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

}  // namespace

}  // namespace i8mm
