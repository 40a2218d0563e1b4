// Upkeep of a key-value cache's pages: copying, reserving, forking, freeing
// and compacting, with the page tables, lengths and reference counts on the
// device, so that a serving loop neither waits for the GPU nor copies them.
//
// Bound by HBM where pages move (each read and written once), else by the
// launches (copy and free are one kernel, the others two) and, in reserve and
// fork, by the plan: one workgroup compares every row named with every other
// (32 pairs 6.7 us, 64 rows 13, of 16 us for the whole reserve call).  The first
// of the two kernels snapshots which pages are free: one bit a page, a running
// count per 64-page word and a count per 4096-page block.  From these any thread
// of the second kernel finds the i-th free (or used) page by two binary
// searches, so pages are handed out lowest id first without a list, a queue or
// an atomic, and the result does not depend on timing.  Only reference counts
// use atomics (integer additions, whose order does not matter).
#include "device_common.h"
#include "serving_launch.h"

namespace i8mm {

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kBlockPages = 4096;  // pages per block of the snapshot: 64 words of 64
constexpr int kMaxBlocks = INT8MM_KV_MAX_PAGES / kBlockPages;
constexpr int kScanThreads = 1024;
constexpr int kThreads = 256;
constexpr int kSlice = 32768;  // bytes of a page that one workgroup copies at a time
constexpr uint32_t kSat = 1u << 30;  // page counts saturate here (more than any pool)

struct Snapshot {
  uint64_t* words;    // [blocks][64], bit set: free
  uint32_t* before;   // [blocks][64], free pages of the block before the word
  uint32_t* counts;   // [blocks], free pages
  int32_t* plan;      // [n], status so far
  uint32_t* first;    // [n], free pages that earlier rows take
  uint32_t* need;     // [n], free pages that this row takes
};

int blocks_of(int num_pages) { return (num_pages + kBlockPages - 1) / kBlockPages; }

Snapshot carve(void* ws, int64_t num_pages, int64_t n, size_t* total) {
  Snapshot s;
  const int64_t nb = blocks_of((int)num_pages);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    void* p = static_cast<char*>(ws) + off;
    off += (bytes + 255) / 256 * 256;
    return p;
  };
  s.words = static_cast<uint64_t*>(take(nb * 64 * 8));
  s.before = static_cast<uint32_t*>(take(nb * 64 * 4));
  s.counts = static_cast<uint32_t*>(take(nb * 4));
  s.plan = static_cast<int32_t*>(take(n * 4));
  s.first = static_cast<uint32_t*>(take(n * 4));
  s.need = static_cast<uint32_t*>(take(n * 4));
  if (total != nullptr) *total = off;
  return s;
}

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
  const uint32_t c = a + b;  // both at most kSat
  return c < kSat ? c : kSat;
}

// Inclusive saturating scan over the block's threads (a multiple of 64).
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = __shfl_up(x, o, 64);
    if (lane >= o) x = sat_add(x, y);
  }
  __syncthreads();
  if (lane == 63) part[wave] = x;
  __syncthreads();
  for (int w = 0; w < wave; ++w) x = sat_add(x, part[w]);
  return x;
}

// The free pages of pages [4096*block, ..).
__device__ void scan_pages(const int32_t* __restrict__ ref, int num_pages, int block,
                           const Snapshot& s, uint32_t* sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int w = wave; w < 64; w += kScanThreads / 64) {
    const int page = block * kBlockPages + w * 64 + lane;
    const uint64_t free = __ballot(page < num_pages && ref[page] <= 0);
    if (lane == 0) {
      s.words[block * 64 + w] = free;
      sh[w] = __popcll(free);
    }
  }
  __syncthreads();
  if (wave == 0) {
    const uint32_t own = sh[lane];
    uint32_t x = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t y = __shfl_up(x, o, 64);
      if (lane >= o) x += y;
    }
    s.before[block * 64 + lane] = x - own;
    if (lane == 63) s.counts[block] = x;
  }
}

__global__ __launch_bounds__(kScanThreads) void k_pages_scan(const int32_t* __restrict__ ref,
                                                             int num_pages, Snapshot s) {
  __shared__ uint32_t sh[64];
  scan_pages(ref, num_pages, blockIdx.x, s, sh);
}

// Rows named by a call, with what decides about them.
struct Rows {
  int32_t* table;
  int32_t* lengths;
  int32_t* refcount;
  const int32_t* a;  // fork: parents; reserve: rows
  const int32_t* b;  // fork: children; reserve: new lengths
  int32_t* status;
  int table_rows, table_width, n, num_pages, lps;
};

// One workgroup beside the scan: which rows are in order, and how many free
// pages each takes after how many.  It reads lengths and tables before the
// second kernel changes them.
template <bool FORK>
__device__ void plan_rows(const Rows& r, const Snapshot& s, uint32_t* part, int32_t* names) {
  uint32_t taken = 0;
  const int ps = 1 << r.lps;
  const int64_t room = (int64_t)r.table_width << r.lps;
  // fork: a child is named once and is no parent; reserve: a row's first naming counts
  const int32_t* named = FORK ? r.b : r.a;
  for (int i0 = 0; i0 < r.n; i0 += kScanThreads) {
    const int i = i0 + threadIdx.x;
    int own = -1, parent = -1;
    if (i < r.n) {
      own = named[i];
      if (FORK) parent = r.a[i];
    }
    bool ok = (unsigned)own < (unsigned)r.table_rows;
    if (FORK) ok = ok && (unsigned)parent < (unsigned)r.table_rows;
    // what decides, requested before the names are compared
    const int own_len = ok ? r.lengths[own] : 0;
    const int len = FORK ? (ok ? r.lengths[parent] : 0) : own_len;
    const int want = !FORK && ok ? r.b[i] : 0;
    int page = -1;
    if (FORK && ok && len >= 0 && len < room) page = r.table[(int64_t)parent * r.table_width + (len >> r.lps)];
    for (int j0 = 0; j0 < r.n; j0 += kScanThreads) {
      __syncthreads();
      if (j0 + (int)threadIdx.x < r.n) names[threadIdx.x] = named[j0 + threadIdx.x];
      __syncthreads();
      const int top = min(kScanThreads, r.n - j0);
      for (int j = 0; j < top; ++j) {
        if (j0 + j < i && names[j] == own) ok = false;
        if (FORK && names[j] == parent) ok = false;
      }
    }
    uint32_t need = 0;
    if (ok && FORK) {
      ok = own_len == 0 && len >= 0 && len <= room;
      if (ok && (len & (ps - 1)) != 0) {
        need = 1;
        ok = (unsigned)page < (unsigned)r.num_pages;
      }
    } else if (ok) {
      ok = len >= 0 && want >= len && want <= room;
      // (len + ps - 1) may pass 2^31 near the largest length
      if (ok) need = (uint32_t)((((int64_t)want + ps - 1) >> r.lps) - (((int64_t)len + ps - 1) >> r.lps));
    }
    if (!ok) need = 0;
    if (need > kSat) need = kSat;
    const uint32_t upto = sat_add(taken, block_scan(need, part));
    if (i < r.n) {
      s.plan[i] = ok ? INT8MM_KV_DONE : INT8MM_KV_BAD_ROW;
      s.need[i] = need;
      // only the rows before count: upto may be saturated, and then nothing fits
      s.first[i] = upto >= kSat ? kSat : upto - need;
    }
    __syncthreads();
    if (threadIdx.x == kScanThreads - 1) part[16] = upto;
    __syncthreads();
    taken = part[16];
  }
}

template <bool FORK>
__global__ __launch_bounds__(kScanThreads) void k_pages_plan(Rows r, Snapshot s) {
  __shared__ uint32_t sh[64];
  __shared__ int32_t names[kScanThreads];
  if ((int)blockIdx.x < (int)gridDim.x - 1)
    scan_pages(r.refcount, r.num_pages, blockIdx.x, s, sh);
  else
    plan_rows<FORK>(r, s, sh, names);
}

// ------------------------------------------------- reading the snapshot

// pre[b] = free pages before block b, b = 0 .. blocks; every thread calls it.
__device__ void load_prefix(const Snapshot& s, int blocks, uint32_t* pre, uint32_t* part) {
  constexpr int per = kMaxBlocks / kThreads;
  uint32_t c[per], sum = 0;
#pragma unroll
  for (int e = 0; e < per; ++e) {
    const int b = threadIdx.x * per + e;
    c[e] = b < blocks ? s.counts[b] : 0;
    sum += c[e];
  }
  uint32_t at = block_scan(sum, part) - sum;
#pragma unroll
  for (int e = 0; e < per; ++e) {
    const int b = threadIdx.x * per + e;
    if (b <= blocks) pre[b] = at;
    at += c[e];
  }
  if (threadIdx.x == kThreads - 1 && blocks == kMaxBlocks) pre[kMaxBlocks] = at;
  __syncthreads();
}

// Free pages below `page` (0 .. num_pages).
__device__ __forceinline__ uint32_t free_below(const Snapshot& s, const uint32_t* pre, int blocks,
                                               int page) {
  const int b = page / kBlockPages;
  if (b >= blocks) return pre[blocks];
  const int w = page >> 6;
  return pre[b] + s.before[w] + __popcll(s.words[w] & ((1ull << (page & 63)) - 1));
}

// The i-th free (FREE) or used page, counted from 0; i is below their number.
template <bool FREE>
__device__ __forceinline__ int select_page(const Snapshot& s, const uint32_t* pre, int blocks,
                                           uint32_t i) {
  auto before_block = [&](int b) { return FREE ? pre[b] : (uint32_t)b * kBlockPages - pre[b]; };
  int lo = 0, hi = blocks - 1;  // the last block with at most i of them before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (before_block(mid) <= i) lo = mid; else hi = mid - 1;
  }
  i -= before_block(lo);
  const uint32_t* wb = s.before + lo * 64;
  auto before_word = [&](int w) { return FREE ? wb[w] : (uint32_t)w * 64 - wb[w]; };
  int wl = 0, wh = 63;
  while (wl < wh) {
    const int mid = (wl + wh + 1) / 2;
    if (before_word(mid) <= i) wl = mid; else wh = mid - 1;
  }
  i -= before_word(wl);
  uint64_t bits = s.words[lo * 64 + wl];
  if (!FREE) bits = ~bits;
  // the i-th set bit: halve the range six times
  int at = 0;
#pragma unroll
  for (int width = 32; width > 0; width >>= 1) {
    const uint32_t c = __popcll((bits >> at) & ((1ull << width) - 1));
    if (i >= c) {
      i -= c;
      at += width;
    }
  }
  return (lo * 64 + wl) * 64 + (at & 63);
}

// --------------------------------------------------------- moving pages

struct Copier {
  uint8_t* base[4];
  int64_t layer_stride[4], page_stride[4];  // bytes
  int bytes[4];                             // of one page
  int slices[4];                            // running number of slices, [3] = per layer
  int layers;
};

Copier copier_of(const int8mm_kv& kv) {
  Copier c{};
  const int eb = kv.dtype == INT8MM_I8 ? 1 : 2;
  const int data = kv.kv_heads * kv.page_size * kv.head_dim * eb;
  const int scale = kv.dtype == INT8MM_I8 ? kv.kv_heads * kv.page_size * 4 : 0;
  void* base[4] = {kv.k, kv.v, kv.k_scale, kv.v_scale};
  const int64_t ls[4] = {kv.k_layer_stride * eb, kv.v_layer_stride * eb, kv.ks_layer_stride * 4, kv.vs_layer_stride * 4};
  const int64_t pgs[4] = {kv.k_page_stride * eb, kv.v_page_stride * eb, kv.ks_page_stride * 4, kv.vs_page_stride * 4};
  int at = 0;
  for (int i = 0; i < 4; ++i) {
    c.base[i] = static_cast<uint8_t*>(base[i]);
    c.layer_stride[i] = ls[i];
    c.page_stride[i] = pgs[i];
    c.bytes[i] = i < 2 ? data : scale;
    at += (c.bytes[i] + kSlice - 1) / kSlice;
    c.slices[i] = at;
  }
  c.layers = kv.layers;
  return c;
}

// Slice `at` (0 .. layers * slices[3] - 1) of page src to page dst, by one
// workgroup; at, src and dst are the same for all its threads.
__device__ __forceinline__ void copy_slice(const Copier& c, int at, int src, int dst) {
  const int layer = at / c.slices[3];
  const int sl = at % c.slices[3];
  uint8_t* base = nullptr;
  int64_t page_stride = 0;
  int size = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int first = i > 0 ? c.slices[i - 1] : 0;
    if (sl >= first && sl < c.slices[i]) {
      const int from = (sl - first) * kSlice;
      base = c.base[i] + layer * c.layer_stride[i] + from;
      page_stride = c.page_stride[i];
      size = min(kSlice, c.bytes[i] - from);
    }
  }
  const uint8_t* a = base + src * page_stride;
  uint8_t* b = base + dst * page_stride;
  constexpr uint32_t kStep = kThreads * 16;
  constexpr int kU = kSlice / kStep;  // 8 loads in flight
  const uint32_t e = threadIdx.x * 16u;
  if (size == kSlice) {  // (with a condition on each load they would wait for one another)
    v4u x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      x[u] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(a + (e + u * kStep)));
#pragma unroll
    for (int u = 0; u < kU; ++u)
      __builtin_nontemporal_store(x[u], reinterpret_cast<v4u*>(b + (e + u * kStep)));
  } else {
    for (uint32_t i = e; i < (uint32_t)size; i += kStep)
      __builtin_nontemporal_store(__builtin_nontemporal_load(reinterpret_cast<const v4u*>(a + i)),
                                  reinterpret_cast<v4u*>(b + i));
  }
}

__global__ __launch_bounds__(kThreads) void k_pages_copy(Copier c, const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst, int n,
                                                         int num_pages) {
  const int per = c.layers * c.slices[3];
  const int64_t total = (int64_t)n * per;
#pragma unroll 1
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int64_t k = w / per;
    const int a = __builtin_amdgcn_readfirstlane(src[k]), b = __builtin_amdgcn_readfirstlane(dst[k]);
    if ((unsigned)a < (unsigned)num_pages && (unsigned)b < (unsigned)num_pages && a != b)
      copy_slice(c, (int)(w - k * per), a, b);
  }
}

__global__ __launch_bounds__(kThreads) void k_pages_reserve(Rows r, Snapshot s, int blocks) {
  __shared__ uint32_t pre[kMaxBlocks + 1];
  __shared__ uint32_t part[kThreads / 64];
  load_prefix(s, blocks, pre, part);
  const int i = blockIdx.x;
  int st = s.plan[i];
  const uint32_t first = s.first[i], need = s.need[i];
  if (st == INT8MM_KV_DONE && need > 0 && sat_add(first, need) > pre[blocks]) st = INT8MM_KV_NO_PAGES;
  if (threadIdx.x == 0) r.status[i] = st;
  if (st != INT8MM_KV_DONE) return;
  const int row = r.a[i], want = r.b[i];
  const uint32_t have = (uint32_t)(((int64_t)r.lengths[row] + (1 << r.lps) - 1) >> r.lps);
  for (uint32_t j = threadIdx.x; j < need; j += kThreads) {
    const int page = select_page<true>(s, pre, blocks, first + j);
    r.table[(int64_t)row * r.table_width + have + j] = page;
    r.refcount[page] = 1;
  }
  __syncthreads();  // every thread has read the old length
  if (threadIdx.x == 0) r.lengths[row] = want;
}

// Workgroups of pair i: they share the `per` slices of the partly filled page,
// the first also writes the child's row.
__global__ __launch_bounds__(kThreads) void k_pages_fork(Rows r, Snapshot s, int blocks, Copier c,
                                                         int per) {
  __shared__ uint32_t pre[kMaxBlocks + 1];
  __shared__ uint32_t part[kThreads / 64];
  const int i = blockIdx.y, sl = blockIdx.x;
  int st = s.plan[i];
  const uint32_t first = s.first[i], need = s.need[i];
  int fresh = -1;
  if (st == INT8MM_KV_DONE && need > 0) {
    load_prefix(s, blocks, pre, part);
    if (first >= pre[blocks])
      st = INT8MM_KV_NO_PAGES;
    else
      fresh = __builtin_amdgcn_readfirstlane(select_page<true>(s, pre, blocks, first));
  }
  if (sl == 0 && threadIdx.x == 0) r.status[i] = st;
  if (st != INT8MM_KV_DONE) return;
  const int parent = r.a[i], child = r.b[i];
  const int len = r.lengths[parent], whole = len >> r.lps;  // a parent is no pair's child
  const int32_t* from = r.table + (int64_t)parent * r.table_width;
  int32_t* to = r.table + (int64_t)child * r.table_width;
  if (sl == 0) {
    for (int j = threadIdx.x; j < r.table_width; j += kThreads) {
      int page = -1;
      if (j < whole) {
        page = from[j];
        if ((unsigned)page < (unsigned)r.num_pages) atomicAdd(r.refcount + page, 1);
      } else if (j == whole) {
        page = fresh;
      }
      to[j] = page;
    }
    if (threadIdx.x == 0) {
      if (fresh >= 0) r.refcount[fresh] = 1;
      r.lengths[child] = len;
    }
  }
  if (fresh >= 0) {
    const int src = __builtin_amdgcn_readfirstlane(from[whole]);
#pragma unroll 1
    for (int w = sl; w < per; w += gridDim.x) copy_slice(c, w, src, fresh);
  }
}

__global__ __launch_bounds__(kThreads) void k_pages_free(Rows r) {
  const int row = r.a[blockIdx.x];
  if ((unsigned)row >= (unsigned)r.table_rows) return;
  int32_t* t = r.table + (int64_t)row * r.table_width;
  for (int j = threadIdx.x; j < r.table_width; j += kThreads) {
    // a row named twice: the exchange gives each entry to one workgroup
    const int page = atomicExch(t + j, -1);
    if ((unsigned)page < (unsigned)r.num_pages && atomicSub(r.refcount + page, 1) <= 0)
      atomicAdd(r.refcount + page, 1);  // it was free already
  }
  if (threadIdx.x == 0) r.lengths[row] = 0;
}

// With n_live used pages, hole k is the k-th free page below n_live and mover
// k the k-th used page at or above it; there are as many of one as of the other.
__global__ __launch_bounds__(kThreads) void k_pages_compact(
    const int32_t* table, int32_t* table_out, int64_t entries, const int32_t* ref,
    int32_t* ref_out, int num_pages, Snapshot s, int blocks, Copier c,
    int32_t* __restrict__ n_live) {
  __shared__ uint32_t pre[kMaxBlocks + 1];
  __shared__ uint32_t part[kThreads / 64];
  load_prefix(s, blocks, pre, part);
  const int live = num_pages - (int)pre[blocks];
  const uint32_t holes = free_below(s, pre, blocks, live);
  const uint32_t stay = (uint32_t)live - holes;  // used pages below n_live
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_live = live;

  // pages
  const int per = c.layers * c.slices[3];
  const int64_t total = (int64_t)holes * per;
  // each workgroup takes slices that follow one another: few pairs to find
  const int64_t each = (total + gridDim.x - 1) / gridDim.x;
  const int64_t w1 = min(total, (blockIdx.x + 1) * each);
  int64_t pair = -1;
  int src = 0, dst = 0;
#pragma unroll 1
  for (int64_t w = blockIdx.x * each; w < w1; ++w) {
    const int64_t k = w / per;
    if (k != pair) {
      pair = k;
      src = __builtin_amdgcn_readfirstlane(select_page<false>(s, pre, blocks, stay + (uint32_t)k));
      dst = __builtin_amdgcn_readfirstlane(select_page<true>(s, pre, blocks, (uint32_t)k));
    }
    copy_slice(c, (int)(w - k * per), src, dst);
  }

  const int64_t step = (int64_t)gridDim.x * kThreads;
  const int64_t me = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  // table entries
  for (int64_t e = me; e < entries; e += step) {
    int page = table[e];
    if ((unsigned)page >= (unsigned)num_pages) {
      page = -1;
    } else if (page >= live) {
      const bool used = ((s.words[page >> 6] >> (page & 63)) & 1) == 0;
      page = used ? select_page<true>(s, pre, blocks, (uint32_t)page - free_below(s, pre, blocks, page) - stay) : -1;
    }
    table_out[e] = page;
  }
  // counts: a hole's thread also clears its mover's, so that they may be
  // changed in place
  for (int64_t e = me; e < num_pages; e += step) {
    const int page = (int)e;
    const bool used = ((s.words[page >> 6] >> (page & 63)) & 1) == 0;
    if (page < live) {
      if (used) {
        ref_out[page] = ref[page];
      } else {
        const int from = select_page<false>(s, pre, blocks, stay + free_below(s, pre, blocks, page));
        ref_out[page] = ref[from];
        ref_out[from] = 0;
      }
    } else if (!used) {
      ref_out[page] = 0;
    }
  }
}

}  // namespace

size_t kv_pages_workspace(int64_t num_pages, int64_t n) {
  size_t total = 0;
  carve(nullptr, num_pages, n, &total);
  return total < 256 ? 256 : total;
}

hipError_t launch_kv_pages_copy(const int8mm_kv& kv, const int32_t* src, const int32_t* dst, int n,
                                hipStream_t s) {
  const Copier c = copier_of(kv);
  const int64_t work = (int64_t)n * c.layers * c.slices[3];
  hipLaunchKernelGGL(k_pages_copy, dim3((unsigned)(work < 65536 ? work : 65536)), dim3(kThreads), 0,
                     s, c, src, dst, n, kv.num_pages);
  return hipGetLastError();
}

hipError_t launch_kv_pages_reserve(int num_pages, int page_size, int32_t* table, int table_rows,
                                   int table_width, int32_t* lengths, int32_t* refcount,
                                   const int32_t* rows, const int32_t* new_lengths, int n,
                                   int32_t* status, void* ws, hipStream_t s) {
  const Snapshot sn = carve(ws, num_pages, n, nullptr);
  const int blocks = blocks_of(num_pages);
  const Rows r{table, lengths, refcount, rows, new_lengths, status,
               table_rows, table_width, n, num_pages, __builtin_ctz(page_size)};
  hipLaunchKernelGGL(k_pages_plan<false>, dim3(blocks + 1), dim3(kScanThreads), 0, s, r, sn);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_pages_reserve, dim3(n), dim3(kThreads), 0, s, r, sn, blocks);
  return hipGetLastError();
}

hipError_t launch_kv_pages_fork(const int8mm_kv& kv, int32_t* table, int table_rows,
                                int table_width, int32_t* lengths, int32_t* refcount,
                                const int32_t* parents, const int32_t* children, int n,
                                int32_t* status, void* ws, hipStream_t s) {
  const Snapshot sn = carve(ws, kv.num_pages, n, nullptr);
  const int blocks = blocks_of(kv.num_pages);
  const Rows r{table, lengths, refcount, parents, children, status,
               table_rows, table_width, n, kv.num_pages, __builtin_ctz(kv.page_size)};
  hipLaunchKernelGGL(k_pages_plan<true>, dim3(blocks + 1), dim3(kScanThreads), 0, s, r, sn);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const Copier c = copier_of(kv);
  const int per = c.layers * c.slices[3];
  hipLaunchKernelGGL(k_pages_fork, dim3((unsigned)(per < 65536 ? per : 65536), (unsigned)n),
                     dim3(kThreads), 0, s, r, sn, blocks, c, per);
  return hipGetLastError();
}

hipError_t launch_kv_pages_free(int num_pages, int32_t* table, int table_rows, int table_width,
                                int32_t* lengths, int32_t* refcount, const int32_t* rows, int n,
                                hipStream_t s) {
  const Rows r{table, lengths, refcount, rows, nullptr, nullptr,
               table_rows, table_width, n, num_pages, 0};
  hipLaunchKernelGGL(k_pages_free, dim3(n), dim3(kThreads), 0, s, r);
  return hipGetLastError();
}

hipError_t launch_kv_pages_compact(const int8mm_kv& kv, const int32_t* table, int32_t* table_out,
                                   int table_rows, int table_width, const int32_t* refcount,
                                   int32_t* refcount_out, int32_t* n_live, void* ws,
                                   hipStream_t s) {
  const Snapshot sn = carve(ws, kv.num_pages, 0, nullptr);
  const int blocks = blocks_of(kv.num_pages);
  if (blocks > 0) {
    hipLaunchKernelGGL(k_pages_scan, dim3(blocks), dim3(kScanThreads), 0, s, refcount, kv.num_pages,
                       sn);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_pages_compact, dim3(2048), dim3(kThreads), 0, s, table, table_out,
                     (int64_t)table_rows * table_width, refcount, refcount_out, kv.num_pages, sn,
                     blocks, copier_of(kv), n_live);
  return hipGetLastError();
}

}  // namespace i8mm
