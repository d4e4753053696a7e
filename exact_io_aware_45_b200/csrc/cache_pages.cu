// Pages of the paged key/value cache: growing, writing, forking, copying,
// freeing and compacting.
//
// Each operation is a plan and, where K and V move, a data kernel. The plan
// validates the whole list before anything changes (a refused call leaves the
// cache as it was) and hands out free pages lowest first, so its result does
// not depend on timing: with f_p = 1 for a free page p, the k-th new page is
// the p with f_p = 1 and sum_{q < p} f_q = k. Plans touch little data (4
// bytes a page, 4 bytes a table entry) and are bound by latency: a plan is one block, or for
// large pools one cluster of eight, which can synchronise between the steps of a plan
// without another launch and shares the scan over the pages through distributed shared
// memory.
//
// The data kernels move bytes and nothing else (16-byte loads and stores, 4 KB
// in flight a warp), bound by HBM: every byte is read once and written once.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "paged.h"

namespace cg = cooperative_groups;

namespace fa {
namespace {

constexpr int kPlanThreads = 512;

// The threads of a plan: kCtas blocks (one, or a cluster).
template <int kCtas>
struct Plan {
  static constexpr int kAll = kCtas * kPlanThreads;
  static __device__ int rank() { return kCtas > 1 ? (int)blockIdx.x : 0; }
  static __device__ int thread() { return rank() * kPlanThreads + threadIdx.x; }
  static __device__ void sync() {
    if constexpr (kCtas > 1) cg::this_cluster().sync();
    else __syncthreads();
  }
};

// Workspace of a plan, in int32 words: header, one bit per slot or page, one
// prefix sum per list entry, two page lists and a page map.
struct PlanWs {
  int* bad;      // [1] the call is refused
  int* count;    // [1] entries of the page lists
  unsigned* bits;
  int* at;       // [n + 1]
  int* from;     // [pages]
  int* to;       // [pages]
  int* map;      // [pages]
};

constexpr int kHeaderWords = 64;

__host__ __device__ inline int bit_words(int pages, int slots) {
  return ((pages > slots ? pages : slots) + 31) / 32;
}

PlanWs plan_ws(void* ws, int pages, int slots, int n) {
  int* w = static_cast<int*>(ws);
  PlanWs p;
  p.bad = w;
  p.count = w + 1;
  w += kHeaderWords;
  p.bits = reinterpret_cast<unsigned*>(w);
  w += bit_words(pages, slots);
  p.at = w;
  w += n + 1;
  p.from = w;
  p.to = w + pages;
  p.map = w + 2 * (size_t)pages;
  return p;
}

struct PlanShared {
  long long warp[kPlanThreads / 32];
  int mine;      // this CTA's count, read by the others through the cluster
};

// Exclusive prefix sum of v over the block; `total` is the block's sum.
template <class T>
__device__ T block_scan(T v, PlanShared& s, T& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s.warp[w] = x;
  __syncthreads();
  if (w == 0) {
    T y = lane < kPlanThreads / 32 ? (T)s.warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < kPlanThreads / 32; o <<= 1) {
      const T z = __shfl_up_sync(~0u, y, o);
      if (lane >= o) y += z;
    }
    if (lane < kPlanThreads / 32) s.warp[lane] = y;
  }
  __syncthreads();
  total = (T)s.warp[kPlanThreads / 32 - 1];
  return x - v + (w ? (T)s.warp[w - 1] : 0);
}

// Zeroes the header and the bits; everyone sees them afterwards.
template <class P>
__device__ void plan_begin(const PlanWs& p, int bits) {
  if (P::thread() == 0) *p.bad = 0, *p.count = 0;
  for (int i = P::thread(); i < bits; i += P::kAll) p.bits[i] = 0;
  P::sync();
}

// Sets bit i; true if it was set already.
__device__ __forceinline__ bool set_bit(unsigned* bits, int i) {
  return (atomicOr(bits + (i >> 5), 1u << (i & 31)) >> (i & 31)) & 1u;
}
__device__ __forceinline__ bool get_bit(const unsigned* bits, int i) {
  return (__ldcg(bits + (i >> 5)) >> (i & 31)) & 1u;
}

__device__ __forceinline__ bool in_range(int i, int n) { return (unsigned)i < (unsigned)n; }

// Calls emit(rank, i) for every i in [0, n) with pred(i), rank counting from 0 in
// the order of i, for ranks below `limit`; returns how many i there are. The
// whole plan takes part; each block has a contiguous part of the range.
template <int kCtas, class Pred, class Emit>
__device__ int plan_pick(int n, int limit, PlanShared& s, Pred pred, Emit emit) {
  using P = Plan<kCtas>;
  constexpr int kPer = 4;
  const int per = ((n + kCtas - 1) / kCtas + kPer - 1) / kPer * kPer;
  const int lo = min(n, P::rank() * per), hi = min(n, lo + per);
  int mine = 0;
#pragma unroll 4
  for (int i = lo + threadIdx.x; i < hi; i += kPlanThreads) mine += pred(i) ? 1 : 0;
  int total;
  block_scan(mine, s, total);
  int before = 0, all = total;
  if constexpr (kCtas > 1) {
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x == 0) s.mine = total;
    cl.sync();
    all = 0;
    for (int r = 0; r < kCtas; ++r) {
      const int v = *cl.map_shared_rank(&s.mine, r);
      if (r < P::rank()) before += v;
      all += v;
    }
    cl.sync();
  }
  for (int base = lo; base < hi && before < limit; base += kPlanThreads * kPer) {
    const int i0 = base + threadIdx.x * kPer;
    bool f[kPer];
    int c = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      f[j] = i0 + j < hi && pred(i0 + j);
      c += f[j] ? 1 : 0;
    }
    int rank = before + block_scan(c, s, total);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (f[j]) {
        if (rank < limit) emit(rank, i0 + j);
        ++rank;
      }
    before += total;
  }
  return all;
}

// at[i] = sum of need(i') for i' < i, at[n] = the sum of all, saturated at 2^30.
// The first block does it; the others meet it at the next barrier of the plan.
template <class P, class Need>
__device__ void list_scan(int n, int* at, PlanShared& s, Need need) {
  if (P::rank() == 0) {
    long long base = 0;                         // needs of a bad list may add up to anything
    for (int b = 0; b < n; b += kPlanThreads) {
      const int i = b + threadIdx.x;
      long long total;
      const long long x = block_scan<long long>(i < n ? need(i) : 0, s, total);
      if (i < n) at[i] = (int)min(base + x, 1ll << 30);
      base = min(base + total, 1ll << 30);
    }
    if (threadIdx.x == 0) at[n] = (int)base;
  }
}

__device__ __forceinline__ void refuse(const CacheView& c) { atomicOr(c.err, (unsigned)kErrCache); }

// ---------------------------------------------------------------- extend

__device__ __forceinline__ int new_tokens(const int* cu, int tokens, int i) {
  return cu ? cu[i + 1] - cu[i] : tokens;
}

template <int kCtas>
__global__ void __launch_bounds__(kPlanThreads)
    extend_kernel(CacheView c, const int* seqs, int n, const int* cu, int tokens, int* pos,
                  PlanWs p) {
  __shared__ PlanShared s;
  using P = Plan<kCtas>;
  const int t = P::thread();
  const int ps = 1 << c.page_log2;
  const long long most = (long long)c.width * ps;
  plan_begin<P>(p, bit_words(0, c.slots));
  // sequence i: its slot, length and new tokens; false if any is wrong
  auto get = [&](int i, int& slot, int& len, int& more) {
    slot = seqs[i];
    more = new_tokens(cu, tokens, i);
    if (!in_range(slot, c.slots) || more < 0) return false;
    len = c.lens[slot];
    return len >= 0 && (long long)len + more <= most;
  };
  auto need = [&](int i) {
    int slot, len, more;
    if (!get(i, slot, len, more)) return 0;
    return ((len + more + ps - 1) >> c.page_log2) - ((len + ps - 1) >> c.page_log2);
  };
  for (int i = t; i < n; i += P::kAll) {
    int slot, len, more;
    if (!get(i, slot, len, more) || set_bit(p.bits, slot)) *p.bad = 1;
  }
  list_scan<P>(n, p.at, s, need);
  P::sync();
  const int total = __ldcg(p.at + n);
  int found = 0;
  if (total > 0 && total <= c.pages)
    found = plan_pick<kCtas>(c.pages, total, s, [&](int i) { return __ldcg(c.refs + i) == 0; },
                         [&](int k, int i) { p.to[k] = i; });
  const bool bad = __ldcg(p.bad) || found < total;
  P::sync();   // the lists are complete, and everyone has read what follows changes
  if (bad) {
    for (int i = t; i < n; i += P::kAll) pos[i] = -1;
    if (t == 0) refuse(c);
    return;
  }
  for (int k = t; k < total; k += P::kAll) {
    int a = 0, b = n - 1;   // the sequence that the k-th new page belongs to
    while (a < b) {
      const int m = (a + b + 1) >> 1;
      if (__ldcg(p.at + m) <= k) a = m; else b = m - 1;
    }
    const int slot = seqs[a], page = __ldcg(p.to + k);
    const int have = (__ldcg(c.lens + slot) + ps - 1) >> c.page_log2;
    c.table[(size_t)slot * c.width + have + k - __ldcg(p.at + a)] = page;
    c.refs[page] = 1;
  }
  P::sync();
  for (int i = t; i < n; i += P::kAll) {
    const int slot = seqs[i], len = __ldcg(c.lens + slot);
    pos[i] = len;
    c.lens[slot] = len + new_tokens(cu, tokens, i);
  }
}

// ---------------------------------------------------------------- write

// One warp per token: its position follows from the list (a chain of five dependent
// loads, for which its data does not wait), then 16-byte pieces of its Hkv heads go to the
// heads' rows of the page. 76 MB of tokens take 28 us (5.4 TB/s read and written), the 48
// tokens of a decoding step 3.4 us (3.7 with the data's loads behind the chain).
__global__ void __launch_bounds__(256)
    write_kernel(CacheView c, char* lk, char* lv, const char* K, const char* V, const int* seqs,
                 const int* pos, int n, const int* cu, int total) {
  const int lane = threadIdx.x & 31;
  constexpr int kAtOnce = 4;                          // loads of K and of V a lane in flight
  const int row_vecs = c.row_bytes >> 4;              // 16-byte pieces of a head's row (2^n)
  const int row_log2 = 31 - __clz(row_vecs);
  const int vecs = c.Hkv * row_vecs;
  const int ps_mask = (1 << c.page_log2) - 1;
  const unsigned warps = gridDim.x * (blockDim.x >> 5);
  // (unsigned: the last step may pass 2^31)
  for (unsigned row = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); row < (unsigned)total;
       row += warps) {
    const int r = (int)row;
    const int4* k = reinterpret_cast<const int4*>(K + (size_t)r * c.Hkv * c.row_bytes);
    const int4* v = reinterpret_cast<const int4*>(V + (size_t)r * c.Hkv * c.row_bytes);
    int4 x[kAtOnce], y[kAtOnce];
    auto load = [&](int v0) {
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e)
        if (v0 + 32 * e < vecs) x[e] = __ldcs(k + v0 + 32 * e), y[e] = __ldcs(v + v0 + 32 * e);
    };
    load(lane);                                       // on its way while the place is looked up
    int i, j;
    if (cu) {
      int a = 0, b = n - 1;                           // the last sequence that begins at or before r
      while (a < b) {
        const int m = (a + b + 1) >> 1;
        if (cu[m] <= r) a = m; else b = m - 1;
      }
      i = a;
      j = r - cu[a];
      if (j < 0 || r >= cu[a + 1]) continue;          // no sequence's row
    } else {
      const int each = total / n;
      i = r / each;
      j = r - i * each;
    }
    const int p0 = pos[i];
    if (p0 < 0) continue;
    const int slot = seqs[i];
    bool ok = in_range(slot, c.slots) && j <= 0x7fffffff - p0;
    const int at = p0 + j;
    int page = -1;
    if (ok) ok = at < c.lens[slot] && (at >> c.page_log2) < c.width;
    if (ok) {
      page = c.table[(size_t)slot * c.width + (at >> c.page_log2)];
      ok = in_range(page, c.pages) && c.refs[page] == 1;
    }
    if (!ok) {
      if (lane == 0) refuse(c);
      continue;
    }
    const size_t dst0 = (size_t)page * c.page_stride + (size_t)(at & ps_mask) * c.row_bytes;
    for (int v0 = lane; v0 < vecs; v0 += 32 * kAtOnce) {
      if (v0 != lane) load(v0);
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const int i = v0 + 32 * e;
        if (i < vecs) {
          const int h = i >> row_log2;
          const size_t dst = dst0 + (size_t)h * c.head_bytes + (size_t)(i & (row_vecs - 1)) * 16;
          *reinterpret_cast<int4*>(lk + dst) = x[e];
          *reinterpret_cast<int4*>(lv + dst) = y[e];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- page data

// Copies pages from[k] -> to[k] for k < *count in all layers of K and V: a warp
// takes 4 KB pieces, eight 16-byte loads a lane in flight.
__device__ void copy_pages(const CacheView& c, const int* from, const int* to, int count) {
  constexpr int kPiece = 4096;
  const int lane = threadIdx.x & 31;
  const int pieces = (c.page_bytes + kPiece - 1) / kPiece;
  const long long units = (long long)count * c.layers * 2 * pieces;
  const int per_block = blockDim.x >> 5;
  const long long warps = (long long)gridDim.x * per_block;
  for (long long u = (long long)blockIdx.x * per_block + (threadIdx.x >> 5); u < units;
       u += warps) {
    const long long q = u / pieces;
    const int piece = (int)(u - q * pieces);
    const long long pair = q >> 1;                    // (layer, k), k fastest
    const int layer = (int)(pair / count);
    const int k = (int)(pair - (long long)layer * count);
    const int a = from[k], b = to[k];
    if (!in_range(a, c.pages) || !in_range(b, c.pages) || a == b) continue;
    char* base = ((q & 1) ? c.V : c.K) + layer * c.layer_stride + (size_t)piece * kPiece;
    const int4* src = reinterpret_cast<const int4*>(base + a * c.page_stride);
    int4* dst = reinterpret_cast<int4*>(base + b * c.page_stride);
    const int left = (min(kPiece, c.page_bytes - piece * kPiece)) >> 4;
    int4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < left) x[i] = __ldcs(src + lane + 32 * i);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < left) __stcs(dst + lane + 32 * i, x[i]);
  }
}

__global__ void __launch_bounds__(256) copy_kernel(CacheView c, PlanWs p, const int* from,
                                                   const int* to, int n) {
  chain_wait();
  if (*p.bad) return;
  copy_pages(c, from, to, n);
}

// ---------------------------------------------------------------- fork

template <int kCtas>
__global__ void __launch_bounds__(kPlanThreads)
    fork_plan_kernel(CacheView c, const int* src, const int* dst, int n, PlanWs p) {
  chain_next();
  __shared__ PlanShared s;
  using P = Plan<kCtas>;
  const int t = P::thread();
  const int ps = 1 << c.page_log2;
  const long long most = (long long)c.width * ps;
  plan_begin<P>(p, bit_words(0, c.slots));
  for (int i = t; i < n; i += P::kAll) {
    const int d = dst[i];
    if (!in_range(d, c.slots) || set_bit(p.bits, d) || c.lens[d] != 0) *p.bad = 1;
  }
  P::sync();
  // a partly filled last page needs a copy of its own
  auto need = [&](int i) {
    const int a = src[i];
    return in_range(a, c.slots) && (c.lens[a] & (ps - 1)) ? 1 : 0;
  };
  for (int i = t; i < n; i += P::kAll) {
    const int a = src[i];
    if (!in_range(a, c.slots) || get_bit(p.bits, a) || c.lens[a] < 0 || c.lens[a] > most)
      *p.bad = 1;
  }
  list_scan<P>(n, p.at, s, need);
  P::sync();
  const int total = __ldcg(p.at + n);
  int found = 0;
  if (total > 0 && total <= c.pages)
    found = plan_pick<kCtas>(c.pages, total, s, [&](int i) { return c.refs[i] == 0; },
                         [&](int k, int i) { p.to[k] = i; });
  if (!__ldcg(p.bad) && found >= total) {
    for (int i = t; i < n; i += P::kAll)
      if (need(i)) {
        const int a = src[i];
        p.from[p.at[i]] = c.table[(size_t)a * c.width + (c.lens[a] >> c.page_log2)];
      }
    if (t == 0) *p.count = total;
  } else {
    P::sync();   // every CTA has read `bad` before it is set for want of pages
    if (t == 0) {
      *p.bad = 1;
      refuse(c);
    }
    return;
  }
  P::sync();
}

__global__ void __launch_bounds__(256)
    fork_kernel(CacheView c, const int* src, const int* dst, int n, PlanWs p) {
  chain_wait();
  if (*p.bad) return;
  const int ps = 1 << c.page_log2;
  const long long all = (long long)gridDim.x * blockDim.x;
  const long long entries = (long long)n * c.width;
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < entries; e += all) {
    const int i = (int)(e / c.width), w = (int)(e - (long long)i * c.width);
    const int a = src[i], d = dst[i], len = c.lens[a];
    const int full = len >> c.page_log2;
    int page = -1;
    if (w < full) {
      page = c.table[(size_t)a * c.width + w];
      if (in_range(page, c.pages)) atomicAdd(c.refs + page, 1);
    } else if (w == full && (len & (ps - 1))) {
      page = p.to[p.at[i]];
      c.refs[page] = 1;
    }
    c.table[(size_t)d * c.width + w] = page;
    if (w == 0) c.lens[d] = len;
  }
  copy_pages(c, p.from, p.to, *p.count);
}

// ---------------------------------------------------------------- free

template <int kCtas>
__global__ void __launch_bounds__(kPlanThreads)
    free_kernel(CacheView c, const int* seqs, int n, PlanWs p) {
  using P = Plan<kCtas>;
  const int t = P::thread();
  plan_begin<P>(p, bit_words(0, c.slots));
  for (int i = t; i < n; i += P::kAll) {
    const int slot = seqs[i];
    if (!in_range(slot, c.slots) || set_bit(p.bits, slot)) *p.bad = 1;
  }
  P::sync();
  if (__ldcg(p.bad)) {
    if (t == 0) refuse(c);
    return;
  }
  const long long entries = (long long)n * c.width;
  for (long long e = t; e < entries; e += P::kAll) {
    const int i = (int)(e / c.width), w = (int)(e - (long long)i * c.width);
    const int slot = seqs[i];
    int* at = c.table + (size_t)slot * c.width + w;
    const int page = *at;
    if (in_range(page, c.pages)) atomicSub(c.refs + page, 1);
    if (page != -1) *at = -1;
    if (w == 0) c.lens[slot] = 0;
  }
}

// ---------------------------------------------------------------- copy

template <int kCtas>
__global__ void __launch_bounds__(kPlanThreads)
    copy_plan_kernel(CacheView c, const int* src, const int* dst, int n, PlanWs p) {
  chain_next();
  using P = Plan<kCtas>;
  const int t = P::thread();
  plan_begin<P>(p, bit_words(c.pages, 0));
  for (int i = t; i < n; i += P::kAll) {
    const int d = dst[i];
    if (!in_range(d, c.pages) || set_bit(p.bits, d)) *p.bad = 1;
  }
  P::sync();
  for (int i = t; i < n; i += P::kAll) {
    const int a = src[i];
    if (!in_range(a, c.pages) || get_bit(p.bits, a)) *p.bad = 1;
  }
  P::sync();
  if (t == 0 && __ldcg(p.bad)) refuse(c);
}

// ---------------------------------------------------------------- compact

template <int kCtas>
__global__ void __launch_bounds__(kPlanThreads)
    compact_plan_kernel(CacheView c, PlanWs p) {
  chain_next();
  __shared__ PlanShared s;
  using P = Plan<kCtas>;
  const int t = P::thread();
  plan_begin<P>(p, 0);
  const int live = plan_pick<kCtas>(c.pages, 0, s, [&](int i) { return c.refs[i] > 0; },
                                [](int, int) {});
  // as many pages in use lie behind the first `live` as there are holes among them
  const int moves = plan_pick<kCtas>(c.pages, c.pages, s,
                                 [&](int i) { return i >= live && c.refs[i] > 0; },
                                 [&](int k, int i) { p.from[k] = i; });
  plan_pick<kCtas>(c.pages, c.pages, s, [&](int i) { return i < live && c.refs[i] <= 0; },
               [&](int k, int i) { p.to[k] = i; });
  for (int i = t; i < c.pages; i += P::kAll) p.map[i] = i;
  P::sync();
  for (int k = t; k < moves; k += P::kAll) {
    const int a = __ldcg(p.from + k), b = __ldcg(p.to + k);
    p.map[a] = b;
    c.refs[b] = c.refs[a];
    c.refs[a] = 0;
  }
  if (t == 0) *p.count = moves;
}

__global__ void __launch_bounds__(256) compact_kernel(CacheView c, PlanWs p) {
  chain_wait();
  const int count = *p.count;
  if (count == 0) return;
  const long long all = (long long)gridDim.x * blockDim.x;
  const long long entries = (long long)c.slots * c.width;
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < entries; e += all) {
    const int page = c.table[e];
    if (in_range(page, c.pages)) {
      const int to = p.map[page];
      if (to != page) c.table[e] = to;
    }
  }
  copy_pages(c, p.from, p.to, count);
}

// Enough blocks of 256 threads to fill the device, fewer for little work.
int data_blocks(long long threads) {
  const long long b = (threads + 255) / 256, most = 8ll * sm_count();
  return (int)(b < 1 ? 1 : (b > most ? most : b));
}

// Threads that copying n pages in all layers keeps busy (128 bytes a thread).
long long copy_threads(const CacheView& c, long long n) {
  return n * c.layers * 2 * ((c.page_bytes + 127) / 128);
}

cudaError_t done() {
  count_launch();
  return cudaGetLastError();
}

// Launches a plan over `work` pages. One block passes its barriers faster, eight read
// more at a time: an extend takes 6.0 and 8.6 us over 1,000 pages, 9.0 and 9.3 over 8,000, 16
// and 11 over 32,000. Freeing goes over table entries, with an atomic and a store each:
// 5.4 and 3.3 us for 4,096 of them, so they count four times.
template <class... A, class... B>
cudaError_t launch_plan(long long work, cudaStream_t st, void (*one)(A...), void (*eight)(A...),
                        B... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 8;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  const bool large = work > 8192;
  cfg.gridDim = dim3(large ? 8 : 1);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = large ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, large ? eight : one, static_cast<A>(args)...);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

size_t cache_workspace_bytes(int pages, int slots, int n) {
  return 4 * ((size_t)kHeaderWords + bit_words(pages, slots) + (size_t)n + 1 +
              3 * (size_t)pages);
}

cudaError_t cache_extend(const CacheView& c, const int* seqs, int n, const int* cu, int tokens,
                         int* pos, void* ws, cudaStream_t st) {
  return launch_plan(c.pages, st, extend_kernel<1>, extend_kernel<8>, c, seqs, n, cu, tokens, pos,
                     plan_ws(ws, c.pages, c.slots, n));
}

cudaError_t cache_write(const CacheView& c, int layer, const void* K, const void* V,
                        const int* seqs, const int* pos, int n, const int* cu, int total,
                        cudaStream_t st) {
  char* lk = c.K + layer * c.layer_stride;
  char* lv = c.V + layer * c.layer_stride;
  write_kernel<<<data_blocks((long long)total * 32), 256, 0, st>>>(
      c, lk, lv, static_cast<const char*>(K), static_cast<const char*>(V), seqs, pos, n, cu,
      total);
  return done();
}

cudaError_t cache_fork(const CacheView& c, const int* src, const int* dst, int n, void* ws,
                       cudaStream_t st) {
  const PlanWs p = plan_ws(ws, c.pages, c.slots, n);
  if (cudaError_t e = launch_plan(c.pages, st, fork_plan_kernel<1>, fork_plan_kernel<8>, c, src,
                                  dst, n, p))
    return e;
  const long long entries = (long long)n * c.width, copies = copy_threads(c, n);
  return launch_chained(fork_kernel, data_blocks(entries > copies ? entries : copies), 256, 0, st,
                        true, c, src, dst, n, p);
}

cudaError_t cache_free(const CacheView& c, const int* seqs, int n, void* ws, cudaStream_t st) {
  return launch_plan(4ll * n * c.width, st, free_kernel<1>, free_kernel<8>, c, seqs, n,
                     plan_ws(ws, c.pages, c.slots, n));
}

cudaError_t cache_copy(const CacheView& c, const int* src, const int* dst, int n, void* ws,
                       cudaStream_t st) {
  const PlanWs p = plan_ws(ws, c.pages, c.slots, n);
  if (cudaError_t e = launch_plan(n, st, copy_plan_kernel<1>, copy_plan_kernel<8>, c, src, dst, n,
                                  p))
    return e;
  return launch_chained(copy_kernel, data_blocks(copy_threads(c, n)), 256, 0, st, true, c, p, src,
                        dst, n);
}

cudaError_t cache_compact(const CacheView& c, void* ws, cudaStream_t st) {
  const PlanWs p = plan_ws(ws, c.pages, c.slots, 0);
  if (cudaError_t e = launch_plan(c.pages, st, compact_plan_kernel<1>, compact_plan_kernel<8>, c, p))
    return e;
  const long long entries = (long long)c.slots * c.width, copies = copy_threads(c, c.pages);
  return launch_chained(compact_kernel, data_blocks(entries > copies ? entries : copies), 256, 0,
                        st, true, c, p);
}

}  // namespace fa
