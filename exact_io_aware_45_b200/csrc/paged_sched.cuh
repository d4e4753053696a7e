// Work division of the paged attention kernels, shared by the kernels that
// compute partial results and the kernel that joins them.
//
// A phase's items (row tiles of packed query rows over one key range) are laid
// end to end as W key tiles. CTA i of n takes tiles [x_i, x_{i+1}), x_i = i W / n:
// the load is even whatever the lengths are, and no length has to be known on
// the host. A cut closer than kSnap tiles to an item's end moves to that end,
// which spares partial results of a few tiles; n shrinks to W / kMinTiles for
// little work.
//
// An item that one CTA covers whole and that no other phase adds to is written
// to O and LSE directly. Otherwise each of its pieces goes to a slot of its
// own: the piece with the item's first tile to slot `item`, a piece that begins
// at CTA i's first tile to slot items + i.
#pragma once

#include "paged.h"

namespace fa {
namespace sched {

constexpr int kSnap = 4;
constexpr int kMinTiles = 8;

// Length of sequence b of the batch: 0 for a slot out of range.
__device__ __forceinline__ int slot_of(const PagedArgs& a, int b) {
  return a.seqs ? a.seqs[b] : b;
}
__device__ __forceinline__ int len_of(const PagedArgs& a, int b) {
  const int s = slot_of(a, b);
  if ((unsigned)s >= (unsigned)a.c.slots) return 0;
  return max(0, min(a.c.lens[s], a.c.width << a.c.page_log2));
}

// Keys [lo, hi) of sequence b that its queries can see behind the shared prefix
// (own phase), and its number of key tiles: at least one, so that every item
// has a CTA that writes its result.
__device__ __forceinline__ void own_keys(const PagedArgs& a, int len, int& lo, int& hi) {
  hi = len;
  lo = a.shared;
  // the window bound of the first query; in 64 bits, wl may be any int
  if (a.wl >= 0) lo = max((long long)lo, (long long)len - a.T - a.wl);
}
__device__ __forceinline__ int tiles_of(int lo, int hi, int tile) {
  return hi > lo ? (hi - 1) / tile - lo / tile + 1 : 1;
}

// Keys [lo, hi) that any query sees of the shared prefix, from the smallest and
// the largest length of the batch.
__device__ __forceinline__ void pre_keys(const PagedArgs& a, int least, int most, int& lo,
                                         int& hi) {
  lo = 0;
  hi = min(a.shared, most);
  if (a.wl >= 0) lo = max(0ll, min((long long)hi, (long long)least - a.T - a.wl));
}

// CTAs that take part, and the raw cut of CTA i.
__device__ __forceinline__ int ctas_of(int n, long long W) {
  return (int)max(1ll, min((long long)n, W / kMinTiles));
}
__device__ __forceinline__ long long raw_cut(int i, long long W, int n) { return i * W / n; }

// The cut x, moved to an end of its item [s, s + nt) when it lies close to one.
__device__ __forceinline__ long long snap(long long x, long long s, int nt) {
  if (x - s < kSnap) return s;
  if (s + nt - x < kSnap) return s + nt;
  return x;
}

// Pieces of the item [s, s + nt): CTAs first + 1 .. first + more begin inside it.
__device__ __forceinline__ void pieces_of(long long s, int nt, long long W, int n, int& first,
                                          int& more) {
  more = 0;
  first = 0;
  if (nt < 2 * kSnap) return;
  const long long a = s + kSnap, b = s + nt - kSnap;   // cuts in [a, b] stay inside
  first = (int)((a * n + W - 1) / W) - 1;              // floor(i W / n) >= a from first + 1 on
  more = max(0, (int)(((b + 1) * n + W - 1) / W) - 1 - first);   // ... and <= b up to there
}

// Where a walk over a CTA's tiles stands.
struct Walk {
  long long x;       // next tile
  long long s;       // first tile of the current item
  int b;             // sequence (own phase), 0 in the shared phase
  int item;          // (b * Hkv + h) * rt + row tile; (h * rt + row tile) in the shared phase
  int h, r;          // KV head and row tile
  int lo, hi;        // keys of the item
  int nt;            // tiles of the item
  int len;           // length of sequence b
};

// One piece of an item.
struct Piece {
  int h, b;          // KV head; sequence whose table names the keys
  int row0, rows;    // packed query rows ((b * T + t) * G + g)
  int lo, hi;        // keys in sight of any row
  int t0, t1;        // key tiles [t0, t1), in units of `tile` keys from key 0
  int slot;          // partial slot, or -1: write the result
};

// Per-block scratch of begin().
struct Scratch {
  long long warp[32];
  long long cut[2], start[2];
  int cut_b[2];
  int least[32], most[32];
};

// Finds this CTA's tiles [w.x, end) and sets up the walk; all `threads` threads
// of the block call it. Returns false if the CTA has none. Contains block barriers.
__device__ inline bool begin(const PagedArgs& a, const Phase& ph, bool pre, int cta, int threads,
                             Scratch& s, Walk& w, long long& end) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, warps = threads >> 5;
  const int per_b = pre ? 0 : a.c.Hkv * ph.rt;
  const int per = (a.B + threads - 1) / threads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long sum = 0;
  int least = 0x7fffffff, most = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = len_of(a, b);
    least = min(least, len);
    most = max(most, len);
    int lo, hi;
    own_keys(a, len, lo, hi);
    sum += (long long)tiles_of(lo, hi, ph.tile) * per_b;
  }
  long long x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  least = __reduce_min_sync(~0u, least);
  most = __reduce_max_sync(~0u, most);
  if (lane == 31) s.warp[wid] = x, s.least[wid] = least, s.most[wid] = most;
  __syncthreads();
  long long before = 0, W = 0;
  for (int i = 0; i < warps; ++i) {
    if (i < wid) before += s.warp[i];
    W += s.warp[i];
    least = min(least, s.least[i]);
    most = max(most, s.most[i]);
  }
  before += x - sum;
  if (pre) {
    int lo, hi;
    pre_keys(a, least, most, lo, hi);
    const int nt = tiles_of(lo, hi, ph.tile);
    W = (long long)ph.items * nt;
    const int n = ctas_of(ph.n, W);
    if (cta >= n) return false;
    long long c[2];
    for (int k = 0; k < 2; ++k) {
      const long long r = raw_cut(cta + k, W, n);
      const long long it = r / nt;
      c[k] = snap(r, it * nt, nt);
    }
    if (c[0] >= c[1]) return false;
    end = c[1];
    w.x = c[0];
    w.item = (int)(c[0] / nt);
    w.s = (long long)w.item * nt;
    w.b = 0;
    w.h = w.item / ph.rt;
    w.r = w.item - w.h * ph.rt;
    w.lo = lo;
    w.hi = hi;
    w.nt = nt;
    w.len = 0;
    return true;
  }
  const int n = ctas_of(ph.n, W);
  if (cta >= n) return false;
  // the thread whose sequences hold a cut places it
  for (int k = 0; k < 2; ++k) {
    const long long r = raw_cut(cta + k, W, n);
    const bool last = r == W;
    if (sum > 0 && r >= before && (r < before + sum || (last && before + sum == W))) {
      long long at = before;
      for (int b = b0; b < b1; ++b) {
        int lo, hi;
        own_keys(a, len_of(a, b), lo, hi);
        const int nt = tiles_of(lo, hi, ph.tile);
        const long long all = (long long)nt * per_b;
        if (r < at + all || (last && b == b1 - 1)) {
          const long long it = last ? per_b - 1 : (r - at) / nt;
          s.cut[k] = last ? W : snap(r, at + it * nt, nt);
          s.cut_b[k] = b;
          s.start[k] = at;
          break;
        }
        at += all;
      }
    }
  }
  __syncthreads();
  if (s.cut[0] >= s.cut[1]) return false;
  end = s.cut[1];
  w.x = s.cut[0];
  w.b = s.cut_b[0];
  long long at = s.start[0];
  w.len = len_of(a, w.b);
  own_keys(a, w.len, w.lo, w.hi);
  w.nt = tiles_of(w.lo, w.hi, ph.tile);
  if (w.x >= at + (long long)w.nt * per_b) {   // moved to the next sequence's first tile
    at += (long long)w.nt * per_b;
    ++w.b;
    w.len = len_of(a, w.b);
    own_keys(a, w.len, w.lo, w.hi);
    w.nt = tiles_of(w.lo, w.hi, ph.tile);
  }
  const int in = (int)((w.x - at) / w.nt);
  w.s = at + (long long)in * w.nt;
  w.h = in / ph.rt;
  w.r = in - w.h * ph.rt;
  w.item = w.b * per_b + in;
  return true;
}

// The next piece of the walk (w.x < end), which it moves past.
__device__ __forceinline__ Piece next(const PagedArgs& a, const Phase& ph, bool pre, int cta,
                                      long long end, Walk& w) {
  Piece p;
  p.h = w.h;
  p.b = w.b;
  p.lo = w.lo;
  p.hi = w.hi;
  const int all = pre ? a.B * a.TG : a.TG;
  p.row0 = w.r * ph.rows;
  p.rows = min(ph.rows, all - p.row0);
  if (!pre) p.row0 += w.b * a.TG;
  const int from = (int)(w.x - w.s);
  const int to = (int)min((long long)w.nt, end - w.s);
  const int base = w.lo / ph.tile;
  p.t0 = base + from;
  p.t1 = base + to;
  const bool whole = from == 0 && to == w.nt;
  p.slot = whole && a.shared == 0 ? -1 : (from == 0 ? w.item : ph.items + cta);
  w.x = w.s + to;
  if (w.x < end) {
    w.s = w.x;
    ++w.item;
    if (++w.r == ph.rt) {
      w.r = 0;
      if (++w.h == a.c.Hkv && !pre) {
        w.h = 0;
        ++w.b;
        w.len = len_of(a, w.b);
        own_keys(a, w.len, w.lo, w.hi);
        w.nt = tiles_of(w.lo, w.hi, ph.tile);
      }
    }
  }
  return p;
}

// Keys [lo, hi) that packed row r sees in the phase, and where it is in Q and O.
struct Row {
  int lo, hi;
  long long at;      // element offset of its d values
  long long lse;     // offset in LSE
};
__device__ __forceinline__ Row row_of(const PagedArgs& a, bool pre, int h, int r) {
  Row o;
  const int b = r / a.TG, q = r - b * a.TG, t = q / a.G, g = q - t * a.G;
  const int len = len_of(a, b);
  const int pos = len - a.T + t;
  o.lo = pre ? 0 : a.shared;
  o.hi = a.causal ? max(0, min(len, pos + 1)) : len;
  if (pre) o.hi = min(o.hi, a.shared);
  if (a.wl >= 0) o.lo = max((long long)o.lo, (long long)pos - a.wl);
  o.lse = ((long long)b * a.Hq + h * a.G + g) * a.T + t;
  o.at = o.lse * a.c.d;
  return o;
}

// Byte offset of key j (head h) in the layer's K or V, through a table row.
__device__ __forceinline__ long long key_offset(const CacheView& c, const int* trow, int h, int j) {
  int page = trow[j >> c.page_log2];
  if ((unsigned)page >= (unsigned)c.pages) page = 0;
  return page * c.page_stride + (long long)h * c.head_bytes +
         (long long)(j & ((1 << c.page_log2) - 1)) * c.row_bytes;
}

// The table row of a piece: the first sequence's in the shared phase.
__device__ __forceinline__ const int* table_row(const PagedArgs& a, int b) {
  int s = slot_of(a, b);
  if ((unsigned)s >= (unsigned)a.c.slots) s = 0;
  return a.c.table + (long long)s * a.c.width;
}

}  // namespace sched
}  // namespace fa
