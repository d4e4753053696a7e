// Work division of the paged attention kernels, shared by the kernels that
// compute partial results and the kernel that joins them.
//
// A phase's items (row tiles of packed query rows over one key range) are laid
// end to end as W units: Phase::over for an item's set-up and result, then one for each
// key tile. Stream i of n (a warp, or a block) takes units [x_i, x_{i+1}), all
// streams as even as whole units allow: the load does not depend on how the
// lengths are spread, and no length has to be known on the host. A cut in an item's first
// `over` units or closer than `snap` tiles to either end moves to that end, which
// spares partial results of a few tiles; n shrinks to W / `least` for little work.
//
// An item that one stream covers whole and that no other phase adds to is written
// to O and LSE directly. Otherwise each of its pieces goes to a slot of its
// own: the piece with the item's first tile to slot `item`, a piece that begins
// with stream i's first tile to slot items + i.
//
// The packed rows of a sequence and KV head are (g, t), t fastest: contiguous in Q
// and O. Units fit an int (checked on the host).
#pragma once

#include "paged.h"

namespace fa {
namespace sched {

// Length of sequence b of the batch: 0 for a slot out of range.
__device__ __forceinline__ int slot_of(const PagedArgs& a, int b) {
  return a.seqs ? __ldg(a.seqs + b) : b;
}
__device__ __forceinline__ int len_at(const PagedArgs& a, int s) {
  if ((unsigned)s >= (unsigned)a.c.slots) return 0;
  return max(0, min(__ldg(a.c.lens + s), a.c.width << a.c.page_log2));
}
__device__ __forceinline__ int len_of(const PagedArgs& a, int b) {
  return len_at(a, slot_of(a, b));
}

// Keys [lo, hi) of a sequence that its queries can see behind the shared prefix
// (own phase), and units of an item over them: one tile at least, so that every
// item has a stream that writes its result.
__device__ __forceinline__ void own_keys(const PagedArgs& a, int len, int& lo, int& hi) {
  hi = len;
  lo = a.shared;
  // the window bound of the first query; in 64 bits, wl may be any int
  if (a.wl >= 0) lo = max((long long)lo, (long long)len - a.T - a.wl);
}
__device__ __forceinline__ int units_of(const Phase& ph, int lo, int hi) {
  return ph.over + (hi > lo ? ((hi - 1) >> ph.tile_log2) - (lo >> ph.tile_log2) + 1 : 1);
}
__device__ __forceinline__ int own_units(const PagedArgs& a, int len) {
  int lo, hi;
  own_keys(a, len, lo, hi);
  return units_of(a.own, lo, hi);
}

// Keys [lo, hi) that any query sees of the shared prefix, from the smallest and
// the largest length of the sequences that are not empty.
__device__ __forceinline__ void pre_keys(const PagedArgs& a, int least, int most, int& lo,
                                         int& hi) {
  lo = 0;
  hi = min(a.shared, most);
  if (a.wl >= 0) lo = max(0ll, min((long long)hi, (long long)least - a.T - a.wl));
}

// W units in n even ranges: the first `extra` are one longer.
struct Cuts {
  int W, n, each, extra;
  // `beside`: units of the own phase, when this is the shared one
  __device__ Cuts(const Phase& ph, int units, int beside = 0) : W(units) {
    n = W >= ph.n * ph.least ? ph.n : max(1, W / ph.least);
    // leaves the own phase, which runs beside it, the SMs that let both end together; in
    // fp32, rounded alike in every kernel (a 64-bit division took 0.5 us more)
    if (ph.yield) {
      const float all = __fmaf_rn((float)beside, __frcp_rn((float)ph.yield), (float)W);
      n = max(1, min(n, (int)__fdiv_rn(__fmul_rn((float)ph.sms, (float)W), all)));
    }
    each = W / n;
    extra = W - each * n;
  }
  // where range i begins
  __device__ int at(int i) const { return i * each + min(i, extra); }
  // the first cut at x or behind
  __device__ int first(int x) const {
    const int y = x - extra * (each + 1);
    return y <= 0 ? (x + each) / (each + 1) : extra + (y + each - 1) / each;
  }
};

// The cut x, moved to an end of its item [s, s + u) when it lies close to one.
__device__ __forceinline__ int snap(const Phase& ph, int x, int s, int u) {
  if (x - s < ph.over + ph.snap) return s;
  if (s + u - x < ph.snap) return s + u;
  return x;
}

// Pieces of the item [s, s + u): streams first + 1 .. first + more begin inside it.
__device__ __forceinline__ void pieces_of(const Phase& ph, int s, int u, const Cuts& c, int& first,
                                          int& more) {
  const int a = s + ph.over + ph.snap, b = s + u - ph.snap;   // cuts in [a, b] stay inside
  first = more = 0;
  if (b < a) return;
  first = c.first(a) - 1;
  more = c.first(b + 1) - 1 - first;
}

// The batch as one warp sees it: units of all sequences, those before sequence
// `b`, the smallest and the largest length, and that of b. All lanes call it.
struct Batch {
  int W, before, least, most, len;   // (least: of the sequences that are not empty)
  int lead;          // the first sequence that reaches farthest into the shared prefix
  int lane_len;      // of sequence `lane`
};
__device__ __forceinline__ Batch scan_batch(const PagedArgs& a, int b) {
  Batch t{0, 0, 0x7fffffff, 0, 0, 0, 0};
  int reach = -1;
  const int per_b = a.c.Hkv * a.own.rt, lane = threadIdx.x & 31;
  constexpr int kAtOnce = 4;                      // dependent loads in flight per lane
  for (int i0 = lane; i0 < a.B; i0 += 32 * kAtOnce) {
    int slot[kAtOnce], len[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) slot[k] = i0 + 32 * k < a.B ? slot_of(a, i0 + 32 * k) : -1;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) len[k] = len_at(a, slot[k]);
    if (i0 == lane) t.lane_len = len[0];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + 32 * k;
      if (i >= a.B) break;
      const int u = own_units(a, len[k]) * per_b;
      t.W += u;
      if (i < b) t.before += u;
      if (i == b) t.len = len[k];
      if (len[k] > 0) t.least = min(t.least, len[k]);
      const int into = min(len[k], a.shared);
      if (into > reach) reach = into, t.lead = i;
      t.most = max(t.most, len[k]);
    }
  }
  t.W = __reduce_add_sync(~0u, t.W);
  t.before = __reduce_add_sync(~0u, t.before);
  t.least = __reduce_min_sync(~0u, t.least);
  t.most = __reduce_max_sync(~0u, t.most);
  t.lead = __reduce_min_sync(~0u, reach == __reduce_max_sync(~0u, reach) ? t.lead : 0x7fffffff);
  t.len = __reduce_max_sync(~0u, t.len);
  return t;
}

// A stream's way through its units.
struct Walk {
  int x, end;        // next unit, and the first that is not its own
  int stream;
  int s, u;          // first unit and units of the current item
  int item;          // (b * Hkv + h) * rt + row tile; (h * rt + row tile) in the shared phase
  int b, h, r;       // sequence (own phase), KV head, row tile
  int lo, hi;        // keys of the item
  int slot, len;     // of sequence b; the leading sequence's slot in the shared phase, where len
                     // says whether there may be keys in [lo, hi) that no query sees
  int slot1, len1;   // of the next sequence, and the slot after it: loaded ahead, since a
  int slot2;         // chain of loads per sequence would stall short ones
};

__device__ __forceinline__ int slot_ahead(const PagedArgs& a, int b) {
  return b < a.B ? slot_of(a, b) : -1;
}
__device__ __forceinline__ void enter(const PagedArgs& a, int b, Walk& w) {
  w.b = b;
  w.slot = slot_of(a, b);
  w.slot1 = slot_ahead(a, b + 1);
  w.slot2 = slot_ahead(a, b + 2);
  w.len = len_at(a, w.slot);
  w.len1 = len_at(a, w.slot1);
  own_keys(a, w.len, w.lo, w.hi);
  w.u = units_of(a.own, w.lo, w.hi);
}
__device__ __forceinline__ void advance(const PagedArgs& a, Walk& w) {
  ++w.b;
  w.slot = w.slot1;
  w.len = w.len1;
  w.slot1 = w.slot2;
  w.len1 = len_at(a, w.slot1);
  w.slot2 = slot_ahead(a, w.b + 2);
  own_keys(a, w.len, w.lo, w.hi);
  w.u = units_of(a.own, w.lo, w.hi);
}

// Sets up the walk of a stream; all lanes of a warp call it and get the same.
// Returns false if the stream has no units.
__device__ inline bool begin(const PagedArgs& a, bool pre, int i, Walk& w) {
  const int lane = threadIdx.x & 31;
  const Batch t = scan_batch(a, 0);
  w.stream = i;
  if (pre) {
    pre_keys(a, t.least, t.most, w.lo, w.hi);
    // windows of sequences that all reach behind the prefix lie within one another, others may
    // leave keys between them
    w.len = a.wl >= 0 && t.least < w.hi;
    w.u = units_of(a.pre, w.lo, w.hi);
    const Cuts c(a.pre, a.pre.items * w.u, t.W);
    if (i >= c.n) return false;
    const int x0 = c.at(i), x1 = c.at(i + 1);
    w.item = x0 / w.u;
    w.x = snap(a.pre, x0, w.item * w.u, w.u);
    w.end = x1 == c.W ? c.W : snap(a.pre, x1, x1 / w.u * w.u, w.u);
    if (w.x >= w.end) return false;
    if (w.x >= (w.item + 1) * w.u) ++w.item;
    w.s = w.item * w.u;
    w.h = w.item / a.pre.rt;
    w.r = w.item - w.h * a.pre.rt;
    w.b = 0;
    w.slot = slot_of(a, t.lead);   // its table names all of the prefix that is in sight (the
                                   // first sequence may be padding, or shorter)
    return true;
  }
  const Cuts c(a.own, t.W);
  if (i >= c.n) return false;
  const int per_b = a.c.Hkv * a.own.rt;
  const int x0 = c.at(i), x1 = c.at(i + 1);
  int at0 = 0, b0 = -1, base = 0;
  w.end = x1 == c.W ? c.W : -1;
  for (int g = 0; g < a.B && (b0 < 0 || w.end < 0); g += 32) {
    const int u = g + lane < a.B ? own_units(a, g ? len_of(a, g + lane) : t.lane_len) : 0;
    int to = u * per_b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, to, o);
      if (lane >= o) to += y;
    }
    to += base;                                   // units up to and with this sequence
    const int from = to - u * per_b;
    const unsigned has0 = __ballot_sync(~0u, x0 >= from && x0 < to);
    const unsigned has1 = __ballot_sync(~0u, x1 >= from && x1 < to);
    if (has0) {
      const int k = __ffs(has0) - 1;
      b0 = g + k;
      at0 = __shfl_sync(~0u, from, k);
      const int v = __shfl_sync(~0u, u, k);
      w.x = snap(a.own, x0, at0 + (x0 - at0) / v * v, v);
    }
    if (has1) {
      const int k = __ffs(has1) - 1;
      const int f = __shfl_sync(~0u, from, k), v = __shfl_sync(~0u, u, k);
      w.end = snap(a.own, x1, f + (x1 - f) / v * v, v);
    }
    base = __shfl_sync(~0u, to, 31);
  }
  if (w.x >= w.end) return false;
  enter(a, b0, w);
  if (w.x >= at0 + w.u * per_b) {                 // moved to the next sequence's first unit
    at0 += w.u * per_b;
    advance(a, w);
  }
  const int in = (w.x - at0) / w.u;
  w.s = at0 + in * w.u;
  w.h = in / a.own.rt;
  w.r = in - w.h * a.own.rt;
  w.item = w.b * per_b + in;
  return true;
}

// One piece of an item.
struct Piece {
  int h;             // KV head
  int b, len;        // sequence and its length (own phase), or whether there may be gaps (shared)
  int table;         // slot whose table names the keys (the leading one's in the shared phase)
  int row0, rows;    // rows: (g, t) of sequence b, or (b, g, t) in the shared phase
  int lo, hi;        // keys in sight of any row
  int t0, t1;        // key tiles [t0, t1), counted from key 0
  int slot;          // partial slot, or -1: write the result
};

// The next piece of the walk (w.x < w.end), which it moves past.
__device__ __forceinline__ Piece next(const PagedArgs& a, bool pre, Walk& w) {
  const Phase& ph = pre ? a.pre : a.own;
  Piece p;
  p.h = w.h;
  p.b = w.b;
  p.len = w.len;
  p.table = w.slot;
  p.lo = w.lo;
  p.hi = w.hi;
  p.row0 = w.r * ph.rows;
  p.rows = min(ph.rows, (pre ? a.B * a.TG : a.TG) - p.row0);
  const int from = w.x - w.s, to = min(w.u, w.end - w.s);
  const int base = w.lo >> ph.tile_log2;
  p.t0 = base + max(0, from - ph.over);
  p.t1 = base + to - ph.over;
  const bool alone = from == 0 && to == w.u && a.shared == 0;
  p.slot = alone ? -1 : (from == 0 ? w.item : ph.items + w.stream);
  w.x = w.s + to;
  if (w.x < w.end) {
    w.s = w.x;
    ++w.item;
    if (++w.r == ph.rt) {
      w.r = 0;
      if (++w.h == a.c.Hkv && !pre) {
        w.h = 0;
        advance(a, w);
      }
    }
  }
  return p;
}

// Bits f .. e - 1 of a word, as far as they lie in it.
__device__ __forceinline__ unsigned bits_of(int f, int e) {
  f = max(f, 0), e = min(e, 32);
  return f < e ? (~0u >> (32 - (e - f))) << f : 0u;
}
// Of the keys j0 .. j0 + 31 those of a piece's range that some query sees, one bit each: the others
// may hold anything, and a V row that is not finite would spread through weights of 0. All lanes
// call it. Where there may be gaps it goes through the batch once.
__device__ __forceinline__ unsigned seen_of(const PagedArgs& a, const Piece& p, int j0,
                                            bool gaps) {
  unsigned m = ~0u;
  if (gaps) {
    m = 0;
    for (int b = threadIdx.x & 31; b < a.B; b += 32) {
      const int len = len_of(a, b);
      const int lo = max(0ll, (long long)len - a.T - a.wl);
      if (len > 0) m |= bits_of(lo - j0, min(len, a.shared) - j0);
    }
    m = __reduce_or_sync(~0u, m);
  }
  return m & bits_of(p.lo - j0, p.hi - j0);
}

// Keys [lo, hi) that a packed row sees in the phase, and its index in LSE (and,
// times d, in Q and O).
struct Row {
  int lo, hi, out;
};
__device__ __forceinline__ Row row_at(const PagedArgs& a, bool pre, int h, int b, int q, int len) {
  Row o;
  const int pos = len - a.T + q % a.T;
  o.lo = pre ? 0 : a.shared;
  o.hi = a.causal ? max(0, min(len, pos + 1)) : len;
  if (pre) o.hi = min(o.hi, a.shared);
  if (a.wl >= 0) o.lo = max((long long)o.lo, (long long)pos - a.wl);
  o.out = (b * a.Hq + h * a.G) * a.T + q;
  return o;
}
// Index of row r of a piece in LSE (and, times d, in Q and O).
__device__ __forceinline__ int out_of(const PagedArgs& a, bool pre, const Piece& p, int r) {
  int b = p.b, q = p.row0 + r;
  if (pre) b = q / a.TG, q -= b * a.TG;
  return (b * a.Hq + p.h * a.G) * a.T + q;
}
// Row r of a piece.
__device__ __forceinline__ Row row_of(const PagedArgs& a, bool pre, const Piece& p, int r) {
  if (!pre) return row_at(a, false, p.h, p.b, p.row0 + r, p.len);
  const int b = (p.row0 + r) / a.TG;
  return row_at(a, true, p.h, b, p.row0 + r - b * a.TG, len_of(a, b));
}

// The table row of a slot (slot 0's for one out of range, whose sequence has no keys).
__device__ __forceinline__ const int* table_row(const PagedArgs& a, int slot) {
  if ((unsigned)slot >= (unsigned)a.c.slots) slot = 0;
  return a.c.table + (long long)slot * a.c.width;
}

// Byte offset of key j (head h) in the layer's K or V, through a table row.
__device__ __forceinline__ long long key_offset(const CacheView& c, const int* trow, int h, int j) {
  int page = __ldg(trow + (j >> c.page_log2));
  if ((unsigned)page >= (unsigned)c.pages) page = 0;
  return page * c.page_stride + (long long)h * c.head_bytes +
         (long long)(j & ((1 << c.page_log2) - 1)) * c.row_bytes;
}

}  // namespace sched
}  // namespace fa
