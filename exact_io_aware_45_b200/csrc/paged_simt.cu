// Paged attention on the CUDA cores for one to four query rows per KV head (fp32 inputs, and head
// sizes the tensor-core kernels do not take), and the kernel that joins partial results.
//
// For each packed query row r of a piece, over the keys j in [lo_r, hi_r):
//   x_rj = scale q_r . k_j (soft-capped), and the running
//   m = max(m, max_j x_rj), l = e^(m_old - m) l + sum_j e^(x_rj - m), likewise O,
// in base 2. A warp takes tiles of 32 keys. For the scores up to eight lanes read a key's row
// side by side, 16 bytes each, against their part of the query rows in registers; the sums over
// these lanes are exchanged so that each lane ends with the scores of one key (7 shuffles a row and
// tile). For P V a lane owns d / 32 columns and reads each V row together with its warp. The
// four warps of a block take tiles in turn and are merged once per piece.
//
// (A lane per key needs no sums across lanes, but reads 32 rows at once, half a sector of each: 64
// sequences of 1,000 to 3,000 tokens, 8 heads, fp32, took 190 us at d 16, now 52, and 16 of 50 to
// 4,000 at d 128 43, now 26.)
//
// Bound: HBM for long sequences (64 of 1,000 to 3,000 tokens, 8 heads, d 128, fp32, 1 GB: 175 us
// with two rows, 180 with four), latency for short ones. The rows are a template argument, one,
// two or four: more go to paged_fma.cu. Four rows of d 128 are read from shared memory (in
// registers they spilled, 304 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "paged_sched.cuh"

namespace fa {
namespace {

constexpr int kTile = 1 << kSimtTileLog2;
constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int N>
__device__ __forceinline__ void load_f(const float* p, float (&x)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __ldg(p + i);
  }
}
template <int N>
__device__ __forceinline__ void load_f(const __nv_bfloat16* p, float (&x)[N]) {
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + i));
      const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i + 2 * j] = __uint_as_float(w[j] << 16);
        x[i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __bfloat162float(p[i]);
  }
}
// Partial results: the join is resident while other kernels write them, so by plain loads, which its
// wait orders, and not by __ldg, which is for what no one writes in a kernel's lifetime. (__ldcg took
// 1 us more behind a prefix of 4,096 tokens.)
template <int N>
__device__ __forceinline__ void load_partial(const float* p, float (&x)[N]) {
  if constexpr (N == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = p[i];
  }
}
__device__ __forceinline__ void store_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

// The query rows in shared memory where registers would not hold them.
template <int D, int kRows>
constexpr bool kShareQ = D * kRows >= 512;

template <int D, int kRows>
struct SimtShared {
  alignas(16) float q[kShareQ<D, kRows> ? kRows : 1][kShareQ<D, kRows> ? D : 4];
  alignas(16) float p[kWarps][kRows][kTile];          // read as float4
  float o[kWarps][kRows][D];
  float m[kWarps][kRows], l[kWarps][kRows];
  int lo[kRows], hi[kRows];
  int out[kRows];
};

// kGaps: a shared phase under a window, where rows that no query sees may lie between others
// (sched::seen_of). A test of it at run time cost the other calls 2 to 17 %.
template <typename T, int D, int kRows, bool kGaps>
__global__ void __launch_bounds__(kWarps * 32, simt_blocks_per_sm(D, kRows))
    simt_kernel(const __grid_constant__ PagedArgs a, const bool pre) {
  __shared__ SimtShared<D, kRows> s;
  constexpr int kPer = D >= 32 ? D / 32 : 1;          // columns of a lane in P V
  // 16-byte pieces: kLanes lanes read kLanes x 16 bytes of a key side by side, kChunks times
  constexpr int kVec = 16 / (int)sizeof(T), kPieces = D / kVec;
  constexpr int kLanes = kPieces < 8 ? kPieces : 8, kChunks = kPieces / kLanes;
  constexpr int kSide = 32 / kLanes;                  // keys side by side
  constexpr int kRowBytes = D * (int)sizeof(T);
  constexpr int kHeld = kShareQ<D, kRows> ? 1 : kChunks;   // chunks of Q in registers
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = lane % kLanes, side = lane / kLanes;
  const int mine_key = part * kSide + side;           // whose scores this lane ends up with
  const Phase& ph = pre ? a.pre : a.own;
  warm_args(a);
  chain_next();
  sched::Walk w;
  if (!sched::begin(a, pre, blockIdx.x, w)) {         // the block's warps walk alike
    chain_end();
    return;
  }
  const T* Q = static_cast<const T*>(a.Q);
  while (w.x < w.end) {
    const sched::Piece pc = sched::next(a, pre, w);
    __syncthreads();
    if (tid < kRows) {
      sched::Row r;
      r.lo = r.hi = r.out = 0;
      if (tid < pc.rows) r = sched::row_of(a, pre, pc, tid);
      s.lo[tid] = r.lo, s.hi[tid] = r.hi, s.out[tid] = r.out;
    }
    __syncthreads();
    float q[kRows][kHeld][kVec];                        // this lane's part, scaled
    if constexpr (kShareQ<D, kRows>) {
      for (int i = tid; i < kRows * D; i += kWarps * 32) {
        float x[1] = {0.f};
        if (i / D < pc.rows) load_f<1>(Q + (size_t)s.out[i / D] * D + i % D, x);
        s.q[i / D][i % D] = x[0] * a.scale;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (r < pc.rows) {
            load_f<kVec>(Q + (size_t)s.out[r] * D + (c * kLanes + part) * kVec, q[r][c]);
          } else {
#pragma unroll
            for (int v = 0; v < kVec; ++v) q[r][c][v] = 0.f;
          }
#pragma unroll
          for (int v = 0; v < kVec; ++v) q[r][c][v] *= a.scale;
        }
    }
    float m[kRows], l[kRows], o[kRows][kPer];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[r][i] = 0.f;
    }
    const int* trow = sched::table_row(a, pc.table);
    const long long head = (long long)pc.h * a.c.head_bytes;
    // pages of a tile's halves (a page has 16 keys at least), asked for one tile ahead
    int page0, page1;
    auto find = [&](int t) {
      const int j = t * kTile;
      page0 = j < pc.hi ? __ldg(trow + (j >> a.c.page_log2)) : 0;
      page1 = j + 16 < pc.hi ? __ldg(trow + ((j + 16) >> a.c.page_log2)) : 0;
    };
    auto offset = [&](int page, int j) {              // of key j in this page
      if ((unsigned)page >= (unsigned)a.c.pages) page = 0;
      return page * a.c.page_stride + head +
             (long long)(j & ((1 << a.c.page_log2) - 1)) * kRowBytes;
    };
    find(pc.t0 + warp);
    for (int t = pc.t0 + warp; t < pc.t1; t += kWarps) {
      const int j0 = t * kTile, j = j0 + mine_key;
      const bool in = j >= pc.lo && j < pc.hi;
      const long long off0 = offset(page0, j0), off1 = offset(page1, j0 + 16);
      find(t + kWarps);
      unsigned seen = ~0u;
      if constexpr (kGaps) seen = sched::seen_of(a, pc, j0, pc.len);
      float x[kLanes][kRows];
#pragma unroll
      for (int g = 0; g < kLanes; ++g)
#pragma unroll
        for (int r = 0; r < kRows; ++r) x[g][r] = 0.f;
      const char* k0 = a.K + off0 + side * kRowBytes + part * 16;
      const char* k1 = a.K + off1 + side * kRowBytes + part * 16;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int held = kShareQ<D, kRows> ? 0 : c;
        if constexpr (kShareQ<D, kRows>) {
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            const float4 x4 = *reinterpret_cast<const float4*>(&s.q[r][(c * kLanes + part) * 4]);
            q[r][0][0] = x4.x, q[r][0][1] = x4.y, q[r][0][2] = x4.z, q[r][0][3] = x4.w;
          }
        }
        float kv[kLanes][kVec];
#pragma unroll
        for (int g = 0; g < kLanes; ++g) {
          const int i = g * kSide + side;
          const char* from = g < kLanes / 2 ? k0 + g * kSide * kRowBytes
                                            : k1 + (g - kLanes / 2) * kSide * kRowBytes;
          if (j0 + i >= pc.lo && j0 + i < pc.hi) {
            load_f<kVec>(reinterpret_cast<const T*>(from + c * kLanes * 16), kv[g]);
          } else {
#pragma unroll
            for (int v = 0; v < kVec; ++v) kv[g][v] = 0.f;
          }
        }
#pragma unroll
        for (int g = 0; g < kLanes; ++g)
#pragma unroll
          for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int v = 0; v < kVec; ++v) x[g][r] = fmaf(q[r][held][v], kv[g][v], x[g][r]);
      }
      // sums over the kLanes lanes of a key, each lane ending with one of kLanes keys
#pragma unroll
      for (int half = kLanes / 2; half; half >>= 1)
#pragma unroll
        for (int g = 0; g < half; ++g)
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            const bool up = part & half;
            const float give = up ? x[g][r] : x[g + half][r];
            const float keep = up ? x[g + half][r] : x[g][r];
            x[g][r] = keep + __shfl_xor_sync(~0u, give, half);
          }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float y = x[0][r];
        if (a.softcap > 0.f) y = a.softcap * tanhf(y / a.softcap);
        y *= kLog2e;
        if (!(in && j >= s.lo[r] && j < s.hi[r])) y = -INFINITY;
        float top = y;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        top = fmaxf(top, m[r]);
        const float ref = top == -INFINITY ? 0.f : top;
        const float e = exp2f(y - ref), c = exp2f(m[r] - ref);
        float sum = e;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
        m[r] = top;
        l[r] = l[r] * c + sum;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[r][i] *= c;
        s.p[warp][r][mine_key] = e;
      }
      __syncwarp();
      const bool mine = lane * kPer < D;
#pragma unroll 2
      for (int i = 0; i < kTile; i += 4) {
        float p[kRows][4], v[4][kPer];
        const char* from = a.V + (i < 16 ? off0 + i * kRowBytes : off1 + (i - 16) * kRowBytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // what no row sees is not read
          if (mine && j0 + i + k >= pc.lo && j0 + i + k < pc.hi &&
              (!kGaps || (seen >> (i + k)) & 1)) {
            load_f<kPer>(reinterpret_cast<const T*>(from + k * kRowBytes) + lane * kPer, v[k]);
          } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e) v[k][e] = 0.f;
          }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float4 x4 = *reinterpret_cast<const float4*>(&s.p[warp][r][i]);
          p[r][0] = x4.x, p[r][1] = x4.y, p[r][2] = x4.z, p[r][3] = x4.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[r][e] = fmaf(p[r][k], v[k][e], o[r][e]);
      }
      __syncwarp();
    }
    // merge the warps
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (lane == 0) s.m[warp][r] = m[r], s.l[warp][r] = l[r];
      if (lane * kPer < D)
#pragma unroll
        for (int i = 0; i < kPer; ++i) s.o[warp][r][lane * kPer + i] = o[r][i];
    }
    __syncthreads();
    for (int i = tid; i < pc.rows * D; i += kWarps * 32) {
      const int r = i / D, e = i % D;
      float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s.m[k][r]);
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float c = exp2f(s.m[k][r] - ref);
        sum = fmaf(c, s.l[k][r], sum);
        acc = fmaf(c, s.o[k][r][e], acc);
      }
      const float y = sum > 0.f ? acc / sum : (sum == 0.f ? 0.f : acc);
      const float lse2 = top + log2f(sum);
      if (pc.slot < 0) {
        store_f(static_cast<T*>(a.O) + (size_t)s.out[r] * D + e, y);
        if (e == 0) a.LSE[s.out[r]] = lse2 * 0.6931471805599453f;
      } else {
        const long long at = (long long)pc.slot * ph.rows + r;
        ph.o[at * D + e] = y;
        if (e == 0) ph.lse[at] = lse2;
      }
    }
  }
  chain_end();
}

template <typename T, int D, bool kGaps>
cudaError_t launch_simt_rows(const PagedArgs& a, bool pre, cudaStream_t st) {
  const Phase& ph = pre ? a.pre : a.own;
  const auto kernel = ph.rows == 1   ? simt_kernel<T, D, 1, kGaps>
                      : ph.rows == 2 ? simt_kernel<T, D, 2, kGaps>
                                     : simt_kernel<T, D, 4, kGaps>;
  return launch_chained(kernel, ph.n, kWarps * 32, 0, st, !pre && a.shared, a, pre);
}

template <typename T, int D>
cudaError_t launch_simt(const PagedArgs& a, bool pre, cudaStream_t st) {
  return pre && a.wl >= 0 ? launch_simt_rows<T, D, true>(a, pre, st)
                          : launch_simt_rows<T, D, false>(a, pre, st);
}

template <typename T>
cudaError_t launch_simt_d(const PagedArgs& a, bool pre, cudaStream_t st) {
  if (a.c.d == 16) return launch_simt<T, 16>(a, pre, st);
  if constexpr (sizeof(T) == 4) {                       // bf16 has the tensor cores from 64 on
    if (a.c.d == 64) return launch_simt<T, 64>(a, pre, st);
    if (a.c.d == 128) return launch_simt<T, 128>(a, pre, st);
  }
  return launch_simt<T, 32>(a, pre, st);
}

// ---------------------------------------------------------------- join

// O = sum_p 2^(lse_p - lse) O_p, lse = log2 sum_p 2^lse_p over a row's partial
// results, whose slots follow from the same arithmetic that cut them. A block has
// `rows` rows of a sequence; where these are fewer than its warps, several warps share a
// row and meet in shared memory (few rows have many pieces each: a long sequence
// is cut into hundreds). Reads (d + 1) floats a piece and row, from L2 mostly, and is
// bound by instructions: one warp does the arithmetic of the cuts, a lane per row (with
// every warp at it, a batch of 128 spent 20 us there), and per piece a warp
// issues two shuffles, a load and d / 32 multiply-adds.
constexpr int kJoinWarps = 8;
constexpr int kJoinBlocksPerSm = 4;
constexpr int kJoinMaxRows = 16;
constexpr int kChunk = 8;              // at most 16; 10 spilled and took 1 us more

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32, kJoinBlocksPerSm)
    join_kernel(const __grid_constant__ PagedArgs a, const int rows) {
  constexpr int kPer = D >= 32 ? D / 32 : 1;
  struct RowPieces {
    int own, own_head, own_next;   // partial results of the own phase, first slots
    int all, pre_head, pre_next;   // of both phases
    int own_row, pre_row;
  };
  __shared__ float part_o[kJoinWarps][D], part_sum[kJoinWarps], part_top[kJoinWarps];
  __shared__ RowPieces info[kJoinMaxRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y, in_b = a.c.Hkv * a.TG;
  const int r0 = blockIdx.x * rows, count = min(rows, in_b - r0);
  warm_args(a);
  if (warp == 0) {
    const sched::Batch t = sched::scan_batch(a, b);
    if (lane < count) {
      const int h = (r0 + lane) / a.TG, q = r0 + lane - h * a.TG;
      const sched::Cuts cuts(a.own, t.W);
      const int u = sched::own_units(a, t.len);
      const int rt = q / a.own.rows, in = h * a.own.rt + rt;
      int first, more;
      sched::pieces_of(a.own, t.before + in * u, u, cuts, first, more);
      RowPieces p;
      p.own = more + 1;
      p.own_head = b * a.c.Hkv * a.own.rt + in;
      p.own_next = a.own.items + first;
      p.own_row = q - rt * a.own.rows;
      p.all = p.own;
      p.pre_head = p.pre_next = p.pre_row = 0;
      if (a.shared) {
        int lo, hi;
        sched::pre_keys(a, t.least, t.most, lo, hi);
        const int pu = sched::units_of(a.pre, lo, hi);
        const int pr = b * a.TG + q, prt = pr / a.pre.rows;
        p.pre_head = h * a.pre.rt + prt;
        p.pre_row = pr - prt * a.pre.rows;
        sched::pieces_of(a.pre, p.pre_head * pu, pu, sched::Cuts(a.pre, a.pre.items * pu, t.W),
                         first, more);
        p.pre_next = a.pre.items + first;
        p.all += more + 1;
      } else if (more == 0) {
        p.all = 0;                                      // written by its only piece
      }
      info[lane] = p;
    }
  }
  __syncthreads();
  // `ways` warps a row
  int ways = kJoinWarps;
  while (ways > 1 && ways * count > kJoinWarps) ways >>= 1;
  const int way = warp & (ways - 1);
  bool waited = false;
  // shared rows are done in one go, all warps meeting below
  const int stop = ways > 1 ? kJoinWarps / ways : count;
  for (int i = warp / ways; i < stop; i += kJoinWarps / ways) {
    RowPieces p;
    p.all = 0;
    if (i < count) p = info[i];
    // row index of partial result k in its phase's buffers
    auto at_of = [&](int k) {
      const bool own = k < p.own;
      const Phase& ph = own ? a.own : a.pre;
      if (!own) k -= p.own;
      const int slot = k ? (own ? p.own_next : p.pre_next) + k : (own ? p.own_head : p.pre_head);
      return slot * ph.rows + (own ? p.own_row : p.pre_row);
    };
    float top = -INFINITY, sum = 0.f, acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    // kChunk partial results at a time: their O and LSE are on their way together
    for (int k0 = way * kChunk; k0 < p.all; k0 += ways * kChunk) {
      const int n = min(kChunk, p.all - k0), own = p.own - k0;
      const int at = lane < n ? at_of(k0 + lane) : 0;   // lane k: of partial result k0 + k
      if (!waited) chain_wait();                        // the partial results are there
      waited = true;
      float lse = -INFINITY;
      if (lane < n) lse = (lane < own ? a.own.lse : a.pre.lse)[at];
      float v[kChunk][kPer];
      const int col = lane * kPer;
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        const int row = __shfl_sync(~0u, at, k);
        const Phase& ph = k < own ? a.own : a.pre;
        const float* from = ph.o + (size_t)row * D + col;
        if (ph.blocked)
          from = ph.o + (size_t)(row >> 7) * (128 * D) + (col >> 3) * (128 * 8) +
                 (row & 127) * 8 + (col & 7);
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[k][e] = 0.f;
        if (k < n && col < D) load_partial<kPer>(from, v[k]);
      }
      float m = lse;
#pragma unroll
      for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
      m = fmaxf(__shfl_sync(~0u, m, 0), top);
      const float ref = m == -INFINITY ? 0.f : m;
      const float old = exp2f(top - ref), weight = exp2f(lse - ref);
      top = m;
      sum *= old;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] *= old;
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        const float c = __shfl_sync(~0u, weight, k);    // 0 for k >= n
        sum += c;
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(c, v[k][e], acc[e]);
      }
    }
    if (ways > 1) {
      if (lane * kPer < D)
#pragma unroll
        for (int e = 0; e < kPer; ++e) part_o[warp][lane * kPer + e] = acc[e];
      if (lane == 0) part_top[warp] = top, part_sum[warp] = sum;
      __syncthreads();
      if (way) break;
      for (int k = 0; k < ways; ++k) top = fmaxf(top, part_top[warp + k]);
      const float ref = top == -INFINITY ? 0.f : top;
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
      for (int k = 0; k < ways; ++k) {
        const float c = exp2f(part_top[warp + k] - ref);
        sum = fmaf(c, part_sum[warp + k], sum);
        if (lane * kPer < D)
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            acc[e] = fmaf(c, part_o[warp + k][lane * kPer + e], acc[e]);
      }
    }
    if (p.all == 0) continue;
    const int h = (r0 + i) / a.TG, q = r0 + i - h * a.TG;
    const size_t out = (size_t)(b * a.Hq + h * a.G) * a.T + q;
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    if (lane * kPer < D)
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        store_f(static_cast<T*>(a.O) + out * D + lane * kPer + e, acc[e] * inv);
    if (lane == 0) a.LSE[out] = (top + log2f(sum)) * 0.6931471805599453f;
  }
  if (!waited) chain_wait();                            // this kernel's end implies the others'
}

template <typename T, int D>
cudaError_t launch_join(const PagedArgs& a, cudaStream_t st) {
  // as many blocks as are resident at once, then rows that share a block's set-up
  const long long all = (long long)a.B * a.c.Hkv * a.TG, resident = kJoinBlocksPerSm * a.own.sms;
  int rows = 1;
  while (rows < kJoinMaxRows && all > resident * rows) rows *= 2;
  const dim3 grid((a.c.Hkv * a.TG + rows - 1) / rows, a.B);
  return launch_chained(join_kernel<T, D>, grid, kJoinWarps * 32, 0, st, true, a, rows);
}

template <typename T>
cudaError_t launch_join_d(const PagedArgs& a, cudaStream_t st) {
  switch (a.c.d) {
    case 16: return launch_join<T, 16>(a, st);
    case 32: return launch_join<T, 32>(a, st);
    case 64: return launch_join<T, 64>(a, st);
    default: return launch_join<T, 128>(a, st);
  }
}

}  // namespace

cudaError_t paged_simt(const PagedArgs& a, bool pre, int dtype, cudaStream_t st) {
  return dtype == FA_F32 ? launch_simt_d<float>(a, pre, st)
                         : launch_simt_d<__nv_bfloat16>(a, pre, st);
}

cudaError_t paged_join(const PagedArgs& a, int dtype, cudaStream_t st) {
  return dtype == FA_F32 ? launch_join_d<float>(a, st) : launch_join_d<__nv_bfloat16>(a, st);
}

}  // namespace fa
