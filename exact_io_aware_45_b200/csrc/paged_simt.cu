// Paged attention on the CUDA cores (fp32 inputs, and head sizes the tensor-core
// kernels do not take), and the kernel that joins partial results.
//
// For each packed query row r of a piece, over the keys j in [lo_r, hi_r):
//   x_rj = scale q_r . k_j (soft-capped), and the running
//   m = max(m, max_j x_rj), l = e^(m_old - m) l + sum_j e^(x_rj - m), likewise O,
// in base 2. A warp takes tiles of 32 keys. For the scores a lane owns a key:
// it reads its row in 16-byte pieces and the query rows from shared memory, so
// no score needs a reduction across lanes; for P V a lane owns d / 32 columns and
// reads each V row together with its warp. The four warps of a block
// take tiles in turn and are merged once per piece.
//
// Bound: 4 d rows flops a key in fp32 against 2 d elements read: at 8 rows and
// fp32 4 flops a byte, above which the CUDA cores (not HBM) are the limit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "paged_sched.cuh"

namespace fa {
namespace {

constexpr int kRows = kSimtRows;
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
__device__ __forceinline__ void store_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

template <typename T, int D>
struct SimtShared {
  alignas(16) float q[kRows][D];                      // read as float4
  float p[kWarps][kRows][kTile];
  float o[kWarps][kRows][D];
  float m[kWarps][kRows], l[kWarps][kRows];
  int lo[kRows], hi[kRows];
  int out[kRows];
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) simt_kernel(const PagedArgs a, const bool pre) {
  __shared__ SimtShared<T, D> s;
  constexpr int kPer = D >= 32 ? D / 32 : 1;          // columns of a lane in P V
  constexpr int kVec = 16 / (int)sizeof(T);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Phase& ph = pre ? a.pre : a.own;
  chain_next();
  sched::Walk w;
  if (!sched::begin(a, pre, blockIdx.x, w)) {         // the block's warps walk alike
    chain_wait();
    return;
  }
  const T* Q = static_cast<const T*>(a.Q);
  while (w.x < w.end) {
    const sched::Piece pc = sched::next(a, pre, blockIdx.x, w);
    __syncthreads();
    if (tid < kRows) {
      sched::Row r;
      r.lo = r.hi = r.out = 0;
      if (tid < pc.rows) r = sched::row_of(a, pre, pc, tid);
      s.lo[tid] = r.lo, s.hi[tid] = r.hi, s.out[tid] = r.out;
    }
    __syncthreads();
    for (int i = tid; i < kRows * D; i += kWarps * 32) {
      const int r = i / D;
      float x = 0.f;
      if (r < pc.rows) {
        float y[1];
        load_f<1>(Q + (size_t)s.out[r] * D + i % D, y);
        x = y[0] * a.scale;
      }
      s.q[r][i % D] = x;
    }
    __syncthreads();
    float m[kRows], l[kRows], o[kRows][kPer];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[r][i] = 0.f;
    }
    const int* trow = sched::table_row(a, pc.table);
    for (int t = pc.t0 + warp; t < pc.t1; t += kWarps) {
      const int j = t * kTile + lane;
      const bool in = j >= pc.lo && j < pc.hi;
      const long long off = in ? sched::key_offset(a.c, trow, pc.h, j) : 0;
      float x[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) x[r] = 0.f;
      if (in) {
        const T* k = reinterpret_cast<const T*>(a.K + off);
#pragma unroll
        for (int i = 0; i < D; i += kVec) {
          float kv[kVec];
          load_f<kVec>(k + i, kv);
#pragma unroll
          for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int v = 0; v < kVec; v += 4) {
              const float4 qv = *reinterpret_cast<const float4*>(&s.q[r][i + v]);
              x[r] = fmaf(qv.x, kv[v], x[r]);
              x[r] = fmaf(qv.y, kv[v + 1], x[r]);
              x[r] = fmaf(qv.z, kv[v + 2], x[r]);
              x[r] = fmaf(qv.w, kv[v + 3], x[r]);
            }
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float y = x[r];
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
        s.p[warp][r][lane] = e;
      }
      __syncwarp();
      const bool mine = lane * kPer < D;
#pragma unroll 4
      for (int i = 0; i < kTile; ++i) {
        const long long vo = __shfl_sync(~0u, off, i);
        if (!__shfl_sync(~0u, (int)in, i)) continue;   // what no row sees is not read
        float v[kPer];
        if (mine) {
          load_f<kPer>(reinterpret_cast<const T*>(a.V + vo) + lane * kPer, v);
        } else {
#pragma unroll
          for (int e = 0; e < kPer; ++e) v[e] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float p = s.p[warp][r][i];
#pragma unroll
          for (int e = 0; e < kPer; ++e) o[r][e] = fmaf(p, v[e], o[r][e]);
        }
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
  chain_wait();
}

template <typename T, int D>
cudaError_t launch_simt(const PagedArgs& a, bool pre, cudaStream_t st) {
  return launch_chained(simt_kernel<T, D>, (pre ? a.pre : a.own).n, kWarps * 32, 0, st,
                        !pre && a.shared, a, pre);
}

template <typename T>
cudaError_t launch_simt_d(const PagedArgs& a, bool pre, cudaStream_t st) {
  switch (a.c.d) {
    case 16: return launch_simt<T, 16>(a, pre, st);
    case 32: return launch_simt<T, 32>(a, pre, st);
    case 64: return launch_simt<T, 64>(a, pre, st);
    default: return launch_simt<T, 128>(a, pre, st);
  }
}

// ---------------------------------------------------------------- join

// O = sum_p 2^(lse_p - lse) O_p, lse = log2 sum_p 2^lse_p over a row's partial
// results, whose slots follow from the same arithmetic that cut them. A block has
// up to eight rows of a sequence and KV head; where it has fewer, several warps share a
// row and meet in shared memory, since few rows have many pieces each (a long
// sequence is cut into hundreds). One warp finds where the cuts are: with every warp
// at it, a batch of 128 spent 20 us on the arithmetic alone. Reads (d + 1) floats a piece and row, from L2 mostly.
constexpr int kJoinWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const PagedArgs a) {
  constexpr int kPer = D >= 32 ? D / 32 : 1;
  __shared__ float part_o[kJoinWarps][D], part_sum[kJoinWarps];
  __shared__ sched::Batch batch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x, b = blockIdx.y;
  if (warp == 0) {
    const sched::Batch mine = sched::scan_batch(a, b);
    if (lane == 0) batch = mine;
  }
  __syncthreads();
  const sched::Batch t = batch;
  const sched::Cuts cuts(a.own, t.W);
  const int u = sched::own_units(a, t.len);
  int pu = 1;
  if (a.shared) {
    int lo, hi;
    sched::pre_keys(a, t.least, t.most, lo, hi);
    pu = sched::units_of(a.pre, lo, hi);
  }
  const sched::Cuts pre_cuts(a.pre, max(1, a.pre.items) * pu);
  // `ways` warps a row, the block's rows side by side
  int ways = kJoinWarps;
  while (ways > 1 && kJoinWarps / ways < a.TG) ways >>= 1;
  const int side = kJoinWarps / ways, way = warp % ways;
  chain_wait();                                         // the partial results are there
  for (int q0 = blockIdx.z * kJoinWarps; q0 < min(a.TG, (int)(blockIdx.z + 1) * kJoinWarps);
       q0 += side) {
    const int q = q0 + warp / ways;
    const int r = q / a.own.rows, in = h * a.own.rt + r;
    int first = 0, more = 0, pre_first = 0, pre_more = -1, pre_item = 0, pre_row = 0;
    bool mine = q < a.TG;
    if (mine) {
      sched::pieces_of(a.own, t.before + in * u, u, cuts, first, more);
      if (a.shared) {
        const int pr = b * a.TG + q;
        pre_item = h * a.pre.rt + pr / a.pre.rows;
        pre_row = pr % a.pre.rows;
        sched::pieces_of(a.pre, pre_item * pu, pu, pre_cuts, pre_first, pre_more);
      } else if (more == 0 && a.own.fold == 1) {
        mine = false;                                   // written by its only piece
      }
    }
    const int own_count = (more + 1) * a.own.fold;
    const int count = mine ? own_count + (pre_more + 1) * a.pre.fold : 0;
    // row index of partial p in its phase's buffers
    auto at_of = [&](int p) -> long long {
      const bool own = p < own_count;
      const Phase& ph = own ? a.own : a.pre;
      if (!own) p -= own_count;
      int f = 0;
      if (ph.fold == 2) f = p & 1, p >>= 1;
      const int slot = own ? (p == 0 ? b * a.c.Hkv * a.own.rt + in : a.own.items + first + p)
                           : (p == 0 ? pre_item : a.pre.items + pre_first + p);
      return ((long long)slot * ph.fold + f) * ph.rows + (own ? q - r * a.own.rows : pre_row);
    };
    float top = -INFINITY;
    for (int p = lane; p < count; p += 32)
      top = fmaxf(top, (p < own_count ? a.own.lse : a.pre.lse)[at_of(p)]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f, acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int p = way; p < count; p += ways) {
      const long long at = at_of(p);
      const float c = exp2f((p < own_count ? a.own.lse : a.pre.lse)[at] - ref);
      sum += c;
      if (lane * kPer < D) {
        float v[kPer];
        load_f<kPer>((p < own_count ? a.own.o : a.pre.o) + at * D + lane * kPer, v);
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(c, v[e], acc[e]);
      }
    }
    if (ways > 1) {
      __syncthreads();
      if (lane * kPer < D)
#pragma unroll
        for (int e = 0; e < kPer; ++e) part_o[warp][lane * kPer + e] = acc[e];
      if (lane == 0) part_sum[warp] = sum;
      __syncthreads();
      if (way) continue;
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
      for (int k = 0; k < ways; ++k) {
        sum += part_sum[warp + k];
        if (lane * kPer < D)
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] += part_o[warp + k][lane * kPer + e];
      }
    }
    if (!mine) continue;
    const size_t out = (size_t)(b * a.Hq + h * a.G) * a.T + q;
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    if (lane * kPer < D)
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        store_f(static_cast<T*>(a.O) + out * D + lane * kPer + e, acc[e] * inv);
    if (lane == 0) a.LSE[out] = (top + log2f(sum)) * 0.6931471805599453f;
  }
}

template <typename T, int D>
cudaError_t launch_join(const PagedArgs& a, cudaStream_t st) {
  const dim3 grid(a.c.Hkv, a.B, (a.TG + kJoinWarps - 1) / kJoinWarps);
  return launch_chained(join_kernel<T, D>, grid, kJoinWarps * 32, 0, st, true, a);
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
