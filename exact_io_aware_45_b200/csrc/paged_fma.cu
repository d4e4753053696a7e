// Paged attention on the CUDA cores for many query rows per KV head (fp32 inputs, and
// head sizes the tensor-core kernels do not take): a shared prefix, or a chunk of tokens.
//
// The mathematics is that of simt_kernel (paged_simt.cu): running maximum and sum per row, in base
// 2. There a lane owns a key and a row's score costs it a read of K and of Q per four
// multiply-adds, which is the cheapest for 8 rows but bound by the load and shuffle pipe.
// Here products are tiled in registers: a block has 64 rows and takes tiles of 32 keys through
// shared memory (cp.async, two stages), a warp 16 of the rows, a lane 4 rows x 4 keys of the
// scores and 4 rows x d / 8 columns of O. Per four of d a lane reads 8 x 16 bytes for 64
// multiply-adds. Rows of K, V and Q are padded by 16 bytes:
// eight keys (or four rows) read side by side fall into different banks.
//
// 64 sequences of 4 rows and 8 heads behind 4,096 tokens (fp32, d 128, 4.3 GFLOP) take 157 us in
// all, 232 by simt_kernel; 128 of 8 rows and 4 heads behind 8,192 (d 64, 8.6 GFLOP) 278. The FMA
// pipe is active in 48 % of the cycles, the scheduler issues in 62 %: three warps each, which the
// registers allow, do not hide all latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "paged_sched.cuh"
#include "sm100_common.cuh"

namespace fa {
namespace {

constexpr int kRows = kFmaRows;
constexpr int kTile = 1 << kSimtTileLog2;
constexpr int kWarps = 4, kWarpRows = kRows / kWarps;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T, int D>
struct FmaShared {
  static constexpr int kStride = D * (int)sizeof(T) + 16;   // bytes of a row of K or V
  alignas(16) unsigned char k[2][kTile * kStride];
  alignas(16) unsigned char v[2][kTile * kStride];
  alignas(16) float q[kRows][D + 4];
  alignas(16) float p[kWarps][kWarpRows][kTile + 8];        // four rows a bank line
  int lo[kRows], hi[kRows], out[kRows];
};

// N elements from shared memory (N is 2 or 4), as floats.
template <int N>
__device__ __forceinline__ void load_s(const float* p, float (&x)[N]) {
  if constexpr (N == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x, x[1] = v.y;
  }
}
template <int N>
__device__ __forceinline__ void load_s(const __nv_bfloat16* p, float (&x)[N]) {
  unsigned w[N / 2];
  if constexpr (N == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const unsigned*>(p);
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ float load_g(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_g(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <int N>
__device__ __forceinline__ void store_g(float* p, const float (&x)[N]) {
  if constexpr (N == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
}
template <int N>
__device__ __forceinline__ void store_g(__nv_bfloat16* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2)
    *reinterpret_cast<__nv_bfloat162*>(p + i) = __floats2bfloat162_rn(x[i], x[i + 1]);
}
// 16 bytes global -> shared; `bytes` of them are read, the rest become zero.
__device__ __forceinline__ void copy16(void* dst, const char* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}

// kGaps: a shared phase under a window, where rows that no query sees may lie between others
// (sched::seen_of). A test of it at run time cost the other calls up to 5 %.
template <typename T, int D, bool kGaps>
__global__ void __launch_bounds__(kThreads, fma_blocks_per_sm(D))
    fma_kernel(const __grid_constant__ PagedArgs a, const bool pre) {
  using Shared = FmaShared<T, D>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Shared& s = *reinterpret_cast<Shared*>(smem_raw);
  constexpr int kPer = D / 8, kVec = kPer < 4 ? kPer : 4;    // columns of a lane in P V
  constexpr int kRowVecs = D * (int)sizeof(T) / 16;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r4 = lane >> 3, c8 = lane & 7;   // rows r4 + 4 i, keys c8 + 8 j, columns from c8 kVec on
  const Phase& ph = pre ? a.pre : a.own;
  warm_args(a);
  chain_next();
  sched::Walk w;
  if (!sched::begin(a, pre, blockIdx.x, w)) {           // the block's warps walk alike
    chain_end();
    return;
  }
  const T* Q = static_cast<const T*>(a.Q);
  while (w.x < w.end) {
    const sched::Piece pc = sched::next(a, pre, w);
    const int* trow = sched::table_row(a, pc.table);
    const long long head = (long long)pc.h * a.c.head_bytes;
    // pages of a tile's two halves (a page has 16 keys at least), asked for one tile ahead
    int page0, page1;
    auto find = [&](int t) {
      const int j = t * kTile;
      page0 = j < pc.hi ? __ldg(trow + (j >> a.c.page_log2)) : 0;
      page1 = j + 16 < pc.hi ? __ldg(trow + ((j + 16) >> a.c.page_log2)) : 0;
    };
    auto load = [&](int t) {
      const int st = (t - pc.t0) & 1;
      constexpr int kAll = kTile * kRowVecs;
      unsigned seen = ~0u;
      if constexpr (kGaps) seen = sched::seen_of(a, pc, t * kTile, pc.len);
#pragma unroll
      for (int i0 = 0; i0 < kAll; i0 += kThreads) {
        const int i = i0 + tid, row = i / kRowVecs, c = i % kRowVecs;
        if (kAll % kThreads && i >= kAll) break;
        const int j = t * kTile + row;
        // rows that no query sees are not read and count as zero
        const bool in = j >= pc.lo && j < pc.hi && (!kGaps || (seen >> row) & 1);
        const int named = row < 16 ? page0 : page1;
        const int page = (unsigned)named < (unsigned)a.c.pages ? named : 0;
        const long long off = page * a.c.page_stride + head +
                              (long long)(j & ((1 << a.c.page_log2) - 1)) * a.c.row_bytes + c * 16;
        copy16(&s.k[st][row * Shared::kStride + c * 16], a.K + off, in ? 16 : 0);
        copy16(&s.v[st][row * Shared::kStride + c * 16], a.V + off, in ? 16 : 0);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    find(pc.t0);
    load(pc.t0);
    find(pc.t0 + 1);
    if (tid < kRows) {
      sched::Row r;
      r.lo = r.hi = r.out = 0;
      if (tid < pc.rows) r = sched::row_of(a, pre, pc, tid);
      s.lo[tid] = r.lo, s.hi[tid] = r.hi, s.out[tid] = r.out;
    }
    __syncthreads();
    for (int i = tid; i < kRows * D; i += kThreads) {
      const int r = i / D;
      s.q[r][i % D] = r < pc.rows ? load_g(Q + (size_t)s.out[r] * D + i % D) * a.scale : 0.f;
    }
    const int r0 = warp * kWarpRows;
    const bool busy = r0 < pc.rows;                     // any of this warp's rows is real
    int lo[4], hi[4];
    float m[4], l[4], o[4][kPer];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = s.lo[r0 + r4 + 4 * i], hi[i] = s.hi[r0 + r4 + 4 * i];
      m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < kPer; ++c) o[i][c] = 0.f;
    }
    for (int t = pc.t0; t < pc.t1; ++t) {
      if (t + 1 < pc.t1) load(t + 1);
      else asm volatile("cp.async.commit_group;" ::: "memory");
      find(t + 2);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      if (busy) {
        const int st = (t - pc.t0) & 1;
        const unsigned char* kt = s.k[st] + c8 * Shared::kStride;
        float x[4][4] = {};
#pragma unroll (D < 64 ? D / 4 : 8)
        for (int e = 0; e < D; e += 4) {
          float q[4][4], k[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) load_s<4>(&s.q[r0 + r4 + 4 * i][e], q[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            load_s<4>(reinterpret_cast<const T*>(kt + 8 * j * Shared::kStride) + e, k[j]);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) x[i][j] = fmaf(q[i][c], k[j][c], x[i][j]);
        }
        const int j0 = t * kTile + c8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float y = x[i][j];
            if (a.softcap > 0.f) y = a.softcap * tanhf(y / a.softcap);
            y *= kLog2e;
            x[i][j] = j0 + 8 * j >= lo[i] && j0 + 8 * j < hi[i] ? y : -INFINITY;
          }
          float top = fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3]));
#pragma unroll
          for (int d = 4; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
          top = fmaxf(top, m[i]);
          const float ref = top == -INFINITY ? 0.f : top;
          const float c = exp2f(m[i] - ref);
          m[i] = top;
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = exp2f(x[i][j] - ref);
            sum += p;
            s.p[warp][r4 + 4 * i][c8 + 8 * j] = p;
          }
          l[i] = l[i] * c + sum;                        // of this lane's keys
#pragma unroll
          for (int e = 0; e < kPer; ++e) o[i][e] *= c;
        }
        __syncwarp();
        const unsigned char* vt = s.v[st] + c8 * kVec * sizeof(T);
#pragma unroll 2
        for (int k = 0; k < kTile; k += 4) {
          float p[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) load_s<4>(&s.p[warp][r4 + 4 * i][k], p[i]);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const T* row = reinterpret_cast<const T*>(vt + (k + kk) * Shared::kStride);
#pragma unroll
            for (int e = 0; e < kPer; e += kVec) {
              float v[kVec];
              load_s<kVec>(row + 8 * e, v);
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < kVec; ++c) o[i][e + c] = fmaf(p[i][kk], v[c], o[i][e + c]);
            }
          }
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sum = l[i];
#pragma unroll
      for (int d = 4; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      const int r = r0 + r4 + 4 * i;
      if (r >= pc.rows) continue;
      const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
      const float lse2 = m[i] + log2f(sum);
      const long long at = pc.slot < 0 ? s.out[r] : (long long)pc.slot * ph.rows + r;
      if (c8 == 0) {
        if (pc.slot < 0) a.LSE[at] = lse2 * kLn2;
        else ph.lse[at] = lse2;
      }
#pragma unroll
      for (int e = 0; e < kPer; e += kVec) {
        float y[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) y[c] = o[i][e + c] * inv;
        const long long to = at * D + 8 * e + c8 * kVec;
        if (pc.slot < 0) store_g<kVec>(static_cast<T*>(a.O) + to, y);
        else store_g<kVec>(ph.o + to, y);
      }
    }
    __syncthreads();                                    // s.out is read until here
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  chain_end();
}

template <typename T, int D, bool kGaps>
cudaError_t launch_gaps(const PagedArgs& a, bool pre, cudaStream_t st) {
  constexpr int kSmem = (int)sizeof(FmaShared<T, D>);
  static_assert((kSmem + 1024) * fma_blocks_per_sm(D) <= 228 * 1024, "shared memory of an SM");
  const auto kernel = fma_kernel<T, D, kGaps>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), kSmem)) return e;
  return launch_chained(kernel, (pre ? a.pre : a.own).n, kThreads, kSmem, st, !pre && a.shared, a,
                        pre);
}

template <typename T, int D>
cudaError_t launch(const PagedArgs& a, bool pre, cudaStream_t st) {
  return pre && a.wl >= 0 ? launch_gaps<T, D, true>(a, pre, st)
                          : launch_gaps<T, D, false>(a, pre, st);
}

template <typename T>
cudaError_t launch_d(const PagedArgs& a, bool pre, cudaStream_t st) {
  if (a.c.d == 16) return launch<T, 16>(a, pre, st);
  if constexpr (sizeof(T) == 4) {                       // bf16 has the tensor cores from 64 on
    if (a.c.d == 64) return launch<T, 64>(a, pre, st);
    if (a.c.d == 128) return launch<T, 128>(a, pre, st);
  }
  return launch<T, 32>(a, pre, st);
}

}  // namespace

cudaError_t paged_fma(const PagedArgs& a, bool pre, int dtype, cudaStream_t st) {
  return dtype == FA_F32 ? launch_d<float>(a, pre, st) : launch_d<__nv_bfloat16>(a, pre, st);
}

}  // namespace fa
