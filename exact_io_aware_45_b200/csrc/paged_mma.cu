// Paged attention for few query rows per KV head (decoding): bound by reading K
// and V once, so the kernel is a stream of TMA loads with just enough
// arithmetic behind it.
//
// One CTA per SM walks its share of the key tiles (paged_sched.cuh). A producer
// warp looks pages up and keeps a ring of 32-key stages filled (112 to 196 KB of K
// and V per SM in flight or in use; at 6.5 TB/s over 148 SMs and ~1 us of
// latency 45 KB would already do); seven to ten consumer warps take stages in turn,
// each with running statistics of its own, and merge once per piece.
//
// The products are transposed so that the packed query rows are the narrow side:
//   S^T = K Q^T   m16n8k16, A = 16 keys x 16 of d (ldmatrix), B = Q^T in registers
//   O^T += V^T P^T  A = 16 of d x 16 keys (ldmatrix.trans), B = P^T
// with 8 query rows per n-tile: decoding has 1 to 8 rows per KV head, of which an
// m16 tile of queries would waste half or more. P^T comes from S^T's accumulator
// layout by an 8x8 transpose (movmatrix). The tensor pipe does 2 * 32 rows-padded
// products of d a key and stays far from its limit, so mma.sync's lower
// peak costs nothing here; from about 64 rows on the tcgen05 kernel is faster.
//
// P is rounded to bf16 for the second product (the row sum takes it unrounded);
// sums, maxima and O stay in fp32.
#include <math.h>

#include "paged_sched.cuh"
#include "sm100_common.cuh"

namespace fa {
namespace {

using namespace sm100;

constexpr int kTile = kMmaTile;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Nine to twelve warps have 168 registers a thread (the register file is dealt out
// in four-warp steps), eight have 255: one n-tile fits the former, more want the
// latter. Stages are a multiple of the consumers, so that a stage is always the
// same warp's: loads complete in any order, and a warp that came to a stage while
// another warp's load of it was still in flight would take the phase before
// that load for its own (the two have the same parity).
template <int D, int NT>
struct Cfg {
  static constexpr int kConsumers = NT == 1 ? (D == 128 ? 10 : 8) : 7;
  static constexpr int kThreads = (kConsumers + 1) * 32;
  static constexpr int kHalf = kTile * D * 2;            // bytes of a stage's K (or V)
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = kConsumers * (D == 128 ? 1 : 3);
  static constexpr int kPitch = D + 4;                   // floats; rows 4 banks apart
  static constexpr int kMerge = kConsumers * 8 * kPitch * 4;
  static constexpr int kQPitch = D * 2 + 16;             // bytes; rows 4 banks apart
  static constexpr int kQ = NT * 8 * kQPitch;
  static constexpr int kRing = kStages * kStage;
};

struct Control {
  uint64_t full[24], empty[24], never;
  sched::Scratch scratch;
  float m[10][kMmaMaxRows], l[10][kMmaMaxRows];
  int abort, skip;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// NT: n-tiles of eight packed query rows.
template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
    mma_kernel(const PagedArgs a, const bool pre, const __grid_constant__ CUtensorMap km,
               const __grid_constant__ CUtensorMap vm, const long long stall) {
  using C = Cfg<D, NT>;
  constexpr int kConsumers = C::kConsumers, kThreads = C::kThreads;
  constexpr bool kQRegs = NT <= 2;     // four n-tiles of Q stay in shared memory
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  float* merge = reinterpret_cast<float*>(ring + C::kRing);
  uint8_t* qs = ring + C::kRing + C::kMerge;
  __shared__ Control s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Phase& ph = pre ? a.pre : a.own;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    mbar_init(&s.never, 1);
    s.abort = 0;
    s.skip = *reinterpret_cast<volatile unsigned*>(a.c.err) & kErrTimeout;
    fence_mbar_init();
  }
  sched::Walk w;
  long long end;
  // the barriers of begin() also publish what thread 0 set up
  if (!sched::begin(a, ph, pre, blockIdx.x, kThreads, s.scratch, w, end)) return;
  if (s.skip) return;
  const Guard guard{&s.abort, a.c.err};
  const int box = min(kTile, 1 << a.c.page_log2);        // rows of one load
  uint32_t gt = 0;                                       // tiles of the ring so far

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&km);
      prefetch_tmap(&vm);
      injected_stall(&s.never, stall, guard);
    }
    __syncwarp();
    while (w.x < end) {
      const sched::Piece pc = sched::next(a, ph, pre, blockIdx.x, end, w);
      const int* trow = sched::table_row(a, pc.b);
      // 32 table entries a load, the next 32 on their way
      const int last = pc.hi > pc.lo ? (pc.hi - 1) >> a.c.page_log2 : -1;
      int at = (pc.t0 * kTile) >> a.c.page_log2;
      int cur = at + lane <= last ? __ldg(trow + at + lane) : -1;
      int nxt = at + 32 + lane <= last ? __ldg(trow + at + 32 + lane) : -1;
      for (int t = pc.t0; t < pc.t1; ++t, ++gt) {
        const int st = gt % C::kStages;
        if (gt >= C::kStages &&
            !__all_sync(~0u, mbar_wait(&s.empty[st], ((gt / C::kStages) & 1) ^ 1, guard)))
          break;
        uint8_t* kd = ring + st * C::kStage;
        uint8_t* vd = kd + C::kHalf;
        // loads that hold a visible key
        int count = 0;
        for (int j = t * kTile; j < (t + 1) * kTile; j += box)
          count += j < pc.hi && j + box > pc.lo ? 1 : 0;
        if (lane == 0) mbar_expect_tx(&s.full[st], (uint32_t)(count * box * D * 4));
        for (int i = 0, j = t * kTile; j < (t + 1) * kTile; ++i, j += box) {
          const int p = j >> a.c.page_log2;
          while (p - at >= 32) {
            at += 32;
            cur = nxt;
            nxt = at + 32 + lane <= last ? __ldg(trow + at + 32 + lane) : -1;
          }
          int page = __shfl_sync(~0u, cur, p - at);
          if ((unsigned)page >= (unsigned)a.c.pages) page = 0;
          if (lane == 0 && j < pc.hi && j + box > pc.lo) {
            const int row = j & ((1 << a.c.page_log2) - 1);
            tma_load_page(kd + i * box * D * 2, &km, &s.full[st], row, pc.h, page);
            tma_load_page(vd + i * box * D * 2, &vm, &s.full[st], row, pc.h, page);
          }
        }
      }
      if (__any_sync(~0u, *guard.abort)) break;
    }
    // after an abort nobody else waits for the copies in flight
    if (*guard.abort && lane == 0) {
      const uint32_t from = gt > C::kStages ? gt - C::kStages : 0;
      for (uint32_t g = from; g < gt; ++g) {
        const long long t0 = clock64();
        while (!mbar_try_wait(&s.full[g % C::kStages], (g / C::kStages) & 1) &&
               clock64() - t0 < kWaitLimitCycles) {
        }
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int gid = lane >> 2, tig = lane & 3;
  const int box_log2 = 31 - __clz(box);
  // byte strides between 16-key groups and 64-column halves of a stage
  const uint32_t group = box == 16 ? 16 * D * 2 : 16 * 128;
  const uint32_t half = (uint32_t)box * 128;
  const uint32_t k_row = ((lane & 7) + ((lane >> 3) & 1) * 8) * 128;
  const uint32_t v_row = ((lane & 7) + (lane >> 4) * 8) * 128;
  const float scale2 = a.scale * kLog2e;
  const float cap2 = a.softcap * kLog2e;
  const float to_cap = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q);

  while (w.x < end) {
    const sched::Piece pc = sched::next(a, ph, pre, blockIdx.x, end, w);
    const uint32_t g0 = gt;
    // lane r keeps row r
    sched::Row row;
    row.lo = 0, row.hi = 0x7fffffff, row.at = 0, row.lse = 0;
    if (lane < pc.rows) row = sched::row_of(a, pre, pc.h, pc.row0 + lane);
    // keys that every row sees
    const int lo_all = __reduce_max_sync(~0u, row.lo), hi_all = __reduce_min_sync(~0u, row.hi);
    for (int i = tid; i < NT * 8 * (D / 8); i += kConsumers * 32) {
      const int r = i / (D / 8), v = i % (D / 8);
      int4 x = make_int4(0, 0, 0, 0);
      if (r < pc.rows)
        x = __ldg(reinterpret_cast<const int4*>(
                Q + sched::row_of(a, pre, pc.h, pc.row0 + r).at) + v);
      *reinterpret_cast<int4*>(qs + r * C::kQPitch + v * 16) = x;
    }
    named_sync(1, kConsumers * 32);
    // B = Q^T: one ldmatrix gives both halves of 16 d columns for two n-tiles or steps
    const uint32_t q_at = smem_u32(qs) + (lane & 7) * C::kQPitch + (lane >> 3) * 16;
    const uint32_t q_at2 =
        smem_u32(qs) + ((lane & 7) + (lane >> 4) * 8) * C::kQPitch + ((lane >> 3) & 1) * 16;
    uint32_t qf[kQRegs ? NT : 1][kQRegs ? D / 32 : 1][4];
    if constexpr (kQRegs) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < D / 32; ++k) ldsm4(qf[n][k], q_at + n * 8 * C::kQPitch + k * 64);
    }
    int lo[NT][2], hi[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lo[n][i] = __shfl_sync(~0u, row.lo, n * 8 + tig * 2 + i);
        hi[n][i] = __shfl_sync(~0u, row.hi, n * 8 + tig * 2 + i);
      }
    float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) m[n][i] = -INFINITY, l[n][i] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][k][i] = 0.f;
    }
    // this warp's stages: every eighth
    gt += (warp - gt % kConsumers + kConsumers) % kConsumers;
    const uint32_t g1 = g0 + (uint32_t)(pc.t1 - pc.t0);
    for (; gt < g1; gt += kConsumers) {
      const int st = gt % C::kStages;
      const int j0 = (pc.t0 + (int)(gt - g0)) * kTile;
      // after an abort every warp still runs through all pieces (their merges
      // are block-wide), with waits that return at once
      if (!__all_sync(~0u, mbar_wait(&s.full[st], (gt / C::kStages) & 1, guard))) break;
      const uint32_t kb = smem_u32(ring + st * C::kStage);
      const uint32_t vb = kb + C::kHalf;
      if (j0 < pc.lo || j0 + kTile > pc.hi) {
        // rows of V that no query sees may hold anything: 0 * NaN must not reach O
        const int j = j0 + lane;
        if (j < pc.lo || j >= pc.hi) {
          uint8_t* vr = ring + st * C::kStage + C::kHalf + (lane >> box_log2) * (box * D * 2) +
                        (lane & (box - 1)) * 128;
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<int4*>(vr + h * half)[i] = make_int4(0, 0, 0, 0);
        }
        fence_async_smem();     // the next load into these rows comes after
        __syncwarp();
      }
      float x[2][NT][4];
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[g][n][i] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t at = kb + (k / 4) * half + k_row +
                            ((((k % 4) * 2 + (lane >> 4)) ^ (lane & 7)) << 4);
        uint32_t f[2][4];
        ldsm4(f[0], at);
        ldsm4(f[1], at + group);
        if constexpr (kQRegs) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int g = 0; g < 2; ++g)
              mma16816(x[g][n], f[g], qf[n][k / 2][(k % 2) * 2], qf[n][k / 2][(k % 2) * 2 + 1]);
        } else {
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t q[4];
            ldsm4(q, q_at2 + n * 8 * C::kQPitch + k * 32);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              mma16816(x[g][n], f[g], q[0], q[1]);
              mma16816(x[g][n + 1], f[g], q[2], q[3]);
            }
          }
        }
      }
      if (a.softcap > 0.f) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[g][n][i] = cap2 * tanh_ex2(x[g][n][i] * to_cap);
      } else {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[g][n][i] *= scale2;
      }
      if (j0 < lo_all || j0 + kTile > hi_all) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + g * 16 + gid + (i >> 1) * 8;
              if (j < lo[n][i & 1] || j >= hi[n][i & 1]) x[g][n][i] = -INFINITY;
            }
      }
      uint32_t pf[2][NT][2];
      bool moved = false;
      float corr[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = fmaxf(fmaxf(x[0][n][i], x[0][n][i + 2]), fmaxf(x[1][n][i], x[1][n][i + 2]));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
          top = fmaxf(top, m[n][i]);
          const float ref = top == -INFINITY ? 0.f : top;
          moved |= top > m[n][i];
          corr[n][i] = ex2(m[n][i] - ref);
          m[n][i] = top;
          float sum = 0.f;
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p = ex2(x[g][n][i + 2 * e] - ref);
              x[g][n][i + 2 * e] = p;
              sum += p;
            }
          l[n][i] = l[n][i] * corr[n][i] + sum;
        }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][k][i] *= corr[n][i & 1];
      }
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            pf[g][n][e] = transpose8x8(pack_bf16(x[g][n][2 * e], x[g][n][2 * e + 1]));
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t f[4];
          ldsm4t(f, vb + g * group + (k / 4) * half + v_row +
                        ((((k % 4) * 2 + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(o[n][k], f, pf[g][n][0], pf[g][n][1]);
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.empty[st]);
    }
    gt = g1;

    // merge the warps that had a stage of this piece
    const int parts = min(kConsumers, (int)(g1 - g0));
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float y = l[n][i];
        y += __shfl_xor_sync(~0u, y, 4);
        y += __shfl_xor_sync(~0u, y, 8);
        y += __shfl_xor_sync(~0u, y, 16);
        if (gid == 0) {
          s.m[warp][n * 8 + tig * 2 + i] = m[n][i];
          s.l[warp][n * 8 + tig * 2 + i] = y;
        }
      }
    const int first = (int)(g0 % kConsumers);
    const bool part = (warp - first + kConsumers) % kConsumers < parts;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n * 8 >= pc.rows) break;
      if (part) {
        float* to = merge + warp * 8 * C::kPitch;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            to[(tig * 2 + (i & 1)) * C::kPitch + k * 16 + gid + (i >> 1) * 8] = o[n][k][i];
      }
      named_sync(1, kConsumers * 32);
      constexpr int kPer = D / 32;
      for (int q = warp; q < 8 && n * 8 + q < pc.rows; q += kConsumers) {   // this warp's rows
        const int r = n * 8 + q;
        float top = -INFINITY, sum = 0.f, acc[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
        for (int i = 0; i < parts; ++i) top = fmaxf(top, s.m[(first + i) % kConsumers][r]);
        const float ref = top == -INFINITY ? 0.f : top;
        for (int i = 0; i < parts; ++i) {
          const int p = (first + i) % kConsumers;
          const float c = ex2(s.m[p][r] - ref);
          sum = fmaf(c, s.l[p][r], sum);
          const float* from = merge + (p * 8 + q) * C::kPitch + lane * kPer;
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] = fmaf(c, from[e], acc[e]);
        }
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        const float lse2 = top + log2f(sum);
        const long long out = __shfl_sync(~0u, row.at, r), out_lse = __shfl_sync(~0u, row.lse, r);
        if (pc.slot < 0) {
          uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.O) + out +
                                                     lane * kPer);
#pragma unroll
          for (int e = 0; e < kPer; e += 2)
            to[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
          if (lane == 0) a.LSE[out_lse] = lse2 * kLn2;
        } else {
          const long long at = (long long)pc.slot * ph.rows + r;
#pragma unroll
          for (int e = 0; e < kPer; e += 2)
            *reinterpret_cast<float2*>(ph.o + at * D + lane * kPer + e) =
                make_float2(acc[e] * inv, acc[e + 1] * inv);
          if (lane == 0) ph.lse[at] = lse2;
        }
      }
      named_sync(1, kConsumers * 32);
    }
  }
}

template <int D, int NT>
cudaError_t launch(const PagedArgs& a, bool pre, const CUtensorMap& km, const CUtensorMap& vm,
                   cudaStream_t st) {
  using C = Cfg<D, NT>;
  constexpr int bytes = C::kRing + C::kMerge + C::kQ + 1024;
  static_assert(bytes + sizeof(Control) <= 227 * 1024, "shared memory");
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(mma_kernel<D, NT>), bytes))
    return e;
  mma_kernel<D, NT><<<(pre ? a.pre : a.own).n, C::kThreads, bytes, st>>>(
      a, pre, km, vm, debug_stall_cycles(kStallFwd));
  count_launch();
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const PagedArgs& a, bool pre, const CUtensorMap& km, const CUtensorMap& vm,
                     cudaStream_t st) {
  const int rows = (pre ? a.pre : a.own).rows;
  if (rows <= 8) return launch<D, 1>(a, pre, km, vm, st);
  if (rows <= 16) return launch<D, 2>(a, pre, km, vm, st);
  return launch<D, 4>(a, pre, km, vm, st);
}

}  // namespace

cudaError_t paged_mma(const PagedArgs& a, bool pre, cudaStream_t st) {
  CUtensorMap km, vm;
  const int ps = 1 << a.c.page_log2, box = ps < kTile ? ps : kTile;
  if (!make_tmap_pages(&km, a.K, a.c.d, ps, a.c.Hkv, a.c.pages, a.c.page_stride, box) ||
      !make_tmap_pages(&vm, a.V, a.c.d, ps, a.c.Hkv, a.c.pages, a.c.page_stride, box))
    return cudaErrorInvalidValue;
  return a.c.d == 128 ? launch_d<128>(a, pre, km, vm, st) : launch_d<64>(a, pre, km, vm, st);
}

}  // namespace fa
