// Paged attention for few query rows per KV head (decoding): bound by reading K
// and V once, so the kernel is many independent streams of loads with just
// enough arithmetic behind each.
//
// A stream is a warp: it walks its share of the key tiles (paged_sched.cuh) with a
// ring of three 8 KB stages of its own (16 keys of d = 128 or 32 of d = 64), filled
// with cp.async and swizzled on the way (16-byte chunk c of a row goes to c ^ (row
// & 7), so that the eight rows of an ldmatrix hit different banks). Two blocks of four warps an
// SM keep up to 128 KB of loads in flight (at 6.5 TB/s over 148 SMs and ~1 us of
// latency 45 KB would do). Warps never meet: no barrier, no merge in shared memory. A
// first form with one TMA producer per SM and a merge per piece ran a ragged
// batch (page 16) at 3.5 TB/s: a 4 KB box cost the producer 260 cycles and a set-up or merge
// stalled the whole SM.
//
// The products are transposed so that the packed query rows are the narrow side:
//   S^T = K Q^T     m16n8k16, A = 16 keys x 16 of d (ldmatrix), B = Q^T in registers
//   O^T += V^T P^T  A = 16 of d x 16 keys (ldmatrix.trans), B = P^T
// with 8 query rows per n-tile: decoding has 1 to 8 rows per KV head, of which an
// m16 tile of queries would waste half or more. P^T comes from S^T's accumulator
// layout by an 8x8 transpose (movmatrix). The tensor pipe stays far from its limit, so
// mma.sync's lower peak costs nothing here.
//
// P goes into the second product as two bf16 numbers, its rounding and what that left
// (the row sum takes it unrounded), so the output's own rounding is the only one that
// counts; at the memory's pace the extra products cost at most 2 % (a ragged batch 104
// us, 102 without). Sums, maxima and O stay in fp32.
#include <math.h>

#include "paged_sched.cuh"
#include "sm100_common.cuh"

namespace fa {
namespace {

using namespace sm100;

constexpr int kStages = 3;
constexpr int kStageBytes = 8192;      // K and V, 4 KB each
constexpr int kSmem = kMmaWarps * kStages * kStageBytes + 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
// 16 bytes global -> shared; `bytes` of them are read, the rest become zero.
__device__ __forceinline__ void copy16(uint32_t dst, const char* src, int bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::256B [%0], [%1], 16, %2, %3;" ::"r"(
                   dst),
               "l"(src), "r"(bytes), "l"(policy)
               : "memory");
}
// K and V that one row tile reads leave L2 first: the partial results are to stay there.
__device__ __forceinline__ uint64_t l2_policy(bool once) {
  uint64_t p;
  if (once) asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Page numbers of a table row: 32 entries in the lanes, the next 32 on their way.
struct Pages {
  const int* row;
  int at, last, cur, nxt;
  __device__ void open(const int* r, int first, int last_entry) {
    row = r;
    at = first;
    last = last_entry;
    cur = load(at);
    nxt = load(at + 32);
  }
  __device__ int load(int i) {
    i += threadIdx.x & 31;
    return i <= last ? __ldg(row + i) : -1;
  }
  // the page of entry p, which never goes back (all lanes call it)
  __device__ int get(int p, int pages) {
    while (p - at >= 32) {
      at += 32;
      cur = nxt;
      nxt = load(at + 32);
    }
    const int page = __shfl_sync(~0u, cur, p - at);
    return (unsigned)page < (unsigned)pages ? page : 0;
  }
};

// NT: n-tiles of eight packed query rows.
template <int D, int NT>
__global__ void __launch_bounds__(kMmaWarps * 32, kMmaBlocksPerSm)
    mma_kernel(const __grid_constant__ PagedArgs a, const bool pre) {
  constexpr int kTile = 1 << mma_tile_log2(D), kGroups = kTile / 16;   // 16 keys a group
  constexpr int kGroupBytes = 16 * D * 2;
  constexpr int kRowVecs = D / 8;                            // 16-byte chunks of a row
  extern __shared__ uint8_t smem_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t ring = ((smem_u32(smem_raw) + 1023) & ~1023u) + warp * kStages * kStageBytes;
  const Phase& ph = pre ? a.pre : a.own;
  // neighbouring streams on different SMs: little work is spread over all of them
  const int stream = warp * gridDim.x + blockIdx.x;
  warm_args(a);
  chain_next();
  sched::Walk w;
  if (!sched::begin(a, pre, stream, w)) {
    chain_end();
    return;
  }

  const int gid = lane >> 2, tig = lane & 3;
  const uint32_t k_row = ((lane & 7) + ((lane >> 3) & 1) * 8) * 128;
  const uint32_t v_row = ((lane & 7) + (lane >> 4) * 8) * 128;
  const float scale2 = a.scale * kLog2e;
  const float cap2 = a.softcap * kLog2e;
  const float to_cap = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q);
  const uint64_t policy = l2_policy(ph.rt == 1);

  while (w.x < w.end) {
    const sched::Piece pc = sched::next(a, pre, w);
    Pages pages;
    pages.open(sched::table_row(a, pc.table), (pc.t0 * kTile) >> a.c.page_log2,
               pc.hi > pc.lo ? (pc.hi - 1) >> a.c.page_log2 : -1);
    const long long head = (long long)pc.h * a.c.head_bytes;

    const bool gaps = pre && pc.len;

    // tile t into its stage: 16 keys of one head and page are 16 * d contiguous elements
    auto load = [&](int t) {
      const uint32_t to = ring + (uint32_t)(t - pc.t0) % kStages * kStageBytes;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int j = t * kTile + g * 16;
        const int page = pages.get(j >> a.c.page_log2, a.c.pages);
        const long long off = page * a.c.page_stride + head +
                              (long long)(j & ((1 << a.c.page_log2) - 1)) * (D * 2) + lane * 16;
        const char* k = a.K + off;
        const char* v = a.V + off;
        const bool edge = j < pc.lo || j + 16 > pc.hi || gaps;
        const unsigned seen = edge ? sched::seen_of(a, pc, j, gaps) : ~0u;
#pragma unroll
        for (int i = 0; i < kGroupBytes / 512; ++i) {
          const int vec = i * 32 + lane, row = vec / kRowVecs, c = vec % kRowVecs;
          const uint32_t dst = to + g * kGroupBytes + (c >> 3) * 2048 + row * 128 +
                               (((c & 7) ^ (row & 7)) << 4);
          // rows that no query sees are not read and count as zero
          const int bytes = (seen >> row) & 1 ? 16 : 0;
          copy16(dst, k + i * 512, bytes, policy);
          copy16(dst + kStageBytes / 2, v + i * 512, bytes, policy);
        }
      }
    };
    // lane r keeps row r
    sched::Row row;
    row.lo = 0, row.hi = 0x7fffffff, row.out = 0;
    if (lane < pc.rows) row = sched::row_of(a, pre, pc, lane);
    uint32_t qf[NT][D / 16][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int out = __shfl_sync(~0u, row.out, n * 8 + gid);
      const uint32_t* from = reinterpret_cast<const uint32_t*>(Q + (size_t)out * D) + tig;
      const bool real = n * 8 + gid < pc.rows;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) qf[n][k][i] = real ? __ldg(from + k * 8 + i * 4) : 0u;
    }
    // keys that every row sees
    const int lo_all = __reduce_max_sync(~0u, row.lo), hi_all = __reduce_min_sync(~0u, row.hi);
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

    // one loop for filling the ring and working from it: code that runs once is slow (its
    // instructions come from L2)
    for (int t = pc.t0 - kStages; t < pc.t1; ++t) {
      if (t >= pc.t0) {
        const uint32_t kb = ring + (uint32_t)(t - pc.t0) % kStages * kStageBytes;
        const uint32_t vb = kb + kStageBytes / 2;
        const int j0 = t * kTile;
        copy_wait<kStages - 1>();
        __syncwarp();
        // two chains of products a group, for latency
        float x[kGroups][NT][4], y[kGroups][NT][4];
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[g][n][i] = y[g][n][i] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            uint32_t f[4];
            ldsm4(f, kb + g * kGroupBytes + (k / 4) * 2048 + k_row +
                         ((((k % 4) * 2 + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(k & 1 ? y[g][n] : x[g][n], f, qf[n][k][0], qf[n][k][1]);
          }
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float z = x[g][n][i] + y[g][n][i];
              if (a.softcap > kWideCap)
                z = kLog2e * soft_cap(z * a.scale, a.softcap, cap_inverse(a.softcap));
              else if (a.softcap > 0.f)
                z = cap2 * tanh_ex2(z * to_cap);
              else
                z *= scale2;
              x[g][n][i] = z;
            }
        if (j0 < lo_all || j0 + kTile > hi_all) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int lo = __shfl_sync(~0u, row.lo, n * 8 + tig * 2 + i);
              const int hi = __shfl_sync(~0u, row.hi, n * 8 + tig * 2 + i);
#pragma unroll
              for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int j = j0 + g * 16 + gid + e * 8;
                  if (j < lo || j >= hi) x[g][n][i + 2 * e] = -INFINITY;
                }
            }
        }
        bool moved = false;
        float corr[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(x[0][n][i], x[0][n][i + 2]);
            if constexpr (kGroups == 2) top = fmaxf(top, fmaxf(x[1][n][i], x[1][n][i + 2]));
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
            for (int g = 0; g < kGroups; ++g)
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
        uint32_t pf[kGroups][NT][2], pr[kGroups][NT][2];   // P rounded, and the rest
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a0 = x[g][n][2 * e], a1 = x[g][n][2 * e + 1];
              const uint32_t p = pack_bf16(a0, a1);
              pf[g][n][e] = transpose8x8(p);
              pr[g][n][e] = transpose8x8(pack_bf16(a0 - __uint_as_float(p << 16),
                                                   a1 - __uint_as_float(p & 0xffff0000u)));
            }
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t f[4];
            ldsm4t(f, vb + g * kGroupBytes + (k / 4) * 2048 + v_row +
                          ((((k % 4) * 2 + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(o[n][k], f, pf[g][n][0], pf[g][n][1]);
              mma16816(o[n][k], f, pr[g][n][0], pr[g][n][1]);
            }
          }
        __syncwarp();
      }
      if (t + kStages < pc.t1) load(t + kStages);
      copy_commit();
    }

#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float inv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[n][i];
        sum += __shfl_xor_sync(~0u, sum, 4);
        sum += __shfl_xor_sync(~0u, sum, 8);
        sum += __shfl_xor_sync(~0u, sum, 16);
        inv[i] = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        const int r = n * 8 + tig * 2 + i;
        const int out = __shfl_sync(~0u, row.out, r);
        if (gid == 0 && r < pc.rows) {
          const float lse2 = m[n][i] + log2f(sum);
          if (pc.slot < 0) a.LSE[out] = lse2 * kLn2;
          else ph.lse[(long long)pc.slot * ph.rows + r] = lse2;
        }
      }
      if (pc.slot < 0) {
        const int r = n * 8 + gid;
        const int out = __shfl_sync(~0u, row.out, r);
        uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.O) +
                                                   (size_t)out * D) + tig;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t v = transpose8x8(
                pack_bf16(o[n][k][2 * e] * inv[0], o[n][k][2 * e + 1] * inv[1]));
            if (r < pc.rows) to[k * 8 + e * 4] = v;
          }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = n * 8 + tig * 2 + i;
          float* to = ph.o + ((long long)pc.slot * ph.rows + r) * D + gid;
          if (r < pc.rows)
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              to[k * 16] = o[n][k][i] * inv[i];
              to[k * 16 + 8] = o[n][k][i + 2] * inv[i];
            }
        }
      }
    }
  }
  copy_wait<0>();
  chain_end();
}

template <int D, int NT>
cudaError_t launch(const PagedArgs& a, bool pre, cudaStream_t st) {
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(mma_kernel<D, NT>), kSmem))
    return e;
  return launch_chained(mma_kernel<D, NT>, (pre ? a.pre : a.own).n / kMmaWarps, kMmaWarps * 32,
                        kSmem, st, !pre && a.shared, a, pre);
}

template <int D>
cudaError_t launch_d(const PagedArgs& a, bool pre, cudaStream_t st) {
  switch ((pre ? a.pre : a.own).rows / 8) {
    case 1: return launch<D, 1>(a, pre, st);
    case 2: return launch<D, 2>(a, pre, st);
    default: return launch<D, 3>(a, pre, st);
  }
}

}  // namespace

cudaError_t paged_mma(const PagedArgs& a, bool pre, cudaStream_t st) {
  return a.c.d == 128 ? launch_d<128>(a, pre, st) : launch_d<64>(a, pre, st);
}

}  // namespace fa
