// Paged attention for many query rows per KV head (a batch behind a shared
// prefix, long chunks of new tokens): bound by the tensor cores and the softmax
// between the two products, so S = Q K^T and O += P V run on tcgen05 with
// S, P and O in tensor memory.
//
// A stream is a CTA (one per SM): it walks its share of the 128-key tiles
// (paged_sched.cuh). Two softmax warpgroups keep the tensor core busy in
// turn, in one of two forms:
//  * two query tiles (more than 128 packed rows): warpgroup t has rows
//    128 t .. 128 t + 127 of the item, and every K/V tile serves both;
//  * one query tile: the warpgroups take the item's key tiles alternately, with running
//    statistics and an accumulator each. At the end each reads half the columns of both
//    accumulators (a row is the same TMEM lane in both) and joins them.
//
// K and V pages are copied by three loader warps with cp.async (any page size;
// a TMA box ends with its page, and at 16 tokens a page the boxes of one 128-key tile cost
// their issuing thread 6,900 cycles, twice what the tile's products and softmax take).
// They are written in the 128-byte swizzled layout of the MMA descriptors: 64-column
// block cb at 16 KB * cb, row r at 128 r, 16-byte chunk c at c ^ (r & 7). Each
// copying thread's arrival on a tile's barrier is tied to its copies, so loaders never
// wait for data, only for free slots; the MMA thread orders the landed bytes before
// its reads with a proxy fence.
//
// The running maximum is a reference that moves only when a tile exceeds it by 2^8 (the
// recurrence holds for any reference), so most tiles leave the accumulator alone.
// P is rounded to bf16 for the second product (the row sum takes it unrounded); sums, statistics
// and O stay in fp32. The rounding of P is of the size of O's own: together they are off by 2.3e-3
// (relative norm against 64 bits, 1,000 random keys), O's alone by 1.7e-3. A second number for the
// rest of P, as in paged_mma.cu, gives 1.7e-3 too, and room for it is there (the lower half of
// S), but the products and the softmax are the bound here: 256 rows over 8 sequences of 4,096 tokens
// take 76 us instead of 63, a batch of 64 behind 4,096 tokens 30 instead of 26.
#include <math.h>

#include "paged_sched.cuh"
#include "sm100_common.cuh"

namespace fa {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kLoaders = 3;            // warps 0, 2 and 3
constexpr int kM = kTcRows, kN = 1 << kTcTileLog2;  // query rows and keys of a tile
constexpr float kTau = 8.0f;           // slack of the reference maximum, log2 units
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxSlots = 8;

// kTwo: two query tiles.
template <int D, bool kTwo>
struct Cfg {
  static constexpr int kSlots = D == 64 ? 8 : 5;
  static constexpr int kTileBytes = kN * D * 2;      // one K or V tile
  static constexpr int kQBytes = kM * D * 2;
  static constexpr int kBlock = 128 * 128;           // one 64-column block
  static constexpr int kOffKV = (kTwo ? 2 : 1) * kQBytes;
  static constexpr int kOffStat = kOffKV + kSlots * kTileBytes;
  static constexpr int kBytes = kOffStat + (kTwo ? 0 : 2 * kM * 8) + 1024;
  static constexpr uint32_t kS = 128;                // TMEM columns: S_t at 128 t,
  static constexpr uint32_t kO = 256;                // O_t at 256 + D t,
  static constexpr uint32_t kP = 64;                 // P_t in the upper half of S_t
};

struct Control {
  uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots];
  uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_ready[2];
  uint64_t done, never;
  uint32_t tmem;
  int abort, skip;
  sched::Walk walk[8];                   // of the softmax warps, out of their registers
};

// Position of a tile in the order of loading and use, from the piece's first: two
// query tiles use K0 V0 K1 V1 ..., one query tile K0 K1 V0 K2 V1 ... (the scores of
// both warpgroups run ahead).
template <bool kTwo>
__device__ __forceinline__ uint32_t k_at(uint32_t j) {
  return kTwo ? 2 * j : (j ? 2 * j - 1 : 0);
}
template <bool kTwo>
__device__ __forceinline__ uint32_t v_at(uint32_t j, uint32_t tiles) {
  return kTwo ? 2 * j + 1 : (j + 1 < tiles ? 2 * j + 2 : 2 * tiles - 1);
}

__device__ __forceinline__ void copy16(uint32_t dst, const char* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(bytes)
               : "memory");
}
// Arrives on `bar` (whose count includes it) when this thread's copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// 32 bytes of registers to global memory, on a 32-byte boundary.
static_assert(kPartialAlign % 32 == 0, "partial results go out with store32");
__device__ __forceinline__ void store32(float* to, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
__device__ __forceinline__ void copy_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// kRare: a shared phase under a window, where rows that no query sees may lie between others
// (sched::seen_of), or a wide soft cap (soft_cap). Code for them in the usual kernel, never run,
// costs it up to 4 %.
template <int D, bool kTwo, bool kRare>
__global__ void __launch_bounds__(kThreads, 1)
    tc_kernel(const __grid_constant__ PagedArgs a, const bool pre, const long long stall) {
  using C = Cfg<D, kTwo>;
  constexpr uint32_t kSlots = C::kSlots;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control s;
  uint8_t* const base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Phase& ph = pre ? a.pre : a.own;
  warm_args(a);
  chain_next();
  sched::Walk w;
  if (!sched::begin(a, pre, blockIdx.x, w)) {            // the same answer in every warp
    chain_end();
    return;
  }
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < kSlots; ++i) {
      mbar_init(&s.kv_full[i], kLoaders * 32);
      mbar_init(&s.kv_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s.q_full[t], kTwo ? 4 : 8);
      mbar_init(&s.s_full[t], 1);
      mbar_init(&s.p_half[t], 4);
      mbar_init(&s.p_full[t], 4);
      mbar_init(&s.o_ready[t], 1);
    }
    mbar_init(&s.done, 1);
    mbar_init(&s.never, 1);
    s.abort = 0;
    s.skip = *reinterpret_cast<volatile unsigned*>(a.c.err) & kErrTimeout;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&s.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = s.tmem;
  if (s.skip) {                                          // nothing is in flight yet
    __syncthreads();
    if (warp == 2) tmem_dealloc(tm, 512);
    chain_end();
    return;
  }
  const Guard guard{&s.abort, a.c.err};
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait_ready_first(bar, parity, guard);
  };

  // Softmax warps: row `r` of query tile t (of the one query tile).
  const int t = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
  const int item_row = kTwo ? t * kM + r : r;
  sched::Piece pc;
  sched::Row row;
  // Q of a piece: this warp's rows of it (half of them, when two warpgroups share a tile),
  // whole rows at a time, first into registers ...
  constexpr int kQVecs = D / 8, kQRows = 32 / kQVecs, kQLoads = (kTwo ? 32 : 16) / kQRows;
  const int q_chunk = lane % kQVecs, q_row = (kTwo ? 0 : t * 16) + lane / kQVecs;
  auto next_piece = [&](int4 (&x)[kQLoads]) {
    sched::Walk v = s.walk[warp - 4];
    pc = sched::next(a, pre, v);
    __syncwarp();
    if (lane == 0) s.walk[warp - 4] = v;
    __syncwarp();
    row.lo = 0, row.hi = 0x7fffffff, row.out = 0;
    if (item_row < pc.rows) row.out = sched::out_of(a, pre, pc, item_row);
#pragma unroll
    for (int i = 0; i < kQLoads; ++i) {
      const int rr = q_row + i * kQRows, out = __shfl_sync(~0u, row.out, rr);
      x[i] = make_int4(0, 0, 0, 0);
      if ((kTwo ? t * kM : 0) + (warp & 3) * 32 + rr < pc.rows)
        x[i] = __ldg(reinterpret_cast<const int4*>(static_cast<const __nv_bfloat16*>(a.Q) +
                                                   (size_t)out * D) + q_chunk);
    }
    if (item_row < pc.rows) row = sched::row_of(a, pre, pc, item_row);   // Q is on its way
  };
  // ... and, once nothing reads the last piece's any more, into the swizzled tile.
  auto give_q = [&](const int4 (&x)[kQLoads]) {
    uint8_t* to = base + (kTwo ? t * C::kQBytes : 0) + (q_chunk >> 3) * C::kBlock;
#pragma unroll
    for (int i = 0; i < kQLoads; ++i) {
      const int rr = (warp & 3) * 32 + q_row + i * kQRows;
      *reinterpret_cast<int4*>(to + rr * 128 + (((q_chunk & 7) ^ (rr & 7)) << 4)) = x[i];
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.q_full[kTwo ? t : 0]);
  };

  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------ loaders
    const int me = warp == 0 ? 0 : warp - 1;
    uint32_t n = 0;                                      // tiles issued
    bool ok = true;
    while (ok && w.x < w.end) {
      const sched::Piece pc = sched::next(a, pre, w);
      const int* trow = sched::table_row(a, pc.table);
      const uint32_t tiles = pc.t1 - pc.t0;
      const long long head = (long long)pc.h * a.c.head_bytes;
      const int last = pc.hi > pc.lo ? (pc.hi - 1) >> a.c.page_log2 : -1;
      // lane i looks up the page of keys 16 i .. 16 i + 15 of a tile (pages hold 16 keys or
      // more), one tile ahead
      auto look_up = [&](uint32_t j) {
        const int e = ((pc.t0 + (int)j) * kN + (lane & 7) * 16) >> a.c.page_log2;
        const int page = e <= last ? __ldg(trow + e) : 0;
        return (unsigned)page < (unsigned)a.c.pages ? page : 0;
      };
      int page_n = look_up(0), page_k = 0, page_v = 0;   // of the next K, the last K, the next V
      for (uint32_t i = 0; i < 2 * tiles; ++i, ++n) {
        // the i-th tile in order of use: which of K and V, and its index
        uint32_t j;
        bool is_v;
        if (kTwo) {
          j = i >> 1, is_v = i & 1;
        } else {
          is_v = i + 1 == 2 * tiles || (i && !(i & 1));
          j = is_v ? (i + 1 == 2 * tiles ? tiles - 1 : i / 2 - 1) : (i + 1) / 2;
        }
        const uint32_t slot = n % kSlots;
        if (n >= kSlots && !__all_sync(~0u, wait(&s.kv_empty[slot], ((n / kSlots) & 1) ^ 1))) {
          ok = false;
          break;
        }
        const uint32_t to = smem_u32(base + C::kOffKV + slot * C::kTileBytes);
        const int j0 = (pc.t0 + (int)j) * kN;
        const char* from = is_v ? a.V : a.K;
        if (!is_v) {
          page_v = page_k;
          page_k = page_n;
          page_n = look_up(j + 1);
        }
        // V_j follows K_j, or (one query tile, but for the last) K_{j+1}
        const int page = is_v && !kTwo && j + 1 < tiles ? page_v : page_k;
        const bool edge = j0 < pc.lo || j0 + kN > pc.hi;
        constexpr int kVecs = D / 8, kRows = 32 / kVecs;  // chunks of a row; rows of an instruction
        constexpr int kGroup = 16 / kRows;               // instructions for 16 keys
        const int c = lane % kVecs, rl = lane / kVecs;
        // 16 keys of a head and page are contiguous: the loaders take them in turn
        for (int g = me; g < kN / 16; g += kLoaders) {
          const int pg = __shfl_sync(~0u, page, g);
          const char* src = from + pg * a.c.page_stride + head +
                            (long long)((j0 + g * 16) & ((1 << a.c.page_log2) - 1)) * (D * 2) +
                            lane * 16;
          const uint32_t dst = to + (c >> 3) * C::kBlock + g * 16 * 128;
          unsigned seen = ~0u;
          if constexpr (kRare) seen = sched::seen_of(a, pc, j0 + g * 16, pre && pc.len);
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            const int r = i * kRows + rl, j = j0 + g * 16 + r;
            // rows that no query sees are not read and count as zero
            const bool out = edge && (j < pc.lo || j >= pc.hi);
            const int bytes = out || (kRare && !((seen >> r) & 1)) ? 0 : 16;
            copy16(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4), src + i * 512, bytes);
          }
        }
        copy_arrive(&s.kv_full[slot]);
      }
    }
    copy_wait_all();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_bf16(kM, kN, false, false);
      constexpr uint32_t id_o = idesc_bf16(kM, D, false, true);
      const uint64_t dq0 = sdesc_sw128(smem_u32(base), 16, 1024);
      const uint64_t dk0 = sdesc_sw128(smem_u32(base + C::kOffKV), 16, 1024);
      const uint64_t dv0 = sdesc_sw128(smem_u32(base + C::kOffKV), C::kBlock, 1024);
      auto slot_of = [&](uint32_t n) { return n % kSlots; };
      auto have = [&](uint32_t n) {
        const bool got = wait(&s.kv_full[slot_of(n)], (n / kSlots) & 1);
        fence_async_smem();
        return got;
      };
      auto release = [&](uint32_t n) { mma_commit(&s.kv_empty[slot_of(n)]); };
      // S_t = Q K^T with the tile at ring position n
      auto issue_s = [&](int t, uint32_t n) {
        const uint64_t dq = sdesc_at(dq0, kTwo ? t * C::kQBytes : 0);
        const uint64_t dk = sdesc_at(dk0, slot_of(n) * C::kTileBytes);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * C::kBlock + (k & 3) * 32;
          mma_ss(tm + t * C::kS, sdesc_at(dq, off), sdesc_at(dk, off), id_s, k > 0);
        }
        mma_commit(&s.s_full[t]);
      };
      // O_t (+)= P_t V over keys 64 half .. 64 half + 63 of the tile at ring position n
      auto issue_pv = [&](int t, uint32_t n, bool acc, int half) {
        const uint64_t dv = sdesc_at(dv0, slot_of(n) * C::kTileBytes);
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          const int k = 4 * half + k4;
          mma_ts(tm + C::kO + t * D, tm + t * C::kS + C::kP + k * 8, sdesc_at(dv, k * 16 * 128),
                 id_o, acc || k > 0);
        }
      };
      uint32_t cnt[2] = {0, 0};                          // tiles of each warpgroup so far
      auto pv = [&](int t, uint32_t n, bool acc) {
        if (!wait(&s.p_half[t], cnt[t] & 1)) return false;
        tc_fence_after();
        issue_pv(t, n, acc, 0);
        if (!wait(&s.p_full[t], cnt[t] & 1)) return false;
        tc_fence_after();
        issue_pv(t, n, acc, 1);
        ++cnt[t];
        return true;
      };
      bool ok = injected_stall(&s.never, stall, guard);
      uint32_t n0 = 0;
      for (uint32_t np = 0; ok && w.x < w.end; ++np) {
        const sched::Piece pc = sched::next(a, pre, w);
        const uint32_t tiles = pc.t1 - pc.t0;
        if (kTwo) {
          // the K tile serves both query tiles; warpgroup 1 runs half a tile behind
          ok = wait(&s.q_full[0], np & 1) && have(n0);
          if (!ok) break;
          tc_fence_after();
          issue_s(0, n0);
          if (!(ok = wait(&s.q_full[1], np & 1))) break;
          tc_fence_after();
          issue_s(1, n0);
          release(n0);
          for (uint32_t j = 0; j < tiles; ++j) {
            const bool more = j + 1 < tiles;
            const uint32_t nv = n0 + v_at<true>(j, tiles), nk = n0 + k_at<true>(j + 1);
            if (!(ok = have(nv) && (!more || have(nk)) && pv(0, nv, j > 0))) break;
            if (more) issue_s(0, nk);
            else mma_commit(&s.o_ready[0]);
            if (!(ok = pv(1, nv, j > 0))) break;
            release(nv);
            if (more) {
              issue_s(1, nk);
              release(nk);
            } else {
              mma_commit(&s.o_ready[1]);
            }
          }
        } else {
          if (!(ok = wait(&s.q_full[0], np & 1))) break;
          for (uint32_t j = 0; j < min(2u, tiles); ++j) {
            const uint32_t nk = n0 + k_at<false>(j);
            if (!(ok = have(nk))) break;
            tc_fence_after();
            issue_s(j, nk);
            release(nk);
          }
          for (uint32_t j = 0; ok && j < tiles; ++j) {
            const int t = j & 1;
            const uint32_t nv = n0 + v_at<false>(j, tiles), nk = n0 + k_at<false>(j + 2);
            const bool more = j + 2 < tiles;
            if (!(ok = have(nv) && (!more || have(nk)) && pv(t, nv, j > 1))) break;
            release(nv);
            if (more) {
              issue_s(t, nk);
              release(nk);
            }
          }
          if (ok) {
            mma_commit(&s.o_ready[0]);
            mma_commit(&s.o_ready[1]);
          }
        }
        n0 += 2 * tiles;
      }
      // no MMA may still run when TMEM is freed, after an abort either
      mma_commit(&s.done);
      const long long t0 = clock64();
      while (!mbar_try_wait(&s.done, 0) && clock64() - t0 < kWaitLimitCycles) {
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_reg = tm + t * C::kS + lanes;
    const uint32_t o_reg = tm + C::kO + t * D + lanes;
    const bool xform = a.softcap > 0.f || a.scale <= 0.f;
    const float scale2 = a.scale * kLog2e;
    const bool wide = kRare && a.softcap > kWideCap;
    const float c = wide ? kLog2e : xform ? 1.f : scale2;
    const float cap2 = a.softcap * kLog2e;
    const float to_cap = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
    uint32_t cnt = 0;                                    // this warpgroup's tiles so far
    if (lane == 0) s.walk[warp - 4] = w;
    __syncwarp();
    {
      int4 q[kQLoads];
      next_piece(q);
      give_q(q);
    }
    for (uint32_t np = 0;; ++np) {
      const int lo_all = __reduce_max_sync(~0u, row.lo), hi_all = __reduce_min_sync(~0u, row.hi);
      float m_ref = -INFINITY, l = 0.f;
      bool first = true;
      for (int j = pc.t0 + (kTwo ? 0 : t); j < pc.t1; j += kTwo ? 1 : 2) {
        if (!__all_sync(~0u, wait(&s.s_full[t], cnt & 1))) break;   // whole warps go on or not
        tc_fence_after();
        uint32_t x[128];
        tmem_ld128(s_reg, x);
        if (xform) {
          if (wide) {
            const float inv = cap_inverse(a.softcap);
#pragma unroll
            for (int i = 0; i < 128; ++i)
              x[i] = __float_as_uint(soft_cap(__uint_as_float(x[i]) * a.scale, a.softcap, inv));
          } else if (a.softcap > 0.f) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              x[i] = __float_as_uint(cap2 * tanh_ex2(__uint_as_float(x[i]) * to_cap));
          } else {
#pragma unroll
            for (int i = 0; i < 128; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * scale2);
          }
        }
        const int j0 = j * kN;
        if (j0 < lo_all || j0 + kN > hi_all) {
          const int lo = row.lo - j0, hi = row.hi - j0;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i < lo || i >= hi) x[i] = __float_as_uint(-INFINITY);
        }
        // row maximum in eight chains
        float m8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t* v = &x[16 * k];
          float m = fmax3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
#pragma unroll
          for (int i = 3; i < 15; i += 2)
            m = fmax3(m, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
          m8[k] = fmaxf(m, __uint_as_float(v[15]));
        }
        const float top = c * fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                                    fmaxf(m8[6], m8[7]));
        const bool grow = top > m_ref + kTau;
        float alpha = 1.f;
        if (grow) {
          alpha = ex2(m_ref - top);                      // 0 without a reference yet
          m_ref = top;
          l *= alpha;
        }
        const float mu = m_ref == -INFINITY ? 0.f : m_ref;
        const float2 c2 = make_float2(c, c), nmu2 = make_float2(-mu, -mu);
        float2 acc[4] = {};
        // P in two halves: P V of the first 64 keys starts while the second is computed
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 z = ffma2(make_float2(__uint_as_float(x[64 * hf + 2 * i]),
                                               __uint_as_float(x[64 * hf + 2 * i + 1])), c2, nmu2);
            const float2 e = make_float2(ex2(z.x), ex2(z.y));
            acc[i & 3] = fadd2(acc[i & 3], e);
            pk[i] = pack_bf16(e.x, e.y);
          }
          tmem_st32(s_reg + C::kP + 32 * hf, pk);
          // earlier P V are complete (the commit behind S_t came after them)
          if (hf == 0 && __any_sync(~0u, grow && !first)) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              uint32_t o[32];
              tmem_ld32(o_reg + k * 32, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(o_reg + k * 32, o);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(hf ? &s.p_full[t] : &s.p_half[t]);
        }
        const float2 s01 = fadd2(acc[0], acc[1]), s23 = fadd2(acc[2], acc[3]);
        l += (s01.x + s01.y) + (s23.x + s23.y);
        first = false;
        ++cnt;
      }
      // The piece is done but for its result. The next one's Q goes in before the result goes
      // out, so that its first scores are not waited for (and with one query tile, whose
      // pieces are short, it is fetched before the last P V has completed).
      const int slot = pc.slot, out = row.out;
      const bool real = item_row < pc.rows, both = pc.t1 - pc.t0 > 1;
      const bool more = s.walk[warp - 4].x < s.walk[warp - 4].end;
      int4 q[kQLoads];
      if (!kTwo && more) next_piece(q);
      // every S and P V has completed: the accumulators may be read, the Q buffers overwritten
      bool got = wait(&s.o_ready[t], np & 1);
      if (!kTwo) got = wait(&s.o_ready[t ^ 1], np & 1) && got;
      got = __all_sync(~0u, got);
      tc_fence_after();
      if (kTwo && more) next_piece(q);
      if (more) give_q(q);
      // this thread's factors for the accumulators of warpgroups 0 and 1 (kTwo: its own)
      float f0, f1 = 0.f, lse2;
      if constexpr (kTwo) {
        f0 = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        lse2 = m_ref + log2f(l);
      } else {
        float2* const stat = reinterpret_cast<float2*>(base + C::kOffStat);   // (m, l) of both
        stat[t * kM + r] = make_float2(m_ref, l);
        named_sync(1, 256);
        const float2 a0 = stat[r], a1 = stat[kM + r];
        const float top = fmaxf(a0.x, a1.x), ref = top == -INFINITY ? 0.f : top;
        f0 = ex2(a0.x - ref), f1 = ex2(a1.x - ref);
        const float sum = f0 * a0.y + f1 * a1.y;
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        f0 *= inv, f1 *= inv;
        lse2 = top + log2f(sum);
      }
      const long long at = (long long)slot * ph.rows + (kTwo ? t * kM : 0);   // partial row 0
      if (real && (kTwo || t == 0)) {
        if (slot < 0) a.LSE[out] = lse2 * kLn2;
        else ph.lse[at + r] = lse2;
      }
      // Partial results go out with a row in each lane, [32-byte chunk][row], so that a
      // warp writes 1 KB at once straight from its registers, and the join reads whole sectors.
      constexpr int kChunks = kTwo ? D / 32 : D / 64;    // 32 columns each
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int k = kTwo ? i : t * kChunks + i;
        uint32_t o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
        if (got) {
          tmem_ld32((kTwo ? o_reg : tm + C::kO + lanes) + k * 32, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
          if (!kTwo && both) {
            uint32_t o1[32];
            tmem_ld32(tm + C::kO + D + lanes + k * 32, o1);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e])));
          }
        }
        if (slot >= 0) {
          float* to = ph.o + at * D + (k * 4 * kM + r) * 8;
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8) store32(to + c8 * kM * 8, &o[8 * c8]);
        } else if (real) {
          uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.O) +
                                               (size_t)out * D + k * 32);
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8) {
            const uint32_t* v = &o[8 * c8];
            to[c8] = make_uint4(
                pack_bf16(__uint_as_float(v[0]), __uint_as_float(v[1])),
                pack_bf16(__uint_as_float(v[2]), __uint_as_float(v[3])),
                pack_bf16(__uint_as_float(v[4]), __uint_as_float(v[5])),
                pack_bf16(__uint_as_float(v[6]), __uint_as_float(v[7])));
          }
        }
      }
      // both warpgroups have read both accumulators before the next piece's P V
      if (!kTwo) {
        tc_fence_before();
        named_sync(1, 256);
      }
      tc_fence_before();
      if (!more) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
  chain_end();
}

template <int D, bool kTwo, bool kRare>
cudaError_t launch_as(const PagedArgs& a, bool pre, cudaStream_t st) {
  using C = Cfg<D, kTwo>;
  static_assert(C::kBytes + sizeof(Control) <= 227 * 1024, "shared memory");
  const auto kernel = tc_kernel<D, kTwo, kRare>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), C::kBytes))
    return e;
  return launch_chained(kernel, (pre ? a.pre : a.own).n, kThreads, C::kBytes, st,
                        !pre && a.shared, a, pre, debug_stall_cycles(kStallFwd));
}

template <int D, bool kTwo>
cudaError_t launch(const PagedArgs& a, bool pre, cudaStream_t st) {
  return (pre && a.wl >= 0) || a.softcap > kWideCap ? launch_as<D, kTwo, true>(a, pre, st)
                                                    : launch_as<D, kTwo, false>(a, pre, st);
}

}  // namespace

cudaError_t paged_tc(const PagedArgs& a, bool pre, cudaStream_t st) {
  const bool two = (pre ? a.pre : a.own).rows > kM;
  if (a.c.d == 128) return two ? launch<128, true>(a, pre, st) : launch<128, false>(a, pre, st);
  return two ? launch<64, true>(a, pre, st) : launch<64, false>(a, pre, st);
}

}  // namespace fa
