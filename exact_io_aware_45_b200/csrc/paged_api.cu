// C ABI of the paged cache and its attention: argument checks, workspace
// layout, kernel choice. See include/fa.h for the contract.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "paged.h"

namespace fa {

int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, unsigned to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}

int elem_bytes(int dtype) { return dtype == FA_F32 ? 4 : 2; }

// Checks a cache's description and fills the kernels' view of it.
fa_status view_of(const fa_cache* c, CacheView& v) {
  if (!c) return FA_ERR_INVALID_ARG;
  if (c->layers <= 0 || c->pages <= 0 || c->Hkv <= 0 || c->seqs <= 0 || c->seq_pages <= 0)
    return FA_ERR_INVALID_ARG;
  if (c->dtype != FA_F32 && c->dtype != FA_BF16) return FA_ERR_INVALID_ARG;
  if (c->d <= 0 || c->page_size <= 0) return FA_ERR_INVALID_ARG;
  if (c->d != 16 && c->d != 32 && c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  int lg = 4;
  while (lg < 8 && (1 << lg) != c->page_size) ++lg;
  if (lg == 8) return FA_ERR_UNSUPPORTED;
  const long long es = elem_bytes(c->dtype);
  const long long page = (long long)c->Hkv * c->page_size * c->d;
  if (page * es >= (1ll << 30) || c->pages >= (1 << 28) || c->layers >= (1 << 16) ||
      (long long)c->seq_pages * c->page_size >= (1ll << 30) ||
      (long long)c->seqs * c->seq_pages >= (1ll << 31) - (1 << 16))   // loops step past it
    return FA_ERR_UNSUPPORTED;
  if (c->page_stride < page || (c->layers > 1 && c->layer_stride < page))
    return FA_ERR_INVALID_ARG;
  if (c->page_stride >= (1ll << 36) || c->layer_stride >= (1ll << 44)) return FA_ERR_UNSUPPORTED;
  if ((c->page_stride * es) & 15 || (c->layers > 1 && ((c->layer_stride * es) & 15)))
    return FA_ERR_INVALID_ARG;
  if (!c->K || !c->V || !c->table || !c->lens || !c->refs || !c->err) return FA_ERR_INVALID_ARG;
  if (!aligned(c->K, 16) || !aligned(c->V, 16) || !aligned(c->table, 4) || !aligned(c->lens, 4) ||
      !aligned(c->refs, 4) || !aligned(c->err, 4))
    return FA_ERR_INVALID_ARG;
  v.K = static_cast<char*>(c->K);
  v.V = static_cast<char*>(c->V);
  v.layer_stride = c->layer_stride * es;
  v.page_stride = c->page_stride * es;
  v.layers = c->layers;
  v.pages = c->pages;
  v.width = c->seq_pages;
  v.slots = c->seqs;
  v.page_log2 = lg;
  v.row_bytes = (int)(c->d * es);
  v.head_bytes = c->page_size * v.row_bytes;
  v.page_bytes = c->Hkv * v.head_bytes;
  v.Hkv = c->Hkv;
  v.d = c->d;
  v.table = c->table;
  v.lens = c->lens;
  v.refs = c->refs;
  v.err = c->err;
  return FA_OK;
}

fa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Checks of a list of n int32 entries, and of the workspace.
bool bad_list(const int* p, int n) { return n > 0 && (!p || !aligned(p, 4)); }
fa_status check_ws(const CacheView& v, int n, const void* ws, size_t bytes) {
  if (!ws || !aligned(ws, 16) || bytes < cache_workspace_bytes(v.pages, v.slots, n))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Kernels of a phase: bf16 with d of 64 or 128 runs on the tensor cores, all else
// on the CUDA cores. There the kernel tiled in registers takes 64 rows at once, the other up
// to four: 64 sequences of 4 rows and 8 heads behind 4,096 tokens (fp32, d 128, 256 rows of the
// prefix) take 157 us with the first and 232 with the second, 16 of 16 rows and 4,000 tokens 329
// and 361. For 5 to 8 rows the second, in tiles of four, would be quicker: the same with 6 rows 319
// and 189, 32 sequences of 8 rows and 20 to 200 tokens (bf16, d 32) 16 and 14, 8 of 5 rows and 100
// to 4,000 (fp32, d 64) 48 and 31. The mma.sync kernel reads K and V once per 16 or 24 packed rows
// and is quick with short sequences; the tcgen05 kernel takes 128 or 256 rows at once, which
// costs an item more to begin and end. Two row tiles (25 to 32 rows) of d 128 bind the first by
// its work, so the second has them where a sequence may be long (`keys`: what its table can
// hold, since no length is known on the host: a table wider than its sequences is taken for long
// ones): 64 sequences of 20 to 300 tokens take 29 and 43 us, 32 of 100 to 2,000 37 and 44, 80 of
// 1,562 (behind 2,144 shared) 285 and 200, 8 of 8,192 91 and 66. At d 64 they are level.
// Where nothing can be long, up to 64 rows are quicker in tiles of 16 or 24: 61 sequences of
// 40 rows and 8 heads with 1 to 49 tokens behind 128 shared take 41 us, 74 with an item each.
enum Family { kSimt, kFma, kMma, kTc };
Family family(const CacheView& v, int rows, long long keys) {
  if (v.row_bytes != 2 * v.d || v.d < 64) return rows <= kSimtRows ? kSimt : kFma;
  const int most = keys <= 256 ? 64 : v.d == 64 || keys <= 1024 ? 32 : 24;
  return rows <= most ? kMma : kTc;
}

// Behind the prefix a sequence has at most what its table holds.
Family own_family(const PagedArgs& a) {
  return family(a.c, a.TG, ((long long)a.c.width << a.c.page_log2) - a.shared);
}
// A short prefix has few items, which the tcgen05 kernel begins side by side.
Family pre_family(const PagedArgs& a) {
  return family(a.c, a.B * a.TG, a.shared < 512 ? 512 : a.shared);
}

// The work division of a phase of `groups` sequences and KV heads with `rows`
// packed rows each, over `keys` keys at most. It depends on sizes and types only, so the
// workspace query and the call agree.
Phase divide(const CacheView& v, Family kind, int groups, int rows, long long keys, int sms) {
  Phase p;
  p.sms = sms;
  int per = 1;           // streams of a block
  switch (kind) {
    case kSimt:
      p.rows = rows <= 2 ? rows : kSimtRows;
      p.tile_log2 = kSimtTileLog2;
      p.n = sms * simt_blocks_per_sm(v.d, p.rows);
      // (4, 2, 4 of them: 64 sequences of 1 to 300 tokens 29 us instead of 19)
      p.over = 3;
      p.snap = 1;
      p.least = 2;
      break;
    case kFma:
      p.rows = kFmaRows;
      p.tile_log2 = kSimtTileLog2;
      p.n = sms * fma_blocks_per_sm(v.d);
      // a tile takes a lone block 1.5 us, and beginning little more: 89 sequences of 35 tokens 18
      // us, 2 with chunks of 64 tokens 30; 31 and 36 with (4, 2, 4)
      p.over = 1;
      p.snap = 1;
      p.least = 1;
      break;
    case kMma:
      // 17 to 24 rows are one tile where the heads alone fill the GPU (8 sequences of 8,192
      // tokens, 8 heads, d 128: 56 us, 84 as two of 16), else two, for latency (one of 3,000, 4
      // heads: 12.7 us, 14.3 as one). Tiles of 32 spill at d 128 and gained little at 64.
      p.rows = rows <= 8 ? 8 : groups >= 32 && (rows + 23) / 24 < (rows + 15) / 16 ? 24 : 16;
      p.tile_log2 = mma_tile_log2(v.d);
      per = kMmaWarps;
      p.n = sms * kMmaWarps * kMmaBlocksPerSm;
      break;
    case kTc:
      p.rows = rows <= kTcRows ? kTcRows : 2 * kTcRows;
      p.blocked = true;
      p.tile_log2 = kTcTileLog2;
      p.n = sms;
      // A piece costs a stream about 10 us beside its tiles of 2 us each; still, short
      // prefixes are cut down to single tiles: 512 tokens behind 128 sequences of 8 heads took
      // 98 us in one stream per head, 31 us in one per tile.
      p.over = 5;
      p.snap = 1;
      p.least = 1;
      break;
  }
  p.rt = (rows + p.rows - 1) / p.rows;
  p.items = groups * p.rt;
  // no more streams than the longest sequences could use
  const long long units = p.items * ((keys >> p.tile_log2) + 2 + p.over);
  const long long most = units / p.least + per;
  if (most < p.n) p.n = (int)(most / per * per);
  return p;
}

cudaError_t run_phase(const PagedArgs& a, bool pre, int dtype, cudaStream_t st) {
  switch (pre ? pre_family(a) : own_family(a)) {
    case kSimt: return paged_simt(a, pre, dtype, st);
    case kFma: return paged_fma(a, pre, dtype, st);
    case kMma: return paged_mma(a, pre, st);
    default: return paged_tc(a, pre, st);
  }
}

// Fills in both phases; false if their units or partial rows do not fit an int.
bool plan(PagedArgs& a, int sms) {
  const long long keys = (long long)a.c.width << a.c.page_log2;
  a.own = divide(a.c, own_family(a), a.B * a.c.Hkv, a.TG, keys - a.shared, sms);
  if (a.shared) a.pre = divide(a.c, pre_family(a), a.c.Hkv, a.B * a.TG, a.shared, sms);
  // The tcgen05 kernel leaves the memory idle and the mma.sync kernel the tensor cores: they
  // run side by side on different SMs. A tile of 256 rows takes an SM 2.2 us at d 128, 8 KB of an
  // own stream 0.14 us: 16, and 8 for 128 rows. At d 64 the tiles of both are half the work. 128
  // sequences with up to 2,048 tokens of their own behind 16,384 take 121 us (d 128) and 69 (d 64)
  // with 16, 144 and 74 with 12, 184 and 91 with 8, 119 and 87 with 22; 24 of them 43 and 33 with
  // 8, 58 and 30 with 4, 39 and 33 with 11.
  if (a.shared && pre_family(a) == kTc && own_family(a) == kMma)
    a.pre.yield = a.pre.rows == kTcRows ? 8 : 16;
  const long long most = keys / 16 + 8;
  for (const Phase* p : {&a.own, &a.pre})
    if (((long long)p->items + p->n) * p->rows >= (1ll << 31)) return false;
  return a.own.items * most < (1ll << 31) - (1 << 20) &&
         a.pre.items * most < (1ll << 31) - (1 << 20);
}

size_t phase_bytes(const Phase& p, int d, size_t* lse_at) {
  const size_t rows = (size_t)(p.items + p.n) * p.rows;
  *lse_at = align256(rows * d * 4);
  return *lse_at + align256(rows * 4);
}

// Where the partial results begin in a workspace.
char* partials_at(void* ws) {
  return reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws) + kPartialAlign - 1) &
                                 ~uintptr_t(kPartialAlign - 1));
}

fa_status check_fwd(const CacheView& v, int B, int T, int Hq, int shared) {
  if (B < 0 || T < 0 || Hq <= 0 || Hq % v.Hkv != 0 || shared < 0) return FA_ERR_INVALID_ARG;
  if (shared & ((1 << v.page_log2) - 1)) return FA_ERR_INVALID_ARG;
  if (shared > v.width << v.page_log2) return FA_ERR_INVALID_ARG;
  // packed rows, items and table indexes stay in int, and the join's grid in its limits
  if (B > 65535 || (long long)B * T * Hq >= (1ll << 28) || (long long)T * (Hq / v.Hkv) >= (1ll << 20))
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

void sizes(PagedArgs& a, const CacheView& v, int B, int T, int Hq, int shared) {
  a.c = v;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.G = Hq / v.Hkv;
  a.TG = T * a.G;
  a.shared = shared;
}

fa_status fwd(const fa_cache* cache, int layer, const void* Q, void* O, float* LSE,
              const int* seqs, int B, int T, int Hq, int shared, float scale, int causal,
              int window_left, float softcap, void* ws, size_t ws_bytes, void* stream) {
  reset_launch_count();
  PagedArgs a;
  CacheView v;
  if (fa_status s = view_of(cache, v)) return s;
  if (fa_status s = check_fwd(v, B, T, Hq, shared)) return s;
  if (layer < 0 || layer >= v.layers || (causal != 0 && causal != 1) || window_left < -1 ||
      !isfinite(scale) || !isfinite(softcap) || softcap < 0.f)
    return FA_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return FA_OK;
  if (!seqs && B > v.slots) return FA_ERR_INVALID_ARG;
  if (!Q || !O || !LSE || !aligned(Q, 16) || !aligned(O, 16) || !aligned(LSE, 4) ||
      !aligned(seqs, 4))
    return FA_ERR_INVALID_ARG;
  sizes(a, v, B, T, Hq, shared);
  a.K = v.K + layer * v.layer_stride;
  a.V = v.V + layer * v.layer_stride;
  a.Q = Q;
  a.O = O;
  a.LSE = LSE;
  a.seqs = seqs;
  a.causal = causal;
  a.wl = window_left;
  a.scale = scale;
  a.softcap = softcap;
  if (!plan(a, sm_count())) return FA_ERR_UNSUPPORTED;
  size_t own_lse, pre_lse;
  const size_t own = phase_bytes(a.own, v.d, &own_lse), pre = phase_bytes(a.pre, v.d, &pre_lse);
  if (!ws || !aligned(ws, kWorkspaceAlign)) return FA_ERR_INVALID_ARG;
  char* const w = partials_at(ws);
  if (ws_bytes < own + pre + (w - static_cast<char*>(ws))) return FA_ERR_INVALID_ARG;
  a.own.o = reinterpret_cast<float*>(w);
  a.own.lse = reinterpret_cast<float*>(w + own_lse);
  a.pre.o = reinterpret_cast<float*>(w + own);
  a.pre.lse = reinterpret_cast<float*>(w + own + pre_lse);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shared)
    if (cudaError_t e = run_phase(a, true, cache->dtype, st)) return from_cuda(e);
  if (cudaError_t e = run_phase(a, false, cache->dtype, st)) return from_cuda(e);
  return from_cuda(paged_join(a, cache->dtype, st));
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_cache_workspace_size(const fa_cache* cache, int n) {
  CacheView v;
  if (n < 0 || view_of(cache, v) != FA_OK) return 0;
  return cache_workspace_bytes(v.pages, v.slots, n);
}

fa_status fa_cache_extend(const fa_cache* cache, const int* seqs, int n, const int* cu_seqlens,
                          int tokens, int* pos, void* workspace, size_t workspace_bytes,
                          void* stream) {
  reset_launch_count();
  CacheView v;
  if (fa_status s = view_of(cache, v)) return s;
  if (n < 0 || n > v.slots || bad_list(seqs, n) || bad_list(pos, n) || !aligned(cu_seqlens, 4) ||
      (!cu_seqlens && tokens < 0))
    return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (fa_status s = check_ws(v, n, workspace, workspace_bytes)) return s;
  return from_cuda(cache_extend(v, seqs, n, cu_seqlens, tokens, pos, workspace,
                                static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache_write(const fa_cache* cache, int layer, const void* K, const void* V,
                         const int* seqs, const int* pos, int n, const int* cu_seqlens,
                         int total, void* stream) {
  reset_launch_count();
  CacheView v;
  if (fa_status s = view_of(cache, v)) return s;
  if (layer < 0 || layer >= v.layers || n < 0 || total < 0 || bad_list(seqs, n) ||
      bad_list(pos, n) || !aligned(cu_seqlens, 4))
    return FA_ERR_INVALID_ARG;
  if (n == 0 || total == 0) return FA_OK;
  if (!cu_seqlens && total % n != 0) return FA_ERR_INVALID_ARG;
  if (!K || !V || !aligned(K, 16) || !aligned(V, 16)) return FA_ERR_INVALID_ARG;
  return from_cuda(cache_write(v, layer, K, V, seqs, pos, n, cu_seqlens, total,
                               static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache_fork(const fa_cache* cache, const int* src, const int* dst, int n,
                        void* workspace, size_t workspace_bytes, void* stream) {
  reset_launch_count();
  CacheView v;
  if (fa_status s = view_of(cache, v)) return s;
  if (n < 0 || n > v.slots || bad_list(src, n) || bad_list(dst, n)) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (fa_status s = check_ws(v, n, workspace, workspace_bytes)) return s;
  return from_cuda(cache_fork(v, src, dst, n, workspace, static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache_free(const fa_cache* cache, const int* seqs, int n, void* workspace,
                        size_t workspace_bytes, void* stream) {
  reset_launch_count();
  CacheView v;
  if (fa_status s = view_of(cache, v)) return s;
  if (n < 0 || n > v.slots || bad_list(seqs, n)) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (fa_status s = check_ws(v, n, workspace, workspace_bytes)) return s;
  return from_cuda(cache_free(v, seqs, n, workspace, static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache_copy(const fa_cache* cache, const int* src, const int* dst, int n,
                        void* workspace, size_t workspace_bytes, void* stream) {
  reset_launch_count();
  CacheView v;
  if (fa_status s = view_of(cache, v)) return s;
  if (n < 0 || n > v.pages || bad_list(src, n) || bad_list(dst, n)) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (fa_status s = check_ws(v, n, workspace, workspace_bytes)) return s;
  return from_cuda(cache_copy(v, src, dst, n, workspace, static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache_compact(const fa_cache* cache, void* workspace, size_t workspace_bytes,
                           void* stream) {
  reset_launch_count();
  CacheView v;
  if (fa_status s = view_of(cache, v)) return s;
  if (fa_status s = check_ws(v, 0, workspace, workspace_bytes)) return s;
  return from_cuda(cache_compact(v, workspace, static_cast<cudaStream_t>(stream)));
}

size_t fa_paged_workspace_size(const fa_cache* cache, int B, int T, int Hq, int shared) {
  CacheView v;
  if (view_of(cache, v) != FA_OK || check_fwd(v, B, T, Hq, shared) != FA_OK) return 0;
  if (B == 0 || T == 0) return kPartialAlign;           // launches nothing, and there is no plan
  PagedArgs a;
  sizes(a, v, B, T, Hq, shared);
  if (!plan(a, sm_count())) return 0;
  size_t at;
  return phase_bytes(a.own, v.d, &at) + phase_bytes(a.pre, v.d, &at) + kPartialAlign -
         kWorkspaceAlign;
}

fa_status fa_fwd_paged(const fa_cache* cache, int layer, const void* Q, void* O, float* LSE,
                       const int* seqs, int B, int T, int Hq, float scale, int causal,
                       int window_left, float softcap, void* workspace, size_t workspace_bytes,
                       void* stream) {
  return fwd(cache, layer, Q, O, LSE, seqs, B, T, Hq, 0, scale, causal, window_left, softcap,
             workspace, workspace_bytes, stream);
}

fa_status fa_fwd_shared(const fa_cache* cache, int layer, const void* Q, void* O, float* LSE,
                        const int* seqs, int B, int T, int Hq, int shared, float scale,
                        int causal, int window_left, float softcap, void* workspace,
                        size_t workspace_bytes, void* stream) {
  return fwd(cache, layer, Q, O, LSE, seqs, B, T, Hq, shared, scale, causal, window_left,
             softcap, workspace, workspace_bytes, stream);
}

}  // extern "C"
