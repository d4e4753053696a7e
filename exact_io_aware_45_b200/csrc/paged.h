// Internal interface of the paged key/value cache: the device's view of a
// cache, and the work division of the attention kernels that read it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa.h"
#include "internal.h"

namespace fa {

// A cache as the kernels see it; strides in bytes.
struct CacheView {
  char* K;
  char* V;
  long long layer_stride, page_stride;
  int layers, pages, width, slots;
  int page_log2;       // page_size = 1 << page_log2
  int head_bytes;      // page_size * d * element size: one head's rows of one page
  int page_bytes;      // Hkv * head_bytes
  int row_bytes;       // d * element size
  int Hkv, d;
  int* table;
  int* lens;
  int* refs;
  unsigned* err;
};

// SMs of the current device, asked for once per device.
int sm_count();

cudaError_t cache_extend(const CacheView& c, const int* seqs, int n, const int* cu, int tokens,
                         int* pos, void* ws, cudaStream_t st);
cudaError_t cache_write(const CacheView& c, int layer, const void* K, const void* V,
                        const int* seqs, const int* pos, int n, const int* cu, int total,
                        cudaStream_t st);
cudaError_t cache_fork(const CacheView& c, const int* src, const int* dst, int n, void* ws,
                       cudaStream_t st);
cudaError_t cache_free(const CacheView& c, const int* seqs, int n, void* ws, cudaStream_t st);
cudaError_t cache_copy(const CacheView& c, const int* src, const int* dst, int n, void* ws,
                       cudaStream_t st);
cudaError_t cache_compact(const CacheView& c, void* ws, cudaStream_t st);
size_t cache_workspace_bytes(int pages, int slots, int n);

// The partial results begin on such a boundary: the widest store of them (32 bytes, paged_tc.cu)
// needs it. A workspace need not, so its size has room for the step up from kWorkspaceAlign.
constexpr int kPartialAlign = 32, kWorkspaceAlign = 16;

// One phase of an attention call: `items` row tiles (of up to `rows` packed
// query rows that share a KV head), each over its own key tiles, cut
// into even ranges for `n` streams (paged_sched.cuh).
struct Phase {
  int rows = 0;        // query rows per item, at most
  int tile_log2 = 0;   // keys per tile = 1 << tile_log2
  int rt = 0;          // row tiles per (sequence, KV head); per KV head in the shared phase
  int n = 0;           // streams
  int items = 0;
  bool blocked = false;  // partial O lies as [128-row block][d / 8][row][8]
  int over = 4;        // units of an item beside its tiles
  int snap = 2;        // tiles that a cut keeps from an item's ends
  int least = 4;       // units that a stream is worth
  int yield = 0;       // shared phase: units of the own phase that take an SM as long as one
                       // of its own, where the own phase runs beside it
  int sms = 0;         // SMs of the device
  float* o = nullptr;  // partial results: [items + n][rows][d], normalised
  float* lse = nullptr;  // [items + n][rows], base 2
};

struct PagedArgs {
  CacheView c;
  const char* K;       // the layer's pages
  const char* V;
  const void* Q;
  void* O;
  float* LSE;
  const int* seqs;
  int B, T, Hq, G;
  int TG;              // T * G: packed query rows of one sequence and KV head
  int shared;          // tokens of the shared prefix
  int causal, wl;
  float scale, softcap;
  Phase own, pre;
};

// Launches a kernel of a call's chain (shared phase, own phase, join). With `after`
// it may start before the kernel ahead of it in the stream has finished, once that
// has let it (chain_next); it then has to wait (chain_wait) before it reads that
// kernel's results, or, if it reads none, let one block wait before it ends (chain_end): the end
// of the chain's last kernel implies the end of all, and the other blocks make room.
template <class... P, class... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                           cudaStream_t st, bool after, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e == cudaSuccess) count_launch();
  return e;
}
#ifdef __CUDACC__
// Brings the arguments of a kernel into its SM's constant cache: their lines (64 bytes) are
// asked for at once, by a warp each, instead of one after the other as the code first needs
// them. 64 sequences behind a prefix of 4,096 take 26.7 us instead of 27.2, one short one 10.4
// instead of 10.6.
__device__ __forceinline__ void warm_args(const PagedArgs& a) {
  for (int i = (int)(threadIdx.x >> 5) * 16; i < (int)sizeof(PagedArgs) / 4;
       i += (int)(blockDim.x >> 5) * 16)
    asm volatile("" ::"r"(reinterpret_cast<const int*>(&a)[i]) : "memory");
}
__device__ __forceinline__ void chain_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void chain_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void chain_end() {
  if (blockIdx.x == 0) chain_wait();
}
#endif

// Kernel families. Each runs one phase (`pre`: the shared prefix).
cudaError_t paged_simt(const PagedArgs& a, bool pre, int dtype, cudaStream_t st);
constexpr int kSimtRows = 4, kSimtTileLog2 = 5;
constexpr int simt_blocks_per_sm(int d, int rows) { return d * rows >= 512 ? 3 : 4; }  // registers
// The same for many packed rows, tiled in registers; a stream is a block.
cudaError_t paged_fma(const PagedArgs& a, bool pre, int dtype, cudaStream_t st);
constexpr int kFmaRows = 64;
constexpr int fma_blocks_per_sm(int d) { return d == 128 ? 2 : d == 64 ? 3 : 4; }   // shared memory
// mma.sync kernel for few packed rows (bf16, d in {64, 128}); a stream is a warp.
cudaError_t paged_mma(const PagedArgs& a, bool pre, cudaStream_t st);
constexpr int kMmaWarps = 4, kMmaBlocksPerSm = 2;
constexpr int mma_tile_log2(int d) { return d == 128 ? 4 : 5; }
// tcgen05 kernel for many packed rows (bf16, d in {64, 128}); a stream is a CTA.
// Items of 128 rows (one query tile, its key tiles dealt to two warpgroups) or 256.
cudaError_t paged_tc(const PagedArgs& a, bool pre, cudaStream_t st);
constexpr int kTcTileLog2 = 7, kTcRows = 128;
// Joins the partial results of both phases.
cudaError_t paged_join(const PagedArgs& a, int dtype, cudaStream_t st);

}  // namespace fa
