// Shared definitions of the paged-cache step: layout of its metadata buffer.
#pragma once

#include <atomic>

#include "fork_common.cuh"

namespace fork {

constexpr int32_t kCacheMagic = 0x46434348;  // 'FCCH'
constexpr int kKeyTile = 128;                // keys of one attention tile

// Header words of a step's metadata buffer.
enum CacheHdr : int {
  C_MAGIC = 0, C_STATUS,
  C_HEAD = 8, C_NFREE, C_TAKEN, C_GIVEN,        // ring before the step, pages taken and returned
  C_VALID = 4, C_TREE = 5, C_NITEM = 6, C_T = 7,  // read together (one 16-byte load)
  C_WORDS = 32
};

// Query rows (token x grouped head) of one attention work item: chosen from the most rows a
// request can have in a step, because the launch may not read the device.  16 rows, and 32 of
// heads of 64, go to the kernel on warp-level products, more to the tcgen05 one (128, or 256 in
// two tiles).  Measured, warp-level / tcgen05: 64 requests x 1 token x 4 heads of 128 (0.95 GB)
// 147 / 160 us; with 32-row items, 32 requests x 8 tokens x 4 heads of 128 116 / 94 us (when both were
// timed), but of 64 (64 requests) 107 / 129 us, and 32 requests of 2 to 8 tokens x 3 heads of 64
// 22.5 / 29 us.
__host__ __device__ inline int cache_item_rows(int max_new, int G, int d) {
  const int64_t most = static_cast<int64_t>(max_new) * G;
  return most <= 16 ? 16 : (most <= 32 && d == 64 ? 32 : (most <= 128 / G * G ? 128 : 256));
}
// 256 rows are two tensor-core tiles, whole tokens in each
__host__ __device__ inline int cache_item_tokens(int max_new, int G, int d) {
  const int rows = cache_item_rows(max_new, G, d);
  return rows == 256 ? 2 * (128 / G) : rows / G;
}

inline int page_shift(int page_tokens) {
  int s = 0;
  while ((1 << s) < page_tokens) ++s;
  return s;
}

// A work item's record, 8 words, is everything the attention kernels need of it, in two loads:
// request, first stream row, first new token, tokens | cached tokens, tree?, the request's only item?

struct CacheLayout {
  int32_t T_cap, max_req, max_item;
  int64_t row_start, len0, kv_len, have, page_off, given_off, item_off;  // per request
  int64_t tok_req, tok_pos, tok_slot, tok_mask;                          // per row
  int64_t item;  // attention work items, 8 words each (above)
  int64_t total;
};

__host__ __device__ inline CacheLayout cache_layout(int32_t T_cap, int32_t max_req, int32_t max_new, int32_t G, int32_t d) {
  CacheLayout L;
  L.T_cap = T_cap;
  L.max_req = max_req;
  const int tile = cache_item_tokens(max_new, G, d);
  const int64_t most = static_cast<int64_t>(T_cap) / tile + max_req;
  L.max_item = static_cast<int32_t>(most < T_cap ? most : T_cap);
  int64_t o = C_WORDS;
  auto take = [&](int64_t n) { int64_t r = o; o = align_words(o + n); return r; };
  L.row_start = take(static_cast<int64_t>(max_req) + 1);
  L.len0 = take(max_req);
  L.kv_len = take(max_req);
  L.have = take(max_req);
  L.page_off = take(static_cast<int64_t>(max_req) + 1);
  L.given_off = take(static_cast<int64_t>(max_req) + 1);
  L.item_off = take(static_cast<int64_t>(max_req) + 1);
  L.tok_req = take(T_cap);
  L.tok_pos = take(T_cap);
  L.tok_slot = take(T_cap);
  L.tok_mask = take(2 * static_cast<int64_t>(T_cap));
  L.item = take(8 * static_cast<int64_t>(L.max_item));
  L.total = o;
  return L;
}

// Programmatic dependent launch: a kernel launched with it may start before the one ahead of
// it in the stream has ended.  Every thread calls pdl_wait before it touches memory (it
// returns when that kernel has ended and its writes are visible), so also before it exits;
// pdl_launch lets the next kernel of the stream take its place early.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<A&&>(args)...);
}

// Let a kernel use `bytes` of dynamic shared memory on the current device: once per device.
template <auto Kern>
int allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cuda_rc(cudaGetDevice(&dev)) != FORK_OK) return FORK_ECUDA;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev) & 1) return FORK_OK;
  if (cuda_rc(cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes))) != FORK_OK)
    return FORK_ECUDA;
  if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return FORK_OK;
}

// Host: validate a caller's handle; returns FORK_OK and the layout.
int check_cache(const fork_cache* c, CacheLayout* out);

}  // namespace fork
