// Test infrastructure: the split of a paged-cache attention call over its CTAs, by itself.
#include "../tree_forked_hybrid_gb300/csrc/fork_cache_attn.cuh"

__global__ void probe_kernel(const __grid_constant__ fork::CacheAttnParams p, int64_t* out) {
  const fork::CacheSplit s = fork::cache_split(p);
  if (threadIdx.x != 0) return;
  int64_t* o = out + 6 * blockIdx.x;
  o[0] = s.begin;
  o[1] = s.end;
  o[2] = s.head;
  o[3] = s.item;
  o[4] = s.off;
  o[5] = s.end > s.begin ? fork::cache_owner(s, s.end - 1) : -1;
}

// meta: a step's metadata with its item records; out: 6 words for each of `ctas` CTAs
extern "C" int probe_split(int32_t* meta, int T_cap, int max_req, int max_new, int Hq, int Hkv, int d, int ctas,
                           int64_t* out) {
  fork::CacheAttnParams p = {};
  p.meta = meta;
  p.L = fork::cache_layout(T_cap, max_req, max_new, Hq / Hkv, d);
  p.Hkv = Hkv;
  probe_kernel<<<ctas, 32>>>(p, out);
  return cudaDeviceSynchronize();
}

extern "C" int64_t probe_item_offset(int T_cap, int max_req, int max_new, int Hq, int Hkv, int d) {
  return fork::cache_layout(T_cap, max_req, max_new, Hq / Hkv, d).item;
}
