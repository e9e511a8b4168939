// What the attention kernels over the paged cache share: the step's work, its split over the
// CTAs, the partial results that CTAs leave for one another.
//
// A work item is up to `rows` query rows (tokens of one request x the grouped heads of one kv
// head); its keys are a run of 128-key tiles.  All tiles of a call, ordered by (kv head,
// item, tile), are cut into equal runs, one per CTA: every CTA reads the same
// number of keys, whatever the requests' lengths.  A CTA's run is a sequence of pieces of
// items; an item cut between CTAs leaves one partial result per piece (running maximum, sum
// and unnormalised output in float32), joined by cache_join_kernel in the order of the CTAs.
#pragma once

#include <cuda.h>

#include "fork_cache.cuh"
#include "tc_ptx.cuh"

namespace fork {

namespace tc {
// A tile by TMA with an L2 policy (evict first: what is read once does not push out what is kept)
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_normal() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
      "{%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}
}  // namespace tc

constexpr int kMaxCtas = 256;  // CTAs of a call, at most (sizes the workspace)

struct CacheAttnParams {
  int32_t* meta;
  CacheLayout L;
  const int32_t* table;
  const uint16_t* q;
  uint16_t* o;
  int Hq, Hkv, G, d, P, P_shift, max_blocks, n_pages, tile, rows, window;
  float scale_log2;  // scale * log2(e)
  uint64_t wait_ns;
  int stall;     // FORK_TEST_STALL
  int4* desc;    // [2 * CTAs]: an item cut after CTA c: (joined?, head, first row, rows), (CTAs, -, -, -)
  float2* ml;    // [2 * CTAs][rows]: running maximum (log2 domain) and sum
  float4* part;  // [2 * CTAs][d / 4][rows]: unnormalised output, a row's neighbours beside it (a thread has a row)
};

// An item of a call: request b's new tokens r0 .. r0 + nt - 1, stream rows row .. row + nt - 1;
// some row sees keys in [lo, hi), tiles t0 .. t0 + kt - 1.
struct CacheItem {
  int b, row, r0, nt, len, tree, only, lo, hi, t0, kt;  // only: no other item reads the request's keys
};

__device__ __forceinline__ CacheItem cache_item(const CacheAttnParams& p, int i) {
  const int4* rec = reinterpret_cast<const int4*>(p.meta + p.L.item + 8 * static_cast<int64_t>(i));
  const int4 x = rec[0], y = rec[1];
  CacheItem it;
  it.b = x.x;
  it.row = x.y;
  it.r0 = x.z;
  it.nt = x.w;
  it.len = y.x;
  it.tree = y.y;
  it.only = y.z;
  it.hi = it.len + it.r0 + it.nt;  // a node's ancestors come before it
  const int first = it.len + (it.tree ? 0 : it.r0);  // no row's position is lower
  it.lo = p.window > 0 ? max(0, first - p.window + 1) : 0;
  it.t0 = it.lo / kKeyTile;
  it.kt = (it.hi - 1) / kKeyTile - it.t0 + 1;
  return it;
}

// A piece of an item: key tiles [t0, t0 + n) for one kv head.  slot < 0: the whole item (its
// rows are finished); else the partial result's place.
struct CachePiece {
  int ok, g, t0, n, slot;
  CacheItem it;
};

// Place of columns 4 c .. 4 c + 3 of a row of a partial result.
__device__ __forceinline__ int64_t cache_part(const CacheAttnParams& p, int slot, int row, int c) {
  return (static_cast<int64_t>(slot) * (p.d / 4) + c) * p.rows + row;
}

// What a query row sees: cache indices [lo, full), and new token j where bit j of mask is set.
struct CacheRow {
  int lo, full;
  uint64_t mask;
};

__device__ __forceinline__ CacheRow cache_row(const CacheAttnParams& p, const CacheItem& it, int tok) {
  CacheRow r;
  const int32_t* m = p.meta;
  if (tok >= it.nt) {  // padding: finite and never written
    r.lo = it.lo;
    r.full = it.hi;
    r.mask = 0;
    return r;
  }
  const int pos = m[p.L.tok_pos + it.row + tok];
  r.lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  if (it.tree) {
    r.full = it.len;
    r.mask = reinterpret_cast<const uint64_t*>(m + p.L.tok_mask)[it.row + tok];
    // a path's nodes lie in the order of their positions: a window keeps the last ones
    if (p.window > 0 && p.window < FORK_CACHE_MAX_TREE)
      while (__popcll(r.mask) > p.window) r.mask &= r.mask - 1;
  } else {
    r.full = pos + 1;
    r.mask = 0;
  }
  return r;
}

// The 32 keys from cache index y0 that a row sees, as bits.
__device__ __forceinline__ uint32_t cache_seen(const CacheRow& r, int len, int y0) {
  const int a = r.lo - y0, b = r.full - y0;  // bits [a, b)
  uint32_t w = b <= 0 ? 0u : (b >= 32 ? 0xffffffffu : (1u << b) - 1u);
  if (a > 0) w = a >= 32 ? 0u : w & ~((1u << a) - 1u);
  const int s = y0 - len;  // new token of bit 0
  if (s >= 0) {
    if (s < 64) w |= static_cast<uint32_t>(r.mask >> s);
  } else if (s > -32) {
    w |= static_cast<uint32_t>(r.mask << -s);
  }
  return w;
}

// Whether some row of the item does not see some key of tile t.
__device__ __forceinline__ bool cache_masked(const CacheAttnParams& p, const CacheItem& it, int t) {
  const int y0 = t * kKeyTile;
  const int all = it.tree ? it.len : it.len + it.r0 + 1;  // every row sees the keys before (but for a window)
  const int last = it.len + it.r0 + it.nt - 1;                   // no row's position is higher
  return all - y0 < kKeyTile || (p.window > 0 && y0 <= last - p.window);
}

constexpr int kMaxRun = 1 << 30;  // tiles of one CTA, at most (the kernels count them in 32 bits)

// x / y, mostly of small numbers (a 64-bit division takes some hundred cycles)
__device__ __forceinline__ int64_t quotient_of(int64_t x, int64_t y) {
  return (x | y) <= 0x7fffffff ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y)) : x / y;
}

// Where a CTA's run begins and ends: one warp counts the call's tiles, 32 items at a time (no
// barrier: only the producers need it).  No run (begin == end) for CTAs beyond the tiles.
// Runs differ by one tile at most: the first `more` CTAs have base + 1.  A call whose runs would be
// longer than kMaxRun does nothing but raise FORK_STATUS_CAPACITY.
struct CacheSplit {
  int head, item, off, n_item, base, more;
  int64_t begin, end;
};

// CTA whose run holds the call's tile x
__device__ __forceinline__ int cache_owner(const CacheSplit& s, int64_t x) {
  const int64_t wide = static_cast<int64_t>(s.more) * (s.base + 1);
  return static_cast<int>(x < wide ? quotient_of(x, s.base + 1) : s.more + quotient_of(x - wide, s.base));
}

__device__ __forceinline__ CacheSplit cache_split(const CacheAttnParams& p) {
  CacheSplit s;
  const int lane = threadIdx.x & 31;
  // the first items are read beside the header (their records exist whatever the step holds)
  const CacheItem first = cache_item(p, min(lane, p.L.max_item - 1));
  s.n_item = p.meta[C_NITEM];
  auto tiles = [&](int i) { return i < s.n_item ? cache_item(p, i).kt : 0; };
  const int v0 = lane < s.n_item ? first.kt : 0;
  int64_t per_head = v0;  // (131072 items of 8 tokens over 2.2 million cached ones: 2.8e9 tiles)
#pragma unroll 4
  for (int i = 32 + lane; i < s.n_item; i += 32) per_head += tiles(i);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) per_head += __shfl_xor_sync(0xffffffffu, per_head, k);
  const int64_t total = per_head * p.Hkv;
  const int ctas = static_cast<int>(total < gridDim.x ? total : gridDim.x);
  s.head = s.item = s.off = s.base = s.more = 0;
  s.begin = s.end = 0;
  const int c = blockIdx.x;
  if (c >= ctas) return s;
  const int64_t base_run = quotient_of(total, ctas);
  if (base_run >= kMaxRun) {
    if (lane == 0) atomicOr(p.meta + C_STATUS, FORK_STATUS_CAPACITY);
    return s;
  }
  s.base = static_cast<int>(base_run);
  s.more = static_cast<int>(total - static_cast<int64_t>(s.base) * ctas);
  s.begin = static_cast<int64_t>(s.base) * c + min(c, s.more);
  s.end = s.begin + s.base + (c < s.more ? 1 : 0);
  s.head = static_cast<int>(quotient_of(s.begin, per_head));
  int64_t left = s.begin - s.head * per_head;  // tiles of this head before the run
  for (int base = 0; base < s.n_item; base += 32) {
    const int v = base == 0 ? v0 : tiles(base + lane);
    int x = v;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, k);
      if (lane >= k) x += y;
    }
    const int all = __shfl_sync(0xffffffffu, x, 31);
    if (left < all) {
      const int at = __ffs(__ballot_sync(0xffffffffu, x > left)) - 1;
      s.item = base + at;
      s.off = static_cast<int>(left) - __shfl_sync(0xffffffffu, x - v, at);
      break;
    }
    left -= all;
  }
  return s;
}

// The pieces of a CTA's run in order (one thread or warp walks them).
struct CacheWalk {
  int g, i, off, n_item;
  int64_t at, end;
  __device__ __forceinline__ explicit CacheWalk(const CacheSplit& s)
      : g(s.head), i(s.item), off(s.off), n_item(s.n_item), at(s.begin), end(s.end) {}
  __device__ __forceinline__ CachePiece next(const CacheAttnParams& p) {
    CachePiece c;
    c.ok = at < end;
    if (!c.ok) return c;
    c.it = cache_item(p, i);
    c.g = g;
    c.t0 = c.it.t0 + off;
    const int64_t left = end - at;
    c.n = static_cast<int>(left < c.it.kt - off ? left : c.it.kt - off);
    const bool whole = off == 0 && c.n == c.it.kt;
    c.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (off == 0 ? 1 : 0);
    at += c.n;
    off = 0;
    if (++i == n_item) {
      i = 0;
      ++g;
    }
    return c;
  }
};

// What CTA c leaves for cache_join_kernel: the item that its run begins and does not finish.
// `at_end`: the call's tile behind the item's last one.
__device__ __forceinline__ void cache_describe(const CacheAttnParams& p, const CacheSplit& s, const CachePiece& c,
                                               int64_t at_end) {
  const bool cut = c.ok && c.slot >= 0 && (c.slot & 1);
  p.desc[2 * blockIdx.x] = make_int4(cut ? 1 : 0, c.g, c.it.row, c.it.nt);
  if (cut)
    p.desc[2 * blockIdx.x + 1] =
        make_int4(cache_owner(s, at_end - 1) - static_cast<int>(blockIdx.x) + 1, 0, 0, 0);
}


// maps: queries [T_cap][Hq][d], keys and values of the layer [n_pages * Hkv][page_tokens][d]
template <int D>
int launch_cache_attn_tc(const CacheAttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                         int ctas, cudaStream_t s);

}  // namespace fork
