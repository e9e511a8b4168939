// Attention over the paged cache for steps of few query rows per kv head (a decoded token, a
// small tree), the join of rows shared by several CTAs, and the entry point.
//
// o = sum_y softmax_y(<q, k_y> scale) v_y in one pass over the keys with the running maximum
// and sum of the exponentials (log2 domain).  With up to 32 rows a key is used too little for
// the products to matter: the kernel has to keep HBM busy.  One CTA per SM; a producer warp
// keeps four 32-KB tiles in flight by TMA (page by page, the page numbers read ahead), and
// eight warps take 16 rows x 16 of a tile's 128 keys each (of 32 rows: 16 x 32 keys), with a
// running maximum, sum and output of their own: no warp waits for another until the piece
// ends, when they are joined in shared memory.  One more warp fetches the next piece's queries
// and what its rows see while this one is worked on (in the consumers' own time that was 2000
// to 2500 of the 24000 cycles of a small call).  The maximum of a row only moves when a score
// exceeds it by 2^8: the usual tile needs one vote instead of shuffles and a rescaling.  Products
// on mma.sync m16n8k16: 16 or 32 query rows would fill an eighth or a quarter of a 128-row tcgen05
// tile, and registers take the exponentials without a trip through tensor memory.
// 64 requests x 1 token x 4 heads of 128 over 1,000 to 6,000 keys (0.95 GB): 145 us, 0.98 of the
// measured HBM rate.  Of 64 (half the bytes of a tile for the same latencies; 64 requests x 8 x 4,
// 0.48 GB): 107 us.  A call of one request and a few short tiles: 9.6 us, the latency of the
// tables, the queries and the first tile.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fork_attn.cuh"
#include "fork_cache_attn.cuh"

namespace fork {

namespace {

constexpr int kWarps = 8;                     // consumer warps
constexpr int kThreads = (kWarps + 2) * 32;   // and the producers of keys and values, and of queries
constexpr int kRingBytes = 128 * 1024;        // K and V tiles in flight
constexpr float kRescale = 8.f;               // a row's maximum moves when a score exceeds it by 2^8
constexpr int kPieces = 4;                    // pieces handed from the producer to the consumers

template <int D, int MT>
struct SmallLayout {
  static constexpr int NB = D / 64;             // 64-element boxes of a row
  static constexpr int BOX = kKeyTile * 128;    // bytes of one box of a tile
  static constexpr int SLOT = NB * BOX;
  static constexpr int NS = kRingBytes / SLOT;  // slots; K and V tiles alternate
  static constexpr int ROWS = 16 * MT;
  static constexpr int KW = kWarps / MT;        // warps side by side on 16 rows: 16 * MT keys each
  static constexpr int QBYTES = ROWS * D * 2;
  static constexpr int STAGE_LD = D + 4;        // floats of a staged row (off the banks of the next)
  static constexpr int Q = NS * SLOT;           // two query tiles, by the piece's parity
  static constexpr int STAGE = Q + 2 * QBYTES;  // the warps' outputs at the end of a piece
  static constexpr int ML = STAGE + kWarps * 16 * STAGE_LD * 4;  // [2][warps][16] (m, l)
  static constexpr int SEE = ML + 2 * kWarps * 16 * 8;  // [2][ROWS] what the rows see
  static constexpr int BAR = SEE + 2 * ROWS * 16;
  static constexpr int BYTES = BAR + 1024;
  static constexpr int SMEM = BYTES + 1024;
};

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// a bf16 pair with an infinity or NaN in it
__device__ __forceinline__ bool odd_pair(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// byte offset of element `col` of row `row` in a 128-byte-swizzled tile of `rows`-row boxes
__device__ __forceinline__ uint32_t swz(int rows, int row, int col) {
  return static_cast<uint32_t>((col >> 6) * rows * 128 + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4));
}

template <int D, int MT>
__global__ void __launch_bounds__(kThreads, 1)
    cache_small_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ CacheAttnParams p) {
  using LY = SmallLayout<D, MT>;
  constexpr int NS = LY::NS, ROWS = LY::ROWS, KW = LY::KW;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + LY::BAR);  // [NS] tile landed
  uint64_t* empty = full + NS;                                   // [NS] read by the eight warps
  uint64_t* pfull = empty + NS;                                  // [kPieces]
  uint64_t* pempty = pfull + kPieces;                            // [kPieces]
  uint64_t* meet = pempty + kPieces;                             // the consumers' own
  uint64_t* never = meet + 1;                                    // FORK_TEST_STALL: completed by nothing
  uint64_t* qfull = never + 1;                                   // [2] the piece's queries are there
  volatile int* abort = reinterpret_cast<volatile int*>(qfull + 2);
  CachePiece* pieces = reinterpret_cast<CachePiece*>(qfull + 3);
  static_assert(sizeof(CacheRow) == 16, "a row's entry");
  static_assert((2 * NS + 2 * kPieces + 5) * 8 + kPieces * sizeof(CachePiece) <= 1024, "barriers");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], kWarps);
    }
    for (int i = 0; i < kPieces; ++i) {
      tc::mbar_init(&pfull[i], 1);
      tc::mbar_init(&pempty[i], kWarps + 1);  // the consumers have begun it, the queries' warp has read it
    }
    tc::mbar_init(meet, kWarps);
    tc::mbar_init(never, 1);
    tc::mbar_init(&qfull[0], 1);
    tc::mbar_init(&qfull[1], 1);
    *abort = 0;
    tc::fence_mbar_init();
  }
  if (tid == kWarps * 32) {
    tc::prefetch_tmap(&kmap);
    tc::prefetch_tmap(&vmap);
  }
  pdl_launch();
  pdl_wait();
  __syncthreads();
  if (p.meta[C_VALID] == 0) return;

  if (warp == kWarps) {
    // ===================== producer =====================
    const CacheSplit split = cache_split(p);
    if (lane == 0) p.desc[2 * blockIdx.x].x = 0;
    const uint64_t first = tc::policy_evict_first(), normal = tc::policy_normal();
    CacheWalk walk(split);
    int f = 0;  // tiles issued, K and V counted apart
    bool ok = !p.stall || __all_sync(0xffffffffu, tc::mbar_wait(never, 0, abort, p.wait_ns));
    for (int n = 0; ok; ++n) {
      const CachePiece c = walk.next(p);
      const int ps = n % kPieces;
      if (n >= kPieces && !(ok = __all_sync(0xffffffffu, tc::mbar_wait(&pempty[ps], ((n / kPieces) - 1) & 1, abort, p.wait_ns))))
        break;
      if (lane == 0) {
        pieces[ps] = c;
        tc::mbar_arrive(&pfull[ps]);
      }
      if (!c.ok) break;
      // pages of the tiles, 32 blocks read ahead of use; blocks without a visible key and
      // bad pages come as zeros (a box outside the tensor)
      const int32_t* row = p.table + static_cast<int64_t>(c.it.b) * p.max_blocks;
      const int b_lo = c.it.lo >> p.P_shift, b_hi = (c.it.hi - 1) >> p.P_shift;
      const int b0 = (c.t0 * kKeyTile) >> p.P_shift;  // first block
      const int per = max(kKeyTile >> p.P_shift, 1);  // blocks of a tile
      const int box = min(p.P, kKeyTile);
      auto fetch = [&](int blk) {
        if (blk < b_lo || blk > b_hi) return -1;
        const int page = row[blk];
        if (page < 0 || page >= p.n_pages) {
          atomicOr(p.meta + C_STATUS, FORK_STATUS_BAD_PAGE);
          return -1;
        }
        return page;
      };
      int base = b0, cur = fetch(base + lane), nxt = fetch(base + 32 + lane);
      for (int t = 0; ok && t < c.n; ++t) {
        const int blk = ((c.t0 + t) * kKeyTile) >> p.P_shift;
        if (blk - base >= 32) {
          base += 32;
          cur = nxt;
          nxt = fetch(base + 32 + lane);
        }
        int page = __shfl_sync(0xffffffffu, cur, (blk - base + min(lane, per - 1)) & 31);
        const int in_page = ((c.t0 + t) * kKeyTile) & (p.P - 1);  // P = 256: a tile is half a page
        const int64_t z = page < 0 ? static_cast<int64_t>(p.n_pages) * p.Hkv : static_cast<int64_t>(page) * p.Hkv + c.g;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++f) {
          const int s = f % NS;
          if (f >= NS && !(ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[s], ((f / NS) - 1) & 1, abort, p.wait_ns)))) break;
          if (lane == 0) tc::mbar_expect_tx(&full[s], LY::SLOT);
          __syncwarp();
          if (lane < per) {
            unsigned char* dst = smem + s * LY::SLOT + lane * box * 128;
#pragma unroll
            for (int b = 0; b < LY::NB; ++b)
              tc::tma_load_3d(dst + b * LY::BOX, kv ? &vmap : &kmap, &full[s], b * 64, in_page, static_cast<int>(z), c.it.only ? first : normal);
          }
        }
      }
      if (lane == 0) cache_describe(p, split, c, walk.at - c.n + c.it.kt);
    }
    // the last copies into each slot complete by themselves
    if (lane == 0)
      for (int i = max(0, f - NS); i < f; ++i) tc::mbar_drain(&full[i % NS], (i / NS) & 1);
    __syncwarp();
  } else if (warp == kWarps + 1) {
    // ===================== queries =====================
    auto wait = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, tc::mbar_wait(bar, par, abort, p.wait_ns));
    };
    for (int n = 0;; ++n) {
      const int ps = n % kPieces;
      if (!wait(&pfull[ps], (n / kPieces) & 1)) break;
      const CachePiece c = pieces[ps];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&pempty[ps]);
      if (!c.ok) break;
      // this piece's place is free once every consumer has begun the piece before
      if (n >= 2 && !wait(&pempty[(n - 1) % kPieces], ((n - 1) / kPieces) & 1)) break;
      const CacheItem& it = c.it;
      // the query rows, token by token (rows past the item are zero), and what they see: every
      // load on its way before the first is used
      unsigned char* qt = smem + LY::Q + (n & 1) * LY::QBYTES;
      constexpr int kPer = ROWS * (D / 8) / 32;
      uint4 x[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int e = lane + 32 * k, r = e / (D / 8), v = e % (D / 8), tok = r / p.G;
        x[k] = make_uint4(0, 0, 0, 0);
        if (tok < it.nt)
          x[k] = *reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(it.row + tok) * p.Hq + c.g * p.G + r % p.G) * D + v * 8);
      }
      CacheRow* see = reinterpret_cast<CacheRow*>(smem + LY::SEE) + (n & 1) * ROWS;
      if (lane < ROWS) see[lane] = cache_row(p, it, lane / p.G);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int e = lane + 32 * k;
        *reinterpret_cast<uint4*>(qt + swz(ROWS, e / (D / 8), (e % (D / 8)) * 8)) = x[k];
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&qfull[n & 1]);
    }
  } else {
    // ===================== consumers =====================
    const uint32_t ring = tc::smem_u32(smem);
    const uint32_t qs0 = tc::smem_u32(smem + LY::Q);
    float* stage = reinterpret_cast<float*>(smem + LY::STAGE);
    float2* ml = reinterpret_cast<float2*>(smem + LY::ML);
    const int quad = lane >> 2, ql = lane & 3;  // fragment row, column pair
    const int mt = warp / KW, key0 = warp % KW * 16 * MT;  // this warp's rows and keys of a tile
    int f = 0, met = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, tc::mbar_wait(bar, par, abort, p.wait_ns));
    };
    auto meet_all = [&]() {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(meet);
      const bool r = wait(meet, met & 1);
      ++met;
      return r;
    };
    for (int n = 0; ok; ++n) {
      const int ps = n % kPieces;
      if (!(ok = wait(&pfull[ps], (n / kPieces) & 1))) break;
      const CachePiece c = pieces[ps];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&pempty[ps]);
      if (!c.ok) break;
      const CacheItem& it = c.it;
      const uint32_t qs = qs0 + (n & 1) * LY::QBYTES;
      if (!(ok = wait(&qfull[n & 1], (n >> 1) & 1))) break;
      const CacheRow* see = reinterpret_cast<const CacheRow*>(smem + LY::SEE) + (n & 1) * ROWS + mt * 16;
      const CacheRow rows[2] = {see[quad], see[8 + quad]};
      float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, acc[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
      for (int t = 0; t < c.n; ++t) {
        // ---- scores of this warp's keys
        const int sk = f % NS;
        if (!(ok = wait(&full[sk], (f / NS) & 1))) break;
        ++f;
        float s[MT][2][4];
#pragma unroll
        for (int g = 0; g < MT; ++g)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[g][j][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t qf[4];
          ldsm4(qf, qs + swz(ROWS, mt * 16 + (lane & 15), ks * 16 + (lane >> 4) * 8));
#pragma unroll
          for (int g = 0; g < MT; ++g) {
            uint32_t kf[4];  // keys 0-7: k 0-7, k 8-15; keys 8-15: k 0-7, k 8-15
            ldsm4(kf, ring + sk * LY::SLOT +
                          swz(kKeyTile, key0 + g * 16 + (lane & 7) + ((lane >> 4) << 3), ks * 16 + ((lane >> 3) & 1) * 8));
            mma_16816(s[g][0], qf, kf[0], kf[1]);
            mma_16816(s[g][1], qf, kf[2], kf[3]);
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty[sk]);
        // ---- mask, running maximum, exponentials
        const int tile = c.t0 + t, y0 = tile * kKeyTile + key0;
        const bool masked = cache_masked(p, it, tile);
        float v[2][MT][4], top[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int g = 0; g < MT; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[h][g][e] = s[g][e >> 1][2 * h + (e & 1)];
          if (masked) {
            const uint32_t seen = cache_seen(rows[h], it.len, y0) >> (ql * 2);
#pragma unroll
            for (int g = 0; g < MT; ++g)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!((seen >> (16 * g + 8 * (e >> 1) + (e & 1))) & 1u)) v[h][g][e] = -INFINITY;
          }
          top[h] = fmaxf(fmaxf(v[h][0][0], v[h][0][1]), fmaxf(v[h][0][2], v[h][0][3]));
#pragma unroll
          for (int g = 1; g < MT; ++g)
            top[h] = fmaxf(top[h], fmaxf(fmaxf(v[h][g][0], v[h][g][1]), fmaxf(v[h][g][2], v[h][g][3])));
          top[h] *= p.scale_log2;
        }
        if (__any_sync(0xffffffffu, top[0] > mx[0] + kRescale || top[1] > mx[1] + kRescale)) {
          // (also a row's first visible keys: its maximum was minus infinity)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
            const float m_new = top[h] > mx[h] + kRescale ? top[h] : mx[h];
            const float fac = m_new == mx[h] ? 1.f : ex2(mx[h] - m_new);
            mx[h] = m_new;
            sum[h] *= fac;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              acc[i][2 * h] *= fac;
              acc[i][2 * h + 1] *= fac;
            }
          }
        }
        uint32_t pf[MT][4], pr[MT][4];  // two bf16 numbers per weight
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // A weight goes into the product as two bf16 numbers, to 2^-15 of it: the largest below it
          // and the rest, both positive (times an infinite value they do not make a NaN);
          // the sum takes it in float32.  The second product is hidden by the wait for HBM where there
          // is one: 64 requests x 1 token x 4 heads of 128 143.3 us (rounded to one bf16 number
          // 142.5), of 64 86.1 (85.0), small trees of 27 rows over a window 22.5 (21.6), 64 requests x
          // 32 rows of heads of 64 106.5 (97.3).  The relative error against 64 bits is 0.0017, the
          // rounding of the result (0.0020)
          const float at = mx[h] == -INFINITY ? 0.f : mx[h];
#pragma unroll
          for (int g = 0; g < MT; ++g) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = ex2(fmaf(v[h][g][e], p.scale_log2, -at));
            sum[h] += (x[0] + x[1]) + (x[2] + x[3]);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              // (times 1 - 2^-24: the next float32 down)
              const uint32_t w = __byte_perm(__float_as_uint(x[e] * 0.99999994f), __float_as_uint(x[e + 1] * 0.99999994f), 0x7632);
              pf[g][h + e] = w;
              pr[g][h + e] = pack_bf16(x[e] - lo_f(w), x[e + 1] - hi_f(w));
            }
          }
        }
        // ---- values
        const int sv = f % NS;
        if (!(ok = wait(&full[sv], (f / NS) & 1))) break;
        ++f;
        const unsigned char* vs = smem + sv * LY::SLOT;
        uint32_t keep[MT][2];  // of a fragment's two keys, those that some row of the item sees
        if (masked) {
          bool odd = false;
          // A masked key has p = 0, but 0 * NaN is NaN: values of keys that no row of the item
          // sees are taken as zero; an infinity or NaN among the others is left out of the
          // product and added to the rows that see it.
          for (int e = lane; e < 16 * MT * (D / 8); e += 32) {
            const int r = e / (D / 8), y = y0 + r;
            const uint4 x = *reinterpret_cast<const uint4*>(vs + swz(kKeyTile, key0 + r, (e % (D / 8)) * 8));
            if (y >= it.lo && y < it.hi) odd = odd || odd_pair(x.x) || odd_pair(x.y) || odd_pair(x.z) || odd_pair(x.w);
          }
          odd = __any_sync(0xffffffffu, odd);
#pragma unroll
          for (int g = 0; g < MT; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int y = y0 + g * 16 + h * 8 + ql * 2;
              keep[g][h] = (y >= it.lo && y < it.hi ? 0xffffu : 0u) | (y + 1 >= it.lo && y + 1 < it.hi ? 0xffff0000u : 0u);
            }
          if (odd) {
            for (int r = 0; r < 16 * MT; ++r)
#pragma unroll
              for (int i = 0; i < D / 8; ++i) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(vs + swz(kKeyTile, key0 + r, i * 8) + ql * 4);
                if (!odd_pair(w)) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if ((cache_seen(rows[h], it.len, y0) >> r) & 1u) {
                    if ((w & 0x7f80u) == 0x7f80u) acc[i][2 * h] += lo_f(w);
                    if ((w & 0x7f800000u) == 0x7f800000u) acc[i][2 * h + 1] += hi_f(w);
                  }
              }
          }
        }
        // (two loops: the masked one would cost the other its instructions)
        auto products = [&](auto fix) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
#pragma unroll
            for (int g = 0; g < MT; ++g) {
              uint32_t vf[4];  // columns 16i..: keys 0-7, 8-15; columns 16i + 8..: keys 0-7, 8-15
              ldsm4_t(vf, ring + sv * LY::SLOT + swz(kKeyTile, key0 + g * 16 + (lane & 15), i * 16 + (lane >> 4) * 8));
              if constexpr (decltype(fix)::value) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  vf[e] &= keep[g][e & 1];
                  if ((vf[e] & 0x7f80u) == 0x7f80u) vf[e] &= 0xffff0000u;
                  if ((vf[e] & 0x7f800000u) == 0x7f800000u) vf[e] &= 0xffffu;
                }
              }
              mma_16816(acc[2 * i], pf[g], vf[0], vf[1]);
              mma_16816(acc[2 * i + 1], pf[g], vf[2], vf[3]);
              mma_16816(acc[2 * i], pr[g], vf[0], vf[1]);
              mma_16816(acc[2 * i + 1], pr[g], vf[2], vf[3]);
            }
          }
        };
        if (masked) products(std::true_type{});
        else products(std::false_type{});
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty[sv]);
      }
      if (!ok) break;
      // ---- join the warps: their outputs side by side, weighted by 2^(own maximum - common
      // maximum) as they are summed
      // (every warp has begun this piece, so none still reads the last one's)
      if (!(ok = wait(&pempty[ps], (n / kPieces) & 1))) break;
      float2* ml_n = ml + (n & 1) * kWarps * 16;
      float* st = stage + warp * 16 * LY::STAGE_LD;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = sum[h];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (ql == 0) ml_n[warp * 16 + h * 8 + quad] = make_float2(mx[h], l);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(st + (h * 8 + quad) * LY::STAGE_LD + i * 8 + ql * 2) =
              make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
      }
      if (!(ok = meet_all())) break;
      for (int e = tid; e < ROWS * (D / 8); e += kWarps * 32) {
        const int row = e / (D / 8), v = (e % (D / 8)) * 8, tok = row / p.G;
        if (tok >= it.nt) continue;
        const int w0 = row / 16 * KW, r = row % 16;  // the row's warps
        float2 a[KW];
        float top = -INFINITY, l = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          a[w] = ml_n[(w0 + w) * 16 + r];
          top = fmaxf(top, a[w].x);
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          // (a warp without a visible key has a zero output and sum)
          const float f1 = a[w].x == -INFINITY ? 0.f : ex2(a[w].x - top);
          l = fmaf(a[w].y, f1, l);
          const float4* sp = reinterpret_cast<const float4*>(stage + ((w0 + w) * 16 + r) * LY::STAGE_LD + v);
          const float4 a0 = sp[0], a1 = sp[1];
          x[0] = fmaf(a0.x, f1, x[0]); x[1] = fmaf(a0.y, f1, x[1]); x[2] = fmaf(a0.z, f1, x[2]); x[3] = fmaf(a0.w, f1, x[3]);
          x[4] = fmaf(a1.x, f1, x[4]); x[5] = fmaf(a1.y, f1, x[5]); x[6] = fmaf(a1.z, f1, x[6]); x[7] = fmaf(a1.w, f1, x[7]);
        }
        if (c.slot < 0) {
          const float inv = 1.f / l;
          uint4 y;
          y.x = pack_bf16(x[0] * inv, x[1] * inv);
          y.y = pack_bf16(x[2] * inv, x[3] * inv);
          y.z = pack_bf16(x[4] * inv, x[5] * inv);
          y.w = pack_bf16(x[6] * inv, x[7] * inv);
          *reinterpret_cast<uint4*>(p.o + (static_cast<int64_t>(it.row + tok) * p.Hq + c.g * p.G + row % p.G) * D + v) = y;
        } else {
          p.part[cache_part(p, c.slot, row, v / 4)] = make_float4(x[0], x[1], x[2], x[3]);
          p.part[cache_part(p, c.slot, row, v / 4 + 1)] = make_float4(x[4], x[5], x[6], x[7]);
          if (v == 0) p.ml[static_cast<int64_t>(c.slot) * p.rows + row] = make_float2(top, l);
        }
      }
    }
  }
  if (*abort && lane == 0) atomicOr(p.meta + C_STATUS, FORK_STATUS_TIMEOUT);
}

// Rows that several CTAs share: CTA c's run begins an item and the next ones finish it.  A CTA
// of this kernel joins 8 rows, a row and 4 columns per thread: the pieces' outputs weighted by 2^(maximum - common maximum), in the
// order of the CTAs.  The weights are formed first, by the warps a row each.
constexpr int kJoinRows = 8;
constexpr int kJoinMany = 64;  // pieces whose weights are kept at a time

template <int D>
__global__ void __launch_bounds__(kJoinRows * D / 4) cache_join_kernel(const __grid_constant__ CacheAttnParams p) {
  __shared__ float s_w[kJoinRows][kJoinMany];
  __shared__ float s_inv[kJoinRows];
  pdl_launch();
  pdl_wait();
  if (p.meta[C_VALID] == 0) return;
  const int c = blockIdx.x, row0 = blockIdx.y * kJoinRows;
  const int4 de = p.desc[2 * c];
  if (de.x == 0 || row0 >= de.w * p.G) return;
  const int n = p.desc[2 * c + 1].x;
  auto slot = [&](int k) { return k == 0 ? 2 * c + 1 : 2 * (c + k); };
  const int r = threadIdx.x % kJoinRows, c4 = threadIdx.x / kJoinRows, row = row0 + r;  // row < rows (a multiple of 8)
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kJoinRows * D / 4 / 32;
  for (int k0 = 0; k0 < n; k0 += kJoinMany) {
    const int m = min(n - k0, kJoinMany);
    if (k0 > 0) __syncthreads();
    for (int q = warp; q < kJoinRows; q += warps) {
      float top = -INFINITY, l = 0.f;
      for (int k = lane; k < n; k += 32) top = fmaxf(top, p.ml[static_cast<int64_t>(slot(k)) * p.rows + row0 + q].x);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
      for (int k = lane; k < n; k += 32) {
        const float2 a = p.ml[static_cast<int64_t>(slot(k)) * p.rows + row0 + q];
        const float w = a.x == -INFINITY ? 0.f : ex2(a.x - top);
        l = fmaf(a.y, w, l);
        if (k >= k0 && k < k0 + m) s_w[q][k - k0] = w;
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
      if (lane == 0) s_inv[q] = 1.f / l;
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < m; ++k) {
      const float4 y = p.part[cache_part(p, slot(k0 + k), row, c4)];
      const float w = s_w[r][k];
      x.x = fmaf(y.x, w, x.x);
      x.y = fmaf(y.y, w, x.y);
      x.z = fmaf(y.z, w, x.z);
      x.w = fmaf(y.w, w, x.w);
    }
  }
  if (row >= de.w * p.G) return;
  const float inv = s_inv[r];
  uint2 o;
  o.x = pack_bf16(x.x * inv, x.y * inv);
  o.y = pack_bf16(x.z * inv, x.w * inv);
  *reinterpret_cast<uint2*>(p.o + (static_cast<int64_t>(de.z + row / p.G) * p.Hq + de.y * p.G + row % p.G) * D + c4 * 4) = o;
}

template <int D, int MT>
int launch_small(const CacheAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int ctas, cudaStream_t s) {
  using LY = SmallLayout<D, MT>;
  if (allow_smem<cache_small_kernel<D, MT>>(LY::SMEM) != FORK_OK) return FORK_ECUDA;
  return cuda_rc(launch_pdl(cache_small_kernel<D, MT>, ctas, kThreads, LY::SMEM, s, kmap, vmap, p));
}

template <int D>
int launch_cache_attn(const CacheAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap,
                      cudaStream_t s) {
  const int ctas = std::min(sm_count(), kMaxCtas);
  int rc;
  if (p.rows == 16) {
    rc = launch_small<D, 1>(p, kmap, vmap, ctas, s);
  } else if (p.rows == 32) {
    if constexpr (D == 64) rc = launch_small<D, 2>(p, kmap, vmap, ctas, s);
    else rc = FORK_EINVAL;  // (cache_item_rows gives 32 rows for heads of 64 alone)
  } else {
    rc = launch_cache_attn_tc<D>(p, qmap, kmap, vmap, ctas, s);
  }
  if (rc != FORK_OK) return rc;
  return cuda_rc(launch_pdl(cache_join_kernel<D>, dim3(ctas, p.rows / kJoinRows), kJoinRows * D / 4, 0, s, p));
}

struct CacheAttnWs {
  size_t desc, ml, part, total;
};
CacheAttnWs cache_attn_ws(int rows, int d) {
  CacheAttnWs w;
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  w.desc = 0;
  w.ml = al(w.desc + 2 * kMaxCtas * sizeof(int4));
  w.part = al(w.ml + static_cast<size_t>(2 * kMaxCtas) * rows * sizeof(float2));
  w.total = al(w.part + static_cast<size_t>(2 * kMaxCtas) * rows * d * sizeof(float));
  return w;
}

}  // namespace
}  // namespace fork

using namespace fork;

extern "C" size_t fork_cache_attn_workspace_bytes(const fork_cache* c) {
  CacheLayout L;
  if (check_cache(c, &L) != FORK_OK) return 0;
  return cache_attn_ws(cache_item_rows(c->max_new, c->Hq / c->Hkv, c->d), c->d).total;
}

extern "C" int fork_cache_attn(const fork_cache* c, const uint16_t* q, const uint16_t* kc, const uint16_t* vc,
                               uint16_t* o, int32_t window, float scale, void* workspace, size_t ws_bytes,
                               uint32_t flags, void* stream) {
  CacheLayout L;
  int rc = check_cache(c, &L);
  if (rc != FORK_OK) return rc;
  if (!q || !kc || !vc || !o || !workspace) return FORK_EINVAL;
  if (!is_aligned16(q) || !is_aligned16(kc) || !is_aligned16(vc) || !is_aligned16(o) || !is_aligned16(workspace))
    return FORK_EINVAL;
  if (window < 0 || !(scale > 0.f) || !std::isfinite(scale)) return FORK_EINVAL;
  const int G = c->Hq / c->Hkv, rows = cache_item_rows(c->max_new, G, c->d);
  const CacheAttnWs w = cache_attn_ws(rows, c->d);
  if (ws_bytes < w.total) return FORK_EINVAL;
  if ((rc = check_device()) != FORK_OK) return rc;
  CacheAttnParams p;
  p.meta = static_cast<int32_t*>(c->d_buf);
  p.L = L;
  p.table = c->table;
  p.q = q;
  p.o = o;
  p.Hq = c->Hq;
  p.Hkv = c->Hkv;
  p.G = G;
  p.d = c->d;
  p.P = c->page_tokens;
  p.P_shift = page_shift(p.P);
  p.max_blocks = c->max_blocks;
  p.n_pages = c->n_pages;
  p.tile = cache_item_tokens(c->max_new, G, c->d);
  p.rows = rows;
  p.window = window;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_ns = c->wait_us == 0 ? 2000000000ull : static_cast<uint64_t>(c->wait_us) * 1000ull;
  p.stall = (flags & FORK_TEST_STALL) ? 1 : 0;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.desc = reinterpret_cast<int4*>(ws + w.desc);
  p.ml = reinterpret_cast<float2*>(ws + w.ml);
  p.part = reinterpret_cast<float4*>(ws + w.part);
  alignas(64) CUtensorMap kmap, vmap, qmap;
  const int64_t planes = static_cast<int64_t>(c->n_pages) * c->Hkv;
  if (planes > 0x7fffffff) return FORK_EINVAL;
  const int box = std::min(c->page_tokens, kKeyTile);
  if (!encode_map_3d(&kmap, kc, c->d, c->page_tokens, planes, 64, box, 1, true) ||
      !encode_map_3d(&vmap, vc, c->d, c->page_tokens, planes, 64, box, 1, true))
    return FORK_ECUDA;
  if (rows >= 128 && !encode_map_3d(&qmap, q, c->d, c->Hq, c->T_cap, 64, G, 128 / G, true)) return FORK_ECUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return c->d == 64 ? launch_cache_attn<64>(p, kmap, vmap, qmap, s) : launch_cache_attn<128>(p, kmap, vmap, qmap, s);
}
