// Attention over the paged cache for steps of many query rows per kv head (drafted trees,
// prompt chunks), on tcgen05.
//
// A piece of an item (fork_cache_attn.cuh) is two streams of 128 query rows x 128 keys.  An
// item of more than 128 rows has two query tiles and each stream takes one of them over every
// key tile; an item of up to 128 rows has one query tile, and the streams take the even and
// the odd key tiles, each with a running maximum, sum and output of its own, joined at the
// end.  Either way one stream's exponentials run while the other's products do.
//   warps 1, 10 producers: the pieces, query tiles and K tiles (warp 1) and V tiles (warp 10)
//               by TMA, page by page, into two rings.  Two, because a V tile waits for its
//               exponentials while its K tile is long done: K runs ahead of V
//   warp 0      one lane issues tcgen05.mma: by turns for the two streams O_t += P_t V, S_t =
//               Q K^T, all waits of a turn at once before its products, a barrier per lane.  An
//               issuer per stream measured 8% slower (131,000 keys x 256 rows: 165 / 152 us when
//               it was tried)
//   warps 2-5, 6-9  softmax of stream 0 / 1, thread = row = TMEM lane: S from TMEM, what the
//               row sees, running maximum (moved only when it grows by more than 2^8, so
//               that O is rescaled rarely), exponentials as bf16 into the columns of S, from
//               where the PV product reads them; at the end O / l or a partial result
// 131,000 keys x 256 rows (8 kv heads of 128; 538 MB, 137 GFLOP): 133 us back to back (135 to 138
// among other calls), 0.60 of the measured HBM rate and 0.54 of the measured tensor rate at once;
// bound by the turn of softmax and products
// (without exponentials 113 us, without copies 143 of then 148, without both 107).  16 requests x
// 64 nodes: 99 us, 839 TFLOP/s.  32 requests x 8 nodes x 4 heads of 128 (0.53 GB): 94 us, 5.6 TB/s.
// TMEM: S_t / P_t at columns 128 t, O_t at 256 + t D.  QK^T and PV in bf16 with float32 sums.
// Every wait is bounded; on a timeout the CTA drains its own copies and products, frees TMEM
// and exits with FORK_STATUS_TIMEOUT.
#include "fork_attn.cuh"
#include "fork_cache_attn.cuh"

namespace fork {

namespace {

constexpr int kRows = 128;
constexpr int kBox = 128 * 128;  // bytes of 128 rows x 64 bf16
constexpr int kThreads = 352;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescale = 8.f;
constexpr int kPieces = 4;

// NQ: query tiles that an item can have.  One leaves room for another slot: a third of K, which
// is asked for first (32 requests x 8 tokens x 4 heads of 128: 93.7 us, with the third for V 95.1).
template <int D, int NQ>
struct TcLayout {
  static constexpr int NB = D / 64;
  static constexpr int SLOT = NB * kBox;
  static constexpr int NK = NB == 2 ? (NQ == 1 ? 3 : 2) : 4;  // K slots
  static constexpr int NV = NB == 2 ? 2 : (NQ == 1 ? 6 : 4);  // V slots, behind them
  static constexpr int NS = NK + NV;
  static constexpr int Q = NS * SLOT;
  static constexpr int MLX = Q + NQ * NB * kBox;  // [2 pieces][2 streams][128] (m, l)
  static constexpr int BAR = MLX + 2 * 2 * kRows * 8;
  static constexpr int BYTES = BAR + 1536;
  static constexpr int SMEM = BYTES + 1024 > 120 * 1024 ? BYTES + 1024 : 120 * 1024;  // one CTA per SM (TMEM)
};

// barriers behind full[NS] and empty[NS]
enum Bar { B_QFULL = 0, B_QEMPTY, B_SFULL0, B_SFULL1, B_PFULL0, B_PFULL1, B_OFULL0, B_OFULL1, B_OFREE0, B_OFREE1, B_VFIX0,
           B_VFIX1, B_VFIXALL, B_MLX, B_FIN, B_STALL, B_VGO, B_PIECEF, B_PIECEE = B_PIECEF + kPieces, B_COUNT = B_PIECEE + kPieces };

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
__device__ __forceinline__ bool odd_pair(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// two float32 product-sums in one instruction
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float* lo, float* hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// both halves of a bf16 pair added to float32 sums, without a conversion
__device__ __forceinline__ void add_halves(uint32_t w, float* lo, float* hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n add.rn.f32.bf16 %0, a, %0;\n add.rn.f32.bf16 %1, b, %1;\n}"
      : "+f"(*lo), "+f"(*hi)
      : "r"(w));
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(tc::smem_u32(bar)), "r"(n) : "memory");
}
// element `col` of row `row` of a 128-byte-swizzled tile of 128-row boxes
__device__ __forceinline__ uint32_t swz(int row, int col) {
  return static_cast<uint32_t>((col >> 6) * kBox + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4));
}

}  // namespace

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
    cache_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CacheAttnParams p) {
  using LY = TcLayout<D, NQ>;
  constexpr int NB = LY::NB, NS = LY::NS, NK = LY::NK, NV = LY::NV;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + LY::BAR);
  uint64_t* empty = full + NS;
  uint64_t* bars = empty + NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* acc_first = reinterpret_cast<volatile int*>(tmem_slot + 2);  // [2]: O_t holds something before its first product
  uint32_t* odd_keys = tmem_slot + 4;  // [stream 0, 1, both][2][4] bits: keys with an infinity or NaN
  CachePiece* pieces = reinterpret_cast<CachePiece*>(tmem_slot + 28);
  static_assert((2 * NS + B_COUNT) * 8 + 28 * 4 + kPieces * sizeof(CachePiece) <= 1536, "barrier region");
  float2* mlx = reinterpret_cast<float2*>(smem + LY::MLX);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(&bars[B_SFULL0 + t], 1);
      tc::mbar_init(&bars[B_PFULL0 + t], 128);
      tc::mbar_init(&bars[B_OFULL0 + t], 1);
      tc::mbar_init(&bars[B_OFREE0 + t], 256);
      tc::mbar_init(&bars[B_VFIX0 + t], 4);
    }
    tc::mbar_init(&bars[B_QFULL], 1);
    tc::mbar_init(&bars[B_QEMPTY], 1);
    tc::mbar_init(&bars[B_FIN], 1);
    tc::mbar_init(&bars[B_VFIXALL], 8);
    tc::mbar_init(&bars[B_MLX], 8);
    tc::mbar_init(&bars[B_STALL], 1);
    tc::mbar_init(&bars[B_VGO], 1);
    for (int i = 0; i < kPieces; ++i) {
      tc::mbar_init(&bars[B_PIECEF + i], 1);
      tc::mbar_init(&bars[B_PIECEE + i], 9);  // the issuer, eight softmax warps
    }
    *abort = 0;
    acc_first[0] = acc_first[1] = 0;
    for (int i = 0; i < 24; ++i) odd_keys[i] = 0;
    tc::fence_mbar_init();
  }
  if (tid == 32) {
    tc::prefetch_tmap(&qmap);
    tc::prefetch_tmap(&kmap);
    tc::prefetch_tmap(&vmap);
  }
  if (warp == 0) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  pdl_launch();
  pdl_wait();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool valid_step = p.meta[C_VALID] != 0;
  auto tm_s = [&](int t) -> uint32_t { return tmem + static_cast<uint32_t>(t) * 128u; };
  auto tm_o = [&](int t) -> uint32_t { return tmem + 256u + static_cast<uint32_t>(t * D); };
  const int tile_tok = kRows / p.G;  // tokens of a query tile

  if (!valid_step) {
    // a refused step: nothing is read or written
  } else if (warp == 1 || warp == 10) {
    // ===================== producers: pieces, queries and keys / values =====================
    const bool keys = warp == 1;
    const CUtensorMap* map = keys ? &kmap : &vmap;
    const CacheSplit split = cache_split(p);
    if (keys && lane == 0) p.desc[2 * blockIdx.x].x = 0;
    const uint64_t evict = tc::policy_evict_first(), normal = tc::policy_normal();
    CacheWalk walk(split);
    auto wait = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, tc::mbar_wait(bar, par, abort, p.wait_ns));
    };
    const int first = keys ? 0 : NK, slots = keys ? NK : NV;
    int f = 0, s = 0, ring = 0;  // tiles issued, the next one's slot and turn
    int nq = 0;                  // pieces whose query tiles were issued
    // the first values come after the first keys: all SMs start at once, and what is needed
    // first would share HBM with what is needed last
    bool ok = keys || split.begin == split.end || wait(&bars[B_VGO], 0);
    for (int n = 0; ok; ++n) {
      const CachePiece c = walk.next(p);
      if (keys) {
        const int ps = n % kPieces;
        if (n >= kPieces && !(ok = wait(&bars[B_PIECEE + ps], ((n / kPieces) - 1) & 1))) break;
        if (lane == 0) {
          pieces[ps] = c;
          tc::mbar_arrive(&bars[B_PIECEF + ps]);
        }
      }
      if (!c.ok) break;
      if (keys) {
        // the query tiles, once the previous piece's products have read theirs
        const int ntiles = NQ == 2 && c.it.nt > tile_tok ? 2 : 1;
        if (nq > 0 && !(ok = wait(&bars[B_QEMPTY], (nq - 1) & 1))) break;
        if (lane == 0) {
          tc::mbar_expect_tx(&bars[B_QFULL], ntiles * NB * 128 * p.G * tile_tok);
          for (int t = 0; t < ntiles; ++t)
            for (int b = 0; b < NB; ++b)
              tc::tma_load_3d(smem + LY::Q + (t * NB + b) * kBox, &qmap, &bars[B_QFULL], b * 64, c.g * p.G,
                              c.it.row + t * tile_tok);
        }
        ++nq;
      }
      // pages read ahead, 32 blocks at a time; blocks without a visible key and bad pages come
      // as zeros (a box outside the tensor)
      const int32_t* row = p.table + static_cast<int64_t>(c.it.b) * p.max_blocks;
      const int b_lo = c.it.lo >> p.P_shift, b_hi = (c.it.hi - 1) >> p.P_shift;
      const int per = max(kKeyTile >> p.P_shift, 1), box = min(p.P, kKeyTile);
      const uint64_t policy = c.it.only ? evict : normal;
      auto fetch = [&](int blk) {
        if (blk < b_lo || blk > b_hi) return -1;
        const int page = row[blk];
        if (page < 0 || page >= p.n_pages) {
          atomicOr(p.meta + C_STATUS, FORK_STATUS_BAD_PAGE);
          return -1;
        }
        return page;
      };
      int base = (c.t0 * kKeyTile) >> p.P_shift;
      int cur = fetch(base + lane), nxt = fetch(base + 32 + lane);
      for (int j = 0; j < c.n; ++j) {
        const int blk = ((c.t0 + j) * kKeyTile) >> p.P_shift;
        if (blk - base >= 32) {
          base += 32;
          cur = nxt;
          nxt = fetch(base + 32 + lane);
        }
        const int page = __shfl_sync(0xffffffffu, cur, (blk - base + min(lane, per - 1)) & 31);
        const int in_page = ((c.t0 + j) * kKeyTile) & (p.P - 1);
        const int64_t z = page < 0 ? static_cast<int64_t>(p.n_pages) * p.Hkv : static_cast<int64_t>(page) * p.Hkv + c.g;
        uint64_t* bar = &full[first + s];
        if (f >= slots && !(ok = wait(&empty[first + s], (ring - 1) & 1))) break;
        if (lane == 0) tc::mbar_expect_tx(bar, LY::SLOT);
        __syncwarp();
        if (lane < per) {
          unsigned char* dst = smem + (first + s) * LY::SLOT + lane * box * 128;
#pragma unroll
          for (int b = 0; b < NB; ++b) tc::tma_load_3d(dst + b * kBox, map, bar, b * 64, in_page, static_cast<int>(z), policy);
        }
        ++f;
        if (++s == slots) {
          s = 0;
          ++ring;
        }
      }
      if (keys && lane == 0) cache_describe(p, split, c, walk.at - c.n + c.it.kt);
    }
    // the last copies complete by themselves
    if (lane == 0) {
      if (nq > 0) tc::mbar_drain(&bars[B_QFULL], (nq - 1) & 1);
      for (int i = max(0, f - slots); i < f; ++i) tc::mbar_drain(&full[first + i % slots], (i / slots) & 1);
    }
    __syncwarp();
  } else if (warp == 0) {
    // ===================== MMA issuer (lane 0) =====================
    if (lane == 0) {
      constexpr uint32_t idesc_qk = tc::idesc_bf16(128, kKeyTile, 0, 0);
      constexpr uint32_t idesc_pv = tc::idesc_bf16(128, D, 0, 1);
      const uint64_t dq = tc::sdesc_sw128(tc::smem_u32(smem + LY::Q), 16, 1024);
      const uint64_t dk = tc::sdesc_sw128(tc::smem_u32(smem), 16, 1024);
      const uint64_t dv = tc::sdesc_sw128(tc::smem_u32(smem), kBox, 1024);
      constexpr uint64_t kBoxU = kBox / 16, kSlotU = LY::SLOT / 16;
      auto wait = [&](uint64_t* bar, uint32_t par) -> bool { return tc::mbar_wait(bar, par, abort, p.wait_ns); };
      bool ok = !p.stall || wait(&bars[B_STALL], 0);  // FORK_TEST_STALL: runs out, nothing is issued
      int F = 0, nS[2] = {0, 0}, nO[2] = {0, 0};
      for (int n = 0; ok; ++n) {
        const int ps = n % kPieces;
        if (!(ok = wait(&bars[B_PIECEF + ps], (n / kPieces) & 1))) break;
        const int alive = pieces[ps].ok, total = pieces[ps].n, two = NQ == 2 && pieces[ps].it.nt > tile_tok;
        tc::mbar_arrive(&bars[B_PIECEE + ps]);
        if (!alive) break;
        if (!(ok = wait(&bars[B_QFULL], n & 1))) break;
        // round i, stream t: key tile i (two query tiles) or 2 i + t (one)
        const int rounds = two ? total : (total + 1) / 2;
        for (int i = 0; ok && i <= rounds; ++i) {
          for (int t = 0; ok && t < 2; ++t) {
            const int jp = two ? i - 1 : 2 * (i - 1) + t, j = two ? i : 2 * i + t;
            const bool prev = i > 0 && jp < total, next = i < rounds && j < total;
            const int kf = F + j, ks = kf % NK, vf = F + jp, vs = NK + vf % NV;
            // (with two query tiles stream 0 has waited for both)
            if (next && !(two && t)) {
              if (!(ok = wait(&full[ks], (kf / NK) & 1))) break;
              if (kf == 0) tc::mbar_arrive(&bars[B_VGO]);
            }
            if (prev) {
              // O_t += P_t V(jp): V landed, P_t published, O_t free of the previous piece
              if (!(two && t) && !(ok = wait(&full[vs], (vf / NV) & 1))) break;
              if (!(ok = wait(&bars[B_PFULL0 + t], (nS[t] - 1) & 1))) break;
              const bool first = i == 1;
              if (first && nO[t] > 0 && !(ok = wait(&bars[B_OFREE0 + t], (nO[t] - 1) & 1))) break;
              const bool over = first && !acc_first[t];
              if (first) acc_first[t] = 0;
              tc::tc_fence_after();
              const uint64_t d0 = dv + vs * kSlotU;
#pragma unroll
              for (int s = 0; s < kKeyTile / 16; ++s)
                tc::mma_f16_ts(tm_o(t), tm_s(t) + s * 8, d0 + s * (2048 / 16), idesc_pv, (!over || s > 0) ? 1u : 0u);
              if (!two || t) tc::mma_commit(&empty[vs]);
            }
            if (next) {
              const uint64_t a0 = dq + (two ? t : 0) * NB * kBoxU, b0 = dk + ks * kSlotU;
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  tc::mma_bf16(tm_s(t), a0 + b * kBoxU + k * 2, b0 + b * kBoxU + k * 2, idesc_qk, (b | k) ? 1u : 0u);
              tc::mma_commit(&bars[B_SFULL0 + t]);
              ++nS[t];
              if (!two || t) tc::mma_commit(&empty[ks]);
            }
          }
          if (ok && i + 1 == rounds) tc::mma_commit(&bars[B_QEMPTY]);  // the last readers of Q are issued
        }
        if (!ok) break;
        // a stream without a tile in this piece: its outputs of the previous piece are read
        // before its barrier moves on
        if (!two && total == 1 && nO[1] > 0 && !(ok = wait(&bars[B_OFREE1], (nO[1] - 1) & 1))) break;
        for (int t = 0; t < 2; ++t) {
          tc::mma_commit(&bars[B_OFULL0 + t]);
          ++nO[t];
        }
        F += total;
      }
      tc::mma_commit(&bars[B_FIN]);
      tc::mbar_drain(&bars[B_FIN], 0);
    }
    __syncwarp();
  } else {
    // ===================== softmax of stream t =====================
    const int t = (warp - 2) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tm_s(t) + lane_base, to = tm_o(t) + lane_base;
    const int lrow = (warp & 3) * 32 + lane;  // row of the query tile = TMEM lane
    const float sl2 = p.scale_log2;
    auto wait = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, tc::mbar_wait(bar, par, abort, p.wait_ns));
    };
    int F = 0, nS = 0, nO = 0, nFix = 0, nFixAll = 0, nMlx = 0, nOdd = 0, nOddAll = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int ps = n % kPieces;
      if (!(ok = wait(&bars[B_PIECEF + ps], (n / kPieces) & 1))) break;
      const CachePiece c = pieces[ps];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars[B_PIECEE + ps]);
      if (!c.ok) break;
      const CacheItem& it = c.it;
      const bool two = NQ == 2 && it.nt > tile_tok;
      const int tok = lrow < tile_tok * p.G ? lrow / p.G + (two ? t * tile_tok : 0) : it.nt;
      const CacheRow see = cache_row(p, it, tok);
      // padding rows (whatever their queries) never move their maximum
      const bool pad = tok >= it.nt;
      float l = 0.f, m_used = pad ? 0.f : -INFINITY;
      const int step = two ? 1 : 2;
      for (int j = two ? 0 : t; j < c.n; j += step) {
        const int tile = c.t0 + j, y0 = tile * kKeyTile;
        if (!(ok = wait(&bars[B_SFULL0 + t], nS & 1))) break;
        ++nS;
        tc::tc_fence_after();
        float sv[kKeyTile];
        {
          uint32_t raw[kKeyTile];
#pragma unroll
          for (int i = 0; i < kKeyTile / 32; ++i) tc::tmem_ld32(ts + i * 32, raw + i * 32);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kKeyTile; ++i) sv[i] = __uint_as_float(raw[i]);
        }
        const bool masked = cache_masked(p, it, tile);
        if (masked) {
#pragma unroll
          for (int w = 0; w < kKeyTile / 32; ++w) {
            const uint32_t bits = cache_seen(see, it.len, y0 + 32 * w);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((bits >> i) & 1u)) sv[32 * w + i] = -INFINITY;
          }
        }
        float mx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mx[e] = sv[e];
#pragma unroll
        for (int i = 8; i < kKeyTile - 8; i += 16)
#pragma unroll
          for (int e = 0; e < 8; ++e) mx[e] = max3(mx[e], sv[i + e], sv[i + 8 + e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx[e] = fmaxf(mx[e], sv[kKeyTile - 8 + e]);
        const float mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sl2;
        const bool resc = !pad && (mt > m_used + kRescale || m_used == -INFINITY);
        const float m_new = resc ? mt : m_used;
        const float at = m_new == -INFINITY ? 0.f : m_new;
        const float factor = resc ? ex2(m_used - at) : 1.f;
        // Rounded to bf16 for the product; the sum takes the rounded values, so that the rounding
        // cancels where one key carries the row (unrounded: 131 us for 135 us, and up to 1.4 times
        // the error of the output's own rounding).  The products bound this kernel: with a second one
        // for what the rounding leaves, as the kernel for few rows has it, 131,000 keys x 256 rows
        // take 184 us for 132, 16 requests x 64 nodes 137 for 99, prompt chunks 196 for 138; the
        // relative error against 64 bits would fall from 0.0021 to 0.0017 (the result's rounding)
        const uint64_t sl2x2 = pair(sl2, sl2), atx2 = pair(-at, -at);
        float fs[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int i = h * 32 + 2 * e;
            float lo, hi;
            unpair(fma2(pair(sv[i], sv[i + 1]), sl2x2, atx2), &lo, &hi);
            pk[e] = pack_bf16(ex2(lo), ex2(hi));
            add_halves(pk[e], &fs[e & 3], &fs[4 + (e & 3)]);
          }
          tc::tmem_st16(ts + h * 16, pk);
        }
        {
          l = fmaf(l, factor, ((fs[0] + fs[1]) + (fs[2] + fs[3])) + ((fs[4] + fs[5]) + (fs[6] + fs[7])));
        }
        m_used = m_new;
        const bool first = j < step;
        // O_t holds the products of this stream's earlier tiles (all complete: S_t was
        // committed after them); none is issued before P_t is published
        if (!first && __any_sync(0xffffffffu, factor != 1.f)) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t ov[32];
            tc::tmem_ld32(to + i * 32, ov);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * factor);
            tc::tmem_st32(to + i * 32, ov);
          }
        }
        if (masked) {
          // A masked key has p = 0, but 0 * NaN is NaN: values of keys that no row of the item
          // sees are set to zero; an infinity or NaN among the others is taken out of the
          // product and added to the rows that see it.
          const int vf = F + j, slot = NK + vf % NV;
          if (!(ok = wait(&full[slot], (vf / NV) & 1))) break;
          unsigned char* vs = smem + slot * LY::SLOT;
          // this thread's keys: with one query tile a key each; with two, stream t has half
          const int nthr = two ? 256 : 128, me = two ? t * 128 + lrow : lrow;
          // its flags, by turns: a slow warp may still read those of the tile before
          uint32_t* odd = odd_keys + (two ? 16 + 4 * (nOddAll++ & 1) : 8 * t + 4 * (nOdd++ & 1));
          uint64_t* bar = &bars[two ? B_VFIXALL : B_VFIX0 + t];
          auto meet = [&]() {
            __syncwarp();
            int& k = two ? nFixAll : nFix;
            if (lane == 0) tc::mbar_arrive(bar);
            const bool r = wait(bar, k & 1);
            ++k;
            return r;
          };
          for (int e = me; e < kKeyTile * (D / 8); e += nthr) {
            const int r = e / (D / 8), y = y0 + r;
            uint4* x = reinterpret_cast<uint4*>(vs + swz(r, (e % (D / 8)) * 8));
            if (y < it.lo || y >= it.hi) *x = make_uint4(0, 0, 0, 0);
            else if (odd_pair(x->x) || odd_pair(x->y) || odd_pair(x->z) || odd_pair(x->w)) atomicOr(&odd[r >> 5], 1u << (r & 31));
          }
          tc::fence_proxy_async_smem();
          if (!(ok = meet())) break;
          const uint32_t o0 = odd[0], o1 = odd[1], o2 = odd[2], o3 = odd[3];
          if (o0 | o1 | o2 | o3) {
            if (first) {  // O_t, free of the previous piece, starts at zero instead of being overwritten
              if (nO > 0 && !(ok = wait(&bars[B_OFREE0 + t], (nO - 1) & 1))) break;
              tc::tc_fence_after();
              uint32_t zero[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) zero[e] = 0;
              for (int i = 0; i < D / 32; ++i) tc::tmem_st32(to + i * 32, zero);
              tc::tmem_wait_st();
              if (lane == 0) acc_first[t] = 1;
            }
            for (int i = 0; i < D / 32; ++i) {
              uint32_t ov[32];
              tc::tmem_wait_st();
              tc::tmem_ld32(to + i * 32, ov);
              tc::tmem_wait_ld();
              for (int r = 0; r < kKeyTile; ++r) {
                const uint32_t w = r < 32 ? o0 : (r < 64 ? o1 : (r < 96 ? o2 : o3));
                if (!((w >> (r & 31)) & 1u)) continue;
                if (!(cache_seen(see, it.len, y0 + r) & 1u)) continue;
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  const uint32_t x = *reinterpret_cast<const uint32_t*>(vs + swz(r, i * 32 + (e & ~7)) + (e & 7) * 2);
                  if ((x & 0x7f80u) == 0x7f80u) ov[e] = __float_as_uint(__uint_as_float(ov[e]) + lo_f(x));
                  if ((x & 0x7f800000u) == 0x7f800000u) ov[e + 1] = __float_as_uint(__uint_as_float(ov[e + 1]) + hi_f(x));
                }
              }
              __syncwarp();
              tc::tmem_st32(to + i * 32, ov);
            }
            tc::tmem_wait_st();
            if (!(ok = meet())) break;
            for (int e = me; e < kKeyTile * (D / 8); e += nthr) {
              uint4* x = reinterpret_cast<uint4*>(vs + swz(e / (D / 8), (e % (D / 8)) * 8));
              uint32_t w[4] = {x->x, x->y, x->z, x->w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if ((w[q] & 0x7f80u) == 0x7f80u) w[q] &= 0xffff0000u;
                if ((w[q] & 0x7f800000u) == 0x7f800000u) w[q] &= 0xffffu;
              }
              *x = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (me < 4) odd[me] = 0;
            tc::fence_proxy_async_smem();
            if (!(ok = meet())) break;
          }
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        tc::mbar_arrive(&bars[B_PFULL0 + t]);
      }
      if (!ok) break;
      F += c.n;
      // ---- the piece's result
      float a[2] = {1.f, 0.f}, m = m_used;
      if (!two) {  // one query tile: the two streams' shares of its rows
        float2* mine = mlx + (nMlx & 1) * 2 * kRows;
        mine[t * kRows + lrow] = make_float2(m_used, l);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[B_MLX]);
        if (!(ok = wait(&bars[B_MLX], nMlx & 1))) break;
        ++nMlx;
        const float2 x = mine[lrow], y = mine[kRows + lrow];
        m = fmaxf(x.x, y.x);
        a[0] = x.x == -INFINITY ? 0.f : ex2(x.x - m);
        a[1] = y.x == -INFINITY ? 0.f : ex2(y.x - m);
        l = x.y * a[0] + y.y * a[1];
      }
      // streams of this thread's output, and its columns
      const int s0 = two ? t : 0, s1 = two ? t : (c.n > 1 ? 1 : 0);
      for (int s = s0; ok && s <= s1; ++s) ok = wait(&bars[B_OFULL0 + s], nO & 1);
      if (!ok) break;
      ++nO;
      tc::tc_fence_after();
      const int i0 = two ? 0 : t * (D / 64), i1 = two ? D / 32 : i0 + D / 64;
      const bool valid = !pad;
      const int rrow = (two ? t * tile_tok * p.G : 0) + lrow;
      const float inv = c.slot < 0 ? 1.f / l : 1.f;
      uint16_t* orow = p.o + (static_cast<int64_t>(it.row + tok) * p.Hq + c.g * p.G + lrow % p.G) * D;
      const int64_t at = static_cast<int64_t>(max(c.slot, 0)) * p.rows + rrow;
      for (int i = i0; i < i1; ++i) {
        float ov[32];
        {
          uint32_t raw[32];
          tc::tmem_ld32(tm_o(s0) + lane_base + i * 32, raw);
          tc::tmem_wait_ld();
          const float w = two ? inv : a[0] * inv;
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = __uint_as_float(raw[e]) * w;
          if (s1 != s0) {
            tc::tmem_ld32(tm_o(1) + lane_base + i * 32, raw);
            tc::tmem_wait_ld();
            const float w1 = a[1] * inv;
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = fmaf(__uint_as_float(raw[e]), w1, ov[e]);
          }
        }
        if (valid && c.slot < 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 v4;
            v4.x = pack_bf16(ov[q * 8 + 0], ov[q * 8 + 1]);
            v4.y = pack_bf16(ov[q * 8 + 2], ov[q * 8 + 3]);
            v4.z = pack_bf16(ov[q * 8 + 4], ov[q * 8 + 5]);
            v4.w = pack_bf16(ov[q * 8 + 6], ov[q * 8 + 7]);
            *reinterpret_cast<uint4*>(orow + i * 32 + q * 8) = v4;
          }
        } else if (valid) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            p.part[cache_part(p, c.slot, rrow, i * 8 + q)] = make_float4(ov[q * 4], ov[q * 4 + 1], ov[q * 4 + 2], ov[q * 4 + 3]);
        }
      }
      if (valid && c.slot >= 0 && (two || t == 0)) p.ml[at] = make_float2(m, l);
      // the outputs are read: the next piece's products may overwrite them
      tc::tc_fence_before();
      if (two) {
        mbar_arrive_n(&bars[B_OFREE0 + t], 2);
      } else {
        tc::mbar_arrive(&bars[B_OFREE0]);
        tc::mbar_arrive(&bars[B_OFREE1]);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*abort && tid == 0) atomicOr(p.meta + C_STATUS, FORK_STATUS_TIMEOUT);
  if (warp == 0) {
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int NQ>
static int launch_tc(const CacheAttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                     int ctas, cudaStream_t s) {
  using LY = TcLayout<D, NQ>;
  if (allow_smem<cache_tc_kernel<D, NQ>>(LY::SMEM) != FORK_OK) return FORK_ECUDA;
  return cuda_rc(launch_pdl(cache_tc_kernel<D, NQ>, ctas, kThreads, LY::SMEM, s, qmap, kmap, vmap, p));
}

template <int D>
int launch_cache_attn_tc(const CacheAttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                         int ctas, cudaStream_t s) {
  return p.rows == 128 ? launch_tc<D, 1>(p, qmap, kmap, vmap, ctas, s) : launch_tc<D, 2>(p, qmap, kmap, vmap, ctas, s);
}

template int launch_cache_attn_tc<64>(const CacheAttnParams&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, int,
                                      cudaStream_t);
template int launch_cache_attn_tc<128>(const CacheAttnParams&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, int,
                                       cudaStream_t);

}  // namespace fork
