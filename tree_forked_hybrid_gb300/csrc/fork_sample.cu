// Sampling: one token per row of logits, from given uniform numbers.
//
// For a row x with temperature t: z_i = (x_i - max x) / t, w_i = e^(z_i).  Top-k keeps the k
// largest (ties: the lowest index), top-p of those the shortest prefix in the same order whose
// mass reaches top_p of theirs, min-p of those the tokens with w_i >= min_p.  The token is the
// first in index order whose cumulative kept weight exceeds u times their sum.
//
// Which token is drawn must not depend on the order of a sum, so weights are 64-bit fixed
// point (44 fractional bits) and every sum is an exact integer sum, whatever splits it: z
// log2(e) as a pair of floats, 2^f by a table of 64 and a short series, accurate to about
// 2^-35 (float32's own 2^-23 would move one draw in some thousand on a flat row; float64
// arithmetic runs at a 64th of the rate).  That costs some 80 instructions, so it is left to
// the tokens within 5 octaves of the maximum, gathered 32 at a time; below, weights to 2^-29 of
// themselves do and are formed in place, two tokens at a time.
//
// One CTA per row, or a cluster of up to 8 for few long rows; a warp owns a contiguous run of
// its CTA's part, so that index order is warp order.  The first pass reads the row from HBM
// and keeps maxima; later ones find it in L2.  What can be drawn is narrowed without a sort:
// for min-p by its own level; for top-k by the k-th largest of some 3000 maxima of parts; for
// top-p (and a large k) by a pass that sorts mass (or counts) into 256 bins below the maximum:
// the cut lies in one of them, whose tokens are sorted again while they are many.  The few that
// are left are copied, in index order, to the shared memory of one CTA, where the exact cut is
// a radix select over their keys, 8 bits at a time.  When they do not get few (ties by the
// thousand) the select runs over the row itself.  A row drawn from without a list is summed by
// runs, then the run that holds the draw by all warps once more.
//
// 512 rows of 131072 floats (normal, sigma 2, and 24 that stand out), thousands of cycles of a
// row: the maximum 29 (HBM), a list of candidates 28 (L2), all weights 62 to 70 (some 45
// instructions a token), bins of light weights 85 (two shared-memory atomics a token).  Greedy
// 62 to 65 us (4.2 TB/s), top-k 127, min-p 113, none 197; top-p 0.9 at temperature 0.5 (the cut
// among the listed) 212 to 230, at 0.9 (some rows' cut among light tokens) 454, at 1.3 604; all kinds
// mixed 155 to 174, by the draw of the kinds.  Other rows, top-p 0.9 at 0.9: normal of sigma 4 363, of
// sigma 1 842, Laplace of scale 2 215, uniform over 20 628, all equal 6057 (atomics at one address).
#include <algorithm>
#include <cmath>

#include "fork_cache.cuh"

namespace fork {

namespace {

// Warps of a CTA.  16 where rows are few (clusters): the block-wide steps are shorter (5 rows of
// 32003, top-k: 17.7 / 23.9 us with 24 when both were timed); 24 where there are more rows than
// SMs, for the passes over the vocabulary (512 rows of 131072, no filter: 221 us; two CTAs of 12
// warps 225, and all kinds mixed 344 for 242; 32 warps 274).
constexpr int warps_of(bool cluster) { return cluster ? 16 : 24; }
constexpr int seg_of(int warps) { return warps == 16 ? 128 : 96; }  // survivors of one warp's run that fit in shared memory
constexpr int kFew = 256;            // survivors that are compared with one another instead of sorted by digits
constexpr int kUnroll = 4;      // maxima kept per thread
constexpr int kRing = 8;        // 16-byte vectors in flight per thread
constexpr int kRounds = 4;      // rounds of bins
constexpr int kBins = 256, kSlots = kBins + kBins / 8;  // (a gap every 8 bins: no bank conflicts where a lane reads 8)
constexpr int kDeep = 10;       // values in a lane's stack (a step adds 8)
constexpr int kMaxCluster = 8;
constexpr int kOrderedRows = 4096;
constexpr int kClusterPart = 8192;  // elements of a row per CTA of a cluster, at least
constexpr int kFrac = 44;       // fractional bits of a weight: 2^18 of them stay below 2^63
constexpr int kNone = 0x7fffffff;
constexpr float kLowest = -3.4028235e38f;
// A level that all light tokens are below: 30 of a weight's bits do (Row::light).  Where min-p
// compares single weights, further down.
constexpr float kLightOctaves = 5.1f, kLightOctavesMinP = 14.1f;
// What the first pass of top-p sorts into bins (131072 logits, normal with sigma 2 and some that
// stand out, temperature 1.3: 2% of the tokens; with 14 octaves 20%).
constexpr float kPickOctaves = 10.f;
constexpr float kNextOctaves = 24.f;  // and a second pass, where the cut lies further down

template <int kWarps>
struct SampleShared {
  static constexpr int kSeg = seg_of(kWarps), kCap = kWarps * kSeg;  // of a warp's run, of a row
  uint4 ring[kWarps][kRing][32];
  uint32_t tab_hi[64][32];  // 2^(j/64), rounded to 30 fractional bits, and its rest (14 more), once per lane (no bank conflicts)
  int tab_lo[64][32];
  uint32_t cnt[kSlots], lo[kSlots], hi[kSlots];
  uint64_t warp_sum[kWarps];
  float warp_max[kWarps];
  int warp_arg[kWarps], warp_cnt[kWarps];
  // read by the other CTAs of the cluster
  uint64_t rank_sum;
  float rank_max;
  int rank_arg, rank_cnt, rank_over;
  // one thread's findings for all
  uint64_t f_above, f_total, f_mass;
  int f_bin, f_cnt, f_idx;
  uint32_t f_cut;
  // heavy values that wait: stacks of the lanes and a line of as many (Row::masses), or a queue (Row::scan)
  float queue[kWarps][2 * 32 * kDeep];
  float lv[kWarps][kSeg];  // the warps' survivors
  int li[kWarps][kSeg];
  uint32_t few_key[kFew];
  uint64_t few_w[kFew];
  float fv[kCap];          // the row's, in index order (the first CTA of a cluster)
  int fi[kCap];
};

// 2^(j/64), 44 fractional bits (formed on the host)
struct SampleTable {
  uint64_t t[64];
};

struct SampleParams {
  const void* x;
  int64_t stride;
  int rows, V, ordered;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* token;
  float* prob;
};

__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
};
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
};

__device__ __forceinline__ float as_f(float x) { return x; }
__device__ __forceinline__ float as_f(uint16_t x) { return bf2f(x); }
// order-preserving bits (minus zero is zero)
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// the cluster: this CTA's rank, their number, a barrier, another CTA's shared memory
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
template <typename S>
__device__ __forceinline__ const S* of_rank(const S* p, int rank) {
  uint64_t a;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<const S*>(a);
}

// two float32 operations in one instruction, each rounded as by itself
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return (static_cast<uint64_t>(__float_as_uint(hi)) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ float low_of(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p)); }
__device__ __forceinline__ float high_of(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ int slot_of(int bin) { return bin + (bin >> 3); }

// total * x for a float x in [0, 1], rounded down or up: exact, by integers
__device__ __forceinline__ uint64_t part_of(uint64_t total, float x, bool up) {
  const uint32_t b = __float_as_uint(x);
  const int e = b >> 23;
  const uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int s = 150 - max(e, 1);  // x = m 2^-s, s >= 23
  const uint64_t lo = total * m, hi = __umul64hi(total, m);
  if (s >= 87) return up && m ? 1 : 0;  // total < 2^62, m < 2^24
  uint64_t q, rest;
  if (s >= 64) {
    q = hi >> (s - 64);
    rest = lo | (hi & ((1ull << (s - 64)) - 1));
  } else {
    q = (lo >> s) | (hi << (64 - s));
    rest = lo & ((1ull << s) - 1);
  }
  return q + (up && rest ? 1 : 0);
}
// a 2^-sh / b to one rounding: both as pairs of floats
__device__ __forceinline__ float quotient(uint64_t a, int sh, uint64_t b) {
  const float ah = __ull2float_rz(a), al = __ull2float_rn(a - static_cast<uint64_t>(ah));
  const float bh = __ull2float_rz(b), bl = __ull2float_rn(b - static_cast<uint64_t>(bh));
  const float q = ah / bh;
  const float r = (fmaf(-q, bh, ah) + al) - q * bl;
  return ldexpf(q + r / bh, -sh);
}

template <typename T, bool CL>
struct Row {
  static constexpr int N = Vec<T>::N;
  static constexpr int kWarps = warps_of(CL), kThreads = kWarps * 32;
  using Shared = SampleShared<kWarps>;
  static constexpr int kSeg = Shared::kSeg, kCap = Shared::kCap;
  Shared& s;
  const T* x;      // the row, from the 16-byte boundary at or before its first element
  int V, mis;      // mis: elements between that boundary and the row
  int rank, ranks;  // CTAs that work on the row together (one, once a CTA is left alone with the survivors)
  int first, last;  // this warp's 16-byte vectors
  int tid, warp, lane;
  bool endless;     // the largest logit is plus infinity: those count as 0, the others not at all
  float top;        // largest logit
  float none;       // a value whose weight rounds to zero, kLowest if there is none
  float light_c, light_rest;  // see light
  float heavy;      // tokens below weigh light (kLowest: none does)
  float ch, cl;     // log2(e) / temperature as a pair
  // what is left: at least thr, and past the cut: key above it, or equal with an index up to cut_idx
  float thr, below;  // below: upper end (not included) while a bracket is open
  uint32_t cut;
  int cut_idx;
  bool listed;
  int e0, e1, n_all;  // this warp's part of the survivors, and how many there are

  __device__ __forceinline__ void sync() {
    if (CL && ranks > 1) cluster_sync();
    else __syncthreads();
  }
  __device__ __forceinline__ const Shared* of(int r) const { return CL && ranks > 1 ? of_rank(&s, r) : &s; }

  // ---- the warp's run, in steps of 32 vectors of N elements: a ring of kRing of them per warp
  // in shared memory, filled by asynchronous copies.  A lane reads back what it asked for itself.
  // (The first pass over 131072 floats: 30 thousand cycles; with the vectors in registers, four in
  // flight and four on their way, 35.)
  __device__ __forceinline__ int steps_of_run() const { return (last - first + 31) / 32; }
  // vectors before it, but the row's first, lie inside the row
  __device__ __forceinline__ int inner() const { return endless ? 0 : min(last, (mis + V + N - 1) / N - 1); }
  __device__ __forceinline__ void ask(int it, int end) {
    const int v = first + it * 32 + lane;
    if (v > 0 && v < end)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(&s.ring[warp][it % kRing][lane]))),
                   "l"(reinterpret_cast<const uint4*>(x) + v)
                   : "memory");
  }
  // behind the requests of a group of U steps
  static __device__ __forceinline__ void close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // all but the last kRing / U - 1 groups are there
  template <int U>
  static __device__ __forceinline__ void await() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing / U - 1) : "memory");
  }
  template <int U>
  __device__ __forceinline__ void start(int end) {
#pragma unroll
    for (int it = 0; it < kRing; ++it) {
      ask(it, end);
      if (it % U == U - 1) close();
    }
  }
  // this lane's values of a step.  Elements outside the row and the run are minus infinity; NaN
  // stays NaN (no comparison holds for it).
  __device__ __forceinline__ void values(int it, int end, float* val) const {
    const int v = first + it * 32 + lane;
    const uint4 w = s.ring[warp][it % kRing][lane];
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int j = 0; j < N; ++j) val[j] = as_f(e[j]);
    if (!(v > 0 && v < end)) {  // the row's ends, element by element
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int i = v * N + j - mis;
        val[j] = v < last && i >= 0 && i < V ? as_f(x[v * N + j]) : -INFINITY;
        if (endless) val[j] = val[j] == INFINITY ? 0.f : -INFINITY;
      }
    }
  }
  // f(values, first index, slot) over the run, `slot` counting to kUnroll over and over
  template <typename F>
  __device__ __forceinline__ void run(F&& f) {
    constexpr int U = 2;
    const int its = steps_of_run(), end = inner();
    start<U>(end);
    for (int it0 = 0; it0 < its; it0 += kUnroll) {
#pragma unroll
      for (int g = 0; g < kUnroll; g += U) {
        const int it = it0 + g;
        if (it >= its) break;
        await<U>();
        float val[U][N];
#pragma unroll
        for (int k = 0; k < U; ++k) values(it + k, end, val[k]);
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (it + k < its) f(val[k], (first + (it + k) * 32 + lane) * N - mis, g + k);
#pragma unroll
        for (int k = 0; k < U; ++k) ask(it + kRing + k, end);
        close();
      }
    }
  }
  // The same with f(values, first index) written once (a long one), step by step; `step(it,
  // its)` after each.
  template <typename F, typename M>
  __device__ __forceinline__ void roll(F&& f, M&& step) {
    const int its = steps_of_run(), end = inner();
    start<1>(end);
#pragma unroll 1
    for (int it = 0; it < its; ++it) {
      await<1>();
      float val[N];
      values(it, end, val);
      f(val, (first + it * 32 + lane) * N - mis);
      ask(it + kRing, end);
      close();
      step(it, its);
    }
  }

  __device__ __forceinline__ bool alive(float v, int i) const {
    if (!(v >= thr && v < below)) return false;
    const uint32_t k = key_of(v);
    return k > cut || (k == cut && i <= cut_idx);
  }
  // a value at or below every v with (top - v) log2(e) / temperature <= octaves
  __device__ __forceinline__ float level(float octaves) const {
    const float d = octaves / ch;
    const float t = top - d - (fabsf(top) + d) * 1e-6f;
    return t > kLowest ? t : kLowest;
  }

  // e^((v - top) / t), 44 fractional bits.  Additions of a constant round to a fixed grid, so
  // that differences of the sums' bits are the integers (a conversion runs at a quarter of
  // the rate).
  __device__ __forceinline__ uint64_t weight(float v) const {
    int sh;
    const uint64_t w = mantissa(v, &sh);
    const bool any = sh > 0;
    return ((w >> (any ? sh - 1 : 0)) + (any ? 1 : 0)) >> (any ? 1 : 0);
  }
  // the same before its last shift: weight = result 2^-sh, result in [2^44, 2^45) or 0
  __device__ __forceinline__ uint64_t mantissa(float v, int* sh) const {
    // v - top exactly, as dh + dl
    const float dh = v - top, bb = dh - v;
    const float dl = (v - (dh - bb)) + (-top - bb);
    const float y0 = dh * ch;
    const bool some = y0 > -46.f;  // not for NaN, nor where the difference or the quotient overflowed
    const float yh = fmaxf(y0, -46.f);
    const float yl = some ? fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch) : 0.f;
    // y = m / 64 + r, |r| <= 2^-7
    const float t0 = yh + 196608.f;  // 1.5 * 2^17: a grid of 2^-6
    const int m = __float_as_int(t0) - 0x48400000;
    const float rf = yh - (t0 - 196608.f);
    const float rs = rf + yl, re = (rf - rs) + yl;
    // r with 37 fractional bits: 29 of them, then the rest
    const float t1 = rs + 0.0234375f;  // 1.5 * 2^-6: a grid of 2^-29
    const float rest = (rs - (t1 - 0.0234375f)) + re;
    const float t2 = rest + 9.1552734375e-5f;  // 1.5 * 2^-14: a grid of 2^-37
    const int rq = (__float_as_int(t1) - 0x3cc00000) * 256 + (__float_as_int(t2) - 0x38c00000);
    // 2^r - 1 with 36 fractional bits: r ln 2 in integers, the series' squares and above in float
    constexpr int kLn2 = 1488522236;  // ln 2 * 2^31
    const float c = rs * rs * fmaf(rs, fmaf(rs, 0.009618129f, 0.05550411f), 0.24022651f);
    const float t3 = c + 1.8310546875e-4f;  // 1.5 * 2^-13: a grid of 2^-36
    const int q = __mulhi(rq, kLn2) + (__float_as_int(t3) - 0x39400000);
    const uint32_t th = s.tab_hi[m & 63][lane];
    const uint64_t t = (static_cast<uint64_t>(th) << 14) + static_cast<int64_t>(s.tab_lo[m & 63][lane]);
    *sh = -(m >> 6);
    return some ? t + ((static_cast<int64_t>(static_cast<int>(th)) * q) >> 22) : 0;
  }

  // weight(v) for v from none (a value without weight) up to level(kLightOctaves), to 2^-29 of
  // itself (half a unit of 2^-30 from the table, 0.72 from the product's last bit, 0.7 from the
  // series): v log2(e) / t rounded to a grid of 2^-6 by an addition of light_c = 1.5 * 2^17 -
  // (top's own, on that grid), the rest by a product-sum that rounds once (2^-32), top's rest off.
  __device__ __forceinline__ uint64_t light(float v) const {
    const float t0 = fmaf(v, ch, light_c);
    const float r = fmaf(v, cl, fmaf(v, ch, light_c - t0)) - light_rest;
    uint32_t rest;
    const uint64_t w = light_of(__float_as_uint(t0), fmaf(r, fmaf(r, fmaf(r, fmaf(r, kL4, kL3), kL2), kL1), kL0), 0, &rest);
    return w + rest;
  }
  // q = (2^r - 1) 2^32, and what makes the rounding down of w's last bit one to nearest on average
  static constexpr float kL0 = 1.4427f, kL1 = 2977044472.f, kL2 = 1031764992.f, kL3 = 238388334.f, kL4 = 41309550.f;
  // t0: the grid point, in the low bits.  Returns `sum` plus the weight's bits from 2^-14 up, its others in `rest`.
  __device__ __forceinline__ uint64_t light_of(uint32_t t0, float q, uint64_t sum, uint32_t* rest) const {
    // (1.5 * 2^17 itself has none of the bits that are looked at)
    const int th = static_cast<int>(s.tab_hi[t0 & 63][lane]);
    int w;  // 30 fractional bits
    asm("mad.hi.s32 %0, %1, %2, %1;" : "=r"(w) : "r"(th), "r"(__float2int_rn(q)));
    // w 2^(14 - sh), -sh the grid point without its 6 fractional bits: for sh <= 14 a product
    // with 2^(14 - sh), for more the rounded upper half of one with 2^(46 - sh); a shift of 32
    // or more leaves nothing
    const uint32_t up = (t0 >> 6) - ((0x48400000u >> 6) - 46u);
    uint32_t lo, hi;
    asm("shl.b32 %0, 1, %1;" : "=r"(lo) : "r"(up));
    asm("shl.b32 %0, 1, %1;" : "=r"(hi) : "r"(up - 32u));
    const uint64_t r64 = static_cast<uint64_t>(static_cast<uint32_t>(w)) * lo + 0x80000000ull;
    *rest = static_cast<uint32_t>(r64 >> 32);
    return static_cast<uint64_t>(static_cast<uint32_t>(w)) * hi + sum;
  }
  // The weight of a token that can be drawn: one form, by its logit alone, for every sum and every
  // cut.  All sums are then sums of the same integers, and where a cut falls does not depend on
  // which of the passes below found it.
  __device__ __forceinline__ uint64_t mass(float v) const { return v < heavy ? light(fmaxf(v, none)) : weight(v); }
  // sum and four of them, two at a time in the float operations (the rests: below 2^30 each)
  __device__ __forceinline__ uint64_t light4(const float* v, uint64_t sum) const {
    const uint64_t c = pair(light_c, light_c), h = pair(ch, ch), l = pair(cl, cl), off = pair(-light_rest, -light_rest);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const uint64_t x2 = pair(v[j], v[j + 1]);
      const uint64_t t0 = fma2(x2, h, c);
      const uint64_t d = fma2(t0, pair(-1.f, -1.f), c);
      const uint64_t r = add2(fma2(x2, l, fma2(x2, h, d)), off);
      const uint64_t q = fma2(r, fma2(r, fma2(r, fma2(r, pair(kL4, kL4), pair(kL3, kL3)), pair(kL2, kL2)), pair(kL1, kL1)), pair(kL0, kL0));
      sum = light_of(static_cast<uint32_t>(t0), low_of(q), sum, &w[j]);
      sum = light_of(static_cast<uint32_t>(t0 >> 32), high_of(q), sum, &w[j + 1]);
    }
    return sum + (w[0] + w[1] + w[2] + w[3]);
  }

  // The weights of the warp's run, from `low` (not below `none`) up, where light weights exist:
  // light ones are added to `sum` in place, a heavy value counts there as one at `heavy`.  Values
  // from `pick` (at most heavy) up go, 32 at a time, to `dense(v, valid)`, which adds what is
  // missing.  Of values equal to low those past index `upto` do not count.  `seen(values, first
  // index)` gets every vector.
  template <typename F, typename O>
  __device__ __forceinline__ void masses(float low, int upto, float pick, uint64_t& sum, F&& dense, O&& seen) {
    constexpr int S = 8 / N;  // vectors of a lane in a step
    const int its = steps_of_run(), end = inner();
    const float above = from_key(key_of(low) + 1u);
    // picked values: a stack per lane; `drain` lines them up behind the stacks
    float* q = s.queue[warp];
    int n = 0;
    auto drain = [&] {
      int at = n;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, at, k);
        if (lane >= k) at += y;
      }
      const int all = __shfl_sync(0xffffffffu, at, 31);
      if (all == 0) return;
      at -= n;
      float* line = q + 32 * kDeep;
#pragma unroll 1
      for (int k = 0; k < n; ++k) line[at + k] = q[32 * k + lane];
      n = 0;
      __syncwarp();
#pragma unroll 1
      for (int e = 0; e < all; e += 32) dense(e + lane < all ? line[e + lane] : -INFINITY, e + lane < all);
      __syncwarp();
    };
    start<S>(end);
#pragma unroll 1
    for (int it = 0; it < its; it += S) {
      await<S>();
      float val[S * N];
#pragma unroll
      for (int k = 0; k < S; ++k) values(it + k, end, val + k * N);
      const int i0 = (first + it * 32) * N - mis;
#pragma unroll
      for (int k = 0; k < S; ++k) seen(val + k * N, i0 + (k * 32 + lane) * N);
      const bool before = i0 + S * 32 * N <= upto;  // all indices up to `upto`
      if (!before && i0 <= upto) {
#pragma unroll
        for (int e = 0; e < S * N; ++e)
          if (i0 + ((e / N) * 32 + lane) * N + e % N > upto && val[e] == low) val[e] = -INFINITY;
      }
      const float from = before || i0 <= upto ? low : above;
      float most = val[0];
#pragma unroll
      for (int j = 1; j < S * N; ++j) most = fmaxf(most, val[j]);
#pragma unroll
      for (int j = 0; j < S * N; j += 4) {
        float c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = fminf(val[j + e] >= from ? val[j + e] : none, heavy);
        sum = light4(c, sum);
      }
      if (most >= pick) {
#pragma unroll
        for (int j = 0; j < S * N; ++j)
          if (val[j] >= pick) q[32 * n++ + lane] = val[j];
      }
#pragma unroll
      for (int k = 0; k < S; ++k) ask(it + kRing + k, end);
      close();
      if (__any_sync(0xffffffffu, n > kDeep - S * N)) drain();
    }
    drain();
  }

  // One pass over the warp's run of the row.  The values that `take(v, i)` picks go, 32 at a
  // time, one per lane, to `dense(v, valid)`; `other(values, i)` sees every vector.
  template <typename P, typename O, typename F>
  __device__ __forceinline__ void scan(P&& take, O&& other, F&& dense) {
    float* q = s.queue[warp];
    int n = 0;
    roll(
        [&](const float* v, int i) {
          other(v, i);
          bool t[N], any = false;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            t[j] = take(v[j], i + j);
            any = any || t[j];
          }
          if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const uint32_t m = __ballot_sync(0xffffffffu, t[j]);
            if (t[j]) q[n + __popc(m & ((1u << lane) - 1u))] = v[j];
            n += __popc(m);
          }
        },
        [&](int it, int its) {
          // full warps' worth, from the end; the rest after the last step
          __syncwarp();
#pragma unroll 1
          while (n >= 32 || (it + 1 == its && n > 0)) {
            const int from = max(n - 32, 0);
            const float x = lane < n - from ? q[from + lane] : -INFINITY;
            dense(x, lane < n - from);
            n = from;
          }
          __syncwarp();
        });
  }

  // ---- the survivors: this warp's part of the list, or its run of the row
  template <typename F>
  __device__ __forceinline__ void each(F&& f) {
    if (listed) {
      for (int e = e0 + lane; e < e1; e += 32) {
        const float v = s.fv[e];
        const int i = s.fi[e];
        if (alive(v, i)) f(v, i);
      }
    } else {
      run(
          [&](const float* v, int i, int) {
#pragma unroll 1
            for (int j = 0; j < N; ++j)
              if (alive(v[j], i + j)) f(v[j], i + j);
          });
    }
  }

  __device__ __forceinline__ void zero_bins() {
    for (int e = tid; e < kSlots; e += kThreads) s.cnt[e] = s.lo[e] = s.hi[e] = 0;
    __syncthreads();
  }
  __device__ __forceinline__ void add_mass(int b, uint64_t w) {
    const uint32_t l = static_cast<uint32_t>(w);
    const uint32_t was = atomicAdd(&s.lo[slot_of(b)], l);
    atomicAdd(&s.hi[slot_of(b)], static_cast<uint32_t>(w >> 32) + (was + l < l ? 1u : 0u));
  }
  // The bins of all CTAs, from the last down or from the first up: the bin at which the running
  // total reaches `want`.  Leaves the bin, the total before it and its own count in s (f_bin
  // -1: the total of all bins is below `want`).
  template <bool MASS>
  __device__ __forceinline__ void find(bool down, uint64_t want) {
    sync();
    if (warp == 0) {
      uint64_t v[kBins / 32];
      uint32_t n[kBins / 32];
      uint64_t mine = 0;
#pragma unroll
      for (int k = 0; k < kBins / 32; ++k) {
        v[k] = 0;
        n[k] = 0;
      }
      for (int r = 0; r < ranks; ++r) {
        const Shared* o = of(r);
#pragma unroll
        for (int k = 0; k < kBins / 32; ++k) {
          const int at = lane * (kBins / 32) + k, b = down ? kBins - 1 - at : at;
          n[k] += o->cnt[slot_of(b)];
          if (MASS) v[k] += (static_cast<uint64_t>(o->hi[slot_of(b)]) << 32) + o->lo[slot_of(b)];
        }
      }
#pragma unroll
      for (int k = 0; k < kBins / 32; ++k) {
        if (!MASS) v[k] = n[k];
        mine += v[k];
      }
      uint64_t x = mine;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, k);
        if (lane >= k) x += y;
      }
      uint64_t before = x - mine;
      const uint64_t all = __shfl_sync(0xffffffffu, x, 31);
      if (lane == 0) {
        s.f_total = all;
        if (all < want) s.f_bin = -1;
      }
      if (before < want && want <= x) {
#pragma unroll
        for (int k = 0; k < kBins / 32; ++k) {
          if (before < want && want <= before + v[k]) {
            const int at = lane * (kBins / 32) + k;
            s.f_bin = down ? kBins - 1 - at : at;
            s.f_above = before;
            s.f_cnt = static_cast<int>(n[k]);
            s.f_mass = v[k];
          }
          before += v[k];
        }
      }
    }
    sync();  // nobody clears its bins before all have read them
  }

  // The cut among the survivors: the key at which the running count (or mass) from the
  // largest key down reaches `want`, and of its ties in index order how many are kept.
  template <bool MASS>
  __device__ __forceinline__ void select(uint64_t want) {
    if (listed && n_all <= kFew) {
      // few: a thread sums what comes before its own (the list is in index order)
      __syncthreads();
      if (tid == 0) s.f_bin = -1;
      const bool mine = tid < n_all && alive(s.fv[min(tid, kCap - 1)], s.fi[min(tid, kCap - 1)]);
      if (tid < n_all) {
        s.few_key[tid] = mine ? key_of(s.fv[tid]) : 0;
        if (MASS) s.few_w[tid] = mine ? mass(s.fv[tid]) : 0;
      }
      __syncthreads();
      if (mine) {
        const uint32_t k = s.few_key[tid];
        uint64_t before = 0;
#pragma unroll 4
        for (int j = 0; j < n_all; ++j) {
          const uint32_t kj = s.few_key[j];
          const uint64_t w = MASS ? s.few_w[j] : 1;
          if (kj > k || (kj == k && j < tid)) before += w;
        }
        const uint64_t own = MASS ? s.few_w[tid] : 1;
        if (before < want && want <= before + own) {
          s.f_bin = 0;
          s.f_cut = k;
          s.f_idx = s.fi[tid];
        }
      }
      __syncthreads();
      if (s.f_bin >= 0) {
        cut = s.f_cut;
        cut_idx = s.f_idx;
      }
      __syncthreads();
      return;
    }
    uint32_t prefix = 0, mask = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      zero_bins();
      each([&](float v, int) {
        const uint32_t k = key_of(v);
        if ((k & mask) != prefix) return;
        const int b = (k >> shift) & 255;
        atomicAdd(&s.cnt[slot_of(b)], 1u);
        if (MASS) add_mass(b, mass(v));
      });
      find<MASS>(true, want);
      if (s.f_bin < 0) return;  // all of them together stay below `want`: no cut
      want -= s.f_above;
      prefix |= static_cast<uint32_t>(s.f_bin) << shift;
      mask |= 255u << shift;
    }
    const int ties = s.f_cnt;
    uint64_t quota = want;
    if (MASS) {
      const uint64_t w = mass(from_key(prefix));
      quota = (want + w - 1) / w;
    }
    const int idx = quota >= static_cast<uint64_t>(ties) ? kNone : nth_tie(prefix, static_cast<int>(quota));
    cut_idx = prefix == cut ? min(idx, cut_idx) : idx;
    cut = prefix;
  }

  // Sum of v over the lower CTAs (v the same in all threads of a CTA, handed over in `slot`)
  template <typename I>
  __device__ __forceinline__ I lower(I Shared::*slot, I v, I* all) {
    if (!CL || ranks == 1) {
      *all = v;
      return 0;
    }
    __syncthreads();
    if (tid == 0) s.*slot = v;
    sync();
    I before = 0, total = 0;
    for (int r = 0; r < ranks; ++r) {
      const I y = of(r)->*slot;
      if (r < rank) before += y;
      total += y;
    }
    sync();
    *all = total;
    return before;
  }

  // Index of the quota-th survivor with this key, in index order.
  __device__ __forceinline__ int nth_tie(uint32_t key, int quota) {
    int n = 0;
    each([&](float v, int) { n += key_of(v) == key; });
    for (int k = 16; k > 0; k >>= 1) n += __shfl_xor_sync(0xffffffffu, n, k);
    __syncthreads();
    if (lane == 0) s.warp_cnt[warp] = n;
    if (tid == 0) s.f_idx = kNone;
    __syncthreads();
    int mine = 0, before = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s.warp_cnt[w];
      mine += s.warp_cnt[w];
    }
    int all;
    before += lower(&Shared::rank_cnt, mine, &all);
    if (before < quota && quota <= before + n) {
      int left = quota - before;  // in this warp's run
      if (listed) {
        for (int e = e0; e < e1; e += 32) {  // one element per lane, lanes in index order
          const bool in = e + lane < e1;
          const float v = in ? s.fv[e + lane] : -INFINITY;
          const int i = in ? s.fi[e + lane] : 0;
          const bool tie = in && alive(v, i) && key_of(v) == key;
          const uint32_t m = __ballot_sync(0xffffffffu, tie);
          if (tie && __popc(m & ((2u << lane) - 1u)) == left) s.f_idx = i;
          left -= __popc(m);
        }
      } else {
        run(
            [&](const float* v, int i, int) {
              int c = 0;
              for (int j = 0; j < N; ++j) c += alive(v[j], i + j) && key_of(v[j]) == key;
              int x = c;
              for (int k = 1; k < 32; k <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, k);
                if (lane >= k) x += y;
              }
              int at = x - c;
              for (int j = 0; j < N; ++j)
                if (alive(v[j], i + j) && key_of(v[j]) == key && ++at == left) s.f_idx = i + j;
              left -= __shfl_sync(0xffffffffu, x, 31);
            });
      }
    }
    sync();
    int idx = kNone;
    for (int r = 0; r < ranks; ++r) idx = min(idx, of(r)->f_idx);
    sync();
    return idx;
  }

  // What lies in [thr, below) of a vector per lane, in index order, to this warp's list behind its
  // first n entries
  __device__ __forceinline__ void note(const float* v, int i, int& n) {
    if (n > kSeg) return;  // (too many for the list already)
    int c = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) c += v[j] >= thr && v[j] < below;
    if (!__any_sync(0xffffffffu, c)) return;
    int x = c;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, k);
      if (lane >= k) x += y;
    }
    int at = n + x - c;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (v[j] >= thr && v[j] < below) {
        if (at < kSeg) {
          s.lv[warp][at] = v[j];
          s.li[warp][at] = i + j;
        }
        ++at;
      }
    n += __shfl_sync(0xffffffffu, x, 31);
  }
  __device__ __forceinline__ void compact() {
    int n = 0;
    run([&](const float* v, int i, int) { note(v, i, n); });
    gather(n);
  }
  // The warps' lists, n entries in this one's, to the list of the first CTA, if they fit.  Leaves
  // `listed`, and the warps' parts of the list in the first CTA.
  __device__ __forceinline__ void gather(int n) {
    if (lane == 0) s.warp_cnt[warp] = n;
    int over = __syncthreads_or(n > kSeg);
    int mine = 0, before = 0, total;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s.warp_cnt[w];
      mine += s.warp_cnt[w];
    }
    total = mine;
    if (CL && ranks > 1) {
      if (tid == 0) {
        s.rank_cnt = mine;
        s.rank_over = over;
      }
      sync();
      total = 0;
      for (int r = 0; r < ranks; ++r) {
        const Shared* o = of(r);
        const int y = o->rank_cnt;
        if (r < rank) before += y;
        total += y;
        over |= o->rank_over;
      }
    }
    // one form for the whole cluster: its CTAs meet equally often
    listed = !over && total <= kCap;
    if (listed) {
      Shared* to = const_cast<Shared*>(of(0));
      for (int e = lane; e < n; e += 32) {
        to->fv[before + e] = s.lv[warp][e];
        to->fi[before + e] = s.li[warp][e];
      }
    }
    sync();
    n_all = total;
    const int per = ((total + kWarps - 1) / kWarps + 31) & ~31;
    e0 = min(warp * per, total);
    e1 = min(e0 + per, total);
  }

  // Brackets around the cut, the token at which the running mass (or count) from the largest
  // logit down reaches `want`: ends with [thr, below) and `want` less what lies above it.  The
  // first pass sorts the picked tokens (for counts, those within 32 of the maximum) into bins of
  // their logits; for top-p it also sums the row's mass, from which `want` follows, and, if they
  // are said to be few, lists them: where they fit and the cut is one of them, `listed` is set and
  // `want` counts from the top.
  template <bool MASS>
  __device__ __forceinline__ void narrow(uint64_t* want, float keep, float pick, bool few) {
    float lo = MASS ? fmaxf(pick, level(46.5f)) : fmaxf(top - 32.f, kLowest), hi = top;
    const float least = MASS ? level(46.5f) : kLowest;  // no weight below
    uint64_t sum = 0;
    int n = few ? 0 : kSeg + 1;  // entries of this warp's list
    bool refined = false;        // inside a bin
    for (int round = 0;; ++round) {
      const float scale = fminf(kBins / (hi - lo), 1e30f);
      auto bin = [&](float v) { return static_cast<int>(fminf((v - lo) * scale, kBins - 1.f)); };
      const bool whole = MASS && round == 0;
      const bool uncounted = MASS && !whole && heavy > kLowest && hi <= pick && !refined;
      zero_bins();
      const uint64_t counted = MASS && heavy > kLowest ? light(heavy) : 0;  // (of a heavy token, in place)
      auto dense = [&](float v, bool valid) {
        if (!valid) return;
        atomicAdd(&s.cnt[slot_of(bin(v))], 1u);
        if (MASS) {
          uint64_t w;
          if (v < heavy) {
            w = light(fmaxf(v, none));
          } else {
            w = weight(v);
            sum += w - counted;
          }
          add_mass(bin(v), w);
        }
      };
      auto take = [&](float v, int) { return v >= lo && v < below; };
      if (whole && heavy > kLowest) {
        // the picked ones in a list too: mostly the cut is among them
        thr = pick;
        masses(none, kNone, pick, sum, dense, [&](const float* v, int i) { note(v, i, n); });
      } else if (uncounted) {
        // All light tokens, too many for a queue to gain anything.  Sums in 16 copies, a lane's by its
        // number (two lanes meet at most), in two words that need no carry: weights below 2^34 in
        // halves of 17 bits, at most 2^14 + 2 N kWarps of them in a copy.  How many tokens a bin has
        // follows from its mass.  (64 rows of 131072 bf16, top-p 0.9: 89 us; in one copy, with carries
        // and counts, 94.)
        uint32_t* h = reinterpret_cast<uint32_t*>(s.queue);
        static_assert(sizeof(s.queue) >= 2 * 16 * kBins * sizeof(uint32_t), "the copies fit in the queues");
        for (int e = tid; e < 2 * 16 * kBins; e += kThreads) h[e] = 0;
        __syncthreads();
        roll(
            [&](const float* v, int) {
#pragma unroll
              for (int j = 0; j < N; ++j) {
                const uint64_t w = light(fmaxf(v[j], none));
                if (!take(v[j], 0)) continue;
                uint32_t* to = h + bin(v[j]) * 16 + (lane & 15);
                atomicAdd(to, static_cast<uint32_t>(w) & 0x1ffffu);
                atomicAdd(to + 16 * kBins, static_cast<uint32_t>(w >> 17));
              }
            },
            [](int, int) {});
        __syncthreads();
        for (int e = tid; e < kBins; e += kThreads) {
          uint64_t lo17 = 0, hi17 = 0;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            lo17 += h[e * 16 + (k + e) % 16];
            hi17 += h[16 * kBins + e * 16 + (k + e) % 16];
          }
          const uint64_t w = lo17 + (hi17 << 17);
          s.lo[slot_of(e)] = static_cast<uint32_t>(w);
          s.hi[slot_of(e)] = static_cast<uint32_t>(w >> 32);
        }
      } else {
        scan(take, [](const float*, int) {}, dense);
      }
      if (whole) {
        for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        __syncthreads();
        if (lane == 0) s.warp_sum[warp] = sum;
        __syncthreads();
        sum = 0;
        for (int w = 0; w < kWarps; ++w) sum += s.warp_sum[w];
        uint64_t total;
        lower(&Shared::rank_sum, sum, &total);
        *want = max(part_of(total, keep, true), static_cast<uint64_t>(1));
      }
      find<MASS>(true, *want);
      const int b = s.f_bin;
      if (whole && heavy > kLowest) {
        gather(n);
        if (listed && b >= 0) return;
        listed = false;
        thr = kLowest;
      }
      if (b < 0) {  // further down than the bins: the next part of the row
        if (refined || lo <= least) return;
        *want -= s.f_total;
        below = hi = lo;
        lo = MASS && round == 0 ? fmaxf(least, fminf(level(kNextOctaves), lo)) : least;
        if (!MASS) return;  // (no scale to bin it by)
        continue;
      }
      refined = true;
      if (bin(hi) != kBins - 1) return;  // a single value, or neighbours that no bins tell apart
      // the values of bin b: [first with bin b, first with bin b + 1), by bisection of their keys
      auto first_of = [&](int bb) {
        uint32_t a = key_of(lo), z = key_of(hi);  // bin(a) < bb <= bin of z or beyond
        while (z - a > 1) {
          const uint32_t m = a + (z - a) / 2;
          if (bin(from_key(m)) >= bb) z = m;
          else a = m;
        }
        return from_key(z);
      };
      const float t = b > 0 ? first_of(b) : lo, u = b + 1 < kBins ? first_of(b + 1) : below;
      const bool same = t == thr && u == below;
      const uint64_t n_bin = uncounted ? s.f_mass / max(light(fmaxf(t, none)), static_cast<uint64_t>(1)) : s.f_cnt;  // (at most this many)
      *want -= s.f_above;
      thr = t;
      below = u;
      if (n_bin <= kCap / 2 || same || round == kRounds) return;  // few enough for the list, or nothing gained
      lo = thr;
      hi = below < INFINITY ? below : top;
    }
  }
};

// Rows that take long come first, so that the last CTAs to start have little to do: top-p over
// the whole vocabulary, then every token drawn from, then the rest.  Every CTA sorts for itself
// (one read of the parameters).
template <int kWarps>
__device__ __forceinline__ int ordered_row(const SampleParams& p, SampleShared<kWarps>& s, int at) {
  constexpr int kThreads = kWarps * 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto kind = [&](int r) {
    if (r >= p.rows) return 3;
    const float t = p.temperature ? p.temperature[r] : 1.f;
    const int k = p.top_k ? p.top_k[r] : 0;
    if (!(t > 0.f) || (k > 0 && k < p.V)) return 2;
    if (p.top_p && p.top_p[r] < 1.f) return 0;
    return p.min_p && p.min_p[r] > 0.f ? 2 : 1;
  };
  for (int want = 0; want < 3; ++want)
    for (int base = 0; base < p.rows; base += kThreads) {
      const bool is = kind(base + tid) == want;
      const uint32_t m = __ballot_sync(0xffffffffu, is);
      __syncthreads();
      if (lane == 0) s.warp_cnt[warp] = __popc(m);
      __syncthreads();
      int before = 0, all = 0;
      for (int w = 0; w < kWarps; ++w) {
        const int c = s.warp_cnt[w];
        if (w < warp) before += c;
        all += c;
      }
      if (at < all) {
        if (is && before + __popc(m & ((1u << lane) - 1u)) == at) s.f_idx = base + tid;
        __syncthreads();
        return s.f_idx;
      }
      at -= all;
    }
  return 0;  // (not reached: every row has a kind)
}

template <typename T, bool CL>
__global__ void __launch_bounds__(warps_of(CL) * 32, 1)
    sample_kernel(const __grid_constant__ SampleParams p, const __grid_constant__ SampleTable table) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using R = Row<T, CL>;
  constexpr int N = R::N, kWarps = R::kWarps, kThreads = R::kThreads, kCap = R::kCap;
  typename R::Shared& s = *reinterpret_cast<typename R::Shared*>(smem_raw);
  const int ranks = CL ? cluster_size() : 1;
  const int rank = CL ? cluster_rank() : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  const int row = p.ordered ? ordered_row(p, s, blockIdx.x) : (CL ? blockIdx.x / ranks : blockIdx.x);
  const T* x0 = static_cast<const T*>(p.x) + row * p.stride;
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(x0) & 15u) / sizeof(T));
  const int nvec = (mis + p.V + N - 1) / N;
  const int part = rank * kWarps + warp, parts = ranks * kWarps;
  R r{s, x0 - mis, p.V, mis, rank, ranks,
      static_cast<int>(static_cast<int64_t>(nvec) * part / parts), static_cast<int>(static_cast<int64_t>(nvec) * (part + 1) / parts),
      tid, warp, lane, false, 0.f, 0.f, 0.f, 0.f, kLowest, 0.f, 0.f, kLowest, INFINITY, 0u, kNone, false, 0, 0, 0};
  for (int e = tid; e < 64 * 32; e += kThreads) {
    const uint64_t t = table.t[e >> 5];
    const uint32_t hi = static_cast<uint32_t>((t + 0x2000u) >> 14);
    s.tab_hi[e >> 5][e & 31] = hi;
    s.tab_lo[e >> 5][e & 31] = static_cast<int>(static_cast<int64_t>(t) - (static_cast<int64_t>(hi) << 14));
  }

  const float temp = p.temperature ? p.temperature[row] : 1.f;
  const int k = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  float min_p = p.min_p ? p.min_p[row] : 0.f;
  const float u = p.u[row];
  const bool greedy = !(temp > 0.f);

  // ---- the largest logit; a thread keeps one maximum per slot, and the vector of its own
  float best[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) best[j] = -INFINITY;
  float most = -INFINITY;
  int where = kNone;  // first index of the first vector that holds `most`
  r.run(
      [&](const float* v, int i, int slot) {
        float m = v[0];
#pragma unroll
        for (int j = 1; j < N; ++j) m = fmaxf(m, v[j]);
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
          if (j == slot) best[j] = fmaxf(best[j], m);
        if (m > most) {
          most = m;
          where = i;
        }
      });
  {
    float b = most;
    int a = where;
    if (greedy && b > -INFINITY) {  // its index within the vector
      for (int j = N - 1; j >= 0; --j) {
        const int i = where + j;
        if (i >= 0 && i < p.V && as_f(x0[i]) == b) a = i;
      }
    }
    auto take = [&](float b2, int a2) {
      if (b2 > b || (b2 == b && a2 < a)) {
        b = b2;
        a = a2;
      }
    };
    for (int m = 16; m > 0; m >>= 1) take(__shfl_xor_sync(0xffffffffu, b, m), __shfl_xor_sync(0xffffffffu, a, m));
    if (lane == 0) {
      s.warp_max[warp] = b;
      s.warp_arg[warp] = a;
    }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) take(s.warp_max[w], s.warp_arg[w]);
    if (CL) {
      if (tid == 0) {
        s.rank_max = b;
        s.rank_arg = a;
      }
      r.sync();
      for (int q = 0; q < ranks; ++q) take(r.of(q)->rank_max, r.of(q)->rank_arg);
      r.sync();
    }
    r.top = b;
    if (b == -INFINITY || greedy) {  // nothing to draw, or nothing to draw by
      if (rank == 0 && tid == 0) {
        p.token[row] = b == -INFINITY ? -1 : a;
        if (p.prob) p.prob[row] = b == -INFINITY ? 0.f : 1.f;
      }
      return;
    }
  }
  if (r.top == INFINITY) {
    r.endless = true;
    r.top = 0.f;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) best[j] = best[j] == INFINITY ? 0.f : -INFINITY;
  }
  // log2(e) / temperature as a pair (log2(e) itself is 1.442695f + 1.925963e-8f)
  r.ch = fminf(1.44269502f / temp, 3e38f);
  r.cl = r.ch < 3e38f ? (fmaf(-r.ch, temp, 1.44269502f) + 1.92596299e-8f) / temp : 0.f;
  if (!(fabsf(r.cl) < r.ch)) r.cl = 0.f;
  // light tokens: from 2^-45.9 (nothing is left of less) to 2^-5.1, where the logits are not so
  // large that their grid is coarser than the light form's
  r.none = r.level(45.9f);
  const float top2 = r.top * r.ch, reach = fmaxf(fabsf(r.top), fabsf(r.none)) * r.ch;
  const bool lights = r.none > kLowest && reach < 16384.f;
  const float heavy = r.heavy = lights ? r.level(p.min_p && min_p > 0.f ? kLightOctavesMinP : kLightOctaves) : kLowest;
  const float pick = lights ? fminf(heavy, r.level(kPickOctaves)) : kLowest;
  {
    const float grid = rintf(top2 * 64.f) * 0.015625f;
    r.light_c = 196608.f - grid;
    r.light_rest = (top2 - grid) + fmaf(r.top, r.ch, -top2) + r.top * r.cl;
  }
  min_p = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;
  const bool use_k = k > 0 && k < p.V, use_p = top_p < 1.f;
  const float keep = fmaxf(top_p, 0.f);

  // ---- narrow what can be drawn, then cut it exactly.  A cut found in a list that does not
  // reach up to the maximum (a bracket) goes back to the whole row.
  uint64_t kept_sum = 0;  // of the lane: what is kept of the run, where a pass has already summed it
  int noted = -1;         // entries of the warp's own list then
  auto cut_of = [&](bool mass, uint64_t want) {
    if (mass && !r.listed && lights && min_p == 0.f && r.below <= heavy) {
      // all tokens from `below` up are kept: their sum in the same pass
      int n = 0;
      const uint64_t counted = r.light(heavy);
      r.masses(r.below, kNone, heavy, kept_sum, [&](float v, bool valid) {
        if (valid) kept_sum += r.weight(v) - counted;
      }, [&](const float* v, int i) { r.note(v, i, n); });
      r.gather(n);
      if (r.listed) noted = n;
    } else if (!r.listed) {
      r.compact();
    }
    const bool bracket = r.below < INFINITY, shared = r.listed;
    if (!shared || rank == 0) {
      const int with = r.ranks;
      if (shared) r.ranks = 1;
      if (mass) r.template select<true>(want);
      else r.template select<false>(want);
      r.ranks = with;
    }
    r.below = INFINITY;
    if (shared && bracket) {
      r.listed = false;
      if (CL && r.ranks > 1) {
        if (tid == 0) {
          s.f_cut = r.cut;
          s.f_idx = r.cut_idx;
        }
        r.sync();
        r.cut = r.of(0)->f_cut;
        r.cut_idx = r.of(0)->f_idx;
        r.sync();
      }
      return true;
    }
    if (shared) {
      r.ranks = 1;
      return rank == 0;  // the first CTA goes on alone
    }
    return true;
  };
  if (use_k) {
    // k of the parts' maxima lie above a bound, so k tokens do
    r.zero_bins();
    auto bin = [&](float v) { return static_cast<int>(fminf((r.top - v) * 8.f, kBins - 1.f)); };
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (best[j] > -INFINITY) atomicAdd(&s.cnt[slot_of(bin(best[j]))], 1u);
    r.template find<false>(false, k);
    uint64_t want = k;
    if (s.f_bin >= 0 && s.f_bin < kBins - 1 && k <= kCap / 2) {
      const float d = (s.f_bin + 1) * 0.125f;
      r.thr = fmaxf(r.top - d - (fabsf(r.top) + d) * 1e-6f, kLowest);
    } else {
      r.template narrow<false>(&want, 0.f, kLowest, false);
    }
    // (without effect when fewer than k tokens are above minus infinity)
    if (!cut_of(false, want)) return;
    if (use_p) {
      uint64_t sum = 0, total;
      r.each([&](float v, int) { sum += r.mass(v); });
      for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      __syncthreads();
      if (lane == 0) s.warp_sum[warp] = sum;
      __syncthreads();
      sum = 0;
      for (int w = 0; w < kWarps; ++w) sum += s.warp_sum[w];
      r.lower(&R::Shared::rank_sum, sum, &total);
      r.template select<true>(max(part_of(total, keep, true), static_cast<uint64_t>(1)));
    }
  } else if (use_p) {
    uint64_t want = 0;
    // few tokens to pick where few threads have met one (512 rows of 131072 at temperature 0.5:
    // 278 us, with the list 250; at 1.3 600, and 640 when it is tried in vain)
    bool met = false;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) met = met || best[j] >= pick;
    const bool few = __syncthreads_count(met) <= kThreads / 3;
    r.template narrow<true>(&want, keep, pick, few);
    if (!cut_of(true, want)) return;
  } else if (min_p > 0.f) {
    r.thr = r.level(0.01f - log2f(min_p));
    r.compact();
    if (r.listed) {
      if (rank != 0) return;
      r.ranks = 1;
    }
  }

  // ---- draw: sums in index order
  const uint64_t floor_w = min_p > 0.f ? part_of(1ull << kFrac, min_p, true) : 0;
  const bool all = !use_k && !use_p && min_p == 0.f;  // every token can be drawn
  auto kept = [&](float v, int i) { return all ? v > -INFINITY : r.alive(v, i); };
  auto weigh = [&](float v) -> uint64_t {
    const uint64_t w = r.mass(v);
    return w >= floor_w ? w : 0;
  };
  uint64_t before = 0, left = 0, total = 0;
  const float least = r.cut ? fmaxf(r.thr, from_key(r.cut)) : r.thr;
  // a warp's sum over its part of the list or its run; then, unless its share is short, the same
  // over its share of the one run that holds the draw
  const int whole = (nvec + parts - 1) / parts;
  uint64_t sum;
  for (int round = 0;; ++round) {
    sum = 0;
    auto dense = [&](float v, bool valid) {
      if (valid) sum += weigh(v);
    };
    if (r.listed) {
      for (int e = r.e0 + lane; e < r.e1; e += 32)
        if (kept(s.fv[e], s.fi[e])) sum += weigh(s.fv[e]);
    } else if (round == 0 && noted >= 0) {
      sum = kept_sum;
      for (int e = lane; e < noted; e += 32)
        if (kept(s.lv[warp][e], s.li[warp][e])) sum += weigh(s.lv[warp][e]);
    } else if (min_p == 0.f && least < heavy) {
      const uint64_t counted = r.light(heavy);
      r.masses(fmaxf(least, r.none), r.cut && least == from_key(r.cut) ? r.cut_idx : kNone, heavy, sum, [&](float v, bool valid) {
        if (valid) sum += r.weight(v) - counted;
      }, [](const float*, int) {});
    } else {
      r.scan([&](float v, int i) { return v >= heavy && kept(v, i); },
             [&](const float* v, int i) {
               bool any = false;
#pragma unroll
               for (int j = 0; j < N; ++j) any = any || (v[j] >= r.thr && v[j] < heavy);
               if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
               for (int j = 0; j < N; ++j) {
                 const uint64_t w = r.light(v[j] < heavy ? fmaxf(v[j], r.none) : r.none);
                 if (v[j] < heavy && w >= floor_w && kept(v[j], i + j)) sum += w;
               }
             },
             dense);
    }
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = sum;
    __syncthreads();
    uint64_t mine = 0;
    for (int w = 0; w < kWarps; ++w) mine += s.warp_sum[w];
    if (round == 0) {
      before = r.lower(&R::Shared::rank_sum, mine, &total);
      // first token whose cumulative weight exceeds u * total (floor: both sides are integers)
      uint64_t target = u > 0.f ? part_of(total, fminf(u, 1.f), false) : 0;
      if (target >= total) target = total - 1;
      if (target < before || target - before >= mine) return;  // not in this CTA's part
      left = target - before;
    }
    int w = 0;
    uint64_t up_to = 0, below = 0;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      up_to += s.warp_sum[q];
      if (left >= up_to) {
        w = q + 1;
        below = up_to;
      }
    }
    left -= below;
    if (round == 1 || r.listed || whole <= 128) {
      if (w != warp) return;
      break;
    }
    const int64_t at = rank * kWarps + w;
    const int f0 = static_cast<int>(nvec * at / parts), n = static_cast<int>(nvec * (at + 1) / parts) - f0;
    r.first = f0 + n * warp / kWarps;
    r.last = f0 + n * (warp + 1) / kWarps;
    __syncthreads();
  }
  bool done = false;
  auto hit = [&](float v, int i) {
    p.token[row] = i;
    if (!p.prob) return;
    int sh;
    const uint64_t w = r.mantissa(v, &sh);
    p.prob[row] = quotient(w, sh, total);
  };
  if (r.listed) {
    for (int e = r.e0; e < r.e1 && !done; e += 32) {
      const float v = e + lane < r.e1 ? s.fv[e + lane] : -INFINITY;
      const int i = e + lane < r.e1 ? s.fi[e + lane] : 0;
      const uint64_t w = kept(v, i) ? weigh(v) : 0;
      uint64_t x = w;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x += y;
      }
      if (w && x - w <= left && left < x) hit(v, i);
      const uint64_t all32 = __shfl_sync(0xffffffffu, x, 31);
      done = left < all32;
      left -= done ? 0 : all32;
    }
    return;
  }
  // the vectors of the warp's share one by one
  const int first = r.first, last = r.last;
  for (int from = first; from < last && !done; from += 32) {
    r.first = from;
    r.last = min(last, from + 32);
    r.run(
        [&](const float* v, int i, int) {
          uint64_t w[N], mine1 = 0;
#pragma unroll
          for (int j = 0; j < N; ++j) mine1 += w[j] = kept(v[j], i + j) ? weigh(v[j]) : 0;
          uint64_t x = mine1;
#pragma unroll
          for (int m = 1; m < 32; m <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, x, m);
            if (lane >= m) x += y;
          }
          uint64_t at = x - mine1;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            if (w[j] && at <= left && left < at + w[j]) hit(v[j], i + j);
            at += w[j];
          }
          const uint64_t all32 = __shfl_sync(0xffffffffu, x, 31);
          done = left < all32;
          left -= done ? 0 : all32;
        });
  }
}

template <typename T>
int launch_sample(const SampleParams& p, cudaStream_t s) {
  // a cluster per row while there are SMs to spare and a part stays long enough to be worth it
  int cs = 1;
  while (cs < kMaxCluster && static_cast<int64_t>(p.rows) * cs * 2 <= sm_count() && p.V / (cs * 2) >= kClusterPart) cs *= 2;
  const bool many = p.rows > sm_count();
  // more rows than SMs, and not so many that sorting them would cost more than the last ones do
  SampleParams q = p;
  q.ordered = many && p.rows <= kOrderedRows;
  auto kern = many ? sample_kernel<T, false> : sample_kernel<T, true>;
  static_assert(sizeof(SampleShared<warps_of(false)>) <= 227 * 1024 && sizeof(SampleShared<warps_of(true)>) <= 227 * 1024, "shared memory of a CTA");
  const size_t smem = many ? sizeof(SampleShared<warps_of(false)>) : sizeof(SampleShared<warps_of(true)>);
  const int rc = many ? allow_smem<sample_kernel<T, false>>(smem) : allow_smem<sample_kernel<T, true>>(smem);
  if (rc != FORK_OK) return FORK_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * cs);
  cfg.blockDim = dim3(warps_of(!many) * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cs;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = many ? 1 : 2;
  static const SampleTable table = [] {
    SampleTable t;
    for (int j = 0; j < 64; ++j) t.t[j] = static_cast<uint64_t>(std::llrint(std::exp2(j / 64.0) * static_cast<double>(1ull << kFrac)));
    return t;
  }();
  if (cuda_rc(cudaLaunchKernelEx(&cfg, kern, q, table)) != FORK_OK) return FORK_ECUDA;
  return cuda_rc(cudaGetLastError());
}

}  // namespace
}  // namespace fork

using namespace fork;

extern "C" int fork_sample(const void* logits, int32_t type, int32_t rows, int32_t V, int64_t row_stride,
                           const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                           const float* u, int32_t* token, float* prob, uint32_t flags, void* stream) {
  (void)flags;
  if (type != FORK_LOGITS_F32 && type != FORK_LOGITS_BF16) return FORK_EINVAL;
  if (rows < 0 || V < 1 || V > (1 << 18) || row_stride < V || rows > (1 << 24)) return FORK_EINVAL;
  if (rows == 0) return FORK_OK;
  if (!logits || !u || !token) return FORK_EINVAL;
  if ((reinterpret_cast<uintptr_t>(logits) & (type == FORK_LOGITS_F32 ? 3u : 1u)) != 0) return FORK_EINVAL;
  const void* words[] = {temperature, top_k, top_p, min_p, u, token, prob};
  for (const void* w : words)
    if ((reinterpret_cast<uintptr_t>(w) & 3u) != 0) return FORK_EINVAL;
  int rc;
  if ((rc = check_device()) != FORK_OK) return rc;
  SampleParams p;
  p.x = logits;
  p.stride = row_stride;
  p.rows = rows;
  p.V = V;
  p.ordered = 0;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.u = u;
  p.token = token;
  p.prob = prob;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == FORK_LOGITS_F32 ? launch_sample<float>(p, s) : launch_sample<uint16_t>(p, s);
}
