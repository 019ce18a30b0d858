// Drawing tokens from logits: temperature, top-k, top-p and min-p, with the
// random numbers given by the caller.
//
// For a row of logits x with the largest value m and temperature T > 0, the
// weights are w_i = e^((x_i - m) / T), ordered by falling x and, among equal
// x, by rising index.  Kept are
//   top-k: the first k of that order;
//   top-p: of these, the smallest prefix whose weight is at least p times theirs;
//   min-p: of these, the ones with w >= min_p * (the largest w = 1);
// and always the first.  Every filter keeps a prefix of the order, so the kept
// set is "x above a cut, or equal to it and among the first `ties` indices".
// The draw walks the kept tokens by rising index: the first whose cumulated
// weight exceeds u times the kept weight.
//
// A token on a border must fall where 64-bit arithmetic puts it, so a weight
// is a 64-bit integer (2^44 for the largest), good to 2^-29 of itself and
// 2^-45 of the largest (lighter ones are 0): the exponent in two fp32 words,
// 2^(j/128) from a table, the rest a cubic.  FP64 would do the same at a
// fortieth of the rate.  Integers also add up to the
// same sum in any order, so histograms and sums may use atomics.
//
// A row belongs to a cluster of up to 16 CTAs that keep it in shared memory:
// it is read from global memory once, and every later sweep is on chip.  A
// warp owns a run of consecutive indices, so index order is warp order.  A
// cut is found in two steps: a histogram over 1/32-wide steps of log2(w), of
// counts for top-k and of weights for top-p, names the step that holds it;
// the logits of that step, a few hundred as a rule, are gathered by every
// CTA and searched there, by a histogram of their ordered bit patterns and,
// among what is left in a bin of that, one against the other.  (A step that
// holds more than 2048, as in a row of equal logits, is searched where it
// lies, by histograms over ten bits of the patterns at a time.)  Top-k mostly
// needs no histogram of the row: the threads' largest logits bound the cut.
// The CTAs add up histograms through distributed shared memory: each sums a
// share of the bins and writes it to all.
//
// What bounds it is latency: a chain of sweeps and barriers, 1300 cycles each
// across a cluster (they lead the stalls; of the issue slots 40% are busy, with
// about 31 instructions for a weight and two shared atomics for one in a
// histogram).  Rows of 151936 fp32 logits, us for 1 / 32 / 128 rows: no filter
// 8.8 / 20 / 69, top-k 14 / 21 / 76, top-p 22 / 42 / 151; reading 32 takes 3.  A histogram
// of the whole row for top-k took 15 / 25 / 89.  64-bit shared atomics, which
// are loops of compare and swap, took 59 for 32 mixed rows (now 42).
#include <cooperative_groups.h>
#include <float.h>
#include <stddef.h>

#include <type_traits>

#include "common.cuh"
#include "errors.h"

namespace cg = cooperative_groups;

namespace bm {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kTile = 128;            // indices a warp takes at once, four to a lane
constexpr int kMaxTiles = 32;         // tiles of a warp
constexpr int kMaxCluster = 16;
constexpr int kBins = 1024;           // bins of a histogram: two to a thread
constexpr int kSteps = 32;            // steps to a factor of two of the weight
constexpr int kLastStep = kBins - 1;  // one step for all weights below 2^-31.97
constexpr int kList = 2 * kBins;      // logits a gathered step may have
constexpr int kOne = 44;              // log2 of the largest weight

// round(2^(30 + j/128))
__device__ const uint32_t kExp2[128] = {
    1073741824u, 1079572136u, 1085434106u, 1091327906u, 1097253708u, 1103211687u, 1109202018u, 1115224875u,
    1121280436u, 1127368878u, 1133490379u, 1139645120u, 1145833280u, 1152055042u, 1158310587u, 1164600099u,
    1170923762u, 1177281762u, 1183674286u, 1190101520u, 1196563654u, 1203060876u, 1209593378u, 1216161350u,
    1222764986u, 1229404479u, 1236080024u, 1242791816u, 1249540052u, 1256324931u, 1263146652u, 1270005413u,
    1276901417u, 1283834865u, 1290805962u, 1297814910u, 1304861917u, 1311947188u, 1319070932u, 1326233356u,
    1333434672u, 1340675091u, 1347954824u, 1355274085u, 1362633090u, 1370032052u, 1377471191u, 1384950723u,
    1392470869u, 1400031848u, 1407633882u, 1415277195u, 1422962010u, 1430688553u, 1438457051u, 1446267730u,
    1454120821u, 1462016553u, 1469955159u, 1477936870u, 1485961921u, 1494030547u, 1502142985u, 1510299473u,
    1518500250u, 1526745556u, 1535035634u, 1543370725u, 1551751076u, 1560176931u, 1568648537u, 1577166143u,
    1585730000u, 1594340357u, 1602997467u, 1611701585u, 1620452965u, 1629251865u, 1638098541u, 1646993254u,
    1655936265u, 1664927835u, 1673968228u, 1683057710u, 1692196547u, 1701385007u, 1710623359u, 1719911875u,
    1729250827u, 1738640488u, 1748081133u, 1757573041u, 1767116489u, 1776711757u, 1786359126u, 1796058879u,
    1805811301u, 1815616678u, 1825475297u, 1835387448u, 1845353420u, 1855373507u, 1865448001u, 1875577199u,
    1885761398u, 1896000896u, 1906295993u, 1916646992u, 1927054196u, 1937517909u, 1948038440u, 1958616096u,
    1969251188u, 1979944027u, 1990694927u, 2001504204u, 2012372174u, 2023299156u, 2034285470u, 2045331439u,
    2056437387u, 2067603638u, 2078830522u, 2090118366u, 2101467502u, 2112878262u, 2124350982u, 2135885998u,
};

struct SampleArgs {
  const void* x;
  long long ld;
  int V, B, tiles;                    // tiles: of a warp
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* ids;
  float* logp;
};

// Order-preserving bit pattern of a logit without NaN and -0; -infinity is 0.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return b == 0xFF800000u ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return k == 0 ? -INFINITY : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// NaN counts as -infinity, -0 as +0.
template <typename T>
__device__ __forceinline__ float clean(T v) {
  const float f = (float)v + 0.0f;
  return f != f ? -INFINITY : f;
}

constexpr uint32_t kLowest = 0x00800000u;   // key of the lowest finite value

struct Smem {
  uint2 exp2[128];                    // kExp2 and its fp32 value
  // by rank; each is told once, so no CTA overwrites what another still reads
  float top[kMaxCluster];             // largest logit
  uint32_t listed[3][kMaxCluster];    // logits gathered for a cut: top-k's twice, top-p's
  u64 kept[kMaxCluster];              // weight above the cut
  uint32_t equal[kMaxCluster];        // logits equal to the cut
  u64 warp64[kWarps];
  uint32_t warp32[kWarps];
  float warpf[kWarps];
  u64 tile64[kMaxTiles];
  uint32_t tile32[kMaxTiles];
  u64 mine[kBins], all[kBins];        // a histogram, the CTA's and the row's; counts in 32-bit words.  mine: also the CTA's list
  float list[kList];                  // the row's list
  uint32_t few[32];                   // keys that a search has left
  int at;
  uint32_t count, few_count;
  u64 before;
  float x[1];                         // [kWarps][tiles][kTile]
};

// The first step of a search, from its histogram: what the bins above it hold.
struct Found {
  int bin;
  u64 before;
};

// 2^y for y = hi + lo <= 0: 2^30 * 2^(j/128 + g) in w, and the power of two it is to be divided by.
__device__ __forceinline__ uint32_t exp2_parts(float hi, float lo, const uint2* table, int& down) {
  hi = fmaxf(hi, -60.f);
  // hi = (128 n + j) / 128 + g; the bits of z hold 128 n + j
  const float z = fmaf(hi, 128.f, 12582912.f);
  const float g = fmaf(z - 12582912.f, -1.f / 128, hi) + lo;
  const int N = __float_as_int(z) - 0x4B400000;
  down = -(N >> 7);
  // 2^g - 1 for |g| <= 1/256: the next term of the series is below 2^-38
  const float q = g * fmaf(g, fmaf(g, 0.05550411f, 0.24022651f), 0.69314718f);
  const uint2 t = table[N & 127];
  // t * 2^g, in steps of two: |t q| < 2^23
  return t.x + 2u * (uint32_t)(__float_as_int(fmaf(__uint_as_float(t.y), q, 25165824.f)) - 0x4BC00000);
}

// Weights of a row: 2^((x - m) * c) with c = log2(e) / T in two words.
struct Weights {
  float m, ch, cl;
  // log2 of x's weight as hi + lo
  __device__ __forceinline__ float exponent(float x, float& lo) const {
    const float d = x - m, bb = d - x, e = (x - (d - bb)) + (-m - bb);   // x - m = d + e
    const float hi = d * ch;
    lo = fmaf(d, cl, fmaf(e, ch, fmaf(d, ch, -hi)));
    return hi;
  }
  // sum + (take ? the weight of x : 0).  The weight is 2^30..2^31 in 32 bits, multiplied up or, where it is
  // below 2^-14 of the largest, shifted down and rounded: one wide multiply-add, and no 64-bit shift.
  __device__ __forceinline__ u64 add(u64 sum, float x, const uint2* table, bool take = true) const {
    float lo;
    int down;
    const float hi = exponent(x, lo);
    const uint32_t w = exp2_parts(hi, lo, table, down);
    const int up = kOne - 30 - down;
    const uint32_t v = (__funnelshift_rc(2 * w, 0u, max(0, -up)) + (up < 0)) >> 1;
    return (u64)v * (take ? 1u << max(0, up) : 0u) + sum;
  }
  __device__ __forceinline__ u64 operator()(float x, const uint2* table) const { return add(0, x, table); }
  // The weight of x, of step `bin`, in units of 2^(kOne - 31 - octave): below 2^32, for all of a step the same unit.
  __device__ __forceinline__ uint32_t in_step(float x, int bin, const uint2* table) const {
    float lo;
    int down;
    const float hi = exponent(x, lo);
    const uint32_t w = exp2_parts(hi, lo, table, down);
    const int up = bin / kSteps + 1 - down;              // 0 or 1, but for the last step
    return up >= 0 ? w << up : __funnelshift_rc(w, 0u, -up);
  }
  static __device__ __forceinline__ u64 from_step(u64 sum, int bin) {
    const int up = kOne - 31 - bin / kSteps;
    return up >= 0 ? sum << up : (sum + (1ull << (-up - 1))) >> -up;
  }
  // step of 1/kSteps in log2 of the weight, from the top
  __device__ __forceinline__ int bin(float x) const { return (int)fminf((m - x) * (kSteps * ch), (float)kLastStep); }
};

// ln(w / total) to fp32, of a token whose weight is w = 2^(hi + lo) of the largest: from its exponent and not from
// its integer, which has few bits left for a light token.  The logarithm of total, at least 2^kOne, is an fp32
// one of its mantissa, corrected once by its exponential in integers.
__device__ float log_share(float hi, float lo, u64 total, const uint2* table) {
  const int z = __clzll(total);
  const u64 b = total << z;                                // 2^63 / b: in (1/2, 1]
  const float y = fminf(-log2f((float)b * 1.0842021724855044e-19f), 0.f);
  int down;
  const uint32_t w = exp2_parts(y, 0.f, table, down);
  const u64 back = __umul64hi(b, (u64)w << (33 - down)) << 1;   // b * 2^y
  const float off = (float)(long long)((1ull << 63) - back) * (1.0842021724855044e-19f * 1.44269502f);
  // log2(2^kOne / total) = h + l, and the weight's to it
  const float e = (float)(z - 63 + kOne);
  const float h = e + y, l = (y - (h - e)) + off;
  const float s = h + hi, bb = s - h, t = (h - (s - bb)) + (hi - bb) + l + lo;
  const float r = s * 0.693147182f;
  return r + fmaf(t, 0.693147182f, fmaf(s, 0.693147182f, -r) + s * -1.90465421e-09f);
}

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// A histogram's sums of 32-bit weights: 16 bits to a word, as a CTA has fewer than 2^16 logits (no carry,
// so nothing waits for an atomic's old value).
struct Halves {
  uint32_t lo, hi;
  __device__ __forceinline__ void add(uint32_t v) {
    atomicAdd(&lo, v & 0xFFFFu);
    atomicAdd(&hi, v >> 16);
  }
  __device__ __forceinline__ u64 sum() const { return lo + ((u64)hi << 16); }
};
static_assert(kWarps * kMaxTiles * kTile <= 1 << 16, "a word of Halves holds a CTA's sum");

// 64-bit sum in shared memory from two 32-bit atomics: the low word's old value tells the carry.
__device__ __forceinline__ void add64(u64* at, u64 v) {
  uint32_t* p = reinterpret_cast<uint32_t*>(at);
  const uint32_t lo = (uint32_t)v, old = atomicAdd(p, lo), hi = (uint32_t)(v >> 32) + (old + lo < old);
  if (hi) atomicAdd(p + 1, hi);
}
// Sum over the lanes below this one and this one.
template <typename T>
__device__ __forceinline__ T warp_scan(T v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T n = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += n;
  }
  return v;
}
// Sum over the threads before this one; `tot` of all.  warp: kWarps words of shared memory.
template <typename T>
__device__ __forceinline__ T block_before(T v, T* warp, T* tot) {
  const T inc = warp_scan(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 31) warp[threadIdx.x >> 5] = inc;
  __syncthreads();
  T b = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < (int)(threadIdx.x >> 5)) b += warp[w];
    all += warp[w];
  }
  *tot = all;
  return b + inc - v;
}

struct Row {
  cg::cluster_group cl;
  Smem& s;
  int rank, n, tiles;
  Weights w;
  float4* tile;                       // this warp's tiles; lane's four logits of tile t at [32 t + lane]

  __device__ void sync() const {
    if (n == 1) __syncthreads();
    else cl.sync();
  }
  // f(four logits) over this thread's
  template <typename F>
  __device__ __forceinline__ void sweep4(F f) const {
    for (int t = 0; t < tiles; ++t) f(tile[32 * t + (threadIdx.x & 31)]);
  }
  template <typename F>
  __device__ __forceinline__ void sweep(F f) const {
    sweep4([&](const float4 v) {
      f(v.x);
      f(v.y);
      f(v.z);
      f(v.w);
    });
  }
  // f(x, x > cut) over the logits, where any of four is above it: with a branch
  // to each, their latencies would add up
  template <typename F>
  __device__ __forceinline__ void sweep_above(float cut, F f) const {
    sweep4([&](const float4 v) {
      const bool a = v.x > cut, b = v.y > cut, c = v.z > cut, d = v.w > cut;
      if (a || b || c || d) {
        f(v.x, a);
        f(v.y, b);
        f(v.z, c);
        f(v.w, d);
      }
    });
  }
  // f(x) over the logits in [lo, hi], which are few
  template <typename F>
  __device__ __forceinline__ void sweep_range(float lo, float hi, F f) const {
    sweep4([&](const float4 v) {
      const bool a = v.x >= lo && v.x <= hi, b = v.y >= lo && v.y <= hi, c = v.z >= lo && v.z <= hi, d = v.w >= lo && v.w <= hi;
      if (a || b || c || d) {
        if (a) f(v.x);
        if (b) f(v.y);
        if (c) f(v.z);
        if (d) f(v.w);
      }
    });
  }
  // This CTA's value to slot[rank] of every CTA; read after the next sync().
  template <typename T>
  __device__ __forceinline__ void tell(T* slot, T v) const {
    if ((int)threadIdx.x < n) cl.map_shared_rank(slot, threadIdx.x)[rank] = v;
  }
  template <typename T>
  __device__ __forceinline__ T total(const T* slot) const {
    T v = 0;
    for (int r = 0; r < n; ++r) v += slot[r];
    return v;
  }
  // all[] = the CTAs' mine[] added up; mine[] is free again afterwards.  A CTA
  // sums kBins / n of the bins, n / 2 lanes to a bin, and tells all CTAs.  What
  // is rounded of a bin is its sum over the row, the same for any n.
  template <typename M, typename T>
  __device__ void add_up(M* mine, T* all) const {
    sync();
    if (n == 1) {
      for (int b = threadIdx.x; b < kBins; b += kThreads) all[b] = scaled(mine[b], whole(mine[b]), b);
    } else {
      const int per = n / 2, b = rank * (kBins / n) + threadIdx.x / per, q = threadIdx.x & (per - 1);
      const M v0 = cl.map_shared_rank(mine, q)[b], v1 = cl.map_shared_rank(mine, q + per)[b];
      T v = whole(v0) + whole(v1);
      for (int o = per / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      v = scaled(v0, v, b);
      cl.map_shared_rank(all, q)[b] = v;
      cl.map_shared_rank(all, q + per)[b] = v;
    }
    sync();
  }
  static __device__ __forceinline__ uint32_t whole(uint32_t v) { return v; }
  static __device__ __forceinline__ u64 whole(u64 v) { return v; }
  static __device__ __forceinline__ u64 whole(Halves v) { return v.sum(); }   // of 16 CTAs: below 2^52
  // a bin's sum in weights, by what its histogram holds
  template <typename T>
  static __device__ __forceinline__ T scaled(T, T v, int) { return v; }
  static __device__ __forceinline__ u64 scaled(Halves, u64 v, int bin) { return Weights::from_step(v, bin); }
  // The bin at which the histogram all[], of sum s, reaches need(s), counted
  // on from `base`; the last one that holds anything, should it not.
  // Between two calls there is a barrier.
  template <typename Word, typename F>
  __device__ Found reach(const Word* all, u64 base, F need_of) const {
    if (threadIdx.x == 0) {
      s.at = 0;
      s.before = base;
    }
    const u64 v0 = all[2 * threadIdx.x], v1 = all[2 * threadIdx.x + 1];
    u64 sum;
    const u64 b0 = base + block_before<u64>(v0 + v1, s.warp64, &sum), need = min((u64)need_of(sum), base + sum);
    if (b0 < need && b0 + v0 + v1 >= need) {
      const bool second = b0 + v0 < need;
      s.at = 2 * threadIdx.x + second;
      s.before = second ? b0 + v0 : b0;
    }
    __syncthreads();
    return Found{s.at, s.before};
  }
  // Bounds of the keys of a step; a little wider than they are.
  __device__ void key_range(int bin, uint32_t& lo, uint32_t& hi) const {
    const float step = 1.0f / (kSteps * w.ch);
    const float d1 = bin * step, d2 = (bin + 1) * step;
    hi = key_of(w.m);
    if (bin > 0) hi = min(hi, key_of(w.m - d1 + 1e-5f * (fabsf(w.m) + d1)));
    lo = kLowest;
    const float v = w.m - d2 - 1e-5f * (fabsf(w.m) + d2);
    if (bin < kLastStep && v > -FLT_MAX) lo = key_of(v);
  }
  // The key at which the weight (MASS) or the number of the logits of step
  // f.bin that are at least `least` reaches `need`, from the largest down,
  // counted on from f.before; *before is what the keys above it hold.  FROM_TOP:
  // of all steps down to f.bin; 0 if those are more than a list holds.
  template <bool MASS, bool FROM_TOP>
  __device__ uint32_t find(Found f, uint32_t least, u64 need, uint32_t* listed, u64* before) const {
    using Word = typename std::conditional<MASS, u64, uint32_t>::type;
    uint32_t lo, hi;
    key_range(f.bin, lo, hi);
    if (FROM_TOP) hi = key_of(w.m);
    lo = max(lo, least);
    hi = max(hi, lo);
    const float vlo = value_of(lo), vhi = value_of(hi);
    auto in = [&](float x) { return FROM_TOP ? w.bin(x) <= f.bin : w.bin(x) == f.bin; };
    // every CTA's logits of the step to every CTA
    float* own = reinterpret_cast<float*>(s.mine);
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
    sweep_range(vlo, vhi, [&](float x) {
      if (!in(x)) return;
      const uint32_t i = atomicAdd(&s.count, 1u);
      if (i < kList) own[i] = x;
    });
    __syncthreads();
    tell(listed, s.count);
    sync();
    const uint32_t count = total(listed);
    const bool gathered = count <= kList;
    if (FROM_TOP && !gathered) return 0;
    if (gathered) {
      const int i = threadIdx.x >> 5;   // warp i takes the list of CTA i
      if (i < n) {
        uint32_t off = 0;
        for (int j = 0; j < i; ++j) off += listed[j];
        const float* theirs = cl.map_shared_rank(own, i);
        for (uint32_t j = threadIdx.x & 31; j < listed[i]; j += 32) s.list[off + j] = theirs[j];
      }
    }
    Word* mine = reinterpret_cast<Word*>(gathered ? s.all : s.mine);
    Word* all = reinterpret_cast<Word*>(s.all);
    u64 base = f.before;
    for (;;) {
      const int shift = max(0, 32 - __clz(hi - lo) - 10);
      for (int i = threadIdx.x; i < kBins; i += kThreads) mine[i] = 0;
      __syncthreads();
      if (threadIdx.x == 0) s.few_count = 0;
      auto put = [&](float x) {
        const uint32_t k = key_of(x);
        if (k >= lo && k <= hi) {
          if (MASS) add64(reinterpret_cast<u64*>(&mine[(hi - k) >> shift]), w(x, s.exp2));
          else atomicAdd(reinterpret_cast<uint32_t*>(&mine[(hi - k) >> shift]), 1u);
        }
      };
      if (gathered) {
        for (uint32_t i = threadIdx.x; i < count; i += kThreads) put(s.list[i]);
        __syncthreads();
      } else {
        sweep_range(vlo, vhi, [&](float x) {
          if (in(x)) put(x);
        });
        add_up(mine, all);
      }
      const Found g = reach(all, base, [&](u64) { return need; });
      base = g.before;
      hi -= (uint32_t)g.bin << shift;
      const uint32_t span = (1u << shift) - 1;
      lo = hi - lo > span ? hi - span : lo;
      if (lo == hi) break;
      if (gathered) {                 // up to 32 keys: every warp ranks them
        for (uint32_t i = threadIdx.x; i < count; i += kThreads) {
          const uint32_t k = key_of(s.list[i]);
          if (k >= lo && k <= hi) {
            const uint32_t at = atomicAdd(&s.few_count, 1u);
            if (at < 32) s.few[at] = k;
          }
        }
        __syncthreads();
        const int few = (int)s.few_count, lane = threadIdx.x & 31;
        if (few <= 32) {
          const uint32_t k = lane < few ? s.few[lane] : 0u;
          const u64 v = lane >= few ? 0 : MASS ? w(value_of(k), s.exp2) : 1;
          u64 above = base, upto = base, sum = base;
          for (int j = 0; j < few; ++j) {
            const uint32_t kj = __shfl_sync(0xffffffffu, k, j);
            const u64 vj = __shfl_sync(0xffffffffu, v, j);
            sum += vj;
            above += kj > k ? vj : 0;
            upto += kj >= k ? vj : 0;
          }
          need = min(need, sum);
          unsigned hit = __ballot_sync(0xffffffffu, above < need && need <= upto && lane < few);
          if (!hit) hit = __ballot_sync(0xffffffffu, above == base && lane < few);   // weights that round to nothing
          if (hit) {
            lo = __shfl_sync(0xffffffffu, k, __ffs(hit) - 1);
            base = __shfl_sync(0xffffffffu, above, __ffs(hit) - 1);
          }
          break;
        }
      }
    }
    *before = base;
    return lo;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(SampleArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), n = cl.num_blocks(), b = blockIdx.x / n;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tiles = a.tiles, V = a.V;
  float* xs = reinterpret_cast<float*>(raw + ((offsetof(Smem, x) + 15) & ~size_t(15)));
  Row r{cl, s, rank, n, tiles, Weights{}, reinterpret_cast<float4*>(xs) + 32 * tiles * warp};

  // Every CTA of the cluster has to have started before another writes to its shared memory.
  if (n > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  // ---- the row to shared memory, with its largest logit
  const T* src = static_cast<const T*>(a.x) + b * a.ld;
  const int first = (rank * kWarps + warp) * tiles * kTile;   // this warp's first index
  const bool vec = (reinterpret_cast<uintptr_t>(src) & (4 * sizeof(T) - 1)) == 0;
  // the row's settings, and log2(e) / T in two words, while the row is on its way
  const float temp = a.temperature ? a.temperature[b] : 1.f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.f, least = a.min_p ? a.min_p[b] : 0.f, u = fmaxf(a.u[b], 0.f);   // NaN u: 0
  float best = -INFINITY;
#pragma unroll 5
  for (int t = 0; t < tiles; ++t) {
    const int i = first + t * kTile + 4 * lane;
    float v[4];
    if (vec && i + 3 < V) {
      if (sizeof(T) == 4) {
        const float4 f = __ldcs(reinterpret_cast<const float4*>(src + i));
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
      } else {
        const uint2 f = __ldcs(reinterpret_cast<const uint2*>(src + i));
        v[0] = bf_lo(f.x); v[1] = bf_hi(f.x); v[2] = bf_lo(f.y); v[3] = bf_hi(f.y);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = i + e < V ? (float)src[i + e] : -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = clean(v[e]);
      best = fmaxf(best, v[e]);
    }
    r.tile[32 * t + lane] = make_float4(v[0], v[1], v[2], v[3]);
  }
  float thread_best = best;
  best = warp_max(best);
  if (lane == 0) s.warpf[warp] = best;
  if (tid < 128) s.exp2[tid] = make_uint2(kExp2[tid], __float_as_uint((float)kExp2[tid]));
  {
    // below 2^-120 any two different logits of a model are infinitely far apart
    const float t = fmaxf(temp, 7.5231638452626401e-37f);
    r.w.ch = 1.44269502f / t;
    r.w.cl = t < INFINITY ? (fmaf(-r.w.ch, t, 1.44269502f) + 1.92596303e-08f) / t : 0.f;
  }
  if (n > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) best = fmaxf(best, s.warpf[i]);
  r.tell(s.top, best);
  r.sync();
  for (int i = 0; i < n; ++i) best = fmaxf(best, s.top[i]);
  if (best == -INFINITY) {            // nothing to draw
    if (rank == 0 && tid == 0) {
      a.ids[b] = -1;
      if (a.logp) a.logp[b] = -INFINITY;
    }
    return;
  }
  if (best == INFINITY) {             // the infinite logits share the row: they become 0, all others are masked
    for (int t = 0; t < tiles; ++t) {
      float4& v = r.tile[32 * t + lane];
      v.x = v.x == INFINITY ? 0.f : -INFINITY;
      v.y = v.y == INFINITY ? 0.f : -INFINITY;
      v.z = v.z == INFINITY ? 0.f : -INFINITY;
      v.w = v.w == INFINITY ? 0.f : -INFINITY;
    }
    best = 0.f;
    thread_best = thread_best == INFINITY ? 0.f : -INFINITY;
  }
  r.w.m = best;
  const Weights& w = r.w;

  // ---- the cut: kept are the keys above it, and the first `ties` that equal it
  uint32_t cut = 0, ties = 0;
  if (!(temp > 0.f)) {                // the argmax, lowest index first
    cut = key_of(best);
    ties = 1;
  } else {
    if (k > 0 && k < V) {
      uint32_t* mine = reinterpret_cast<uint32_t*>(s.mine);
      uint32_t* all = reinterpret_cast<uint32_t*>(s.all);
      u64 have = 0, before = 0;
      auto count = [&](bool maxima) {
        for (int i = tid; i < kBins; i += kThreads) mine[i] = 0;
        __syncthreads();
        if (maxima) {
          if (thread_best > -INFINITY) atomicAdd(&mine[w.bin(thread_best)], 1u);
        } else {
          r.sweep([&](float x) {
            if (x > -INFINITY) atomicAdd(&mine[w.bin(x)], 1u);
          });
        }
        r.add_up(mine, all);
        return r.reach(all, 0, [&](u64 sum) {
          have = sum;
          return (u64)k;
        });
      };
      // The k-th of the threads' largest logits is no larger than the k-th of all, and while k is a fraction of the
      // threads not many are between the two: those down to its step are listed without a histogram of the row.
      if (k <= n * (kThreads / 4)) {
        const Found f = count(true);
        if (have >= (u64)k) cut = r.template find<false, true>(Found{f.bin, 0}, 1, (u64)k, s.listed[0], &before);
      }
      if (!cut) {
        const Found f = count(false);
        if (have > (u64)k) cut = r.template find<false, false>(f, 1, (u64)k, s.listed[1], &before);   // else there are no more than k
      }
      if (cut) {
        ties = (uint32_t)(k - before);
        if (p < 1.f) r.sync();        // every CTA has read the lists
      }
    }
    if (p < 1.f) {
      const float kv = value_of(cut);
      Halves* mine = reinterpret_cast<Halves*>(s.mine);
      for (int i = tid; i < kBins; i += kThreads) s.mine[i] = 0;
      __syncthreads();
      r.sweep_above(kv, [&](float x, bool above) {
        const int bin = w.bin(x);
        const uint32_t v = w.in_step(x, bin, s.exp2);
        if (above) mine[bin].add(v);
      });
      r.add_up(mine, s.all);
      if (ties) {                     // the logits that top-k's cut shares, by count
        if (tid == 0) s.all[w.bin(kv)] += ties * w(kv, s.exp2);
        __syncthreads();
      }
      const u64 p64 = __float2ull_rz(fmaxf(p, 0.f) * 18446744073709551616.f);   // p < 1 in 64 binary places
      u64 need = 0;
      const Found f = r.reach(s.all, 0, [&](u64 sum) { return need = max(1ull, __umul64hi(sum, p64) + (sum * p64 != 0)); });
      const uint32_t k_cut = cut, k_ties = ties;
      u64 before;
      cut = r.template find<true, false>(f, max(1u, k_cut), need, s.listed[2], &before);
      const u64 wc = w(value_of(cut), s.exp2);
      const u64 rest = need - min(need, before), want = rest <= wc ? 1 : wc ? (rest + wc - 1) / wc : 1;
      ties = (uint32_t)min(want, (u64)V);
      if (cut == k_cut) ties = min(ties, k_ties);
    }
  }
  const float cv = value_of(cut);
  const u64 one = 1ull << kOne;
  const u64 wmin = least > 0.f && temp > 0.f ? __float2ull_rz(fminf(least, 1.f) * (float)one) : 0;
  const u64 wcut = ties ? w(cv, s.exp2) : 0;
  if (wcut < wmin) ties = 0;

  // ---- kept weight by warp, CTA and row
  u64 mass = 0;
  uint32_t eq = 0;
  if (cut == 0 && wmin == 0) {
    r.sweep([&](float x) { mass = w.add(mass, x, s.exp2); });
  } else {
    if (wmin) {
      r.sweep_above(cv, [&](float x, bool above) {
        const u64 v = w(x, s.exp2);
        mass += above && v >= wmin ? v : 0;
      });
    } else {
      r.sweep_above(cv, [&](float x, bool above) { mass = w.add(mass, x, s.exp2, above); });
    }
    if (ties) r.sweep([&](float x) { eq += x == cv; });
  }
  mass = warp_sum64(mass);
  eq = warp_sum(eq);
  __syncthreads();
  if (lane == 0) {
    s.warp64[warp] = mass;
    s.warp32[warp] = eq;
  }
  __syncthreads();
  {
    u64 m = 0;
    uint32_t e = 0;
    for (int i = 0; i < kWarps; ++i) {
      m += s.warp64[i];
      e += s.warp32[i];
    }
    r.tell(s.kept, m);
    r.tell(s.equal, e);
  }
  r.sync();
  const u64 kept = r.total(s.kept) + min((u64)ties, (u64)r.total(s.equal)) * wcut;
  u64 target = u >= 1.f ? kept - 1 : __umul64hi(kept, __float2ull_rz(u * 18446744073709551616.f));
  // the CTA, then the warp, then the tile that holds the target
  int left = (int)ties, owner = -1;
  for (int i = 0; i < n; ++i) {
    const int e = min(left, (int)min(s.equal[i], 0x7FFFFFFFu));
    const u64 v = s.kept[i] + e * wcut;
    if (target < v) {
      owner = i;
      break;
    }
    target -= v;
    left -= e;
  }
  if (owner != rank) return;
  int own = 0;
  for (; own < kWarps - 1; ++own) {
    const int e = min(left, (int)s.warp32[own]);
    const u64 v = s.warp64[own] + e * wcut;
    if (target < v) break;
    target -= v;
    left -= e;
  }
  const float4* tile = reinterpret_cast<const float4*>(xs) + 32 * tiles * own;
  auto four = [&](int t, u64 (&v)[4], uint32_t& same) {
    const float4 x = tile[32 * t + lane];
    const float xe[4] = {x.x, x.y, x.z, x.w};
    same = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = 0;
      if (xe[i] > cv) {
        v[i] = w(xe[i], s.exp2);
        if (v[i] < wmin) v[i] = 0;
      }
      same |= (uint32_t)(xe[i] == cv) << i;
    }
  };
  u64 v[4];
  uint32_t same;
  for (int t = warp; t < tiles; t += kWarps) {
    four(t, v, same);
    const u64 m = warp_sum64(v[0] + v[1] + v[2] + v[3]);
    const uint32_t e = warp_sum((uint32_t)__popc(same));
    if (lane == 0) {
      s.tile64[t] = m;
      s.tile32[t] = e;
    }
  }
  __syncthreads();
  if (warp != 0) return;
  int at = 0;
  for (; at < tiles - 1; ++at) {
    const int e = min(left, (int)s.tile32[at]);
    const u64 m = s.tile64[at] + e * wcut;
    if (target < m) break;
    target -= m;
    left -= e;
  }
  four(at, v, same);
  int e = left - ((int)warp_scan((uint32_t)__popc(same)) - __popc(same));   // ties left to this lane
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (same >> i & 1 && e-- > 0) v[i] = wcut;
  const u64 sum = v[0] + v[1] + v[2] + v[3], upto = warp_scan(sum);
  u64 cum = upto - sum;
  if (!(cum <= target && target < upto)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (cum <= target && target < cum + v[i]) {
      a.ids[b] = (rank * kWarps + own) * tiles * kTile + at * kTile + 4 * lane + i;
      if (a.logp) {
        const float4 x = tile[32 * at + lane];
        float lo;
        const float hi = w.exponent(i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w, lo);
        a.logp[b] = temp > 0.f ? log_share(hi, lo, kept, s.exp2) : 0.f;
      }
    }
    cum += v[i];
  }
}

// Shared-memory and cluster attributes of both kernels on the current device.
cudaError_t ensure_attributes() {
  static std::atomic<unsigned long long> done{0};
  return once_per_device(done, [] {
    const void* kernels[] = {(const void*)k_sample<float>, (const void*)k_sample<bf16>};
    cudaError_t e = cudaSuccess;
    for (const void* f : kernels) {
      if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    }
    return e;
  });
}

// CTAs per row: the largest cluster that still pays, and at least one whose shared memory holds the row (20 tiles a
// warp).  A wider cluster shortens every sweep but costs barriers, and its rows start together only while they fit:
// 15 clusters of 8 or 7 of 16 (they lie within a GPC), 128 CTAs of the smaller ones an SM each, two an SM after that.
// Sharing an SM, or waiting for a second wave, pays for longer rows only.  Times of 4 / 8 / 16 CTAs a row, us:
//   V = 32000:   9 rows 17.8 / 15.2 / 18.1;  16 rows 19.3 / 21.6 / 23.0;  128 rows 43.7 / 61.6 / 120 (2 CTAs: 36.3)
//   V = 151936:  8 rows 58.3 / 37.1 / 25.6;  16 rows 58.8 / 38.9 / 31.0;  32 rows 48.2 / 45.1 / 53.8
//   V = 1000:   any rows below 64, 1 CTA 10.5, 4 12.5
int cluster_size(int B, int V) {
  int n = kMaxCluster;
  for (; n > 1 && n * kWarps * kTile * 10 >= V; n /= 2) {
    const int64_t ctas = (int64_t)B * n;
    if (ctas <= (n > 4 ? 120 : 128) && n * 2048 <= V) break;
    if (ctas <= 256 && n * 4096 <= V) break;
    if (ctas <= 512 && n * 12288 <= V) break;
  }
  return n;
}

}  // namespace
}  // namespace bm

extern "C" bm_status bm_sample(const void* logits, int dtype, int64_t ld, int V, int B, const float* temperature,
                               const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* ids,
                               float* logprobs, void* stream) {
  using namespace bm;
  if (!logits || !u || !ids) return set_error(BM_ERR_INVALID_ARG, "bm_sample: null pointer");
  if (dtype != BM_F32 && dtype != BM_BF16) return set_error(BM_ERR_INVALID_ARG, "bm_sample: dtype must be BM_F32 or BM_BF16");
  if (B < 1 || B > 65535 || V < 1 || V > BM_SAMPLE_MAX_VOCAB)
    return set_error(BM_ERR_INVALID_ARG, "bm_sample: need 1 <= B <= 65535 and 1 <= V <= " + std::to_string(BM_SAMPLE_MAX_VOCAB));
  if (ld < V) return set_error(BM_ERR_INVALID_ARG, "bm_sample: ld must be at least V");
  if ((uintptr_t)logits & (dtype == BM_F32 ? 3 : 1)) return set_error(BM_ERR_INVALID_ARG, "bm_sample: misaligned logits");
  if (((uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)u | (uintptr_t)ids | (uintptr_t)logprobs) & 3)
    return set_error(BM_ERR_INVALID_ARG, "bm_sample: temperature, top_k, top_p, min_p, u, ids and logprobs must be 4-byte aligned");
  cudaError_t e = ensure_attributes();
  if (e == cudaSuccess) {
    const int n = cluster_size(B, V);
    const int tiles = (V + n * kWarps * kTile - 1) / (n * kWarps * kTile);
    const SampleArgs a{logits, ld, V, B, tiles, temperature, top_k, top_p, min_p, u, ids, logprobs};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)B * n);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem) + 16 + (size_t)kWarps * tiles * kTile * sizeof(float);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = dtype == BM_F32 ? cudaLaunchKernelEx(&cfg, k_sample<float>, a) : cudaLaunchKernelEx(&cfg, k_sample<bf16>, a);
  }
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, std::string("bm_sample: ") + cudaGetErrorString(e));
  return ok();
}
