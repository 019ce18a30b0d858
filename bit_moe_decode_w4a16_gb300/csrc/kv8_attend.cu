// Single-token attention over the 8-bit K/V cache, alone or behind a prefix
// that the whole batch shares.
//
// For head h of stream b, over the prefix's positions and then the stream's
// own, with k = kc * ks and v = vc * vs (codes times scales):
//   s_j = scale * (q . k_j),  o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
// The positions are split into chunks (kv8.cuh); a chunk's running maximum m,
// sum l and unnormalised o are a record, and a stream's records are merged in
// ascending order: prefix chunks first, then its own.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "kv8_attend.cuh"

namespace bm {
namespace {

using namespace kv8;

// ---------------------------------------------------------------- one pass over a chunk
//
// A work item is a chunk of a stream's positions and the query rows of one
// of its kv heads.  The item's four warps take 32 positions each of every stage
// of 128; each keeps a running maximum, sum and output of its own, and the
// four are merged at the end of the item.  A warp streams its positions
// through a ring of its own in shared memory (cp.async, a stage ahead,
// across items), so the loop has no barrier between warps.
//
// On the tensor cores (mma.sync m16n8k16, fp16, fp32 sums), with g = lane / 4
// and t = lane % 4:
//   S = Q K^T: rows are heads (8 to 15 are zero), columns positions.  The
//     reduction over d is permuted: lane t takes the 16-byte pieces of a K
//     row that it reads whole, and q in the same order.  Codes become fp16
//     exactly; the score is multiplied by the position's scale in fp32.
//   O^T = V^T P^T: rows are elements of d, columns heads.  S's layout is
//     P^T's: no exchange.  Row g of tile j is element 16g + 2j, row g + 8 the
//     next one, so that lane (g, t) reads 16 bytes of each of its four
//     positions and interleaves them by byte.
// A weight enters as fp16(p * vs).  Its reference is the running maximum of
// s + log2(vs), not of s: the product stays in fp16's range whatever V's
// magnitude (its scales are 0 or lie in 2^-100 .. 2^100: the sum of the weights
// has the same reference and fp32's range), and what is rounded away is small
// against the largest term of the sum.  The reference moves only when it is
// passed by 2^8 (an fp16 holds that), so the output is seldom rescaled.
//
// Three CTAs an SM (two in batches of hundreds of rows, see the launch) take
// items in order of size, so the grid ends together.
// 32 streams of 8192 positions, 32 + 2 x 4 heads of 128, e4m3: 53 us with the
// merge, 5.2 TB/s of codes and scales; 12 warps an SM keep 69% of HBM busy
// (four CTAs with stages of half the size took longer, two with twice as
// much shared memory 84 us).  16 streams of 8192: 33 us, 4.2 TB/s, as 2.25
// rounds of items take 3.  16 streams of 1 to 8192: 21 us, 17 from L2, where the
// items' uneven ends and the chain of two launches show.  One stream of 4096:
// 7 us, latency alone.
constexpr int kWarpsPerItem = 4, kTake = 32, kStage = kWarpsPerItem * kTake, kRing = 2;

template <int D>
struct alignas(16) Ring {
  uint8_t k[kTake * D], v[kTake * D];
  float ks[kTake], vs[kTake];
};

template <int D>
using WarpOut = float[8][D + 8];

template <int D>
struct ChunkSmem {
  static_assert(sizeof(WarpOut<D>) <= sizeof(Ring<D>), "a warp's output fits a slot");
  Ring<D> ring[kWarpsPerItem][kRing];   // at an item's end a warp's output lies in the slot it has just used
  float m[kWarpsPerItem][8], l[kWarpsPerItem][8];
  int streams;                        // live ones of some length
  int table[1];                       // [B] slots, [B] lengths, [B] the live streams in item order, [2 B + 1] items before each entry's
};

// 16-byte piece c of a position's codes in the ring: swizzled so that both products read without bank conflicts.
template <int D>
__device__ __forceinline__ int piece(int token, int c) {
  return token * D + 16 * (D == 128 ? c ^ (token & 7) : c ^ (token >> 1 & 3));
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t shared_address(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(shared_address(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(shared_address(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(void* dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(shared_address(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4_or_zero(void* dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(shared_address(dst)), "l"(src), "r"(live ? 4 : 0) : "memory");
}
struct Item {
  const uint8_t *K, *V;
  const float *Ks, *Vs;
  int n, kh, b, rec;                  // positions; kv head; stream; chunk of the stream
};

template <int D, int FMT>
__global__ void __launch_bounds__(kWarpsPerItem * 32, 3) k_kv8_chunk(AttendArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  ChunkSmem<D>& sm = *reinterpret_cast<ChunkSmem<D>*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int kvh = a.c.kvh, G = a.qh / kvh;
  pdl_trigger();   // the whole grid is resident: the merge may take the free slots
  int *slots = sm.table, *lens = slots + a.B, *order = lens + a.B, *first = order + a.B;

  // ---- the items: the streams' whole chunks, streams of the largest chunks first, then their last, shorter ones.
  // CTA i takes item i of every even block of gridDim items and the opposite one of every odd block, which
  // evens out their sizes.
  int streams = 0;
  if (warp == 0) {
    int top = 0, low = 1 << 30, sum = 0;   // chunk sizes there are
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      if (b < a.B) {
        int slot, len;
        if (!a.live(b, slot, len)) len = 0;
        slots[b] = slot;
        lens[b] = len;
        if (len > 0) {
          top = max(top, chunk_of(len));
          low = min(low, chunk_of(len));
        }
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    low = __reduce_min_sync(0xffffffffu, low);
    // an entry's items before it, the lanes' entries in their order
    auto enter = [&](bool has, int count, int at) {
      int inc = has ? count : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (has) first[at] = sum + inc - count;
      sum += __shfl_sync(0xffffffffu, inc, 31);
    };
    for (int size = top; size >= low; size /= 2)
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane, len = b < a.B ? lens[b] : 0;
        const bool has = len > 0 && chunk_of(len) == size;
        const unsigned votes = __ballot_sync(0xffffffffu, has);
        const int at = streams + __popc(votes & ((1u << lane) - 1));
        if (has) order[at] = b;
        enter(has, len / size * kvh, at);
        streams += __popc(votes);
      }
    __syncwarp();
    for (int e0 = 0; e0 < streams; e0 += 32) {
      const int e = e0 + lane, len = e < streams ? lens[order[e]] : 0;
      enter(e < streams, len > 0 && len % chunk_of(len) ? kvh : 0, streams + e);
    }
    if (lane == 0) {
      first[2 * streams] = sum;
      sm.streams = streams;
    }
  }
  __syncthreads();
  streams = sm.streams;
  const int items = first[2 * streams], step = gridDim.x;
  const float inv_kvh = 1.f / kvh;
  auto take = [&](int round) { return round * step + (round & 1 ? step - 1 - (int)blockIdx.x : (int)blockIdx.x); };
  auto item_of = [&](int it) {
    int lo = 0, hi = 2 * streams;     // the last entry with first <= it
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= it) lo = mid;
      else hi = mid;
    }
    Item i;
    i.b = order[lo < streams ? lo : lo - streams];
    const int r = it - first[lo], len = lens[i.b], size = chunk_of(len);
    const int c = (int)((r + 0.5f) * inv_kvh);   // r / kvh, exact below 2^17
    i.kh = r - c * kvh;
    i.rec = lo < streams ? c : len / size;
    const size_t row = a.c.row(slots[i.b], i.kh, i.rec * size);
    i.K = a.c.K + row * D;
    i.V = a.c.V + row * D;
    i.Ks = a.c.Ks + row;
    i.Vs = a.c.Vs + row;
    i.n = min(size, len - i.rec * size);
    return i;
  };

  // ---- loads run a stage ahead of the arithmetic, into the next item too
  constexpr int kPieces = D / 16, kRows = 32 / kPieces, kCopies = kTake / kRows;   // a lane copies a piece of every kRows-th position
  const int my_row = lane / kPieces, my_piece = lane % kPieces;
  int load_round = 0, load_it = take(0), load_j = kTake * warp, load_slot = 0;
  Item li{};
  if (load_it < items) li = item_of(load_it);
  auto load = [&]() {
    if (load_it < items) {
      Ring<D>& s = sm.ring[warp][load_slot];
      const int left = li.n - load_j;
      const size_t off = (size_t)(load_j + my_row) * D + 16 * my_piece;
      const uint8_t *pk = li.K + off, *pv = li.V + off;
      const float *ps = li.Ks + load_j + lane, *pz = li.Vs + load_j + lane;
      if (left >= kTake) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int at = piece<D>(my_row + kRows * i, my_piece);
          copy16(s.k + at, pk + kRows * D * i);
          copy16(s.v + at, pv + kRows * D * i);
        }
        copy4(s.ks + lane, ps);
        copy4(s.vs + lane, pz);
      } else {                        // the stream's last positions, then zeros
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int at = piece<D>(my_row + kRows * i, my_piece);
          const bool live = my_row + kRows * i < left;
          copy16_or_zero(s.k + at, live ? pk + kRows * D * i : li.K, live);
          copy16_or_zero(s.v + at, live ? pv + kRows * D * i : li.V, live);
        }
        const bool live = lane < left;
        copy4_or_zero(s.ks + lane, live ? ps : li.Ks, live);
        copy4_or_zero(s.vs + lane, live ? pz : li.Vs, live);
      }
      load_slot = load_slot + 1 == kRing ? 0 : load_slot + 1;
      load_j += kStage;
      if (load_j - kTake * warp >= li.n) {
        load_it = take(++load_round);
        load_j = kTake * warp;
        if (load_it < items) li = item_of(load_it);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) load();

  int slot = 0;
  constexpr int kPer = D / 64;        // 16-byte pieces of a K row per lane
  uint32_t q[kPer][4][2];
  float qf = 0.f;
  // this lane's query row (head g), read while the item before is merged
  uint4 x[kPer][2];
  auto ask = [&](const Item& i) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        x[j][u] = make_uint4(0, 0, 0, 0);
        if (g < G) x[j][u] = *reinterpret_cast<const uint4*>(a.Q + ((size_t)i.b * a.qh + i.kh * G + g) * D + 16 * (kPer * t + j) + 8 * u);
      }
  };
  Item i{};
  if (take(0) < items) {
    i = item_of(take(0));
    ask(i);
  }
  for (int round = 0; take(round) < items; ++round) {
    // ---- as fp16 of about its own magnitude
    {
      float mx = 0.f, down, up;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t w[4] = {x[j][u].x, x[j][u].y, x[j][u].z, x[j][u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(w[e])), fabsf(bf_hi(w[e]))));
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      row_scale(mx, down, up);
      qf = a.scale_log2 * up;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t w[4] = {x[j][u].x, x[j][u].y, x[j][u].z, x[j][u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 v = __floats2half2_rn(bf_lo(w[e]) * down, bf_hi(w[e]) * down);
            q[j][2 * u + e / 2][e & 1] = *reinterpret_cast<const uint32_t*>(&v);
          }
        }
    }
    constexpr int kTiles = D / 16;
    float o[kTiles][4], m = -1e30f, l = 0.f;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    for (int j0 = 0; j0 < i.n; j0 += kStage) {
      load();
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      __syncwarp();
      const Ring<D>& s = sm.ring[warp][slot];
      slot = slot + 1 == kRing ? 0 : slot + 1;
      const int left = i.n - j0 - kTake * warp;   // positions of this warp's
      if (left > 0) {
        constexpr int kN = kTake / 8;
        float c[kN][4];
#pragma unroll
        for (int nt = 0; nt < kN; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          uint32_t w[kN][4];
#pragma unroll
          for (int nt = 0; nt < kN; ++nt) {
            const uint4 k = *reinterpret_cast<const uint4*>(s.k + piece<D>(8 * nt + g, kPer * t + j));
            w[nt][0] = k.x; w[nt][1] = k.y; w[nt][2] = k.z; w[nt][3] = k.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int nt = 0; nt < kN; ++nt) {
              uint32_t b0, b1;
              codes4<FMT>(w[nt][e], b0, b1);
              mma16816(c[nt], q[j][e][0], 0u, q[j][e][1], 0u, b0, b1);
            }
        }
        // head g, positions 8 nt + 2 t + e
        float p[kN][2], vs[kN][2], mx = -1e30f;
#pragma unroll
        for (int nt = 0; nt < kN; ++nt) {
          const float2 kf = *reinterpret_cast<const float2*>(&s.ks[8 * nt + 2 * t]);
          const float2 vf = *reinterpret_cast<const float2*>(&s.vs[8 * nt + 2 * t]);
          vs[nt][0] = vf.x;
          vs[nt][1] = vf.y;
          p[nt][0] = c[nt][0] * (kf.x * qf);
          p[nt][1] = c[nt][1] * (kf.y * qf);
        }
        if (left < kTake) {
#pragma unroll
          for (int nt = 0; nt < kN; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (8 * nt + 2 * t + e >= left) p[nt][e] = -INFINITY;
        }
#pragma unroll
        for (int nt = 0; nt < kN; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) mx = fmaxf(mx, p[nt][e] + fmaxf(log2_fast(vs[nt][e]), -100.f));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (__any_sync(0xffffffffu, mx > m + 8.f)) {
          const float mn = mx > m + 8.f ? mx : m, f = exp2_fast(m - mn);
          l = scaled_down(l, m - mn);
          m = mn;
          const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            o[j][0] *= f0;
            o[j][1] *= f1;
            o[j][2] *= f0;
            o[j][3] *= f1;
          }
        }
        uint32_t pb[kN];
#pragma unroll
        for (int nt = 0; nt < kN; ++nt) {
          const float p0 = exp2_fast(p[nt][0] - m), p1 = exp2_fast(p[nt][1] - m);
          l += p0 + p1;
          const __half2 w = __floats2half2_rn(p0 * vs[nt][0], p1 * vs[nt][1]);
          pb[nt] = *reinterpret_cast<const uint32_t*>(&w);
        }
#pragma unroll
        for (int u = 0; u < kTake / 16; ++u) {
          uint32_t v[4][D / 32];      // this lane's D / 8 codes of positions 16u + 2t, + 1, + 8, + 9
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int token = 16 * u + 2 * t + (r & 1) + 8 * (r >> 1);
            if (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(s.v + piece<D>(token, g));
              v[r][0] = x.x; v[r][1] = x.y; v[r][D / 32 - 2] = x.z; v[r][D / 32 - 1] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(s.v + piece<D>(token, g >> 1) + 8 * (g & 1));
              v[r][0] = x.x; v[r][1] = x.y;
            }
          }
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            const uint32_t sel = j & 1 ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            codes4<FMT>(__byte_perm(v[0][j / 2], v[1][j / 2], sel), a0, a1);
            codes4<FMT>(__byte_perm(v[2][j / 2], v[3][j / 2], sel), a2, a3);
            mma16816(o[j], a0, a1, a2, a3, pb[2 * u], pb[2 * u + 1]);
          }
        }
      }
      __syncwarp();                   // every lane has read the slot before it is loaded again
    }

    // ---- the item's record from the four warps'
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const int used = slot == 0 ? kRing - 1 : slot - 1;
    WarpOut<D>& out = *reinterpret_cast<WarpOut<D>*>(&sm.ring[warp][used]);
    if (t == 0) {
      sm.m[warp][g] = m;
      sm.l[warp][g] = l;
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      const int d = D / 8 * g + 2 * j;
      *reinterpret_cast<float2*>(&out[2 * t][d]) = make_float2(o[j][0], o[j][2]);
      *reinterpret_cast<float2*>(&out[2 * t + 1][d]) = make_float2(o[j][1], o[j][3]);
    }
    const Item done = i;
    if (take(round + 1) < items) {
      i = item_of(take(round + 1));
      ask(i);
    }
    __syncthreads();
#pragma unroll 1
    for (int r = warp; r < G; r += kWarpsPerItem) {
      float f[kWarpsPerItem], mx = sm.m[0][r], den = 0.f;
#pragma unroll
      for (int w = 1; w < kWarpsPerItem; ++w) mx = fmaxf(mx, sm.m[w][r]);
#pragma unroll
      for (int w = 0; w < kWarpsPerItem; ++w) {
        f[w] = exp2_fast(sm.m[w][r] - mx);
        den += scaled_down(sm.l[w][r], sm.m[w][r] - mx);
      }
      const size_t rec = a.record(done.b, done.kh * G + r, a.p_chunks + done.rec);
#pragma unroll
      for (int d = 2 * lane; d < D; d += 64) {
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarpsPerItem; ++w) {
          const float2 v = *reinterpret_cast<const float2*>(&(*reinterpret_cast<const WarpOut<D>*>(&sm.ring[w][used]))[r][d]);
          acc.x = fmaf(v.x, f[w], acc.x);
          acc.y = fmaf(v.y, f[w], acc.y);
        }
        *reinterpret_cast<float2*>(a.rec_o + rec * D + d) = acc;
      }
      if (lane == 0) a.rec_ml[rec] = make_float2(mx, den);
    }
    __syncthreads();                  // the slots are loaded again
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  pdl_wait();                         // done means done: the prefix's records are there too
}

// One head of one stream to a warp: its records in ascending order, a lane
// d / 32 elements.  The kernel is a chain of latencies, so everything is
// asked for at once: the maxima and sums (a record to a lane), and the first
// outputs before their weights are known (16 of them: a lone stream of 4096
// took 7.2 us with 8 and 6.9 with 16, 32 streams behind a prefix 46.8 and 45.6).  It
// starts with the chunks (programmatic dependent launch) and ends 2 to 5 us
// behind them.
constexpr int kMergeWarps = 4, kMergeAhead = 16;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) k_kv8_merge(AttendArgs a) {
  constexpr int E = D / 32;
  using Part = typename std::conditional<E == 4, float4, float2>::type;
  const int at = blockIdx.x * kMergeWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (at >= a.B * a.qh) return;
  const int b = at / a.qh, h = at - b * a.qh;
  int slot, len;
  const bool live = a.live(b, slot, len);   // inputs of the call: not written by the kernels before
  pdl_wait();
  if (!live) return;
  const int n = a.p_chunks + chunks_of(len);
  const Part* o = reinterpret_cast<const Part*>(a.rec_o + a.record(b, h, 0) * D) + lane;
  const float2* ml = a.rec_ml + a.record(b, h, 0);
  float2 mine = lane < n ? ml[lane] : make_float2(-FLT_MAX, 0.f);
  Part part[kMergeAhead];
#pragma unroll
  for (int k = 0; k < kMergeAhead; ++k)
    if (k < n) part[k] = o[k * 32];
  float mx = mine.x;
  for (int r = lane + 32; r < n; r += 32) mx = fmaxf(mx, ml[r].x);
  mx = warp_max(mx);
  float den = 0.f, acc[E] = {};
  for (int r0 = 0; r0 < n; r0 += 32) {
    if (r0) mine = r0 + lane < n ? ml[r0 + lane] : make_float2(-FLT_MAX, 0.f);
    const float f = exp2f(mine.x - mx);
    den += mine.y * exp2f(fmaxf(mine.x - mx, -120.f)) * exp2f(fminf(mine.x - mx + 120.f, 0.f));   // scaled_down, not approximated
    for (int k0 = 0; k0 < 32 && r0 + k0 < n; k0 += kMergeAhead) {
      Part next[kMergeAhead];
      const int ahead = r0 + k0 + kMergeAhead;
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k)
        if (ahead + k < n) next[k] = o[(ahead + k) * 32];
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, k0 + k);
        if (r0 + k0 + k < n) {
          const float* p = reinterpret_cast<const float*>(&part[k]);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(p[e], fk, acc[e]);
        }
        part[k] = next[k];
      }
    }
  }
  den = warp_sum(den);
  const float inv = n == 0 ? 0.f : 1.f / den;   // no positions: zeros
  __nv_bfloat162 out[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = __floats2bfloat162_rn(n == 0 ? 0.f : acc[2 * e] * inv, n == 0 ? 0.f : acc[2 * e + 1] * inv);
  bf16* to = a.O + ((size_t)b * a.qh + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E / 2; ++e) *reinterpret_cast<__nv_bfloat162*>(to + 2 * e) = out[e];
}

// CTAs of the chunk kernel that an SM holds at once: three, but two where the table of a large batch (20 bytes a row;
// head_dim 128 from 448 rows on) leaves no room for a third.  The items are dealt out evenly to all CTAs of the grid,
// so none of them may have to wait for another's end: 460 streams of 1000 positions, 32 + 2 x 4 heads of 128, took
// 186 us with a grid of three CTAs an SM and take 143 with two (440 streams, three CTAs: 120).
int ctas_per_sm(size_t smem) {
  constexpr size_t kSmShared = 228 * 1024, kReserved = 1024;   // of an SM; of a CTA besides its own
  return smem + kReserved <= kSmShared / 3 ? 3 : 2;
}

template <int D, int FMT>
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
  const size_t most = sizeof(ChunkSmem<D>) + 5 * kMaxBatch * sizeof(int), items = (size_t)a.B * a.c.kvh * a.own_chunks;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(
      done, [&] { return cudaFuncSetAttribute(k_kv8_chunk<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most); });
  if (e == cudaSuccess && a.p_chunks > 0) e = launch_kv8_prefix(a, FMT, D, s);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(ChunkSmem<D>) + 5 * a.B * sizeof(int);
  const unsigned grid = (unsigned)std::min<size_t>(items, kSms * ctas_per_sm(smem));
  e = launch_k(a.p_chunks > 0, k_kv8_chunk<D, FMT>, dim3(grid), dim3(kWarpsPerItem * 32), smem, s, a);
  if (e != cudaSuccess) return e;
  return launch_k(true, k_kv8_merge<D>, dim3((a.B * a.qh + kMergeWarps - 1) / kMergeWarps), dim3(kMergeWarps * 32), 0, s, a);
}

bool shapes_ok(int B, int qh, int kvh, int d) {
  return B >= 1 && B <= kMaxBatch && kvh >= 1 && qh >= 1 && qh % kvh == 0 && qh / kvh <= kMaxGroup && qh <= 1024 &&
         (d == 64 || d == 128);
}

size_t records(int ctx_cap, int prefix_len, int kvh) { return (size_t)most_prefix_chunks(prefix_len, kvh) + most_chunks(ctx_cap); }

bm_status attend(const char* who, const bm_kv8_cache* c, const bm_kv8_cache* p, int p_slot, int p_len, const uint16_t* Q,
                 const int32_t* slots, const int32_t* lens, int q_heads, float scale, uint16_t* O, int B, void* ws,
                 size_t ws_bytes, void* stream) {
  auto refuse = [&](bm_status st, const std::string& what) { return set_error(st, std::string(who) + ": " + what); };
  AttendArgs a{};
  bm_status st = check_cache(c, who, &a.c);
  if (st != BM_OK) return st;
  if (p) {
    if ((st = check_cache(p, who, &a.p)) != BM_OK) return st;
    if (p->format != c->format || p->kv_heads != c->kv_heads || p->head_dim != c->head_dim)
      return refuse(BM_ERR_INVALID_ARG, "the prefix's cache must have the streams' format, kv_heads and head_dim");
    if (p_slot < 0 || p_slot >= p->slots) return refuse(BM_ERR_INVALID_ARG, "prefix_slot out of range");
    if (p_len < 0 || p_len > p->ctx_cap) return refuse(BM_ERR_CTX_CAP, "prefix_len outside the slot");
  }
  if (!Q || !slots || !lens || !O || !ws) return refuse(BM_ERR_INVALID_ARG, "null pointer");
  if (((uintptr_t)Q | (uintptr_t)O | (uintptr_t)ws) & 15)
    return refuse(BM_ERR_INVALID_ARG, "Q, O and the workspace must be 16-byte aligned");
  if (((uintptr_t)slots | (uintptr_t)lens) & 3) return refuse(BM_ERR_INVALID_ARG, "slots and lens must be 4-byte aligned");
  if (!shapes_ok(B, q_heads, c->kv_heads, c->head_dim))
    return refuse(BM_ERR_INVALID_ARG, "need 1 <= B <= 1024, q_heads <= 1024 and a multiple of kv_heads, at most 8 query heads per kv head");
  if (!(scale > 0.f) || !(scale < INFINITY)) return refuse(BM_ERR_INVALID_ARG, "scale must be positive and finite");
  const size_t need = kv8_workspace_bytes(B, q_heads, c->kv_heads, c->head_dim, c->ctx_cap, p_len);
  if (ws_bytes < need)
    return refuse(BM_ERR_INVALID_ARG, "workspace of " + std::to_string(ws_bytes) + " bytes, " + std::to_string(need) + " needed");
  a.p_slot = p_slot;
  a.p_len = p_len;
  a.p_chunk = prefix_chunk(p_len, c->kv_heads);
  a.p_chunks = prefix_chunks(p_len, c->kv_heads);
  a.Q = reinterpret_cast<const bf16*>(Q);
  a.slots = slots;
  a.lens = lens;
  a.O = reinterpret_cast<bf16*>(O);
  a.B = B;
  a.qh = q_heads;
  a.own_chunks = most_chunks(c->ctx_cap);
  a.rec_o = static_cast<float*>(ws);
  a.rec_ml = reinterpret_cast<float2*>(a.rec_o + a.record(B, 0, 0) * c->head_dim);
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4 = c->format == BM_KV8_E4M3, d128 = c->head_dim == 128;
  const cudaError_t e = d128 ? (e4 ? launch_attend<128, BM_KV8_E4M3>(a, s) : launch_attend<128, BM_KV8_INT8>(a, s))
                             : (e4 ? launch_attend<64, BM_KV8_E4M3>(a, s) : launch_attend<64, BM_KV8_INT8>(a, s));
  if (e != cudaSuccess) return refuse(BM_ERR_CUDA, cudaGetErrorString(e));
  return ok();
}

}  // namespace
}  // namespace bm

extern "C" {

size_t kv8_workspace_bytes(int B, int q_heads, int kv_heads, int head_dim, int ctx_cap, int prefix_len) {
  using namespace bm;
  if (!shapes_ok(B, q_heads, kv_heads, head_dim) || ctx_cap < 1 || prefix_len < 0) return 0;
  return (size_t)B * q_heads * records(ctx_cap, prefix_len, kv_heads) * (head_dim + 2) * sizeof(float);
}

bm_status kv8_attend(const bm_kv8_cache* c, const uint16_t* Q, const int32_t* slots, const int32_t* lens, int q_heads,
                     float scale, uint16_t* O, int B, void* ws, size_t ws_bytes, void* stream) {
  return bm::attend("kv8_attend", c, nullptr, 0, 0, Q, slots, lens, q_heads, scale, O, B, ws, ws_bytes, stream);
}

bm_status kv8_attend_prefix(const bm_kv8_cache* c, const bm_kv8_cache* prefix, int prefix_slot, int prefix_len,
                            const uint16_t* Q, const int32_t* slots, const int32_t* lens, int q_heads, float scale,
                            uint16_t* O, int B, void* ws, size_t ws_bytes, void* stream) {
  if (!prefix) return bm::set_error(BM_ERR_INVALID_ARG, "kv8_attend_prefix: null prefix cache");
  return bm::attend("kv8_attend_prefix", c, prefix, prefix_slot, prefix_len, Q, slots, lens, q_heads, scale, O, B, ws,
                    ws_bytes, stream);
}

}  // extern "C"
