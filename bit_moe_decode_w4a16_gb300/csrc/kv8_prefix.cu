// Attention over a prefix that a batch shares, computed once for all of it.
//
// The query rows of a kv head are gathered from the whole batch (row r is
// head r % G of its group of stream r / G), 128 at a time: over a prefix of P
// positions that is a dense product of 128 x P x d, and the prefix's codes
// are read and converted once per 128 rows instead of once per stream.  A CTA
// takes 128 rows and one or more chunks of the prefix, one behind the other,
// and leaves a record (o, m, l) per row and chunk; the records are merged with
// those of the streams' own positions.
//
// Per tile of 128 positions, on the 5th-generation tensor cores (fp16
// operands, fp32 sums in tensor memory):
//   S[row][position] = Q K^T, MMAs of 128 x 128 x 16, both operands in shared
//     memory (K-major, 128-byte swizzle);
//   p and the weights p * vs as in kv8_attend.cu, in two sweeps of S, two
//     positions to an instruction (f32x2); the weights go to tensor memory as
//     the fp16 A operand.  S is read in the fragment layout (2 rows x 32
//     positions to a thread): with a row to a thread, every thread reads every
//     position's scales, and those reads alone took 2000 cycles a tile;
//   O[row][element] += P V, MMAs of 128 x d x 16, A in tensor memory, B = V^T
//     in shared memory, positions contiguous (K-major).
// Eight warps do the softmax; eight convert codes to fp16 (V is transposed on
// the way, 8 positions x 4 bytes to a thread; its elements are stored at row
// d / 4 (e % 4) + e / 4 of B so that a warp's stores meet no bank conflict,
// and O's columns come out in that order); one lane issues the MMAs.
// K, V and S have two buffers each, so the next tile's scores are made
// while this one's softmax runs, and O is waited for only to rescale it.
//
// An MMA takes about 100 cycles whether N is 16 or 128, so the tile is as
// wide as tensor memory allows (two S of 128 columns and O; 64-position tiles
// at two CTAs an SM measured 55 us where these took 44).
//
// 32 streams of 8 heads a group over 32768 positions of 4 kv heads of 128: 43
// us with the merge, 402 TFLOP/s; the kernel alone 34, of which 14 tiles 1.9
// each.  The chain of a tile bounds it, scores to weights to product: a tile of
// 128 x 128 weights is about 9 thousand warp instructions, which keep the issue
// slots busy for half of the time and the tensor pipe for a fifth, while the
// softmax warps wait for tensor memory.  Storing the records takes 3.5 us.  A CTA walks over consecutive chunks
// rather than leave them to a second wave (128 streams behind 8192: 87 -> 75
// us); taking a chunk's tiles of query rows through one CTA instead took 48
// us, as query rows and records then wait for each other.
//
// Every wait is bounded.  A wait that gives up leaves NaN in its CTA's
// records, and so in the output rows.
#include <type_traits>

#include "kv8_attend.cuh"
#include "tc_ptx.cuh"

namespace bm {
namespace {

using namespace kv8;

constexpr int kRows = 128, kTokens = 128;          // a tile
constexpr int kSoftmax = 256, kConvert = 256, kThreads = kSoftmax + kConvert + 32;
constexpr uint32_t kTmemCols = 512;                // S of even and of odd tiles, O, P of even and of odd tiles
constexpr uint32_t kWaitLimit = 1u << 18;          // polls of ~3.7 us: a wait gives up after about a second

template <int D>
struct PrefixSmem {
  uint8_t q[kRows * D * 2];                        // [d / 64][row][64] fp16, swizzled
  uint8_t k[2][kTokens * D * 2];                   // [d / 64][position][64]
  uint8_t v[2][kTokens * D * 2];                   // [position / 64][element][64]
  // scales and log2 of V's, of four tiles: they are written with a tile's K, when the softmax may be two tiles back
  float ks[4][kTokens], vs[4][kTokens], lg[4][kTokens];
  float up[kRows];
  // by the tile's parity; their phase is the tile's half
  uint64_t k_full[2], v_full[2], s_ready[2], p_ready[2], o_ready[2], drained;
  uint32_t tmem;
  int gave_up;
};
// 16-byte piece c of row r of a K-major operand of `rows` rows: 128-byte rows of 64 fp16, pieces swizzled by the row.
__device__ __forceinline__ uint32_t piece(int rows, int r, int c) { return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

// Descriptor of a K-major operand with the 128-byte swizzle: 8-row atoms of
// 1024 bytes (SBO), LBO unused (encoded 1), layout type 2; the start address
// moves by 32 bytes per 16 values of K.
__device__ __forceinline__ uint64_t operand(uint32_t base, int rows, int k16) {
  const uint32_t at = base + (k16 >> 2) * rows * 128 + (k16 & 3) * 32;
  return (uint64_t)((at >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) k_kv8_prefix(AttendArgs a, int per_cta) {
  extern __shared__ unsigned char raw[];
  const uint32_t raw_at = tc::smem_u32(raw);
  PrefixSmem<D>& sm = *reinterpret_cast<PrefixSmem<D>*>(raw + ((1024u - (raw_at & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk0 = blockIdx.x * per_cta, row0 = blockIdx.y * kRows, kh = blockIdx.z;
  const int kvh = a.c.kvh, G = a.qh / kvh, rows = a.B * G;
  // the CTA's chunks lie one behind the other, each of `per_chunk` tiles but for the prefix's last
  const int j0 = chunk0 * a.p_chunk, n = (int)min((long long)per_cta * a.p_chunk, (long long)(a.p_len - j0));
  const int tiles = (n + kTokens - 1) / kTokens, per_chunk = a.p_chunk / kTokens;
  const float inv_g = 1.f / G;
  auto stream_of = [&](int r) { return (int)((r + 0.5f) * inv_g); };   // r / G, exact below 2^20
  const size_t at = a.p.row(a.p_slot, kh, j0);
  pdl_trigger();                                   // the streams' own chunks do not depend on this

  if (warp == kSoftmax / 32) {
    tc::tmem_alloc(tc::smem_u32(&sm.tmem), kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tc::smem_u32(&sm.k_full[b]), kConvert);
      tc::mbar_init(tc::smem_u32(&sm.v_full[b]), kConvert);
      tc::mbar_init(tc::smem_u32(&sm.p_ready[b]), kSoftmax);
      tc::mbar_init(tc::smem_u32(&sm.s_ready[b]), 2);
      tc::mbar_init(tc::smem_u32(&sm.o_ready[b]), 1);
    }
    tc::mbar_init(tc::smem_u32(&sm.drained), 1);
    tc::fence_mbar_init();
    sm.gave_up = 0;
  }
  // ---- the query rows as fp16 of about their own magnitude, d / 8 lanes to a row
  constexpr int kPieces = D / 8;
  if (tid < kSoftmax + kConvert)
#pragma unroll
  for (int u = tid; u < kRows * kPieces; u += kSoftmax + kConvert) {
    const int at_row = u / kPieces, c = u % kPieces, r = row0 + at_row, b = stream_of(r), h = kh * G + r - b * G;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < rows) x = *reinterpret_cast<const uint4*>(a.Q + ((size_t)b * a.qh + h) * D + 8 * c);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float mx = 0.f, down, up;
#pragma unroll
    for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(w[e])), fabsf(bf_hi(w[e]))));
#pragma unroll
    for (int o = kPieces / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    row_scale(mx, down, up);
    uint32_t f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 v = __floats2half2_rn(bf_lo(w[e]) * down, bf_hi(w[e]) * down);
      f[e] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(sm.q + piece(kRows, at_row, c)) = make_uint4(f[0], f[1], f[2], f[3]);
    if (c == 0) sm.up[at_row] = up;
  }
  tc::fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t s_cols = sm.tmem, o_cols = s_cols + 2 * kTokens, p_cols = o_cols + 128;
  // tile i's phase of a pair of barriers.  No thread can miss one: a tile's barrier completes again only after
  // every thread that waits for it has arrived at another barrier of that tile.
  // try_wait suspends the thread: sixteen polling warps would take the issue slots of the one that works.
  auto wait = [](uint64_t* bars, int i) { return tc::mbar_wait(tc::smem_u32(&bars[i & 1]), i >> 1 & 1, kWaitLimit); };
  bool ok = true;

  if (warp == (kSoftmax + kConvert) / 32) {
    // ---------------- MMAs: issuing one takes as long as running it, so a lane does nothing else
    if (lane == 0) {
      const uint32_t qk = tc::idesc_f16_f32(kRows, kTokens), pv = tc::idesc_f16_f32(kRows, D);
      const uint32_t q_at = tc::smem_u32(sm.q);
      int in_chunk = 0;                            // tiles of the chunk before the next output's
      // tile i's scores, once its K is there
      auto issue_scores = [&](int i) {
        if (!wait(sm.k_full, i)) return false;
        tc::fence_after_sync();
        const uint32_t k_at = tc::smem_u32(sm.k[i & 1]);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_f16_ss(s_cols + (i & 1) * kTokens, operand(q_at, kRows, k), operand(k_at, kTokens, k), qk, k > 0);
        tc::mma_commit(tc::smem_u32(&sm.s_ready[i & 1]));
        tc::mbar_arrive(tc::smem_u32(&sm.s_ready[i & 1]));   // a release by this thread: it passes the scales on
        return true;
      };
      // tile i's part of O, once its weights and its V are there
      auto issue_output = [&](int i) {
        if (!wait(sm.v_full, i) || !wait(sm.p_ready, i)) return false;
        tc::fence_after_sync();
        const uint32_t v_at = tc::smem_u32(sm.v[i & 1]);
#pragma unroll
        for (int k = 0; k < kTokens / 16; ++k)
          tc::mma_f16_tmem_a(o_cols, p_cols + (i & 1) * (kTokens / 2) + 8 * k, operand(v_at, D, k), pv, in_chunk > 0 || k > 0);
        if (++in_chunk == per_chunk) in_chunk = 0;
        tc::mma_commit(tc::smem_u32(&sm.o_ready[i & 1]));
        return true;
      };
      ok = issue_scores(0) && (tiles < 2 || issue_scores(1));
      // scores go where those of two tiles before were, which that tile's weights say have been read
      for (int i = 0; ok && i < tiles; ++i) ok = issue_output(i) && (i + 2 >= tiles || issue_scores(i + 2));
      // nothing of this CTA's is in flight when it ends
      tc::mma_commit(tc::smem_u32(&sm.drained));
      if (!tc::mbar_wait(tc::smem_u32(&sm.drained), 0, kWaitLimit)) ok = false;
    }
    __syncwarp();
  } else if (warp >= kSoftmax / 32) {
    // ---------------- conversion: warp w takes positions 16 w .. of a tile
    const int cw = warp - kSoftmax / 32, ct = tid - kSoftmax;
    constexpr int kRowsAt = D == 128 ? 4 : 8;      // K rows to a warp's load
    constexpr int kK = 16 / kRowsAt;      // loads of 16 codes
    constexpr int kG = D == 128 ? 2 : 1;           // groups of 8 positions to a thread
    const int k_row = lane / (32 / kRowsAt), k_piece = lane % (32 / kRowsAt);
    const int v_word = D == 128 ? lane : lane & 15, v_half = D == 128 ? 0 : lane >> 4;
    const uint8_t *K = a.p.K + at * D, *V = a.p.V + at * D;
    uint4 kr[kK];
    uint32_t vr[kG][8];
    float scale;                                   // K's in the first half of the threads, V's in the others
    auto load = [&](int i) {
      const int t0 = i * kTokens + 16 * cw;        // positions of the chunk
      const bool whole = t0 + 16 <= n;
#pragma unroll
      for (int r = 0; r < kK; ++r) {
        const int p = t0 + kRowsAt * r + k_row;
        kr[r] = whole || p < n ? ldg_nc_v4(K + (size_t)p * D + 16 * k_piece) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int q = 0; q < kG; ++q)
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int p = t0 + (D == 128 ? 8 * q : 8 * v_half) + r;
          vr[q][r] = whole || p < n ? __ldg(reinterpret_cast<const uint32_t*>(V + (size_t)p * D) + v_word) : 0u;
        }
      const int p = i * kTokens + (ct & (kTokens - 1));
      scale = p < n ? __ldg((ct < kTokens ? a.p.Ks : a.p.Vs) + at + p) : 0.f;
    };
    load(0);
    for (int i = 0; i < tiles; ++i) {
      // the K buffer is free once tile i - 2 has its scores
      if (i > 1) {
        if (lane == 0) ok = wait(sm.s_ready, i - 2);
        if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) break;
      }
      uint8_t *k_to = sm.k[i & 1], *v_to = sm.v[i & 1];
      if (ct < kTokens) {
        sm.ks[i & 3][ct] = scale;
      } else {
        sm.vs[i & 3][ct - kTokens] = scale;
        sm.lg[i & 3][ct - kTokens] = fmaxf(log2_fast(scale), -100.f);
      }
#pragma unroll
      for (int r = 0; r < kK; ++r) {
        const int row = 16 * cw + kRowsAt * r + k_row;
        uint32_t f[8];
        codes4<FMT>(kr[r].x, f[0], f[1]);
        codes4<FMT>(kr[r].y, f[2], f[3]);
        codes4<FMT>(kr[r].z, f[4], f[5]);
        codes4<FMT>(kr[r].w, f[6], f[7]);
        // the pieces of the row's second half in the other order: no bank conflict
        const bool swap = k_piece & 4;
        *reinterpret_cast<uint4*>(k_to + piece(kTokens, row, 2 * k_piece + swap)) =
            swap ? make_uint4(f[4], f[5], f[6], f[7]) : make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4*>(k_to + piece(kTokens, row, 2 * k_piece + !swap)) =
            swap ? make_uint4(f[0], f[1], f[2], f[3]) : make_uint4(f[4], f[5], f[6], f[7]);
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(tc::smem_u32(&sm.k_full[i & 1]));
      if (i > 1) {
        if (lane == 0) ok = wait(sm.o_ready, i - 2);
        if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) break;
      }
#pragma unroll
      for (int q = 0; q < kG; ++q) {
        const int group = 2 * cw + (D == 128 ? q : v_half);   // of 8 positions
        uint32_t f[4][4];                          // [element of the word][pair of positions]
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          codes4<FMT>(__byte_perm(vr[q][2 * r], vr[q][2 * r + 1], 0x5140), f[0][r], f[1][r]);
          codes4<FMT>(__byte_perm(vr[q][2 * r], vr[q][2 * r + 1], 0x7362), f[2][r], f[3][r]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(v_to + piece(D, D / 4 * e + v_word, group)) = make_uint4(f[e][0], f[e][1], f[e][2], f[e][3]);
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(tc::smem_u32(&sm.v_full[i & 1]));
      if (i + 1 < tiles) load(i + 1);
    }
  } else {
    // ---------------- softmax: 16 rows to a warp.  Thread (g, t) has rows g and g + 8 of them and positions
    // 8 j + 2 t and the next, j = 0 .. 15.
    const int row = 32 * (warp & 3) + 16 * (warp >> 2), g = lane >> 2, t = lane & 3;
    const uint32_t lanes = (uint32_t)row << 16;
    float qf[2], m[2], l[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      qf[r] = a.scale_log2 * sm.up[row + g + 8 * r];
      m[r] = -1e30f;
      l[r] = 0.f;
    }
    // a chunk's records, once its last tile `i` is in O.  B's row n is element 4 (n % (d / 4)) + n / (d / 4): what a
    // thread has of the four quarters of the columns are 4 consecutive elements
    auto store = [&](int i, int chunk) {
      if (lane == 0) ok = wait(sm.o_ready, i);
      if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) return;
      tc::fence_after_sync();
      float4* to[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        const int q = row0 + row + g + 8 * r, b = stream_of(q);
        to[r] = nullptr;
        if (q < rows) {
          const size_t rec = a.record(b, kh * G + q - b * G, chunk);
          if (t == 0) a.rec_ml[rec] = make_float2(m[r], l[r]);
          to[r] = reinterpret_cast<float4*>(a.rec_o + rec * D) + 2 * t;
        }
        m[r] = -1e30f;
        l[r] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < D / 4; j += 8) {
        uint32_t o[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) tc::tmem_ld_frag8(o_cols + lanes + k * (D / 4) + j, o[k]);
        tc::tmem_wait_ld();
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (to[r]) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              to[r][j + e] = make_float4(__uint_as_float(o[0][2 * r + e]), __uint_as_float(o[1][2 * r + e]), __uint_as_float(o[2][2 * r + e]), __uint_as_float(o[3][2 * r + e]));
          }
      }
    };
    int in_chunk = 0, chunk = chunk0;
    for (int i = 0; i < tiles; ++i, ++in_chunk) {
      if (in_chunk == per_chunk) {
        store(i - 1, chunk++);
        if (!ok) break;
        in_chunk = 0;
      }
      // tile i's scores, and tile i - 2's output, which read the weights that these will overwrite
      if (lane == 0) ok = wait(sm.s_ready, i) && (i < 2 || wait(sm.o_ready, i - 2));
      if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) break;
      tc::fence_after_sync();
      const int here = n - i * kTokens, left = here - 2 * t, b = i & 3;   // positions of the chunk from here on
      const uint32_t s_at = s_cols + lanes + (i & 1) * kTokens, p_at = p_cols + lanes + (i & 1) * (kTokens / 2);
      auto pair = [&](const float* of, int at) { return *reinterpret_cast<const uint64_t*>(of + at + 2 * t); };
      float mx[2] = {-1e30f, -1e30f};
      auto largest = [&](auto whole) {             // a branch per score would cost more than the score
#pragma unroll
        for (int c = 0; c < kTokens; c += 32) {
          uint32_t v[16];
          tc::tmem_ld_frag32(s_at + c, v);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t ks = pair(sm.ks[b], c + 8 * j), lg = pair(sm.lg[b], c + 8 * j);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint64_t x = fma2(mul2((uint64_t)v[4 * j + 2 * r] | (uint64_t)v[4 * j + 2 * r + 1] << 32, ks), pack2(qf[r], qf[r]), lg);
              if (decltype(whole)::value) {
                mx[r] = fmaxf(mx[r], fmaxf(first(x), second(x)));
              } else {
                if (c + 8 * j < left) mx[r] = fmaxf(mx[r], first(x));
                if (c + 8 * j + 1 < left) mx[r] = fmaxf(mx[r], second(x));
              }
            }
          }
        }
      };
      if (here >= kTokens) largest(std::true_type());
      else largest(std::false_type());
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
        // each row by itself: its neighbours are other streams'
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float mn = mx[r] > m[r] + 8.f ? mx[r] : m[r];
          f[r] = exp2_fast(m[r] - mn);
          l[r] = scaled_down(l[r], m[r] - mn);
          m[r] = mn;
        }
        if (in_chunk > 0) {                        // O holds the chunk's tiles before
          if (lane == 0) ok = wait(sm.o_ready, i - 1);
          if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) break;
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[16];
            tc::tmem_ld_frag32(o_cols + lanes + c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f[k >> 1 & 1]);
            tc::tmem_st_frag32(o_cols + lanes + c, o);
          }
        }
      }
      auto weights = [&](auto whole) {
#pragma unroll
        for (int c = 0; c < kTokens; c += 32) {
          uint32_t v[16], w[8];
          tc::tmem_ld_frag32(s_at + c, v);
          tc::tmem_wait_ld();
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t ks = pair(sm.ks[b], c + 8 * j), vs = pair(sm.vs[b], c + 8 * j);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint64_t x = fma2(mul2((uint64_t)v[4 * j + 2 * r] | (uint64_t)v[4 * j + 2 * r + 1] << 32, ks), pack2(qf[r], qf[r]), pack2(-m[r], -m[r]));
              uint64_t p = pack2(exp2_fast(first(x)), exp2_fast(second(x)));
              if (!decltype(whole)::value) p = pack2(c + 8 * j < left ? first(p) : 0.f, c + 8 * j + 1 < left ? second(p) : 0.f);
              sum[r] = add2(sum[r], p);
              const uint64_t x2 = mul2(p, vs);
              const __half2 h2 = __floats2half2_rn(first(x2), second(x2));
              w[2 * j + r] = *reinterpret_cast<const uint32_t*>(&h2);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) l[r] += first(sum[r]) + second(sum[r]);
          tc::tmem_st_frag16(p_at + c / 2, w);
        }
      };
      if (here >= kTokens) weights(std::true_type());
      else weights(std::false_type());
      tc::tmem_wait_st();
      tc::fence_before_sync();
      tc::mbar_arrive(tc::smem_u32(&sm.p_ready[i & 1]));
    }
    if (ok) store(tiles - 1, chunk);
    tc::fence_before_sync();
  }
  if (!ok) sm.gave_up = 1;
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kSoftmax / 32) tc::tmem_dealloc(s_cols, kTmemCols);
  if (sm.gave_up && tid < kRows && row0 + tid < rows) {   // NaN in all of this CTA's records
    const int r = row0 + tid, b = stream_of(r);
    for (int c = chunk0; c < min(chunk0 + per_cta, a.p_chunks); ++c)
      a.rec_ml[a.record(b, kh * G + r - b * G, c)] = make_float2(0.f, __uint_as_float(0x7FC00000u));
  }
}

// Chunks that a CTA takes one after the other.  A CTA's start and end cost about as much as three tiles, so the
// chunks of a second wave are better some CTA's next ones: 32 streams of 8 heads behind 32768 positions 43.8 -> 42.7 us,
// 512 behind 4096 315 -> 248 us.  The records are the same either way.
int chunks_per_cta(int chunks, int tiles, int others) {
  int best = 1, waves = 2;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= chunks && waves > 1; ++n) {
    waves = ((chunks + n - 1) / n * others + kSms - 1) / kSms;
    const int64_t cost = waves * ((int64_t)n * tiles + 3);
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

template <int D, int FMT>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(PrefixSmem<D>) + 1024;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = once_per_device(
      done, [&] { return cudaFuncSetAttribute(k_kv8_prefix<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); });
  if (e != cudaSuccess) return e;
  const int row_tiles = (a.B * (a.qh / a.c.kvh) + kRows - 1) / kRows;
  const int per_cta = chunks_per_cta(a.p_chunks, a.p_chunk / kTokens, row_tiles * a.c.kvh);
  return launch_k(false, k_kv8_prefix<D, FMT>, dim3((a.p_chunks + per_cta - 1) / per_cta, row_tiles, a.c.kvh), dim3(kThreads), smem, s, a, per_cta);
}

}  // namespace

namespace kv8 {

cudaError_t launch_kv8_prefix(const AttendArgs& a, int format, int d, cudaStream_t s) {
  if (d == 128) return format == BM_KV8_E4M3 ? launch<128, BM_KV8_E4M3>(a, s) : launch<128, BM_KV8_INT8>(a, s);
  return format == BM_KV8_E4M3 ? launch<64, BM_KV8_E4M3>(a, s) : launch<64, BM_KV8_INT8>(a, s);
}

}  // namespace kv8
}  // namespace bm
