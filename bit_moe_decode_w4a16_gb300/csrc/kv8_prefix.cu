// Attention over a prefix that a batch shares, computed once for all of it.
//
// The query rows of a kv head are gathered from the whole batch (row r is
// head r % G of its group of stream r / G), 128 at a time: over a prefix of P
// positions that is a dense product of 128 x P x d, and the prefix's codes
// are read and converted once per 128 rows instead of once per stream.  A CTA
// takes 128 rows and one chunk of the prefix and leaves one record (o, m, l)
// per row; the records are merged with those of the streams' own positions.
//
// Per tile of 64 positions, on the 5th-generation tensor cores (fp16
// operands, fp32 sums in tensor memory):
//   S[row][position] = Q K^T, MMAs of 128 x 64 x 16, both operands in shared
//     memory (K-major, 128-byte swizzle);
//   p and the weights p * vs as in kv8_attend.cu, a thread to a row, two
//     positions to an instruction (f32x2); the weights go back over S as the
//     fp16 A operand;
//   O[row][element] += P V, MMAs of 128 x d x 16, A in tensor memory, B = V^T
//     in shared memory, positions contiguous (K-major).
// Four warps do the softmax; four convert codes to fp16 (V is transposed on
// the way, 8 positions x 4 bytes to a thread; its elements are stored at row
// d / 4 (e % 4) + e / 4 of B so that a warp's stores meet no bank conflict,
// and O's columns come out in that order), and a lane of theirs issues the
// MMAs.  K, V and S have two buffers each: a commit is seen about 2000 cycles
// after its MMAs were issued, so the next tile's scores are on their way
// while this one's softmax runs, and O is waited for only to rescale it.  Two
// CTAs share an SM (256 of its 512 tensor memory columns and about 100 KB of
// shared memory each).
//
// What bounds it is the issue of the softmax's instructions, about 6 per
// score, and the conversions'.
//
// Every wait is bounded.  A wait that gives up leaves NaN in its CTA's
// records, and so in the output rows.
#include <mutex>
#include <set>
#include <utility>

#include "kv8_attend.cuh"
#include "tc_ptx.cuh"

namespace bm {
namespace {

using namespace kv8;

constexpr int kRows = 128, kTokens = 64;           // a tile
constexpr int kSoftmax = 128, kConvert = 128, kThreads = kSoftmax + kConvert;   // 8 warps: 128 registers at two CTAs an SM
constexpr uint32_t kTmemCols = 256;                // S (then P) of even tiles, of odd tiles, O
constexpr uint32_t kWaitLimit = 1u << 18;          // polls of ~3.7 us: a wait gives up after about a second

template <int D>
struct PrefixSmem {
  uint8_t q[kRows * D * 2];                        // [d / 64][row][64] fp16, swizzled
  uint8_t k[2][kTokens * D * 2];                   // [d / 64][position][64]
  uint8_t v[2][kTokens * D * 2];                   // [element][64 positions]
  float ks[2][kTokens], vs[2][kTokens], lg[2][kTokens];   // scales, log2 of V's
  // by the tile's parity; their phase is the tile's half
  uint64_t k_full[2], v_full[2], s_ready[2], p_ready[2], o_ready[2], drained;
  uint32_t tmem;
  int gave_up;
};
constexpr int kOutStride = 129;                    // floats of a row of O on its way out, over q, k and v
static_assert(kRows * kOutStride * 4 <= 3 * kRows * 128 * 2, "O fits over the operands (d = 128)");
static_assert(kRows * (64 + 1) * 4 <= 3 * kRows * 64 * 2, "O fits over the operands (d = 64)");

// 16-byte piece c of row r of a K-major operand of `rows` rows: 128-byte rows of 64 fp16, pieces swizzled by the row.
__device__ __forceinline__ uint32_t piece(int rows, int r, int c) { return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

// Descriptor of a K-major operand with the 128-byte swizzle: 8-row atoms of
// 1024 bytes (SBO), LBO unused (encoded 1), layout type 2; the start address
// moves by 32 bytes per 16 values of K.
__device__ __forceinline__ uint64_t operand(uint32_t base, int rows, int k16) {
  const uint32_t at = base + (k16 >> 2) * rows * 128 + (k16 & 3) * 32;
  return (uint64_t)((at >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ uint64_t pack2(float a, float b) { return (uint64_t)__float_as_uint(a) | (uint64_t)__float_as_uint(b) << 32; }
__device__ __forceinline__ float first(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float second(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 2) k_kv8_prefix(AttendArgs a) {
  extern __shared__ unsigned char raw[];
  const uint32_t raw_at = tc::smem_u32(raw);
  PrefixSmem<D>& sm = *reinterpret_cast<PrefixSmem<D>*>(raw + ((1024u - (raw_at & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk = blockIdx.x, row0 = blockIdx.y * kRows, kh = blockIdx.z;
  const int kvh = a.c.kvh, G = a.qh / kvh, rows = a.B * G;
  const int j0 = chunk * a.p_chunk, n = min(a.p_chunk, a.p_len - j0), tiles = (n + kTokens - 1) / kTokens;
  const size_t at = a.p.row(a.p_slot, kh, j0);
  pdl_trigger();                                   // the streams' own chunks do not depend on this

  if (warp == 4) {
    tc::tmem_alloc(tc::smem_u32(&sm.tmem), kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tc::smem_u32(&sm.k_full[b]), kConvert);
      tc::mbar_init(tc::smem_u32(&sm.v_full[b]), kConvert);
      tc::mbar_init(tc::smem_u32(&sm.p_ready[b]), kSoftmax);
      tc::mbar_init(tc::smem_u32(&sm.s_ready[b]), 1);
      tc::mbar_init(tc::smem_u32(&sm.o_ready[b]), 1);
    }
    tc::mbar_init(tc::smem_u32(&sm.drained), 1);
    tc::fence_mbar_init();
    sm.gave_up = 0;
  }
  float up = 1.f;
  if (tid < kSoftmax) {
    // ---- this thread's query row, as fp16 of about its own magnitude
    const int r = row0 + tid, b = r / G, h = kh * G + r - b * G;
    uint4 x[D / 8];
    float mx = 0.f;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      x[c] = make_uint4(0, 0, 0, 0);
      if (r < rows) x[c] = *reinterpret_cast<const uint4*>(a.Q + ((size_t)b * a.qh + h) * D + 8 * c);
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(w[e])), fabsf(bf_hi(w[e]))));
    }
    float down;
    row_scale(mx, down, up);
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
      uint32_t f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 v = __floats2half2_rn(bf_lo(w[e]) * down, bf_hi(w[e]) * down);
        f[e] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(sm.q + piece(kRows, tid, c)) = make_uint4(f[0], f[1], f[2], f[3]);
    }
    tc::fence_proxy_async_smem();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t s_cols = sm.tmem, o_cols = s_cols + 2 * kTokens;
  // tile i's phase of a pair of barriers.  No thread can miss one: a tile's barrier completes again only after
  // every thread that waits for it has arrived at another barrier of that tile.
  auto wait = [](uint64_t* bars, int i) { return tc::mbar_wait_spin(tc::smem_u32(&bars[i & 1]), i >> 1 & 1, kWaitLimit); };
  bool ok = true;
  float m = -1e30f, l = 0.f;

  if (warp >= 4) {
    // ---------------- conversion: warp w takes positions 16 w .. of a tile
    const int cw = warp - 4, ct = tid - kSoftmax;
    constexpr int kRowsAt = D == 128 ? 4 : 8;      // K rows to a warp's load
    constexpr int kK = kTokens / 4 / kRowsAt;      // loads of 16 codes
    constexpr int kG = D == 128 ? 2 : 1;           // groups of 8 positions to a thread
    const int k_row = lane / (32 / kRowsAt), k_piece = lane % (32 / kRowsAt);
    const int v_word = D == 128 ? lane : lane & 15, v_half = D == 128 ? 0 : lane >> 4;
    const uint8_t *K = a.p.K + at * D, *V = a.p.V + at * D;
    uint4 kr[kK];
    uint32_t vr[kG][8];
    float scale;                                   // K's in threads 0 .. 63, V's in the others
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
      const int p = i * kTokens + (ct & 63);
      scale = p < n ? __ldg((ct < 64 ? a.p.Ks : a.p.Vs) + at + p) : 0.f;
    };
    const bool issuer = ct == 0;
    const uint32_t qk = tc::idesc_f16_f32(kRows, kTokens), pv = tc::idesc_f16_f32(kRows, D);
    const uint32_t q_at = tc::smem_u32(sm.q);
    // tile i's scores, once its K is there
    auto issue_scores = [&](int i) {
      if (!wait(sm.k_full, i)) return false;
      tc::fence_after_sync();
      const uint32_t k_at = tc::smem_u32(sm.k[i & 1]);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        tc::mma_f16_ss(s_cols + (i & 1) * kTokens, operand(q_at, kRows, k), operand(k_at, kTokens, k), qk, k > 0);
      tc::mma_commit(tc::smem_u32(&sm.s_ready[i & 1]));
      return true;
    };
    // tile i's part of O, once its weights and its V are there
    auto issue_output = [&](int i) {
      if (!wait(sm.v_full, i) || !wait(sm.p_ready, i)) return false;
      tc::fence_after_sync();
      const uint32_t v_at = tc::smem_u32(sm.v[i & 1]);
#pragma unroll
      for (int k = 0; k < kTokens / 16; ++k)
        tc::mma_f16_tmem_a(o_cols, s_cols + (i & 1) * kTokens + 8 * k, operand(v_at, D, k), pv, i > 0 || k > 0);
      tc::mma_commit(tc::smem_u32(&sm.o_ready[i & 1]));
      return true;
    };
    load(0);
    for (int i = 0; i < tiles; ++i) {
      // the K buffer is free once tile i - 2 has its scores
      if (i > 1 && !(ok = wait(sm.s_ready, i - 2))) break;
      uint8_t *k_to = sm.k[i & 1], *v_to = sm.v[i & 1];
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
      // these scores go where tile i - 2's weights are: after its output's MMAs
      if (issuer) ok = (i < 2 || issue_output(i - 2)) && issue_scores(i);
      __syncwarp();
      // V, and the scales that tile i - 2's softmax has read
      if (i > 1) ok = ok && wait(sm.o_ready, i - 2);
      if (!ok) break;
      if (ct < 64) {
        sm.ks[i & 1][ct] = scale;
      } else {
        sm.vs[i & 1][ct - 64] = scale;
        sm.lg[i & 1][ct - 64] = fmaxf(log2_fast(scale), -100.f);
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
    if (issuer) {
      if (ok && tiles > 1) ok = issue_output(tiles - 2);
      if (ok) ok = issue_output(tiles - 1);
      // nothing of this CTA's is in flight when it ends
      tc::mma_commit(tc::smem_u32(&sm.drained));
      if (!tc::mbar_wait(tc::smem_u32(&sm.drained), 0, kWaitLimit)) ok = false;
    }
    __syncwarp();
  } else {
    // ---------------- softmax: a thread to a row
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const float qf = a.scale_log2 * up;
    const uint64_t qf2 = pack2(qf, qf);
    for (int i = 0; i < tiles; ++i) {
      ok = wait(sm.v_full, i) && wait(sm.s_ready, i) && (i < 2 || wait(sm.o_ready, i - 2));
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const int left = n - i * kTokens;
      const ulonglong2 *ks = reinterpret_cast<const ulonglong2*>(sm.ks[i & 1]), *vs = reinterpret_cast<const ulonglong2*>(sm.vs[i & 1]),
                       *lg = reinterpret_cast<const ulonglong2*>(sm.lg[i & 1]);
      const uint32_t cols = s_cols + lanes + (i & 1) * kTokens;
      uint32_t v[2][32];
      tc::tmem_ld32(cols, v[0]);
      tc::tmem_ld32(cols + 32, v[1]);
      tc::tmem_wait_ld();
      uint64_t t[kTokens / 2];                     // q . k * ks, two positions each
      float mx = -1e30f, my = -1e30f;
#pragma unroll
      for (int k = 0; k < kTokens / 4; ++k) {
        const ulonglong2 kk = ks[k], gg = lg[k];
        const uint32_t* x = &v[k / 8][4 * (k % 8)];
        t[2 * k] = mul2((uint64_t)x[0] | (uint64_t)x[1] << 32, kk.x);
        t[2 * k + 1] = mul2((uint64_t)x[2] | (uint64_t)x[3] << 32, kk.y);
        const uint64_t x0 = fma2(t[2 * k], qf2, gg.x), x1 = fma2(t[2 * k + 1], qf2, gg.y);
        if (left >= kTokens) {
          mx = fmaxf(mx, fmaxf(first(x0), second(x0)));
          my = fmaxf(my, fmaxf(first(x1), second(x1)));
        } else {
          if (4 * k < left) mx = fmaxf(mx, first(x0));
          if (4 * k + 1 < left) mx = fmaxf(mx, second(x0));
          if (4 * k + 2 < left) mx = fmaxf(mx, first(x1));
          if (4 * k + 3 < left) mx = fmaxf(mx, second(x1));
        }
      }
      mx = fmaxf(mx, my);
      if (__any_sync(0xffffffffu, mx > m + 8.f)) {
        const float mn = mx > m + 8.f ? mx : m, f = exp2_fast(m - mn);   // each row by itself: its neighbours are other streams'
        m = mn;
        l *= f;
        if (i > 0) {                               // O holds the tiles before
          ok = wait(sm.o_ready, i - 1);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tc::tmem_ld16(o_cols + lanes + c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tc::tmem_st16(o_cols + lanes + c, o);
          }
        }
      }
      const uint64_t m2 = pack2(-m, -m);
      uint64_t sum0 = 0, sum1 = 0;
      uint32_t w[kTokens / 2];
#pragma unroll
      for (int k = 0; k < kTokens / 4; ++k) {
        const ulonglong2 vv = vs[k];
        const uint64_t x0 = fma2(t[2 * k], qf2, m2), x1 = fma2(t[2 * k + 1], qf2, m2);
        uint64_t p0 = pack2(exp2_fast(first(x0)), exp2_fast(second(x0))), p1 = pack2(exp2_fast(first(x1)), exp2_fast(second(x1)));
        if (left < kTokens) {
          p0 = pack2(4 * k < left ? first(p0) : 0.f, 4 * k + 1 < left ? second(p0) : 0.f);
          p1 = pack2(4 * k + 2 < left ? first(p1) : 0.f, 4 * k + 3 < left ? second(p1) : 0.f);
        }
        sum0 = add2(sum0, p0);
        sum1 = add2(sum1, p1);
        const uint64_t w0 = mul2(p0, vv.x), w1 = mul2(p1, vv.y);
        const __half2 h0 = __floats2half2_rn(first(w0), second(w0)), h1 = __floats2half2_rn(first(w1), second(w1));
        w[2 * k] = *reinterpret_cast<const uint32_t*>(&h0);
        w[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&h1);
      }
      tc::tmem_st32(cols, w);
      sum0 = add2(sum0, sum1);
      l += first(sum0) + second(sum0);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      tc::mbar_arrive(tc::smem_u32(&sm.p_ready[i & 1]));
    }
    if (ok) ok = (tiles < 2 || wait(sm.o_ready, tiles - 2)) && wait(sm.o_ready, tiles - 1);
    tc::fence_after_sync();
    if (__all_sync(0xffffffffu, ok)) {
      // every MMA is done: O goes out over the operands, a row to a thread
      float* out = reinterpret_cast<float*>(&sm) + tid * (D == 128 ? kOutStride : 65);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tc::tmem_ld32(o_cols + lanes + c, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const int col = c + k;                   // B's row: element 4 (col % (d / 4)) + col / (d / 4)
          out[4 * (col % (D / 4)) + col / (D / 4)] = __uint_as_float(o[k]);
        }
      }
    }
    tc::fence_before_sync();
  }
  if (!ok) sm.gave_up = 1;
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 4) tc::tmem_dealloc(s_cols, kTmemCols);
  const bool bad = sm.gave_up != 0;
  // ---- records, a row to a warp at a time
  const float* out = reinterpret_cast<const float*>(&sm);
  for (int r = warp; r < kRows && row0 + r < rows; r += kThreads / 32) {
    const int b = (row0 + r) / G, h = kh * G + row0 + r - b * G;
    float* rec = a.record(b, h, chunk, D);
#pragma unroll
    for (int d = lane; d < D; d += 32) rec[d] = out[r * (D == 128 ? kOutStride : 65) + d];
  }
  if (tid < kSoftmax && row0 + tid < rows) {
    const int b = (row0 + tid) / G, h = kh * G + row0 + tid - b * G;
    float* rec = a.record(b, h, chunk, D);
    *reinterpret_cast<float2*>(rec + D) = make_float2(bad ? 0.f : m, bad ? __uint_as_float(0x7FC00000u) : l);
  }
}

std::mutex g_mu;
std::set<std::pair<int, const void*>> g_set;

template <int D, int FMT>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(PrefixSmem<D>) + 1024;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    const void* f = (const void*)k_kv8_prefix<D, FMT>;
    if (!g_set.count({dev, f})) {
      if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
      g_set.insert({dev, f});
    }
  }
  const int rows = a.B * (a.qh / a.c.kvh);
  return launch_k(false, k_kv8_prefix<D, FMT>, dim3(a.p_chunks, (rows + kRows - 1) / kRows, a.c.kvh), dim3(kThreads), smem, s, a);
}

}  // namespace

namespace kv8 {

cudaError_t launch_kv8_prefix(const AttendArgs& a, int format, int d, cudaStream_t s) {
  if (d == 128) return format == BM_KV8_E4M3 ? launch<128, BM_KV8_E4M3>(a, s) : launch<128, BM_KV8_INT8>(a, s);
  return format == BM_KV8_E4M3 ? launch<64, BM_KV8_E4M3>(a, s) : launch<64, BM_KV8_INT8>(a, s);
}

}  // namespace kv8
}  // namespace bm
