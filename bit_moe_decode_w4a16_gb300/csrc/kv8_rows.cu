// Attention of a ragged step's rows over the 8-bit cache, each behind its own
// stream's positions.
//
// Row j of a stream with n rows and len positions (its own n included) attends
// to positions 0 .. len - n + j of its slot, or, in a tree, to 0 .. len - n - 1
// and those of its ancestors and itself:
//   o = sum_p w_p v_p / sum_p w_p,   w_p = 2^(x_p - m),  x_p = scale log2(e) q . k_p
// A stream's rows are gathered per kv head (row r is head r % G of row r / G),
// 256 to a block; a CTA takes pieces of blocks from the plan's list (longest
// first, dealt out back and forth) and walks over a piece's tiles of 128
// positions on the 5th-generation tensor cores (fp16 operands, fp32 sums in
// tensor memory):
//   S[row][position] = Q K^T, MMAs of 128 x 128 x 16, both in shared memory;
//   weights 2^(S ks qf - m) vs, as fp16, over S's place in tensor memory; m is
//     the running maximum of x + log2 vs, moved only when it rises by 2^8;
//   O[row][element] += P V, MMAs of 128 x d x 16, A in tensor memory, B the
//     tile's V as it lies (positions down, elements along: N-major).
// K and V are converted to fp16 with the same layout (128-byte swizzle), once
// for the block's two halves of 128 rows, which two warpgroups of softmax work
// on in turn: while one makes weights the other's products run.  A block of up
// to 128 rows instead gives its even tiles to one warpgroup and the odd ones
// to the other, each with sums of its own, which are joined at the end.
// A thread has 4 rows x 32 positions of a tile, so that a load of scales serves
// 8 scores, and holds the scores in registers between maximum and weights.
// A warpgroup converts codes, one lane issues the MMAs.
//
// Every wait is bounded.  A CTA in which one gave up leaves NaN in the rows of all
// of its pieces.
#include <type_traits>

#include "kv8_attend.cuh"
#include "kv8_step.cuh"
#include "tc_ptx.cuh"

namespace bm {
namespace {

using namespace kv8;

struct RowsArgs {
  Cache c;
  const void* plan;
  const bf16* Q;
  bf16* O;
  float* rec_o;        // records: unnormalised output [d]
  float2* rec_ml;      // and its maximum and sum
  int B, T, qh;
  float scale_log2;
};

// The plan is for these sizes.
__device__ __forceinline__ bool fits(const PlanHead& h, const RowsArgs& a) {
  return h.magic == kPlanMagic && h.B == a.B && h.T == a.T && h.qh == a.qh && h.kvh == a.c.kvh && h.slots == a.c.slots && h.cap == a.c.cap;
}

constexpr int kSub = 128;                                   // rows of a half block
constexpr int kConvert = 256, kThreads = 128 + kConvert + 256;   // a warpgroup that issues MMAs, two of conversion, two of softmax
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 160, kConvertRegs = 64, kIssueRegs = 32;
static_assert(2 * kSoftmaxRegs + 2 * kConvertRegs + kIssueRegs <= 5 * kLaunchRegs, "warpgroups share what the launch has");
constexpr uint32_t kTmemCols = 512;                         // S of both halves (later P), O of both halves
constexpr float kLargest = 32768.f;                         // a weight above it moves its row's maximum; fp16 ends at 65504
constexpr float kLargestSum = 2.028240960365167e31f;        // 2^104: V scales below 2^-100 count as that in a maximum
constexpr uint32_t kWaitLimit = 1u << 18;                   // polls of ~3.7 us: a wait gives up after about a second

template <int D>
struct RowsSmem {
  uint8_t q[2][kSub * D * 2];                               // [d / 64][row][64] fp16, swizzled
  uint8_t k[2][kTile * D * 2], v[2][kTile * D * 2];         // [d / 64][position][64]
  // scales and log2 of V's, of four tiles: they are written with a tile's K, when the softmax may be two tiles back
  float ks[4][kTile], vs[4][kTile], lg[4][kTile];
  float up[kBlockRows];
  float m[kSub], l[kSub];                                   // of the second warpgroup, where both have the same rows
  uint64_t k_full[2], v_full[2];                            // by the tile's parity
  uint64_t s_ready[2][2], o_ready[2][2];                    // by half and the tile's parity: they also say that K, V may be overwritten
  uint64_t p_ready[2], turn[2];                             // by half
  uint64_t q_full, drained;
  uint32_t tmem;
  int gave_up;
};

// 16-byte piece c of row r: 128-byte rows of 64 fp16, pieces swizzled by the row.
__device__ __forceinline__ uint32_t piece(int r, int c) { return (c >> 3) * kTile * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4); }
// Descriptors with the 128-byte swizzle (layout type 2), 8-row atoms of 1024 bytes: the low word, to which a start 16 bytes further on
// adds 1, and the whole.  Rows of K and Q: the start moves by 32 bytes per 16 elements.  V, N-major: by 16 rows per 16
// positions, and blocks of 64 elements lie 128 rows apart.
__device__ __forceinline__ uint32_t k_major(uint32_t at) { return at >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t n_major(uint32_t at) { return at >> 4 | (uint32_t)(kTile * 128 >> 4) << 16; }
__device__ __forceinline__ uint64_t operand(uint32_t low) { return (uint64_t)low | (uint64_t)((1024u >> 4) | 1u << 14 | 2u << 29) << 32; }

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void sync_some(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

__device__ __forceinline__ uint64_t join(uint32_t lo, uint32_t hi) { return (uint64_t)lo | (uint64_t)hi << 32; }

// Of a thread's positions 8 j + e (j < 16, e < 2), as bits 2 j + e: those below `left`; and those whose bit (offset + 8 j + e) of `bits` is set.
__device__ __forceinline__ uint32_t below(int left) {
  const int k = left <= 0 ? 0 : 2 * (left >> 3) + min(left & 7, 2);
  return k >= 32 ? 0xffffffffu : (1u << k) - 1;
}
__device__ __forceinline__ uint32_t two_of_eight(unsigned long long x) {   // bits 0 and 1 of each byte, together
  x &= 0x0303030303030303ull;
  x = (x | x >> 6) & 0x000F000F000F000Full;
  x = (x | x >> 12) & 0x000000FF000000FFull;
  return (uint32_t)(x | x >> 24) & 0xFFFFu;
}
__device__ __forceinline__ uint32_t among(unsigned long long bits, int offset) {
  const int up = -offset;
  unsigned long long lo = 0, hi = 0;
  if (offset >= 0) lo = offset < 64 ? bits >> offset : 0;
  else if (up < 64) lo = bits << up, hi = bits >> (64 - up);
  else hi = up < 128 ? bits << (up - 64) : 0;
  return two_of_eight(lo) | two_of_eight(hi) << 16;
}

// The CTA's r-th piece.
__device__ __forceinline__ int turn(int r) { return r * (int)gridDim.x + (int)(r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); }

// A piece as all roles see it.
struct Work {
  PlanStream st;
  int kh, q0, rows, tiles, t0, piece;   // kv head; first of its rows and their number; tiles from t0 on; 65535: the whole block
  bool wide;                            // both halves have rows
  __device__ Work(const Plan& plan, int i, int G) {
    const PlanItem it = plan.items[i];
    st = plan.streams[it.who & 1023];
    kh = it.who >> 10;
    q0 = (it.what & 65535) * kBlockRows;
    rows = min(kBlockRows, st.n * G - q0);
    t0 = it.t0;
    tiles = it.t1 - it.t0;
    piece = it.what >> 16;
    wide = rows > kSub;
  }
};

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) k_kv8_rows(RowsArgs a) {
  extern __shared__ unsigned char raw[];
  const uint32_t raw_at = tc::smem_u32(raw);
  RowsSmem<D>& sm = *reinterpret_cast<RowsSmem<D>*>(raw + ((1024u - (raw_at & 1023u)) & 1023u));
  const Plan plan(const_cast<void*>(a.plan), a.B, a.T);
  pdl_trigger();                                            // the merge starts when this grid lets it
  // the same in all lanes by construction, which spares the warps that issue MMAs most of their instructions
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const int items = uniform(fits(*plan.head, a) ? plan.head->items : 0);
  if ((int)blockIdx.x >= items) return;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, G = a.qh / a.c.kvh;

  if (warp == 0) {
    tc::tmem_alloc(tc::smem_u32(&sm.tmem), kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tc::smem_u32(&sm.k_full[b]), kConvert);
      tc::mbar_init(tc::smem_u32(&sm.v_full[b]), kConvert);
      for (int s = 0; s < 2; ++s) {
        tc::mbar_init(tc::smem_u32(&sm.s_ready[s][b]), 2);
        tc::mbar_init(tc::smem_u32(&sm.o_ready[s][b]), 1);
      }
      tc::mbar_init(tc::smem_u32(&sm.p_ready[b]), 128);
      tc::mbar_init(tc::smem_u32(&sm.turn[b]), 1);
    }
    tc::mbar_init(tc::smem_u32(&sm.q_full), 256);
    tc::mbar_init(tc::smem_u32(&sm.drained), 2);
    tc::fence_mbar_init();
    sm.gave_up = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t s_cols = sm.tmem, o_cols = s_cols + 2 * kTile;
  // Completion number n (from 0) of a barrier.  A thread whose wait gave up goes on without waiting and arrives nowhere, so that
  // all threads take the same way through the barriers of their warpgroup.
  bool ok = true;
  auto wait = [&](uint64_t& bar, int n) {
    if (ok) ok = tc::mbar_wait(tc::smem_u32(&bar), n & 1, kWaitLimit);
  };
  auto arrive = [&](uint64_t& bar) {
    if (ok) tc::mbar_arrive(tc::smem_u32(&bar));
  };

  if (warp < 4) {
    // ---------------- MMAs, a warp for each half.  They run in the order in which a warp issues them, so a half's scores may be issued
    // behind the product that reads the weights they overwrite.  The two take turns, a product and the next scores each: issued
    // at once, both halves' MMAs end together, and the tensor cores wait while both make weights (a prompt of 8192 rows: 659 us;
    // in turns 566; one warp for both, 702, as the pipe runs dry between its MMAs).
    regs_down<kIssueRegs>();
    if (warp < 2) {
      const int s = warp;
      constexpr uint32_t qk = tc::idesc_f16_f32(kSub, kTile), pv = tc::idesc_f16_f32(kSub, D) | tc::kIdescBMajorN;
      constexpr uint32_t kBuffer = kTile * D * 2 >> 4, kBlock = kTile * 128 >> 4;
      const uint32_t k_at = k_major(tc::smem_u32(sm.k[0])), v_at = n_major(tc::smem_u32(sm.v[0])), q_at = k_major(tc::smem_u32(sm.q[0]));
      const uint32_t leader = tc::elect_one();
      const uint32_t s_at = s_cols + s * kTile, o_at = o_cols + s * 128;
      int turns = 0;                                        // s = 0 begins
      auto my_turn = [&]() {
        if (turns >= 1 - s) wait(sm.turn[s], turns - (1 - s));
        ++turns;
      };
      auto pass = [&]() {
        if (leader && ok) tc::mbar_arrive(tc::smem_u32(&sm.turn[1 - s]));
        __syncwarp();
      };
      int tile0 = 0, uses = 0;                              // tiles before this piece, the half's steps so far
      for (int r = 0; turn(r) < items; ++r) {
        const Work w(plan, turn(r), G);
        const int wide = uniform(w.wide), tiles = uniform(w.tiles), steps = wide ? 2 * tiles : tiles;   // step k is half k % 2's
        auto tile_of = [&](int k) { return tile0 + (wide ? k >> 1 : k); };
        auto scores = [&](int k) {
          const int b = tile_of(k) & 1;
          __syncwarp();
          tc::fence_after_sync();
          const uint32_t q = q_at + (wide ? s * kBuffer : 0), kk = k_at + b * kBuffer, on = leader && ok;
#pragma unroll
          for (int e = 0; e < D / 16; ++e)
            tc::warp_mma_f16_ss(s_at, operand(q + (e >> 2) * kBlock + (e & 3) * 2), operand(kk + (e >> 2) * kBlock + (e & 3) * 2), qk, e > 0, on);
          if (on) {
            tc::mma_commit(tc::smem_u32(&sm.s_ready[s][b]));
            tc::mbar_arrive(tc::smem_u32(&sm.s_ready[s][b]));   // a release by this thread: it passes the scales on
          }
          __syncwarp();
        };
        auto product = [&](int k) {
          const int b = tile_of(k) & 1;
          wait(sm.v_full[b], tile_of(k) >> 1);
          wait(sm.p_ready[s], uses++);
          my_turn();
          __syncwarp();
          tc::fence_after_sync();
          const uint32_t v = v_at + b * kBuffer, on = leader && ok;
#pragma unroll
          for (int e = 0; e < kTile / 16; ++e) tc::warp_mma_f16_tmem_a(o_at, s_at + 8 * e, operand(v + e * (16 * 128 >> 4)), pv, k > 1 || e > 0, on);
          if (on) tc::mma_commit(tc::smem_u32(&sm.o_ready[s][b]));
          __syncwarp();
        };
        wait(sm.q_full, r);
        if (s < steps) wait(sm.k_full[tile_of(s) & 1], tile_of(s) >> 1);
        my_turn();
        if (s < steps) scores(s);
        pass();
        for (int k = s; k < steps; k += 2) {
          if (k + 2 < steps) wait(sm.k_full[tile_of(k + 2) & 1], tile_of(k + 2) >> 1);
          product(k);
          if (k + 2 < steps) scores(k + 2);
          pass();
        }
        if (s == 1 && (steps & 1)) {                        // the other half has one more
          my_turn();
          pass();
        }
        tile0 += tiles;
      }
      // nothing of this CTA's is in flight when it ends
      tc::warp_mma_commit(tc::smem_u32(&sm.drained), leader);
      if (!tc::mbar_wait(tc::smem_u32(&sm.drained), 0, kWaitLimit)) ok = false;
    }
  } else if (warp < 4 + kConvert / 32) {
    // ---------------- conversion: 16 codes to a thread and turn
    regs_down<kConvertRegs>();
    constexpr int kLanes = D / 16, kTurns = kTile * kLanes / kConvert;
    const int ct = tid - 128, row0 = ct / kLanes, c = ct % kLanes;
    const bool swap = c & 4;                                // the second half's pieces in the other order: no bank conflict
    uint4 kr[kTurns], vr[kTurns];
    float scale = 0.f;                                      // of position ct % 128: K's in the first warpgroup, V's in the other
    auto load = [&](const Work& w, int i, bool v) {
      const int p0 = (w.t0 + i) * kTile;
      const size_t at = a.c.row(w.st.slot, w.kh, p0);
      const uint8_t* from = (v ? a.c.V : a.c.K) + at * D + 16 * ct;
      const int left = w.st.len - p0;
      uint4* to = v ? vr : kr;
#pragma unroll
      for (int u = 0; u < kTurns; ++u)
        to[u] = u * (kConvert / kLanes) + row0 < left ? ldg_nc_v4(from + u * kConvert * 16) : make_uint4(0, 0, 0, 0);
      if (!v) scale = (ct & 127) < left ? __ldg((ct < 128 ? a.c.Ks : a.c.Vs) + at + (ct & 127)) : 0.f;
    };
    auto convert = [&](uint8_t* to, const uint4 (&x)[kTurns]) {
#pragma unroll
      for (int u = 0; u < kTurns; ++u) {
        const int row = u * (kConvert / kLanes) + row0;
        uint32_t f[8];
        codes4<FMT>(x[u].x, f[0], f[1]);
        codes4<FMT>(x[u].y, f[2], f[3]);
        codes4<FMT>(x[u].z, f[4], f[5]);
        codes4<FMT>(x[u].w, f[6], f[7]);
        *reinterpret_cast<uint4*>(to + piece(row, 2 * c + swap)) = swap ? make_uint4(f[4], f[5], f[6], f[7]) : make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4*>(to + piece(row, 2 * c + !swap)) = swap ? make_uint4(f[0], f[1], f[2], f[3]) : make_uint4(f[4], f[5], f[6], f[7]);
      }
    };
    int tile = 0;
    // bit 2 half + buffer: the parity of the half's steps with the buffer so far; the buffer's tile was a step of the half
    unsigned uses = 0, theirs = 0;
    for (int r = 0; turn(r) < items; ++r) {
      const Work w(plan, turn(r), G);
      const int own = w.st.len - w.st.n, all_see = own + (w.st.tree ? 0 : w.q0 / G + 1);   // positions that every row attends to
      load(w, 0, false);
      load(w, 0, true);
      for (int i = 0; i < w.tiles; ++i, ++tile) {
        const int b = tile & 1, slot = tile & 3;
        // the buffer's last tile was a step of one half or of both: its scores (its products) have been made
        auto free_again = [&](uint64_t (&done)[2][2]) {
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (theirs >> (2 * s + b) & 1) wait(done[s][b], (uses >> (2 * s + b) & 1) ^ 1);
        };
        free_again(sm.s_ready);
        if (ct < 128) {
          sm.ks[slot][ct] = scale;
        } else {
          sm.vs[slot][ct - 128] = scale;
          sm.lg[slot][ct - 128] = fmaxf(log2_fast(scale), -100.f);
        }
        if (FMT == BM_KV8_E4M3 && (w.t0 + i + 1) * kTile > all_see) {
          // some rows do not attend to some of these positions, and 0 * NaN is NaN: a NaN code becomes 0, and its position's scale NaN
          sync_some(2, kConvert);
#pragma unroll
          for (int u = 0; u < kTurns; ++u) {
            uint32_t* x = reinterpret_cast<uint32_t*>(&vr[u]);
            uint32_t any = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t nan = ((x[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
              x[e] &= ~((nan >> 7) * 0xFFu);
              any |= nan;
            }
            if (any) sm.vs[slot][u * (kConvert / kLanes) + row0] = __uint_as_float(0x7FC00000u);
          }
        }
        convert(sm.k[b], kr);
        tc::fence_proxy_async_smem();
        arrive(sm.k_full[b]);
        if (i + 1 < w.tiles) load(w, i + 1, false);
        free_again(sm.o_ready);
        convert(sm.v[b], vr);
        tc::fence_proxy_async_smem();
        arrive(sm.v_full[b]);
        const unsigned now = (w.wide ? 5u : 1u << (2 * (i & 1))) << b;
        theirs = (theirs & ~(5u << b)) | now;
        uses ^= now;
        if (i + 1 < w.tiles) load(w, i + 1, true);
      }
    }
  } else {
    // ---------------- softmax: thread (g, t) of a warp has rows g, g + 8, g + 16, g + 24 of its 32 (index r) and positions
    // 8 j + 2 t and the next, j = 0 .. 15.
    regs_up<kSoftmaxRegs>();
    const int s = (warp >> 2) - 1 - kConvert / 128, g = lane >> 2, t = lane & 3, wt = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, half = 16u << 16;
    const uint32_t s_at = s_cols + s * kTile + lanes, o_at = o_cols + s * 128 + lanes;
    int tile0 = 0;                                          // the CTA's tiles so far
    unsigned uses = 0, last = 0, last_use = 0;              // bit b: the parity of this half's steps with buffer b; the latest step's buffer, and that parity before it
    auto products_done = [&]() { wait(sm.o_ready[s][last], last_use); };
    for (int turn_no = 0; turn(turn_no) < items; ++turn_no) {
      const Work w(plan, turn(turn_no), G);
      const int n_rows = w.st.n * G, own = w.st.len - w.st.n;
      sync_some(1, 256);                                    // both warpgroups are done with the piece before: its rows may go
      // ---- the query rows as fp16 of about their own magnitude, d / 8 lanes to a row; a batch is asked for at once
      {
        constexpr int kPieces = D / 8, kStep = 128 / kPieces, kBatch = 64 / kStep;
        const int c = wt % kPieces, first = (w.wide ? kSub * s : 64 * s) + wt / kPieces, end = first + (w.wide ? kSub : 64);
        const bf16* from = a.Q + ((size_t)w.st.start * a.qh + w.kh * G) * D + 8 * c;
        const float inv_g = 1.f / G;
#pragma unroll 1
        for (int row0 = first; row0 < end; row0 += kBatch * kStep) {
          uint4 x[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int q = w.q0 + row0 + u * kStep, j = w.q0 / G + (int)((w.q0 % G + row0 + u * kStep + 0.5f) * inv_g);   // q / G: exact, as the rest is below 2^20
            x[u] = make_uint4(0, 0, 0, 0);
            if (q < n_rows) x[u] = *reinterpret_cast<const uint4*>(from + ((size_t)j * a.qh + q - j * G) * D);
          }
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int row = row0 + u * kStep;
            const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            float mx = 0.f, down, up;
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(in[e])), fabsf(bf_hi(in[e]))));
#pragma unroll
            for (int o = kPieces / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            row_scale(mx, down, up);
            uint32_t f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 v = __floats2half2_rn(bf_lo(in[e]) * down, bf_hi(in[e]) * down);
              f[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            *reinterpret_cast<uint4*>(sm.q[row >> 7] + piece(row & 127, c)) = make_uint4(f[0], f[1], f[2], f[3]);
            if (c == 0) sm.up[row] = up;
          }
        }
      }
      tc::fence_proxy_async_smem();
      arrive(sm.q_full);
      sync_some(1, 256);
      const int sub = w.wide ? kSub * s : 0, row = 32 * (warp & 3) + g;   // this thread's rows: sub + row + 8 r
      float qf[4], m[4], l[4];
      int lim[4];                                           // positions below it are attended to,
      unsigned long long bits[4];                           // and of the step's own rows these
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int q = w.q0 + sub + row + 8 * r;
        qf[r] = a.scale_log2 * sm.up[sub + row + 8 * r];
        m[r] = -1e30f;
        l[r] = 0.f;
        lim[r] = q >= n_rows ? 0 : w.st.tree ? own : own + q / G + 1;
        bits[r] = q < n_rows && w.st.tree ? plan.masks[w.st.start + q / G] : 0;
      }
      const int all_see = own + (w.st.tree ? 0 : (w.q0 + sub) / G + 1);   // positions that every row of this half attends to
      const int steps = w.wide ? w.tiles : (w.tiles + 1 - s) >> 1;
      for (int it = 0; it < steps; ++it) {
        const int i = w.wide ? it : 2 * it + s, tile = tile0 + i, slot = tile & 3, p0 = (w.t0 + i) * kTile + 2 * t;   // this thread's first position
        wait(sm.s_ready[s][tile & 1], uses >> (tile & 1) & 1);
        tc::fence_after_sync();
        const float *ks_at = sm.ks[slot] + 2 * t, *vs_at = sm.vs[slot] + 2 * t, *lg_at = sm.lg[slot] + 2 * t;
        auto pair = [](const float* of, int j) { return *reinterpret_cast<const uint64_t*>(of + 8 * j); };
        // Scores of 16 positions, rows 2 h and 2 h + 1: v[h][4 j + 2 (r & 1) + e].
        auto read = [&](int c, uint32_t (&v)[2][8]) {
          tc::tmem_ld_frag16(s_at + 16 * c, v[0]);
          tc::tmem_ld_frag16(s_at + half + 16 * c, v[1]);
        };
        auto landed = [](uint32_t (&v)[2][8]) {             // nothing that was read is used before
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) asm volatile("" : "+r"(v[0][e]), "+r"(v[1][e]));
        };
        const bool masked = (w.t0 + i + 1) * kTile > all_see;
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};             // bit 2 j + e: position 8 j + e of this thread's is attended to
        if (masked) {
#pragma unroll
          for (int r = 0; r < 4; ++r) see[r] = below(lim[r] - p0) | (bits[r] ? among(bits[r], p0 - own) : 0);
        }
        // ---- weights in one sweep against the present maxima; stored if none turned out too large
        auto sweep = [&](auto partly) {
          constexpr bool kPartly = decltype(partly)::value;
          uint32_t v[2][2][8], out[2][32];                  // out[pair of rows][2 j + (r & 1)]: weights of two positions
          uint64_t sum[4] = {0, 0, 0, 0};
          __half2 top = __float2half2_rn(0.f);              // the largest
          read(0, v[0]);
          landed(v[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (c < 7) read(c + 1, v[(c + 1) & 1]);
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
              const int j = 2 * c + jj;
              const uint64_t ks = pair(ks_at, j), vs = pair(vs_at, j);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const uint32_t* x = &v[c & 1][r >> 1][4 * jj + 2 * (r & 1)];
                const uint64_t e = fma2(mul2(join(x[0], x[1]), ks), pack2(qf[r], qf[r]), pack2(-m[r], -m[r]));
                uint64_t p = pack2(exp2_fast(first(e)), exp2_fast(second(e))), pv = mul2(p, vs);
                if (kPartly) {                              // both: a scale that is not attended to may be NaN
                  const bool s0 = see[r] >> (2 * j) & 1, s1 = see[r] >> (2 * j + 1) & 1;
                  p = pack2(s0 ? first(p) : 0.f, s1 ? second(p) : 0.f);
                  pv = pack2(s0 ? first(pv) : 0.f, s1 ? second(pv) : 0.f);
                }
                sum[r] = add2(sum[r], p);
                const __half2 h2 = __floats2half2_rn(first(pv), second(pv));
                out[r >> 1][2 * j + (r & 1)] = *reinterpret_cast<const uint32_t*>(&h2);
                top = __hmax2(top, h2);
              }
            }
            if (c < 7) landed(v[(c + 1) & 1]);
          }
          float sums[4], most = 0.f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sums[r] = first(sum[r]) + second(sum[r]);
            most = fmaxf(most, sums[r]);
          }
          // a sum by itself too: where V is zero the weight is, or NaN, whatever p is
          const bool good = __all_sync(0xffffffffu, fmaxf(__low2float(top), __high2float(top)) <= kLargest && most < kLargestSum);
          if (good) {
#pragma unroll
            for (int r = 0; r < 4; ++r) l[r] += sums[r];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int c = 0; c < 2; ++c) tc::tmem_st_pairs32(s_at + h * half + 32 * c, *reinterpret_cast<const uint32_t(*)[16]>(&out[h][16 * c]));
          }
          return good;
        };
        // ---- the rows' maxima of score + log2 of V's scale, of the tile's first `many` positions, and what goes by them
        auto move = [&](float (&mx)[4]) {
          float f[4];
          bool moves = false;
#pragma unroll
          for (int r = 0; r < 4; ++r) {                     // each row by itself: its neighbours stand elsewhere in another step
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            const float mn = mx[r] > m[r] + 8.f ? mx[r] : m[r];
            moves |= mn != m[r];
            f[r] = exp2_fast(m[r] - mn);
            l[r] = scaled_down(l[r], m[r] - mn);
            m[r] = mn;
          }
          if (it > 0 && __any_sync(0xffffffffu, moves)) {   // O holds the tiles before
            products_done();
            tc::fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[2][16];
#pragma unroll
              for (int h = 0; h < 2; ++h) tc::tmem_ld_frag32(o_at + h * half + c, o[h]);
              tc::tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(o[h][e]));
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[h][e] = __float_as_uint(__uint_as_float(o[h][e]) * f[2 * h + (e >> 1 & 1)]);
#pragma unroll
              for (int h = 0; h < 2; ++h) tc::tmem_st_frag32(o_at + h * half + c, o[h]);
            }
          }
        };
        auto maxima = [&](int many) {
          float mx[4] = {-1e30f, -1e30f, -1e30f, -1e30f};
#pragma unroll 1
          for (int c = 0; c < many / 16; c += 2) {
            uint32_t v[2][2][8];
            read(c, v[0]);
            read(c + 1, v[1]);
            landed(v[0]);
            landed(v[1]);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              const uint64_t ks = pair(ks_at + 16 * c, jj), lg = pair(lg_at + 16 * c, jj);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const uint32_t* x = &v[jj >> 1][r >> 1][4 * (jj & 1) + 2 * (r & 1)];
                const uint64_t e = fma2(mul2(join(x[0], x[1]), ks), pack2(qf[r], qf[r]), lg);
                if (see[r] >> (4 * c + 2 * jj) & 1) mx[r] = fmaxf(mx[r], first(e));
                if (see[r] >> (4 * c + 2 * jj + 1) & 1) mx[r] = fmaxf(mx[r], second(e));
              }
            }
          }
          move(mx);
        };
        // A quarter's maxima will do to begin with: the sweep notices if they do not.
        bool good = false;
#pragma unroll 1
        for (int many = it == 0 ? 32 : 0; !good && many <= kTile; many = many < kTile ? kTile : kTile + 1) {
          if (many) maxima(many);
          good = masked ? sweep(std::true_type()) : sweep(std::false_type());
        }
        // ---- or, where scores are so large that fp32's steps between them matter, in two roundings throughout
        if (!good) {
          // A score in two roundings: a maximum is one of the scores, and none lies above it by the product's own rounding.
          auto score = [&](const uint32_t (&v)[2][8], int r, int jj, int e, float ks) {
            return __fmul_rn(__fmul_rn(__uint_as_float(v[r >> 1][4 * jj + 2 * (r & 1) + e]), ks), qf[r]);
          };
          float mx[4] = {-1e30f, -1e30f, -1e30f, -1e30f};
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t v[2][8];
            read(c, v);
            landed(v);
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float ks = ks_at[16 * c + 8 * jj + e], lg = lg_at[16 * c + 8 * jj + e];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (see[r] >> (4 * c + 2 * jj + e) & 1) mx[r] = fmaxf(mx[r], __fadd_rn(score(v, r, jj, e, ks), lg));
              }
          }
          move(mx);
          float sum[4] = {};
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {                     // weights go where scores of an earlier turn were, or this one's
            uint32_t v[2][8], out[2][4];
            read(c, v);
            landed(v);
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
              const float2 ks = *reinterpret_cast<const float2*>(ks_at + 16 * c + 8 * jj), vs = *reinterpret_cast<const float2*>(vs_at + 16 * c + 8 * jj);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                // the product is selected too: a scale that is not attended to may be NaN
                const uint32_t here = see[r] >> (4 * c + 2 * jj);
                const float x0 = exp2_fast(__fadd_rn(score(v, r, jj, 0, ks.x), -m[r])), x1 = exp2_fast(__fadd_rn(score(v, r, jj, 1, ks.y), -m[r]));
                const float y0 = here & 1 ? x0 : 0.f, y1 = here & 2 ? x1 : 0.f;
                sum[r] += y0 + y1;
                const __half2 h2 = __floats2half2_rn(here & 1 ? x0 * vs.x : 0.f, here & 2 ? x1 * vs.y : 0.f);
                out[r >> 1][2 * jj + (r & 1)] = *reinterpret_cast<const uint32_t*>(&h2);
              }
            }
            tc::tmem_st_pairs8(s_at + 8 * c, out[0]);
            tc::tmem_st_pairs8(s_at + half + 8 * c, out[1]);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) l[r] += sum[r];
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        arrive(sm.p_ready[s]);
        last = tile & 1;
        last_use = uses >> last & 1;
        uses ^= 1u << last;
      }
      tile0 += w.tiles;

      // ---- the rows' outputs, or this piece's records
      if (steps > 0) products_done();
      tc::fence_after_sync();
      float f0[4], f1[4];                                   // factors of this warpgroup's sums, and of the other's
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        f0[r] = 1.f;
        f1[r] = 0.f;
      }
      if (!w.wide) {
        if (s == 1 && t == 0) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sm.m[row + 8 * r] = m[r];
            sm.l[row + 8 * r] = l[r];
          }
        }
      }
      float* other = reinterpret_cast<float*>(sm.q[1]) + wt;   // the second half's rows are free where both have the same
#pragma unroll 1
      for (int hc = 0; hc < 2; ++hc) {                      // a half of the elements
        constexpr int kF = D / 64;
        float o[2][kF][16];                                 // [pair of rows][32 elements]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int f = 0; f < kF; ++f) {
            uint32_t x[16];
            tc::tmem_ld_frag32(o_at + h * half + hc * (D / 2) + 32 * f, x);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(x[e]));
#pragma unroll
            for (int e = 0; e < 16; ++e) o[h][f][e] = steps > 0 ? __uint_as_float(x[e]) : 0.f;
          }
        if (!w.wide) {
          if (s == 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int f = 0; f < kF; ++f)
#pragma unroll
                for (int e = 0; e < 16; ++e) other[((h * kF + f) * 16 + e) * 128] = o[h][f][e];
          }
          sync_some(1, 256);
          if (s == 0) {
            if (hc == 0) {
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float om = sm.m[row + 8 * r], mn = fmaxf(m[r], om);
                f0[r] = exp2_fast(m[r] - mn);
                f1[r] = exp2_fast(om - mn);
                l[r] = scaled_down(l[r], m[r] - mn) + scaled_down(sm.l[row + 8 * r], om - mn);
                m[r] = mn;
              }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int f = 0; f < kF; ++f)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const int r = 2 * h + (e >> 1 & 1);
                  o[h][f][e] = fmaf(other[((h * kF + f) * 16 + e) * 128], f1[r], o[h][f][e] * f0[r]);
                }
          }
          sync_some(1, 256);
          if (s == 1) continue;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int q = w.q0 + sub + row + 8 * r, j = q / G, head = w.kh * G + q - j * G;
          if (w.piece != (int)kWhole) {
            if (q < n_rows) {
              const size_t rec = (size_t)w.st.rec + ((size_t)j * a.qh + head) * w.st.most + w.piece;
              if (hc == 0 && t == 0) a.rec_ml[rec] = make_float2(m[r], l[r]);
              float* to = a.rec_o + rec * D + hc * (D / 2) + 2 * t;
#pragma unroll
              for (int f = 0; f < kF; ++f)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float* x = &o[r >> 1][f][4 * e + 2 * (r & 1)];
                  *reinterpret_cast<float2*>(to + 32 * f + 8 * e) = make_float2(x[0], x[1]);
                }
            }
          } else {
            const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];   // nothing to attend to: zeros
#pragma unroll
            for (int f = 0; f < kF; ++f) {
              uint32_t p[4];                                // elements 8 e + 2 t and the next of 32
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float* x = &o[r >> 1][f][4 * e + 2 * (r & 1)];
                const __nv_bfloat162 v = __floats2bfloat162_rn(x[0] * inv, x[1] * inv);
                p[e] = *reinterpret_cast<const uint32_t*>(&v);
              }
              // turned among the row's four threads: elements 8 t .. 8 t + 7
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const uint32_t back = __shfl_xor_sync(0xffffffffu, t & 1 ? p[e] : p[e + 1], 1);
                if (t & 1) p[e] = back;
                else p[e + 1] = back;
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t back = __shfl_xor_sync(0xffffffffu, t & 2 ? p[e] : p[e + 2], 2);
                if (t & 2) p[e] = back;
                else p[e + 2] = back;
              }
              if (q < n_rows)
                *reinterpret_cast<uint4*>(a.O + ((size_t)(w.st.start + j) * a.qh + head) * D + hc * (D / 2) + 32 * f + 8 * t) = make_uint4(p[0], p[1], p[2], p[3]);
            }
          }
        }
      }
      tc::fence_before_sync();                              // O is read before the next piece's products
    }
  }
  if (!ok) sm.gave_up = 1;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(s_cols, kTmemCols);
  if (sm.gave_up) {                                         // NaN in all rows of this CTA's pieces
    for (int r = 0; turn(r) < items; ++r) {
      const Work w(plan, turn(r), G);
      for (int u = tid; u < w.rows * D; u += kThreads) {
        const int q = w.q0 + u / D, j = q / G, head = w.kh * G + q - j * G;
        if (w.piece != (int)kWhole) a.rec_ml[(size_t)w.st.rec + ((size_t)j * a.qh + head) * w.st.most + w.piece] = make_float2(0.f, __uint_as_float(0x7FC00000u));
        else a.O[((size_t)(w.st.start + j) * a.qh + head) * D + u % D] = __ushort_as_bfloat16(0x7FC0);
      }
    }
  }
}

// The rows of cut blocks: a head of a row to a warp and turn, its records in
// ascending order, a lane d / 32 elements.
constexpr int kMergeWarps = 8, kMergeAhead = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) k_kv8_rows_merge(RowsArgs a) {
  constexpr int E = D / 32;
  using Part = typename std::conditional<E == 4, float4, float2>::type;
  __shared__ int unit[kMaxStreams];
  const Plan plan(const_cast<void*>(a.plan), a.B, a.T);
  const bool mine = fits(*plan.head, a);
  const int units = mine ? plan.head->units : 0, lane = threadIdx.x & 31, G = a.qh / a.c.kvh;
  for (int b = threadIdx.x; b < a.B && mine; b += kMergeWarps * 32) unit[b] = plan.streams[b].unit;
  __syncthreads();
  pdl_wait();
  for (int u = blockIdx.x * kMergeWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kMergeWarps) {
    int lo = 0, hi = a.B;                                   // the last stream whose units begin at or before u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (unit[mid] <= u) lo = mid;
      else hi = mid;
    }
    const PlanStream st = plan.streams[lo];
    const int local = u - st.unit, j = local / a.qh, head = local - j * a.qh, kh = head / G, block = (j * G + head - kh * G) / kBlockRows;
    const int n = Pieces(block * a.c.kvh + kh, Cut{st.cut, st.pitch}, extent_of(block, st.n, st.len, G, st.tree)).count;
    if (n == 1) continue;                                   // the block is whole: its outputs are there
    const size_t rec = (size_t)st.rec + (size_t)local * st.most;
    const Part* o = reinterpret_cast<const Part*>(a.rec_o + rec * D) + lane;
    const float2* ml = a.rec_ml + rec;
    float mx = -1e30f, den = 0.f, acc[E] = {};
    for (int r = lane; r < n; r += 32) mx = fmaxf(mx, ml[r].x);
    mx = warp_max(mx);
    for (int r0 = 0; r0 < n; r0 += kMergeAhead) {
      Part part[kMergeAhead];
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k)
        if (r0 + k < n) part[k] = o[(r0 + k) * 32];
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k)
        if (r0 + k < n) {
          const float2 x = ml[r0 + k];
          const float f = exp2f(x.x - mx);
          den += x.y * exp2f(fmaxf(x.x - mx, -120.f)) * exp2f(fminf(x.x - mx + 120.f, 0.f));   // as scaled_down
          const float* p = reinterpret_cast<const float*>(&part[k]);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(p[e], f, acc[e]);
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    bf16* to = a.O + ((size_t)(st.start + j) * a.qh + head) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) *reinterpret_cast<__nv_bfloat162*>(to + 2 * e) = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  }
}

template <int D, int FMT>
cudaError_t launch_rows(const RowsArgs& a, int64_t records, cudaStream_t s) {
  const size_t smem = sizeof(RowsSmem<D>) + 1024;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [&] {
    cudaFuncAttributes at;
    cudaError_t x = cudaFuncGetAttributes(&at, k_kv8_rows<D, FMT>);
    // the warpgroups' shares are cut from this many; with fewer, one would wait for registers that never come
    if (x == cudaSuccess && at.numRegs != kLaunchRegs) x = cudaErrorInvalidKernelImage;
    return x != cudaSuccess ? x : cudaFuncSetAttribute(k_kv8_rows<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min<int64_t>(kSms, most_items(a.B, a.T, a.qh, a.c.kvh));
  e = launch_k(false, k_kv8_rows<D, FMT>, dim3(grid), dim3(kThreads), smem, s, a);
  if (e != cudaSuccess || records == 0) return e;
  const int64_t units = std::min<int64_t>(records, (int64_t)a.T * a.qh);
  return launch_k(true, k_kv8_rows_merge<D>, dim3((unsigned)std::min<int64_t>((units + kMergeWarps - 1) / kMergeWarps, 4 * kSms)), dim3(kMergeWarps * 32), 0, s, a);
}

}  // namespace
}  // namespace bm

extern "C" {

size_t kv8_rows_workspace_bytes(int B, int T, int q_heads, int kv_heads, int head_dim, int ctx_cap) {
  using namespace bm::kv8;
  if (!step_shapes_ok(B, T, q_heads, kv_heads) || (head_dim != 64 && head_dim != 128) || ctx_cap < 1) return 0;
  return 16 + (size_t)most_records(B, T, q_heads, kv_heads, ctx_cap) * (head_dim + 2) * sizeof(float);
}

bm_status kv8_attend_rows(const bm_kv8_cache* c, const void* plan, size_t plan_bytes, const uint16_t* Q, int q_heads, float scale, uint16_t* O,
                          int B, int T, void* ws, size_t ws_bytes, void* stream) {
  using namespace bm;
  auto refuse = [](const std::string& what) { return set_error(BM_ERR_INVALID_ARG, "kv8_attend_rows: " + what); };
  RowsArgs a{};
  bm_status st = kv8::check_cache(c, "kv8_attend_rows", &a.c);
  if (st != BM_OK) return st;
  if (!plan || !Q || !O || !ws) return refuse("null pointer");
  if (((uintptr_t)Q | (uintptr_t)O | (uintptr_t)ws | (uintptr_t)plan) & 15) return refuse("Q, O, the plan and the workspace must be 16-byte aligned");
  if (!kv8::step_shapes_ok(B, T, q_heads, c->kv_heads))
    return refuse("need 1 <= B <= 1024, 1 <= T <= 1048576, q_heads <= 1024 and a multiple of kv_heads, at most 8 query heads per kv head");
  if (!(scale > 0.f) || !(scale < INFINITY)) return refuse("scale must be positive and finite");
  if (plan_bytes < kv8::plan_bytes(B, T, q_heads, c->kv_heads)) return refuse("a plan of " + std::to_string(plan_bytes) + " bytes is none of this B, T and heads");
  const size_t need = kv8_rows_workspace_bytes(B, T, q_heads, c->kv_heads, c->head_dim, c->ctx_cap);
  if (ws_bytes < need) return refuse("workspace of " + std::to_string(ws_bytes) + " bytes, " + std::to_string(need) + " needed");
  const int64_t records = kv8::most_records(B, T, q_heads, c->kv_heads, c->ctx_cap);
  a.plan = plan;
  a.Q = reinterpret_cast<const bf16*>(Q);
  a.O = reinterpret_cast<bf16*>(O);
  a.rec_o = static_cast<float*>(ws);
  a.rec_ml = reinterpret_cast<float2*>(a.rec_o + (size_t)records * c->head_dim);
  a.B = B;
  a.T = T;
  a.qh = q_heads;
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4 = c->format == BM_KV8_E4M3, d128 = c->head_dim == 128;
  const cudaError_t e = d128 ? (e4 ? launch_rows<128, BM_KV8_E4M3>(a, records, s) : launch_rows<128, BM_KV8_INT8>(a, records, s))
                             : (e4 ? launch_rows<64, BM_KV8_E4M3>(a, records, s) : launch_rows<64, BM_KV8_INT8>(a, records, s));
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, std::string("kv8_attend_rows: ") + cudaGetErrorString(e));
  return ok();
}

}  // extern "C"
