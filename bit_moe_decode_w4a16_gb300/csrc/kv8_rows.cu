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
// positions on the 5th-generation tensor cores (fp32 sums in tensor memory):
//   S[row][position] = Q K^T, bf16 MMAs of 128 x 128 x 16, both in shared memory;
//   weights 2^(S ks qf - m) vs, as fp16, over S's place in tensor memory; m is
//     a reference at or below the running maximum of x + log2 vs, moved only when a weight passes 2^15;
//   O[row][element] += P V, MMAs of 128 x d x 16, A in tensor memory, B the
//     tile's V as it lies (positions down, elements along: N-major).
// K is converted to bf16 and V to fp16, in the same layout (128-byte swizzle), once
// for the block's two halves of 128 rows, which two warpgroups of softmax work
// on in turn: while one makes weights the other's products run.  A block of up
// to 128 rows instead gives its even tiles to one warpgroup and the odd ones
// to the other, each with sums of its own, which are joined at the end.
// Every code of either format is exact in both types.  Queries are bf16, scaled by
// a power of two so that no score overflows: exact down to 2^-126 of the row's
// largest element (in fp16 what lay 2^-17 below it lost bits, and 2^-25 all).
// Weights are fp16, which has three bits more: one loses at most
// 2^-11 of itself, or half of fp16's last step, 2^-25.  The largest weight of a row is 1 or
// more, in long pieces 2^4 or 2^8: what many light weights lose together is then at most
// 2^-12 of it in a piece of up to 2^21 positions (with 1 throughout, 2^19 positions of
// 2^-25.1 each were lost, 1.5% of it, also for elements to which the large one gives nothing).
// A reference that begins lower has less room before it is moved: 4% of the time of 1000
// rows behind 65536 positions.  Beside a large sum the tensor cores themselves cut products off
// at 2^-25 of its binary order, and sums of 16 of them at 2^-23: pieces of more than 2^17
// positions can lose more than the output's rounding to that.
// Roles: two warps issue MMAs, two warpgroups convert, K a tile ahead of V, and
// two make weights.  A thread of these has 4 rows x 32 positions of a tile, so
// that a load of scales serves 8 scores, and works on half a tile at a time
// against the reference as it stands: weights that come out too large are made
// again with the reference moved.
//
// What bounds it: the chain of a tile of 256 x 128 scores, about 4750 clocks: one
// half's weights (2400; 64 multiplications, exponentials and roundings to a
// thread, twice as long as the half's MMAs), its product, its next scores.
// Tensor cores are at work 42% of the time; then the start and end of a piece,
// 5000 to 7000 clocks of query rows, whose place comes free with the last scores,
// 5000 of outputs beside the next scores, and a first and a masked tile of
// twice the work: what short prompts and trees mostly are.  Measured, d = 128, 32 query and 4 kv heads, e4m3: a prompt of 8192
// rows 577 us (953 TFLOP/s; a warp to a row's head, fp32: 58.7 ms), 1000 rows behind
// 65536 positions (int8) 1287 us (841), 16 prompts of up to 1000 rows 118 to 123 us, 32 trees
// of up to 16 rows behind 4096 positions 47 us, one of 13 rows 23.7 us, 32 single rows
// behind 4096 75 us (they fill 8 of a half's 128 rows; kv8_attend 33).  Instructions count: at 147 KB
// of them, with weights of a whole tile at a time, the same prompts took 127 to
// 135 us; spills inside the tiles' loop cost more than a second read of tensor memory (for d = 128
// ptxas spills four bytes outside it, read once a piece).
//
// Every wait is bounded.  A CTA in which one gave up leaves NaN in the rows of all
// of its pieces and counts itself, for kv8_rows_status.
#include <type_traits>

#include "kv8_attend.cuh"
#include "kv8_step.cuh"
#include "tc_ptx.cuh"

namespace bm {
namespace {

using namespace kv8;

// What a CTA holds back, so that waits run out: failure-detection tests only.
enum Hold { kHoldNone, kHoldKeys, kHoldValues, kHoldQueries, kHoldWeights };

struct RowsArgs {
  Cache c;
  const void* plan;
  const bf16* Q;
  bf16* O;
  float4* rec_o;       // records of 16 rows: unnormalised outputs [d / 32][4][lane], in the order in which a warp holds them
  float2* rec_ml;      // [16] their maxima and sums
  int B, T, qh;
  float scale_log2;
  int hold, hold_cta, hold_at;   // a Hold; of this CTA; which of its tiles (queries: pieces; weights: the first half's steps)
};

__device__ unsigned gave_up_count;   // CTAs in which a wait gave up, ever

// The plan is for these sizes.
__device__ __forceinline__ bool fits(const PlanHead& h, const RowsArgs& a) {
  return h.magic == kPlanMagic && h.B == a.B && h.T == a.T && h.qh == a.qh && h.kvh == a.c.kvh && h.slots == a.c.slots && h.cap == a.c.cap;
}

constexpr int kSub = 128;                                   // rows of a half block
constexpr int kConvert = 256, kThreads = 128 + kConvert + 256;   // a warpgroup that issues MMAs, two of conversion, two of softmax
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 160, kConvertRegs = 64, kIssueRegs = 32;
static_assert(2 * kSoftmaxRegs + 2 * kConvertRegs + kIssueRegs <= 5 * kLaunchRegs, "warpgroups share what the launch has");
constexpr uint32_t kTmemCols = 512;                         // S of both halves (later P), O of both halves
constexpr float kLargest = 32768.f;                         // a weight above it moves its row's reference; fp16 ends at 65504
// Binary orders by which references lie below their maxima, in pieces of up to 2^13, 2^17 and more positions.
__device__ __forceinline__ float lowered(int tiles) { return tiles <= 64 ? 0.f : tiles <= 1024 ? 4.f : 8.f; }
// V scales below it count as it in a maximum: weights of positions without V are below 2^102, whatever the reference.
__device__ __forceinline__ float least_scale_log(int tiles) { return lowered(tiles) - 100.f; }
constexpr float kLargestSum = 4.056481920730334e31f;        // 2^105, of 16 positions
constexpr uint32_t kWaitLimit = 1u << 18;                   // polls of ~3.7 us: a wait gives up after about a second

// A piece as all roles see it.
struct Work {
  int start, n, slot, len;              // of the stream: first row, rows, slot, positions
  long long rec;                        // its first record
  int most, tree;
  int kh, q0, rows, wide;               // kv head; first of the block's query rows and their number; both halves have some
  int t0, tiles, piece, j0;             // tiles from t0 on; 65535: the whole block; the stream's row of the first query row
  Work() = default;
  __device__ Work(const Plan& plan, int i, int G) {
    const PlanItem it = plan.items[i];
    const PlanStream& st = plan.streams[it.who & 1023];
    start = st.start;
    n = st.n;
    slot = st.slot;
    len = st.len;
    rec = st.rec;
    most = st.most;
    tree = st.tree;
    kh = it.who >> 10;
    q0 = (it.what & 65535) * kBlockRows;
    rows = min(kBlockRows, n * G - q0);
    wide = rows > kSub;
    j0 = q0 / G;
    t0 = it.t0;
    tiles = it.t1 - it.t0;
    piece = it.what >> 16;
  }
};

template <int D>
struct RowsSmem {
  uint8_t q[2][kSub * D * 2];                               // [d / 64][row][64] bf16, swizzled
  uint8_t k[2][kTile * D * 2], v[2][kTile * D * 2];         // [d / 64][position][64], bf16 and fp16
  // scales and log2 of V's, of four tiles: they are written with a tile's K, when the softmax may be two tiles back
  float ks[4][kTile], vs[4][kTile], lg[4][kTile];
  // of the query rows of this piece and of the next: the factor that its scores are short of, its place among all heads of all rows
  // (-1: none), below which position it attends to all, and which of the step's own rows it attends to besides
  float up[2][kBlockRows];
  int to[2][kBlockRows], lim[2][kBlockRows];
  unsigned long long bits[2][kBlockRows];
  Work work[8];                                             // by turn: written two ahead of the conversion's, which is up to four ahead of the softmax's
  float m[2][kSub], l[2][kSub];                             // maxima and sums of halves that have the same rows
  uint64_t k_full[2], v_full[2];                            // by the tile's parity
  uint64_t s_ready[2][2], o_ready[2][2];                    // by half and the tile's parity: they also say that K, V may be overwritten
  uint64_t p_ready[2], turn[2];                             // by half
  uint64_t q_full, drained;
  uint32_t tmem;
  int gave_up, stop[2];                                     // a wait gave up; one of the softmax's, by the turn's parity
};

// 16-byte piece c of row r: 128-byte rows of 64 elements, pieces swizzled by the row.
__device__ __forceinline__ uint32_t piece(int r, int c) { return (c >> 3) * kTile * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4); }
// Descriptors with the 128-byte swizzle (layout type 2), 8-row atoms of 1024 bytes: the low word, to which a start 16 bytes further on
// adds 1, and the whole.  Rows of K and Q: the start moves by 32 bytes per 16 elements.  V, N-major: by 16 rows per 16
// positions, and blocks of 64 elements lie 128 rows apart.
__device__ __forceinline__ uint32_t k_major(uint32_t at) { return at >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t n_major(uint32_t at) { return at >> 4 | (uint32_t)(kTile * 128 >> 4) << 16; }
__device__ __forceinline__ uint64_t operand(uint32_t low) { return (uint64_t)low | (uint64_t)((1024u >> 4) | 1u << 14 | 2u << 29) << 32; }

// Four codes -> two bf16 pairs (exact).
template <int FMT>
__device__ __forceinline__ void codes4_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == BM_KV8_E4M3) {
    codes4<FMT>(w, lo, hi);
    auto again = [](uint32_t& x) {
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x));
      const __nv_bfloat162 z = __floats2bfloat162_rn(y.x, y.y);
      x = *reinterpret_cast<const uint32_t*>(&z);
    };
    again(lo);
    again(hi);
  } else {
    // a code is its low seven bits less 128 if its sign is set: 0x43 in front of u < 128 is the bf16 128 + u, in front of 128 it is 256
    auto pair = [](uint32_t x) {
      const uint32_t a = x & 0xFF7FFF7Fu, b = x & 0xFF80FF80u;
      const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&y);
    };
    lo = pair(__byte_perm(w, 0x43434343u, 0x4140));
    hi = pair(__byte_perm(w, 0x43434343u, 0x4342));
  }
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// As tc::mbar_wait with kWaitLimit, in a few instructions: what all warps run has to fit the instruction cache.
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 0;\n"
      "again:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " @p bra over;\n add.u32 n, n, 1;\n setp.lt.u32 q, n, %3;\n @q bra again;\n"
      "over:\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "n"(kWaitLimit)
      : "memory");
  return done;
}
__device__ __forceinline__ void sync_some(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t join(uint32_t lo, uint32_t hi) { return (uint64_t)lo | (uint64_t)hi << 32; }

// A row's 32 elements, of which thread t of its four has x[4 j + e], element 8 j + 2 t + e: scaled and rounded to bf16, and turned among
// the four so that thread t gets elements 8 t .. 8 t + 7.
__device__ __forceinline__ uint4 rounded_row(const float* x, float by, int t) {
  uint32_t p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[4 * j] * by, x[4 * j + 1] * by);
    p[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const uint32_t back = __shfl_xor_sync(0xffffffffu, t & 1 ? p[j] : p[j + 1], 1);
    if (t & 1) p[j] = back;
    else p[j + 1] = back;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t back = __shfl_xor_sync(0xffffffffu, t & 2 ? p[j] : p[j + 2], 2);
    if (t & 2) p[j] = back;
    else p[j + 2] = back;
  }
  return make_uint4(p[0], p[1], p[2], p[3]);
}

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
    sm.work[0] = Work(plan, turn(0), G);
    if (turn(1) < items) sm.work[1] = Work(plan, turn(1), G);
    sm.gave_up = sm.stop[0] = sm.stop[1] = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t s_cols = sm.tmem, o_cols = s_cols + 2 * kTile;
  // Completion number n (from 0) of a barrier.  A thread whose wait gave up goes on without waiting and arrives nowhere, so that
  // all threads take the same way through the barriers of their warpgroup.
  bool ok = true;
  auto wait = [&](uint64_t& bar, int n) {
    if (ok) ok = bounded_wait(tc::smem_u32(&bar), n & 1);
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
      constexpr uint32_t qk = tc::idesc_bf16_f32(kSub, kTile), pv = tc::idesc_f16_f32(kSub, D) | tc::kIdescBMajorN;
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
        if (s < steps) wait(sm.q_full, r);
        if (s < steps) wait(sm.k_full[tile_of(s) & 1], tile_of(s) >> 1);
        my_turn();
        if (s < steps) scores(s);
        pass();
        // the next piece's query rows into L2; its fields were there before this piece's first codes
        if (ok && s < steps && turn(r + 1) < items) {
          const Work& next = sm.work[(r + 1) & 7];
          const int q0 = next.q0 + s * kSub + lane, end = min(next.n * G, next.q0 + kBlockRows);
          const bf16* from = a.Q + ((size_t)next.start * a.qh + next.kh * G) * D;
          for (int q = q0; q < min(end, q0 - lane + kSub); q += 32) {
            const bf16* at = from + ((size_t)(q / G) * a.qh + q % G) * D;
#pragma unroll
            for (int e = 0; e < D; e += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + e));
          }
        }
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
    } else if (warp == 2 && lane == 0 && a.hold != kHoldNone && a.hold_cta == (int)blockIdx.x) {
      // A warp without work, so that the others' code is what always runs: bytes are awaited on the barrier's phase that never come.
      const bool by_tile = a.hold == kHoldKeys || a.hold == kHoldValues;
      uint64_t& bar = a.hold == kHoldKeys ? sm.k_full[a.hold_at & 1] : a.hold == kHoldValues ? sm.v_full[a.hold_at & 1]
                      : a.hold == kHoldQueries ? sm.q_full : sm.p_ready[0];
      bool there = true;
      for (int n = 0; n < (by_tile ? a.hold_at >> 1 : a.hold_at) && there; ++n) there = bounded_wait(tc::smem_u32(&bar), n & 1);
      if (there) tc::mbar_expect_tx(tc::smem_u32(&bar), 16);
    }
  } else if (warp < 4 + kConvert / 32) {
    // ---------------- conversion: 16 codes to a thread and turn
    regs_down<kConvertRegs>();
    constexpr int kLanes = D / 16, kTurns = kTile * kLanes / kConvert;
    const int ct = tid - 128, row0 = ct / kLanes, c = ct % kLanes;
    const bool swap = c & 4;                                // the second half's pieces in the other order: no bank conflict
    uint4 kr[kTurns], vr[kTurns];
    float scale = 0.f;                                      // of position ct % 128: K's in the first warpgroup, V's in the other
    auto convert = [&](uint8_t* to, const uint4 (&x)[kTurns], bool to_bf16) {
#pragma unroll
      for (int u = 0; u < kTurns; ++u) {
        const int row = u * (kConvert / kLanes) + row0;
        const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        uint32_t f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (to_bf16) codes4_bf16<FMT>(in[e], f[2 * e], f[2 * e + 1]);
          else codes4<FMT>(in[e], f[2 * e], f[2 * e + 1]);
        }
        *reinterpret_cast<uint4*>(to + piece(row, 2 * c + swap)) = swap ? make_uint4(f[4], f[5], f[6], f[7]) : make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4*>(to + piece(row, 2 * c + !swap)) = swap ? make_uint4(f[0], f[1], f[2], f[3]) : make_uint4(f[4], f[5], f[6], f[7]);
      }
    };
    // A buffer's last tile was a step of one half or of both: it is free when that one's scores (its products) have been made.
    // Bit 2 half + buffer: the parity of the half's steps with the buffer so far; the buffer's tile was a step of the half.
    struct Buffers {
      unsigned uses = 0, theirs = 0;
      int tile = 0;
      __device__ void given(const Work& w, int i) {
        const unsigned now = (w.wide ? 5u : 1u << (2 * (i & 1))) << (tile & 1);
        theirs = (theirs & ~(5u << (tile & 1))) | now;
        uses ^= now;
        ++tile;
      }
    } of_k, of_v;
    auto free_again = [&](const Buffers& of, uint64_t (&done)[2][2]) {
      const int b = of.tile & 1;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (of.theirs >> (2 * s + b) & 1) wait(done[s][b], (of.uses >> (2 * s + b) & 1) ^ 1);
    };
    for (int r = 0; turn(r) < items; ++r) {
      const Work w(plan, turn(r), G);
      const int all_see = w.len - w.n + (w.tree ? 0 : w.j0 + 1);   // positions that every row attends to
      const size_t at0 = a.c.row(w.slot, w.kh, w.t0 * kTile);
      auto load = [&](int i, uint4 (&to)[kTurns], const uint8_t* of) {
        const uint8_t* from = of + (at0 + (size_t)i * kTile) * D + 16 * ct;
        const int left = w.len - (w.t0 + i) * kTile;
#pragma unroll
        for (int u = 0; u < kTurns; ++u)
          to[u] = u * (kConvert / kLanes) + row0 < left ? ldg_nc_v4(from + u * kConvert * 16) : make_uint4(0, 0, 0, 0);
      };
      auto load_k = [&](int i) {
        load(i, kr, a.c.K);
        scale = (ct & 127) < w.len - (w.t0 + i) * kTile ? __ldg((ct < 128 ? a.c.Ks : a.c.Vs) + at0 + (size_t)i * kTile + (ct & 127)) : 0.f;
      };
      // Some rows may not attend to some of these positions, and 0 * NaN is NaN: NaN codes of V become 0, and their positions' scales NaN.
      auto partly = [&](int i) { return FMT == BM_KV8_E4M3 && (w.t0 + i) * kTile > all_see - kTile; };
      load_k(0);
      load(0, vr, a.c.V);
      // two pieces ahead: a half without steps in a piece waits for nothing there, and has seen only what was written before the piece
      // before; not by a thread that waits for nothing any more
      if (ct == 0) {
        if (ok && turn(r + 2) < items) sm.work[(r + 2) & 7] = Work(plan, turn(r + 2), G);
      }
      // K goes a tile ahead of V, whose buffer comes free later; where V's codes are looked at with K's, it waits until they are here.
      int ik = 0, iv = 0;
#pragma unroll 1
      while (iv < w.tiles) {
        if (ik < w.tiles && (ik == iv || (ik == iv + 1 && !partly(ik)))) {
          free_again(of_k, sm.s_ready);
          const int slot = of_k.tile & 3;
          if (ct < 128) {
            sm.ks[slot][ct] = scale;
          } else {
            sm.vs[slot][ct - 128] = scale;
            sm.lg[slot][ct - 128] = fmaxf(log2_fast(scale), least_scale_log(w.tiles));
          }
          if (partly(ik)) {
            sync_some(2, kConvert);                         // the scales are there
#pragma unroll
            for (int u = 0; u < kTurns; ++u) {
              uint32_t* y = reinterpret_cast<uint32_t*>(&vr[u]);
              uint32_t any = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t nan = ((y[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                y[e] &= ~((nan >> 7) * 0xFFu);
                any |= nan;
              }
              if (any) sm.vs[slot][u * (kConvert / kLanes) + row0] = __uint_as_float(0x7FC00000u);
            }
          }
          convert(sm.k[of_k.tile & 1], kr, true);
          tc::fence_proxy_async_smem();
          arrive(sm.k_full[of_k.tile & 1]);
          of_k.given(w, ik);
          if (++ik < w.tiles) load_k(ik);
        } else {
          free_again(of_v, sm.o_ready);
          convert(sm.v[of_v.tile & 1], vr, false);
          tc::fence_proxy_async_smem();
          arrive(sm.v_full[of_v.tile & 1]);
          of_v.given(w, iv);
          if (++iv < w.tiles) load(iv, vr, a.c.V);
        }
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
    unsigned uses = 0, last = 0;                            // bit b: the parity of this half's steps with buffer b; the latest step's buffer
    auto products_done = [&]() { wait(sm.o_ready[s][last], (uses >> last & 1) ^ 1); };
    // ---- a block's query rows, brought to a magnitude of about 1, d / 8 lanes to a row, asked for while the piece before ends.  All rows
    // of the halves in use are written, whatever the block's own: 128 of this half's, or 64 of the half that both share.
    auto first_row = [&](const Work& w) { return w.wide ? kSub * s : 64 * s; };
    constexpr int kPieces = D / 8, kStep = 128 / kPieces, kBatch = 64 / kStep;
    // x / G, x below 2^9: the quotient is off by a few 2^-24 of itself, and at least 2^-4 from a border
    auto of_group = [&](int x) { return (int)__fdividef(x + 0.5f, (float)G); };
    auto ask = [&](const Work& w, int row0, uint4 (&x)[kBatch]) {
      const int c = wt % kPieces, j0 = w.j0, rest = w.q0 - j0 * G;
      const bf16* from = a.Q + ((size_t)w.start * a.qh + w.kh * G) * D + 8 * c;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int row = row0 + wt / kPieces + u * kStep, q = w.q0 + row, j = j0 + of_group(rest + row);
        x[u] = make_uint4(0, 0, 0, 0);
        if (q < w.n * G) x[u] = *reinterpret_cast<const uint4*>(from + ((size_t)j * a.qh + q - j * G) * D);
      }
    };
    auto place = [&](const Work& w, int row0, int slot, const uint4 (&x)[kBatch]) {
      static_assert(kStep % 8 == 0, "a thread's rows have one swizzle");
      const int c = wt % kPieces, j0 = w.j0, rest = w.q0 - j0 * G, own = w.len - w.n;
      uint8_t* to = sm.q[row0 >> 7] + piece((row0 & 127) + wt / kPieces, c);
      float* up_to = sm.up[slot] + row0 + wt / kPieces;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        uint32_t mx2 = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) mx2 = max_bf16x2(mx2, in[e] & 0x7FFF7FFFu);
#pragma unroll
        for (int o = kPieces / 2; o > 0; o >>= 1) mx2 = max_bf16x2(mx2, __shfl_xor_sync(0xffffffffu, mx2, o));
        float down, up;
        row_scale(fmaxf(bf_lo(mx2), bf_hi(mx2)), down, up);
        uint32_t f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t y = mul2(pack2(bf_lo(in[e]), bf_hi(in[e])), pack2(down, down));
          const __nv_bfloat162 v = __floats2bfloat162_rn(first(y), second(y));
          f[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(to + u * kStep * 128) = make_uint4(f[0], f[1], f[2], f[3]);
        if (c == 0) up_to[u * kStep] = up;
      }
      // a row to a thread: what else there is to know of it
      if (wt < 64) {
        const int row = row0 + wt, q = w.q0 + row, j = j0 + of_group(rest + row);
        const bool live = q < w.n * G;
        sm.to[slot][row] = live ? (w.start + j) * a.qh + w.kh * G + q - j * G : -1;
        sm.lim[slot][row] = w.tree ? own : own + j + 1;
        sm.bits[slot][row] = live && w.tree ? plan.masks[w.start + j] : 0;
      }
    };
    auto place_all = [&](const Work& w, int slot, uint4 (&x)[kBatch]) {
#pragma unroll 1
      for (int k = 0; k <= w.wide; ++k) {
        if (k) ask(w, first_row(w) + 64, x);
        place(w, first_row(w) + 64 * k, slot, x);
      }
      tc::fence_proxy_async_smem();
      arrive(sm.q_full);
    };
    const int row = 32 * (warp & 3) + g;                    // this thread's rows of its half: row + 8 r
#pragma unroll 1
    for (int turn_no = -1;; ++turn_no) {                    // a piece, and the next one's query rows: -1, the first one's alone
      const bool more = turn(turn_no + 1) < items;
      const Work& next = sm.work[(turn_no + 1) & 7];
      float m[4], l[4];
      if (turn_no >= 0) {
        // a piece's other fields are read where they are needed rather than held: the tiles' loop needs the registers
        bool wide;
        int tiles, t0, lowest, highest;                       // below `lowest` all of the warp's rows attend to, from `highest` on none does
        {
          const Work w = sm.work[turn_no & 7];
          wide = w.wide;
          tiles = w.tiles;
          t0 = w.t0;
          const int own = w.len - w.n, rest = w.q0 - w.j0 * G, a_at = (wide ? kSub * s : 0) + 32 * (warp & 3), z_at = min(a_at + 31, w.rows - 1);
          lowest = own + (w.tree ? 0 : w.j0 + of_group(rest + a_at) + 1);
          highest = z_at < a_at ? 0 : own + (w.tree ? min(w.n, kDrafts) : w.j0 + of_group(rest + z_at) + 1);
        }
        const int info = turn_no & 1, mine_at = (wide ? kSub * s : 0) + row;
        float qf[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          m[r] = -1e30f;
          l[r] = 0.f;
        }
        const int steps = wide ? tiles : (tiles + 1 - s) >> 1;
        for (int it = 0; it < steps; ++it) {
          const int i = wide ? it : 2 * it + s, tile = tile0 + i, slot = tile & 3, p0 = (t0 + i) * kTile + 2 * t;   // this thread's first position
          wait(sm.s_ready[s][tile & 1], uses >> (tile & 1) & 1);
          tc::fence_after_sync();
          if (it == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) qf[r] = a.scale_log2 * sm.up[info][mine_at + 8 * r];
          }
          const float *ks_at = sm.ks[slot] + 2 * t, *vs_at = sm.vs[slot] + 2 * t, *lg_at = sm.lg[slot] + 2 * t;
          auto pair = [](const float* of, int j) { return *reinterpret_cast<const uint64_t*>(of + 8 * j); };
          // Scores of 32 positions, rows 2 h and 2 h + 1: v[h][4 j + 2 (r & 1) + e].
          auto read = [&](int c, uint32_t (&v)[2][16]) {
            tc::tmem_ld_frag32(s_at + 32 * c, v[0]);
            tc::tmem_ld_frag32(s_at + half + 32 * c, v[1]);
          };
          auto landed = [](auto& v) {                         // nothing that was read is used before
            tc::tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (auto& x : v[h]) asm volatile("" : "+r"(x));
          };
          // of this tile's positions; a row that ends among them has bits of its own
          const int lo = lowest - (t0 + i) * kTile, hi = highest - (t0 + i) * kTile;
          uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};             // bit 2 j + e: position 8 j + e of this thread's is attended to
          if (lo < kTile) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int lim = sm.lim[info][mine_at + 8 * r];
              const unsigned long long bits = sm.bits[info][mine_at + 8 * r];
              see[r] = below(lim - p0);
              if (bits) see[r] |= among(bits, p0 - lim);      // a tree's rows attend to all before the step's own
            }
          }
          // None of them too large, nor a sum by itself (where V is zero the weight is, or NaN, whatever p is): the sums are kept.
          auto keep = [&](const uint64_t (&sum)[4], __half2 top, bool held) {
            float sums[4], most = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              sums[r] = first(sum[r]) + second(sum[r]);
              most = fmaxf(most, sums[r]);
            }
            const bool good = held || __all_sync(0xffffffffu, fmaxf(__low2float(top), __high2float(top)) <= kLargest && most < kLargestSum);
            if (good) {
#pragma unroll
              for (int r = 0; r < 4; ++r) l[r] += sums[r];
            }
            return good;
          };
          // Weights of 32 positions against the present references.
          auto weights = [&](int c, const uint32_t (&v)[2][16], uint32_t (&out)[2][8], bool held) {
            uint64_t sum[4] = {0, 0, 0, 0};
            __half2 top = __float2half2_rn(0.f);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              const uint64_t ks = pair(ks_at + 32 * c, jj), vs = pair(vs_at + 32 * c, jj);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const uint32_t* x = &v[r >> 1][4 * jj + 2 * (r & 1)];
                const uint64_t e = fma2(mul2(join(x[0], x[1]), ks), pack2(qf[r], qf[r]), pack2(-m[r], -m[r]));
                float e0 = first(e), e1 = second(e);
                if (held) {
                  // a maximum is less than low + 1 above its reference
                  const float low = lowered(tiles), most0 = low + 2.f - lg_at[32 * c + 8 * jj], most1 = low + 2.f - lg_at[32 * c + 8 * jj + 1];
                  e0 = e0 > most0 ? most0 : e0;               // NaN stays
                  e1 = e1 > most1 ? most1 : e1;
                }
                uint64_t p = pack2(exp2_fast(e0), exp2_fast(e1)), pv = mul2(p, vs);
                // both: a scale that is not attended to may be NaN
                const bool s0 = see[r] >> (8 * c + 2 * jj) & 1, s1 = see[r] >> (8 * c + 2 * jj + 1) & 1;
                p = pack2(s0 ? first(p) : 0.f, s1 ? second(p) : 0.f);
                pv = pack2(s0 ? first(pv) : 0.f, s1 ? second(pv) : 0.f);
                sum[r] = add2(sum[r], p);
                const __half2 h2 = __floats2half2_rn(first(pv), second(pv));
                out[r >> 1][2 * jj + (r & 1)] = *reinterpret_cast<const uint32_t*>(&h2);
                top = __hmax2(top, h2);
              }
            }
            return keep(sum, top, held);
          };
          // Weights go where scores were read: 32 positions' into 16 columns.
          auto put = [&](int c, const uint32_t (&out)[2][8]) {
            tc::tmem_st_frag16(s_at + 16 * c, out[0]);
            tc::tmem_st_frag16(s_at + half + 16 * c, out[1]);
          };
          // References of rows whose maxima have risen follow them, in whole numbers: the weights of the tile's positions before 32 c,
          // which are made already, scale exactly.  (Where maxima are so large that fp32 has no such numbers, they are the references.)
          auto move = [&](int c, float (&mx)[4]) {
            float f[4];
            bool moves = false;
            const float low = lowered(tiles);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
              mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
              f[r] = 1.f;
              if (mx[r] > m[r] + low + 1.f) {                 // each row by itself: its neighbours stand elsewhere in another step
                float mn = floorf(mx[r]) - low;
                if (!(mx[r] - mn <= 9.f)) mn = mx[r];
                const float by = mn - m[r];                   // the first time 2^99 and more
                f[r] = by <= 126.f ? __uint_as_float((uint32_t)(127 - (int)by) << 23) : 0.f;
                l[r] = scaled_down(l[r], -by);
                m[r] = mn;
                moves = true;
              }
            }
            if (!__any_sync(0xffffffffu, moves) || it + c == 0) return;
            if (it > 0) {                                     // O holds the tiles before
              products_done();
              tc::fence_after_sync();
#pragma unroll 1
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t at = o_at + (k & 1 ? half : 0) + 32 * (k >> 1);
                const float fa = k & 1 ? f[2] : f[0], fb = k & 1 ? f[3] : f[1];
                uint32_t o[16];
                tc::tmem_ld_frag32(at, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(o[e]));
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * (e & 2 ? fb : fa));
                tc::tmem_st_frag32(at, o);
              }
            }
            tc::tmem_wait_st();
#pragma unroll 1
            for (int k = 0; k < 4 * c; ++k) {
              const uint32_t at = s_at + (k & 1 ? half : 0) + 8 * (k >> 1);
              const float fa = k & 1 ? f[2] : f[0], fb = k & 1 ? f[3] : f[1];   // in fp32: weights reach 2^15, and fp16 has no 2^-25
              uint32_t p[4];
              tc::tmem_ld_pairs8(at, p);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                asm volatile("" : "+r"(p[e]));
                const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&p[e]));
                const __half2 y = __floats2half2_rn(w.x * (e & 1 ? fb : fa), w.y * (e & 1 ? fb : fa));
                p[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
              tc::tmem_st_pairs8(at, p);
            }
          };
          // The maxima of score + log2 of V's scale.
          auto maxima = [&](int c, const uint32_t (&v)[2][16]) {
            float mx[4] = {-1e30f, -1e30f, -1e30f, -1e30f};
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              const uint64_t ks = pair(ks_at + 32 * c, jj), lg = pair(lg_at + 32 * c, jj);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const uint32_t* x = &v[r >> 1][4 * jj + 2 * (r & 1)];
                const uint64_t e = fma2(mul2(join(x[0], x[1]), ks), pack2(qf[r], qf[r]), lg);
                if (see[r] >> (8 * c + 2 * jj) & 1) mx[r] = fmaxf(mx[r], first(e));
                if (see[r] >> (8 * c + 2 * jj + 1) & 1) mx[r] = fmaxf(mx[r], second(e));
              }
            }
            move(c, mx);
          };
#pragma unroll 1
          for (int c2 = 0; c2 < 4; c2 += 2) {                 // half a tile at a time
            bool good = false;
            if (it + c2 > 0 && 32 * c2 + 64 <= lo) {          // every row attends to all of it: the same way for all of the warp
              uint32_t v[2][2][8], out[2][2][8];
              uint64_t sum[4] = {0, 0, 0, 0};
              __half2 top = __float2half2_rn(0.f);
              auto read16 = [&](int c, uint32_t (&to)[2][8]) {
                tc::tmem_ld_frag16(s_at + 16 * c, to[0]);
                tc::tmem_ld_frag16(s_at + half + 16 * c, to[1]);
              };
              read16(2 * c2, v[0]);
              landed(v[0]);
#pragma unroll
              for (int k = 0; k < 4; ++k) {                   // read ahead by 16 positions
                if (k < 3) read16(2 * c2 + k + 1, v[(k + 1) & 1]);
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                  const int j = 2 * k + jj;
                  const uint64_t ks = pair(ks_at + 32 * c2, j), vs = pair(vs_at + 32 * c2, j);
#pragma unroll
                  for (int r = 0; r < 4; ++r) {
                    const uint32_t* x = &v[k & 1][r >> 1][4 * jj + 2 * (r & 1)];
                    const uint64_t e = fma2(mul2(join(x[0], x[1]), ks), pack2(qf[r], qf[r]), pack2(-m[r], -m[r]));
                    const uint64_t p = pack2(exp2_fast(first(e)), exp2_fast(second(e))), pv = mul2(p, vs);
                    sum[r] = add2(sum[r], p);
                    const __half2 h2 = __floats2half2_rn(first(pv), second(pv));
                    out[k >> 1][r >> 1][2 * (j & 3) + (r & 1)] = *reinterpret_cast<const uint32_t*>(&h2);
                    top = __hmax2(top, h2);
                  }
                }
                if (k < 3) landed(v[(k + 1) & 1]);
              }
              if ((good = keep(sum, top, false))) {
                put(c2, out[0]);
                put(c2 + 1, out[1]);
              }
            }
            if (!good) {
#pragma unroll 1
              for (int c = c2; c < c2 + 2; ++c) {             // 32 positions at a time
                uint32_t out[2][8] = {};
                if (32 * c < hi) {
                  uint32_t v[2][16];
                  read(c, v);
                  landed(v);
                  // against the present references, and against moved ones; where scores are so large that fp32's steps between them
                  // matter, some lie above their maximum by its rounding, and are held
                  good = false;
#pragma unroll 1
                  for (int turn = it + c == 0; turn < 3 && !good; ++turn) {
                    if (turn) maxima(c, v);
                    good = weights(c, v, out, turn == 2);
                  }
                }
                put(c, out);
              }
            }
          }
          tc::tmem_wait_st();
          tc::fence_before_sync();
          arrive(sm.p_ready[s]);
          last = tile & 1;
          uses ^= 1u << last;
        }
        tile0 += tiles;
      }
      // ---- the next piece's query rows go first, so that its first scores are made while this one's outputs are written
      if (more) {
        if (!ok) sm.stop[turn_no & 1] = 1;
        uint4 x[kBatch];
        ask(next, first_row(next), x);
        sync_some(1, 256);                                  // both halves' scores are made
        if (sm.stop[turn_no & 1]) break;                    // both halves or none: the flag is next written behind another such barrier
        place_all(next, (turn_no + 1) & 1, x);
      }
      if (turn_no >= 0) {
        // ---- the rows' outputs, or this piece's records
        const Work& w = sm.work[turn_no & 7];
        const int n_rows = w.n * G, sub = w.wide ? kSub * s : 0, mine_at = sub + row, info = turn_no & 1;
        if (w.wide || w.tiles > s) products_done();           // this half has had steps
        tc::fence_after_sync();
        float f[2][4];                                        // where both halves have the same rows: the factors of their sums
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
          l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
        if (!w.wide) {
          if (t == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              sm.m[s][row + 8 * r] = m[r];
              sm.l[s][row + 8 * r] = l[r];
            }
          }
          tc::fence_before_sync();
          sync_some(1, 256);
          tc::fence_after_sync();
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float ma = sm.m[0][row + 8 * r], mb = sm.m[1][row + 8 * r], mn = fmaxf(ma, mb);
            f[0][r] = exp2_fast(ma - mn);
            f[1][r] = exp2_fast(mb - mn);
            l[r] = scaled_down(sm.l[0][row + 8 * r], ma - mn) + scaled_down(sm.l[1][row + 8 * r], mb - mn);
            m[r] = mn;
          }
        }
        const bool whole = w.piece == (int)kWhole;
        // the records of the warp's rows, 16 by 16: the stream's slabs of a kv head, piece by piece
        const int slabs = (n_rows + 15) >> 4, slab = (w.q0 + sub + 32 * (warp & 3)) >> 4;
        const size_t rec = (size_t)w.rec + ((size_t)w.kh * slabs + slab) * w.most + w.piece;
        float inv[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) inv[r] = l[r] == 0.f ? 0.f : 1.f / l[r];   // nothing to attend to: zeros
        if (!whole && (w.wide || s == 0) && t == 0) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (slab + (r >> 1) < slabs) a.rec_ml[(rec + (size_t)(r >> 1) * w.most) * 16 + g + 8 * (r & 1)] = make_float2(m[r], l[r]);
        }
        // 32 elements at a time: o[pair of rows][4 j + 2 (r & 1) + e] is element 8 j + 2 t + e.  Both halves' sums lie in the same lanes of
        // tensor memory, so either warpgroup can join them, and takes half of the elements.
        const uint32_t o_first = o_cols + lanes;
#pragma unroll 1
        for (int c = w.wide ? 0 : s * (D / 64); c < (w.wide ? D / 32 : (s + 1) * (D / 64)); ++c) {
          float o[2][16];
          {
            uint32_t x[2][16];
#pragma unroll
            for (int h = 0; h < 2; ++h) tc::tmem_ld_frag32((w.wide ? o_at : o_first) + h * half + 32 * c, x[h]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                asm volatile("" : "+r"(x[h][e]));
                o[h][e] = __uint_as_float(x[h][e]);
              }
          }
          if (!w.wide && w.tiles > 1) {                       // with one tile, the second half has no sums
            uint32_t x[2][16];
#pragma unroll
            for (int h = 0; h < 2; ++h) tc::tmem_ld_frag32(o_first + 128 + h * half + 32 * c, x[h]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                asm volatile("" : "+r"(x[h][e]));
                const int r = 2 * h + (e >> 1 & 1);
                o[h][e] = fmaf(__uint_as_float(x[h][e]), f[1][r], o[h][e] * f[0][r]);
              }
          }
          if (!whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (slab + h < slabs) {
                float4* at = a.rec_o + ((rec + (size_t)h * w.most) * (D / 32) + c) * 128 + lane;
#pragma unroll
                for (int e = 0; e < 4; ++e) at[32 * e] = make_float4(o[h][4 * e], o[h][4 * e + 1], o[h][4 * e + 2], o[h][4 * e + 3]);
              }
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint4 p = rounded_row(o[r >> 1] + 2 * (r & 1), inv[r], t);
              const int to = sm.to[info][mine_at + 8 * r];
              if (to >= 0) *reinterpret_cast<uint4*>(a.O + (size_t)to * D + 32 * c + 8 * t) = p;
            }
          }
        }
        tc::fence_before_sync();                            // O is read before the next piece's products
        if (!w.wide) sync_some(1, 256);                     // by both halves
      }
      if (!more) break;
    }
  }
  if (!ok) sm.gave_up = 1;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(s_cols, kTmemCols);
  if (sm.gave_up) {                                         // NaN in all rows of this CTA's pieces
    if (tid == 0) atomicAdd(&gave_up_count, 1u);
    for (int r = 0; turn(r) < items; ++r) {
      const Work w(plan, turn(r), G);
      const int slabs = (w.n * G + 15) >> 4;
      for (int u = tid; u < w.rows * D; u += kThreads) {
        const int row = u / D, q = w.q0 + row, j = q / G, head = w.kh * G + q - j * G;
        if (w.piece != (int)kWhole)
          a.rec_ml[((size_t)w.rec + ((size_t)w.kh * slabs + (q >> 4)) * w.most + w.piece) * 16 + (q & 15)] = make_float2(0.f, __uint_as_float(0x7FC00000u));
        else a.O[((size_t)(w.start + j) * a.qh + head) * D + u % D] = __ushort_as_bfloat16(0x7FC0);
      }
    }
  }
}

// The rows of cut blocks: 32 elements of 16 rows to a warp and turn, the
// pieces' records in ascending order and in the layout of the warp that wrote
// them (thread (g, t): rows g and g + 8, elements 8 j + 2 t and the next).
constexpr int kMergeWarps = 4, kMergeAhead = 4;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) k_kv8_rows_merge(RowsArgs a) {
  __shared__ int unit[kMaxStreams];
  const Plan plan(const_cast<void*>(a.plan), a.B, a.T);
  const bool mine = fits(*plan.head, a);
  const int units = mine ? plan.head->units * (D / 32) : 0, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, G = a.qh / a.c.kvh;
  for (int b = threadIdx.x; b < a.B && mine; b += kMergeWarps * 32) unit[b] = plan.streams[b].unit;
  __syncthreads();
  bool waited = false;
  for (int u = blockIdx.x * kMergeWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kMergeWarps) {
    const int slab_no = u / (D / 32), c = u % (D / 32);
    int lo = 0, hi = a.B;                                   // the last stream whose units begin at or before this one
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (unit[mid] <= slab_no) lo = mid;
      else hi = mid;
    }
    const PlanStream st = plan.streams[lo];
    const int n_rows = st.n * G, slabs = (n_rows + 15) >> 4, local = slab_no - st.unit, kh = local / slabs, slab = local - kh * slabs;
    const int block = slab / (kBlockRows / 16);
    const int n = Pieces(block * a.c.kvh + kh, Cut{st.cut, st.pitch}, extent_of(block, st.n, st.len, G, st.tree)).count;
    if (n == 1) continue;                                   // the block is whole: its outputs are there
    if (!waited) pdl_wait();                                // the plan was there before; the records are now
    waited = true;
    const size_t rec = (size_t)st.rec + (size_t)local * st.most;
    const float4* o = a.rec_o + (rec * (D / 32) + c) * 128 + lane;
    const float2* ml = a.rec_ml + rec * 16 + g;
    float mx[2] = {-1e30f, -1e30f}, den[2] = {0.f, 0.f}, acc[16] = {};
    for (int r = 0; r < n; ++r) {
      mx[0] = fmaxf(mx[0], ml[16 * r].x);
      mx[1] = fmaxf(mx[1], ml[16 * r + 8].x);
    }
    for (int r0 = 0; r0 < n; r0 += kMergeAhead) {
      float4 part[kMergeAhead][4];
      float2 x[kMergeAhead][2];
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k)
        if (r0 + k < n) {
#pragma unroll
          for (int j = 0; j < 4; ++j) part[k][j] = o[(size_t)(r0 + k) * (D / 32) * 128 + 32 * j];
          x[k][0] = ml[16 * (r0 + k)];
          x[k][1] = ml[16 * (r0 + k) + 8];
        }
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k)
        if (r0 + k < n) {
          float f[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float d = x[k][h].x - mx[h];
            f[h] = exp2f(d);
            den[h] += x[k][h].y * exp2f(fmaxf(d, -120.f)) * exp2f(fminf(d + 120.f, 0.f));   // as scaled_down
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[4 * j] = fmaf(part[k][j].x, f[0], acc[4 * j]);
            acc[4 * j + 1] = fmaf(part[k][j].y, f[0], acc[4 * j + 1]);
            acc[4 * j + 2] = fmaf(part[k][j].z, f[1], acc[4 * j + 2]);
            acc[4 * j + 3] = fmaf(part[k][j].w, f[1], acc[4 * j + 3]);
          }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 p = rounded_row(acc + 2 * h, den[h] == 0.f ? 0.f : 1.f / den[h], t);
      const int q = 16 * slab + g + 8 * h, j = q / G;
      if (q < n_rows) *reinterpret_cast<uint4*>(a.O + ((size_t)(st.start + j) * a.qh + kh * G + q - j * G) * D + 32 * c + 8 * t) = p;
    }
  }
  if (!waited) pdl_wait();                                  // done means done: the kernel before is
}

std::atomic<int> test_hold{kHoldNone}, test_hold_cta{0}, test_hold_at{0};

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
  const int64_t units = (records / 16 + (int64_t)a.T * a.qh / 16) * (D / 32);   // more than there can be
  return launch_k(true, k_kv8_rows_merge<D>, dim3((unsigned)std::min<int64_t>((units + kMergeWarps - 1) / kMergeWarps, 8 * kSms)), dim3(kMergeWarps * 32), 0, s, a);
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
  a.rec_o = static_cast<float4*>(ws);
  a.rec_ml = reinterpret_cast<float2*>(a.rec_o + (size_t)records * c->head_dim / 4);
  a.B = B;
  a.T = T;
  a.qh = q_heads;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.hold = test_hold;
  a.hold_cta = test_hold_cta;
  a.hold_at = test_hold_at;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4 = c->format == BM_KV8_E4M3, d128 = c->head_dim == 128;
  const cudaError_t e = d128 ? (e4 ? launch_rows<128, BM_KV8_E4M3>(a, records, s) : launch_rows<128, BM_KV8_INT8>(a, records, s))
                             : (e4 ? launch_rows<64, BM_KV8_E4M3>(a, records, s) : launch_rows<64, BM_KV8_INT8>(a, records, s));
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, std::string("kv8_attend_rows: ") + cudaGetErrorString(e));
  return ok();
}

bm_status kv8_rows_status(void* stream) {
  using namespace bm;
  auto fail = [](cudaError_t e) { return set_error(BM_ERR_CUDA, std::string("kv8_rows_status: ") + cudaGetErrorString(e)); };
  static std::atomic<unsigned> told[64] = {};               // per device, of what was counted on it
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(s, &capture);
  if (e != cudaSuccess) return fail(e);
  if (capture != cudaStreamCaptureStatusNone) return set_error(BM_ERR_INVALID_ARG, "kv8_rows_status: the stream is being captured");
  int dev = 0;
  unsigned count = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return fail(e);
  if (dev >= 64) return set_error(BM_ERR_UNSUPPORTED, "kv8_rows_status: more than 64 devices");
  if ((e = cudaMemcpyFromSymbolAsync(&count, gave_up_count, sizeof(count), 0, cudaMemcpyDeviceToHost, s)) != cudaSuccess) return fail(e);
  if ((e = cudaStreamSynchronize(s)) != cudaSuccess) return fail(e);
  unsigned before = told[dev];                              // two threads that ask at once tell each CTA once
  while ((int)(count - before) > 0 && !told[dev].compare_exchange_weak(before, count)) {}
  if ((int)(count - before) <= 0) return ok();
  return set_error(BM_ERR_DEVICE_CHECK, "kv8_attend_rows: a bounded wait gave up in " + std::to_string(count - before) +
                                            " CTAs; the rows that they had are NaN");
}

bm_status bm_test_kv8_rows_hold(int what, int cta, int at) {
  using namespace bm;
  if (what < kHoldNone || what > kHoldWeights || cta < 0 || at < 0)
    return set_error(BM_ERR_INVALID_ARG, "bm_test_kv8_rows_hold: need 0 <= what <= 4, cta >= 0, at >= 0");
  test_hold = what;
  test_hold_cta = cta;
  test_hold_at = at;
  return ok();
}

}  // extern "C"
