// Planning a ragged step over the 8-bit cache, and ending one of drafted trees.
//
// kv8_plan: start = the running sum of the streams' row counts; row j of
// stream b goes to position lens[b] + j, and is rotated for lens[b] + j (a run
// of consecutive rows) or lens[b] + its depth in the stream's tree.  Row j of a
// tree attends to its ancestors and itself: mask[j] = bit j | mask[parent], by
// doubling (mask |= mask[up], up = up[up]) in six rounds for 64 rows, a warp to
// a tree and two rows to a lane.  Then the attention's pieces (kv8_step.cuh),
// longest first by a counting sort.
// kv8_tree_accept: from row 0 on, the first child whose token is the model's
// choice behind its parent.  kv8_tree_keep: the kept rows' codes and scales to
// consecutive positions, all of a stream and head read before any is written.
//
// All three are latency: a few kB in the ordinary step.  One cluster of eight
// CTAs plans it: every CTA makes the streams' running sum and table for itself (at most
// 1024 of them), and rows and pieces are spread over all.
#include <cooperative_groups.h>

#include "kv8_step.cuh"

namespace bm {
namespace {

using namespace kv8;
namespace cg = cooperative_groups;

constexpr int kPlanCtas = 8, kPlanThreads = 1024, kBins = 1024;
constexpr unsigned kAll = 0xffffffffu;

struct PlanArgs {
  void* plan;
  const int32_t *slots, *lens, *counts, *parents;
  int32_t *row_start, *after, *row_slot, *row_index, *row_pos;
  int B, T, qh, kvh, num_slots, cap;
};

struct PlanSmem {
  int start[kMaxStreams + 1], count[kMaxStreams], slot[kMaxStreams], base[kMaxStreams];   // slot -1: refused
  int bad[kMaxStreams];                       // trees that are none, reported by the warp that looked, to all CTAs
  int from[kMaxStreams + 1];                  // a stream's first piece before sorting
  Cut cuts[kMaxStreams];
  int bins[kBins], places[kBins];             // this CTA's pieces by length; where the next of each goes
  long long sums[3][kPlanThreads / 32];
};

// Sums of the values of the threads before this one, and of all; every thread of the CTA calls it.
template <int N>
__device__ __forceinline__ void scan_before(long long (&v)[N], long long (*sums)[kPlanThreads / 32], long long (&all)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kAll, x[i], o);
      if (lane >= o) x[i] += y;
    }
  }
  __syncthreads();                            // `sums` may still be read from the call before
  if (lane == 31) {
#pragma unroll
    for (int i = 0; i < N; ++i) sums[i][warp] = x[i];
  }
  __syncthreads();
  if (warp < N) {
    long long s = sums[warp][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kAll, s, o);
      if (lane >= o) s += y;
    }
    sums[warp][lane] = s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    all[i] = sums[i][kPlanThreads / 32 - 1];
    v[i] = x[i] - v[i] + (warp ? sums[i][warp - 1] : 0);
  }
}

// The last of a[0 .. n - 1] (rising) that is at most x; a[0] is.
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Ancestors of a tree's rows: lane l has rows l and l + 32, `up` their parents (-1: none).
__device__ __forceinline__ void ancestors(int (&up)[2], unsigned long long (&mask)[2]) {
#pragma unroll 1
  for (int round = 0; round < 6; ++round) {   // 2^6 rows
    unsigned long long m[2];
    int u[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int from = up[k] & 31;
      const unsigned long long a = __shfl_sync(kAll, mask[0], from), b = __shfl_sync(kAll, mask[1], from);
      const int ua = __shfl_sync(kAll, up[0], from), ub = __shfl_sync(kAll, up[1], from);
      m[k] = up[k] < 0 ? 0 : up[k] < 32 ? a : b;
      u[k] = up[k] < 0 ? -1 : up[k] < 32 ? ua : ub;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      mask[k] |= m[k];
      up[k] = u[k];
    }
  }
}

// One cluster of one or kPlanCtas CTAs.
__global__ void __launch_bounds__(kPlanThreads) k_kv8_plan(PlanArgs a) {
  __shared__ PlanSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, cta = blockIdx.x, ctas = gridDim.x, B = a.B, T = a.T, G = a.qh / a.kvh;
  const Plan plan(a.plan, B, T);

  // ---- the streams
  int n = 0, base = 0, slot = -1;
  if (tid < B) {
    const int count = a.counts[tid];
    slot = a.slots[tid];
    base = a.lens[tid];
    n = min(max(count, 0), T + 1);            // more than T rows do not fit, however many
    if (slot < 0 || slot >= a.num_slots || base < 0 || count < 0 || (long long)base + count > a.cap) slot = -1;
    sm.bad[tid] = 0;
  }
  long long before[1] = {n}, all_rows[1];
  scan_before(before, sm.sums, all_rows);
  const int start = (int)before[0];           // at most 2^10 (2^20 + 1)
  const long long total = all_rows[0];
  if (tid < B) {
    if (n > 0 && (long long)start + n > T) slot = -1;
    sm.start[tid] = start;
    sm.count[tid] = n;
    sm.slot[tid] = slot;
    sm.base[tid] = base;
  }
  if (tid == 0) sm.start[B] = (int)total;
  cluster.sync();                             // sm.bad is ready for the other CTAs' reports

  auto put = [&](int t, int to, int index, int pos) {
    a.row_slot[t] = to;
    a.row_index[t] = index;
    if (a.row_pos) a.row_pos[t] = pos;
  };
  const int me = cta * kPlanThreads + tid, all = ctas * kPlanThreads;
  if (!a.parents) {
    for (int t = me; t < T; t += all) {
      const int b = last_at_most(sm.start, B + 1, t), at = b < B && sm.slot[b] >= 0 ? sm.base[b] + t - sm.start[b] : 0;
      put(t, b < B ? sm.slot[b] : -1, at, at);
    }
  } else {
    for (int t = (int)min(total, (long long)T) + me; t < T; t += all) put(t, -1, 0, 0);
    for (int b = me >> 5; b < B; b += all >> 5) {
      const int s0 = sm.start[b], c = sm.count[b], p0 = sm.base[b];
      int to = sm.slot[b];
      if (c == 0) continue;
      const bool run = to >= 0 && a.parents[s0] == -2;
      if (to < 0 || run) {
        for (int j = lane; j < c && s0 + j < T; j += 32) put(s0 + j, to, to < 0 ? 0 : p0 + j, to < 0 ? 0 : p0 + j);
        continue;
      }
      int up[2];
      unsigned long long mask[2];
      bool fits = c <= kDrafts;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int j = lane + 32 * k;
        up[k] = -1;
        mask[k] = 1ull << j;
        if (fits && j < c) {
          up[k] = a.parents[s0 + j];
          if (up[k] < -1 || up[k] >= j) {
            fits = false;
            up[k] = -1;
          }
        }
      }
      fits = __all_sync(kAll, fits);
      if (!fits) {
        to = -1;
        if (lane < ctas) cluster.map_shared_rank(sm.bad, lane)[b] = 1;
        for (int j = lane; j < c; j += 32) put(s0 + j, -1, 0, 0);
        continue;
      }
      ancestors(up, mask);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int j = lane + 32 * k;
        if (j < c) {
          plan.masks[s0 + j] = mask[k];
          put(s0 + j, to, p0 + j, p0 + __popcll(mask[k]) - 1);
        }
      }
    }
  }
  cluster.sync();

  // ---- the streams' table
  PlanStream st{};
  int blocks = 0;
  if (tid < B) {
    const bool refused = slot < 0 || sm.bad[tid];
    st.start = min(start, T);
    st.base = base;
    st.refused = refused;
    st.slot = refused ? -1 : slot;
    st.n = refused ? 0 : n;
    st.len = base + st.n;
    st.most = 1;
    if (st.n > 0) {
      st.tree = a.parents && a.parents[start] != -2;
      const Cut cut = cut_of(st.n, st.len, G, a.kvh);
      sm.cuts[tid] = cut;
      st.cut = cut.cut;
      st.pitch = cut.pitch;
      st.most = most_pieces(tiles_of(st.len), cut);
      blocks = blocks_of(st.n, G) * a.kvh;
    }
  }
  const long long slabs = st.most > 1 ? ((long long)st.n * G + 15) / 16 * a.kvh : 0;
  long long at[3] = {(long long)blocks * st.most, slabs, slabs * st.most}, sum[3];
  scan_before(at, sm.sums, sum);
  st.unit = (int)at[1];
  st.rec = at[2];
  const int items = (int)sum[0];
  if (tid < B) {
    if (cta == 0) {
      plan.streams[tid] = st;
      a.row_start[tid] = st.start;
      a.after[tid] = st.refused ? -1 : base + n;
    }
    sm.from[tid] = (int)at[0];
    sm.slot[tid] = st.n;                      // what the loops below need of a stream
    sm.base[tid] = st.len;
    sm.count[tid] = st.most;
    sm.bad[tid] = st.tree;
  }
  if (tid == 0) {
    sm.from[B] = items;
    if (cta == 0) a.row_start[B] = (int)min(total, (long long)T);
  }

  // ---- its pieces, the longest first: each CTA counts a share of them by length, and puts them behind those of the CTAs before it
  int shift = 0;                              // bins of equal width hold the longest possible piece
  for (long long most = 2ll * tiles_of(a.cap) + 8; (most >> shift) >= kBins; ++shift) {}
  sm.bins[tid] = 0;
  __syncthreads();
  auto piece = [&](int x, PlanItem& it) {     // the bin of piece x, -1: it holds nothing
    const int b = last_at_most(sm.from, B + 1, x), most = sm.count[b], local = x - sm.from[b], i = local / most, c = local - i * most;
    const int sn = sm.slot[b], len = sm.base[b], block = i / a.kvh;
    const Pieces p(i, sm.cuts[b], extent_of(block, sn, len, G, sm.bad[b]));
    if (c >= p.count) return -1;
    it.who = (unsigned)b | (unsigned)(i - block * a.kvh) << 10;
    it.what = (unsigned)block | (p.count == 1 ? kWhole : (unsigned)c) << 16;
    it.t0 = p.begin(c);
    it.t1 = p.end(c);
    const int wide = (long long)sn * G - (long long)block * kBlockRows > kBlockRows / 2;
    return kBins - 1 - (int)((((long long)(it.t1 - it.t0) << wide) + 6) >> shift);
  };
  PlanItem it;
  for (int x = me; x < items; x += all) {
    const int bin = piece(x, it);
    if (bin >= 0) atomicAdd(&sm.bins[bin], 1);
  }
  cluster.sync();
  long long first[1] = {0}, kept[1];
  int ahead = 0;
  for (int k = 0; k < ctas; ++k) {
    const int v = cluster.map_shared_rank(sm.bins, k)[tid];
    first[0] += v;
    if (k < cta) ahead += v;
  }
  scan_before(first, sm.sums, kept);
  sm.places[tid] = (int)first[0] + ahead;
  cluster.sync();                             // nobody reads another CTA's counts any more
  for (int x = me; x < items; x += all) {
    const int bin = piece(x, it);
    if (bin >= 0) plan.items[atomicAdd(&sm.places[bin], 1)] = it;
  }
  if (me == 0) *plan.head = PlanHead{kPlanMagic, B, T, a.qh, a.kvh, a.num_slots, a.cap, (int)kept[0], (int)sum[1], {}};
}

// ---------------------------------------------------------------- the end of a step of trees

constexpr int kAcceptWarps = 4;

__global__ void __launch_bounds__(kAcceptWarps * 32) k_kv8_accept(const void* p, const int32_t* tokens, const int32_t* ids, int32_t* path,
                                                                 int32_t* kept, int32_t* fresh, int32_t* n_fresh, int32_t* lens, int B, int T) {
  const Plan plan(const_cast<void*>(p), B, T);
  const int b = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= B || plan.head->magic != kPlanMagic || plan.head->B != B || plan.head->T != T) return;
  const PlanStream st = plan.streams[b];
  int way[2] = {-1, -1}, out[2] = {-1, -1}, rows = 0, made = 0;
  if (st.n > 0 && !st.tree) {
    rows = st.n;
    made = 1;
    if (lane == 0) out[0] = ids[st.start + st.n - 1];
  } else if (st.n > 0) {
    int token[2], id[2], parent[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = lane + 32 * k;
      token[k] = id[k] = -1;
      parent[k] = -1;
      if (j < st.n) {
        token[k] = tokens[st.start + j];
        id[k] = ids[st.start + j];
        const unsigned long long above = plan.masks[st.start + j] & ~(1ull << j);   // a parent is the latest ancestor
        parent[k] = above ? 63 - __clzll(above) : -1;
      }
    }
    int at = 0;
    while (true) {                            // a child comes behind its parent: at most 64 rounds
      const int i0 = __shfl_sync(kAll, id[0], at & 31), i1 = __shfl_sync(kAll, id[1], at & 31), choice = at < 32 ? i0 : i1;
      if (lane == (rows & 31)) {
        if (rows < 32) {
          way[0] = at;
          out[0] = choice;
        } else {
          way[1] = at;
          out[1] = choice;
        }
      }
      ++rows;
      const unsigned c0 = __ballot_sync(kAll, choice >= 0 && parent[0] == at && token[0] == choice);
      const unsigned c1 = __ballot_sync(kAll, choice >= 0 && parent[1] == at && token[1] == choice);
      if (!(c0 | c1)) break;
      at = c0 ? __ffs(c0) - 1 : 31 + __ffs(c1);
    }
    made = rows;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    path[b * kDrafts + lane + 32 * k] = way[k];
    fresh[b * kDrafts + lane + 32 * k] = out[k];
  }
  if (lane == 0) {
    kept[b] = rows;
    n_fresh[b] = made;
    if (!st.refused) lens[b] = st.base + rows;
  }
}

// A kv head of a stream to a CTA, 16 codes to a thread and turn; K first, then V.
constexpr int kKeepThreads = 256;

template <int D>
__global__ void __launch_bounds__(kKeepThreads) k_kv8_keep(Cache c, const void* p, const int32_t* path, const int32_t* kept, int B) {
  constexpr int kLanes = D / 16, kTurns = 2 * kDrafts * kLanes / kKeepThreads;
  __shared__ int from[kDrafts];
  const PlanHead& head = *static_cast<const PlanHead*>(p);
  const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  if (head.magic != kPlanMagic || head.B != B || head.kvh != c.kvh || head.slots != c.slots || head.cap != c.cap) return;
  const PlanStream& st = reinterpret_cast<const PlanStream*>(&head + 1)[b];
  const int rows = kept[b], n = st.n, base = st.base;
  bool wrong = !st.tree || rows < 2 || rows > n;
  if (!wrong && tid < rows) {
    const int src = path[b * kDrafts + tid];
    from[tid] = src;
    wrong = src < 0 || src >= n;
  }
  if (__syncthreads_or(wrong)) return;
  const size_t at = c.row(st.slot, h, base);
  uint4 codes[kTurns];
  float scale = 0.f;
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int u = tid + k * kKeepThreads, v = u / (kDrafts * kLanes), i = u / kLanes % kDrafts;
    if (i < rows) codes[k] = *reinterpret_cast<const uint4*>((v ? c.V : c.K) + (at + from[i]) * D + 16 * (u % kLanes));
  }
  const int i = tid % kDrafts, v = tid / kDrafts;
  if (v < 2 && i < rows) scale = (v ? c.Vs : c.Ks)[at + from[i]];
  __syncthreads();                            // everything is read
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int u = tid + k * kKeepThreads, w = u / (kDrafts * kLanes), j = u / kLanes % kDrafts;
    if (j < rows && from[j] != j) *reinterpret_cast<uint4*>((w ? c.V : c.K) + (at + j) * D + 16 * (u % kLanes)) = codes[k];
  }
  if (v < 2 && i < rows && from[i] != i) (v ? c.Vs : c.Ks)[at + i] = scale;
}

bool aligned(uintptr_t all, int to) { return !(all & (to - 1)); }

}  // namespace
}  // namespace bm

extern "C" {

size_t kv8_plan_bytes(int B, int T, int q_heads, int kv_heads) {
  return bm::kv8::step_shapes_ok(B, T, q_heads, kv_heads) ? bm::kv8::plan_bytes(B, T, q_heads, kv_heads) : 0;
}

bm_status kv8_plan(const bm_kv8_cache* c, int q_heads, const int32_t* slots, const int32_t* lens, const int32_t* counts, const int32_t* parents,
                   int32_t* row_start, int32_t* after, int32_t* row_slot, int32_t* row_index, int32_t* row_pos, int B, int T, void* plan,
                   size_t plan_bytes, void* stream) {
  using namespace bm;
  auto refuse = [](const std::string& what) { return set_error(BM_ERR_INVALID_ARG, "kv8_plan: " + what); };
  kv8::Cache cc{};
  bm_status st = kv8::check_cache(c, "kv8_plan", &cc);
  if (st != BM_OK) return st;
  if (!slots || !lens || !counts || !row_start || !after || !row_slot || !row_index || !plan) return refuse("null pointer");
  if (!kv8::step_shapes_ok(B, T, q_heads, c->kv_heads))
    return refuse("need 1 <= B <= 1024, 1 <= T <= 1048576, q_heads <= 1024 and a multiple of kv_heads, at most 8 query heads per kv head");
  if (!aligned((uintptr_t)slots | (uintptr_t)lens | (uintptr_t)counts | (uintptr_t)parents | (uintptr_t)row_start | (uintptr_t)after |
                   (uintptr_t)row_slot | (uintptr_t)row_index | (uintptr_t)row_pos, 4))
    return refuse("int32 vectors must be 4-byte aligned");
  if (!aligned((uintptr_t)plan, 16)) return refuse("the plan must be 16-byte aligned");
  const size_t need = kv8::plan_bytes(B, T, q_heads, c->kv_heads);
  if (plan_bytes < need) return refuse("plan of " + std::to_string(plan_bytes) + " bytes, " + std::to_string(need) + " needed");
  const PlanArgs a{plan, slots, lens, counts, parents, row_start, after, row_slot, row_index, row_pos, B, T, q_heads, c->kv_heads, c->slots, c->ctx_cap};
  // A CTA alone has less to wait for, eight share the pieces, whose number grows with the streams' blocks.  One and eight, us, 32 / 4 heads:
  // 8 trees of 17 rows behind 4000 positions (128 pieces) 8.0 and 9.2; 32 single rows behind 4096 (640) 8.8 and 10.0; 32 trees of 16 behind 32768
  // (1152) 13.2 and 13.3; 64 single rows behind 4096 (1280) 12.0 and 11.6; 64 trees of 32 behind 131072 (4352) 25.1 and 13.7; 512 single
  // rows 44.5 and 17.9.  Prompts of 2048, 4096 and 8192 rows: 7.4 and 8.2, 8.3 and 8.6, 10.6 and 9.9.
  const int ctas = T <= 2048 && B * c->kv_heads <= 128 ? 1 : kPlanCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_kv8_plan, a);
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, std::string("kv8_plan: ") + cudaGetErrorString(e));
  return ok();
}

bm_status kv8_tree_accept(const void* plan, size_t plan_bytes, const int32_t* tokens, const int32_t* ids, int32_t* path, int32_t* kept,
                          int32_t* fresh, int32_t* n_fresh, int32_t* lens, int B, int T, void* stream) {
  using namespace bm;
  auto refuse = [](const std::string& what) { return set_error(BM_ERR_INVALID_ARG, "kv8_tree_accept: " + what); };
  if (!plan || !tokens || !ids || !path || !kept || !fresh || !n_fresh || !lens) return refuse("null pointer");
  if (!kv8::step_shapes_ok(B, T, 1, 1)) return refuse("need 1 <= B <= 1024, 1 <= T <= 1048576");
  if (!aligned((uintptr_t)tokens | (uintptr_t)ids | (uintptr_t)path | (uintptr_t)kept | (uintptr_t)fresh | (uintptr_t)n_fresh | (uintptr_t)lens, 4))
    return refuse("int32 vectors must be 4-byte aligned");
  if (!aligned((uintptr_t)plan, 16)) return refuse("the plan must be 16-byte aligned");
  if (plan_bytes < kv8::plan_bytes(B, T, 1, 1)) return refuse("a plan of " + std::to_string(plan_bytes) + " bytes is none of this B and T");
  k_kv8_accept<<<(B + kAcceptWarps - 1) / kAcceptWarps, kAcceptWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(plan, tokens, ids, path, kept,
                                                                                                                  fresh, n_fresh, lens, B, T);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, std::string("kv8_tree_accept: ") + cudaGetErrorString(e));
  return ok();
}

bm_status kv8_tree_keep(const bm_kv8_cache* c, const void* plan, size_t plan_bytes, const int32_t* path, const int32_t* kept, int B, void* stream) {
  using namespace bm;
  auto refuse = [](const std::string& what) { return set_error(BM_ERR_INVALID_ARG, "kv8_tree_keep: " + what); };
  kv8::Cache cc{};
  bm_status st = kv8::check_cache(c, "kv8_tree_keep", &cc);
  if (st != BM_OK) return st;
  if (!plan || !path || !kept) return refuse("null pointer");
  if (B < 1 || B > kv8::kMaxStreams) return refuse("need 1 <= B <= 1024");
  if (!aligned((uintptr_t)path | (uintptr_t)kept, 4)) return refuse("int32 vectors must be 4-byte aligned");
  if (!aligned((uintptr_t)plan, 16)) return refuse("the plan must be 16-byte aligned");
  if (plan_bytes < kv8::plan_bytes(B, 1, c->kv_heads, c->kv_heads)) return refuse("a plan of " + std::to_string(plan_bytes) + " bytes is none of this B and cache");
  const dim3 grid(B, c->kv_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c->head_dim == 128) k_kv8_keep<128><<<grid, kKeepThreads, 0, s>>>(cc, plan, path, kept, B);
  else k_kv8_keep<64><<<grid, kKeepThreads, 0, s>>>(cc, plan, path, kept, B);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, std::string("kv8_tree_keep: ") + cudaGetErrorString(e));
  return ok();
}

}  // extern "C"
