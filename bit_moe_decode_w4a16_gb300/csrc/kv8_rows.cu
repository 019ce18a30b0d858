// Attention of a ragged step's rows over the 8-bit cache, each behind its own
// stream's positions.
//
// Row j of a stream with n rows and len positions (its own n included) attends
// to positions 0 .. len - n + j of its slot, or, in a tree, to 0 .. len - n - 1
// and those of its ancestors and itself:
//   o = sum_p w_p v_p / sum_p w_p,   w_p = 2^(x_p - max x),  x_p = scale log2(e) q . k_p
//
// A warp takes a head of a row and walks over its positions, 32 / (d / 16)
// at once and 16 elements to a lane, with the running maximum and sum of the weights.
#include "kv8_attend.cuh"
#include "kv8_step.cuh"

namespace bm {
namespace {

using namespace kv8;

struct RowsArgs {
  Cache c;
  const void* plan;
  const bf16* Q;
  bf16* O;
  int B, T, qh;
  float scale_log2;
};

constexpr int kWarps = 4;

template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) k_kv8_rows(RowsArgs a) {
  constexpr int kLanes = D / 16, kAt = 32 / kLanes;   // lanes of a position, positions at once
  const Plan plan(const_cast<void*>(a.plan), a.B, a.T);
  const PlanHead& h = *plan.head;
  if (h.magic != kPlanMagic || h.B != a.B || h.T != a.T || h.qh != a.qh || h.kvh != a.c.kvh || h.slots != a.c.slots || h.cap != a.c.cap) return;
  const int t = blockIdx.x, lane = threadIdx.x & 31, l = lane % kLanes, g = lane / kLanes, G = a.qh / a.c.kvh;
  int lo = 0, hi = a.B;                               // the last stream that begins at or before the row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (plan.streams[mid].start <= t) lo = mid;
    else hi = mid;
  }
  const PlanStream st = plan.streams[lo];
  const int j = t - st.start;
  if (j < 0 || j >= st.n) return;
  const int own = st.len - st.n;
  const unsigned long long mask = st.tree ? plan.masks[t] : 0;
  const int last = st.tree ? st.len : own + j + 1;
  for (int head = threadIdx.x >> 5; head < a.qh; head += kWarps) {
    float q[16], o[16] = {}, m = -1e30f, den = 0.f;
    const uint32_t* qw = reinterpret_cast<const uint32_t*>(a.Q + ((size_t)t * a.qh + head) * D + 16 * l);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      q[2 * e] = bf_lo(qw[e]);
      q[2 * e + 1] = bf_hi(qw[e]);
    }
    float mx = 0.f, down, up;
#pragma unroll
    for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(q[e]));
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    row_scale(mx, down, up);
#pragma unroll
    for (int e = 0; e < 16; ++e) q[e] *= down;
    const size_t at = a.c.row(st.slot, head / G, 0);
    for (int p0 = 0; p0 < last; p0 += kAt) {
      const int p = p0 + g;
      const bool see = p < last && (!st.tree || p < own || mask >> (p - own) & 1);
      float x = 0.f, v[16] = {};
      if (see) {
        const uint4 kw = *reinterpret_cast<const uint4*>(a.c.K + (at + p) * D + 16 * l), vw = *reinterpret_cast<const uint4*>(a.c.V + (at + p) * D + 16 * l);
        const uint32_t k4[4] = {kw.x, kw.y, kw.z, kw.w}, v4[4] = {vw.x, vw.y, vw.z, vw.w};
        const float vs = a.c.Vs[at + p];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float k[4];
          decode4<FMT>(k4[w], k);
          decode4<FMT>(v4[w], v + 4 * w);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x = fmaf(q[4 * w + e], k[e], x);
            v[4 * w + e] *= vs;
          }
        }
      }
      x = group_sum<kLanes>(x);
      x = see ? x * a.c.Ks[at + p] * (a.scale_log2 * up) : -1e30f;
      const float mn = fmaxf(m, x), f = exp2f(m - mn), w = see ? exp2f(x - mn) : 0.f;
      den = den * f + w;
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = fmaf(o[e], f, see ? w * v[e] : 0.f);
      m = mn;
    }
    // the groups' parts
#pragma unroll
    for (int s = kLanes; s < 32; s <<= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, s), od = __shfl_xor_sync(0xffffffffu, den, s);
      const float mn = fmaxf(m, om), f = exp2f(m - mn), of = exp2f(om - mn);
      den = den * f + od * of;
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = o[e] * f + __shfl_xor_sync(0xffffffffu, o[e], s) * of;
      m = mn;
    }
    if (g == 0) {
      const float inv = den == 0.f ? 0.f : 1.f / den;
      bf16* to = a.O + ((size_t)t * a.qh + head) * D + 16 * l;
#pragma unroll
      for (int e = 0; e < 16; ++e) to[e] = f2bf(o[e] * inv);
    }
  }
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
  a.plan = plan;
  a.Q = reinterpret_cast<const bf16*>(Q);
  a.O = reinterpret_cast<bf16*>(O);
  a.B = B;
  a.T = T;
  a.qh = q_heads;
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4 = c->format == BM_KV8_E4M3, d128 = c->head_dim == 128;
  if (d128 && e4) k_kv8_rows<128, BM_KV8_E4M3><<<T, kWarps * 32, 0, s>>>(a);
  else if (d128) k_kv8_rows<128, BM_KV8_INT8><<<T, kWarps * 32, 0, s>>>(a);
  else if (e4) k_kv8_rows<64, BM_KV8_E4M3><<<T, kWarps * 32, 0, s>>>(a);
  else k_kv8_rows<64, BM_KV8_INT8><<<T, kWarps * 32, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, std::string("kv8_attend_rows: ") + cudaGetErrorString(e));
  return ok();
}

}  // extern "C"
