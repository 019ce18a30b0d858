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

#include "kv8.cuh"

namespace bm {
namespace {

using namespace kv8;

constexpr int kMaxGroup = 8;

struct AttendArgs {
  Cache c, p;            // the streams' cache, the prefix's
  int p_slot, p_len, p_chunk, p_chunks;
  const bf16* Q;
  const int32_t* slots;
  const int32_t* lens;
  bf16* O;
  float* rec;            // [B][q_heads][p_chunks + own chunks] records of d + 2 floats: o, m, l
  int B, qh, own_chunks;
  float scale_log2;      // scale * log2(e): the scores are powers of two
  __device__ float* record(int b, int h, int r, int d) const {
    return rec + (((size_t)b * qh + h) * (p_chunks + own_chunks) + r) * (size_t)(d + 2);
  }
  // A stream that takes part: padding and out-of-range rows are skipped.
  __device__ bool live(int b, int& slot, int& len) const {
    slot = slots[b];
    len = lens[b];
    return slot >= 0 && slot < c.slots && len >= 0 && len <= c.cap;
  }
};

// One chunk of one (stream, kv head): a warp takes every eighth position,
// a lane d / 32 of its elements.
template <int D, int FMT>
__global__ void __launch_bounds__(256) k_kv8_chunk(AttendArgs a) {
  constexpr int E = D / 32;
  __shared__ float so[8][kMaxGroup][D], sm[8][kMaxGroup], sl[8][kMaxGroup];
  const int b = blockIdx.z, kh = blockIdx.y, r = blockIdx.x;
  int slot, len;
  if (!a.live(b, slot, len)) return;
  const bool pre = r < a.p_chunks;
  const int size = pre ? a.p_chunk : chunk_of(len), j0 = (pre ? r : r - a.p_chunks) * size;
  const int n = min(size, (pre ? a.p_len : len) - j0);
  if (n <= 0) return;
  const Cache& c = pre ? a.p : a.c;
  const size_t row0 = c.row(pre ? a.p_slot : slot, kh, j0);
  const int G = a.qh / a.c.kvh, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float q[kMaxGroup][E], o[kMaxGroup][E], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
  for (int g = 0; g < kMaxGroup; ++g) {
    m[g] = -FLT_MAX;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[g][e] = 0.f;
      q[g][e] = g < G ? bf2f(a.Q[((size_t)b * a.qh + kh * G + g) * D + lane * E + e]) : 0.f;
    }
  }
  for (int j = warp; j < n; j += 8) {
    float k[4], v[4];
    uint32_t kw, vw;
    if (E == 4) {
      kw = reinterpret_cast<const uint32_t*>(c.K + (row0 + j) * D)[lane];
      vw = reinterpret_cast<const uint32_t*>(c.V + (row0 + j) * D)[lane];
    } else {
      kw = reinterpret_cast<const uint16_t*>(c.K + (row0 + j) * D)[lane];
      vw = reinterpret_cast<const uint16_t*>(c.V + (row0 + j) * D)[lane];
    }
    decode4<FMT>(kw, k);
    decode4<FMT>(vw, v);
    const float ks = c.Ks[row0 + j], vs = c.Vs[row0 + j];
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[g][e], k[e], s);
      s = warp_sum(s) * ks * a.scale_log2;
      const float mn = fmaxf(m[g], s), f = exp2f(m[g] - mn), p = exp2f(s - mn);
      m[g] = mn;
      l[g] = l[g] * f + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] = o[g][e] * f + p * vs * v[e];
    }
  }
#pragma unroll
  for (int g = 0; g < kMaxGroup; ++g) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][g][lane * E + e] = o[g][e];
    if (lane == 0) {
      sm[warp][g] = m[g];
      sl[warp][g] = l[g];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * D; i += 256) {
    const int g = i / D, d = i - g * D;
    float mx = -FLT_MAX, den = 0.f, acc = 0.f;
    for (int w = 0; w < 8; ++w) mx = fmaxf(mx, sm[w][g]);
    for (int w = 0; w < 8; ++w) {
      const float f = exp2f(sm[w][g] - mx);
      den += sl[w][g] * f;
      acc += so[w][g][d] * f;
    }
    float* rec = a.record(b, kh * G + g, r, D);
    rec[d] = acc;
    if (d == 0) {
      rec[D] = mx;
      rec[D + 1] = den;
    }
  }
}

// One head of one stream: its records in ascending order.
template <int D>
__global__ void __launch_bounds__(D) k_kv8_merge(AttendArgs a) {
  const int h = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
  int slot, len;
  if (!a.live(b, slot, len)) return;
  const int n = a.p_chunks + chunks_of(len);
  float mx = -FLT_MAX, den = 0.f, acc = 0.f;
  for (int r = 0; r < n; ++r) mx = fmaxf(mx, a.record(b, h, r, D)[D]);
  for (int r = 0; r < n; ++r) {
    const float* rec = a.record(b, h, r, D);
    const float f = exp2f(rec[D] - mx);
    den += rec[D + 1] * f;
    acc += rec[d] * f;
  }
  a.O[((size_t)b * a.qh + h) * D + d] = f2bf(n == 0 ? 0.f : acc / den);   // no positions: zeros
}

template <int D, int FMT>
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
  const int per_stream = a.p_chunks + a.own_chunks;
  if (per_stream > 0) k_kv8_chunk<D, FMT><<<dim3(per_stream, a.c.kvh, a.B), 256, 0, s>>>(a);
  k_kv8_merge<D><<<dim3(a.qh, a.B), D, 0, s>>>(a);
  return cudaGetLastError();
}

// Positions per chunk of the shared prefix; a function of its length only.
int prefix_chunk(int len) { return chunk_of(len); }

bool shapes_ok(int B, int qh, int kvh, int d) {
  return B >= 1 && B <= 1024 && kvh >= 1 && qh >= 1 && qh % kvh == 0 && qh / kvh <= kMaxGroup && qh <= 1024 &&
         (d == 64 || d == 128);
}

size_t records(int ctx_cap, int prefix_len) {
  const int pc = prefix_len > 0 ? (prefix_len + prefix_chunk(prefix_len) - 1) / prefix_chunk(prefix_len) : 0;
  return (size_t)pc + std::min(64, (ctx_cap + 255) / 256);
}

bm_status attend(const char* who, const bm_kv8_cache* c, const bm_kv8_cache* p, int p_slot, int p_len, const uint16_t* Q,
                 const int32_t* slots, const int32_t* lens, int q_heads, float scale, uint16_t* O, int B, void* ws,
                 size_t ws_bytes, void* stream) {
  const std::string w(who);
  AttendArgs a{};
  bm_status st = check_cache(c, who, &a.c);
  if (st != BM_OK) return st;
  if (p) {
    if ((st = check_cache(p, who, &a.p)) != BM_OK) return st;
    if (p->format != c->format || p->kv_heads != c->kv_heads || p->head_dim != c->head_dim)
      return set_error(BM_ERR_INVALID_ARG, w + ": the prefix's cache must have the streams' format, kv_heads and head_dim");
    if (p_slot < 0 || p_slot >= p->slots) return set_error(BM_ERR_INVALID_ARG, w + ": prefix_slot out of range");
    if (p_len < 0 || p_len > p->ctx_cap) return set_error(BM_ERR_CTX_CAP, w + ": prefix_len outside the slot");
  }
  if (!Q || !slots || !lens || !O || !ws) return set_error(BM_ERR_INVALID_ARG, w + ": null pointer");
  if (((uintptr_t)Q | (uintptr_t)O | (uintptr_t)ws) & 15)
    return set_error(BM_ERR_INVALID_ARG, w + ": Q, O and the workspace must be 16-byte aligned");
  if (!shapes_ok(B, q_heads, c->kv_heads, c->head_dim))
    return set_error(BM_ERR_INVALID_ARG, w + ": need 1 <= B <= 1024, q_heads <= 1024 and a multiple of kv_heads, at most 8 query heads per kv head");
  if (!(scale > 0.f) || !(scale < INFINITY)) return set_error(BM_ERR_INVALID_ARG, w + ": scale must be positive and finite");
  const size_t need = kv8_workspace_bytes(B, q_heads, c->kv_heads, c->head_dim, c->ctx_cap, p_len);
  if (ws_bytes < need)
    return set_error(BM_ERR_INVALID_ARG, w + ": workspace of " + std::to_string(ws_bytes) + " bytes, " + std::to_string(need) + " needed");
  a.p_slot = p_slot;
  a.p_len = p_len;
  a.p_chunk = prefix_chunk(p_len);
  a.p_chunks = p_len > 0 ? (p_len + a.p_chunk - 1) / a.p_chunk : 0;
  a.Q = reinterpret_cast<const bf16*>(Q);
  a.slots = slots;
  a.lens = lens;
  a.O = reinterpret_cast<bf16*>(O);
  a.rec = static_cast<float*>(ws);
  a.B = B;
  a.qh = q_heads;
  a.own_chunks = std::min(64, (c->ctx_cap + 255) / 256);
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4 = c->format == BM_KV8_E4M3, d128 = c->head_dim == 128;
  const cudaError_t e = d128 ? (e4 ? launch_attend<128, BM_KV8_E4M3>(a, s) : launch_attend<128, BM_KV8_INT8>(a, s))
                             : (e4 ? launch_attend<64, BM_KV8_E4M3>(a, s) : launch_attend<64, BM_KV8_INT8>(a, s));
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, w + ": " + cudaGetErrorString(e));
  return ok();
}

}  // namespace
}  // namespace bm

extern "C" {

size_t kv8_workspace_bytes(int B, int q_heads, int kv_heads, int head_dim, int ctx_cap, int prefix_len) {
  using namespace bm;
  if (!shapes_ok(B, q_heads, kv_heads, head_dim) || ctx_cap < 1 || prefix_len < 0) return 0;
  return (size_t)B * q_heads * records(ctx_cap, prefix_len) * (head_dim + 2) * sizeof(float);
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
