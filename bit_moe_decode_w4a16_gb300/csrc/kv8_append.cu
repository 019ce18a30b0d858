// Writing the 8-bit K/V cache and reading it back.
//
// kv8_append takes rows of the QKV projection.  Per head of a row, in fp32:
//   n = x / sqrt(mean(x^2) + eps) * w          (q and k heads, if norm)
//   y_i       = n_i cos(a_i) - n_{i+d/2} sin(a_i)
//   y_{i+d/2} = n_{i+d/2} cos(a_i) + n_i sin(a_i),   a_i = pos * inv_freq_i
//   q: bf16(y);  k, v: amax = max |y|, scale = amax / M, code = rn(y * (M / amax))
// with M = 448 (e4m3) or 127 (int8).  One rounding each: q and the codes are
// rounded from fp32, with no bf16 step between the norm and the rotation.
//
// It is bound by the bytes of the rows (each read once and written once).  A
// head belongs to d / 8 lanes of 16 bytes each: a head's sums and maxima are
// 3 or 4 shuffles, the other half of a rotated pair is one shuffle away
// (lane ^ d / 16), and no head touches shared memory.  A CTA holds a row's
// heads; its first d / 2 threads turn the position into the row's cosines
// and sines.
#include "kv8.cuh"

namespace bm {
namespace {

using namespace kv8;

struct AppendArgs {
  Cache c;
  const bf16* qkv;
  long long ld;
  int qh;
  int norm;
  float eps;
  const bf16* q_norm;
  const bf16* k_norm;
  const float* inv_freq;
  const int32_t* slots;
  const int32_t* index;
  const int32_t* pos;
  bf16* Q;
  int heads_per_cta;
};

// Cosine and sine of pos * f.  The angle is reduced in 64 bits, in turns:
// at position 2^17 an fp32 product would be off by 2^-7 of a radian.
__device__ __forceinline__ float2 rotation(int pos, float f) {
  const double turns = (double)pos * (double)f * 0.15915494309189533577;   // / (2 pi)
  const float frac = (float)(turns - rint(turns));
  float s, c;
  sincospif(2.0f * frac, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ void unpack8(uint4 r, float (&x)[8]) {
  x[0] = bf_lo(r.x); x[1] = bf_hi(r.x); x[2] = bf_lo(r.y); x[3] = bf_hi(r.y);
  x[4] = bf_lo(r.z); x[5] = bf_hi(r.z); x[6] = bf_lo(r.w); x[7] = bf_hi(r.w);
}

template <int D, int FMT>
__global__ void __launch_bounds__(1024) k_kv8_append(AppendArgs a) {
  constexpr int kLanes = D / 8;   // lanes of a head
  __shared__ float2 cs[D / 2];
  const int t = blockIdx.x;
  const int slot = a.slots[t], idx = a.index[t];
  if (slot < 0 || slot >= a.c.slots || idx < 0 || idx >= a.c.cap) return;   // padding: nothing of the row is written
  const int l = threadIdx.x % kLanes, h = blockIdx.y * a.heads_per_cta + threadIdx.x / kLanes;
  const int kvh = a.c.kvh, heads = a.qh + 2 * kvh;
  const bool live = h < heads && (int)(threadIdx.x / kLanes) < a.heads_per_cta;
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (live) raw = *reinterpret_cast<const uint4*>(a.qkv + t * a.ld + (size_t)h * D + 8 * l);
  const bool rotated = a.inv_freq != nullptr;
  if (rotated) {
    if (threadIdx.x < D / 2) cs[threadIdx.x] = rotation(a.pos ? a.pos[t] : idx, a.inv_freq[threadIdx.x]);
    __syncthreads();
  }
  float x[8];
  unpack8(raw, x);
  const bool is_v = h >= a.qh + kvh, is_q = h < a.qh;
  if (a.norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    ss = group_sum<kLanes>(ss);
    const float inv = 1.0f / sqrtf(ss / (float)D + a.eps);
    const bf16* nw = is_q ? a.q_norm : a.k_norm;
    if (!is_v) {
      float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (nw) unpack8(*reinterpret_cast<const uint4*>(nw + 8 * l), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
    }
  }
  if (rotated) {
    const bool second = l >= kLanes / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, x[i], kLanes / 2);
      const float2 r = cs[(8 * l + i) % (D / 2)];
      if (!is_v) x[i] = fmaf(x[i], r.x, second ? other * r.y : -(other * r.y));
    }
  }
  // the largest magnitude, on the bit patterns: NaN > infinity > any number
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = max(mx, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (!live) return;
  if (is_q) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      p[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(a.Q + ((size_t)t * a.qh + h) * D + 8 * l) = make_uint4(p[0], p[1], p[2], p[3]);
    return;
  }
  const float amax = __uint_as_float(mx);
  float inv = 0.f, scale = 0.f;
  if (mx >= 0x7F800000u) {
    scale = __uint_as_float(0x7FC00000u);   // a head with infinity or NaN reads back as NaN
  } else if (amax >= kTinyHead) {
    inv = code_max<FMT>() / amax;
    scale = amax / code_max<FMT>();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = inv == 0.f ? 0.f : x[i] * inv;
  const size_t row = a.c.row(slot, is_v ? h - a.qh - kvh : h - a.qh, idx);
  uint8_t* codes = is_v ? a.c.V : a.c.K;
  *reinterpret_cast<uint2*>(codes + row * D + 8 * l) = make_uint2(encode4<FMT>(x), encode4<FMT>(x + 4));
  if (l == 0) (is_v ? a.c.Vs : a.c.Ks)[row] = scale;
}

// bf16(code * scale), 16 codes to a thread; K in blockIdx.z = 0, V in 1.
template <int D, int FMT>
__global__ void __launch_bounds__(256) k_kv8_read(Cache c, int slot, int first, int count, bf16* K, bf16* V) {
  constexpr int kLanes = D / 16;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int p = (int)(i / kLanes), l = (int)(i % kLanes), h = blockIdx.y;
  if (p >= count) return;
  const size_t row = c.row(slot, h, first + p);
  const bool v = blockIdx.z != 0;
  const uint4 w = *reinterpret_cast<const uint4*>((v ? c.V : c.K) + row * D + 16 * l);
  const float s = (v ? c.Vs : c.Ks)[row];
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t out[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[4];
    decode4<FMT>(in[j], f);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * q] * s, f[2 * q + 1] * s);
      out[2 * j + q] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  uint4* o = reinterpret_cast<uint4*>((v ? V : K) + ((size_t)h * count + p) * D + 16 * l);
  o[0] = make_uint4(out[0], out[1], out[2], out[3]);
  o[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

template <int D, int FMT>
cudaError_t launch_append(const AppendArgs& args, int T, cudaStream_t s) {
  AppendArgs a = args;
  const int heads = a.qh + 2 * a.c.kvh, per = 1024 / (D / 8);
  const int ny = (heads + per - 1) / per;
  a.heads_per_cta = (heads + ny - 1) / ny;
  const int threads = ((max(a.heads_per_cta * (D / 8), D / 2) + 31) / 32) * 32;
  k_kv8_append<D, FMT><<<dim3(T, ny), threads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

namespace kv8 {

// The cache descriptor's own checks; `who` opens the message.
bm_status check_cache(const bm_kv8_cache* c, const char* who, Cache* out) {
  const std::string w(who);
  if (!c) return set_error(BM_ERR_INVALID_ARG, w + ": null cache");
  if (c->format != BM_KV8_E4M3 && c->format != BM_KV8_INT8)
    return set_error(BM_ERR_INVALID_ARG, w + ": unknown cache format " + std::to_string(c->format));
  if (c->head_dim != 64 && c->head_dim != 128) return set_error(BM_ERR_INVALID_ARG, w + ": head_dim must be 64 or 128");
  if (c->slots < 1 || c->ctx_cap < 1 || c->kv_heads < 1 || c->kv_heads > 1024)
    return set_error(BM_ERR_INVALID_ARG, w + ": slots and ctx_cap must be >= 1, kv_heads in [1, 1024]");
  if (!c->K || !c->V || !c->Ks || !c->Vs) return set_error(BM_ERR_INVALID_ARG, w + ": null cache pointer");
  if (((uintptr_t)c->K | (uintptr_t)c->V) & 15 || ((uintptr_t)c->Ks | (uintptr_t)c->Vs) & 3)
    return set_error(BM_ERR_INVALID_ARG, w + ": codes must be 16-byte aligned and scales 4-byte aligned");
  *out = Cache{c->slots, c->ctx_cap, c->kv_heads, c->K, c->V, c->Ks, c->Vs};
  return BM_OK;
}

}  // namespace kv8
}  // namespace bm

extern "C" {

bm_status kv8_append(const bm_kv8_cache* c, const uint16_t* qkv, int64_t ld, int q_heads, const bm_kv8_rope* rope,
                     const int32_t* slots, const int32_t* index, const int32_t* rope_pos, uint16_t* Q, int T,
                     void* stream) {
  using namespace bm;
  AppendArgs a{};
  bm_status st = kv8::check_cache(c, "kv8_append", &a.c);
  if (st != BM_OK) return st;
  if (!qkv || !rope || !slots || !index || !Q) return set_error(BM_ERR_INVALID_ARG, "kv8_append: null pointer");
  if (T < 1) return set_error(BM_ERR_INVALID_ARG, "kv8_append: T must be >= 1");
  if (q_heads < 1 || q_heads > 1024) return set_error(BM_ERR_INVALID_ARG, "kv8_append: q_heads must be in [1, 1024]");
  const int64_t row = ((int64_t)q_heads + 2 * c->kv_heads) * c->head_dim;
  if (ld < row || ld % 8)
    return set_error(BM_ERR_INVALID_ARG, "kv8_append: ld must be a multiple of 8 and at least (q_heads + 2 kv_heads) * head_dim");
  if (((uintptr_t)qkv | (uintptr_t)Q | (uintptr_t)rope->q_norm | (uintptr_t)rope->k_norm) & 15)
    return set_error(BM_ERR_INVALID_ARG, "kv8_append: qkv, Q and the norm weights must be 16-byte aligned");
  if (rope->norm && !(rope->eps >= 0.f)) return set_error(BM_ERR_INVALID_ARG, "kv8_append: eps must be >= 0");
  a.qkv = reinterpret_cast<const bf16*>(qkv);
  a.ld = ld;
  a.qh = q_heads;
  a.norm = rope->norm != 0;
  a.eps = rope->eps;
  a.q_norm = reinterpret_cast<const bf16*>(rope->q_norm);
  a.k_norm = reinterpret_cast<const bf16*>(rope->k_norm);
  a.inv_freq = rope->inv_freq;
  a.slots = slots;
  a.index = index;
  a.pos = rope_pos;
  a.Q = reinterpret_cast<bf16*>(Q);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4 = c->format == BM_KV8_E4M3, d128 = c->head_dim == 128;
  const cudaError_t e = d128 ? (e4 ? launch_append<128, BM_KV8_E4M3>(a, T, s) : launch_append<128, BM_KV8_INT8>(a, T, s))
                             : (e4 ? launch_append<64, BM_KV8_E4M3>(a, T, s) : launch_append<64, BM_KV8_INT8>(a, T, s));
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, std::string("kv8_append: ") + cudaGetErrorString(e));
  return ok();
}

bm_status kv8_read(const bm_kv8_cache* c, int slot, int first, int count, uint16_t* K_out, uint16_t* V_out, void* stream) {
  using namespace bm;
  kv8::Cache cc{};
  bm_status st = kv8::check_cache(c, "kv8_read", &cc);
  if (st != BM_OK) return st;
  if (slot < 0 || slot >= c->slots) return set_error(BM_ERR_INVALID_ARG, "kv8_read: slot out of range");
  if (first < 0 || count < 0 || (int64_t)first + count > c->ctx_cap)
    return set_error(BM_ERR_CTX_CAP, "kv8_read: positions outside the slot");
  if (count == 0) return ok();
  if (!K_out || !V_out) return set_error(BM_ERR_INVALID_ARG, "kv8_read: null pointer");
  if (((uintptr_t)K_out | (uintptr_t)V_out) & 15) return set_error(BM_ERR_INVALID_ARG, "kv8_read: outputs must be 16-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int lanes = c->head_dim / 16;
  const dim3 grid((unsigned)(((int64_t)count * lanes + 255) / 256), c->kv_heads, 2);
  bf16 *K = reinterpret_cast<bf16*>(K_out), *V = reinterpret_cast<bf16*>(V_out);
  const bool e4 = c->format == BM_KV8_E4M3, d128 = c->head_dim == 128;
  if (d128 && e4) k_kv8_read<128, BM_KV8_E4M3><<<grid, 256, 0, s>>>(cc, slot, first, count, K, V);
  else if (d128) k_kv8_read<128, BM_KV8_INT8><<<grid, 256, 0, s>>>(cc, slot, first, count, K, V);
  else if (e4) k_kv8_read<64, BM_KV8_E4M3><<<grid, 256, 0, s>>>(cc, slot, first, count, K, V);
  else k_kv8_read<64, BM_KV8_INT8><<<grid, 256, 0, s>>>(cc, slot, first, count, K, V);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, std::string("kv8_read: ") + cudaGetErrorString(e));
  return ok();
}

}  // extern "C"
