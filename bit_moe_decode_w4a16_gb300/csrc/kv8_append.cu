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
// Each row is read once and written once.  A head belongs to d / 16 lanes, 8
// elements and their 8 partners of the rotation each: a head's sums and maxima
// are 2 or 3 shuffles, a rotation none.  A thread keeps its place in the row
// and walks over rows, so norm weights and frequencies are read once; two rows
// are on their way while one is worked on, and a CTA's first d / 2 threads make
// the next row's cosines and sines meanwhile.
//
// 4000 rows of 32 + 2 x 4 heads of 128, e4m3: 15.6 us, 5.0 TB/s.  What is paid
// per thread and row (its addresses, loads, shuffles, branches) came before
// the bytes (11.6 us): 8 elements to a thread took 22 us, with fp32 pairs in
// one instruction or without, 4 took 33; a third more threads on an SM, at
// fewer registers, 20.  A call of 1 to 32 rows is one latency chain of 2.1 to
// 2.5 us, longer by 0.4 with CTAs of 320 threads, whose rows start together.
#include <algorithm>

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
  int heads_per_cta, T;
};

// f / (2 pi) in 2^-64 turns, good to 2^-55 for f up to 1 (an fp64 product).  A
// product with a position wraps around at whole turns, so the angle is good to
// 2^-38 of a turn at position 2^17, far below the fp32 rounding of the fraction
// that follows; an fp32 product would be off by 2^-7 of a radian there.
__device__ __forceinline__ unsigned long long turns64(float f) {
  const double t = (double)f * 0.15915494309189533577;
  return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}
__device__ __forceinline__ float2 rotation(int pos, unsigned long long turns) {
  const int frac = (int)(((unsigned long long)(long long)pos * turns) >> 32);   // of a turn, in [-1/2, 1/2)
  float s, c;
  sincospif((float)frac * 4.656612873077393e-10f, &s, &c);   // * 2^-31: half turns
  return make_float2(c, s);
}

// Eight bf16 -> four pairs of fp32, two values to an instruction from there on.
__device__ __forceinline__ void unpack8(uint4 r, uint64_t* x) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pack2(bf_lo(w[i]), bf_hi(w[i]));
}
__device__ __forceinline__ uint4 round8(const uint64_t* x) {
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(first(x[i]), second(x[i]));
    p[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(p[0], p[1], p[2], p[3]);
}
template <int FMT>
__device__ __forceinline__ uint2 encode8(const uint64_t* x, float inv) {
  float f[8];
  const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t v = mul2(x[i], inv2);
    f[2 * i] = first(v);
    f[2 * i + 1] = second(v);
  }
  return make_uint2(encode4<FMT>(f), encode4<FMT>(f + 4));
}

// The largest of three magnitudes; NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

constexpr int kMaxThreads = 160, kCtasPerSm = 4;

struct AppendRow {
  uint4 lo, hi;
  int slot, idx, pos;
};

template <int D, int FMT>
__global__ void __launch_bounds__(kMaxThreads, kCtasPerSm) k_kv8_append(AppendArgs a) {
  constexpr int kLanes = D / 16;   // lanes of a head
  __shared__ __align__(16) float cs[2][2][D / 2];   // cosines and sines of a row's angles
  const int l = threadIdx.x % kLanes, h = blockIdx.y * a.heads_per_cta + threadIdx.x / kLanes;
  const int kvh = a.c.kvh, heads = a.qh + 2 * kvh;
  const bool live = h < heads && (int)(threadIdx.x / kLanes) < a.heads_per_cta;
  const bool is_v = h >= a.qh + kvh, is_q = h < a.qh, all_v = __all_sync(0xffffffffu, is_v), any_kv = __any_sync(0xffffffffu, live && !is_q);
  const bool rotated = a.inv_freq != nullptr, turns_here = rotated && threadIdx.x < D / 2;
  // Rows outside the cache are padding: nothing of theirs is written.
  auto valid = [&](const AppendRow& r) { return (unsigned)r.slot < (unsigned)a.c.slots && (unsigned)r.idx < (unsigned)a.c.cap; };
  // elements 8l .. 8l + 7 and their partners of the rotation, d / 2 further on
  const bf16* mine = a.qkv + (size_t)h * D + 8 * l;
  const int32_t* positions = a.pos ? a.pos : a.index;
  auto load = [&](int t) {
    AppendRow r{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), -1, -1, 0};
    if (t < a.T) {
      r.slot = __ldg(a.slots + t);
      r.idx = __ldg(a.index + t);
      if (turns_here) r.pos = __ldg(positions + t);
      if (live) {
        const uint4* at = reinterpret_cast<const uint4*>(mine + t * a.ld);
        r.lo = __ldg(at);
        r.hi = __ldg(at + D / 16);
      }
    }
    return r;
  };
  const int step = gridDim.x;
  AppendRow now = load(blockIdx.x), next = load(blockIdx.x + step);
  const unsigned long long turns = turns_here ? turns64(a.inv_freq[threadIdx.x]) : 0;
  auto rotate = [&](int b, int pos) {
    const float2 r = rotation(pos, turns);
    cs[b][0][threadIdx.x] = r.x;
    cs[b][1][threadIdx.x] = r.y;
  };
  const bf16* nw = is_q ? a.q_norm : a.k_norm;
  uint4 w_lo = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), w_hi = w_lo;   // ones
  if (a.norm && !is_v && nw) {
    const uint4* at = reinterpret_cast<const uint4*>(nw + 8 * l);
    w_lo = __ldg(at);
    w_hi = __ldg(at + D / 16);
  }
  if (turns_here) rotate(0, now.pos);
  if (rotated) __syncthreads();
  int b = 0;
  for (int t = blockIdx.x; t < a.T; t += step) {
    const AppendRow after = load(t + 2 * step);
    if (turns_here) rotate(b ^ 1, next.pos);
    if (valid(now)) {
      uint64_t x[8];
      unpack8(now.lo, x);
      unpack8(now.hi, x + 4);
      if (a.norm && !all_v) {
        uint64_t s2 = mul2(x[0], x[0]), w[8];
#pragma unroll
        for (int i = 1; i < 8; ++i) s2 = fma2(x[i], x[i], s2);
        const float ss = group_sum<kLanes>(first(s2) + second(s2));
        const float inv = is_v ? 1.f : rsqrtf(fmaf(ss, 1.0f / D, a.eps));
        const uint64_t inv2 = pack2(inv, inv);
        unpack8(w_lo, w);
        unpack8(w_hi, w + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], mul2(inv2, w[i]));
      }
      if (rotated && !is_v) {
        const uint64_t minus = pack2(-1.f, -1.f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&cs[b][0][8 * l + 4 * j]), s = *reinterpret_cast<const ulonglong2*>(&cs[b][1][8 * l + 4 * j]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint64_t p = x[2 * j + i], q = x[2 * j + i + 4], ci = i ? c.y : c.x, si = i ? s.y : s.x;
            x[2 * j + i] = fma2(p, ci, mul2(mul2(q, si), minus));
            x[2 * j + i + 4] = fma2(q, ci, mul2(p, si));
          }
        }
      }
      if (is_q && live) {
        uint4* q = reinterpret_cast<uint4*>(a.Q + ((size_t)t * a.qh + h) * D + 8 * l);
        q[0] = round8(x);
        q[D / 16] = round8(x + 4);
      }
      if (any_kv) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max_abs(amax, first(x[i]), second(x[i]));
        uint32_t mx = __float_as_uint(amax) & 0x7FFFFFFFu;   // as bit patterns, NaN > infinity > any number
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (live && !is_q) {
          amax = __uint_as_float(mx);
          float inv = 0.f, scale = 0.f;
          const bool finite = mx < 0x7F800000u;
          if (finite && amax >= kTinyHead) {
            inv = code_max<FMT>() / amax;
            scale = amax / code_max<FMT>();
          }
          uint2 lo = encode8<FMT>(x, inv), hi = encode8<FMT>(x + 4, inv);
          if (!finite) {   // a head with infinity or NaN reads back as NaN
            lo = hi = make_uint2(0, 0);
            scale = __uint_as_float(0x7FC00000u);
          }
          const size_t row = a.c.row(now.slot, is_v ? h - a.qh - kvh : h - a.qh, now.idx);
          uint2* codes = reinterpret_cast<uint2*>((is_v ? a.c.V : a.c.K) + row * D + 8 * l);
          codes[0] = lo;
          codes[D / 16] = hi;
          if (l == 0) (is_v ? a.c.Vs : a.c.Ks)[row] = scale;
        }
      }
    }
    now = next;
    next = after;
    b ^= 1;
    if (rotated) __syncthreads();
  }
}

// bf16(code * scale), 16 codes to a thread; K in blockIdx.z = 0, V in 1: one
// 16-byte load and two 16-byte stores a thread, bound by HBM.  65536 positions
// of 4 heads of 128: 32.1 us, 6.3 TB/s (94% of a plain copy).
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
  const int heads = a.qh + 2 * a.c.kvh, per = kMaxThreads / (D / 16);
  const int ny = (heads + per - 1) / per;
  a.heads_per_cta = (heads + ny - 1) / ny;
  const int threads = ((max(a.heads_per_cta * (D / 16), D / 2) + 31) / 32) * 32;
  a.T = T;
  // as many CTAs as an SM's registers hold, on every SM
  const int ctas = std::max(1, kSms * (kCtasPerSm * kMaxThreads / threads) / ny);
  k_kv8_append<D, FMT><<<dim3(std::min(T, ctas), ny), threads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

namespace kv8 {

// The cache descriptor's own checks; `who` opens the message.
bm_status check_cache(const bm_kv8_cache* c, const char* who, Cache* out) {
  auto refuse = [&](const std::string& what) { return set_error(BM_ERR_INVALID_ARG, std::string(who) + ": " + what); };
  if (!c) return refuse("null cache");
  if (c->format != BM_KV8_E4M3 && c->format != BM_KV8_INT8)
    return refuse("unknown cache format " + std::to_string(c->format));
  if (c->head_dim != 64 && c->head_dim != 128) return refuse("head_dim must be 64 or 128");
  if (c->slots < 1 || c->ctx_cap < 1 || c->kv_heads < 1 || c->kv_heads > 1024)
    return refuse("slots and ctx_cap must be >= 1, kv_heads in [1, 1024]");
  if (!c->K || !c->V || !c->Ks || !c->Vs) return refuse("null cache pointer");
  if (((uintptr_t)c->K | (uintptr_t)c->V) & 15 || ((uintptr_t)c->Ks | (uintptr_t)c->Vs) & 3)
    return refuse("codes must be 16-byte aligned and scales 4-byte aligned");
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
  if (((uintptr_t)slots | (uintptr_t)index | (uintptr_t)rope_pos | (uintptr_t)rope->inv_freq) & 3)
    return set_error(BM_ERR_INVALID_ARG, "kv8_append: slots, index, rope_pos and inv_freq must be 4-byte aligned");
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
