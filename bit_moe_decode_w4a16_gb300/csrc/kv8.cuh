// The 8-bit K/V cache: layout, code conversions and the split of a stream's
// positions, shared by the kernels that write, read and attend over it.
//
// One layer's cache: codes [slot][kv head][position][d] (one byte each) and
// fp32 scales [slot][kv head][position], for K and for V; the stored value is
// code * scale.  One scale per (position, head): a position is written once,
// by the row that appends it, and never has to be rescaled for a later one.
#pragma once

#include "common.cuh"
#include "errors.h"

namespace bm {
namespace kv8 {

constexpr int kSms = 152;

struct Cache {
  int slots, cap, kvh;
  uint8_t* K;
  uint8_t* V;
  float* Ks;
  float* Vs;
  // index of the scale of (slot, head, position); times d: of its codes
  __host__ __device__ size_t row(int slot, int h, int p) const { return ((size_t)slot * kvh + h) * cap + p; }
};

constexpr float kTinyHead = 7.7037197775489434e-34f;   // 2^-110: 448 / amax stays finite above it

template <int FMT>
__host__ __device__ constexpr float code_max() {
  return FMT == BM_KV8_E4M3 ? 448.0f : 127.0f;
}

// Four codes of a word -> fp32 (exact).
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float* f) {
  if (FMT == BM_KV8_E4M3) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t p;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(p) : "h"((unsigned short)(w >> (16 * h))));
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&p));
      f[2 * h] = v.x;
      f[2 * h + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
  }
}

// Four fp32 values, already divided by the scale, -> four codes, rounded to
// nearest even and clamped to the format's largest finite code.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(const float* f) {
  if (FMT == BM_KV8_E4M3) {
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = max(-127, min(127, __float2int_rn(f[i])));
    w |= ((uint32_t)q & 0xFFu) << (8 * i);
  }
  return w;
}

// Pairs of fp32: one instruction works on both.
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

// Positions per chunk of a stream of `len` positions: 256, doubled each time
// the length passes four times the last border (4096, 16384, 65536), and
// beyond that kept so large that there are at most 64 chunks.  A chunk has
// a fixed cost, a record to merge among it, and a lone stream needs chunks to
// spread over the GPU: half as many of each as the length grows fourfold.  It
// depends on the stream's own length only, so a stream's result does not
// depend on the batch it is attended in.
__host__ __device__ inline int chunk_of(int len) {
  int c = 256;
  for (long long border = 4096; len > border; border *= border < 65536 ? 4 : 2) c *= 2;
  return c;
}
__host__ __device__ inline int chunks_of(int len) {
  const int c = chunk_of(len);
  return len > 0 ? (len - 1) / c + 1 : 0;
}
// The most chunks a stream of up to `cap` positions can have.
__host__ __device__ inline int most_chunks(int cap) {
  int most = 0;
  for (long long border = 4096, n = 16;; border *= border < 65536 ? 4 : 2) {
    if (cap <= border) {
      const int c = chunks_of(cap);
      return most > c ? most : c;
    }
    most = (int)n;
    if (border < 65536) n *= 2;
  }
}

// Checks a caller's cache descriptor (kv8_append.cu); `who` opens the message.
bm_status check_cache(const bm_kv8_cache* c, const char* who, Cache* out);

}  // namespace kv8
}  // namespace bm
