// What the kernels of attention over the 8-bit cache share.
#pragma once

#include <algorithm>

#include "kv8.cuh"

namespace bm {
namespace kv8 {

constexpr int kMaxGroup = 8, kMaxBatch = 1024;

struct AttendArgs {
  Cache c, p;            // the streams' cache, the prefix's
  int p_slot, p_len, p_chunk, p_chunks;
  const bf16* Q;
  const int32_t* slots;
  const int32_t* lens;
  bf16* O;
  float* rec_o;          // records [B][q_heads][p_chunks + own chunks]: unnormalised output [d]
  float2* rec_ml;        // and its maximum and sum
  int B, qh, own_chunks;
  float scale_log2;      // scale * log2(e): the scores are powers of two
  __host__ __device__ size_t record(int b, int h, int r) const { return ((size_t)b * qh + h) * (p_chunks + own_chunks) + r; }
  // A stream that takes part: padding and out-of-range rows are skipped.
  __device__ bool live(int b, int& slot, int& len) const {
    slot = slots[b];
    len = lens[b];
    return slot >= 0 && slot < c.slots && len >= 0 && len <= c.cap;
  }
};

// Four codes -> two fp16 pairs (exact).
template <int FMT>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == BM_KV8_E4M3) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // 0x64 in front of u = code + 128 is the fp16 1024 + u
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 k = __float2half2_rn(1152.f);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), k), y = __hsub2(*reinterpret_cast<const __half2*>(&b), k);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// v * 2^d for d <= 0, in two factors: 2^d alone becomes zero below -126.  A sum of weights needs it, as positions
// whose V is zero set the reference 100 below their score, which leaves the sum that much above 1.
__device__ __forceinline__ float scaled_down(float v, float d) {
  return v * exp2_fast(fmaxf(d, -120.f)) * exp2_fast(fminf(d + 120.f, 0.f));
}
__device__ __forceinline__ float log2_fast(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A power of two that brings a query row of largest magnitude `amax` into fp16's range; exact, and undone
// on the scores by its inverse.  The exponent is held where `down`, `up` and `up` times a score factor of 2^-7 to 2
// are normal numbers: rows of the type's largest binade become 2 .. 4, those below 2^-119 less than 1.
__device__ __forceinline__ void row_scale(float amax, float& down, float& up) {
  down = up = 1.f;
  const uint32_t bits = __float_as_uint(amax);
  if (bits < 0x7F800000u) {             // infinity and NaN stay, and make their scores NaN
    const uint32_t e = min(max(bits >> 23, 8u), 253u);
    down = __uint_as_float((254u - e) << 23);
    up = __uint_as_float(e << 23);
  }
}

// Positions per chunk of the shared prefix, and the chunks: at most as many as fill the GPU, one CTA an SM,
// for one tile of query rows.
inline int prefix_chunk(int len, int kvh) {
  const int most = kSms / kvh > 1 ? kSms / kvh : 1, tiles = len > 0 ? (len - 1) / 128 + 1 : 1;
  return std::min((tiles + most - 1) / most, 1 << 23) * 128;   // below 2^31
}
inline int prefix_chunks(int len, int kvh) {
  return len > 0 ? (len - 1) / prefix_chunk(len, kvh) + 1 : 0;
}

// The most chunks a prefix of up to `len` positions can have: their number falls where a chunk becomes a tile longer,
// and a workspace for the longest prefix has to do for all.
inline int most_prefix_chunks(int len, int kvh) {
  const int most = kSms / kvh > 1 ? kSms / kvh : 1, tiles = len > 0 ? (len - 1) / 128 + 1 : 0;
  return std::max(std::min(tiles, most), prefix_chunks(len, kvh));   // the second where chunks are as long as they get
}

// The prefix's records (kv8_prefix.cu).
cudaError_t launch_kv8_prefix(const AttendArgs& a, int format, int d, cudaStream_t s);

}  // namespace kv8
}  // namespace bm
