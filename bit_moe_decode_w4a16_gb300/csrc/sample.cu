// Drawing tokens from logits: temperature, top-k, top-p and min-p, with the
// random numbers given by the caller.
//
// For a row of logits x with the largest value m and temperature T > 0, the
// weights are w_i = e^((x_i - m) / T), ordered by falling x and, among equal
// x, by rising index.  Kept are
//   top-k: the first k of that order;
//   top-p: of these, the smallest prefix whose weight is at least p times theirs;
//   min-p: of these, the ones with w >= min_p * (the largest w = 1);
// and always the first.  Every filter keeps a prefix of the order, so the kept
// set is "x above a threshold, or equal to it and among the first r indices".
// The draw walks the kept tokens by rising index: the first whose cumulated
// weight exceeds u times the kept weight.
//
// One CTA per row; each threshold is a binary search over the ordered bit
// patterns of x, one sweep of the row per bit.
#include "common.cuh"
#include "errors.h"

namespace bm {
namespace {

constexpr int kThreads = 1024;

struct SampleArgs {
  const void* x;
  long long ld;
  int V, B;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* ids;
  float* logp;
};

// Order-preserving bit pattern; NaN and -infinity are 0 (never drawn).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u || b == 0xFF800000u) return 0u;
  if (b == 0x80000000u) return 0x80000000u;   // -0 equals +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <typename T>
__device__ __forceinline__ float load_logit(const void* x, long long i) {
  if (sizeof(T) == 4) return static_cast<const float*>(x)[i];
  return bf2f(static_cast<const bf16*>(x)[i]);
}

template <typename T>
__device__ T block_sum(T v, T* red) {
  __syncthreads();
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  T s = 0;
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(SampleArgs a) {
  __shared__ double red_d[32];
  __shared__ int red_i[32];
  __shared__ double part[kThreads];
  const int b = blockIdx.x, V = a.V, t = threadIdx.x;
  const long long row = b * a.ld;
  auto key = [&](int i) { return key_of(load_logit<T>(a.x, row + i)); };
  // thread t owns the indices [lo, hi): index order is thread order
  const int lo = (int)((long long)V * t / kThreads), hi = (int)((long long)V * (t + 1) / kThreads);
  const float T0 = a.temperature ? a.temperature[b] : 1.f;
  const bool greedy = !(T0 > 0.f);
  uint32_t best = 0;
  for (int i = lo; i < hi; ++i) best = max(best, key(i));
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if ((t & 31) == 0) red_i[t >> 5] = (int)best;
  __syncthreads();
  for (int w = 0; w < 32; ++w) best = max(best, (uint32_t)red_i[w]);
  __syncthreads();
  if (best == 0) {
    if (t == 0) {
      a.ids[b] = -1;
      if (a.logp) a.logp[b] = -INFINITY;
    }
    return;
  }
  const double top = value_of(best), invT = 1.0 / (double)(greedy ? 1.f : T0);
  auto weight = [&](uint32_t k) -> double {
    if (k == best) return 1.0;
    return k == 0 ? 0.0 : exp(((double)value_of(k) - top) * invT);
  };
  // the kept set: key > cut, or key == cut and among the first `ties` indices
  uint32_t cut = greedy ? best : 1;
  long long ties = greedy ? 1 : V;
  auto count_from = [&](uint32_t k) {
    int n = 0;
    for (int i = lo; i < hi; ++i) n += key(i) >= k;
    return block_sum(n, red_i);
  };
  const int k = a.top_k && !greedy ? a.top_k[b] : 0;
  if (k > 0 && k < V) {
    uint32_t at = 0;   // the largest threshold that at least k keys reach
    for (int bit = 31; bit >= 0; --bit)
      if (count_from(at | (1u << bit)) >= k) at |= 1u << bit;
    if (at > cut) {
      cut = at;
      ties = k - (at == 0xFFFFFFFFu ? 0 : count_from(at + 1));
    }
  }
  // weight of the keys >= thr inside the top-k set
  auto mass_from = [&](uint32_t thr) {
    double s = 0;
    for (int i = lo; i < hi; ++i) {
      const uint32_t v = key(i);
      if (v >= thr && v > cut) s += weight(v);
    }
    s = block_sum(s, red_d);
    if (cut < thr) return s;
    const long long equal = (long long)count_from(cut) - (cut == 0xFFFFFFFFu ? 0 : count_from(cut + 1));
    return equal > 0 ? s + (double)min(ties, equal) * weight(cut) : s;
  };
  const float p = a.top_p && !greedy ? a.top_p[b] : 1.f;
  if (p < 1.f) {
    const double need = (double)p * mass_from(cut);
    uint32_t at = 0;
    for (int bit = 31; bit >= 0; --bit)
      if (mass_from(at | (1u << bit)) >= need) at |= 1u << bit;
    at = min(at, best);
    const double above = at == 0xFFFFFFFFu ? 0.0 : mass_from(at + 1);
    const double w = weight(at);
    long long r = w > 0 ? (long long)ceil((need - above) / w) : 1;
    r = max(r, 1LL);
    if (at > cut || (at == cut && r < ties)) {
      cut = at;
      ties = r;
    }
  }
  const float mp = a.min_p && !greedy ? a.min_p[b] : 0.f;
  if (mp > 0.f) {
    uint32_t at = 0;   // the smallest key whose weight reaches min_p: weights rise with the key
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t cand = at | (1u << bit);
      if (cand <= best && weight(cand - 1) < (double)fminf(mp, 1.f)) at = cand;
    }
    if (at > cut) {
      cut = at;
      ties = V;
    }
  }
  // equal keys before this thread's indices
  int eq = 0;
  for (int i = lo; i < hi; ++i) eq += key(i) == cut;
  __syncthreads();
  part[t] = eq;
  __syncthreads();
  long long before = 0;
  for (int i = 0; i < t; ++i) before += (long long)part[i];
  __syncthreads();
  double s = 0;
  long long seen = before;
  for (int i = lo; i < hi; ++i) {
    const uint32_t v = key(i);
    if (v > cut || (v == cut && seen++ < ties)) s += weight(v);
  }
  part[t] = s;
  __syncthreads();
  if (t == 0) {
    double total = 0;
    for (int i = 0; i < kThreads; ++i) total += part[i];
    const float u = a.u && a.u[b] > 0.f ? a.u[b] : 0.f;
    const double target = (double)u * total;
    double cum = 0;
    int own = 0;
    while (own < kThreads - 1 && cum + part[own] <= target) cum += part[own++];
    // walk the owner's indices; a target past the last kept token takes that token
    int id = -1;
    double wid = 0;
    for (int th = own; th >= 0 && id < 0; --th) {
      const int l2 = (int)((long long)V * th / kThreads), h2 = (int)((long long)V * (th + 1) / kThreads);
      long long eqs = 0;
      for (int i = 0; i < l2; ++i) eqs += key(i) == cut;
      for (int i = l2; i < h2; ++i) {
        const uint32_t v = key(i);
        if (v > cut || (v == cut && eqs++ < ties)) {
          const double w = weight(v);
          if (!(w > 0)) continue;
          id = i;
          wid = w;
          cum += w;
          if (th == own && cum > target) break;
        }
      }
    }
    a.ids[b] = id;
    if (a.logp) a.logp[b] = greedy ? 0.f : (float)log(wid / total);
  }
}

}  // namespace
}  // namespace bm

extern "C" bm_status bm_sample(const void* logits, int dtype, int64_t ld, int V, int B, const float* temperature,
                               const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* ids,
                               float* logprobs, void* stream) {
  using namespace bm;
  if (!logits || !u || !ids) return set_error(BM_ERR_INVALID_ARG, "bm_sample: null pointer");
  if (dtype != BM_F32 && dtype != BM_BF16) return set_error(BM_ERR_INVALID_ARG, "bm_sample: dtype must be BM_F32 or BM_BF16");
  if (B < 1 || B > 65535 || V < 1 || V > BM_SAMPLE_MAX_VOCAB)
    return set_error(BM_ERR_INVALID_ARG, "bm_sample: need 1 <= B <= 65535 and 1 <= V <= " + std::to_string(BM_SAMPLE_MAX_VOCAB));
  if (ld < V) return set_error(BM_ERR_INVALID_ARG, "bm_sample: ld must be at least V");
  if ((uintptr_t)logits & (dtype == BM_F32 ? 3 : 1)) return set_error(BM_ERR_INVALID_ARG, "bm_sample: misaligned logits");
  SampleArgs a{logits, ld, V, B, temperature, top_k, top_p, min_p, u, ids, logprobs};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == BM_F32) k_sample<float><<<B, kThreads, 0, s>>>(a);
  else k_sample<bf16><<<B, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(BM_ERR_CUDA, std::string("bm_sample: ") + cudaGetErrorString(e));
  return ok();
}
