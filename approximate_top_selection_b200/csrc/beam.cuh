// beam.cuh -- one step of beam search: the k best continuations of a
// sentence's beams, and the beams' states brought into the new order.
//
// Continuation (i, t) of beam i by token t is worth s_i + x_it - lse_i, with
// lse_i = log sum_t exp(x_it).  Beams of score -inf have ended, tokens of logit
// -inf are forbidden: neither gives a continuation.  Continuations rank by
// value (held in 64 bits; NaN first, as everywhere in this library), then by
// lower beam, then by larger logit, then by lower token.  A beam whose logits
// hold a NaN or +inf has no log-sum-exp: its values are NaN.
#pragma once

#include "common.cuh"

namespace tk {

constexpr int kBeamThreads = 256;

__device__ __forceinline__ float logit_value(float x) { return x; }
__device__ __forceinline__ float logit_value(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// Unsigned order of a double's value; NaN above all, 0 is never produced.
__device__ __forceinline__ uint64_t order_key64(double v) {
  if (v != v) return ~0ull;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// A continuation: larger `value` first, then larger `rest` (complement of the
// beam, order key of the logit), then lower token.
struct Cont {
  uint64_t value;
  uint64_t rest;
  uint32_t token;
};

__device__ __forceinline__ bool ranks_above(const Cont& a, const Cont& b) {
  if (a.value != b.value) return a.value > b.value;
  if (a.rest != b.rest) return a.rest > b.rest;
  return a.token < b.token;
}

struct BeamArgs {
  const void* logits;   // [batch][beams][n]
  const float* scores;  // [batch][beams]
  int64_t n;
  int beams, k;
  float* out_scores;    // [batch][k]
  int32_t* out_parent;  // [batch][k]
  int32_t* out_token;   // [batch][k]
};

constexpr int kMaxBeams = 128;

// One CTA per sentence: log-sum-exp of every beam, then k rounds that each
// find the best continuation below the last one.
template <typename T>
__global__ void __launch_bounds__(kBeamThreads) topk_beam_simple(BeamArgs p) {
  __shared__ double off[kMaxBeams];
  __shared__ double rsum[kBeamThreads];
  __shared__ float rmax[kBeamThreads];
  __shared__ Cont best[kBeamThreads];
  pdl_wait_then_release();
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x;
  const float ninf = __int_as_float(0xff800000);
  for (int i = 0; i < p.beams; ++i) {
    const T* x = static_cast<const T*>(p.logits) + (b * p.beams + i) * p.n;
    float m = ninf;
    bool bad = false;
    for (int64_t t = tid; t < p.n; t += kBeamThreads) {
      const float v = logit_value(x[t]);
      bad |= v != v || v == __int_as_float(0x7f800000);
      m = fmaxf(m, v);
    }
    rmax[tid] = m;
    bad = __syncthreads_or(bad);
    for (int s = kBeamThreads / 2; s; s >>= 1) {
      if (tid < s) rmax[tid] = fmaxf(rmax[tid], rmax[tid + s]);
      __syncthreads();
    }
    m = rmax[0];
    double sum = 0.0;
    if (!bad && m != ninf)
      for (int64_t t = tid; t < p.n; t += kBeamThreads)
        sum += exp(static_cast<double>(logit_value(x[t])) - static_cast<double>(m));
    rsum[tid] = sum;
    __syncthreads();
    for (int s = kBeamThreads / 2; s; s >>= 1) {
      if (tid < s) rsum[tid] += rsum[tid + s];
      __syncthreads();
    }
    if (tid == 0)
      off[i] = static_cast<double>(p.scores[b * p.beams + i]) -
               (bad ? __longlong_as_double(0x7ff8000000000000ll) : static_cast<double>(m) + log(rsum[0]));
    __syncthreads();
  }
  Cont last = {~0ull, ~0ull, 0};
  bool first = true;
  for (int j = 0; j < p.k; ++j) {
    Cont mine = {0, 0, 0};  // value 0: none
    for (int i = 0; i < p.beams; ++i) {
      if (p.scores[b * p.beams + i] == ninf) continue;
      const T* x = static_cast<const T*>(p.logits) + (b * p.beams + i) * p.n;
      for (int64_t t = tid; t < p.n; t += kBeamThreads) {
        const float v = logit_value(x[t]);
        if (v == ninf) continue;
        const Cont c = {order_key64(off[i] + static_cast<double>(v)),
                        (static_cast<uint64_t>(~static_cast<uint32_t>(i)) << 32) | order_key(v),
                        static_cast<uint32_t>(t)};
        if ((first || ranks_above(last, c)) && ranks_above(c, mine)) mine = c;
      }
    }
    best[tid] = mine;
    __syncthreads();
    for (int s = kBeamThreads / 2; s; s >>= 1) {
      if (tid < s && ranks_above(best[tid + s], best[tid])) best[tid] = best[tid + s];
      __syncthreads();
    }
    last = best[0];
    first = false;
    const bool none = last.value == 0;
    if (tid == 0) {
      const int i = static_cast<int>(~static_cast<uint32_t>(last.rest >> 32));
      const int64_t o = b * p.k + j;
      p.out_scores[o] = none ? ninf : static_cast<float>(off[i] + static_cast<double>(key_value(static_cast<uint32_t>(last.rest))));
      p.out_parent[o] = none ? -1 : i;
      p.out_token[o] = none ? -1 : static_cast<int32_t>(last.token);
    }
    __syncthreads();
    if (none) {
      for (int r = j + 1 + tid; r < p.k; r += kBeamThreads) {
        p.out_scores[b * p.k + r] = ninf;
        p.out_parent[b * p.k + r] = -1;
        p.out_token[b * p.k + r] = -1;
      }
      break;
    }
  }
}

// ---------------------------------------------------------------- reordering
constexpr int kReorderStates = 64;  // tensors per launch

struct ReorderArgs {
  const unsigned char* src[kReorderStates];  // [batch][beams][row_bytes]
  unsigned char* dst[kReorderStates];        // [batch][k][row_bytes]
  int64_t row_bytes[kReorderStates];
  const int32_t* parents;  // [batch][k]
  int64_t batch;
  int beams, k;
};

// One CTA per (new beam, tensor).
__global__ void __launch_bounds__(256) beam_reorder_simple(ReorderArgs p) {
  pdl_wait_then_release();
  const int s = blockIdx.y;
  const int64_t r = blockIdx.x;
  const int64_t nb = p.row_bytes[s];
  const int32_t parent = __ldg(p.parents + r);
  unsigned char* dst = p.dst[s] + r * nb;
  if (parent < 0 || parent >= p.beams) {
    if (parent != -1 && threadIdx.x == 0) atomicOr(&g_device_status, 2);
    for (int64_t i = threadIdx.x; i < nb; i += 256) dst[i] = 0;
    return;
  }
  const unsigned char* src = p.src[s] + (r / p.k * p.beams + parent) * nb;
  for (int64_t i = threadIdx.x; i < nb; i += 256) dst[i] = src[i];
}

}  // namespace tk
