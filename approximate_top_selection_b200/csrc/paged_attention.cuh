// paged_attention.cuh -- attention of one new token per sequence over a paged
// key-value cache: o = sum_j p_j V_j, p = softmax(scale * q . K_j) over the
// sequence's cached tokens, or over the positions a selector listed.
#pragma once

#include "kv_cache.cuh"

namespace tk {

struct AttendArgs {
  const uint16_t* q;  // [batch][heads][d] bf16
  int64_t q_stride;   // elements between sequences
  CacheView k, v;
  TableView tab;
  const int32_t* positions;  // null, or [batch][lists][c]
  int heads, lists, c;
  float scale_log2;  // softmax scale * log2(e)
  uint16_t* out;  // [batch][heads][d] bf16
  float* lse;     // null, or [batch][heads]
};

// One CTA of four warps per (sequence, head): each warp takes every fourth
// key with its own running maximum and sum (the lanes split d), and the four
// are joined at the end.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(128) paged_attention_simple(AttendArgs p) {
  constexpr int PER = D / 32;  // values per lane
  __shared__ float so[4][D];
  __shared__ float sm[4], sl[4];
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x % p.heads, b = blockIdx.x / p.heads;
  const int kvh = static_cast<int>(static_cast<int64_t>(h) * p.k.kv_heads / p.heads);
  const int n = seq_length(p.tab, b);
  const int list = p.positions ? static_cast<int>(static_cast<int64_t>(h) * p.lists / p.heads) : 0;
  const int32_t* pos = p.positions ? p.positions + (static_cast<int64_t>(b) * p.lists + list) * p.c : nullptr;
  const int count = pos ? p.c : n;
  float q[PER], o[PER];
  const uint16_t* qr = p.q + b * p.q_stride + static_cast<int64_t>(h) * D + lane * PER;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    q[i] = __uint_as_float(static_cast<uint32_t>(qr[i]) << 16);
    o[i] = 0.0f;
  }
  float m = __int_as_float(0xff800000), l = 0.0f;
  for (int j = warp; j < count; j += 4) {
    int t = j;
    if (pos) {
      t = __ldg(pos + j);
      if (t < 0) continue;
      if (t >= n) {
        if (t >= p.tab.capacity) atomicOr(&g_device_status, kDevBadIndex);
        continue;
      }
    }
    const int at = t / p.k.page_size, off = t % p.k.page_size;
    const int32_t page = __ldg(p.tab.table + b * p.tab.stride + at);
    if (page < 0 || page >= p.k.pages) {
      atomicOr(&g_device_status, kDevBadIndex);
      continue;
    }
    const unsigned char* kr = p.k.data + page * p.k.page_stride + kvh * p.k.head_stride + off * p.k.token_stride;
    const unsigned char* vr = p.v.data + page * p.v.page_stride + kvh * p.v.head_stride + off * p.v.token_stride;
    float kf[PER], vf[PER];
    if constexpr (kE4m3) {
      const float ks = p.k.scale[page * p.k.s_page_stride + kvh * p.k.s_head_stride + off * p.k.s_token_stride];
      const float vs = p.v.scale[page * p.v.s_page_stride + kvh * p.v.s_head_stride + off * p.v.s_token_stride];
#pragma unroll
      for (int i = 0; i < PER; i += 2) {
        const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kr + lane * PER + i)));
        const float2 c = f16x2_to_float2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(vr + lane * PER + i)));
        kf[i] = a.x * ks;
        kf[i + 1] = a.y * ks;
        vf[i] = c.x * vs;
        vf[i + 1] = c.y * vs;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        kf[i] = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(kr)[lane * PER + i]) << 16);
        vf[i] = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(vr)[lane * PER + i]) << 16);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) s = fmaf(q[i], kf[i], s);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float ref = mn == __int_as_float(0xff800000) ? 0.0f : mn;
    const float f = exp2f(m - ref), w = exp2f(s - ref);
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = o[i] * f + w * vf[i];
    m = mn;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) so[warp][lane * PER + i] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const float ref = mm == __int_as_float(0xff800000) ? 0.0f : mm;
  float f[4], total = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = exp2f(sm[w] - ref);
    total += sl[w] * f[w];
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t row = static_cast<int64_t>(b) * p.heads + h;
  for (int i = threadIdx.x; i < D; i += 128) {
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) a += so[w][i] * f[w];
    p.out[row * D + i] = static_cast<uint16_t>(floats_to_bf16x2(total == 0.0f ? 0.0f : a * inv, 0.0f));
  }
  if (p.lse && threadIdx.x == 0) p.lse[row] = 0.6931471805599453f * (mm + log2f(total));
}

}  // namespace tk
