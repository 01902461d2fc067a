// kv_cache.cuh -- the paged key-value cache: where a cached row lies, the
// e4m3 form of a row, and the kernels that write new tokens' rows into their
// slots and read sequences back as contiguous bf16 rows.
//
// A cache tensor is [pages][kv_heads][page_size][d] (any strides over the
// first three).  Sequence b's token t lies on page block_table[b][t / page_size]
// at offset t % page_size.  The e4m3 form keeps one float32 scale per row
// (page, head, offset): a row x of d values is stored as code_i =
// rn_e4m3(x_i / 2^e), scale = 2^e, with the smallest e >= -127 for which
// max|x_i| <= 448 * 2^e (e = 0 for a row of zeros).  A power of two costs an
// 8-bit float nothing but range, and makes the division exact: the only
// rounding of a stored value is the one to 4 significant bits (relative
// 2^-4, absolute 2^-10 * 2^e below the smallest normal code).
// A row holding a NaN or an infinity has no such e: its scale is NaN and the
// whole row reads back as NaN.
#pragma once

#include "common.cuh"

namespace tk {

constexpr int kDevBadIndex = 2;  // TOPK_DEV_BAD_INDEX

struct CacheView {
  unsigned char* data;
  float* scale;                                   // null for bf16
  int64_t page_stride, head_stride, token_stride;        // bytes
  int64_t s_page_stride, s_head_stride, s_token_stride;  // elements of scale
  int64_t pages;
  int kv_heads, page_size;
};

struct TableView {
  const int32_t* table;  // [batch][stride], `width` entries used
  const int32_t* lens;   // [batch]
  int64_t stride;
  int64_t capacity;  // width * page_size
  int batch;
};

// Length of sequence b: seq_lens[b] held to [0, capacity]; a longer one is flagged.
__device__ __forceinline__ int seq_length(const TableView& t, int b) {
  const int n = __ldg(t.lens + b);
  if (n <= 0) return 0;
  if (n > t.capacity) {
    atomicOr(&g_device_status, kDevBadIndex);
    return static_cast<int>(t.capacity);
  }
  return n;
}

// Two e4m3 codes as two f16 values (exact: 4 significant bits, exponents -9 .. 8).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Two floats as e4m3 codes, a in the low byte (round to nearest even; the
// callers keep |a|, |b| <= 448, so saturation never acts; NaN gives code 0x7F).
__device__ __forceinline__ uint32_t floats_to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ uint32_t floats_to_bf16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// 2^e of a row whose largest magnitude has the float bits `top` (sign clear).
__device__ __forceinline__ int row_exponent(uint32_t top) {
  if (top == 0u) return 0;
  const int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;  // 448 = 1.75 * 2^8
}

__device__ __forceinline__ float power_of_two(int e) {  // -127 <= e <= 127
  return e > -127 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : __uint_as_float(0x00400000u);
}

// ---------------------------------------------------------------- writing
struct WriteArgs {
  const uint16_t* src[2];  // k, v: [tokens][kv_heads][d] bf16
  int64_t token_stride[2], head_stride[2];  // elements
  CacheView cache[2];
  const int64_t* slots;  // [tokens]: page * page_size + offset, negative: skipped
  int64_t tokens;
};

// One group of D / 8 lanes per row (16 bytes a lane).
template <int D, bool kE4m3>
__global__ void __launch_bounds__(256) cache_write_kernel(WriteArgs p) {
  constexpr int L = D / 8;
  pdl_wait_then_release();
  const int heads = p.cache[0].kv_heads;
  const int64_t rows = p.tokens * heads * 2;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (256 / L);
  const int gl = threadIdx.x % L;
  const unsigned mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (threadIdx.x % 32 / L * L);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / L) + threadIdx.x / L; r < rows; r += groups) {
    const int w = static_cast<int>(r & 1);
    const int h = static_cast<int>((r >> 1) % heads);
    const int64_t t = (r >> 1) / heads;
    const int64_t slot = __ldg(p.slots + t);
    if (slot < 0) continue;
    const CacheView& c = p.cache[w];
    const int64_t page = slot / c.page_size;
    if (page >= c.pages) {
      atomicOr(&g_device_status, kDevBadIndex);
      continue;
    }
    const int off = static_cast<int>(slot - page * c.page_size);
    const uint4 x = *reinterpret_cast<const uint4*>(p.src[w] + t * p.token_stride[w] + h * p.head_stride[w] + gl * 8);
    unsigned char* dst = c.data + page * c.page_stride + h * c.head_stride + off * c.token_stride;
    if constexpr (!kE4m3) {
      *reinterpret_cast<uint4*>(dst + gl * 16) = x;
    } else {
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
      float f[8];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(xs[i] << 16);
        f[2 * i + 1] = __uint_as_float(xs[i] & 0xffff0000u);
        top = max(top, max((xs[i] << 16) & 0x7fff0000u, xs[i] & 0x7fff0000u));
      }
#pragma unroll
      for (int o = L / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
      const bool finite = top < 0x7f800000u;
      const int e = row_exponent(top);
      const float inv = finite ? power_of_two(-e) : __uint_as_float(0x7fffffffu);
      uint32_t out[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        out[i] = floats_to_e4m3x2(f[4 * i] * inv, f[4 * i + 1] * inv) |
                 (floats_to_e4m3x2(f[4 * i + 2] * inv, f[4 * i + 3] * inv) << 16);
      *reinterpret_cast<uint2*>(dst + gl * 8) = make_uint2(out[0], out[1]);
      if (gl == 0)
        c.scale[page * c.s_page_stride + h * c.s_head_stride + off * c.s_token_stride] =
            finite ? power_of_two(e) : __uint_as_float(0x7fffffffu);
    }
  }
}

// ---------------------------------------------------------------- reading
struct ReadArgs {
  CacheView cache;
  TableView tab;
  int64_t n;
  uint16_t* out;  // [batch][kv_heads][n][d] bf16
};

// One group of D / 8 lanes per row of the output; rows past a sequence's end
// (and rows whose page does not exist) are zero.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(256) cache_read_kernel(ReadArgs p) {
  constexpr int L = D / 8;
  pdl_wait_then_release();
  const CacheView& c = p.cache;
  const int64_t rows = static_cast<int64_t>(p.tab.batch) * c.kv_heads * p.n;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (256 / L);
  const int gl = threadIdx.x % L;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / L) + threadIdx.x / L; r < rows; r += groups) {
    const int64_t bh = r / p.n;
    const int64_t t = r - bh * p.n;
    const int b = static_cast<int>(bh / c.kv_heads), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.kv_heads);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (t < seq_length(p.tab, b)) {
      const int64_t at = t / c.page_size;
      const int off = static_cast<int>(t - at * c.page_size);
      const int32_t page = __ldg(p.tab.table + b * p.tab.stride + at);
      if (page < 0 || page >= c.pages) {
        atomicOr(&g_device_status, kDevBadIndex);
      } else {
        const unsigned char* src = c.data + page * c.page_stride + h * c.head_stride + off * c.token_stride;
        if constexpr (!kE4m3) {
          x = __ldg(reinterpret_cast<const uint4*>(src + gl * 16));
        } else {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(src + gl * 8));
          const float s = __ldg(c.scale + page * c.s_page_stride + h * c.s_head_stride + off * c.s_token_stride);
          const uint32_t two[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(two[i]));
            o[i] = floats_to_bf16x2(f.x * s, f.y * s);
          }
          x = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    *reinterpret_cast<uint4*>(p.out + r * D + gl * 8) = x;
  }
}

}  // namespace tk
