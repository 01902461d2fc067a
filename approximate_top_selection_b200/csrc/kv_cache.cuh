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
  uint32_t page_magic, page_shift;  // t / page_size = (t * page_magic) >> page_shift for 0 <= t < 2^31

  __device__ __forceinline__ int page_of(int t) const {
    return static_cast<int>((static_cast<uint64_t>(t) * page_magic) >> page_shift);
  }
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

// Four e4m3 codes as f16 values (exact: 4 significant bits, exponents -9 .. 8): the
// lower two and the upper two of a word.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t four, uint32_t& low, uint32_t& high) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(low), "=r"(high)
      : "r"(four));
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Four floats as e4m3 codes, a in the low byte (round to nearest even; the
// callers keep magnitudes within 448, so saturation never acts; NaN gives code
// 0x7F).
__device__ __forceinline__ uint32_t floats_to_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
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

// D / 16 lanes per row, 16 values a lane, two rows of a lane group in flight.  A
// CTA takes 16 tokens (blockIdx.x) by write_lines() of the tokens' lines (k or
// v, head; blockIdx.y), rows numbered by line, then token: the rows of a warp
// are successive tokens of one head, which in a prompt are neighbours in the
// cache, and so are their scales.  Bound by memory as far as bytes go (every
// value read once, 2 bytes, and written once), but near the issue limit too: 16
// values of a lane are widened, scaled and rounded in about 70 instructions, and
// finding the row must not take more.  Measured: 49999 tokens x 8 heads x 128 to
// e4m3 in 62 us, 4.9 TB/s (with 64-bit divisions for the row and the
// page: 68 us, issue slots 75 % busy; rows numbered by token: 73 us).
constexpr int kWriteTokens = 16;

template <int D>
__host__ __device__ constexpr int write_lines() {
  return 2 * 256 / (D / 16) / kWriteTokens;
}

__device__ __noinline__ int64_t divide_wide(int64_t a, int64_t b) { return a / b; }

__device__ __forceinline__ uint32_t larger_bf16x2(uint32_t a, uint32_t b) {  // NaN is the largest
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(256, 5) cache_write_kernel(WriteArgs p) {
  constexpr int L = D / 16, kGroups = 256 / L, kRows = 2;
  pdl_wait_then_release();
  const int heads = p.cache[0].kv_heads;
  const int gl = threadIdx.x % L;
  const unsigned mask = ((1u << L) - 1u) << (threadIdx.x % 32 / L * L);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kWriteTokens;
  for (int line0 = blockIdx.y * write_lines<D>(); line0 < 2 * heads; line0 += gridDim.y * write_lines<D>()) {
    int64_t slot[kRows];
    uint4 x[kRows][2];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int j = i * kGroups + static_cast<int>(threadIdx.x) / L;
      const int64_t t = t0 + j % kWriteTokens;
      const int line = line0 + j / kWriteTokens;
      const bool live = t < p.tokens && line < 2 * heads;
      const int w = line >= heads ? 1 : 0;
      slot[i] = live ? __ldg(p.slots + t) : -1;
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      if (live) {  // not waiting for the slot
        const uint4* src = reinterpret_cast<const uint4*>((w ? p.src[1] : p.src[0]) +
                                                          t * (w ? p.token_stride[1] : p.token_stride[0]) +
                                                          (line - w * heads) * (w ? p.head_stride[1] : p.head_stride[0])) +
                           gl * 2;
        x[i][0] = __ldcs(src);
        x[i][1] = __ldcs(src + 1);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (slot[i] < 0) continue;  // the same for a group's lanes
      const int line = line0 + (i * kGroups + static_cast<int>(threadIdx.x) / L) / kWriteTokens;
      const int w = line >= heads ? 1 : 0, h = line - w * heads;
      const CacheView& c = p.cache[w];
      const int64_t page = slot[i] <= 0x7fffffff ? c.page_of(static_cast<int>(slot[i])) : divide_wide(slot[i], c.page_size);
      if (page >= c.pages) {
        atomicOr(&g_device_status, kDevBadIndex);
        continue;
      }
      const int off = static_cast<int>(slot[i] - page * c.page_size);
      unsigned char* dst = c.data + page * c.page_stride + h * c.head_stride + off * c.token_stride;
      if constexpr (!kE4m3) {
        reinterpret_cast<uint4*>(dst)[gl * 2] = x[i][0];
        reinterpret_cast<uint4*>(dst)[gl * 2 + 1] = x[i][1];
      } else {
        const uint32_t xs[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
        uint32_t both = 0;  // the largest magnitudes of the even and the odd values
#pragma unroll
        for (int y = 0; y < 8; ++y) both = larger_bf16x2(both, xs[y] & 0x7fff7fffu);
#pragma unroll
        for (int o = L / 2; o >= 1; o >>= 1) both = larger_bf16x2(both, __shfl_xor_sync(mask, both, o));
        const uint32_t top = max(both << 16, both & 0xffff0000u);
        const bool finite = top < 0x7f800000u;
        const int e = row_exponent(top);
        const float inv = finite ? power_of_two(-e) : __uint_as_float(0x7fffffffu);
        uint32_t out[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          out[y] = floats_to_e4m3x4(__uint_as_float(xs[2 * y] << 16) * inv, __uint_as_float(xs[2 * y] & 0xffff0000u) * inv,
                                    __uint_as_float(xs[2 * y + 1] << 16) * inv,
                                    __uint_as_float(xs[2 * y + 1] & 0xffff0000u) * inv);
        reinterpret_cast<uint4*>(dst)[gl] = make_uint4(out[0], out[1], out[2], out[3]);
        if (gl == 0)
          c.scale[page * c.s_page_stride + h * c.s_head_stride + off * c.s_token_stride] =
              finite ? power_of_two(e) : __uint_as_float(0x7fffffffu);
      }
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

// A CTA reads read_rows() successive rows (blockIdx.x) of one head (blockIdx.y)
// of one sequence (blockIdx.z): D / 16 lanes per row, 16 values a lane, two rows
// of a lane group in flight.  Rows past a sequence's end (and rows whose page
// does not exist) are zero.  Bound by memory: the cached row read once, 2 bytes
// a value written.  Measured: 16 ragged sequences up to 32768, 8 heads x 128,
// e4m3: 254 us, 5.5 TB/s (with 64-bit divisions for sequence and head: 256
// us, issue slots 75 % busy).
template <int D>
__host__ __device__ constexpr int read_rows() {
  return 2 * 256 / (D / 16);
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(256, 6) cache_read_kernel(ReadArgs p) {
  constexpr int L = D / 16, kGroups = 256 / L, kRows = 2;
  pdl_wait_then_release();
  const CacheView& c = p.cache;
  const int gl = threadIdx.x % L, g = threadIdx.x / L;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * read_rows<D>() + g;
  for (int b = blockIdx.z; b < p.tab.batch; b += gridDim.z) {
    const int len = seq_length(p.tab, b);
    for (int h = blockIdx.y; h < c.kv_heads; h += gridDim.y) {
      int32_t page[kRows];
      int off[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t t = t0 + i * kGroups;
        page[i] = -1;
        off[i] = 0;
        if (t < len && t < p.n) {
          const int at = c.page_of(static_cast<int>(t));
          off[i] = static_cast<int>(t) - at * c.page_size;
          page[i] = __ldg(p.tab.table + b * p.tab.stride + at);
          if (page[i] < 0 || page[i] >= c.pages) {
            atomicOr(&g_device_status, kDevBadIndex);
            page[i] = -1;
          }
        }
      }
      uint4 x[kRows][2];
      float s[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
        s[i] = 0.0f;
        if (page[i] >= 0) {
          const uint4* src = reinterpret_cast<const uint4*>(c.data + page[i] * c.page_stride + h * c.head_stride +
                                                            off[i] * c.token_stride);
          if constexpr (kE4m3) {
            x[i][0] = __ldg(src + gl);
            s[i] = __ldg(c.scale + page[i] * c.s_page_stride + h * c.s_head_stride + off[i] * c.s_token_stride);
          } else {
            x[i][0] = __ldg(src + gl * 2);
            x[i][1] = __ldg(src + gl * 2 + 1);
          }
        }
      }
      uint4* dst = reinterpret_cast<uint4*>(p.out + ((static_cast<int64_t>(b) * c.kv_heads + h) * p.n + t0) * D) + gl * 2;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (t0 + i * kGroups >= p.n) continue;
        uint4 o0 = x[i][0], o1 = x[i][1];
        if constexpr (kE4m3) {
          const uint32_t w[4] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w};
          uint32_t o[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t low, high;
            e4m3x4_to_f16x2(w[y], low, high);
            const float2 a = f16x2_to_float2(low), z = f16x2_to_float2(high);
            o[2 * y] = floats_to_bf16x2(a.x * s[i], a.y * s[i]);
            o[2 * y + 1] = floats_to_bf16x2(z.x * s[i], z.y * s[i]);
          }
          o0 = make_uint4(o[0], o[1], o[2], o[3]);
          o1 = make_uint4(o[4], o[5], o[6], o[7]);
        }
        __stcs(dst + i * kGroups * (D / 8), o0);
        __stcs(dst + i * kGroups * (D / 8) + 1, o1);
      }
    }
  }
}

}  // namespace tk
