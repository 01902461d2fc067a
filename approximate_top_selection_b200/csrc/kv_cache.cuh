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

// Four codes: the lower two and the upper two of a word.
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

// D / 16 lanes per row, 16 values a lane, kWriteRows rows of a lane group in
// flight; a CTA takes 256 / (D / 16) * kWriteRows rows.  Rows are numbered by
// blocks of 16 tokens, in a block by (k or v, head), then by token: the rows of
// a warp are successive tokens of one head, which in a prompt are neighbours
// in the cache, and so are their scales.  Bound by memory: every value is read
// once (2 bytes) and written once.  Measured: 49999 tokens x 8 heads x 128 to
// e4m3 in 68 us, 4.4 TB/s (four rows in flight and a loop over the grid: 86 us;
// rows numbered by token: 73 us).
constexpr int kWriteRows = 2;
constexpr int kWriteBlock = 16;

template <int D>
__host__ __device__ constexpr int write_rows_per_cta() {
  return 256 / (D / 16) * kWriteRows;
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(256, 4) cache_write_kernel(WriteArgs p) {
  constexpr int L = D / 16, kGroups = 256 / L;
  pdl_wait_then_release();
  const int heads = p.cache[0].kv_heads;
  const int64_t block_rows = 2 * static_cast<int64_t>(heads) * kWriteBlock;
  const int64_t rows = (p.tokens + kWriteBlock - 1) / kWriteBlock * block_rows;
  const int gl = threadIdx.x % L;
  const unsigned mask = ((1u << L) - 1u) << (threadIdx.x % 32 / L * L);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * write_rows_per_cta<D>(); r0 < rows;
       r0 += static_cast<int64_t>(gridDim.x) * write_rows_per_cta<D>()) {
    const int64_t block0 = r0 / block_rows, in_block = r0 - block0 * block_rows;
    int64_t slot[kWriteRows];
    int64_t tok[kWriteRows];
    int ln[kWriteRows];
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
      int64_t j = in_block + i * kGroups + threadIdx.x / L, block = block0;
      while (j >= block_rows) {  // at most a few blocks on: a CTA has 128 rows, a block 32 or more
        j -= block_rows;
        ++block;
      }
      ln[i] = static_cast<int>(j / kWriteBlock);
      tok[i] = block * kWriteBlock + j % kWriteBlock;
      slot[i] = tok[i] < p.tokens ? __ldg(p.slots + tok[i]) : -1;
    }
    uint4 x[kWriteRows][2];
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
      const int w = ln[i] >= heads ? 1 : 0, h = ln[i] - w * heads;
      const uint4* src = reinterpret_cast<const uint4*>((w ? p.src[1] : p.src[0]) +
                                                        tok[i] * (w ? p.token_stride[1] : p.token_stride[0]) +
                                                        h * (w ? p.head_stride[1] : p.head_stride[0])) +
                         gl * 2;
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      if (tok[i] < p.tokens) {  // not waiting for the slot
        x[i][0] = __ldcs(src);
        x[i][1] = __ldcs(src + 1);
      }
    }
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
      if (slot[i] < 0) continue;  // the same for a group's lanes
      const int w = ln[i] >= heads ? 1 : 0, h = ln[i] - w * heads;
      const CacheView& c = p.cache[w];
      const int64_t page = (slot[i] >> 32) == 0
                               ? static_cast<int64_t>(static_cast<uint32_t>(slot[i]) / static_cast<uint32_t>(c.page_size))
                               : slot[i] / c.page_size;
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
        uint32_t top = 0;
#pragma unroll
        for (int y = 0; y < 8; ++y) top = max(top, max((xs[y] << 16) & 0x7fff0000u, xs[y] & 0x7fff0000u));
#pragma unroll
        for (int o = L / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
        const bool finite = top < 0x7f800000u;
        const int e = row_exponent(top);
        const float inv = finite ? power_of_two(-e) : __uint_as_float(0x7fffffffu);
        uint32_t out[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          out[y] = floats_to_e4m3x2(__uint_as_float(xs[2 * y] << 16) * inv, __uint_as_float(xs[2 * y] & 0xffff0000u) * inv) |
                   (floats_to_e4m3x2(__uint_as_float(xs[2 * y + 1] << 16) * inv,
                                     __uint_as_float(xs[2 * y + 1] & 0xffff0000u) * inv)
                    << 16);
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

// A CTA reads 256 / (D / 16) * kReadRows successive rows of one sequence and
// head: D / 16 lanes per row, 16 values a lane, kReadRows rows of a lane group
// in flight.  Rows past a sequence's end (and rows whose page does not exist)
// are zero.  Bound by memory: the cached row read once, 2 bytes a value written.
// Measured: 16 ragged sequences up to 32768, 8 heads x 128, e4m3: 256 us, 5.45
// TB/s (four rows in flight at five CTAs per SM: 270 us; eight: 293 us).
constexpr int kReadRows = 2;

template <int D>
__host__ __device__ constexpr int read_rows_per_cta() {
  return 256 / (D / 16) * kReadRows;
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(256, 8) cache_read_kernel(ReadArgs p) {
  constexpr int L = D / 16, kGroups = 256 / L;
  pdl_wait_then_release();
  const CacheView& c = p.cache;
  const int64_t blocks = (p.n + read_rows_per_cta<D>() - 1) / read_rows_per_cta<D>();  // of a sequence and head
  const int64_t items = blocks * p.tab.batch * c.kv_heads;
  const int gl = threadIdx.x % L, g = threadIdx.x / L;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t bh = item / blocks;
    const int b = static_cast<int>(bh / c.kv_heads), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.kv_heads);
    const int64_t t0 = (item - bh * blocks) * read_rows_per_cta<D>() + g;
    const int len = seq_length(p.tab, b);
    int32_t page[kReadRows];
    int off[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      const int64_t t = t0 + i * kGroups;
      page[i] = -1;
      off[i] = 0;
      if (t < len && t < p.n) {
        const int at = static_cast<int>(t) / c.page_size;
        off[i] = static_cast<int>(t) - at * c.page_size;
        page[i] = __ldg(p.tab.table + b * p.tab.stride + at);
        if (page[i] < 0 || page[i] >= c.pages) {
          atomicOr(&g_device_status, kDevBadIndex);
          page[i] = -1;
        }
      }
    }
    uint4 x[kReadRows][2];
    float s[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
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
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      const int64_t t = t0 + i * kGroups;
      if (t >= p.n) continue;
      uint4 o0 = x[i][0], o1 = x[i][1];
      if constexpr (kE4m3) {
        const uint32_t w[4] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w};
        uint32_t o[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(y & 1 ? w[y / 2] >> 16 : w[y / 2] & 0xffffu));
          o[y] = floats_to_bf16x2(f.x * s[i], f.y * s[i]);
        }
        o0 = make_uint4(o[0], o[1], o[2], o[3]);
        o1 = make_uint4(o[4], o[5], o[6], o[7]);
      }
      uint4* dst = reinterpret_cast<uint4*>(p.out + (bh * p.n + t) * D) + gl * 2;
      __stcs(dst, o0);
      __stcs(dst + 1, o1);
    }
  }
}

}  // namespace tk
