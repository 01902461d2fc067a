// paged_attention.cuh -- attention of one new token per sequence over a paged
// key-value cache: o = sum_j p_j V_j, p = softmax(scale * q . K_j) over the
// sequence's cached tokens, or over the positions a selector listed.
//
// One pass over the cache: every warp keeps, for its keys, the running maximum
// m of the scores (in units of log2), l = sum 2^(s_j - m) and O = sum
// 2^(s_j - m) V_j; two such triples join as (max m, ...) with the factors
// 2^(m_a - m).  A key-value head is read once for all query heads that share
// it, eight or sixteen at a time: they are the columns of the matrix products
// S^T = K Q^T (16 keys x 8 heads) and O^T += V^T P^T (16 columns of V x 8
// heads), so that a head that shares its keys with none wastes seven eighths of
// the small operand, not of the large one.  16 flops per element of K and V and
// group of eight heads: 51 TFLOP/s of bf16 at full bandwidth.  The kernel is
// bound by reading K and V from HBM.
//
// Work: a unit is (sequence, list of query heads); its tokens are cut into
// granules of 4 * KT tokens, one tile of KT keys per warp.  All granules of
// all units form one line that the CTAs (two per SM) share evenly, whatever
// the lengths; a unit that lies in several CTAs' shares is joined by the CTA
// that finishes last (an atomic ticket, nobody waits; the parts are added in
// the order of the CTAs, so equal calls give equal bits).
//
// Each warp feeds itself: its lanes look up its tile's rows (a position, then
// a page, each a tile ahead of its use) and copy them by 16-byte cp.async into
// a ring of STAGES tiles of its own, so no barrier of the CTA stands in the
// loop and any page size, stride or list of positions costs the same.
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
  int row_tiles;      // groups of 16 query heads per list
  uint32_t page_magic, page_shift;  // t / page_size = (t * page_magic) >> page_shift for 0 <= t < 2^31
  bool grouped;       // no positions, and 16 | page_size: 16 tokens from a multiple of 16 on share a page
  bool same_strides;  // k and v have equal strides
  float scale_log2;   // softmax scale * log2(e)
  uint16_t* out;      // [batch][heads][d] bf16
  float* lse;         // null, or [batch][heads]
  uint32_t* tickets;  // [kAttendMaxCtas], zero between calls
  float* parts;       // [ctas][2][16 * (d + 2)]
};

constexpr int kAttendWarps = 4;
constexpr int kAttendThreads = 32 * kAttendWarps;
constexpr int kAttendMaxCtas = 1024;

__host__ __device__ constexpr int attend_part_floats(int d) { return 16 * (d + 2); }

template <int D, bool kE4m3, int NT>
struct AttendShape {
  static constexpr int kRowBytes = D * (kE4m3 ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kKeys = D == 256 ? 16 : (D == 128 && !kE4m3) ? 16 : 32;  // per warp tile
  static constexpr int kGranule = kAttendWarps * kKeys;
  static constexpr int kTileBytes = kKeys * kRowBytes;               // K or V
  static constexpr int kScaleBytes = kE4m3 ? 2 * kKeys * 4 : 0;
  static constexpr int kStageBytes = 2 * kTileBytes + kScaleBytes;
  static constexpr bool kQShared = D == 256 && NT == 2;  // Q fragments in shared memory (64 registers otherwise)
  // 8 KB a tile: three stages of four warps and two CTAs fill an SM's shared memory
  static constexpr int kCtasPerSm = D == 256 && (!kE4m3 || NT == 2) ? 1 : 2;
  static constexpr int kStages = D == 64 && kE4m3 ? 6 : D == 256 && kE4m3 && NT == 2 ? 5 : 3;
  static constexpr int kJoinFloats = 2304;
  // shared memory: [warps][stages] tiles, join buffer, Q fragments, (m, l) per warp and joined, valid masks, plan
  static constexpr int kOffJoin = kAttendWarps * kStages * kStageBytes;
  static constexpr int kOffQ = kOffJoin + kJoinFloats * 4;
  static constexpr int kOffMl = kOffQ + (kQShared ? 8192 : 0);
  static constexpr int kOffValid = kOffMl + (kAttendWarps + 1) * 32 * 4;
  static constexpr int kOffPlan = kOffValid + kAttendWarps * kStages * 4;
  static constexpr int kSmem = (kOffPlan + 64 + 127) / 128 * 128;
  static_assert(kOffPlan % 8 == 0, "plan alignment");
  // Columns of O joined at a time: 4 warps x rows x (columns + 4) floats fit
  // the buffer; the 4 spread a lane quad's heads over the banks.
  static __device__ __forceinline__ int join_columns(int rows) {
    return min(D, (kJoinFloats / (kAttendWarps * rows) - 4) & ~15);
  }
};

// ---------------------------------------------------------------- instructions
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  const int bytes = live ? 16 : 0;  // the rest of the 16 is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  const int bytes = live ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void load_matrices_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool kF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two 16x16 matrices of bytes, transposed: r[2 x] holds rows 4t .. 4t + 3 of
// column g of matrix x, r[2 x + 1] the same of column g + 8.
__device__ __forceinline__ void load_bytes_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Transposes an 8x8 matrix of 16-bit values held across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {  // 2^x, relative error below 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t floats_to_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Over the eight lanes of a column (those of equal lane % 4).
__device__ __forceinline__ float column_max(float x) {
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}
__device__ __forceinline__ float column_sum(float x) {
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
__device__ __forceinline__ float finite_or_zero(float m) { return m == __int_as_float(0xff800000) ? 0.0f : m; }

// ---------------------------------------------------------------- work line
// Where a CTA stands on the line of granules.
struct AttendCursor {
  int b, unit;   // sequence, unit of it (list and group of 16 heads)
  int at;        // granule within the unit
  int count;     // tokens or list slots of the unit
  int granules;  // of the unit
};

template <int kGranule>
__device__ __forceinline__ int granules_of(int count) {
  return static_cast<int>((static_cast<uint32_t>(count) + kGranule - 1) / kGranule);
}

template <int kGranule>
__device__ __forceinline__ void cursor_enter(const AttendArgs& p, AttendCursor& u) {
  u.count = p.positions ? p.c : seq_length(p.tab, u.b);
  u.granules = granules_of<kGranule>(u.count);
}

// To the next granule; past the last one `b` is tab.batch and nothing may be read.
template <int kGranule>
__device__ __forceinline__ void cursor_next(const AttendArgs& p, AttendCursor& u) {
  if (++u.at < u.granules) return;
  u.at = 0;
  if (++u.unit < p.lists * p.row_tiles) return;
  u.unit = 0;
  do {
    if (++u.b >= p.tab.batch) {
      u.granules = 0;
      u.count = 0;
      return;
    }
    cursor_enter<kGranule>(p, u);
  } while (u.granules == 0);
}

// ---------------------------------------------------------------- one warp's state
// A lane's place in the products: g = lane / 4, t = lane % 4.  Scores: rows g
// and g + 8 of each 16, heads 2t and 2t + 1 of each 8; O^T: columns g and g + 8
// of each 16 of V, the same heads.  Row r of a score tile is key_of(r): the
// order of summation over keys is free, and bytes of V come transposed four
// keys at a time, so that with the keys 4t, 4t + 1 in rows 2t, 2t + 1 and 4t + 2,
// 4t + 3 in rows 2t + 8, 2t + 9 each half of such a word is an operand pair.
template <int D, bool kE4m3, int NT>
struct AttendWarp {
  using S = AttendShape<D, kE4m3, NT>;
  static constexpr int kGroups = S::kKeys / 16;
  static constexpr int kSteps = D / 16;  // of the product over d
  static constexpr int kQWords = 2;      // registers of Q per step and 8 heads

  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
  float f[NT][2];  // e4m3: O holds sum w_j V8_j / f, with w_j = 2^(s_j - m) * vscale_j
  uint32_t q[NT][S::kQShared ? 1 : kSteps][kQWords];
  float head_scale[NT][2];  // score in log2 units per unit of the product

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][j][i] = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[n][h] = __int_as_float(0xff800000);
        l[n][h] = 0.0f;
        f[n][h] = 0.0f;
      }
    }
  }

  static __device__ __forceinline__ int key_of(int r) {
    return kE4m3 ? ((r & 6) << 1) + (r & 1) + ((r >> 2) & 2) : r;
  }

  // Fragments of the query heads (zeros behind `rows`).  Beside e4m3 keys the
  // products run in f16, which holds every code exactly: a head is scaled by
  // the power of two that brings its largest finite value into [2^14, 2^15),
  // where rounding to f16 moves a value by at most 2^-25 (below 2^-39 of that
  // largest one).  A lane's four codes of a key are the values 4t .. 4t + 3 of
  // 16, and so are its values of q.
  __device__ __forceinline__ void load_q(const AttendArgs& p, const uint16_t* q0, int rows, uint2* shared, int warp) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool live = n * 8 + g < rows;
      const uint16_t* row = q0 + static_cast<int64_t>(n * 8 + g) * D;
      float mul = 1.0f;
      head_scale[n][0] = head_scale[n][1] = p.scale_log2;
      if constexpr (kE4m3) {
        uint32_t top = 0;
#pragma unroll 4
        for (int ks = 0; ks < kSteps; ++ks) {
          const uint2 w = live ? __ldg(reinterpret_cast<const uint2*>(row + ks * 16) + t) : make_uint2(0, 0);
          const uint32_t h[4] = {w.x << 16, w.x, w.y << 16, w.y};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = h[i] & 0x7fff0000u;
            if (v < 0x7f800000u) top = max(top, v);
          }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float scale = p.scale_log2;
        if (top) {
          int e = 14 - (static_cast<int>(top >> 23) - 127);
          e = min(max(e, -126), 126);
          mul = power_of_two(e);
          scale = p.scale_log2 * power_of_two(-e);
        }
        head_scale[n][0] = __shfl_sync(0xffffffffu, scale, 8 * t);
        head_scale[n][1] = __shfl_sync(0xffffffffu, scale, 8 * t + 4);
      }
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        if (S::kQShared && ks % kAttendWarps != warp) continue;
        uint32_t b0 = 0, b1 = 0;
        if (live) {
          if constexpr (kE4m3) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + ks * 16) + t);
            b0 = floats_to_f16x2(__uint_as_float(w.x << 16) * mul, __uint_as_float(w.x & 0xffff0000u) * mul);
            b1 = floats_to_f16x2(__uint_as_float(w.y << 16) * mul, __uint_as_float(w.y & 0xffff0000u) * mul);
          } else {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(row + ks * 16);
            b0 = __ldg(src + t);
            b1 = __ldg(src + t + 4);
          }
        }
        if constexpr (S::kQShared) {
          shared[(ks * NT + n) * 32 + lane] = make_uint2(b0, b1);
        } else {
          q[n][ks][0] = b0;
          q[n][ks][1] = b1;
        }
      }
    }
  }

  __device__ __forceinline__ void fragment(uint32_t (&b)[kQWords], int n, int ks, const uint2* shared) const {
    if constexpr (S::kQShared) {
      const uint2 w = shared[(ks * NT + n) * 32 + (threadIdx.x & 31)];
      b[0] = w.x;
      b[1] = w.y;
    } else {
      b[0] = q[n][ks][0];
      b[1] = q[n][ks][1];
    }
  }

  // Address of 16-byte chunk c of row r in a tile: chunks are permuted within
  // 128-byte lines so that the eight rows of an 8x8 matrix use all banks, the
  // rows 0-7 and 8-15 as well as the rows key_of(0-7) and key_of(8-15).
  static __device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int r, int c) {
    if constexpr (S::kChunks == 4)
      return tile + r * 64 + ((c ^ (((r >> 1) & 2) | (((r >> 1) ^ (r >> 3)) & 1))) << 4);
    else
      return tile + r * S::kRowBytes + ((c ^ (r & 7) ^ ((r >> 2) & 2)) << 4);
  }

  // One tile: scores, softmax, and the products with V.
  __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, const float* scales, uint32_t valid,
                                       const uint2* shared_q) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const float ninf = __int_as_float(0xff800000);
    float s[NT][kGroups][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][k][i] = 0.0f;
    constexpr int kStepsPerLoad = kE4m3 ? 2 : 1;
#pragma unroll
    for (int ks = 0; ks < kSteps; ks += kStepsPerLoad) {
      uint32_t b[kStepsPerLoad][NT][kQWords];
#pragma unroll
      for (int x = 0; x < kStepsPerLoad; ++x)
#pragma unroll
        for (int n = 0; n < NT; ++n) fragment(b[x][n], n, ks + x, shared_q);
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        uint32_t r[4];
        load_matrices(r, chunk_at(kt, k * 16 + key_of(lane & 15), (kE4m3 ? ks : 2 * ks) + (lane >> 4)));
#pragma unroll
        for (int x = 0; x < kStepsPerLoad; ++x) {
          if constexpr (kE4m3) {
            const uint32_t a[4] = {e4m3x2_to_f16x2(r[2 * x] & 0xffffu), e4m3x2_to_f16x2(r[2 * x + 1] & 0xffffu),
                                   e4m3x2_to_f16x2(r[2 * x] >> 16), e4m3x2_to_f16x2(r[2 * x + 1] >> 16)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<true>(s[n][k], a, b[x][n][0], b[x][n][1]);
          } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<false>(s[n][k], r, b[x][n][0], b[x][n][1]);
          }
        }
      }
    }
    // scores in log2 units; keys left out become -inf
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float ks = 1.0f;
        if constexpr (kE4m3) ks = scales[k * 16 + key_of(g + 8 * y)];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& x = s[n][k][2 * y + h];
            if constexpr (kE4m3)
              x *= ks * head_scale[n][h];
            else
              x *= head_scale[n][h];
          }
      }
    if (valid != (S::kKeys == 32 ? 0xffffffffu : (1u << (S::kKeys & 31)) - 1u)) {
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (!((valid >> (k * 16 + key_of(g + 8 * y))) & 1u))
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][k][2 * y] = s[n][k][2 * y + 1] = ninf;
    }
    // The reference m moves only when a score passes it by 2^8: weights up to
    // 256 are harmless in fp32 sums, and most tiles need neither a maximum
    // across lanes nor a rescaling.
    float top[NT][2];
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[n][h] = ninf;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) top[n][h] = fmaxf(top[n][h], fmaxf(s[n][k][h], s[n][k][2 + h]));
        raise |= top[n][h] > m[n][h] + 8.0f;
      }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = fmaxf(m[n][h], column_max(top[n][h]));
          const float x = exp2_fast(m[n][h] - finite_or_zero(mn));
          m[n][h] = mn;
          l[n][h] *= x;
          if constexpr (kE4m3) {
            f[n][h] *= x;
          } else {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[n][j][h] *= x;
              o[n][j][2 + h] *= x;
            }
          }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ref = finite_or_zero(m[n][h]);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          s[n][k][h] = exp2_fast(s[n][k][h] - ref);
          s[n][k][2 + h] = exp2_fast(s[n][k][2 + h] - ref);
          l[n][h] += s[n][k][h] + s[n][k][2 + h];
        }
      }
    if constexpr (kE4m3) {
      // w_j = p_j * vscale_j, held in f16 relative to f: f follows the largest
      // w of the head, so the weights that carry the sum keep 11 bits whatever
      // the scales are.
      float wt[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) wt[n][0] = wt[n][1] = 0.0f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float vs = scales[S::kKeys + k * 16 + key_of(g + 8 * y)];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              s[n][k][2 * y + h] *= vs;
              wt[n][h] = fmaxf(wt[n][h], fabsf(s[n][k][2 * y + h]));
            }
        }
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) grow |= wt[n][h] > f[n][h] * 256.0f;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float fn = fmaxf(f[n][h], fminf(column_max(wt[n][h]), 1e36f));
            const float x = fn > 0.0f ? f[n][h] / fn : 0.0f;
            f[n][h] = fn;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[n][j][h] *= x;
              o[n][j][2 + h] *= x;
            }
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float inv = f[n][h] >= 1.2e-38f ? 1.0f / f[n][h] : 0.0f;  // weights below 2^-126 count as nothing
#pragma unroll
          for (int k = 0; k < kGroups; ++k) {
            s[n][k][h] *= inv;
            s[n][k][2 + h] *= inv;
          }
        }
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      // P^T as the right operand.  Beside bf16 values P is split into two bf16
      // parts (the second takes what rounding the first left), which keeps 16
      // bits of every weight.
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float a = s[n][k][2 * y], b = s[n][k][2 * y + 1];
          if constexpr (kE4m3) {
            hi[n][y] = transpose8x8(floats_to_f16x2(a, b));
          } else {
            const uint32_t h = floats_to_bf16x2(a, b);
            hi[n][y] = transpose8x8(h);
            lo[n][y] = transpose8x8(
                floats_to_bf16x2(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xffff0000u)));
          }
        }
      if constexpr (kE4m3) {
#pragma unroll
        for (int c = 0; c < S::kChunks; c += 2) {
          uint32_t r[4];
          load_bytes_t(r, chunk_at(vt, k * 16 + (lane & 15), c + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a[4] = {e4m3x2_to_f16x2(r[2 * x] & 0xffffu), e4m3x2_to_f16x2(r[2 * x + 1] & 0xffffu),
                                   e4m3x2_to_f16x2(r[2 * x] >> 16), e4m3x2_to_f16x2(r[2 * x + 1] >> 16)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<true>(o[n][c + x], a, hi[n][0], hi[n][1]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          uint32_t a[4];
          load_matrices_t(a, chunk_at(vt, k * 16 + (lane & 7) + (lane >> 4) * 8, 2 * j + ((lane >> 3) & 1)));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816<false>(o[n][j], a, hi[n][0], hi[n][1]);
            mma16816<false>(o[n][j], a, lo[n][0], lo[n][1]);
          }
        }
      }
    }
  }

  // Column of o[.][j][i] for a lane with lane / 4 = g.
  static __device__ __forceinline__ int column(int j, int i, int g) { return 16 * j + g + 8 * (i >> 1); }
};

// ---------------------------------------------------------------- joining
// Joins the parts of a unit that lies in CTAs first .. last (in that order)
// and writes its rows.  All threads of the CTA.
template <int D>
__device__ void attend_join(const AttendArgs& p, int first, int last, int rows, int64_t out_row, float* buf) {
  constexpr int V = D / 32;  // columns per lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_row = rows == 1 ? 4 : rows == 2 ? 2 : 1;  // warps that share a row's parts
  const float ninf = __int_as_float(0xff800000);
  const int n = last - first + 1;
  for (int base = 0; base < rows; base += kAttendWarps / per_row) {
    const int row = base + warp / per_row, sub = warp % per_row;
    float acc[V], total = 0.0f, mm = ninf;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    if (row < rows) {
      for (int i = lane; i < n; i += 32)
        mm = fmaxf(mm, __ldcg(p.parts + static_cast<int64_t>((first + i) * 2 + (i == 0)) * attend_part_floats(D) + row));
#pragma unroll
      for (int x = 16; x; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
      const float ref = finite_or_zero(mm);
      for (int i0 = sub * 32; i0 < n; i0 += per_row * 32) {
        const int i = i0 + lane;
        float w = 0.0f;
        if (i < n) {
          const float* part = p.parts + static_cast<int64_t>((first + i) * 2 + (i == 0)) * attend_part_floats(D);
          w = exp2_fast(__ldcg(part + row) - ref);
          total += w * __ldcg(part + 16 + row);
        }
        const int m = min(32, n - i0);
#pragma unroll 8
        for (int x = 0; x < m; ++x) {
          const float wx = __shfl_sync(0xffffffffu, w, x);
          const float* src = p.parts +
                             static_cast<int64_t>((first + i0 + x) * 2 + (i0 + x == 0)) * attend_part_floats(D) + 32 +
                             row * D + lane * V;
          if constexpr (V == 2) {
            const float2 a = __ldcg(reinterpret_cast<const float2*>(src));
            acc[0] += wx * a.x;
            acc[1] += wx * a.y;
          } else {
#pragma unroll
            for (int y = 0; y < V; y += 4) {
              const float4 a = __ldcg(reinterpret_cast<const float4*>(src + y));
              acc[y] += wx * a.x;
              acc[y + 1] += wx * a.y;
              acc[y + 2] += wx * a.z;
              acc[y + 3] += wx * a.w;
            }
          }
        }
      }
#pragma unroll
      for (int x = 16; x; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
    }
    if (per_row > 1) {  // the row's warps meet in shared memory, added in warp order
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) buf[warp * D + lane * V + i] = acc[i];
      if (lane == 0) buf[4 * D + warp] = total;
      __syncthreads();
      if (sub == 0)
        for (int w = 1; w < per_row; ++w) {
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] += buf[(warp + w) * D + lane * V + i];
          total += buf[4 * D + warp + w];
        }
    }
    if (row < rows && sub == 0) {
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (out_row + row) * D + lane * V);
#pragma unroll
      for (int i = 0; i < V; i += 2) dst[i / 2] = floats_to_bf16x2(acc[i] * inv, acc[i + 1] * inv);
      if (p.lse && lane == 0) p.lse[out_row + row] = 0.6931471805599453f * (mm + log2f(total));
    }
  }
}

// ---------------------------------------------------------------- kernel
template <int D, bool kE4m3, int NT>
__global__ void __launch_bounds__(kAttendThreads, (AttendShape<D, kE4m3, NT>::kCtasPerSm))
    paged_attention_kernel(AttendArgs p) {
  using S = AttendShape<D, kE4m3, NT>;
  using W = AttendWarp<D, kE4m3, NT>;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* join = reinterpret_cast<float*>(smem + S::kOffJoin);
  uint2* shared_q = reinterpret_cast<uint2*>(smem + S::kOffQ);
  float* ml = reinterpret_cast<float*>(smem + S::kOffMl);  // [warp][m of 16 rows, l of 16 rows]
  uint32_t* valid_masks = reinterpret_cast<uint32_t*>(smem + S::kOffValid) + warp * S::kStages;
  int64_t* plan = reinterpret_cast<int64_t*>(smem + S::kOffPlan);
  unsigned char* ring = smem + warp * S::kStages * S::kStageBytes;
  const uint32_t ring_addr = smem_addr(ring);
  pdl_wait_then_release();

  const int units = p.lists * p.row_tiles;
  const int group = p.heads / p.lists;
  // Sequences without a token have no granule: their rows are written here.
  if (!p.positions) {
    for (int b = blockIdx.x; b < p.tab.batch; b += gridDim.x) {
      if (seq_length(p.tab, b) != 0) continue;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + static_cast<int64_t>(b) * p.heads * D);
      for (int i = tid; i < p.heads * D / 2; i += kAttendThreads) dst[i] = 0;
      if (p.lse)
        for (int i = tid; i < p.heads; i += kAttendThreads)
          p.lse[static_cast<int64_t>(b) * p.heads + i] = __int_as_float(0xff800000);
    }
  }
  // This CTA's share [g0, g1) of the line, and where it begins.
  // No share is empty: shares are given to as many CTAs as there are granules.
  int64_t total, g0, g1;
  int ctas;
  AttendCursor cur;
  auto share = [&]() {
    ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total));
    g0 = part_start(total, max(ctas, 1), min(static_cast<int>(blockIdx.x), ctas), 1, total);
    g1 = part_start(total, max(ctas, 1), min(static_cast<int>(blockIdx.x) + 1, ctas), 1, total);
  };
  if (p.positions) {
    cur.b = 0;
    cursor_enter<S::kGranule>(p, cur);
    total = static_cast<int64_t>(p.tab.batch) * units * cur.granules;
    share();
    const int64_t u = g0 / cur.granules;
    cur.b = static_cast<int>(u / units);
    cur.unit = static_cast<int>(u - static_cast<int64_t>(cur.b) * units);
    cur.at = static_cast<int>(g0 - u * cur.granules);
  } else {
    // Running sums of the sequences' granules: a stretch of sequences per thread.
    const int per = (p.tab.batch + kAttendThreads - 1) / kAttendThreads;
    const int b0 = min(tid * per, p.tab.batch), b1 = min(b0 + per, p.tab.batch);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += granules_of<S::kGranule>(seq_length(p.tab, b));
    int64_t upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, x);
      if (lane >= x) upto += y;
    }
    if (lane == 31) plan[warp] = upto;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kAttendWarps; ++w) {
      if (w < warp) upto += plan[w];
      total += plan[w];
    }
    total *= units;
    share();
    int64_t before = (upto - mine) * units;
    if (g0 < g1 && g0 >= before && g0 < upto * units) {
      int b = b0;
      int64_t n = granules_of<S::kGranule>(seq_length(p.tab, b));
      while (g0 >= before + n * units) {
        before += n * units;
        n = granules_of<S::kGranule>(seq_length(p.tab, ++b));
      }
      plan[4] = b;
      plan[5] = g0 - before;
    }
    __syncthreads();
    if (g0 < g1) {
      cur.b = static_cast<int>(plan[4]);
      cursor_enter<S::kGranule>(p, cur);
      cur.unit = static_cast<int>(plan[5] / cur.granules);
      cur.at = static_cast<int>(plan[5] - static_cast<int64_t>(cur.unit) * cur.granules);
    }
  }
  if (g0 >= g1) return;

  // The three steps of a tile's rows, each a tile behind the one before: the
  // lane's token, its page, the copies.  A lane of index < kKeys has a key.
  AttendCursor ahead = cur;
  int64_t ahead_left = g1 - g0;
  int tok = -1, tok_b = 0, tok_kv = 0, tok_len = 0;
  int32_t page = -1;
  int off = 0, page_kv = 0;
  const int kv_per = p.lists / p.k.kv_heads;
  auto next_token = [&]() {
    tok = -1;
    if (ahead_left > 0) {
      const uint32_t i = (static_cast<uint32_t>(ahead.at) * kAttendWarps + warp) * S::kKeys + lane;
      const int list = ahead.unit / p.row_tiles;
      tok_b = ahead.b;
      tok_kv = list / kv_per;
      tok_len = p.positions ? seq_length(p.tab, ahead.b) : ahead.count;
      if (lane < S::kKeys && i < static_cast<uint32_t>(ahead.count))
        tok = p.positions ? __ldg(p.positions + (static_cast<int64_t>(ahead.b) * p.lists + list) * p.c + i) : static_cast<int>(i);
      --ahead_left;
      cursor_next<S::kGranule>(p, ahead);
    }
  };
  auto next_page = [&]() {
    page = -1;
    page_kv = tok_kv;
    if (tok >= 0) {
      if (tok < tok_len) {
        const int at = static_cast<int>((static_cast<uint64_t>(tok) * p.page_magic) >> p.page_shift);
        off = tok - at * p.k.page_size;
        page = __ldg(p.tab.table + tok_b * p.tab.stride + at);
        if (page < 0 || page >= p.k.pages) {
          atomicOr(&g_device_status, kDevBadIndex);
          page = -1;
        }
      } else if (tok >= p.tab.capacity) {
        atomicOr(&g_device_status, kDevBadIndex);
      }
    }
  };
  auto issue = [&](int stage) {
    const bool live = page >= 0;
    const uint32_t valid = __ballot_sync(0xffffffffu, live);
    const int64_t pg = live ? page : 0;
    const int o = live ? off : 0;
    const int64_t ko = pg * p.k.page_stride + page_kv * p.k.head_stride + o * p.k.token_stride;
    int64_t vo = ko;
    if (!p.same_strides) vo = pg * p.v.page_stride + page_kv * p.v.head_stride + o * p.v.token_stride;
    const uint32_t kt = ring_addr + stage * S::kStageBytes, vt = kt + S::kTileBytes;
    if (lane == 0) valid_masks[stage] = valid;
    if (valid) {
      constexpr int kRowsPerCopy = 32 / S::kChunks;
      const int c = lane % S::kChunks, r0 = lane / S::kChunks;
      if (p.grouped && p.same_strides) {  // one address for 16 rows of K and of V
#pragma unroll
        for (int y = 0; y < S::kKeys / 16; ++y) {
          int64_t a = __shfl_sync(0xffffffffu, ko, y * 16) + r0 * p.k.token_stride + c * 16;
#pragma unroll
          for (int i = 0; i < 16 / kRowsPerCopy; ++i) {
            const int r = y * 16 + i * kRowsPerCopy + r0;
            const bool on = (valid >> r) & 1u;
            copy16(W::chunk_at(kt, r, c), p.k.data + a, on);
            copy16(W::chunk_at(vt, r, c), p.v.data + a, on);
            a += kRowsPerCopy * p.k.token_stride;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < S::kKeys / kRowsPerCopy; ++i) {
          const int r = i * kRowsPerCopy + r0;
          const int64_t a = __shfl_sync(0xffffffffu, ko, r) + c * 16;
          const bool on = (valid >> r) & 1u;
          copy16(W::chunk_at(kt, r, c), p.k.data + a, on);
          const int64_t b = p.same_strides ? a : __shfl_sync(0xffffffffu, vo, r) + c * 16;
          copy16(W::chunk_at(vt, r, c), p.v.data + b, on);
        }
      }
      if constexpr (kE4m3) {
        if (lane < S::kKeys) {
          const uint32_t st = vt + S::kTileBytes + lane * 4;
          copy4(st, p.k.scale + (pg * p.k.s_page_stride + page_kv * p.k.s_head_stride + o * p.k.s_token_stride), live);
          copy4(st + S::kKeys * 4,
                p.v.scale + (pg * p.v.s_page_stride + page_kv * p.v.s_head_stride + o * p.v.s_token_stride), live);
        }
      }
    }
    copy_commit();
  };

  next_token();
  next_page();
  next_token();
#pragma unroll 1
  for (int i = 0; i < S::kStages - 1; ++i) {
    issue(i);
    next_page();
    next_token();
  }

  W w;
  w.reset();
  bool fresh = true;
  int stage = 0;
#pragma unroll 1
  for (int64_t g = g0; g < g1; ++g) {
    const int list = cur.unit / p.row_tiles, mt = cur.unit - list * p.row_tiles;
    const int rows = min(16, group - mt * 16);
    const int head = list * group + mt * 16;
    if (fresh) {
      if constexpr (S::kQShared) __syncthreads();
      w.load_q(p, p.q + cur.b * p.q_stride + static_cast<int64_t>(head) * D, rows, shared_q, warp);
      if constexpr (S::kQShared) __syncthreads();
      fresh = false;
    }
    copy_wait<S::kStages - 2>();
    __syncwarp();
    {  // the stage consumed last is free again
      const int s = stage == 0 ? S::kStages - 1 : stage - 1;
      issue(s);
      next_page();
      next_token();
    }
    const uint32_t valid = valid_masks[stage];
    if (valid) {
      const uint32_t kt = ring_addr + stage * S::kStageBytes;
      w.tile(kt, kt + S::kTileBytes,
             reinterpret_cast<const float*>(ring + stage * S::kStageBytes + 2 * S::kTileBytes), valid, shared_q);
    }
    stage = stage == S::kStages - 1 ? 0 : stage + 1;
    if (cur.at + 1 < cur.granules && g + 1 < g1) {
      ++cur.at;
      continue;
    }

    // The unit ends here, or this CTA's share of it: join the four warps.
    const int64_t unit_first = g - cur.at;
    const bool whole = unit_first >= g0 && cur.at + 1 == cur.granules;
    const int t = lane & 3, lane_g = lane >> 2;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float sum = column_sum(w.l[n][h]);
        if (lane_g == 0) {
          ml[warp * 32 + n * 8 + 2 * t + h] = w.m[n][h];
          ml[warp * 32 + 16 + n * 8 + 2 * t + h] = sum;
        }
      }
    __syncthreads();
    float factor[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mm = w.m[n][h];
#pragma unroll
        for (int x = 0; x < kAttendWarps; ++x) mm = fmaxf(mm, ml[x * 32 + n * 8 + 2 * t + h]);
        factor[n][h] = exp2_fast(w.m[n][h] - finite_or_zero(mm));
        if constexpr (kE4m3) factor[n][h] *= w.f[n][h];
      }
    float* part = p.parts + static_cast<int64_t>(blockIdx.x * 2 + (unit_first >= g0)) * attend_part_floats(D);
    const int64_t out_row = static_cast<int64_t>(cur.b) * p.heads + head;
    float* inverse = ml + kAttendWarps * 32;  // 1 / l of every row, for rows that end here
    if (tid < rows) {
      float mm = __int_as_float(0xff800000), sum = 0.0f;
#pragma unroll
      for (int x = 0; x < kAttendWarps; ++x) mm = fmaxf(mm, ml[x * 32 + tid]);
#pragma unroll
      for (int x = 0; x < kAttendWarps; ++x) sum += ml[x * 32 + 16 + tid] * exp2_fast(ml[x * 32 + tid] - finite_or_zero(mm));
      inverse[tid] = sum == 0.0f ? 0.0f : 1.0f / sum;
      if (!whole) {
        part[tid] = mm;
        part[16 + tid] = sum;
      } else if (p.lse) {
        p.lse[out_row + tid] = 0.6931471805599453f * (mm + log2f(sum));
      }
    }
    const int columns = S::join_columns(rows), pitch = columns + 4;
    for (int c0 = 0; c0 < D; c0 += columns) {
      if (c0) __syncthreads();
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        if (j * 16 < c0 || j * 16 >= c0 + columns) continue;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int head_row = n * 8 + 2 * t + (i & 1);
            if (head_row < rows)
              join[(warp * rows + head_row) * pitch + W::column(j, i, lane_g) - c0] = w.o[n][j][i] * factor[n][i & 1];
          }
      }
      __syncthreads();
      const int pairs = min(columns, D - c0) / 2;
      for (int i = tid; i < rows * pairs; i += kAttendThreads) {
        const int y = i / pairs, c = (i - y * pairs) * 2;
        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int x = 0; x < kAttendWarps; ++x) {  // in warp order
          const float2 u = *reinterpret_cast<const float2*>(join + (x * rows + y) * pitch + c);
          v.x += u.x;
          v.y += u.y;
        }
        if (whole)
          *reinterpret_cast<uint32_t*>(p.out + (out_row + y) * D + c0 + c) =
              floats_to_bf16x2(v.x * inverse[y], v.y * inverse[y]);
        else
          *reinterpret_cast<float2*>(part + 32 + y * D + c0 + c) = v;
      }
    }
    if (!whole) {
      const int first = part_of(unit_first, total, ctas, 1);
      const int last = part_of(unit_first + cur.granules - 1, total, ctas, 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t n = static_cast<uint32_t>(last - first);
        const bool done = atomicAdd(p.tickets + first, 1u) == n;
        if (done) p.tickets[first] = 0;
        plan[6] = done;
      }
      __syncthreads();
      if (plan[6]) {
        __threadfence();
        attend_join<D>(p, first, last, rows, out_row, join);
      }
    }
    __syncthreads();
    w.reset();
    fresh = true;
    cursor_next<S::kGranule>(p, cur);
  }
  copy_wait<0>();
}

}  // namespace tk
