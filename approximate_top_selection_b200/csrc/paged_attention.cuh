// paged_attention.cuh -- attention of one new token per sequence over a paged
// key-value cache: o = sum_j p_j V_j, p = softmax(scale * q . K_j) over the
// sequence's cached tokens, or over the positions a selector listed.
//
// One pass over the cache: every warp keeps, for its keys, the running maximum
// m of the scores (in units of log2), l = sum 2^(s_j - m) and O = sum
// 2^(s_j - m) V_j; two such triples join as (max m, ...) with the factors
// 2^(m_a - m).  A key-value head is read once for all query heads that share
// it: up to 16 of them are the 16 rows of m16n8k16 matrix products (S = Q K^T,
// O += P V), so the work per cached byte stays far below the memory's pace:
// 4 * 16 flops per element of K and V, about 100 TFLOP/s at full bandwidth.
// The kernel is bound by reading K and V from HBM.
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

template <int D, bool kE4m3>
struct AttendShape {
  static constexpr int kRowBytes = D * (kE4m3 ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kKeys = D == 256 ? 16 : (D == 128 && !kE4m3) ? 16 : 32;  // per warp tile
  static constexpr int kGranule = kAttendWarps * kKeys;
  static constexpr int kTileBytes = kKeys * kRowBytes;               // K or V
  static constexpr int kScaleBytes = kE4m3 ? 2 * kKeys * 4 : 0;
  static constexpr int kStageBytes = 2 * kTileBytes + kScaleBytes;
  static constexpr int kStages = D == 64 && kE4m3 ? 6 : 3;
  static constexpr int kCtasPerSm = D == 256 && !kE4m3 ? 1 : 2;
  static constexpr bool kQShared = D == 256;  // Q fragments in shared memory (64 registers otherwise)
  static constexpr int kJoinCols = D == 128 ? 128 : 64;
  static constexpr int kJoinPitch = kJoinCols + 8;  // floats; spreads a column's rows over the banks
  // shared memory: [warps][stages] tiles, join buffer, Q fragments, (m, l) per warp and joined, valid masks, plan
  static constexpr int kOffJoin = kAttendWarps * kStages * kStageBytes;
  static constexpr int kOffQ = kOffJoin + 16 * kJoinPitch * 4;
  static constexpr int kOffMl = kOffQ + (kQShared ? D / 16 * 512 : 0);
  static constexpr int kOffValid = kOffMl + (kAttendWarps + 1) * 32 * 4;
  static constexpr int kOffPlan = kOffValid + kAttendWarps * kStages * 4;
  static constexpr int kSmem = (kOffPlan + 64 + 127) / 128 * 128;
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
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
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

template <int D, bool kE4m3>
__device__ __forceinline__ void cursor_enter(const AttendArgs& p, AttendCursor& u) {
  u.count = p.positions ? p.c : seq_length(p.tab, u.b);
  u.granules = granules_of<AttendShape<D, kE4m3>::kGranule>(u.count);
}

// To the next granule; past the last one `b` is tab.batch and nothing may be read.
template <int D, bool kE4m3>
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
    cursor_enter<D, kE4m3>(p, u);
  } while (u.granules == 0);
}

// ---------------------------------------------------------------- one warp's state
template <int D, bool kE4m3, bool kFull>
struct AttendWarp {
  using S = AttendShape<D, kE4m3>;
  static constexpr int kTiles = S::kKeys / 8;  // score tiles of 8 keys
  static constexpr int kRows = kFull ? 2 : 1;  // rows g and g + 8 of a lane

  float o[D / 8][4];
  float m[2], l[2];
  float f[2];        // e4m3: O holds sum w_j V8_j / f, with w_j = 2^(s_j - m) * vscale_j
  uint32_t q[S::kQShared ? 1 : D / 16][4];
  float row_scale[2];  // score in log2 units per unit of the product

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      m[r] = __int_as_float(0xff800000);
      l[r] = 0.0f;
      f[r] = 0.0f;
    }
  }

  // Fragments of the 16 query rows (zeros behind `rows`).  Beside e4m3 keys
  // the products run in f16: a row is scaled by the power of two that brings
  // its largest finite value into [2^14, 2^15), where rounding to f16 moves a
  // value by at most 2^-25 (below 2^-39 of that largest one).
  __device__ __forceinline__ void load_q(const AttendArgs& p, const uint16_t* q0, int rows, uint4* shared, int warp) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float mul[2] = {1.0f, 1.0f};
    row_scale[0] = row_scale[1] = p.scale_log2;
    if constexpr (kE4m3) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        uint32_t top = 0;
        if (g + 8 * r < rows) {
          const uint2* src = reinterpret_cast<const uint2*>(q0 + static_cast<int64_t>(g + 8 * r) * D) + t;
#pragma unroll 4
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint2 w = __ldg(src + ks * 4);
            const uint32_t h[4] = {w.x << 16, w.x, w.y << 16, w.y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t v = h[i] & 0x7fff0000u;
              if (v < 0x7f800000u) top = max(top, v);
            }
          }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (top) {
          int e = 14 - (static_cast<int>(top >> 23) - 127);
          e = min(max(e, -126), 126);
          mul[r] = power_of_two(e);
          row_scale[r] = p.scale_log2 * power_of_two(-e);
        }
      }
    }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      if (S::kQShared && ks % kAttendWarps != warp) continue;
      uint32_t a[4] = {0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (g + 8 * r < rows) {
          const uint16_t* row = q0 + static_cast<int64_t>(g + 8 * r) * D + ks * 16;
          if constexpr (kE4m3) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(row) + t);
            a[r] = floats_to_f16x2(__uint_as_float(w.x << 16) * mul[r], __uint_as_float(w.x & 0xffff0000u) * mul[r]);
            a[2 + r] = floats_to_f16x2(__uint_as_float(w.y << 16) * mul[r], __uint_as_float(w.y & 0xffff0000u) * mul[r]);
          } else {
            a[r] = __ldg(reinterpret_cast<const uint32_t*>(row) + t);
            a[2 + r] = __ldg(reinterpret_cast<const uint32_t*>(row) + t + 4);
          }
        }
      }
      if constexpr (S::kQShared) {
        shared[ks * 32 + lane] = make_uint4(a[0], a[1], a[2], a[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[ks][i] = a[i];
      }
    }
  }

  // Address of 16-byte chunk c of row r in a tile: chunks are permuted within
  // 128-byte lines so that the eight rows of an 8x8 matrix use all banks.
  static __device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int r, int c) {
    if constexpr (S::kChunks == 4)
      return tile + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    else
      return tile + r * S::kRowBytes + ((c ^ (r & 7)) << 4);
  }

  // One tile: scores, softmax, and the products with V.
  __device__ __forceinline__ void tile(const AttendArgs& p, uint32_t kt, uint32_t vt, const float* scales, uint32_t valid,
                                       const uint4* shared_q) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    const float ninf = __int_as_float(0xff800000);
    float s[kTiles][4];
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.0f;
    constexpr int kStepsPerLoad = kE4m3 ? 4 : 2;
#pragma unroll
    for (int j = 0; j < S::kChunks / 4; ++j) {
      uint32_t a[kStepsPerLoad][4];
#pragma unroll
      for (int i = 0; i < kStepsPerLoad; ++i) {
        if constexpr (S::kQShared) {
          const uint4 w = shared_q[(j * kStepsPerLoad + i) * 32 + lane];
          a[i][0] = w.x;
          a[i][1] = w.y;
          a[i][2] = w.z;
          a[i][3] = w.w;
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) a[i][x] = q[j * kStepsPerLoad + i][x];
        }
      }
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        uint32_t b[4];
        load_matrices(b, chunk_at(kt, n * 8 + (lane & 7), j * 4 + (lane >> 3)));
        if constexpr (kE4m3) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma16816<true>(s[n], a[i], e4m3x2_to_f16x2(b[i] & 0xffffu), e4m3x2_to_f16x2(b[i] >> 16));
        } else {
          mma16816<false>(s[n], a[0], b[0], b[1]);
          mma16816<false>(s[n], a[1], b[2], b[3]);
        }
      }
    }
    // scores in log2 units; keys left out become -inf
    float top[2] = {ninf, ninf};
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      float2 ks = make_float2(1.0f, 1.0f);
      if constexpr (kE4m3) ks = *reinterpret_cast<const float2*>(scales + n * 8 + 2 * t);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if constexpr (kE4m3) {
          s[n][2 * r] *= ks.x;
          s[n][2 * r + 1] *= ks.y;
        }
        s[n][2 * r] *= row_scale[r];
        s[n][2 * r + 1] *= row_scale[r];
      }
    }
    if (valid != (S::kKeys == 32 ? 0xffffffffu : (1u << (S::kKeys & 31)) - 1u)) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (!((valid >> (n * 8 + 2 * t + i)) & 1u)) s[n][i] = s[n][2 + i] = ninf;
    }
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int r = 0; r < kRows; ++r) top[r] = fmaxf(top[r], fmaxf(s[n][2 * r], s[n][2 * r + 1]));
#pragma unroll
    for (int r = 0; r < kRows; ++r) top[r] = quad_max(top[r]);
    // The reference m moves only when a score passes it by 2^8: weights up to
    // 256 are harmless in fp32 sums, and most tiles need no rescaling.
    bool raise = top[0] > m[0] + 8.0f;
    if constexpr (kFull) raise |= top[1] > m[1] + 8.0f;
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float mn = fmaxf(m[r], top[r]);
        const float x = exp2_fast(m[r] - finite_or_zero(mn));
        m[r] = mn;
        l[r] *= x;
        if constexpr (kE4m3) {
          f[r] *= x;
        } else {
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[j][2 * r] *= x;
            o[j][2 * r + 1] *= x;
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float ref = finite_or_zero(m[r]);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        s[n][2 * r] = exp2_fast(s[n][2 * r] - ref);
        s[n][2 * r + 1] = exp2_fast(s[n][2 * r + 1] - ref);
        l[r] += s[n][2 * r] + s[n][2 * r + 1];
      }
    }
    if constexpr (kE4m3) {
      // w_j = p_j * vscale_j, held in f16 relative to f: f follows the largest
      // w of the row, so the weights that carry the sum keep 11 bits whatever
      // the scales are.
      float wt[2] = {0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        const float2 vs = *reinterpret_cast<const float2*>(scales + S::kKeys + n * 8 + 2 * t);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          s[n][2 * r] *= vs.x;
          s[n][2 * r + 1] *= vs.y;
          wt[r] = fmaxf(wt[r], fmaxf(fabsf(s[n][2 * r]), fabsf(s[n][2 * r + 1])));
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) wt[r] = fminf(quad_max(wt[r]), 1e36f);
      bool grow = wt[0] > f[0] * 256.0f;
      if constexpr (kFull) grow |= wt[1] > f[1] * 256.0f;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float fn = fmaxf(f[r], wt[r]);
          const float x = fn > 0.0f ? f[r] / fn : 0.0f;
          f[r] = fn;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[j][2 * r] *= x;
            o[j][2 * r + 1] *= x;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float inv = f[r] >= 1.2e-38f ? 1.0f / f[r] : 0.0f;  // weights below 2^-126 count as nothing
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          s[n][2 * r] *= inv;
          s[n][2 * r + 1] *= inv;
        }
      }
    }
#pragma unroll
    for (int kk = 0; kk < S::kKeys / 16; ++kk) {
      // P as the left operand: its C layout is the A layout of 16 keys.  Beside
      // bf16 values P is split into two bf16 parts (the second takes what
      // rounding the first left), which keeps 16 bits of every weight.
      uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float a = s[2 * kk + x][2 * r], b = s[2 * kk + x][2 * r + 1];
          if constexpr (kE4m3) {
            hi[2 * x + r] = floats_to_f16x2(a, b);
          } else {
            const uint32_t h = floats_to_bf16x2(a, b);
            hi[2 * x + r] = h;
            lo[2 * x + r] = floats_to_bf16x2(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xffff0000u));
          }
        }
#pragma unroll
      for (int c = 0; c < S::kChunks; c += 2) {
        uint32_t b[4];
        load_matrices_t(b, chunk_at(vt, kk * 16 + (lane & 15), c + (lane >> 4)));
        if constexpr (kE4m3) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {  // chunk c + x: even columns, then odd ones
            mma16816<true>(o[2 * (c + x)], hi, e4m3x2_to_f16x2(__byte_perm(b[2 * x], 0, 0x4420)),
                           e4m3x2_to_f16x2(__byte_perm(b[2 * x + 1], 0, 0x4420)));
            mma16816<true>(o[2 * (c + x) + 1], hi, e4m3x2_to_f16x2(__byte_perm(b[2 * x], 0, 0x4431)),
                           e4m3x2_to_f16x2(__byte_perm(b[2 * x + 1], 0, 0x4431)));
          }
        } else {
          mma16816<false>(o[c], hi, b[0], b[1]);
          mma16816<false>(o[c + 1], hi, b[2], b[3]);
          mma16816<false>(o[c], lo, b[0], b[1]);
          mma16816<false>(o[c + 1], lo, b[2], b[3]);
        }
      }
    }
  }

  // Column of o[j][i] (i = 0, 1) for a lane with lane % 4 = t.
  static __device__ __forceinline__ int column(int j, int i, int t) {
    return kE4m3 ? (j >> 1) * 16 + 4 * t + 2 * i + (j & 1) : 8 * j + 2 * t + i;
  }
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
template <int D, bool kE4m3, bool kFull>
__global__ void __launch_bounds__(kAttendThreads, AttendShape<D, kE4m3>::kCtasPerSm)
    paged_attention_kernel(AttendArgs p) {
  using S = AttendShape<D, kE4m3>;
  using W = AttendWarp<D, kE4m3, kFull>;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* join = reinterpret_cast<float*>(smem + S::kOffJoin);
  uint4* shared_q = reinterpret_cast<uint4*>(smem + S::kOffQ);
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
    cursor_enter<D, kE4m3>(p, cur);
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
      cursor_enter<D, kE4m3>(p, cur);
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
      cursor_next<D, kE4m3>(p, ahead);
    }
  };
  auto next_page = [&]() {
    page = -1;
    page_kv = tok_kv;
    if (tok >= 0) {
      if (tok < tok_len) {
        const int at = tok / p.k.page_size;
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
      const int c = lane % S::kChunks;
#pragma unroll
      for (int i = 0; i < S::kKeys / kRowsPerCopy; ++i) {
        const int r = i * kRowsPerCopy + lane / S::kChunks;
        const int64_t a = __shfl_sync(0xffffffffu, ko, r);
        const bool on = (valid >> r) & 1u;
        copy16(W::chunk_at(kt, r, c), p.k.data + a + c * 16, on);
        const int64_t b = p.same_strides ? a : __shfl_sync(0xffffffffu, vo, r);
        copy16(W::chunk_at(vt, r, c), p.v.data + b + c * 16, on);
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
      w.tile(p, kt, kt + S::kTileBytes,
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
    const int t = lane & 3, row = lane >> 2;
#pragma unroll
    for (int r = 0; r < W::kRows; ++r) {
      float s = w.l[r];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (t == 0) {
        ml[warp * 32 + row + 8 * r] = w.m[r];
        ml[warp * 32 + 16 + row + 8 * r] = s;
      }
    }
    __syncthreads();
    float factor[2] = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < W::kRows; ++r) {
      float mm = w.m[r];
#pragma unroll
      for (int x = 0; x < kAttendWarps; ++x) mm = fmaxf(mm, ml[x * 32 + row + 8 * r]);
      factor[r] = exp2_fast(w.m[r] - finite_or_zero(mm));
      if constexpr (kE4m3) factor[r] *= w.f[r];
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
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += S::kJoinCols) {
#pragma unroll 1
      for (int x = 0; x < kAttendWarps; ++x) {  // in warp order
        if (warp == x) {
#pragma unroll
          for (int j = c0 / 8; j < (c0 + S::kJoinCols) / 8; ++j)
#pragma unroll
            for (int r = 0; r < W::kRows; ++r)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float* dst = join + (row + 8 * r) * S::kJoinPitch + W::column(j, i, t) - c0;
                const float v = w.o[j][2 * r + i] * factor[r];
                *dst = x == 0 ? v : *dst + v;
              }
        }
        __syncthreads();
      }
      for (int i = tid; i < rows * (S::kJoinCols / 2); i += kAttendThreads) {
        const int y = i / (S::kJoinCols / 2), c = i % (S::kJoinCols / 2) * 2;
        const float2 v = *reinterpret_cast<const float2*>(join + y * S::kJoinPitch + c);
        if (whole)
          *reinterpret_cast<uint32_t*>(p.out + (out_row + y) * D + c0 + c) =
              floats_to_bf16x2(v.x * inverse[y], v.y * inverse[y]);
        else
          *reinterpret_cast<float2*>(part + 32 + y * D + c0 + c) = v;
      }
      if (c0 + S::kJoinCols < D) __syncthreads();
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
    cursor_next<D, kE4m3>(p, cur);
  }
  copy_wait<0>();
}

}  // namespace tk
