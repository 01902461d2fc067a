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
// the small operand, not of the large one.  16 flops per element of K and of e4m3
// V, 32 of bf16 V (a weight has two parts there), and group of eight heads: 78
// TFLOP/s of bf16 at full bandwidth.  The kernel is bound by reading K and V
// from HBM.
//
// Work: a unit is (sequence, list of query heads); its tokens are cut into
// granules of 4 * KT tokens, one tile of KT keys per warp.  All granules of
// all units form one line that the CTAs (two or three per SM) share evenly,
// whatever the lengths; a unit that lies in several CTAs' shares is joined by the CTA
// that finishes last (an atomic ticket, nobody waits; the parts are added in
// the order of the CTAs, so equal calls give equal bits).  Where units are many
// and short, joining is most of the time, and each warp takes whole units by itself
// instead (600 sequences of up to 128, 32 heads on 8: 46 us against 81).
//
// Each warp feeds itself through a ring of STAGES tiles of its own, so no
// barrier of the CTA stands in the loop and any page size, stride or list of
// positions is served.  A tile goes through three steps, STAGES - 1 tiles
// apart: its tokens (a list's positions are copied), its pages (looked up in
// the block table), its rows.  All three are cp.async copies into shared memory
// in the groups that the ring waits for anyway, so neither look-up's latency is
// ever waited for by itself (with look-ups one tile ahead in registers they took
// twice the time of the products on lists of 512 positions).
//
// Measured on one B200, bytes of K, V and scales against its copy bandwidth of
// 6461 GB/s: 16 ragged sequences up to 32768, 32 heads on 8, d 128, bf16: 196 to
// 203 us on several GPUs, 98 to 95 %; 16 x 8192, 32 on 32: 197 us, 98 %; pages of
// one token: 197 us, 98 %; e4m3, 4 ragged sequences up to 131072: 118 us, 87 %
// (issue: the codes' widening); 512 of 8192 positions for 512 heads: 34 us, 61 %,
// e4m3 30 us, 36 % (starts, ends and joins of 13 tiles a warp); 128 heads on 8
// (NT = 2): bf16 211 us, 92 %, e4m3 162 us, 62 % (issue).  One sequence of 1001: 11 us, of which the work takes 1: about 4 us
// pass before the first tile (lengths, table, rows are three dependent trips to
// memory), about 4 in joining 16 parts.
// Rejected: heads as the 16 rows of the products (237 us where this takes 196:
// twice the products and accumulators); q as two e4m3 codes beside e4m3 keys (the
// 8-bit product is made of conversions here: 146 us against 130); one round that
// also fills the ring (1 to 3 us slower on every case).
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
  bool grouped;       // no positions, 16 | page_size (16 tokens from a multiple of 16 on share a page), same strides
  bool same_strides;  // k and v, and their scales, have equal strides
  float scale_log2;   // softmax scale * log2(e)
  uint16_t* out;      // [batch][heads][d] bf16
  float* lse;         // null, or [batch][heads]
  uint32_t* tickets;  // [kAttendMaxCtas] of units by first CTA, [2 kAttendMaxCtas] of groups; zero between calls
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
  static constexpr uint32_t kAllKeys = kKeys == 32 ? 0xffffffffu : (1u << (kKeys & 31)) - 1u;
  static constexpr int kGranule = kAttendWarps * kKeys;
  static constexpr int kTileBytes = kKeys * kRowBytes;               // K or V
  static constexpr int kScaleBytes = kE4m3 ? 2 * kKeys * 4 : 0;
  static constexpr int kStageBytes = 2 * kTileBytes + kScaleBytes;
  static constexpr bool kQShared = D == 256 && NT == 2;  // Q fragments in shared memory (64 registers otherwise)
  // About 8 KB a tile: three stages of four warps and two CTAs fill an SM's
  // shared memory.  Tiles that take more instructions for their bytes (e4m3, or
  // narrow rows) gain more by a third CTA than by a third stage.
  static constexpr bool kThree = NT == 1 && (D == 64 || (D == 128 && kE4m3));
  static constexpr int kCtasPerSm = kThree ? 3 : D == 256 && (!kE4m3 || NT == 2) ? 1 : 2;
  static constexpr int kStages = D == 64 && kE4m3 ? (kThree ? 3 : 5) : kThree ? 2 : D == 256 && kE4m3 && NT == 2 ? 5 : 3;
  static constexpr int kSlots = 2 * kStages - 1;  // tiles from their tokens to their rows
  static constexpr int kJoinFloats = kThree ? 1280 : 1792;
  // shared memory: [warps][stages] tiles, join buffer, Q fragments, (m, l) per warp,
  // [warps][slots] tokens, pages and places, [warps][stages] valid masks, plan
  static constexpr int kOffJoin = kAttendWarps * kStages * kStageBytes;
  static constexpr int kOffQ = kOffJoin + kJoinFloats * 4;
  static constexpr int kOffMl = kOffQ + (kQShared ? 8192 : 0);
  static constexpr int kOffPlace = kOffMl + kAttendWarps * 32 * 4;
  static constexpr int kOffToken = kOffPlace + kAttendWarps * kSlots * 16;
  static constexpr int kOffPage = kOffToken + kAttendWarps * kSlots * kKeys * 4;
  static constexpr int kOffPlan = kOffPage + kAttendWarps * kSlots * kKeys * 4;
  static constexpr int kOffValid = kOffPlan + 64;
  static constexpr int kSmem = (kOffValid + kAttendWarps * kStages * 4 + 127) / 128 * 128;
  static_assert(kOffPlan % 8 == 0 && kOffPlace % 16 == 0, "alignment");
  static_assert((kSmem + 1024) * kCtasPerSm <= 228 * 1024, "shared memory");
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
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
// Where a CTA stands on the line of granules: a unit is a sequence, a list of
// query heads and 16 of the list's heads.
struct AttendCursor {
  int b, list, tile;  // sequence, list, group of 16 heads
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

// To the next granule; past the last one `b` is tab.batch and nothing may be
// read.  Returns whether another unit begins.
template <int kGranule>
__device__ __forceinline__ bool cursor_next(const AttendArgs& p, AttendCursor& u) {
  if (++u.at < u.granules) return false;
  u.at = 0;
  if (++u.tile < p.row_tiles) return true;
  u.tile = 0;
  if (++u.list < p.lists) return true;
  u.list = 0;
  do {
    if (++u.b >= p.tab.batch) {
      u.granules = 0;
      u.count = 0;
      return true;
    }
    cursor_enter<kGranule>(p, u);
  } while (u.granules == 0);
  return true;
}

// The same for a warp that takes whole units, every `step`-th of them: a tile
// of keys is a granule, and a unit without a token has one as well, in which
// its rows are written.
template <int kKeys>
__device__ __forceinline__ void cursor_enter_unit(const AttendArgs& p, AttendCursor& u, uint32_t unit) {
  const uint32_t of_seq = p.lists * p.row_tiles, list = unit % of_seq;
  u.b = static_cast<int>(unit / of_seq);
  u.list = static_cast<int>(list / p.row_tiles);
  u.tile = static_cast<int>(list - u.list * p.row_tiles);
  u.at = 0;
  u.count = p.positions ? p.c : seq_length(p.tab, u.b);
  u.granules = max(granules_of<kKeys>(u.count), 1);
}

// Share c of `total` granules among `ctas`; in 32 bits where that is enough
// (a 64-bit division takes a few hundred cycles of a call's start).
__device__ __forceinline__ int64_t attend_share(int64_t total, int ctas, int c) {
  if (total < (1 << 21)) return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(ctas);
  return part_start(total, ctas, c, 1, total);
}
__device__ __forceinline__ int attend_owner(int64_t granule, int64_t total, int ctas) {
  if (total < (1 << 21))
    return static_cast<int>((static_cast<uint32_t>(granule + 1) * static_cast<uint32_t>(ctas) - 1) /
                            static_cast<uint32_t>(total));
  return part_of(granule, total, ctas, 1);
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
  float f[NT][2];    // e4m3: O holds sum w_j V8_j / f, with w_j = 2^(s_j - m) * vscale_j; at least kLeast
  float inv[NT][2];  // 1 / f
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
        f[n][h] = kLeast;
        inv[n][h] = 1.0f / kLeast;
      }
    }
  }

  // The smallest f, whose inverse is finite: the smallest scale, 2^-127, is half of it.
  static constexpr float kLeast = 1.17549435e-38f;  // 2^-126
  static constexpr float kMost = 3.40282347e38f;    // of a finite w

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
            uint32_t a[4];
            e4m3x4_to_f16x2(r[2 * x], a[0], a[2]);
            e4m3x4_to_f16x2(r[2 * x + 1], a[1], a[3]);
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
    if (valid != S::kAllKeys) {
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
            const float fn = f[n][h] * x;
            f[n][h] = fmaxf(fn, kLeast);
            inv[n][h] = 1.0f / f[n][h];
            if (fn < kLeast) {  // what f cannot follow, O does
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                o[n][j][h] *= fn * (1.0f / kLeast);
                o[n][j][2 + h] *= fn * (1.0f / kLeast);
              }
            }
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
      // w_j = p_j * vscale_j, held in f16 relative to f, which is at most 2^-10 of
      // the head's largest w: a weight keeps 11 bits down to 2^-24 of that, and
      // below is off by 2^-35 of it at most.  (With f at the largest w itself, the
      // tail behind a key of 2^24 times its weight was off by 20 % where that key's
      // value is 0.)  f16 holds up to 65504, so f moves when a w passes 2^15 f.
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
        for (int h = 0; h < 2; ++h) grow |= wt[n][h] > f[n][h] * 32768.0f;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float fn = fmaxf(f[n][h], fminf(column_max(wt[n][h]), kMost) * 0x1p-10f);
            const float x = f[n][h] / fn;
            f[n][h] = fn;
            inv[n][h] = 1.0f / fn;
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
#pragma unroll
          for (int k = 0; k < kGroups; ++k) {
            s[n][k][h] *= inv[n][h];
            s[n][k][2 + h] *= inv[n][h];
          }
        }
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      // P^T as the right operand.  Beside bf16 values P is split into two bf16
      // parts: the upper half of its bits, and what is left, rounded.  That keeps
      // 16 bits of every weight, and both parts are positive (the last of the 24
      // bits is set for it, 2^-23 of the weight), so that an infinite value gives
      // an infinite product with each and not NaN with a second part of zero or
      // below.
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float a = s[n][k][2 * y], b = s[n][k][2 * y + 1];
          if constexpr (kE4m3) {
            hi[n][y] = transpose8x8(floats_to_f16x2(a, b));
          } else {
            const uint32_t x = __float_as_uint(a), z = __float_as_uint(b);
            hi[n][y] = transpose8x8(__byte_perm(x, z, 0x7632));
            lo[n][y] = transpose8x8(floats_to_bf16x2(__uint_as_float(x | 1u) - __uint_as_float(x & 0xffff0000u),
                                                     __uint_as_float(z | 1u) - __uint_as_float(z & 0xffff0000u)));
          }
        }
      if constexpr (kE4m3) {
#pragma unroll
        for (int c = 0; c < S::kChunks; c += 2) {
          uint32_t r[4];
          load_bytes_t(r, chunk_at(vt, k * 16 + (lane & 15), c + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t a[4];
            e4m3x4_to_f16x2(r[2 * x], a[0], a[2]);
            e4m3x4_to_f16x2(r[2 * x + 1], a[1], a[3]);
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

  // The rows of a unit that this warp has had all of.  Lanes g and g ^ 1 swap
  // a column, so that each has two neighbours to write.
  __device__ __forceinline__ void write_rows(const AttendArgs& p, int64_t out_row, int rows) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = n * 8 + 2 * t + h;
        const float sum = column_sum(l[n][h]);
        const float factor = sum == 0.0f ? 0.0f : 1.0f / sum;
        const float unit = kE4m3 ? f[n][h] : 1.0f;  // a factor of its own: f / sum may be a subnormal
        uint16_t* dst = p.out + (out_row + row) * D + (g & 1 ? 7 + g : g);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const float a = o[n][j][h] * factor * unit, b = o[n][j][2 + h] * factor * unit;
          const float c = __shfl_xor_sync(0xffffffffu, g & 1 ? a : b, 4);
          if (row < rows)
            *reinterpret_cast<uint32_t*>(dst + 16 * j) = g & 1 ? floats_to_bf16x2(c, b) : floats_to_bf16x2(a, c);
        }
        if (p.lse && row < rows && g == 0) p.lse[out_row + row] = 0.6931471805599453f * (m[n][h] + log2f(sum));
      }
  }

  // Column of o[.][j][i] for a lane with lane / 4 = g.
  static __device__ __forceinline__ int column(int j, int i, int g) { return 16 * j + g + 8 * (i >> 1); }
};

// ---------------------------------------------------------------- joining
// The part of a unit that CTA c holds: its first CTA writes slot 1, the others
// (which continue a unit) slot 0.  m of 16 rows, l of 16 rows, O / l [16][D]
// (means of V, which fit a float whenever V does).
template <int D>
__device__ __forceinline__ float* attend_part(float* parts, int c, int first) {
  return parts + static_cast<int64_t>(c * 2 + (c == first)) * attend_part_floats(D);
}

// Joins the n (up to 32) parts of CTAs c0, c0 + step, ... in that order: into
// the unit's output rows, or into the first of the parts.  All threads of the
// CTA; buf holds 1056 floats.  (A call of its own; it takes no reference to the
// kernel's arguments, which would move them from constant to local memory.)
template <int D>
__device__ __noinline__ void attend_join(float* parts, int first, int c0, int n, int step, int rows, bool final,
                                         uint16_t* out, float* lse, float* buf) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* weight = buf;        // [rows][32], the parts' shares of the row
  float* mass = buf + 512;    // [rows] max, [rows] sum
  float* half = buf + 544;    // [<= 128][4] partial sums
  for (int r = warp; r < rows; r += kAttendWarps) {
    float m = __int_as_float(0xff800000), l = 0.0f;
    if (lane < n) {
      const float* part = attend_part<D>(parts, c0 + lane * step, first);
      m = __ldcg(part + r);
      l = __ldcg(part + 16 + r);
    }
    float mm = m;
#pragma unroll
    for (int x = 16; x; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
    const float w = exp2_fast(m - finite_or_zero(mm));
    const float mine = lane < n ? w * l : 0.0f;
    float sum = mine;
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    weight[r * 32 + lane] = sum == 0.0f ? 0.0f : __fdividef(mine, sum);
    if (lane == 0) {
      mass[r] = mm;
      mass[16 + r] = sum;
    }
  }
  __syncthreads();
  // Four columns of a row per thread; few rows share their parts out to
  // `split` threads, added in order.
  const int total = rows * (D / 4);
  const int split = total > 64 ? 1 : total > 32 ? 2 : 4;
  float* dst0 = attend_part<D>(parts, c0, first);
  for (int i0 = 0; i0 < total; i0 += kAttendThreads / split) {
    const int i = i0 + tid % (kAttendThreads / split), s = tid / (kAttendThreads / split);
    const int r = i / (D / 4), col = i % (D / 4) * 4;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < total) {
#pragma unroll 8
      for (int x = s; x < n; x += split) {
        const float w = weight[r * 32 + x];
        const float4 v =
            __ldcg(reinterpret_cast<const float4*>(attend_part<D>(parts, c0 + x * step, first) + 32 + r * D + col));
        acc.x += w * v.x;
        acc.y += w * v.y;
        acc.z += w * v.z;
        acc.w += w * v.w;
      }
    }
    if (split > 1) {
      reinterpret_cast<float4*>(half)[tid] = acc;
      __syncthreads();
      if (s == 0)
        for (int x = 1; x < split; ++x) {
          const float4 v = reinterpret_cast<const float4*>(half)[tid + x * (kAttendThreads / split)];
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
        }
    }
    if (i < total && s == 0) {
      if (final) {
        *reinterpret_cast<uint2*>(out + r * D + col) =
            make_uint2(floats_to_bf16x2(acc.x, acc.y), floats_to_bf16x2(acc.z, acc.w));
      } else {
        *reinterpret_cast<float4*>(dst0 + 32 + r * D + col) = acc;  // read by this thread alone
      }
    }
  }
  if (tid < rows) {
    if (final) {
      if (lse) lse[tid] = 0.6931471805599453f * (mass[tid] + log2f(mass[16 + tid]));
    } else {
      dst0[tid] = mass[tid];
      dst0[16 + tid] = mass[16 + tid];
    }
  }
}

// One of `count` arrivals at a ticket; true for all threads of the CTA that
// arrives last, which then sees what the others wrote before they arrived.
__device__ __forceinline__ bool attend_arrive(uint32_t* ticket, int count, int64_t* flag) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const bool last = atomicAdd(ticket, 1u) == static_cast<uint32_t>(count - 1);
    if (last) *ticket = 0;
    __threadfence();
    *flag = last;
  }
  __syncthreads();
  return *flag != 0;
}

// ---------------------------------------------------------------- kernel
// kSolo: every warp takes whole units by itself, an equal number each; there is
// nothing to join and no barrier, which is most of a short unit's time.  Units
// of a sequence go to different warps, so that a long one's are spread.
template <int D, bool kE4m3, int NT, bool kSolo>
__global__ void __launch_bounds__(kAttendThreads, (AttendShape<D, kE4m3, NT>::kCtasPerSm))
    paged_attention_kernel(AttendArgs p) {
  using S = AttendShape<D, kE4m3, NT>;
  using W = AttendWarp<D, kE4m3, NT>;
  static_assert(!(kSolo && S::kQShared), "the shared Q is one unit's");
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* join = reinterpret_cast<float*>(smem + S::kOffJoin);
  uint2* shared_q = reinterpret_cast<uint2*>(smem + S::kOffQ);
  float* ml = reinterpret_cast<float*>(smem + S::kOffMl);  // [warp][m of 16 rows, l of 16 rows]
  uint32_t* valid_masks = reinterpret_cast<uint32_t*>(smem + S::kOffValid) + warp * S::kStages;
  int4* places = reinterpret_cast<int4*>(smem + S::kOffPlace) + warp * S::kSlots;
  int* tokens = reinterpret_cast<int*>(smem + S::kOffToken) + warp * S::kSlots * S::kKeys;
  int* pages = reinterpret_cast<int*>(smem + S::kOffPage) + warp * S::kSlots * S::kKeys;
  int64_t* plan = reinterpret_cast<int64_t*>(smem + S::kOffPlan);
  unsigned char* ring = smem + warp * S::kStages * S::kStageBytes;
  const uint32_t ring_addr = smem_addr(ring);
  pdl_wait_then_release();

  const int units = p.lists * p.row_tiles;
  const int group = p.heads / p.lists;
  // This CTA's share [g0, g1) of the line, and where it begins.
  // No share is empty: shares are given to as many CTAs as there are granules.
  int64_t total, g0, g1;
  int ctas;
  AttendCursor cur;
  auto share = [&]() {
    ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total));
    g0 = static_cast<int>(blockIdx.x) < ctas ? attend_share(total, ctas, blockIdx.x) : total;
    g1 = static_cast<int>(blockIdx.x) < ctas ? attend_share(total, ctas, blockIdx.x + 1) : total;
  };
  if constexpr (kSolo) {
    // g is a unit here
    g0 = warp * gridDim.x + blockIdx.x;
    g1 = static_cast<uint32_t>(p.tab.batch) * static_cast<uint32_t>(units);
    if (g0 >= g1) return;
    cursor_enter_unit<S::kKeys>(p, cur, static_cast<uint32_t>(g0));
  } else if (p.positions) {
    cur.b = 0;
    cursor_enter<S::kGranule>(p, cur);
    total = static_cast<int64_t>(p.tab.batch) * units * cur.granules;
    share();
    if (g0 >= g1) return;
    const int64_t u = g0 / cur.granules;
    cur.b = static_cast<int>(u / units);
    cur.list = static_cast<int>(u - static_cast<int64_t>(cur.b) * units);
    cur.at = static_cast<int>(g0 - u * cur.granules);
  } else {
    // Running sums of the sequences' granules: a stretch of sequences per thread.
    const int per = (p.tab.batch + kAttendThreads - 1) / kAttendThreads;
    const int b0 = min(tid * per, p.tab.batch), b1 = min(b0 + per, p.tab.batch);
    int64_t mine = 0;
    bool empty = false;
    for (int b = b0; b < b1; ++b) {
      const int n = granules_of<S::kGranule>(seq_length(p.tab, b));
      mine += n;
      empty |= n == 0;
    }
    int64_t upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, x);
      if (lane >= x) upto += y;
    }
    if (lane == 31) plan[warp] = upto;
    if (__syncthreads_or(empty)) {
      // Sequences without a token have no granule: their rows are written here.
      for (int b = blockIdx.x; b < p.tab.batch; b += gridDim.x) {
        if (seq_length(p.tab, b) != 0) continue;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + static_cast<int64_t>(b) * p.heads * D);
        for (int i = tid; i < p.heads * (D / 2); i += kAttendThreads) dst[i] = 0;
        if (p.lse)
          for (int i = tid; i < p.heads; i += kAttendThreads)
            p.lse[static_cast<int64_t>(b) * p.heads + i] = __int_as_float(0xff800000);
      }
    }
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
    if (g0 >= g1) return;
    cur.b = static_cast<int>(plan[4]);
    cursor_enter<S::kGranule>(p, cur);
    cur.list = static_cast<int>(plan[5] / cur.granules);
    cur.at = static_cast<int>(plan[5] - static_cast<int64_t>(cur.list) * cur.granules);
  }
  if constexpr (!kSolo) {
    cur.tile = cur.list % p.row_tiles;
    cur.list /= p.row_tiles;
  }
  const int64_t step = kSolo ? gridDim.x * kAttendWarps : 1;  // of g

  // The three steps of a tile.  A lane of index < kKeys has a key.  Where a
  // tile lies: its sequence, its key-value head, the sequence's length and the
  // first of its tokens (or -1 behind the share's end).
  AttendCursor ahead = cur;
  int64_t ahead_left = g1 - g0;  // granules to fetch; kSolo: units from this one to the last
  const int kv_per = p.lists / p.k.kv_heads;
  int ahead_kv = cur.list / kv_per;
  int ahead_len = p.positions ? seq_length(p.tab, cur.b) : cur.count;
  const uint32_t tokens_addr = smem_addr(tokens), pages_addr = smem_addr(pages);
  auto fetch_tokens = [&](int slot) {
    int4 place = make_int4(0, 0, 0, -1);
    if (ahead_left > 0) {
      const uint32_t i0 = (kSolo ? static_cast<uint32_t>(ahead.at)
                                 : static_cast<uint32_t>(ahead.at) * kAttendWarps + warp) * S::kKeys;
      place = make_int4(ahead.b, ahead_kv, ahead_len, static_cast<int>(min(i0, 0x7fffffffu)));
      if (p.positions && lane < S::kKeys) {
        const bool on = i0 + lane < static_cast<uint32_t>(ahead.count);
        copy4(tokens_addr + (slot * S::kKeys + lane) * 4,
              p.positions + (static_cast<int64_t>(ahead.b) * p.lists + ahead.list) * p.c + (on ? i0 + lane : 0), on);
      }
      bool another;
      if constexpr (kSolo) {
        another = ++ahead.at == ahead.granules;
        if (another && (ahead_left -= step) > 0) cursor_enter_unit<S::kKeys>(p, ahead, static_cast<uint32_t>(g1 - ahead_left));
      } else {
        --ahead_left;
        another = cursor_next<S::kGranule>(p, ahead);
      }
      if (another && ahead_left > 0) {
        ahead_kv = ahead.list / kv_per;
        ahead_len = p.positions ? seq_length(p.tab, ahead.b) : ahead.count;
      }
    }
    if (lane == 0) places[slot] = place;
  };
  // The lane's token turns into its page, asked for here, and its offset there
  // (-1: no token).  A list's slots behind its end are told by their index.
  auto fetch_pages = [&](int slot) {
    const int4 place = places[slot];
    if (lane < S::kKeys) {
      const uint32_t i = static_cast<uint32_t>(place.w) + lane;
      int tok = -1;
      if (place.w >= 0 && i < static_cast<uint32_t>(p.positions ? p.c : place.z))
        tok = p.positions ? tokens[slot * S::kKeys + lane] : static_cast<int>(i);
      const bool on = tok >= 0 && tok < place.z;
      if (tok >= p.tab.capacity) atomicOr(&g_device_status, kDevBadIndex);
      const int at = on ? p.k.page_of(tok) : 0;
      copy4(pages_addr + (slot * S::kKeys + lane) * 4, p.tab.table + place.x * p.tab.stride + at, on);
      tokens[slot * S::kKeys + lane] = on ? tok - at * p.k.page_size : -1;
    }
  };
  auto fetch_rows = [&](int stage, int slot) {
    const int page_kv = places[slot].y;
    int o = lane < S::kKeys ? tokens[slot * S::kKeys + lane] : -1;
    bool live = o >= 0;
    int64_t pg = 0;
    if (live) {
      pg = pages[slot * S::kKeys + lane];
      if (pg < 0 || pg >= p.k.pages) {
        atomicOr(&g_device_status, kDevBadIndex);
        live = false;
        pg = 0;
      }
    }
    if (!live) o = 0;
    const uint32_t valid = __ballot_sync(0xffffffffu, live);
    const int64_t ko = pg * p.k.page_stride + page_kv * p.k.head_stride + o * p.k.token_stride;
    int64_t vo = ko;
    if (!p.same_strides) vo = pg * p.v.page_stride + page_kv * p.v.head_stride + o * p.v.token_stride;
    const uint32_t kt = ring_addr + stage * S::kStageBytes, vt = kt + S::kTileBytes;
    if (lane == 0) valid_masks[stage] = valid;
    if (valid) {
      constexpr int kRowsPerCopy = 32 / S::kChunks;
      const int c = lane % S::kChunks, r0 = lane / S::kChunks;
      if (p.grouped && valid == S::kAllKeys) {
        // The common tile: one address for 16 rows of K and of V, no row left
        // out.  r0 is below the power of two kRowsPerCopy, so that the chunk's
        // permutation is the lane's own and a constant of the copy.
        const uint32_t lane_at = W::chunk_at(0, r0, c);
        const int64_t step = kRowsPerCopy * p.k.token_stride;
        const int64_t lane_off = r0 * p.k.token_stride + c * 16;
#pragma unroll
        for (int y = 0; y < S::kKeys / 16; ++y) {
          const int64_t a = __shfl_sync(0xffffffffu, ko, y * 16) + lane_off;
          const unsigned char* ka = p.k.data + a;
          const unsigned char* va = p.v.data + a;
#pragma unroll
          for (int i = 0; i < 16 / kRowsPerCopy; ++i) {
            const uint32_t flip = W::chunk_at(0, y * 16 + i * kRowsPerCopy, 0);
            copy16(kt + ((lane_at ^ (flip & 127)) + (flip & ~127u)), ka);
            copy16(vt + ((lane_at ^ (flip & 127)) + (flip & ~127u)), va);
            ka += step;
            va += step;
          }
        }
      } else {
        // any rows: their addresses from the lanes that looked them up, a few
        // rows at a time so that the exchanges overlap
        constexpr int kCopies = S::kKeys / kRowsPerCopy, kBatch = kCopies < 8 ? kCopies : 8;
#pragma unroll
        for (int i0 = 0; i0 < kCopies; i0 += kBatch) {
          int64_t at[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) at[i] = __shfl_sync(0xffffffffu, ko, (i0 + i) * kRowsPerCopy + r0) + c * 16;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int r = (i0 + i) * kRowsPerCopy + r0;
            copy16(W::chunk_at(kt, r, c), p.k.data + at[i], (valid >> r) & 1u);
          }
          if (!p.same_strides) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) at[i] = __shfl_sync(0xffffffffu, vo, (i0 + i) * kRowsPerCopy + r0) + c * 16;
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int r = (i0 + i) * kRowsPerCopy + r0;
            copy16(W::chunk_at(vt, r, c), p.v.data + at[i], (valid >> r) & 1u);
          }
        }
      }
      if constexpr (kE4m3) {
        if (lane < S::kKeys) {
          const uint32_t st = vt + S::kTileBytes + lane * 4;
          const int64_t ks = pg * p.k.s_page_stride + page_kv * p.k.s_head_stride + o * p.k.s_token_stride;
          int64_t vs = ks;
          if (!p.same_strides) vs = pg * p.v.s_page_stride + page_kv * p.v.s_head_stride + o * p.v.s_token_stride;
          copy4(st, p.k.scale + ks, live);
          copy4(st + S::kKeys * 4, p.v.scale + vs, live);
        }
      }
    }
  };

  // Before the first tile: its tokens, and those of the tiles that the steps
  // are apart; then the pages likewise; then rows.  Slot of tile i: i % kSlots.
  constexpr int kApart = S::kStages - 1;
  int slot_t = 0, slot_p = 0, slot_r = 0;
  auto next_slot = [](int& x) { x = x == S::kSlots - 1 ? 0 : x + 1; };
#pragma unroll 1
  for (int i = 0; i < kApart; ++i) {
    fetch_tokens(slot_t);
    next_slot(slot_t);
  }
  copy_commit();
  copy_wait<0>();
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < kApart; ++i) {
    fetch_pages(slot_p);
    next_slot(slot_p);
    fetch_tokens(slot_t);
    next_slot(slot_t);
  }
  copy_commit();
  copy_wait<0>();
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < kApart; ++i) {
    fetch_rows(i, slot_r);
    next_slot(slot_r);
    fetch_pages(slot_p);
    next_slot(slot_p);
    __syncwarp();  // the tokens' slot held the rows' place
    fetch_tokens(slot_t);
    next_slot(slot_t);
    copy_commit();
  }

  W w;
  w.reset();
  bool fresh = true;
  int stage = 0;
#pragma unroll 1
  for (int64_t g = g0; g < g1;) {
    const int rows = min(16, group - cur.tile * 16);
    const int head = cur.list * group + cur.tile * 16;
    if (fresh) {
      if constexpr (S::kQShared) __syncthreads();
      w.load_q(p, p.q + cur.b * p.q_stride + static_cast<int64_t>(head) * D, rows, shared_q, warp);
      if constexpr (S::kQShared) __syncthreads();
      fresh = false;
    }
    copy_wait<S::kStages - 2>();
    __syncwarp();
    // the stage consumed last is free again, and so is the slot of its rows
    fetch_rows(stage == 0 ? S::kStages - 1 : stage - 1, slot_r);
    next_slot(slot_r);
    fetch_pages(slot_p);
    next_slot(slot_p);
    __syncwarp();
    fetch_tokens(slot_t);
    next_slot(slot_t);
    copy_commit();
    const uint32_t valid = valid_masks[stage];
    if (valid) {
      const uint32_t kt = ring_addr + stage * S::kStageBytes;
      w.tile(kt, kt + S::kTileBytes,
             reinterpret_cast<const float*>(ring + stage * S::kStageBytes + 2 * S::kTileBytes), valid, shared_q);
    }
    stage = stage == S::kStages - 1 ? 0 : stage + 1;
    if (cur.at + 1 < cur.granules && (kSolo || g + 1 < g1)) {
      ++cur.at;
      g += !kSolo;
      continue;
    }

    if constexpr (kSolo) {
      w.write_rows(p, static_cast<int64_t>(cur.b) * p.heads + head, rows);
      w.reset();
      fresh = true;
      g += step;
      if (g < g1) cursor_enter_unit<S::kKeys>(p, cur, static_cast<uint32_t>(g));
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
    // m and l of a row of all four warps
    auto joined = [&](int row, float& mm, float& sum) {
      mm = ml[row];
#pragma unroll
      for (int x = 1; x < kAttendWarps; ++x) mm = fmaxf(mm, ml[x * 32 + row]);
      sum = 0.0f;
#pragma unroll
      for (int x = 0; x < kAttendWarps; ++x) sum += ml[x * 32 + 16 + row] * exp2_fast(ml[x * 32 + row] - finite_or_zero(mm));
    };
    float factor[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mm, sum;
        joined(n * 8 + 2 * t + h, mm, sum);
        factor[n][h] = sum == 0.0f ? 0.0f : __fdividef(exp2_fast(w.m[n][h] - finite_or_zero(mm)), sum);
      }
    float* part = p.parts + static_cast<int64_t>(blockIdx.x * 2 + (unit_first >= g0)) * attend_part_floats(D);
    const int64_t out_row = static_cast<int64_t>(cur.b) * p.heads + head;
    if (tid < rows) {
      float mm, sum;
      joined(tid, mm, sum);
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
              join[(warp * rows + head_row) * pitch + W::column(j, i, lane_g) - c0] =
                  w.o[n][j][i] * factor[n][i & 1] * (kE4m3 ? w.f[n][i & 1] : 1.0f);
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
              floats_to_bf16x2(v.x, v.y);
        else
          *reinterpret_cast<float2*>(part + 32 + y * D + c0 + c) = v;
      }
    }
    if (!whole) {
      // Up to 32 parts are joined at once; more by groups of 32, and then the
      // groups (one CTA reading hundreds of parts would take longer than the
      // cache did).
      const int first = attend_owner(unit_first, total, ctas);
      const int last = attend_owner(unit_first + cur.granules - 1, total, ctas);
      const int n = last - first + 1, me = static_cast<int>(blockIdx.x) - first;
      uint16_t* out = p.out + out_row * D;
      float* lse = p.lse ? p.lse + out_row : nullptr;
      // one call site: the whole unit's parts, a group's, or the groups'
      int c0 = first, members = n, step = 1;
      uint32_t* ticket = p.tickets + first;
      if (n > 32) {
        c0 = first + me / 32 * 32;
        members = min(32, last - c0 + 1);
        ticket = p.tickets + kAttendMaxCtas + 2 * c0 + (c0 == first);
      }
      while (attend_arrive(ticket, members, plan + 6)) {
        const bool final = n <= 32 || step == 32;
        attend_join<D>(p.parts, first, c0, members, step, rows, final, out, lse, join);
        if (final) break;
        c0 = first;
        members = (n + 31) / 32;
        step = 32;
        ticket = p.tickets + first;
      }
    }
    __syncthreads();
    w.reset();
    fresh = true;
    cursor_next<S::kGranule>(p, cur);
    ++g;
  }
  copy_wait<0>();
}

}  // namespace tk
