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

// Two kernels.  A CTA of the first takes a piece of a beam's row: the piece's
// maximum, its sum of exponentials and its k largest logits.  A CTA of the
// second, started as the first drains, turns a sentence's sums into lse_i and
// picks the k best of all pieces' lists.  Within a beam the order is the
// logits', so a piece's list can be cut at k before lse_i is known.  (Leaving
// the second part to the CTA that finishes a sentence last costs every CTA a
// fence and an atomic, 1.1 of its 7 us.)
//
// The k largest of a piece without sorting it: of the 256 threads' maxima, the
// j-th largest of each warp (j = ceil(k / 8)) bounds the k-th largest value
// from below in all; the few vectors that reach the smallest of these bounds
// are set aside, their elements gathered and ranked by counting.  Where that
// leaves too many (equal logits), the bound is bisected, over keys and then over
// indices.
//
// The first kernel has two forms.  Few rows (a round of CTAs at most): pieces of
// at most 64 KB that stay in the CTA's registers, the maximum first, then the
// exponentials relative to it.  Many rows: pieces of up to 256 KB that pass
// through the registers once, in batches, with a running reference; the few
// batches that hold candidates are read again, from a cache.  A piece's start
// and end take about as long as 64 KB of logits, so fewer pieces pay.
//
// Bound by reading the logits.  A logit costs one exponential (16 per clock
// and SM: 4.5e12 a second, against 1.6e12 fp32 or 3.2e12 bf16 logits a second
// at full bandwidth) and about five other instructions.  Measured: 4 x 131072
// fp32, k 8: 9.0 us (held); 32 sentences x 8 x 128255 bf16, k 16: 27 us, 2.4
// TB/s (streaming; 31.9 held, in 3.5 rounds of CTAs); 512 x 128255 fp32, k 8:
// 60 us, 4.4 TB/s (75 held).  About 5 us of these are the second kernel.
// Rejected: resident CTAs with the next held piece on its way into shared memory
// (39 us by cp.async, 38 us by bulk copies: the pieces fit half as many warps);
// batches of 8 vectors by two CTAs per SM instead of 4 by four (equal there, a
// quarter slower on 1024 rows of 32000).

// A piece's largest key (0: nothing) and its sum of 2^(x L - r), with L = log2 e
// rounded to fp32 and r a whole number near max * L (so that sums join by exact
// powers of two), or of exp(x - max), r = kBeamByMax, where max is beyond 1e6.
struct __align__(16) BeamSum {
  double sum;
  uint32_t top;
  int r;
};
constexpr int kBeamByMax = -2147483647 - 1;
constexpr float kBeamLog2e = 1.4426950408889634f;

struct BeamArgs {
  const void* logits;   // [batch][beams][n]
  const float* scores;  // [batch][beams]
  int64_t n;
  int beams, k;
  int pieces;           // per row
  int64_t first;        // sentence of blockIdx.x = 0
  float* out_scores;    // [batch][k]
  int32_t* out_parent;  // [batch][k]
  int32_t* out_token;   // [batch][k]
  BeamSum* sums;        // [rows of the launch][pieces]
  uint64_t* lists;      // [rows of the launch][pieces][k]
};

constexpr int kMaxBeams = 128;
constexpr int kBeamCap = 512;       // gathered candidates; more than the largest k
constexpr int kBeamHits = 384;      // vectors that hold them, or batches
constexpr int kBeamBatch = 4;       // 16-byte vectors that a thread takes at a time
constexpr int kBeamBatches = 16;    // of a thread
constexpr int kBeamCtasPerSm = 4;
constexpr int kBeamVectors = 16;    // of a thread, where a piece stays in registers

// Order key of a candidate logit; 0 for one that gives no continuation.
__device__ __forceinline__ uint32_t beam_key(float x) {
  return x == __int_as_float(0xff800000) ? 0u : order_key(x);
}

// A key that at least k of the CTA's elements reach, given every thread's
// largest key (0: none).  warp_keys: 8 words.
__device__ __forceinline__ uint32_t beam_bound(uint32_t mine, int k, uint32_t* warp_keys) {
  constexpr int kWarps = kBeamThreads / 32;
  const int rounds = (k + kWarps - 1) / kWarps;
  uint32_t last = 0;
  for (int i = 0; i < rounds; ++i) {
    last = __reduce_max_sync(0xffffffffu, mine);
    if (last == 0) break;
    if (mine == last) mine = 0;
  }
  if ((threadIdx.x & 31) == 0) warp_keys[threadIdx.x >> 5] = last;
  __syncthreads();
  // k <= 8: the k-th largest of the eight warps' maxima; else the smallest.
  uint32_t bound = warp_keys[0];
  if (k >= kWarps) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) bound = min(bound, warp_keys[w]);
    return bound;
  }
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    int above = 0;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) above += warp_keys[v] > warp_keys[w] || (warp_keys[v] == warp_keys[w] && v < w);
    if (above == k - 1) bound = warp_keys[w];
  }
  return bound;
}

__device__ __forceinline__ int block_total(int mine, int* slot) {
  __syncthreads();
  if (threadIdx.x == 0) *slot = 0;
  __syncthreads();
  mine = __reduce_add_sync(0xffffffffu, mine);
  if ((threadIdx.x & 31) == 0 && mine) atomicAdd(slot, mine);
  __syncthreads();
  return *slot;
}

struct BeamShared {
  union {
    uint64_t gathered[kBeamCap];
    struct {
      uint64_t value[kBeamCap], rest[kBeamCap];
      uint32_t token[kBeamCap];
    } cont;
  };
  uint4 hit[kBeamHits];   // vectors of a piece that reach its bound
  int hit_at[kBeamHits];  // index of their first element
  int batch[kBeamHits];   // batches that reach it: number * threads + thread
  double off[kMaxBeams];
  double part[kBeamThreads / 32];
  Cont best[kBeamThreads / 32];
  uint32_t warp_keys[kBeamThreads / 32], warp_tops[kBeamThreads / 32];
  int count, hits, batches, total;
};

__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes from byte s (1 .. 15) on of two neighbouring vectors.
__device__ __forceinline__ uint4 shift_together(const uint4& a, const uint4& b, int s) {
  const int w = s >> 2, bits = (s & 3) * 8;
  const uint32_t x0 = w == 0 ? a.x : w == 1 ? a.y : w == 2 ? a.z : a.w;
  const uint32_t x1 = w == 0 ? a.y : w == 1 ? a.z : w == 2 ? a.w : b.x;
  const uint32_t x2 = w == 0 ? a.z : w == 1 ? a.w : w == 2 ? b.x : b.y;
  const uint32_t x3 = w == 0 ? a.w : w == 1 ? b.x : w == 2 ? b.y : b.z;
  const uint32_t x4 = w == 0 ? b.x : w == 1 ? b.y : w == 2 ? b.z : b.w;
  return make_uint4(__funnelshift_r(x0, x1, bits), __funnelshift_r(x1, x2, bits), __funnelshift_r(x2, x3, bits),
                    __funnelshift_r(x3, x4, bits));
}

// The piece of a row that a CTA takes, as vectors of 16 bytes counted from the
// row's start.  Which thread adds which elements in which order, and so every
// bit of the row's sum, is the same wherever the row lies: beams of equal logits
// tie.  A warp takes 128 successive vectors at a time, four a lane.  Where the
// row is off a 16-byte address, a vector lies in two aligned ones: the lane
// loads the one that holds most of it and has the one or two words of the other
// from its neighbour.  Rows off such addresses take a tenth longer than rows on
// them (summed by aligned vectors, in an order that depended on the address, they
// did not): 512 x 128255 fp32 60 us, bf16 42, against 54 and 38.  Rejected: both
// aligned vectors loaded by every lane, from L1 the second time (fp32 62 us, bf16
// 56; the shift chosen word by word instead of by constants: 82, 49).  The
// row's first vector, its last whole one and the rest behind that may have
// neighbours in theirs: they are "edges", read by elements, by one thread each.
// A vector behind the piece, and elements behind the row, read as -inf.
template <typename T>
struct BeamPiece {
  static constexpr int kPer = 16 / sizeof(T);  // elements per vector
  static constexpr uint32_t kFill = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
  const T* row;
  int64_t n;
  int64_t w0, w1;  // vectors of the piece
  int mis;         // elements from an aligned address to the row's start
  int low, live;   // vectors w0 + low .. w0 + live - 1 of the piece are no edges

  __device__ __forceinline__ BeamPiece(const T* row_, int64_t n_, int piece, int pieces) : row(row_), n(n_) {
    mis = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % kPer);
    const uint32_t vectors = static_cast<uint32_t>((n + kPer - 1) / kPer);  // n < 2^31
    const uint32_t each = vectors / static_cast<uint32_t>(pieces), more = vectors - each * pieces;
    w0 = piece * each + min(static_cast<uint32_t>(piece), more);
    w1 = w0 + each + (piece < more);
    low = w0 == 0;
    live = max(low, static_cast<int>(min(w1, last()) - w0));
  }
  // Vector v (of each four successive ones) of this thread.
  static __device__ __forceinline__ int at(int v) { return at(v >> 2, v & 3, static_cast<int>(threadIdx.x)); }
  static __device__ __forceinline__ int at(int four, int v, int thread) {
    return four * (4 * kBeamThreads) + (thread & ~31) * 4 + v * 32 + (thread & 31);
  }
  __device__ __forceinline__ int64_t index(int i) const { return (w0 + i) * kPer; }  // of vector i's first element
  __device__ __forceinline__ int64_t last() const { return n / kPer - 1; }           // the row's last whole vector
  __device__ __forceinline__ bool edge(int64_t w) const { return w == 0 || w >= last(); }
  // The edge that a thread takes, or -1: the first one thread 0, the last whole
  // one thread 32 and the rest thread 64, where the piece has them.
  __device__ __forceinline__ int64_t edge_of(int thread) const {
    const int64_t w = thread == 0 ? 0 : thread == 32 ? last() : thread == 64 ? last() + 1 : -1;
    return w >= w0 && w < w1 && (w > 0 || thread == 0) ? w : -1;
  }
  // Vector i by itself.
  __device__ __forceinline__ uint4 load(int i) const {
    if (i < low || i >= live) return make_uint4(kFill, kFill, kFill, kFill);
    const uint4* src = reinterpret_cast<const uint4*>(row - mis + w0 * kPer) + i;
    const uint4 x = __ldg(src);
    return mis ? shift_together(x, __ldg(src + 1), mis * static_cast<int>(sizeof(T))) : x;
  }

  // Four vectors of every lane.  The row's start lies kWord words and 0 or 16
  // bits behind an aligned address; from kWord = 2 on the second of a vector's
  // two aligned ones is its own, which is one further on.
  __device__ __forceinline__ int word() const { return mis * static_cast<int>(sizeof(T)) / 4; }
  __device__ __forceinline__ const uint4* source() const {
    return reinterpret_cast<const uint4*>(row - mis + w0 * kPer) + (word() >= 2);
  }
  __device__ __forceinline__ bool whole(int four) const {
    return four * 4 * kBeamThreads >= low && (four + 1) * 4 * kBeamThreads <= live;
  }
  // The aligned vectors, and the words that complete the warp's last (first) one,
  // the same for all lanes (loaded by one of them, in a branch of its own, they
  // were waited for at the branch's end: 512 x 128255 fp32 90 us).
  // first: source() + at(0).
  __device__ __forceinline__ void load_four(uint4 (&x)[4], uint2& rest, const uint4* first, int four) const {
    const int back = word() >= 2, lane = static_cast<int>(threadIdx.x) & 31;
    const uint4* src = first + four * (4 * kBeamThreads);
    const uint2* words = reinterpret_cast<const uint2*>(src - lane + (back ? -1 : 128)) + back;
    rest = make_uint2(kFill, kFill);
    if (whole(four)) {
#pragma unroll
      for (int v = 0; v < 4; ++v) x[v] = __ldg(src + v * 32);
      if (mis) rest = __ldg(words);
    } else {
      // those beside the first and the last vector too: their words are needed
      const int from = low < live ? low - back : 0, to = low < live ? live - (back || mis == 0) : -1;
      const int i0 = at(four, 0, static_cast<int>(threadIdx.x)), i = i0 - lane + (back ? -1 : 128);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        x[v] = i0 + v * 32 >= from && i0 + v * 32 <= to ? __ldg(src + v * 32) : make_uint4(kFill, kFill, kFill, kFill);
      if (mis && i >= from && i <= to) rest = __ldg(words);
    }
  }
  template <int kWord>
  static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b, int bits) {
    return sizeof(T) == 4 ? a : __funnelshift_r(a, b, bits);
  }
  template <int kWord>
  __device__ __forceinline__ void join_four(uint4 (&x)[4], const uint2& rest) const {
    constexpr bool kBack = kWord >= 2;
    // words of the other aligned vector: its last two, its last, its first or its first two
    constexpr bool kTwo = kWord == 2 || (kWord == 1 && sizeof(T) == 2);
    if constexpr (kWord == 0 && sizeof(T) == 4) return;
    const int lane = threadIdx.x & 31, bits = mis * static_cast<int>(sizeof(T)) % 4 * 8;
    const int from = kBack ? (lane + 31) & 31 : (lane + 1) & 31;
    const bool turn = lane == (kBack ? 31 : 0);  // gives a word of the vector behind (before)
    const bool end = lane == (kBack ? 0 : 31);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int v = kBack ? 3 - u : u, next = kBack ? max(v - 1, 0) : min(v + 1, 3);
      uint32_t far = kBack ? (turn ? x[next].w : x[v].w) : (turn ? x[next].x : x[v].x), farther = 0;
      far = __shfl_sync(0xffffffffu, far, from);
      if (kTwo) farther = __shfl_sync(0xffffffffu, kBack ? (turn ? x[next].z : x[v].z) : (turn ? x[next].y : x[v].y), from);
      if (u == 3 && end) {
        far = kBack ? rest.y : rest.x;
        farther = kBack ? rest.x : rest.y;
      }
      const uint4 o = x[v];
      if constexpr (kWord == 0)
        x[v] = make_uint4(join<0>(o.x, o.y, bits), join<0>(o.y, o.z, bits), join<0>(o.z, o.w, bits), join<0>(o.w, far, bits));
      else if constexpr (kWord == 1)
        x[v] = make_uint4(join<1>(o.y, o.z, bits), join<1>(o.z, o.w, bits), join<1>(o.w, far, bits),
                          join<1>(far, farther, bits));
      else if constexpr (kWord == 2)
        x[v] = make_uint4(join<2>(farther, far, bits), join<2>(far, o.x, bits), join<2>(o.x, o.y, bits),
                          join<2>(o.y, o.z, bits));
      else
        x[v] = make_uint4(join<3>(far, o.x, bits), join<3>(o.x, o.y, bits), join<3>(o.y, o.z, bits),
                          join<3>(o.z, o.w, bits));
    }
  }
  // Turns what load_four loaded into the vectors themselves.
  __device__ __forceinline__ void finish_four(uint4 (&x)[4], const uint2& rest, int four) const {
    if (mis == 0) return;
    switch (word()) {
      case 0: join_four<0>(x, rest); break;
      case 1: join_four<1>(x, rest); break;
      case 2: join_four<2>(x, rest); break;
      default: join_four<3>(x, rest); break;
    }
    if (whole(four)) return;
    const int i0 = at(four, 0, static_cast<int>(threadIdx.x));
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (i0 + v * 32 < low || i0 + v * 32 >= live) x[v] = make_uint4(kFill, kFill, kFill, kFill);
  }
  __device__ __forceinline__ uint4 load_edge(int64_t w) const {
    uint32_t word[4] = {kFill, kFill, kFill, kFill};
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int64_t i = w * kPer + e;
      if (i >= n) continue;
      if constexpr (sizeof(T) == 4)
        word[e] = __float_as_uint(row[i]);
      else
        word[e / 2] = e & 1 ? (word[e / 2] & 0xffffu) | (static_cast<uint32_t>(row[i]) << 16)
                            : (word[e / 2] & 0xffff0000u) | row[i];
    }
    return make_uint4(word[0], word[1], word[2], word[3]);
  }
  // Elementwise larger (NaN is the largest), two bf16 at a time.
  static __device__ __forceinline__ uint4 larger(const uint4& a, const uint4& b) {
    return make_uint4(larger(a.x, b.x), larger(a.y, b.y), larger(a.z, b.z), larger(a.w, b.w));
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) return __float_as_uint(fmax_nan(__uint_as_float(a), __uint_as_float(b)));
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ float largest(const uint4& x) {
    const uint32_t w = larger(larger(x.x, x.y), larger(x.z, x.w));
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    return fmax_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  // A float's bits (exact in T) as the word reaches() compares with.
  static __device__ __forceinline__ uint32_t bits(uint32_t f) {
    return sizeof(T) == 4 ? f : (f & 0xffff0000u) | (f >> 16);
  }
  // Whether an element (none of them NaN) is at least `least`.
  static __device__ __forceinline__ bool reaches(const uint4& x, uint32_t least) {
    const uint32_t w = larger(larger(x.x, x.y), larger(x.z, x.w));
    if constexpr (sizeof(T) == 4) return __uint_as_float(w) >= __uint_as_float(least);
    uint32_t d;
    asm("set.ge.u32.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(least));
    return d != 0;
  }
  static __device__ __forceinline__ float value(const uint4& x, int e) {
    const int i = e * static_cast<int>(sizeof(T)) / 4;
    const uint32_t w = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
  }
};

__device__ __forceinline__ void beam_push(BeamShared& sh, uint32_t key, int64_t i) {
  const int at = atomicAdd(&sh.count, 1);
  if (at < kBeamCap) sh.gathered[at] = pack(key, static_cast<uint32_t>(i));
}

// Exactly the k best of the piece into sh.gathered: the bound bisected over
// keys (the largest that k elements reach), then over the indices of the
// elements that equal it.  Reads the piece again for every step.
template <typename T>
__device__ __noinline__ void beam_bisect(BeamShared* shp, const T* row, int64_t n, int piece, int pieces, int k) {
  BeamShared& sh = *shp;
  const BeamPiece<T> p(row, n, piece, pieces);
  auto each = [&](auto&& f) {
    const int vectors = static_cast<int>(p.w1 - p.w0);
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < vectors + static_cast<int>(threadIdx.x); i0 += 4 * kBeamThreads) {
      uint4 x[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int i = i0 + v * kBeamThreads;
        x[v] = i < vectors && p.edge(p.w0 + i) ? p.load_edge(p.w0 + i) : p.load(i);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int e = 0; e < p.kPer; ++e) f(beam_key(p.value(x[v], e)), p.index(i0 + v * kBeamThreads) + e);
    }
  };
  uint32_t lo = 1, hi = 0xffffffffu;
  while (lo < hi) {
    const uint32_t mid = lo + ((hi - lo) >> 1) + 1;
    int c = 0;
    each([&](uint32_t key, int64_t) { c += key >= mid; });
    if (block_total(c, &sh.total) >= k)
      lo = mid;
    else
      hi = mid - 1;
  }
  int c = 0;
  each([&](uint32_t key, int64_t) { c += key > lo; });
  const int equal = k - block_total(c, &sh.total);
  int64_t a = 0, b = n - 1;
  while (a < b) {
    const int64_t mid = (a + b) >> 1;
    c = 0;
    each([&](uint32_t key, int64_t i) { c += key == lo && i <= mid; });
    if (block_total(c, &sh.total) >= equal)
      b = mid;
    else
      a = mid + 1;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  each([&](uint32_t key, int64_t i) {
    if (key > lo || (key == lo && i <= a)) beam_push(sh, key, i);
  });
  __syncthreads();
}

// Calls use(i, rank) for every i < n with the number of j that above(j, i)
// holds for: four lanes count a quarter each.
template <typename Above, typename Use>
__device__ __forceinline__ void beam_rank(int n, Above&& above, Use&& use) {
  const int q = threadIdx.x & 3;
  for (int i0 = 0; i0 < n; i0 += kBeamThreads / 4) {
    const int i = i0 + static_cast<int>(threadIdx.x >> 2);
    int r = 0;
    if (i < n) {
#pragma unroll 4
      for (int j = q; j < n; j += 4) r += above(j, i);
    }
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    r += __shfl_xor_sync(0xffffffffu, r, 2);
    if (i < n && q == 0) use(i, r);
  }
}

// The k best continuations of sentence blockIdx.x of the launch, from its rows'
// sums and lists.
__global__ void __launch_bounds__(kBeamThreads) beam_finish_kernel(BeamArgs p) {
  __shared__ BeamShared sh;
  pdl_wait_then_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t local = blockIdx.x;
  const int64_t b = p.first + local;
  const float ninf = __int_as_float(0xff800000);
  const BeamSum* sums = p.sums + local * p.beams * p.pieces;
  const uint64_t* lists = p.lists + local * p.beams * p.pieces * p.k;
  const int total = p.beams * p.pieces * p.k, per_beam = p.k * p.pieces;
  // The first candidates of every thread stay in registers; their loads are in
  // flight with those of the sums.
  constexpr int kHeld = 8;
  uint64_t held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = tid + i * kBeamThreads;
    held[i] = c < total ? __ldcg(lists + c) : 0ull;
  }
  for (int i = warp; i < p.beams; i += kBeamThreads / 32) {
    uint32_t top = 0;
    double sum = 0.0;
    int r = 0;            // of `sum`: 2^r is its unit
    bool by_max = false;  // some piece's sum is relative to its maximum
    const float score = __ldg(p.scores + b * p.beams + i);
    for (int j0 = 0; j0 < p.pieces; j0 += 32) {
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (j0 + lane < p.pieces) raw = __ldcg(reinterpret_cast<const uint4*>(sums + i * p.pieces + j0 + lane));
      const double x = __hiloint2double(static_cast<int>(raw.y), static_cast<int>(raw.x));
      const int rj = static_cast<int>(raw.w);
      top = max(top, __reduce_max_sync(0xffffffffu, raw.z));
      by_max |= __any_sync(0xffffffffu, raw.z && rj == kBeamByMax);
      const int now = max(j0 ? r : kBeamByMax, __reduce_max_sync(0xffffffffu, raw.z ? rj : kBeamByMax));
      // Differences beyond 1100 leave nothing of a sum below 2^32.  No piece so
      // far, or one by its maximum, has no r to subtract from.
      auto down = [now](int from) { return from == kBeamByMax ? -1100 : max(from - now, -1100); };
      if (j0) sum = scalbn(sum, down(r));
      if (raw.z) sum += scalbn(x, down(rj));
      r = now;
    }
    const bool bad = top >= 0xff800000u;  // +inf or NaN
    const double m = top ? static_cast<double>(key_value(top)) : 0.0;
    constexpr double kLn2 = 0.6931471805599453;
    if (by_max && !bad) {
      sum = 0.0;
      for (int j = lane; j < p.pieces; j += 32) {
        const uint4 raw = __ldcg(reinterpret_cast<const uint4*>(sums + i * p.pieces + j));
        const double x = __hiloint2double(static_cast<int>(raw.y), static_cast<int>(raw.x));
        const int rj = static_cast<int>(raw.w);
        if (raw.z) sum += x * exp((rj == kBeamByMax ? static_cast<double>(key_value(raw.z)) : rj * kLn2) - m);
      }
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (lane == 0) {
      // L (1 + e) = log2 e: the terms' exponents are short by e x, all but
      // e (x - m) of which is given back here.
      constexpr double kShort = 1.4426950408889634 / static_cast<double>(kBeamLog2e) - 1.0;
      const double lse = by_max ? m + log(sum) : r * kLn2 + log(sum) + kShort * m;
      sh.off[i] = bad ? __longlong_as_double(0x7ff8000000000000ll) : static_cast<double>(score) - lse;
    }
  }
  if (tid == 0) sh.count = 0;
  __syncthreads();
  // Bound and gather on the values rounded down to float (the order is kept,
  // equal ones stay candidates).
  auto value = [&](int c, uint64_t e) { return sh.off[c / per_beam] + static_cast<double>(key_value(packed_key(e))); };
  auto low_key = [&](double v) { return order_key(__double2float_rd(v)); };
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (held[i]) mine = max(mine, low_key(value(tid + i * kBeamThreads, held[i])));
  for (int c = tid + kHeld * kBeamThreads; c < total; c += kBeamThreads) {
    const uint64_t e = __ldcg(lists + c);
    if (e) mine = max(mine, low_key(value(c, e)));
  }
  // The k-th largest of the threads' maxima, to 16 bits: beams differ in score,
  // so the bound of the weakest warp would let most candidates through.
  uint32_t bound = 0;
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t trial = bound | (1u << bit);
    if (__syncthreads_count(mine >= trial) >= p.k) bound = trial;
  }
  bound = max(bound, 1u);
  auto gather = [&](int c, uint64_t e) {
    const double v = value(c, e);
    if (low_key(v) < bound) return;
    const int at = atomicAdd(&sh.count, 1);
    if (at >= kBeamCap) return;
    sh.cont.value[at] = order_key64(v);
    sh.cont.rest[at] = (static_cast<uint64_t>(~static_cast<uint32_t>(c / per_beam)) << 32) | packed_key(e);
    sh.cont.token[at] = packed_idx(e);
  };
  if (mine >= bound) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (held[i]) gather(tid + i * kBeamThreads, held[i]);
    for (int c = tid + kHeld * kBeamThreads; c < total; c += kBeamThreads) {
      const uint64_t e = __ldcg(lists + c);
      if (e) gather(c, e);
    }
  }
  __syncthreads();
  const int m = sh.count;
  auto write = [&](int64_t o, const Cont& c) {
    const int i = static_cast<int>(~static_cast<uint32_t>(c.rest >> 32));
    p.out_scores[o] = static_cast<float>(sh.off[i] + static_cast<double>(key_value(static_cast<uint32_t>(c.rest))));
    p.out_parent[o] = i;
    p.out_token[o] = static_cast<int32_t>(c.token);
  };
  int done = min(m, p.k);
  if (m <= kBeamCap) {
    auto cont = [&](int i) { return Cont{sh.cont.value[i], sh.cont.rest[i], sh.cont.token[i]}; };
    beam_rank(
        m, [&](int j, int i) { return ranks_above(cont(j), cont(i)); },
        [&](int i, int r) {
          if (r < p.k) write(b * p.k + r, cont(i));
        });
  } else {
    // Too many near-equal values: one round over the lists per continuation (128
    // beams, k 128: 14 ms; 16 beams of equal logits, k 32: 0.6 ms).
    Cont last = {~0ull, ~0ull, 0};
    for (done = 0; done < p.k; ++done) {
      Cont top = {0, 0, 0};
      for (int c = tid; c < total; c += kBeamThreads) {
        const uint64_t e = __ldcg(lists + c);
        if (!e) continue;
        const Cont x = {order_key64(value(c, e)),
                        (static_cast<uint64_t>(~static_cast<uint32_t>(c / per_beam)) << 32) | packed_key(e),
                        packed_idx(e)};
        if ((done == 0 || ranks_above(last, x)) && ranks_above(x, top)) top = x;
      }
#pragma unroll
      for (int x = 16; x; x >>= 1) {
        const Cont y = {__shfl_xor_sync(0xffffffffu, top.value, x), __shfl_xor_sync(0xffffffffu, top.rest, x),
                        __shfl_xor_sync(0xffffffffu, top.token, x)};
        if (ranks_above(y, top)) top = y;
      }
      if (lane == 0) sh.best[warp] = top;
      __syncthreads();
      last = sh.best[0];
      for (int w = 1; w < kBeamThreads / 32; ++w)
        if (ranks_above(sh.best[w], last)) last = sh.best[w];
      __syncthreads();
      if (last.value == 0) break;
      if (tid == 0) write(b * p.k + done, last);
    }
  }
  for (int r = done + tid; r < p.k; r += kBeamThreads) {
    p.out_scores[b * p.k + r] = ninf;
    p.out_parent[b * p.k + r] = -1;
    p.out_token[b * p.k + r] = -1;
  }
}

// The elements of the vectors set aside that reach the bound.  All threads.
template <typename T>
__device__ __forceinline__ void beam_gather(BeamShared& sh, uint32_t bound) {
  constexpr int kPer = BeamPiece<T>::kPer;
  const int n = min(sh.hits, kBeamHits) * kPer;
  for (int i = threadIdx.x; i < n; i += kBeamThreads) {
    const uint32_t key = beam_key(logit_value(reinterpret_cast<const T*>(sh.hit)[i]));
    if (key >= bound) beam_push(sh, key, sh.hit_at[i / kPer] + i % kPer);
  }
}

// The piece's list (its k best of those gathered) and sum.  All threads.
__device__ __forceinline__ void beam_piece_end(const BeamShared& sh, const BeamArgs& p, uint32_t top, int r) {
  uint64_t* list = p.lists + static_cast<int64_t>(blockIdx.x) * p.k;
  const int found = sh.count;
  beam_rank(
      found, [&](int j, int i) { return sh.gathered[j] > sh.gathered[i]; },
      [&](int i, int above) {
        if (above < p.k) list[above] = sh.gathered[i];
      });
  for (int i = found + static_cast<int>(threadIdx.x); i < p.k; i += kBeamThreads) list[i] = 0;
  if (threadIdx.x == 0) {
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kBeamThreads / 32; ++w) t += sh.part[w];
    p.sums[blockIdx.x] = BeamSum{t, top, r};
  }
}

// The piece of a beam that has ended.
__device__ __forceinline__ void beam_piece_ended(const BeamArgs& p) {
  if (threadIdx.x == 0) p.sums[blockIdx.x] = BeamSum{0.0, 0u, 0};
  for (int i = threadIdx.x; i < p.k; i += kBeamThreads) p.lists[static_cast<int64_t>(blockIdx.x) * p.k + i] = 0;
}

// Grid of both kernels: sentence-major, then beam, then piece.
template <typename T>
__global__ void __launch_bounds__(kBeamThreads, 2) topk_beam_held_kernel(BeamArgs p) {
  constexpr int kPer = BeamPiece<T>::kPer;
  __shared__ BeamShared sh;
  pdl_wait_then_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t row = blockIdx.x / static_cast<uint32_t>(p.pieces);  // of the launch
  const int piece = static_cast<int>(blockIdx.x - row * p.pieces);
  const float ninf = __int_as_float(0xff800000);
  if (tid == 0) sh.count = sh.hits = 0;
  if (__ldg(p.scores + p.first * p.beams + row) == ninf) {
    beam_piece_ended(p);
  } else {
    const T* row_x = static_cast<const T*>(p.logits) + (p.first * p.beams + row) * p.n;
    const BeamPiece<T> pc(row_x, p.n, piece, p.pieces);
    // (vectors that no lane of the warp has are passed over)
    auto any = [&](int v) { return pc.at(v / 4, v % 4, tid & ~31) < pc.live; };
    uint4 x[kBeamVectors / 4][4];
    uint2 rest[kBeamVectors / 4];
    const uint4* first = pc.source() + pc.at(0);
#pragma unroll
    for (int f = 0; f < kBeamVectors / 4; ++f) pc.load_four(x[f], rest[f], first, f);
    uint4 edge = make_uint4(pc.kFill, pc.kFill, pc.kFill, pc.kFill);
    const int64_t edge_at = pc.edge_of(tid);
    if (edge_at >= 0) edge = pc.load_edge(edge_at);
#pragma unroll
    for (int f = 0; f < kBeamVectors / 4; ++f)
      if (4 * f * kBeamThreads < pc.live) pc.finish_four(x[f], rest[f], f);
    // largest element of the thread (NaN counts as the largest), and the bound
    uint4 y = edge;
#pragma unroll
    for (int v = 0; v < kBeamVectors; ++v)
      if (any(v)) y = pc.larger(y, x[v / 4][v % 4]);
    const float top = pc.largest(y);
    const uint32_t mine = beam_key(top);
    const uint32_t warp_top = __reduce_max_sync(0xffffffffu, mine);
    if (lane == 0) sh.warp_tops[warp] = warp_top;
    const uint32_t bound = max(beam_bound(mine, p.k, sh.warp_keys), 1u);
    uint32_t key_top = 0;  // the piece's maximum
#pragma unroll
    for (int w = 0; w < kBeamThreads / 32; ++w) key_top = max(key_top, sh.warp_tops[w]);
    // The sum of 2^(x L - r): one fused multiply-add and one exponential a
    // logit.  L's rounding moves the exponent of a term by 2^-26 of x log2 e, of
    // which the part common to all terms is taken out at the end.  Vectors that
    // reach the bound are set aside, and their elements then looked at by all
    // threads.
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int r = 0;
    bool gathered = false;
    const float m = key_top ? key_value(key_top) : 0.0f;
    if (key_top >= 0xff800000u) {  // a NaN or +inf: no sum
    } else if (fabsf(m) > 1e6f) {  // x L would be off by more than a fraction of 1
      r = kBeamByMax;
#pragma unroll 1
      for (int v = 0; v <= kBeamVectors; ++v) {
        const uint4 z = v < kBeamVectors ? pc.load(pc.at(v)) : edge;
#pragma unroll
        for (int e = 0; e < kPer; ++e) sum[e & 3] += exp2_ftz((pc.value(z, e) - m) * kBeamLog2e);
      }
    } else if (key_top) {
      gathered = true;
      const uint32_t least = pc.bits(bound == 1u ? 0xff7fffffu : __float_as_uint(key_value(bound)));
      const float rf = rintf(m * kBeamLog2e);
      r = static_cast<int>(rf);
      auto add = [&](const uint4& z, int64_t i) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) sum[e & 3] += exp2_ftz(fmaf(pc.value(z, e), kBeamLog2e, -rf));
        if (pc.reaches(z, least)) {
          const int at = atomicAdd(&sh.hits, 1);
          if (at < kBeamHits) {
            sh.hit[at] = z;
            sh.hit_at[at] = static_cast<int>(i);
          }
        }
      };
#pragma unroll
      for (int v = 0; v < kBeamVectors; ++v)
        if (any(v)) add(x[v / 4][v % 4], pc.index(pc.at(v)));
      if (edge_at >= 0) add(edge, edge_at * kPer);
      __syncthreads();
      beam_gather<T>(sh, bound);
    }
    float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sh.part[warp] = s;
    __syncthreads();
    if (key_top && (!gathered || sh.hits > kBeamHits || sh.count > kBeamCap)) beam_bisect(&sh, row_x, p.n, piece, p.pieces, p.k);
    beam_piece_end(sh, p, key_top, r);
  }
}

// sum * 2^d for a whole number d <= 0; nothing is left below 2^-126, not of an
// infinite sum either (of logits so large that x L - r is a rounding error).  A
// larger d is that of an empty sum.
__device__ __forceinline__ float beam_shrink(float sum, float d) {
  return d >= -126.0f && d <= 0.0f ? sum * __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(d)) << 23) : 0.0f;
}

template <typename T>
__global__ void __launch_bounds__(kBeamThreads, kBeamCtasPerSm) topk_beam_stream_kernel(BeamArgs p) {
  using Piece = BeamPiece<T>;
  constexpr int kPer = Piece::kPer;
  __shared__ BeamShared sh;
  __shared__ float batch_top[kBeamBatches * kBeamThreads];  // a thread's own
  pdl_wait_then_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float ninf = __int_as_float(0xff800000);
  if (tid == 0) sh.count = sh.hits = sh.batches = 0;
  auto piece_of = [&](uint32_t block) {
    const uint32_t row = block / static_cast<uint32_t>(p.pieces);  // of the launch
    return Piece(static_cast<const T*>(p.logits) + (p.first * p.beams + row) * p.n, p.n,
                 static_cast<int>(block - row * p.pieces), p.pieces);
  };
  auto edge_of = [&](const Piece& pc) {
    const int64_t w = pc.edge_of(tid);
    return w >= 0 ? pc.load_edge(w) : make_uint4(pc.kFill, pc.kFill, pc.kFill, pc.kFill);
  };
  const float score = __ldg(p.scores + p.first * p.beams + blockIdx.x / static_cast<uint32_t>(p.pieces));
  const Piece pass = piece_of(blockIdx.x);

  // One pass: the thread's largest element (NaN counts as the largest), that of
  // each batch, and the sum of 2^(x L - r).  L's rounding moves the exponent of
  // a term by 2^-26 of x log2 e, of which the part common to all terms is taken
  // out at the end.  r is the whole number near the largest x L of the batch that
  // last passed `lift`, one logit above the one before: exponents stay below 2.
  float top = ninf, sum = 0.0f, rf = 0.0f, lift = ninf;
  auto raise = [&](float largest) {
    top = fmax_nan(top, largest);
    if (largest > lift) {
      const float to = rintf(largest * kBeamLog2e);
      sum = beam_shrink(sum, rf - to);
      rf = to;
      lift = largest + 1.0f;
    }
  };
  auto add = [&](float (&part)[4], const uint4& z) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) part[e & 3] += exp2_ftz(fmaf(Piece::value(z, e), kBeamLog2e, -rf));
  };
  const int batches = (pass.live + kBeamBatch * kBeamThreads - 1) / (kBeamBatch * kBeamThreads);
  auto take = [&](const uint4 (&x)[kBeamBatch], int b) {
    uint4 y = x[0];
#pragma unroll
    for (int v = 1; v < kBeamBatch; ++v) y = Piece::larger(y, x[v]);
    const float largest = Piece::largest(y);
    batch_top[b * kBeamThreads + tid] = largest;
    raise(largest);
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < kBeamBatch; ++v)
      if (pass.at(b, v, tid & ~31) < pass.live) add(part, x[v]);
    sum += (part[0] + part[1]) + (part[2] + part[3]);
  };
  static_assert(kBeamBatch == 4, "a batch is four vectors of a lane");
  uint4 x[kBeamBatch], z[kBeamBatch];
  uint2 x_rest, z_rest;
  const uint4* first = pass.source() + pass.at(0);
  pass.load_four(x, x_rest, first, 0);  // not waiting for the score
  if (score == ninf) {
    beam_piece_ended(p);
    return;
  }
  if (pass.edge_of(tid) >= 0) {
    const uint4 edge = edge_of(pass);
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    raise(Piece::largest(edge));
    add(part, edge);
    sum = (part[0] + part[1]) + (part[2] + part[3]);
  }
#pragma unroll 1
  for (int b = 0; b < batches; b += 2) {
    pass.load_four(z, z_rest, first, b + 1);
    pass.finish_four(x, x_rest, b);
    take(x, b);
    if (b + 1 >= batches) break;
    pass.load_four(x, x_rest, first, b + 2);
    pass.finish_four(z, z_rest, b + 1);
    take(z, b + 1);
  }

  // The piece once more: what the loop above does not need of it holds no registers there.
  uint32_t block = blockIdx.x;
  asm volatile("" : "+r"(block));
  const Piece pc = piece_of(block);
  const int64_t edge_at = pc.edge_of(tid);
  const uint32_t mine = beam_key(top);
  const uint32_t warp_top = __reduce_max_sync(0xffffffffu, mine);
  if (lane == 0) sh.warp_tops[warp] = warp_top;
  uint32_t bound = max(beam_bound(mine, p.k, sh.warp_keys), 1u);
  uint32_t key_top = 0;  // the piece's maximum
#pragma unroll
  for (int w = 0; w < kBeamThreads / 32; ++w) key_top = max(key_top, sh.warp_tops[w]);
  int r = 0;
  const float m = key_top ? key_value(key_top) : 0.0f;
  if (key_top >= 0xff800000u) {  // a NaN or +inf: no sum
    sum = 0.0f;
  } else if (fabsf(m) > 1e6f) {  // x L would be off by more than a fraction of 1
    r = kBeamByMax;
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int v = 0; v <= batches * kBeamBatch; ++v) {
      const uint4 y = v < batches * kBeamBatch ? pc.load(pc.at(v)) : edge_of(pc);
#pragma unroll
      for (int e = 0; e < kPer; ++e) part[e & 3] += exp2_ftz((pc.value(y, e) - m) * kBeamLog2e);
    }
    sum = (part[0] + part[1]) + (part[2] + part[3]);
  } else {
    const float to = rintf(m * kBeamLog2e);
    r = static_cast<int>(to);
    sum = beam_shrink(sum, rf - to);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sh.part[warp] = sum;

  // Vectors that reach the bound are set aside, from batches that do, which are
  // read again by a thread per vector (a piece's only batch is still there).
  auto set_aside = [&](const uint4& y, int64_t i) {
    if (beam_key(pc.largest(y)) < bound) return;
    const int at = atomicAdd(&sh.hits, 1);
    if (at >= kBeamHits) return;
    sh.hit[at] = y;
    sh.hit_at[at] = static_cast<int>(i);
  };
  bool over;
  for (bool again = false;; again = true) {
    if (mine >= bound) {
      if (batches <= 1) {
#pragma unroll
        for (int v = 0; v < kBeamBatch; ++v) set_aside(x[v], pc.index(pc.at(v)));
      } else {
        for (int b = 0; b < batches; ++b)
          if (beam_key(batch_top[b * kBeamThreads + tid]) >= bound) {
            const int at = atomicAdd(&sh.batches, 1);
            if (at < kBeamHits) sh.batch[at] = b * kBeamThreads + tid;
          }
      }
      if (edge_at >= 0) set_aside(edge_of(pc), edge_at * kPer);
    }
    __syncthreads();
    if (batches > 1) {
      const int n = min(sh.batches, kBeamHits) * kBeamBatch;
      for (int i = tid; i < n; i += kBeamThreads) {
        const int batch = sh.batch[i / kBeamBatch];
        const int at = pc.at(batch / kBeamThreads, i % kBeamBatch, batch % kBeamThreads);
        set_aside(pc.load(at), pc.index(at));
      }
      __syncthreads();
    }
    beam_gather<T>(sh, bound);
    __syncthreads();
    over = sh.batches > kBeamHits || sh.hits > kBeamHits || sh.count > kBeamCap;
    if (again || !over) break;
    // Too many (logits in falling order, say): the k-th largest of the threads'
    // maxima itself, to 16 bits.
    uint32_t tight = 0;
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t trial = tight | (1u << bit);
      if (__syncthreads_count(mine >= trial) >= p.k) tight = trial;
    }
    bound = max(bound, tight);
    if (tid == 0) sh.count = sh.hits = sh.batches = 0;
    __syncthreads();
  }
  if (over) beam_bisect(&sh, pc.row, p.n, static_cast<int>(block % static_cast<uint32_t>(p.pieces)), p.pieces, p.k);
  beam_piece_end(sh, p, key_top, r);
}

// ---------------------------------------------------------------- reordering
// A copy of rows, bound by memory: every kept row is read and written once.
// Rows may start at any byte.  The body of a row is written in 16-byte vectors
// on 16-byte addresses; where the source lies s bytes off such addresses, each
// vector is shifted together from the two aligned ones that hold it (both
// inside the row; the second is the next lane's first and comes from L1).
// The up to 31 bytes before the body and 47 behind it are copied singly.
// Measured: 8 tensors of 16 rows of 4 MB: 158 us, 6.8 TB/s (rows read twice come
// from L2 the second time).
constexpr int kReorderStates = 64;  // tensors per launch
constexpr int kReorderThreads = 256;
constexpr int kReorderUnroll = 8;
constexpr int64_t kReorderChunk = kReorderThreads * kReorderUnroll * 16;  // bytes of a long row per item
constexpr int64_t kReorderShort = 4096;  // rows up to this long go to one warp each

struct ReorderArgs {
  const unsigned char* src[kReorderStates];  // [batch][beams][row_bytes]
  unsigned char* dst[kReorderStates];        // [batch][k][row_bytes]
  int64_t row_bytes[kReorderStates];
  int64_t end[kReorderStates];  // items of the tensors up to and with this one
  const int32_t* parents;       // [batch][k]
  int64_t rows;                 // batch * k
  int count, beams, k;
};

// Items (one CTA each) of a tensor: eight short rows, or a chunk of a long one.
__host__ __device__ inline int64_t reorder_items(int64_t rows, int64_t row_bytes) {
  if (row_bytes <= kReorderShort) return (rows + kReorderThreads / 32 - 1) / (kReorderThreads / 32);
  return rows * ((row_bytes + kReorderChunk - 1) / kReorderChunk);
}

// Vectors [v0, v1) of a row's body and, where `edges`, the bytes around the
// body, by `width` threads of which this is `id`.  src null: zeros.
__device__ __forceinline__ void copy_row(unsigned char* dst, const unsigned char* src, int64_t bytes, int64_t v0,
                                         int64_t v1, bool edges, int id, int width) {
  int64_t head = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(dst) & 15)) & 15);
  const int s = src ? static_cast<int>((reinterpret_cast<uintptr_t>(src) + head) & 15) : 0;
  if (s > head) head += 16;
  int64_t body = s ? (bytes - head + s) / 16 - 1 : (bytes - head) / 16;  // vectors whose sources lie in the row
  if (bytes < head || body < 0) body = 0;
  v1 = v1 < body ? v1 : body;
  uint4* d = reinterpret_cast<uint4*>(dst + head);
  const uint4* a = reinterpret_cast<const uint4*>(src + head - s);
  for (int64_t i = v0 + id; i < v1; i += static_cast<int64_t>(width) * kReorderUnroll) {
    uint4 x[kReorderUnroll];
#pragma unroll
    for (int u = 0; u < kReorderUnroll; ++u) {
      const int64_t j = i + static_cast<int64_t>(u) * width;
      x[u] = make_uint4(0, 0, 0, 0);
      if (src && j < v1) x[u] = __ldg(a + j);
    }
    if (s) {
#pragma unroll
      for (int u = 0; u < kReorderUnroll; ++u) {
        const int64_t j = i + static_cast<int64_t>(u) * width;
        if (j < v1) x[u] = shift_together(x[u], __ldg(a + j + 1), s);
      }
    }
#pragma unroll
    for (int u = 0; u < kReorderUnroll; ++u) {
      const int64_t j = i + static_cast<int64_t>(u) * width;
      if (j < v1) __stcs(d + j, x[u]);
    }
  }
  if (edges) {
    const int64_t behind = body ? head + body * 16 : 0;  // without a body: the whole row
    const int64_t before = body ? head : 0;
    for (int64_t i = id; i < before; i += width) dst[i] = src ? src[i] : 0;
    for (int64_t i = behind + id; i < bytes; i += width) dst[i] = src ? src[i] : 0;
  }
}

__global__ void __launch_bounds__(kReorderThreads) beam_reorder_kernel(ReorderArgs p) {
  pdl_wait_then_release();
  for (int64_t item = blockIdx.x; item < p.end[p.count - 1]; item += gridDim.x) {
    int t = 0;
    while (item >= p.end[t]) ++t;
    int64_t i = item - (t ? p.end[t - 1] : 0);
    const int64_t bytes = p.row_bytes[t];
    int64_t r, chunk = 0;
    int id = threadIdx.x, width = kReorderThreads;
    if (bytes <= kReorderShort) {
      r = i * (kReorderThreads / 32) + threadIdx.x / 32;
      id = threadIdx.x & 31;
      width = 32;
      if (r >= p.rows) continue;
    } else {
      const int64_t chunks = (bytes + kReorderChunk - 1) / kReorderChunk;
      r = i / chunks;
      chunk = i - r * chunks;
    }
    const int32_t parent = __ldg(p.parents + r);
    const bool live = parent >= 0 && parent < p.beams;
    if (!live && parent != -1) atomicOr(&g_device_status, 2);
    const unsigned char* src = live ? p.src[t] + (r / p.k * p.beams + parent) * bytes : nullptr;
    copy_row(p.dst[t] + r * bytes, src, bytes, chunk * (kReorderChunk / 16), (chunk + 1) * (kReorderChunk / 16),
             chunk == 0, id, width);
  }
}

}  // namespace tk
