// decode_api.cu -- C ABI of the operators of a decoding step around the
// selections: the paged cache, attention over it, and beam search.  A
// translation unit of its own, compiled next to topk_api.cu.

// common.cuh defines the status word and the self-test kernel with external
// linkage for topk_api.cu; in this unit they get names of their own.
#define g_device_status g_decode_device_status
#define wait_timeout_probe decode_wait_timeout_probe

#include <algorithm>
#include <cmath>

#include "beam.cuh"
#include "kv_cache.cuh"
#include "launch.cuh"
#include "paged_attention.cuh"

namespace tk {

namespace {

// The part of a workspace that is zero between calls, of every operator.
constexpr size_t kTicketBytes = TOPK_DECODE_TICKET_BYTES;
static_assert(kTicketBytes >= 12 * kAttendMaxCtas, "tickets");

constexpr int kMaxReorder = 256;
constexpr int64_t kMaxGridX = 2147483647LL;

bool cache_head_dim(int d) { return d == 64 || d == 128 || d == 256; }

// Checks a cache description and builds the device view.
int cache_view(const topk_cache* c, CacheView* v) {
  if (!c || !c->data) return TOPK_EINVAL;
  if (c->pages < 1 || c->kv_heads < 1 || c->page_size < 1 || c->d < 1) return TOPK_EINVAL;
  if (c->type != TOPK_CACHE_BF16 && c->type != TOPK_CACHE_E4M3) return TOPK_EINVAL;
  if (!cache_head_dim(c->d)) return TOPK_EUNSUPPORTED;
  if (c->pages > kMaxN) return TOPK_EUNSUPPORTED;  // page numbers are int32
  if (c->kv_heads > (1 << 20)) return TOPK_EUNSUPPORTED;
  const int64_t esz = c->type == TOPK_CACHE_BF16 ? 2 : 1;
  if (!aligned16(c->data)) return TOPK_EINVAL;
  const int64_t strides[3] = {c->page_stride, c->head_stride, c->token_stride};
  for (int64_t s : strides)
    if (s < 0 || s > kMaxElems || (s * esz) % 16 != 0) return TOPK_EINVAL;
  if (c->type == TOPK_CACHE_E4M3) {
    if (!c->scale || (reinterpret_cast<uintptr_t>(c->scale) & 3u)) return TOPK_EINVAL;
    const int64_t ss[3] = {c->scale_page_stride, c->scale_head_stride, c->scale_token_stride};
    for (int64_t s : ss)
      if (s < 0 || s > kMaxElems) return TOPK_EINVAL;
  }
  v->data = static_cast<unsigned char*>(c->data);
  v->scale = c->type == TOPK_CACHE_E4M3 ? c->scale : nullptr;
  v->page_stride = c->page_stride * esz;
  v->head_stride = c->head_stride * esz;
  v->token_stride = c->token_stride * esz;
  v->s_page_stride = c->scale_page_stride;
  v->s_head_stride = c->scale_head_stride;
  v->s_token_stride = c->scale_token_stride;
  v->pages = c->pages;
  v->kv_heads = c->kv_heads;
  v->page_size = c->page_size;
  // t / page_size for t < 2^31 by a multiplication: 2^shift / page_size rounded up, shift = 31 + ceil(log2 page_size)
  v->page_shift = 31;
  while ((int64_t{1} << (v->page_shift - 31)) < c->page_size) ++v->page_shift;
  v->page_magic = static_cast<uint32_t>(((static_cast<unsigned __int128>(1) << v->page_shift) + c->page_size - 1) /
                                        static_cast<unsigned>(c->page_size));
  return TOPK_OK;
}

bool same_shape(const topk_cache* a, const topk_cache* b) {
  return a->pages == b->pages && a->kv_heads == b->kv_heads && a->page_size == b->page_size && a->d == b->d &&
         a->type == b->type;
}

int table_view(const int32_t* table, int64_t stride, int width, const int32_t* lens, int64_t batch, int page_size,
               TableView* t) {
  if (!table || !lens) return TOPK_EINVAL;
  if (batch < 1 || width < 1 || stride < 0 || stride > kMaxElems) return TOPK_EINVAL;
  if (batch > kMaxN) return TOPK_EUNSUPPORTED;
  t->table = table;
  t->lens = lens;
  t->stride = stride;
  t->capacity = std::min(static_cast<int64_t>(width) * page_size, kMaxN);
  t->batch = static_cast<int>(batch);
  return TOPK_OK;
}

// CTAs of the attention's line: all that are resident at once.  The workspace
// is sized for three per SM, the most any instantiation has.
constexpr int kAttendCtasPerSm = 3;

size_t attend_workspace(int d, const DeviceInfo& dev) {
  const int ctas = std::min(dev.sms * kAttendCtasPerSm, kAttendMaxCtas);
  return kTicketBytes + static_cast<size_t>(ctas) * 2 * attend_part_floats(d) * 4;
}

// Whether warps take whole units, each one by itself.  It saves the joins of
// the warps and CTAs (2 us or more of a CTA's time per unit) and costs the
// evenness of shares, and the time that a unit takes in one warp.  So: a unit
// of one tile always; else as many units as keep the CTAs loading, two per CTA
// where a unit has four granules (a warp's 16 tiles), one per warp at eight,
// and lists, which are all of one length, only in nearly full rounds of the
// warps.  Measured (one way, the other; us; d 128, 8 key heads unless said):
// 85 sequences of up to 3 tokens 6.3, 14.5; 148 of up to 64: 9.3, 18.5; 74 of up to 256:
// 21, 26; 37 of up to 256: 19.3, 18.7; 222 of up to 512: 61, 72; 74 of up to 512: 37, 38;
// 222 of up to 1024: 114, 103; e4m3, 111 of up to 512: 27, 41; 128 heads on 8, 148 of up
// to 512: 48, 98; d 256, 74 of up to 512: 46, 74; lists of 512 from 4096, 2560 of
// them (72 % of three rounds): 129, 118, 3552 (all of three rounds): 142, 153.
bool attend_solo(int64_t units, int64_t granules, bool one_tile, bool lists, int64_t ctas) {
  if (one_tile) return true;
  const int64_t warps = kAttendWarps * ctas;
  if (lists && units > warps && granules > 2) return 7 * units >= 6 * ((units + warps - 1) / warps) * warps;
  return granules <= 8 && 2 * units >= std::max<int64_t>(granules, 2) * ctas;
}

template <int D, bool kE4m3, int NT>
int launch_attend_rows(AttendArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  using S = AttendShape<D, kE4m3, NT>;
  if (S::kSmem > dev.max_smem_optin) return TOPK_EUNSUPPORTED;
  const int64_t most = a.positions ? a.c : a.tab.capacity;  // tokens of a unit
  const int64_t granules = (most + S::kGranule - 1) / S::kGranule;
  const int64_t units = static_cast<int64_t>(a.lists) * a.row_tiles * a.tab.batch;
  int rc, per_sm = 0;
  if constexpr (!S::kQShared) {
    if ((rc = occupancy(paged_attention_kernel<D, kE4m3, NT, true>, kAttendThreads, S::kSmem, &per_sm))) return rc;
    const int64_t ctas = std::min(per_sm, kAttendCtasPerSm) * dev.sms;
    if (attend_solo(units, granules, most <= S::kKeys, a.positions != nullptr, ctas))
      return launch_pdl(paged_attention_kernel<D, kE4m3, NT, true>, dim3(static_cast<unsigned>(std::min(ctas, units))),
                        dim3(kAttendThreads), S::kSmem, st, a);
  }
  if ((rc = occupancy(paged_attention_kernel<D, kE4m3, NT, false>, kAttendThreads, S::kSmem, &per_sm))) return rc;
  int64_t ctas = std::min(std::min(per_sm, kAttendCtasPerSm) * dev.sms, kAttendMaxCtas);
  if (granules <= ctas / units) ctas = std::max<int64_t>(1, granules * units);
  return launch_pdl(paged_attention_kernel<D, kE4m3, NT, false>, dim3(static_cast<unsigned>(ctas)),
                    dim3(kAttendThreads), S::kSmem, st, a);
}

template <int D, bool kE4m3>
int launch_attend(AttendArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  const int group = a.heads / a.lists;
  a.row_tiles = (group + 15) / 16;
  if (static_cast<int64_t>(a.lists) * a.row_tiles > kMaxN / a.tab.batch) return TOPK_EUNSUPPORTED;
  return group > 8 ? launch_attend_rows<D, kE4m3, 2>(a, dev, st) : launch_attend_rows<D, kE4m3, 1>(a, dev, st);
}

template <int D, bool kE4m3>
int launch_write(const WriteArgs& a, cudaStream_t st) {
  int rc = prepare_kernel(cache_write_kernel<D, kE4m3>);
  if (rc) return rc;
  const int64_t blocks = (a.tokens + kWriteTokens - 1) / kWriteTokens;
  if (blocks > kMaxGridX) return TOPK_EUNSUPPORTED;
  const int lines = (2 * a.cache[0].kv_heads + write_lines<D>() - 1) / write_lines<D>();
  return launch_pdl(cache_write_kernel<D, kE4m3>,
                    dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(std::min(lines, 65535))), dim3(256), 0, st, a);
}

template <int D, bool kE4m3>
int launch_read(const ReadArgs& a, cudaStream_t st) {
  int rc = prepare_kernel(cache_read_kernel<D, kE4m3>);
  if (rc) return rc;
  const int64_t blocks = (a.n + read_rows<D>() - 1) / read_rows<D>();
  return launch_pdl(cache_read_kernel<D, kE4m3>,
                    dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(std::min(a.cache.kv_heads, 65535)),
                         static_cast<unsigned>(std::min(a.tab.batch, 65535))),
                    dim3(256), 0, st, a);
}

// Picks the instantiation for (d, cache type).
#define TK_BY_CACHE(fn, d, e4m3, ...)                                          \
  ((d) == 64    ? ((e4m3) ? fn<64, true>(__VA_ARGS__) : fn<64, false>(__VA_ARGS__))   \
   : (d) == 128 ? ((e4m3) ? fn<128, true>(__VA_ARGS__) : fn<128, false>(__VA_ARGS__)) \
                : ((e4m3) ? fn<256, true>(__VA_ARGS__) : fn<256, false>(__VA_ARGS__)))

// How a beam's row is cut into pieces.  Where one round of CTAs can hold all
// rows in registers: into what a CTA holds at most, and down to a quarter of
// that while the pieces are fewer than two per SM.  Else for the streaming
// kernel, which has fewer starts and ends to pay for: so many that the rounds
// of CTAs take the least time, the end of a piece counted as 32 KB of reading.
// Measured, held and streaming, us, k 8: 64 rows of 128255 bf16 (256 pieces)
// 12.7, 16.1; fp32 (512) 16.6, 16.4; 192 rows of 32000 fp32 (384) 14.1, 14.4; 512
// rows of 128255 bf16 48.5, 41.7; fp32 74.6, 59.7; 4 rows of 131072 fp32 8.9, 9.1.
struct BeamCut {
  int pieces;
  bool held;
};
BeamCut beam_cut(int64_t rows, int64_t n, int esz, const DeviceInfo& dev) {
  const int64_t vectors = n / (16 / esz) + 2;
  const int64_t held_most = static_cast<int64_t>(kBeamThreads) * kBeamVectors;
  const int64_t held_least = (vectors + held_most - 1) / held_most;
  if (rows * held_least <= 2 * dev.sms) {
    const int64_t wanted = std::min(2 * dev.sms / rows, 4 * vectors / held_most);
    return {static_cast<int>(std::max(held_least, wanted)), true};
  }
  const int64_t most = static_cast<int64_t>(kBeamThreads) * kBeamBatch * kBeamBatches, slots = kBeamCtasPerSm * dev.sms;
  const int64_t least = (vectors + most - 1) / most, cap = std::max(least, vectors / 1024);
  int64_t best = 0, best_cost = 0;
  for (int rounds = 0; rounds <= 4; ++rounds) {  // the most pieces of so many rounds; 0: the fewest pieces
    const int64_t p = std::min(cap, std::max(least, rounds * slots / rows));
    const int64_t cost = ((rows * p + slots - 1) / slots) * (vectors / p + 2048);
    if (best == 0 || cost < best_cost) {
      best = p;
      best_cost = cost;
    }
  }
  return {static_cast<int>(best), false};
}

struct BeamPlan {
  int pieces;
  bool held;
  int64_t sentences;  // per launch
  size_t sums, lists; // bytes
  size_t total() const { return kTicketBytes + sums + lists; }
};

BeamPlan plan_beam(int64_t batch, int beams, int64_t n, int k, int esz, const DeviceInfo& dev) {
  BeamPlan pl;
  const BeamCut cut = beam_cut(batch * beams, n, esz, dev);
  pl.pieces = cut.pieces;
  pl.held = cut.held;
  // as many sentences as fit a grid and about 1 GB of lists
  const int64_t sentence_bytes = static_cast<int64_t>(pl.pieces) * (sizeof(BeamSum) + 8 * k) * beams;
  const int64_t fit = std::min<int64_t>((int64_t{1} << 30) / sentence_bytes,
                                        kMaxGridX / (static_cast<int64_t>(pl.pieces) * beams));
  pl.sentences = std::min(batch, std::max<int64_t>(fit, 1));
  pl.sums = static_cast<size_t>(pl.sentences) * beams * pl.pieces * sizeof(BeamSum);
  pl.lists = static_cast<size_t>(pl.sentences) * beams * pl.pieces * k * 8;
  return pl;
}

template <typename T>
int run_beam(const T* logits, const float* scores, int64_t batch, int beams, int64_t n, int k, float* out_scores,
             int32_t* out_parent, int32_t* out_token, void* ws, size_t ws_bytes, void* stream) {
  if (!logits || !scores || !out_scores || !out_parent || !out_token) return TOPK_EINVAL;
  if (batch < 1 || beams < 1 || n < 1 || k < 1 || n > kMaxN) return TOPK_EINVAL;
  if (beams > TOPK_BEAM_MAX || k > TOPK_BEAM_MAX) return TOPK_EUNSUPPORTED;
  if (batch > kMaxElems / beams / n || batch > kMaxGridX) return TOPK_EUNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(logits) % sizeof(T)) return TOPK_EINVAL;
  DeviceInfo dev;
  int rc = current_device_info(&dev);
  if (rc) return rc;
  const BeamPlan pl = plan_beam(batch, beams, n, k, sizeof(T), dev);
  if (!ws || ws_bytes < pl.total()) return TOPK_EWORKSPACE;
  if (!aligned16(ws)) return TOPK_EINVAL;
  BeamArgs a{logits, scores, n, beams, k, pl.pieces, 0, out_scores, out_parent, out_token, nullptr, nullptr};
  unsigned char* base = static_cast<unsigned char*>(ws);
  a.sums = reinterpret_cast<BeamSum*>(base + kTicketBytes);
  a.lists = reinterpret_cast<uint64_t*>(base + kTicketBytes + pl.sums);
  for (; a.first < batch; a.first += pl.sentences) {
    const int64_t sentences = std::min(pl.sentences, batch - a.first);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(sentences * beams * pl.pieces));
    rc = pl.held ? launch_pdl(topk_beam_held_kernel<T>, grid, dim3(kBeamThreads), 0, st, a)
                 : launch_pdl(topk_beam_stream_kernel<T>, grid, dim3(kBeamThreads), 0, st, a);
    if (rc) return rc;
    rc = launch_pdl(beam_finish_kernel, dim3(static_cast<unsigned>(sentences)), dim3(kBeamThreads), 0, st, a);
    if (rc) return rc;
  }
  return TOPK_OK;
}

}  // namespace

int decode_take_device_status(int* out) { return take_device_status(out); }

}  // namespace tk

using namespace tk;

extern "C" {

size_t paged_attention_workspace_bytes(int64_t batch, int heads, int lists, int d) {
  DeviceInfo dev;
  if (batch < 1 || heads < 1 || lists < 0 || !cache_head_dim(d) || current_device_info(&dev)) return 0;
  return attend_workspace(d, dev);
}

int paged_attention(const uint16_t* q, int64_t q_stride, int64_t batch, int heads, const topk_cache* k_cache,
                    const topk_cache* v_cache, const int32_t* block_table, int64_t table_stride, int table_width,
                    const int32_t* seq_lens, const int32_t* positions, int lists, int c, float scale, uint16_t* out,
                    float* out_lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !out) return TOPK_EINVAL;
  AttendArgs a{};
  int rc;
  if ((rc = cache_view(k_cache, &a.k)) || (rc = cache_view(v_cache, &a.v))) return rc;
  if (!same_shape(k_cache, v_cache)) return TOPK_EINVAL;
  if ((rc = table_view(block_table, table_stride, table_width, seq_lens, batch, k_cache->page_size, &a.tab)))
    return rc;
  if (heads < 1 || heads % k_cache->kv_heads) return TOPK_EINVAL;
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return TOPK_EINVAL;
  if (!aligned16(q) || !aligned16(out) || q_stride < 0 || q_stride > kMaxElems || q_stride % 8) return TOPK_EINVAL;
  if (positions) {
    if (lists < 1 || c < 1 || lists % k_cache->kv_heads || heads % lists) return TOPK_EINVAL;
    if (c > kMaxElems / lists / batch) return TOPK_EUNSUPPORTED;
  } else if (lists != 0 || c != 0) {
    return TOPK_EINVAL;
  }
  if (batch > kMaxN / heads) return TOPK_EUNSUPPORTED;
  DeviceInfo dev;
  if ((rc = current_device_info(&dev))) return rc;
  if (!workspace || workspace_bytes < attend_workspace(k_cache->d, dev)) return TOPK_EWORKSPACE;
  if (!aligned16(workspace)) return TOPK_EINVAL;
  a.tickets = static_cast<uint32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kTicketBytes);
  a.same_strides = a.k.page_stride == a.v.page_stride && a.k.head_stride == a.v.head_stride &&
                   a.k.token_stride == a.v.token_stride &&
                   (!a.k.scale || (a.k.s_page_stride == a.v.s_page_stride && a.k.s_head_stride == a.v.s_head_stride &&
                                   a.k.s_token_stride == a.v.s_token_stride));
  a.grouped = !positions && k_cache->page_size % 16 == 0 && a.same_strides;
  a.q = q;
  a.q_stride = q_stride;
  a.positions = positions;
  a.heads = heads;
  a.lists = positions ? lists : k_cache->kv_heads;
  a.c = c;
  a.scale_log2 = scale_log2;
  a.out = out;
  a.lse = out_lse;
  return TK_BY_CACHE(launch_attend, k_cache->d, a.k.scale != nullptr, a, dev, static_cast<cudaStream_t>(stream));
}

int cache_write(const uint16_t* k, int64_t k_token_stride, int64_t k_head_stride, const uint16_t* v,
                int64_t v_token_stride, int64_t v_head_stride, int64_t tokens, const topk_cache* k_cache,
                const topk_cache* v_cache, const int64_t* slots, void* stream) {
  if (!k || !v || !slots) return TOPK_EINVAL;
  WriteArgs a{};
  int rc;
  if ((rc = cache_view(k_cache, &a.cache[0])) || (rc = cache_view(v_cache, &a.cache[1]))) return rc;
  if (!same_shape(k_cache, v_cache)) return TOPK_EINVAL;
  if (tokens < 1) return TOPK_EINVAL;
  if (tokens > kMaxElems / k_cache->kv_heads / k_cache->d) return TOPK_EUNSUPPORTED;
  if (!aligned16(k) || !aligned16(v)) return TOPK_EINVAL;
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  for (int64_t s : strides)
    if (s < 0 || s > kMaxElems || s % 8) return TOPK_EINVAL;
  a.src[0] = k;
  a.src[1] = v;
  a.token_stride[0] = k_token_stride;
  a.token_stride[1] = v_token_stride;
  a.head_stride[0] = k_head_stride;
  a.head_stride[1] = v_head_stride;
  a.slots = slots;
  a.tokens = tokens;
  return TK_BY_CACHE(launch_write, k_cache->d, a.cache[0].scale != nullptr, a, static_cast<cudaStream_t>(stream));
}

int cache_read(const topk_cache* cache, const int32_t* block_table, int64_t table_stride, int table_width,
               const int32_t* seq_lens, int64_t batch, int64_t n, uint16_t* out, void* stream) {
  ReadArgs a{};
  int rc;
  if (!out || n < 1 || n > kMaxN) return TOPK_EINVAL;
  if ((rc = cache_view(cache, &a.cache))) return rc;
  if ((rc = table_view(block_table, table_stride, table_width, seq_lens, batch, cache->page_size, &a.tab))) return rc;
  if (batch > kMaxElems / cache->kv_heads / n / cache->d) return TOPK_EUNSUPPORTED;
  if (!aligned16(out)) return TOPK_EINVAL;
  a.n = n;
  a.out = out;
  return TK_BY_CACHE(launch_read, cache->d, a.cache.scale != nullptr, a, static_cast<cudaStream_t>(stream));
}

size_t topk_beam_workspace_bytes(int64_t batch, int beams, int64_t n, int k) {
  if (batch < 1 || beams < 1 || n < 1 || k < 1 || n > kMaxN || beams > TOPK_BEAM_MAX || k > TOPK_BEAM_MAX) return 0;
  if (batch > kMaxElems / beams / n || batch > kMaxGridX) return 0;
  DeviceInfo dev;
  if (current_device_info(&dev)) return 0;
  return std::max(plan_beam(batch, beams, n, k, 4, dev).total(), plan_beam(batch, beams, n, k, 2, dev).total());
}

int topk_beam(const float* logits, const float* beam_scores, int64_t batch, int beams, int64_t n, int k,
              float* out_scores, int32_t* out_parent, int32_t* out_token, void* workspace, size_t workspace_bytes,
              void* stream) {
  return run_beam<float>(logits, beam_scores, batch, beams, n, k, out_scores, out_parent, out_token, workspace,
                         workspace_bytes, stream);
}

int topk_beam_bf16(const uint16_t* logits, const float* beam_scores, int64_t batch, int beams, int64_t n, int k,
                   float* out_scores, int32_t* out_parent, int32_t* out_token, void* workspace,
                   size_t workspace_bytes, void* stream) {
  return run_beam<uint16_t>(logits, beam_scores, batch, beams, n, k, out_scores, out_parent, out_token, workspace,
                            workspace_bytes, stream);
}

int beam_reorder(const void* const* src, void* const* dst, const int64_t* row_bytes, int count, int64_t batch,
                 int beams, int k, const int32_t* parents, void* stream) {
  if (!src || !dst || !row_bytes || !parents) return TOPK_EINVAL;
  if (count < 1 || batch < 1 || beams < 1 || k < 1) return TOPK_EINVAL;
  if (count > kMaxReorder || batch > kMaxN / k || batch > kMaxN / beams) return TOPK_EUNSUPPORTED;
  // No destination may overlap a source or another destination.
  struct Span {
    uintptr_t begin, end;
    bool dst;
  };
  Span span[2 * kMaxReorder];
  for (int i = 0; i < count; ++i) {
    if (!src[i] || !dst[i] || row_bytes[i] < 1) return TOPK_EINVAL;
    if (row_bytes[i] > kMaxElems / batch / std::max(beams, k)) return TOPK_EUNSUPPORTED;
    const uintptr_t s = reinterpret_cast<uintptr_t>(src[i]), d = reinterpret_cast<uintptr_t>(dst[i]);
    span[2 * i] = Span{s, s + static_cast<uintptr_t>(batch * beams * row_bytes[i]), false};
    span[2 * i + 1] = Span{d, d + static_cast<uintptr_t>(batch * k * row_bytes[i]), true};
  }
  std::sort(span, span + 2 * count, [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t any_end = 0, dst_end = 0;
  for (int i = 0; i < 2 * count; ++i) {
    if (span[i].begin < (span[i].dst ? any_end : dst_end)) return TOPK_EINVAL;
    any_end = std::max(any_end, span[i].end);
    if (span[i].dst) dst_end = std::max(dst_end, span[i].end);
  }
  int rc = prepare_kernel(beam_reorder_kernel);
  if (rc) return rc;
  for (int first = 0; first < count; first += kReorderStates) {
    ReorderArgs a{};
    a.count = std::min(kReorderStates, count - first);
    a.rows = batch * k;
    int64_t items = 0;
    for (int i = 0; i < a.count; ++i) {
      a.src[i] = static_cast<const unsigned char*>(src[first + i]);
      a.dst[i] = static_cast<unsigned char*>(dst[first + i]);
      a.row_bytes[i] = row_bytes[first + i];
      items += reorder_items(a.rows, a.row_bytes[i]);
      a.end[i] = items;
    }
    a.parents = parents;
    a.beams = beams;
    a.k = k;
    rc = launch_pdl(beam_reorder_kernel, dim3(static_cast<unsigned>(std::min(items, kMaxGridX))), dim3(kReorderThreads),
                    0, static_cast<cudaStream_t>(stream), a);
    if (rc) return rc;
  }
  return TOPK_OK;
}

}  // extern "C"
