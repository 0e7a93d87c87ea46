// Host entries of the decode-loop operators: pic_write_tokens,
// pic_attend_paged and pic_evict_tokens (include/pic.h).  They check their
// arguments, fill the launch parameters and launch; they allocate nothing,
// upload nothing and wait for nothing, so they can be captured into a graph.
#include "pic_decode.h"

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <limits>

namespace {

using namespace pic;

pic_status fail(pic_ctx* ctx, pic_status st, const char* fmt, ...) __attribute__((format(printf, 3, 4)));
pic_status fail(pic_ctx* ctx, pic_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_error(ctx, st, buf);
}
pic_status cuda_fail(pic_ctx* ctx, cudaError_t e, const char* what) {
  return fail(ctx, PIC_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The launching device, and that every buffer is memory of that device: these
// operators stream with no regard to the host link, and a pageable host
// pointer would fault.
struct Buffer {
  const char* name;
  const void* ptr;
};
pic_status check_device(pic_ctx* ctx, const Buffer* bufs, int n, int* sm_count) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "cudaGetDevice");
  static std::atomic<int> sms_of[32];   // 0: not asked for yet
  *sm_count = dev < 32 ? sms_of[dev].load(std::memory_order_relaxed) : 0;
  if (*sm_count == 0) {
    e = cudaDeviceGetAttribute(sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(ctx, e, "cudaDeviceGetAttribute");
    if (dev < 32) sms_of[dev].store(*sm_count, std::memory_order_relaxed);
  }
  for (int i = 0; i < n; ++i) {
    if (!bufs[i].ptr) continue;
    cudaPointerAttributes a;
    e = cudaPointerGetAttributes(&a, bufs[i].ptr);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(ctx, PIC_ERR_INVALID_ARG, "%s is not memory the GPU can reach", bufs[i].name);
    }
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)
      return fail(ctx, PIC_ERR_UNSUPPORTED, "%s must be device memory", bufs[i].name);
    if (a.type == cudaMemoryTypeDevice && a.device != dev)
      return fail(ctx, PIC_ERR_INVALID_ARG, "%s is on device %d, the current device is %d", bufs[i].name, a.device, dev);
  }
  return PIC_OK;
}

PagedView paged_view(const CtxView& c, const int32_t* d_tables, int32_t n_tables, int32_t max_blocks) {
  PagedView v{};
  v.tables = d_tables;
  v.n_tables = n_tables;
  v.max_blocks = max_blocks;
  v.num_cache_blocks = c.num_cache_blocks;
  v.block_size = c.model->block_size;
  int32_t log2 = 0;
  while (int64_t{1} << log2 < v.block_size) ++log2;
  v.block_shift = 31 + log2;
  v.block_mul = static_cast<uint32_t>(((uint64_t{1} << v.block_shift) + v.block_size - 1) / v.block_size);
  return v;
}

void fill_freq(const CtxView& c, FreqTable* t) { std::memcpy(t->turns, c.freq, c.model->rope_dim / 2 * sizeof(float2)); }

// Longest sequence a block table can hold (none, where the cache has no block).
int32_t table_capacity(const CtxView& c, int32_t max_blocks) {
  if (c.num_cache_blocks == 0) return 0;
  const int64_t n = static_cast<int64_t>(max_blocks) * c.model->block_size;
  return static_cast<int32_t>(std::min<int64_t>(n, kPagedMaxSlots));
}

// Rows of the cache: a sequence whose blocks are all its own is no longer.
int32_t cache_rows(const CtxView& c) {
  return static_cast<int32_t>(std::min<int64_t>(static_cast<int64_t>(c.num_cache_blocks) * c.model->block_size, kPagedMaxSlots));
}

bool weight_heads_ok(const CtxView& c, int32_t n) { return n == 1 || n == c.model->num_kv_heads; }

struct PagedLayout {
  size_t first, lse2, rec_ml, rec_acc, scores, total;
  int64_t score_stride;
};
int32_t paged_passes(int32_t group) { return (group + 15) / 16; }
// Width of an output row: the head's, or the latent's.
int32_t paged_out_dim(const CtxView& c) { return c.model->kind == PIC_KIND_MLA ? c.model->rope_offset : c.model->head_dim; }
int64_t paged_max_parts(int32_t v_heads, int head_dim) {
  return std::max<int64_t>(1, static_cast<int64_t>(kPagedMaxSms) * paged_ranges_per_sm(head_dim) / v_heads);
}
PagedLayout paged_layout(const CtxView& c, int64_t n_req, int64_t q_heads, int64_t max_len, bool weights) {
  const int d = paged_out_dim(c);
  const int32_t group = static_cast<int32_t>(q_heads / c.model->num_kv_heads);
  const int64_t recs = paged_max_parts(c.model->num_kv_heads * paged_passes(group), c.model->head_dim) + n_req;
  PagedLayout L{};
  L.score_stride = weights ? n_req * ((max_len + kPagedTile - 1) / kPagedTile) * kPagedTile : 0;
  L.first = sizeof(WsHeader);
  L.lse2 = align_up(L.first + (n_req + 1) * sizeof(int64_t), kWsAlign);
  L.rec_ml = align_up(L.lse2 + (weights ? n_req * q_heads * sizeof(float) : 0), kWsAlign);
  L.rec_acc = align_up(L.rec_ml + recs * q_heads * sizeof(float2), kWsAlign);
  L.scores = align_up(L.rec_acc + recs * q_heads * d * sizeof(float), kWsAlign);
  L.total = align_up(L.scores + static_cast<size_t>(q_heads) * L.score_stride * sizeof(float), kWsAlign);
  return L;
}
bool paged_heads_ok(const CtxView& c, int32_t num_q_heads) {
  return num_q_heads > 0 && num_q_heads % c.model->num_kv_heads == 0;
}
// What one call takes: sizes beyond it would overflow the kernels' counts (and a workspace's size).
bool paged_size_ok(int64_t n_req, int64_t num_q_heads) {
  return num_q_heads <= kPagedMaxHeads && n_req * num_q_heads <= std::numeric_limits<int32_t>::max() / 2;
}
bool evict_size_ok(const CtxView& c, int64_t num_layers, int64_t n_req) {
  const int64_t row_items = static_cast<int64_t>(c.model->num_kv_heads) * c.model->head_dim * 2 / 32;
  return num_layers <= c.model->num_layers && num_layers * n_req <= std::numeric_limits<int32_t>::max() / 2 / row_items;
}

// How finely the move slices the kept rows of each (layer, request, tensor,
// and head where heads keep sets of their own): into as many slices of whole
// 32-byte items as fill the resident CTAs best.  Slices below 128 bytes cost
// DRAM efficiency (weighed 0.7 and 0.5, by the time of one request's layer).
struct EvictShape {
  int32_t tensors, pieces, piece_heads, slices, slice_items;
};
EvictShape evict_shape(const CtxView& c, int32_t weight_heads, int64_t units, int sm_count) {
  const pic_model_desc& m = *c.model;
  EvictShape s{};
  s.tensors = m.kind == PIC_KIND_GQA ? 2 : 1;
  s.pieces = weight_heads > 1 ? m.num_kv_heads : 1;
  s.piece_heads = weight_heads > 1 ? 1 : m.num_kv_heads;
  const int32_t items = s.piece_heads * (m.head_dim * 2 / 32);
  const int64_t streams = units * s.tensors * s.pieces, room = static_cast<int64_t>(sm_count) * kEvictMoveCtas;
  double best = -1.0;
  for (int32_t per = std::min(items, kEvictMoveThreads); per >= 1; --per) {
    if (items % per != 0) continue;
    const int64_t n = streams * (items / per), waves = (n + room - 1) / room;
    const double fill = static_cast<double>(n) / static_cast<double>(waves * room);
    const double score = fill * (per >= 4 ? 1.0 : (per >= 2 ? 0.7 : 0.5));
    if (score > best * 1.02) {   // the widest of equals
      best = score;
      s.slices = items / per;
      s.slice_items = per;
    }
  }
  return s;
}
struct EvictLayout {
  size_t next_lens, units, total;
};
EvictLayout evict_layout(int64_t layers, int64_t n_req, int64_t weight_heads) {
  EvictLayout L{};
  L.next_lens = sizeof(WsHeader);
  L.units = align_up(L.next_lens + n_req * sizeof(int32_t), kWsAlign);
  L.total = align_up(L.units + layers * n_req * weight_heads * sizeof(EvictUnit), kWsAlign);
  return L;
}

}  // namespace

extern "C" {

pic_status pic_write_tokens(pic_ctx* ctx, const pic_new_tokens* t, void* k_cache, void* v_cache,
                            const int32_t* d_tables, int32_t n_tables, int32_t max_blocks, float* d_weights,
                            int32_t weight_heads, void* d_ws, size_t ws_bytes, pic_stream_t stream) {
  if (!ctx || !t) return fail(ctx, PIC_ERR_INVALID_ARG, "null ctx or tokens");
  const CtxView c = ctx_view(ctx);
  const pic_model_desc& m = *c.model;
  const bool mla = m.kind == PIC_KIND_MLA;
  if (t->n_tokens < 0 || t->num_q_heads < 0) return fail(ctx, PIC_ERR_INVALID_ARG, "negative token or head count");
  if (t->n_axes < 1 || t->n_axes > PIC_MAX_AXES)
    return fail(ctx, PIC_ERR_INVALID_ARG, "n_axes must be 1 .. %d", PIC_MAX_AXES);
  const int32_t half = m.rope_dim / 2;
  for (int32_t i = 0; t->freq_axis && i < half; ++i)
    if (t->freq_axis[i] >= t->n_axes)
      return fail(ctx, PIC_ERR_INVALID_ARG, "freq_axis[%d] is %d, there are %d axes", i, t->freq_axis[i], t->n_axes);
  if (!d_ws || ws_bytes < PIC_STATUS_BYTES) return fail(ctx, PIC_ERR_CAPACITY, "workspace needs %d bytes", PIC_STATUS_BYTES);
  if (t->n_tokens == 0) return set_error(ctx, PIC_OK, "");   // an empty batch has no buffers
  const bool with_q = t->num_q_heads > 0, with_k = t->k != nullptr;
  if (!with_q && !with_k) return fail(ctx, PIC_ERR_INVALID_ARG, "neither queries nor keys given");
  if (!t->d_pos || (with_q && (!t->q || !t->q_out)))
    return fail(ctx, PIC_ERR_INVALID_ARG, "null positions, queries or query output");
  if (with_k) {
    if (!mla != (t->v != nullptr)) return fail(ctx, PIC_ERR_INVALID_ARG, "GQA tokens have keys and values, MLA tokens keys only");
    if (n_tables < 0 || max_blocks < 0) return fail(ctx, PIC_ERR_INVALID_ARG, "bad block table shape");
    if (!k_cache || (!mla && !v_cache) || (!d_tables && n_tables > 0 && max_blocks > 0) || !t->d_req || !t->d_slot)
      return fail(ctx, PIC_ERR_INVALID_ARG, "null cache, block table, request or slot list");
    if (d_weights && !weight_heads_ok(c, weight_heads))
      return fail(ctx, PIC_ERR_INVALID_ARG, "weight_heads must be 1 or num_kv_heads");
  } else if (t->v) {
    return fail(ctx, PIC_ERR_INVALID_ARG, "values without keys");
  }
  const int64_t q_bytes = static_cast<int64_t>(t->num_q_heads) * m.head_dim * 2;
  const int64_t row_bytes = static_cast<int64_t>(m.num_kv_heads) * m.head_dim * 2;
  if (q_bytes > std::numeric_limits<int32_t>::max() || row_bytes > std::numeric_limits<int32_t>::max())
    return fail(ctx, PIC_ERR_RANGE, "a token's heads exceed 2^31 bytes");
  if (t->n_tokens > 1 && ((with_q && (t->q_stride < q_bytes || t->q_out_stride < q_bytes)) ||
                          (with_k && (t->k_stride < row_bytes || (!mla && t->v_stride < row_bytes)))))
    return fail(ctx, PIC_ERR_RANGE, "token strides smaller than a token");
  if (with_q && t->q == t->q_out && t->n_tokens > 1 && t->q_stride != t->q_out_stride)
    return fail(ctx, PIC_ERR_INVALID_ARG, "queries turned in place need one stride");
  if (!aligned(t->q, 16) || !aligned(t->q_out, 16) || !aligned(t->k, 16) || !aligned(t->v, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || (t->q_stride & 15) || (t->q_out_stride & 15) || (t->k_stride & 15) || (t->v_stride & 15))
    return fail(ctx, PIC_ERR_ALIGNMENT, "tokens, caches and strides must be 16-byte aligned");
  if (!aligned(t->d_pos, 4) || !aligned(t->d_req, 4) || !aligned(t->d_slot, 4) || !aligned(d_tables, 4) ||
      !aligned(d_weights, 4) || !aligned(d_ws, kWsAlign))
    return fail(ctx, PIC_ERR_ALIGNMENT, "index arrays and weights must be 4-byte aligned, the workspace 256-byte");
  const Buffer bufs[] = {{"q", with_q ? t->q : nullptr}, {"q_out", with_q ? t->q_out : nullptr}, {"k", t->k}, {"v", t->v},
                         {"positions", t->d_pos}, {"requests", with_k ? t->d_req : nullptr},
                         {"slots", with_k ? t->d_slot : nullptr}, {"k_cache", with_k ? k_cache : nullptr},
                         {"v_cache", with_k && !mla ? v_cache : nullptr}, {"block tables", with_k ? d_tables : nullptr},
                         {"weights", with_k ? d_weights : nullptr}, {"workspace", d_ws}};
  int sms = 0;
  const pic_status st = check_device(ctx, bufs, sizeof(bufs) / sizeof(bufs[0]), &sms);
  if (st != PIC_OK) return st;

  WriteParams p{};
  p.paged = paged_view(c, d_tables, n_tables, max_blocks);
  fill_freq(c, &p.freq);
  if (t->freq_axis) std::memcpy(p.axis, t->freq_axis, half);
  p.pos = t->d_pos;
  p.n_axes = t->n_axes;
  p.n_tokens = t->n_tokens;
  p.req = t->d_req;
  p.slot = t->d_slot;
  p.q = static_cast<const uint8_t*>(t->q);
  p.q_out = static_cast<uint8_t*>(t->q_out);
  p.k = static_cast<const uint8_t*>(t->k);
  p.v = static_cast<const uint8_t*>(t->v);
  p.q_stride = t->q_stride;
  p.q_out_stride = t->q_out_stride;
  p.k_stride = t->k_stride;
  p.v_stride = t->v_stride;
  p.q_heads = t->num_q_heads;
  p.kv_heads = with_k ? m.num_kv_heads : 0;
  p.head_bytes = m.head_dim * 2;
  p.rope_off = m.rope_offset * 2;
  const int lanes = half / 8;  // eight frequencies a lane: 4, 8 or 16
  p.lph_shift = lanes == 4 ? 2 : (lanes == 8 ? 3 : 4);
  const int latent_chunks = mla ? m.rope_offset * 2 / 16 : 0;
  p.q_copy_chunks = with_q && t->q != t->q_out ? latent_chunks : 0;
  p.k_copy_chunks = with_k ? latent_chunks : 0;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.weights = with_k ? d_weights : nullptr;
  p.weight_heads = weight_heads;
  p.status = &static_cast<WsHeader*>(d_ws)->status;
  // A warp's run of heads: all of a token's when there are tokens for 32 warps
  // per SM, so that their cos / sin are made once; shorter runs, down to four
  // steps, when there are few and latency counts.
  const int hpi = 32 / lanes;
  const int64_t iters = (static_cast<int64_t>(p.q_heads) + p.kv_heads + hpi - 1) / hpi;
  const int64_t wanted = (static_cast<int64_t>(sms) * 32 + t->n_tokens - 1) / t->n_tokens;
  p.rot_iters = static_cast<int32_t>(std::max<int64_t>(std::min<int64_t>(iters, 4), (iters + wanted - 1) / wanted));
  p.rot_parts = static_cast<int32_t>((iters + p.rot_iters - 1) / p.rot_iters);
  const int64_t chunks = static_cast<int64_t>(p.q_heads) * p.q_copy_chunks + p.k_copy_chunks +
                         (t->v ? row_bytes / 16 : 0);
  p.copy_parts = static_cast<int32_t>((chunks + 255) / 256);
  if (static_cast<int64_t>(t->n_tokens) * (p.rot_parts + p.copy_parts) > std::numeric_limits<int32_t>::max())
    return fail(ctx, PIC_ERR_RANGE, "more than 2^31 warps of work: write fewer tokens at a time");
  const cudaError_t e = launch_write(p, m.pairing, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(ctx, e, "token write launch");
  return set_error(ctx, PIC_OK, "");
}

size_t pic_attend_paged_workspace_bytes(const pic_ctx* ctx, int32_t n_req, int32_t num_q_heads, int32_t max_seq_len,
                                        int32_t with_weights) {
  if (!ctx || n_req < 0 || max_seq_len < 0) return 0;
  const CtxView c = ctx_view(ctx);
  if (!paged_heads_ok(c, num_q_heads) || !paged_size_ok(n_req, num_q_heads) || max_seq_len > kPagedMaxSlots) return 0;
  return paged_layout(c, n_req, num_q_heads, max_seq_len, with_weights != 0).total;
}

pic_status pic_attend_paged(pic_ctx* ctx, const void* q, int64_t q_stride, int32_t n_req, int32_t num_q_heads,
                            float softmax_scale, const void* k_cache, const void* v_cache, const int32_t* d_tables,
                            int32_t max_blocks, const int32_t* d_seq_lens, int32_t max_seq_len, void* out,
                            int32_t out_type, float* lse, float* d_weights, int32_t weight_heads, void* d_ws,
                            size_t ws_bytes, pic_stream_t stream) {
  if (!ctx) return fail(nullptr, PIC_ERR_INVALID_ARG, "null ctx");
  const CtxView c = ctx_view(ctx);
  const pic_model_desc& m = *c.model;
  const bool mla = m.kind == PIC_KIND_MLA;
  if (!paged_heads_ok(c, num_q_heads))
    return fail(ctx, PIC_ERR_INVALID_ARG, "num_q_heads must be a positive multiple of num_kv_heads");
  if (n_req < 0 || max_blocks < 0 || max_seq_len < 0) return fail(ctx, PIC_ERR_INVALID_ARG, "negative size");
  if (out_type != PIC_F32 && out_type != PIC_BF16) return fail(ctx, PIC_ERR_INVALID_ARG, "unknown out_type %d", out_type);
  if (d_weights && !weight_heads_ok(c, weight_heads))
    return fail(ctx, PIC_ERR_INVALID_ARG, "weight_heads must be 1 or num_kv_heads");
  if (mla) v_cache = nullptr;  // the latent serves as value
  const bool some = n_req > 0;   // an empty batch has no buffers of its own, a table without columns no address
  if (!k_cache || (!mla && !v_cache) || !d_ws || (some && (!q || (!d_tables && max_blocks > 0) || !d_seq_lens || !out)))
    return fail(ctx, PIC_ERR_INVALID_ARG, "null q, cache, block table, lengths, out or workspace");
  const int64_t q_bytes = static_cast<int64_t>(num_q_heads) * m.head_dim * 2;
  const int64_t row_bytes = static_cast<int64_t>(m.num_kv_heads) * m.head_dim * 2;
  if (row_bytes > std::numeric_limits<int32_t>::max() || !paged_size_ok(n_req, num_q_heads))
    return fail(ctx, PIC_ERR_RANGE, "more than %d query heads, or 2^30 in all", kPagedMaxHeads);
  if (n_req > 1 && q_stride < q_bytes) return fail(ctx, PIC_ERR_RANGE, "q_stride smaller than a request's heads");
  if (max_seq_len > table_capacity(c, max_blocks))
    return fail(ctx, PIC_ERR_RANGE, "max_seq_len %d exceeds the %d slots a block table holds", max_seq_len,
                table_capacity(c, max_blocks));
  if (!aligned(q, 16) || (q_stride & 15) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return fail(ctx, PIC_ERR_ALIGNMENT, "q, its stride, caches and out must be 16-byte aligned");
  if (!aligned(d_tables, 4) || !aligned(d_seq_lens, 4) || !aligned(lse, 4) || !aligned(d_weights, 4) || !aligned(d_ws, kWsAlign))
    return fail(ctx, PIC_ERR_ALIGNMENT, "tables, lengths, lse and weights must be 4-byte aligned, the workspace 256-byte");
  const PagedLayout L = paged_layout(c, n_req, num_q_heads, max_seq_len, d_weights != nullptr);
  if (ws_bytes < L.total) return fail(ctx, PIC_ERR_CAPACITY, "workspace has %zu bytes, needs %zu", ws_bytes, L.total);
  if (n_req == 0) return set_error(ctx, PIC_OK, "");
  const Buffer bufs[] = {{"q", q}, {"k_cache", k_cache}, {"v_cache", v_cache}, {"block tables", d_tables},
                         {"lengths", d_seq_lens}, {"out", out}, {"lse", lse}, {"weights", d_weights}, {"workspace", d_ws}};
  int sms = 0;
  const pic_status st = check_device(ctx, bufs, sizeof(bufs) / sizeof(bufs[0]), &sms);
  if (st != PIC_OK) return st;

  uint8_t* ws = static_cast<uint8_t*>(d_ws);
  PagedParams p{};
  p.paged = paged_view(c, d_tables, n_req, max_blocks);
  p.q = static_cast<const uint8_t*>(q);
  p.q_stride = q_stride;
  p.lens = d_seq_lens;
  p.n_req = n_req;
  p.max_len = max_seq_len;
  p.q_heads = num_q_heads;
  p.kv_heads = m.num_kv_heads;
  p.group = num_q_heads / m.num_kv_heads;
  p.passes = paged_passes(p.group);
  p.v_heads = p.kv_heads * p.passes;
  const int used = std::min(sms, kPagedMaxSms);
  p.parts = static_cast<int32_t>(std::max<int64_t>(1, static_cast<int64_t>(used) * paged_ranges_per_sm(m.head_dim) / p.v_heads));
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.row_bytes = static_cast<int32_t>(row_bytes);
  p.first = n_req > kPagedWalkRequests ? reinterpret_cast<int64_t*>(ws + L.first) : nullptr;
  p.rec_acc = reinterpret_cast<float*>(ws + L.rec_acc);
  p.rec_ml = reinterpret_cast<float2*>(ws + L.rec_ml);
  p.lse2 = d_weights ? reinterpret_cast<float*>(ws + L.lse2) : nullptr;
  p.scores = d_weights ? reinterpret_cast<float*>(ws + L.scores) : nullptr;
  p.score_stride = L.score_stride;
  p.out = out;
  p.out_bf16 = out_type == PIC_BF16;
  p.lse = lse;
  p.weights = d_weights;
  p.weight_heads = weight_heads;
  p.status = &reinterpret_cast<WsHeader*>(ws)->status;
  const cudaError_t e = launch_paged(p, m.head_dim, used, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(ctx, e, "paged attention launch");
  return set_error(ctx, PIC_OK, "");
}

size_t pic_evict_workspace_bytes(const pic_ctx* ctx, int32_t num_layers, int32_t n_req, int32_t weight_heads) {
  if (!ctx || num_layers <= 0 || n_req < 0) return 0;
  const CtxView c = ctx_view(ctx);
  if (!weight_heads_ok(c, weight_heads) || !evict_size_ok(c, num_layers, n_req)) return 0;
  return evict_layout(num_layers, n_req, weight_heads).total;
}

pic_status pic_evict_tokens(pic_ctx* ctx, int32_t num_layers, void* k_cache, void* v_cache, int64_t cache_ls,
                            float* d_weights, int64_t weights_ls, int32_t weight_heads, const int32_t* d_tables,
                            int32_t n_req, int32_t max_blocks, const int32_t* d_seq_lens, int32_t budget, int32_t n_first,
                            int32_t n_recent, int32_t renumber, int32_t* d_kept, int32_t* d_new_lens, void* d_ws,
                            size_t ws_bytes, pic_stream_t stream) {
  if (!ctx) return fail(nullptr, PIC_ERR_INVALID_ARG, "null ctx");
  const CtxView c = ctx_view(ctx);
  const pic_model_desc& m = *c.model;
  const bool mla = m.kind == PIC_KIND_MLA;
  if (n_req < 0 || max_blocks < 0) return fail(ctx, PIC_ERR_INVALID_ARG, "negative size");
  if (num_layers < 1 || num_layers > m.num_layers) return fail(ctx, PIC_ERR_RANGE, "num_layers outside the model");
  if (!weight_heads_ok(c, weight_heads)) return fail(ctx, PIC_ERR_INVALID_ARG, "weight_heads must be 1 or num_kv_heads");
  if (budget < 1 || n_first < 0 || n_recent < 0 || static_cast<int64_t>(n_first) + n_recent > budget)
    return fail(ctx, PIC_ERR_INVALID_ARG, "need budget >= 1 and n_first + n_recent <= budget");
  const bool some = n_req > 0;
  if (!k_cache || (!mla && !v_cache) || !d_weights || !d_ws ||
      (some && ((!d_tables && max_blocks > 0) || !d_seq_lens || !d_kept || !d_new_lens)))
    return fail(ctx, PIC_ERR_INVALID_ARG, "null cache, weights, block table, lengths, output or workspace");
  if (mla) v_cache = nullptr;  // a latent row is key and value
  const int64_t rows = static_cast<int64_t>(c.num_cache_blocks) * m.block_size;
  const int64_t row_bytes = static_cast<int64_t>(m.num_kv_heads) * m.head_dim * 2;
  if (num_layers > 1 && (cache_ls < rows * row_bytes || weights_ls < rows * weight_heads * 4))
    return fail(ctx, PIC_ERR_RANGE, "a layer stride is smaller than a layer");
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || (cache_ls & 15))
    return fail(ctx, PIC_ERR_ALIGNMENT, "caches and their layer stride must be 16-byte aligned");
  if (!aligned(d_weights, 4) || (weights_ls & 3) || !aligned(d_tables, 4) || !aligned(d_seq_lens, 4) ||
      !aligned(d_kept, 4) || !aligned(d_new_lens, 4) || !aligned(d_ws, kWsAlign))
    return fail(ctx, PIC_ERR_ALIGNMENT, "weights, tables, lengths and lists must be 4-byte aligned, the workspace 256-byte");
  if (!evict_size_ok(c, num_layers, n_req))
    return fail(ctx, PIC_ERR_RANGE, "layers x requests x row slices must stay below 2^30");
  const EvictLayout L = evict_layout(num_layers, n_req, weight_heads);
  if (ws_bytes < L.total) return fail(ctx, PIC_ERR_CAPACITY, "workspace has %zu bytes, needs %zu", ws_bytes, L.total);
  if (n_req == 0) return set_error(ctx, PIC_OK, "");
  const Buffer bufs[] = {{"k_cache", k_cache}, {"v_cache", v_cache}, {"weights", d_weights}, {"block tables", d_tables},
                         {"lengths", d_seq_lens}, {"kept list", d_kept}, {"new lengths", d_new_lens}, {"workspace", d_ws}};
  int sms = 0;
  const pic_status st = check_device(ctx, bufs, sizeof(bufs) / sizeof(bufs[0]), &sms);
  if (st != PIC_OK) return st;

  uint8_t* ws = static_cast<uint8_t*>(d_ws);
  EvictParams p{};
  p.paged = paged_view(c, d_tables, n_req, max_blocks);
  fill_freq(c, &p.freq);
  p.layers = num_layers;
  p.n_req = n_req;
  p.kv_heads = m.num_kv_heads;
  p.weight_heads = weight_heads;
  p.head_bytes = m.head_dim * 2;
  p.rope_off = m.rope_offset * 2;
  p.head_items = m.head_dim * 2 / 32;
  p.rope_items = m.rope_dim * 2 / 32;
  p.lens = d_seq_lens;
  p.max_len = std::min(table_capacity(c, max_blocks), cache_rows(c));
  if (renumber) p.max_len = std::min(p.max_len, static_cast<int32_t>(PIC_MAX_ABS_DELTA));  // shifts stay exact
  p.budget = budget;
  p.n_first = n_first;
  p.n_recent = n_recent;
  p.renumber = renumber != 0;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.cache_ls = cache_ls;
  p.weights = d_weights;
  p.weights_ls = weights_ls;
  p.kept = d_kept;
  p.new_lens = d_new_lens;
  p.next_lens = reinterpret_cast<int32_t*>(ws + L.next_lens);
  p.units = reinterpret_cast<EvictUnit*>(ws + L.units);
  p.sel_cap = static_cast<int32_t>(std::min<int64_t>((static_cast<int64_t>(p.max_len) + 3) / 4 * 4, kEvictCachedSlots));
  const EvictShape shape = evict_shape(c, weight_heads, static_cast<int64_t>(num_layers) * n_req, sms);
  p.tensors = shape.tensors;
  p.pieces = shape.pieces;
  p.piece_heads = shape.piece_heads;
  p.slices = shape.slices;
  p.slice_items = shape.slice_items;
  p.status = &reinterpret_cast<WsHeader*>(ws)->status;
  const cudaError_t e = launch_evict(p, m.pairing, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(ctx, e, "eviction launch");
  return set_error(ctx, PIC_OK, "");
}

}  // extern "C"
