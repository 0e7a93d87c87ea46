// Host entries of a serving step's operators: pic_map_tokens, pic_attend_tokens
// and pic_attend_shared (include/pic.h).  Like the decode loop's they check their
// arguments, fill the launch parameters and launch; they allocate nothing,
// upload nothing and wait for nothing, so they can be captured into a graph.
#include "pic_entry.h"

#include <cmath>

namespace {

using namespace pic;
using namespace pic::entry;

// The parts of PagedParams that a call over rows takes from its arguments; n_list: the rows that the workspace
// is laid out for.
PagedParams rows_params(const CtxView& c, const void* q, int64_t q_stride, int32_t n_rows, int64_t n_list, int32_t num_q_heads,
                        float scale, const void* k_cache, const void* v_cache, void* out, float* lse, uint8_t* ws, int sms) {
  const pic_model_desc& m = *c.model;
  const PagedLayout L = paged_layout(c, n_list, num_q_heads, 0, false);
  PagedParams p{};
  p.q = static_cast<const uint8_t*>(q);
  p.q_stride = q_stride;
  p.n_req = n_rows;
  p.q_heads = num_q_heads;
  p.kv_heads = m.num_kv_heads;
  p.group = num_q_heads / m.num_kv_heads;
  p.passes = paged_passes(p.group);
  p.v_heads = p.kv_heads * p.passes;
  const int used = std::min(sms, kPagedMaxSms);
  p.parts = static_cast<int32_t>(std::max<int64_t>(1, static_cast<int64_t>(used) * paged_ranges_per_sm(m.head_dim) / p.v_heads));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.row_bytes = m.num_kv_heads * m.head_dim * 2;
  p.first = n_rows > kPagedWalkRequests ? reinterpret_cast<int64_t*>(ws + L.first) : nullptr;
  p.rec_acc = reinterpret_cast<float*>(ws + L.rec_acc);
  p.rec_ml = reinterpret_cast<float2*>(ws + L.rec_ml);
  p.out = out;
  p.out_bf16 = 1;
  p.lse = lse;
  p.status = &reinterpret_cast<WsHeader*>(ws)->status;
  return p;
}

// Requests of a call, at most: the kernels count to one past them, some in steps of 1,024, in 32 bits.
constexpr int32_t kMaxRequests = 1 << 30;

// ---- tiles of rows (pic_tile.cu)

// Bytes of a shared prefix, counted for every request, up to which it is read row by row: 8 requests over
// 1,000 slots 13 us (tiles 22), over 2,000 (63 MB) 17 (19), over 4,000 (125 MB) 23 (18).
constexpr int64_t kSharedPrefixReads = int64_t{64} << 20;

// Row blocks of `tiles` tiles per KV head, at most: of n_tokens tokens of n_req requests (each may leave one half filled).
int64_t tile_blocks(const CtxView& c, int32_t tiles, int64_t n_tokens, int64_t n_req, int32_t num_q_heads) {
  const int64_t block = static_cast<int64_t>(kTileRows) * tiles;
  const int64_t rows = n_tokens * (num_q_heads / c.model->num_kv_heads);
  return n_req <= 1 ? (rows + block - 1) / block : rows / block + std::min(n_req, n_tokens);
}
// Parts that a row block's slots are dealt to, at most: enough for two rounds of the SMs.
int64_t most_splits(const CtxView& c, int64_t blocks, int sms) {
  const int64_t ctas = std::max<int64_t>(1, blocks * c.model->num_kv_heads);
  return ctas < 2 * sms ? (2 * sms - 1) / ctas + 1 : 1;
}
// Parts where several requests' blocks differ in length: as many as there are SMs for, of at least
// four steps each; and parts enough for two rounds of the SMs
// where a part keeps 16 steps (recomputed heads of 4 sequences of 16k, 136 CTAs: 167 us in the three parts that it gives,
// 189 whole, 197 in two, 181 in four).  Requests of one token count as a row block here, though the tiles take none of
// them: a chunk beside many is not split.
int32_t tile_splits(const CtxView& c, int64_t blocks, int sms, int64_t max_slots) {
  const int64_t ctas = std::max<int64_t>(1, blocks * c.model->num_kv_heads), step = tile_slots(c.model->head_dim);
  const int64_t fill = std::min(sms / ctas, max_slots / (4 * step)), even = std::min(most_splits(c, blocks, sms), max_slots / (16 * step));
  return static_cast<int32_t>(std::max<int64_t>(1, std::max(fill, ctas < 2 * sms ? even : 0)));
}
// Tiles of a row block, and its parts.  Two tiles keep the tensor cores busy, as one's products run during the other's
// softmax: a step takes them 1.43 us, one tile 0.9.  But one tile starts and ends sooner, and twice as many
// blocks are there for the SMs before slots have to be split and joined.  So both forms' time is
// estimated, for blocks of equal length, as
//   rounds of the SMs x (start and end + steps of a part) + half a part for the last round + the join,
//   a launch and its records written and read,
// and the smaller taken.  Measured (8 KV heads of 128 dims, 4 query heads each; two tiles, one): a prompt of 128 tokens 10.0,
// 7.9 us, of 512 14.5, 10.7, of 4,096 104, 130; 16 tokens behind 16k slots 27.4, 21.8; 608 behind 4k 60, 33;
// 128 behind 16k 38, 49; 64 requests over a prefix of 8k 38.6, 35.5, of 32k 90, 104.  Parts by the same estimate:
// 400 tokens behind 64k 368 us in 6, 297 in 5 (the sixth began a third round of the SMs).
// (Over a shared prefix, whose weights have two parts, a step takes 1.7 and 1.05 us, in about the same proportion: of nine
// such calls the estimate chose the form and parts that were the fastest, or within 6 % of them.)
// Of several requests only the whole is known here: one tile must be the better for all rows in one request, and
// every request's blocks must fit the SMs at once (256 requests may as well be 255 of one token and a prompt).
struct TileShape {
  int32_t tiles, splits;
  double us;
};
TileShape tile_shape_of(const CtxView& c, int32_t tiles, int64_t n_tokens, int32_t num_q_heads, int sms, int64_t max_slots) {
  const double start = tiles == 2 ? 6.5 : 5.0, step_us = tiles == 2 ? 1.43 : 0.9;
  const double record_us = 8.0 * static_cast<double>(n_tokens) * num_q_heads * c.model->head_dim / 8e6;   // of one part
  const int64_t step = tile_slots(c.model->head_dim), steps = std::max<int64_t>(1, (max_slots + step - 1) / step);
  const int64_t blocks = tile_blocks(c, tiles, n_tokens, 1, num_q_heads);
  const int64_t ctas = std::max<int64_t>(1, blocks * c.model->num_kv_heads);
  const int64_t most = std::max<int64_t>(1, std::min(most_splits(c, blocks, sms), steps / 4));
  TileShape best{tiles, 1, 0.0};
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t rounds = (ctas * s + sms - 1) / sms;
    const double part = static_cast<double>((steps + s - 1) / s) * step_us;
    const double us = static_cast<double>(rounds) * (start + part) + 0.5 * part + (s > 1 ? 4.0 + record_us * static_cast<double>(s) : 0.0);
    if (s == 1 || us < best.us) best = {tiles, static_cast<int32_t>(s), us};
  }
  return best;
}
TileShape tile_shape(const CtxView& c, int64_t n_tokens, int64_t n_req, int32_t num_q_heads, int sms, int64_t max_slots) {
  TileShape best = tile_shape_of(c, 1, n_tokens, num_q_heads, sms, max_slots);
  // (rows of one tile: the same blocks)
  if (most_tiles(c.model->head_dim) == 2 && n_tokens * (num_q_heads / c.model->num_kv_heads) > kTileRows) {
    const TileShape two = tile_shape_of(c, 2, n_tokens, num_q_heads, sms, max_slots);
    const bool at_once = n_req <= 1 || tile_blocks(c, 1, n_tokens, n_req, num_q_heads) * c.model->num_kv_heads <= sms;
    if (two.us <= best.us || !at_once) best = two;
  }
  if (n_req > 1) best.splits = tile_splits(c, tile_blocks(c, best.tiles, n_tokens, n_req, num_q_heads), sms, max_slots);
  return best;
}
// Rows of the row-by-row kernels' list in pic_attend_tokens: beside tiles they take the requests, of which those of
// one token are theirs; else the tokens, which are no more than the requests where the cache has blocks.
int64_t listed_rows(const CtxView& c, int64_t n_tokens, int64_t n_req) {
  return c.num_cache_blocks > 0 ? std::min(n_tokens, n_req) : n_tokens;
}
// Records that a call's tiles leave, at most, whatever the device, the slots and the number of requests.  With rows R of
// a KV head in row blocks of B, thus b = ceil(R / B) of them or more, a row is in at most (2 SMs - 1) / (b KV heads) + 1
// parts, and R / b <= min(R, B):
//   records <= (2 SMs - 1) min(R, B) + R KV heads,
// the second term of pic_attend_shared, where one part leaves records too; the tokens' are only split where
// b KV heads < 2 SMs, so R KV heads <= (2 SMs - 1) B.  As parts fall where blocks are added the records
// themselves go up and down with the rows; this bound never falls, so that a workspace serves smaller calls too.
int64_t tile_records(const CtxView& c, int64_t n_tokens, int32_t num_q_heads, bool shared) {
  const int64_t kv = c.model->num_kv_heads, rows = n_tokens * (num_q_heads / kv);
  const int64_t block = static_cast<int64_t>(kTileRows) * most_tiles(c.model->head_dim), parts = 2 * kPagedMaxSms - 1;
  return parts * std::min(rows, block) + (shared ? rows * kv : std::min(rows * kv, parts * block));
}
// Workspace of a call: the row-by-row kernels' part (n_list rows), then the tiles' records.
struct RowsLayout {
  size_t acc, ml, total;
};
RowsLayout rows_layout(const CtxView& c, int64_t n_list, int64_t num_q_heads, int64_t records) {
  const int64_t kv = c.model->num_kv_heads;
  RowsLayout L{};
  L.acc = paged_layout(c, n_list, num_q_heads, 0, false).total;
  // (a pass more over the query heads halves their ranges: fewer heads may take more)
  for (int64_t p = 1; p < paged_passes(static_cast<int32_t>(num_q_heads / kv)); ++p)
    L.acc = std::max(L.acc, paged_layout(c, n_list, 16 * p * kv, 0, false).total);
  L.ml = align_up(L.acc + records * c.model->head_dim * sizeof(float), kWsAlign);
  L.total = align_up(L.ml + records * sizeof(float2), kWsAlign);
  return L;
}
RowsLayout tokens_layout(const CtxView& c, int64_t n_tokens, int64_t n_req, int32_t num_q_heads) {
  return rows_layout(c, listed_rows(c, n_tokens, n_req), num_q_heads, n_tokens > 1 ? tile_records(c, n_tokens, num_q_heads, false) : 0);
}
RowsLayout shared_layout(const CtxView& c, int64_t n_req, int32_t num_q_heads) {
  return rows_layout(c, n_req, num_q_heads, tile_records(c, n_req, num_q_heads, true));
}

// One cache tensor as the tiles read it: whole groups of 8 rows, planes of 64 dims
// inside; or, where blocks are no multiple of 8, rows of one plane.  Rows past the end read as zeros.
bool encode_cache(CUtensorMap* map, const void* base, const CtxView& c, int32_t box) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const pic_model_desc& m = *c.model;
  const cuuint64_t rows = static_cast<cuuint64_t>(c.num_cache_blocks) * m.block_size, row = static_cast<cuuint64_t>(m.num_kv_heads) * m.head_dim * 2;
  const cuuint64_t heads = m.num_kv_heads, d = m.head_dim;
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  const auto run = [&](cuuint32_t rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* boxes) {
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, boxes, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (box >= 8) {
    const cuuint64_t dims[5] = {64, 8, d / 64, rows / 8, heads}, strides[4] = {row, 128, 8 * row, d * 2};
    const cuuint32_t boxes[5] = {64, 8, static_cast<cuuint32_t>(d / 64), static_cast<cuuint32_t>(box / 8), 1};
    return run(5, dims, strides, boxes);
  }
  const cuuint64_t dims[3] = {d, heads, rows}, strides[2] = {d * 2, row};
  const cuuint32_t boxes[3] = {64, 1, static_cast<cuuint32_t>(box)};
  return run(3, dims, strides, boxes);
}

// The tiles' parameters that follow from a call's rows; false without a tensor map.
bool tile_params(const CtxView& c, const PagedParams& p, float scale, TileParams* t, TileMaps* maps) {
  const pic_model_desc& m = *c.model;
  t->q = p.q;
  t->q_stride = p.q_stride;
  t->n_tokens = p.n_req;
  t->q_heads = p.q_heads;
  t->kv_heads = p.kv_heads;
  t->group = p.group;
  t->sign = scale > 0.0f ? 1 : (scale < 0.0f ? -1 : 0);
  t->scale_log2 = t->sign == 0 ? 1.0f : std::fabs(scale) * 1.4426950408889634f;
  t->box = std::min(m.block_size & -m.block_size, tile_slots(m.head_dim));
  t->cache_rows = c.num_cache_blocks * m.block_size;
  t->status = p.status;
  return encode_cache(&maps->k, p.k_cache, c, t->box) && encode_cache(&maps->v, p.v_cache, c, t->box);
}

// Arguments that both attentions share; PIC_OK to go on.
pic_status check_rows(pic_ctx* ctx, const CtxView& c, const void* q, int64_t q_stride, int32_t n_rows, int32_t num_q_heads,
                      float scale, const void* k_cache, const void* v_cache, const void* out, const float* lse, const void* ws) {
  const pic_model_desc& m = *c.model;
  if (m.kind != PIC_KIND_GQA)
    return fail(ctx, PIC_ERR_UNSUPPORTED, "MLA models: attend with pic_attend_paged or pic_attend_decode");
  if (!paged_heads_ok(c, num_q_heads))
    return fail(ctx, PIC_ERR_INVALID_ARG, "num_q_heads must be a positive multiple of num_kv_heads");
  if (!std::isfinite(scale)) return fail(ctx, PIC_ERR_INVALID_ARG, "softmax_scale must be finite");
  if (!k_cache || !v_cache || !ws || (n_rows > 0 && (!q || !out)))
    return fail(ctx, PIC_ERR_INVALID_ARG, "null q, cache, out or workspace");
  const int64_t q_bytes = static_cast<int64_t>(num_q_heads) * m.head_dim * 2;
  if (static_cast<int64_t>(m.num_kv_heads) * m.head_dim * 2 > std::numeric_limits<int32_t>::max() ||
      !paged_size_ok(n_rows, num_q_heads))
    return fail(ctx, PIC_ERR_RANGE, "more than %d query heads, or 2^30 in all", kPagedMaxHeads);
  if (n_rows > 1 && q_stride < q_bytes) return fail(ctx, PIC_ERR_RANGE, "q_stride smaller than a token's heads");
  if (!aligned(q, 16) || (q_stride & 15) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return fail(ctx, PIC_ERR_ALIGNMENT, "q, its stride, caches and out must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(ws, kWsAlign))
    return fail(ctx, PIC_ERR_ALIGNMENT, "lse must be 4-byte aligned, the workspace 256-byte");
  return PIC_OK;
}

}  // namespace

extern "C" {

size_t pic_map_tokens_workspace_bytes(const pic_ctx* ctx, int32_t n_req) {
  return ctx && n_req >= 0 && n_req <= kMaxRequests ? sizeof(WsHeader) : 0;
}

pic_status pic_map_tokens(pic_ctx* ctx, const pic_token_map* t, void* d_ws, size_t ws_bytes, pic_stream_t stream) {
  if (!ctx || !t) return fail(ctx, PIC_ERR_INVALID_ARG, "null ctx or map");
  const CtxView c = ctx_view(ctx);
  if (t->n_req < 0 || t->max_blocks < 0 || t->n_tokens < 0) return fail(ctx, PIC_ERR_INVALID_ARG, "negative size");
  if (t->n_req > kMaxRequests) return fail(ctx, PIC_ERR_RANGE, "more than 2^30 requests");
  const bool some = t->n_req > 0;
  if (!t->d_n_free || !t->d_new_n_free || !t->d_indptr || (c.num_cache_blocks > 0 && !t->d_free_blocks) ||
      (some && (!t->d_seq_lens || !t->d_grow || !t->d_new_lens || (!t->d_block_tables && t->max_blocks > 0))) ||
      (t->n_tokens > 0 && (!t->d_req || !t->d_slot)))
    return fail(ctx, PIC_ERR_INVALID_ARG, "null lengths, growth, block tables, free blocks, offsets or token lists");
  if (!d_ws || ws_bytes < sizeof(WsHeader)) return fail(ctx, PIC_ERR_CAPACITY, "workspace needs %zu bytes", sizeof(WsHeader));
  for (const void* x : {static_cast<const void*>(t->d_seq_lens), static_cast<const void*>(t->d_grow),
                        static_cast<const void*>(t->d_block_tables), static_cast<const void*>(t->d_free_blocks),
                        static_cast<const void*>(t->d_n_free), static_cast<const void*>(t->d_shift),
                        static_cast<const void*>(t->d_new_lens), static_cast<const void*>(t->d_new_n_free),
                        static_cast<const void*>(t->d_indptr), static_cast<const void*>(t->d_req),
                        static_cast<const void*>(t->d_slot), static_cast<const void*>(t->d_pos)})
    if (!aligned(x, 4)) return fail(ctx, PIC_ERR_ALIGNMENT, "lists must be 4-byte aligned");
  if (!aligned(d_ws, kWsAlign)) return fail(ctx, PIC_ERR_ALIGNMENT, "the workspace must be 256-byte aligned");
  const bool tokens = t->n_tokens > 0;
  const Buffer bufs[] = {{"lengths", some ? t->d_seq_lens : nullptr}, {"growth", some ? t->d_grow : nullptr},
                         {"block tables", some ? t->d_block_tables : nullptr}, {"free blocks", t->d_free_blocks},
                         {"free count", t->d_n_free}, {"shifts", some ? t->d_shift : nullptr},
                         {"new lengths", some ? t->d_new_lens : nullptr}, {"new free count", t->d_new_n_free},
                         {"offsets", t->d_indptr}, {"requests", tokens ? t->d_req : nullptr},
                         {"slots", tokens ? t->d_slot : nullptr}, {"positions", tokens ? t->d_pos : nullptr}, {"workspace", d_ws}};
  int sms = 0;
  const pic_status st = check_device(ctx, bufs, sizeof(bufs) / sizeof(bufs[0]), &sms);
  if (st != PIC_OK) return st;
  MapParams p{};
  p.tables = t->d_block_tables;
  p.n_req = t->n_req;
  p.max_blocks = t->max_blocks;
  p.block_size = c.model->block_size;
  p.max_len = static_cast<int32_t>(std::min<int64_t>(static_cast<int64_t>(t->max_blocks) * c.model->block_size, kPagedMaxSlots));
  p.num_blocks = c.num_cache_blocks;
  p.lens = t->d_seq_lens;
  p.grow = t->d_grow;
  p.free_blocks = t->d_free_blocks;
  p.n_free = t->d_n_free;
  p.new_lens = t->d_new_lens;
  p.new_n_free = t->d_new_n_free;
  p.n_tokens = t->n_tokens;
  p.indptr = t->d_indptr;
  p.req = t->d_req;
  p.slot = t->d_slot;
  p.pos = t->d_pos;
  p.shift = t->d_shift;
  WsHeader* h = static_cast<WsHeader*>(d_ws);
  p.ticket = &h->ticket;
  p.status = &h->status;
  const cudaError_t e = launch_map(p, sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(ctx, e, "token map launch");
  return set_error(ctx, PIC_OK, "");
}

size_t pic_attend_tokens_workspace_bytes(const pic_ctx* ctx, int32_t n_tokens, int32_t n_req, int32_t num_q_heads) {
  if (!ctx || n_tokens < 0 || n_req < 0 || n_req > kMaxRequests) return 0;
  const CtxView c = ctx_view(ctx);
  if (c.model->kind != PIC_KIND_GQA || !paged_heads_ok(c, num_q_heads) || !paged_size_ok(n_tokens, num_q_heads)) return 0;
  return tokens_layout(c, n_tokens, n_req, num_q_heads).total;
}

pic_status pic_attend_tokens(pic_ctx* ctx, const void* q, int64_t q_stride, int32_t n_tokens, int32_t num_q_heads,
                             float softmax_scale, const void* k_cache, const void* v_cache, const int32_t* d_tables, int32_t n_req,
                             int32_t max_blocks, const int32_t* d_indptr, const int32_t* d_slot, int32_t window, int32_t n_first,
                             void* out, float* lse, void* d_ws, size_t ws_bytes, pic_stream_t stream) {
  if (!ctx) return fail(nullptr, PIC_ERR_INVALID_ARG, "null ctx");
  const CtxView c = ctx_view(ctx);
  if (n_tokens < 0 || n_req < 0 || max_blocks < 0) return fail(ctx, PIC_ERR_INVALID_ARG, "negative size");
  if (window < 0 || n_first < 0) return fail(ctx, PIC_ERR_INVALID_ARG, "window and n_first must not be negative");
  if (n_req > kMaxRequests) return fail(ctx, PIC_ERR_RANGE, "more than 2^30 requests");
  const pic_status ok = check_rows(ctx, c, q, q_stride, n_tokens, num_q_heads, softmax_scale, k_cache, v_cache, out, lse, d_ws);
  if (ok != PIC_OK) return ok;
  const bool some = n_tokens > 0 && n_req > 0;
  if (some && (!d_indptr || !d_slot || (!d_tables && max_blocks > 0)))
    return fail(ctx, PIC_ERR_INVALID_ARG, "null block table, offsets or slots");
  if (!aligned(d_tables, 4) || !aligned(d_indptr, 4) || !aligned(d_slot, 4))
    return fail(ctx, PIC_ERR_ALIGNMENT, "tables, offsets and slots must be 4-byte aligned");
  const RowsLayout L = tokens_layout(c, n_tokens, n_req, num_q_heads);
  if (ws_bytes < L.total) return fail(ctx, PIC_ERR_CAPACITY, "workspace has %zu bytes, needs %zu", ws_bytes, L.total);
  if (!some) return set_error(ctx, PIC_OK, "");
  const Buffer bufs[] = {{"q", q}, {"k_cache", k_cache}, {"v_cache", v_cache}, {"block tables", d_tables}, {"offsets", d_indptr},
                         {"slots", d_slot}, {"out", out}, {"lse", lse}, {"workspace", d_ws}};
  int sms = 0;
  const pic_status st = check_device(ctx, bufs, sizeof(bufs) / sizeof(bufs[0]), &sms);
  if (st != PIC_OK) return st;
  const int64_t n_list = listed_rows(c, n_tokens, n_req);
  PagedParams p = rows_params(c, q, q_stride, n_tokens, n_list, num_q_heads, softmax_scale, k_cache, v_cache, out, lse,
                              static_cast<uint8_t*>(d_ws), sms);
  p.paged = paged_view(c, d_tables, n_req, max_blocks);
  p.rows.indptr = d_indptr;
  p.rows.slot = d_slot;
  p.rows.n_req = n_req;
  p.rows.n_tokens = n_tokens;
  p.rows.capacity = table_capacity(c, max_blocks);
  p.rows.window = window;
  p.rows.n_first = n_first;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int used = std::min(sms, kPagedMaxSms);
  // Requests of several tokens go in tiles of rows, single tokens row by row, each
  // request by its own count, which is on the device: both kernels are
  // launched and each leaves the other's alone.  One suffices where there are no more tokens than
  // requests, or one request.
  const bool tiles = n_tokens > n_req && c.num_cache_blocks > 0;   // (of a cache without blocks there is no tensor map)
  if (tiles) {
    TileParams t{};
    TileMaps maps;
    if (!tile_params(c, p, softmax_scale, &t, &maps)) return fail(ctx, PIC_ERR_CUDA, "no tensor map of the cache");
    t.paged = p.paged;
    t.indptr = d_indptr;
    t.slot = d_slot;
    t.n_req = n_req;
    t.capacity = p.rows.capacity;
    t.window = window;
    t.n_first = n_first;
    t.least = n_req > 1 ? 2 : 1;
    const int64_t slots = window > 0 ? std::min<int64_t>(t.capacity, static_cast<int64_t>(window) + n_first + n_tokens) : t.capacity;
    const TileShape shape = tile_shape(c, n_tokens, n_req, num_q_heads, used, slots);
    t.tiles = shape.tiles;
    t.splits = shape.splits;
    t.blocks = static_cast<int32_t>(tile_blocks(c, t.tiles, n_tokens, n_req, num_q_heads));
    t.out = out;
    t.lse = lse;
    if (t.splits > 1) {
      t.rec_acc = reinterpret_cast<float*>(static_cast<uint8_t*>(d_ws) + L.acc);
      t.rec_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(d_ws) + L.ml);
    }
    cudaError_t e = launch_tile(t, maps, c.model->head_dim, cs);
    if (e == cudaSuccess && n_req > 1) {
      p.rows.singles = 1;
      p.rows.after_tiles = 1;
      p.n_req = n_req;   // the list is of requests
      p.first = n_req > kPagedWalkRequests ? p.first : nullptr;
      e = launch_paged_rows(p, c.model->head_dim, used, cs);
    }
    if (e == cudaSuccess && t.splits > 1) e = launch_tile_join(t, c.model->head_dim, cs);
    if (e != cudaSuccess) return cuda_fail(ctx, e, "token attention launch");
  } else {
    const cudaError_t e = launch_paged_rows(p, c.model->head_dim, used, cs);
    if (e != cudaSuccess) return cuda_fail(ctx, e, "token attention launch");
  }
  return set_error(ctx, PIC_OK, "");
}

size_t pic_attend_shared_workspace_bytes(const pic_ctx* ctx, int32_t n_req, int32_t num_q_heads) {
  if (!ctx || n_req < 0) return 0;
  const CtxView c = ctx_view(ctx);
  if (c.model->kind != PIC_KIND_GQA || !paged_heads_ok(c, num_q_heads) || !paged_size_ok(n_req, num_q_heads)) return 0;
  return shared_layout(c, n_req, num_q_heads).total;
}

pic_status pic_attend_shared(pic_ctx* ctx, const void* q, int64_t q_stride, int32_t n_req, int32_t num_q_heads, float softmax_scale,
                             const void* k_cache, const void* v_cache, const int32_t* d_prefix_table, int32_t prefix_blocks,
                             const int32_t* d_prefix_len, const int32_t* d_tables, int32_t max_blocks, const int32_t* d_seq_lens,
                             int32_t max_seq_len, void* out, float* lse, void* d_ws, size_t ws_bytes, pic_stream_t stream) {
  if (!ctx) return fail(nullptr, PIC_ERR_INVALID_ARG, "null ctx");
  const CtxView c = ctx_view(ctx);
  if (n_req < 0 || max_blocks < 0 || max_seq_len < 0 || prefix_blocks < 0) return fail(ctx, PIC_ERR_INVALID_ARG, "negative size");
  const pic_status ok = check_rows(ctx, c, q, q_stride, n_req, num_q_heads, softmax_scale, k_cache, v_cache, out, lse, d_ws);
  if (ok != PIC_OK) return ok;
  const bool some = n_req > 0;
  if (some && (!d_seq_lens || !d_prefix_len || (!d_tables && max_blocks > 0) || (!d_prefix_table && prefix_blocks > 0)))
    return fail(ctx, PIC_ERR_INVALID_ARG, "null block table, prefix table or lengths");
  if (max_seq_len > table_capacity(c, max_blocks))
    return fail(ctx, PIC_ERR_RANGE, "max_seq_len %d exceeds the %d slots a block table holds", max_seq_len,
                table_capacity(c, max_blocks));
  if (!aligned(d_tables, 4) || !aligned(d_seq_lens, 4) || !aligned(d_prefix_table, 4) || !aligned(d_prefix_len, 4))
    return fail(ctx, PIC_ERR_ALIGNMENT, "tables and lengths must be 4-byte aligned");
  const RowsLayout L = shared_layout(c, n_req, num_q_heads);
  if (ws_bytes < L.total) return fail(ctx, PIC_ERR_CAPACITY, "workspace has %zu bytes, needs %zu", ws_bytes, L.total);
  if (!some) return set_error(ctx, PIC_OK, "");
  const Buffer bufs[] = {{"q", q}, {"k_cache", k_cache}, {"v_cache", v_cache}, {"prefix table", d_prefix_table},
                         {"prefix length", d_prefix_len}, {"block tables", d_tables}, {"lengths", d_seq_lens}, {"out", out},
                         {"lse", lse}, {"workspace", d_ws}};
  int sms = 0;
  const pic_status st = check_device(ctx, bufs, sizeof(bufs) / sizeof(bufs[0]), &sms);
  if (st != PIC_OK) return st;
  PagedParams p = rows_params(c, q, q_stride, n_req, n_req, num_q_heads, softmax_scale, k_cache, v_cache, out, lse,
                              static_cast<uint8_t*>(d_ws), sms);
  p.paged = paged_view(c, d_tables, n_req, max_blocks);
  p.lens = d_seq_lens;
  p.max_len = max_seq_len;
  p.rows.shared = 1;
  p.rows.prefix_table = d_prefix_table;
  p.rows.prefix_len = d_prefix_len;
  p.rows.prefix_blocks = prefix_blocks;
  p.rows.max_prefix = table_capacity(c, prefix_blocks);
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int used = std::min(sms, kPagedMaxSms);
  cudaError_t e = cudaSuccess;
  // A short prefix is read row by row like the rest: a launch less, and its repeated reads come from L2.
  const double prefix_reads = 2.0 * n_req * p.rows.max_prefix * p.row_bytes;   // (may pass 64 bits)
  if (prefix_reads > kSharedPrefixReads) {
    // the prefix in tiles of all requests' rows, whose records the join adds to those of the rest
    TileParams t{};
    TileMaps maps;
    if (!tile_params(c, p, softmax_scale, &t, &maps)) return fail(ctx, PIC_ERR_CUDA, "no tensor map of the cache");
    t.paged = paged_view(c, d_prefix_table, 1, prefix_blocks);
    t.n_req = 1;
    t.least = 1;
    t.capacity = p.rows.max_prefix;
    t.lens = d_seq_lens;
    t.prefix_len = d_prefix_len;
    t.max_len = max_seq_len;
    // an eighth of the SMs is left to the slots behind the prefix, whose kernel starts beside the tiles (64
    // requests over 32k slots and 1-2,048 of their own: 12 parts 101 us, 14 96, 16 (128 CTAs) 94, 18 95, 19 (every SM)
    // 106)
    const TileShape shape = tile_shape(c, n_req, 1, num_q_heads, used - used / 8, t.capacity);
    t.tiles = shape.tiles;
    t.splits = shape.splits;
    t.blocks = static_cast<int32_t>(tile_blocks(c, t.tiles, n_req, 1, num_q_heads));
    t.rec_acc = reinterpret_cast<float*>(static_cast<uint8_t*>(d_ws) + L.acc);
    t.rec_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(d_ws) + L.ml);
    e = launch_tile(t, maps, c.model->head_dim, cs);
    p.rows.shared = 2;
    p.rows.after_tiles = 1;
    p.rows.n_extra = t.splits;
    p.rows.extra_acc = t.rec_acc;
    p.rows.extra_ml = t.rec_ml;
  }
  if (e == cudaSuccess) e = launch_paged_rows(p, c.model->head_dim, used, cs);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "shared-prefix attention launch");
  return set_error(ctx, PIC_OK, "");
}

}  // extern "C"
