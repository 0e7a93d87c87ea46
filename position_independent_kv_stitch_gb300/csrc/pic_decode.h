// Internal interface of the decode-loop operators (pic_write_tokens,
// pic_attend_paged, pic_evict_tokens): parameters shared by their host entries
// (pic_decode.cpp) and their kernels (pic_write.cu, pic_paged.cu,
// pic_evict.cu).  Not part of the public ABI.
//
// Everything a launch needs beyond the caller's device buffers travels in its
// parameters (frequencies included), so the calls upload nothing, wait for
// nothing and can be captured into a graph.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "pic.h"
#include "pic_internal.h"

namespace pic {

// Gives a kernel its dynamic shared memory, once per device (the limit of a
// kernel never changes, so threads may race here).
template <typename Kern>
inline cudaError_t allow_smem(Kern kern, int bytes, std::atomic<uint32_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint32_t bit = dev < 32 ? 1u << dev : 0u;
  if ((done.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// What the entries need of a context (defined in pic_host.cpp).
struct CtxView {
  const pic_model_desc* model;
  const float2* freq;  // rope_dim/2 frequencies in turns, (hi, lo)
  int32_t num_cache_blocks;
};
CtxView ctx_view(const pic_ctx* ctx);

// Longest sequence.  Kernels count slots in 32 bits and look past the end of a
// sequence before they compare: 111 slots in the attention over latent rows, a
// sweep of 4 x 1,024 in the selection, five tiles of 384 in the move.
constexpr int32_t kPagedMaxSlots = INT32_MAX - 8192;

constexpr int kMaxFreqs = 128;  // rope_dim / 2 of the widest head

// The paged cache as the kernels see it: one layer's tables and geometry.
struct PagedView {
  const int32_t* tables;     // [n_tables][max_blocks]
  int32_t n_tables;
  int32_t max_blocks;
  int32_t num_cache_blocks;
  int32_t block_size;
  // slot / block_size = slot * block_mul >> block_shift for every 0 <= slot < 2^31:
  // with 2^(L - 1) < block_size <= 2^L, block_mul = ceil(2^(31 + L) / block_size) is
  // less than 1 too large, which adds less than slot / 2^(31 + L) < 1 / block_size
  uint32_t block_mul;
  int32_t block_shift;       // 31 + L
};

struct FreqTable {
  float2 turns[kMaxFreqs];
};

struct WriteParams {
  PagedView paged;
  FreqTable freq;
  uint8_t axis[kMaxFreqs];   // position axis of each frequency
  const int32_t* pos;        // [n_axes][n_tokens]
  int32_t n_axes;
  int32_t n_tokens;
  const int32_t* req;        // [n_tokens]
  const int32_t* slot;       // [n_tokens], < 0: not written
  const uint8_t* q;
  uint8_t* q_out;
  const uint8_t* k;
  const uint8_t* v;
  int64_t q_stride, q_out_stride, k_stride, v_stride;  // bytes between tokens
  int32_t q_heads, kv_heads;
  int32_t head_bytes;        // bytes of one head (MLA: of the row)
  int32_t rope_off;          // byte offset of the rope slice in a head
  int32_t lph_shift;         // log2 of the lanes that turn one head (8 frequencies each)
  int32_t q_copy_chunks;     // 16-byte chunks of a query head that are only copied (MLA: its latent; 0 in place)
  int32_t k_copy_chunks;     // the same of a key row
  int32_t rot_parts, copy_parts;  // warp tasks of one token
  int32_t rot_iters;         // head steps of one rotating task
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* weights;            // [blocks][weight_heads][block_size] or null
  int32_t weight_heads;
  // norms of the heads (launch_write_normed)
  const uint8_t* q_norm;     // [dims] or null: q as it is
  const uint8_t* k_norm;     // [dims] or null; MLA: of the latent
  int32_t norm_f32;          // their type: fp32 or bf16
  int32_t latent_norm;       // 1: a warp task per token of its own normalises the latent
  float norm_eps, norm_offset;
  uint32_t* status;
};
cudaError_t launch_write(const WriteParams& p, int pairing, cudaStream_t s);
cudaError_t launch_write_normed(const WriteParams& p, int pairing, cudaStream_t s);

// ---- block tables and token lists
struct MapParams {
  int32_t* tables;           // [n_req][max_blocks]
  int32_t n_req, max_blocks, block_size;
  int32_t max_len;           // slots a table holds
  int32_t num_blocks;        // of the cache, and places of the pile
  const int32_t* lens;       // [n_req]
  const int32_t* grow;       // [n_req]
  int32_t* free_blocks;      // [num_blocks], the first *n_free of them free
  const int32_t* n_free;
  int32_t* new_lens;         // may be lens
  int32_t* new_n_free;       // may be n_free
  int32_t n_tokens;
  int32_t* indptr;           // [n_req + 1]
  int32_t* req;              // [n_tokens]
  int32_t* slot;
  int32_t* pos;              // or null
  const int32_t* shift;      // [n_req] or null
  uint32_t* ticket;          // CTAs that have read their inputs; left at 0
  uint32_t* status;
};
cudaError_t launch_map(const MapParams& p, int sm_count, cudaStream_t s);

// ---- paged attention
constexpr int kPagedTile = 16;          // positions of one step of a warp
constexpr int kPagedMaxSms = 256;       // SMs used (workspace sizing)
// Up to here the joins walk the requests' lengths themselves, while they wait
// for the records: 64 requests of 64 slots take 8.7 us (11.4 with weights),
// against 9.6 (12.4) from what the attention kernel left.  256 of 64 slots take
// 13.0 (21.7) by walking and 12.7 (18.4) from what was left, 1,024 of 128 slots
// with weights 66 and 54.
constexpr int kPagedWalkRequests = 128;
constexpr int kPagedMaxHeads = 4096;    // query heads

// What a query row attends to, where it is not simply a request's whole sequence
// (pic_attend_tokens, pic_attend_shared; the kernels' ROWS variants).  The row's slots are
// counted without the gap between those that it sees: the first `head` are slots
// 0 .. head - 1, number v from there on is slot v + gap.
struct RowsParams {
  int32_t shared;            // 0: tokens of requests; 1: one token a request, the prefix shared; 2: the same
                             // without the prefix, whose part of each row is in the records `extra`
  int32_t singles;           // tokens: 1 where requests of more than one token are another kernel's; row r of
                             // the list is then request r's token, else token r
  int32_t n_tokens;          // tokens: rows of q and the outputs
  const int32_t* indptr;     // [n_req + 1] tokens: rows of each request
  const int32_t* slot;       // [rows] tokens: slot of each
  int32_t n_req;             // tokens: requests
  int32_t after_tiles;       // 1: launched while the tiles that the join also reads may still run
  int32_t capacity;          // slots a table holds
  int32_t window, n_first;   // window 0: every slot before
  const int32_t* prefix_table;   // shared: [prefix_blocks]
  const int32_t* prefix_len;     // shared: [1]
  int32_t prefix_blocks, max_prefix;
  int32_t n_extra;           // records per row of the prefix's parts: [n_extra][n_req][q_heads]
  const float* extra_acc;    // [..][D]; not written where the sum is 0
  const float2* extra_ml;
};

struct PagedParams {
  PagedView paged;
  RowsParams rows;
  const uint8_t* q;
  int64_t q_stride;          // bytes between requests
  const int32_t* lens;       // [n_req]
  int32_t n_req;
  int32_t max_len;
  int32_t q_heads, kv_heads, group;
  int32_t passes;            // 16-head passes over a group
  int32_t v_heads;           // kv_heads * passes: what ranges are dealt to
  int32_t parts;             // ranges per virtual head
  float scale_log2;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  int32_t row_bytes;         // one token, all KV heads
  int64_t* first;            // [n_req + 1], of many requests: each one's first tile (if it has any); the tiles in all
  float* rec_acc;            // [parts + n_req][q_heads][D]
  float2* rec_ml;            // [parts + n_req][q_heads]: running max (log2 units) and sum
  float* lse2;               // [n_req][q_heads] log2 units (with weights)
  float* scores;             // [q_heads][score_stride] log2 units (with weights)
  int64_t score_stride;
  void* out;
  int32_t out_bf16;
  float* lse;
  float* weights;
  int32_t weight_heads;
  int32_t weight_ctas;       // CTAs of the last kernel that add weights (the others join records)
  int32_t join_wide;         // 1: one per (request, query head); 0: one warp for each
  uint32_t* status;
};
int paged_ranges_per_sm(int head_dim);  // ranges an SM works on at a time (head_dim 576: MLA rows)
cudaError_t launch_paged(const PagedParams& p, int head_dim, int sm_count, cudaStream_t s);
cudaError_t launch_paged_rows(const PagedParams& p, int head_dim, int sm_count, cudaStream_t s);   // bf16 out, no weights

// ---- attention of tiles of query rows (pic_tile.cu)
constexpr int kTileRows = 128;          // rows of a product: (token, query head of the KV head) pairs
__host__ __device__ constexpr int most_tiles(int head_dim) { return head_dim <= 128 ? 2 : 1; }    // tiles of a CTA
__host__ __device__ constexpr int tile_slots(int head_dim) { return head_dim <= 128 ? 128 : 64; } // slots of a step
struct TileMaps {
  CUtensorMap k, v;
};
struct TileParams {
  PagedView paged;           // tokens: the requests' tables; prefix: its table, alone
  const uint8_t* q;
  int64_t q_stride;          // bytes between tokens
  int32_t n_tokens;
  int32_t q_heads, kv_heads, group;
  // tokens: rows of requests
  const int32_t* indptr;     // [n_req + 1]; null: one request of all tokens, the prefix's readers
  const int32_t* slot;       // [n_tokens]
  int32_t n_req;
  int32_t capacity;          // slots a table holds
  int32_t window, n_first;
  // prefix: a token sees the first min(lens, prefix) slots
  const int32_t* lens;       // [n_tokens]
  const int32_t* prefix_len;
  int32_t max_len;
  int32_t least;             // tokens: requests of fewer tokens are another kernel's
  float scale_log2;          // of |scale| (1 where it is 0)
  int32_t sign;              // of scale: the queries enter as they are, negated, or as 0
  int32_t tiles;             // of a row block
  int32_t blocks;            // row blocks launched per KV head, at least those there are
  int32_t splits;            // parts of a row block's slots
  int32_t box;               // slots of one copy
  int32_t cache_rows;        // one past the last row of the cache
  void* out;                 // splits == 1 of tokens: bf16 [n_tokens][q_heads][D]
  float* lse;
  float* rec_acc;            // else [splits][n_tokens][q_heads][D]
  float2* rec_ml;            // and the running max (log2 units) and sum
  uint32_t* status;
};
cudaError_t launch_tile(const TileParams& p, const TileMaps& maps, int head_dim, cudaStream_t s);
cudaError_t launch_tile_join(const TileParams& p, int head_dim, cudaStream_t s);

// ---- eviction
struct EvictUnit {           // per (layer, request, weight head), in the workspace
  int32_t n_keep;            // kept tokens (0: nothing to move)
  int32_t first_moved;       // kept tokens before this rank stay where they are
};
constexpr int kEvictMoveThreads = 384;   // threads and
constexpr int kEvictMoveCtas = 4;        // CTAs per SM of the move
constexpr int kEvictCachedSlots = 46000; // weights the selection keeps in shared memory
struct EvictParams {
  PagedView paged;
  FreqTable freq;
  int32_t layers, n_req;
  int32_t kv_heads, weight_heads;
  int32_t head_bytes;        // bytes of one head (MLA: of the row)
  int32_t head_items;        // 32-byte items of a head
  int32_t rope_off;
  int32_t rope_items;        // of these, the ones that are turned when renumbering
  const int32_t* lens;
  int32_t max_len;           // longest legal length
  int32_t budget, n_first, n_recent;
  int32_t renumber;
  int32_t sel_cap;           // weights the selection keeps in shared memory
  // the move: a CTA per (layer, request, tensor, piece of the heads, slice of the piece)
  int32_t tensors, pieces, piece_heads;
  int32_t slices, slice_items;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int64_t cache_ls;
  float* weights;
  int64_t weights_ls;        // bytes
  int32_t* kept;             // [layers][n_req][weight_heads][budget]
  int32_t* new_lens;
  int32_t* next_lens;        // workspace [n_req]: what new_lens becomes
  EvictUnit* units;          // workspace [layers * n_req * weight_heads]
  uint32_t* status;
};
cudaError_t launch_evict(const EvictParams& p, int pairing, cudaStream_t s);

}  // namespace pic
