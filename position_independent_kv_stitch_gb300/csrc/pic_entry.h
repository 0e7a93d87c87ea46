// What the host entries of the decode loop share (pic_decode.cpp, pic_serve.cpp):
// errors, the device check, the paged view of a context, and the layout of the
// paged attention's workspace.
#pragma once

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <limits>

#include "pic_decode.h"

namespace pic {
namespace entry {

inline pic_status fail(pic_ctx* ctx, pic_status st, const char* fmt, ...) __attribute__((format(printf, 3, 4)));
inline pic_status fail(pic_ctx* ctx, pic_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_error(ctx, st, buf);
}
inline pic_status cuda_fail(pic_ctx* ctx, cudaError_t e, const char* what) {
  return fail(ctx, PIC_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The launching device, and that every buffer is memory of that device: these
// operators stream with no regard to the host link, and a pageable host
// pointer would fault.
struct Buffer {
  const char* name;
  const void* ptr;
};
inline pic_status check_device(pic_ctx* ctx, const Buffer* bufs, int n, int* sm_count) {
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

inline PagedView paged_view(const CtxView& c, const int32_t* d_tables, int32_t n_tables, int32_t max_blocks) {
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

inline void fill_freq(const CtxView& c, FreqTable* t) { std::memcpy(t->turns, c.freq, c.model->rope_dim / 2 * sizeof(float2)); }

// Longest sequence a block table can hold (none, where the cache has no block).
inline int32_t table_capacity(const CtxView& c, int32_t max_blocks) {
  if (c.num_cache_blocks == 0) return 0;
  const int64_t n = static_cast<int64_t>(max_blocks) * c.model->block_size;
  return static_cast<int32_t>(std::min<int64_t>(n, kPagedMaxSlots));
}

// Rows of the cache: a sequence whose blocks are all its own is no longer.
inline int32_t cache_rows(const CtxView& c) {
  return static_cast<int32_t>(std::min<int64_t>(static_cast<int64_t>(c.num_cache_blocks) * c.model->block_size, kPagedMaxSlots));
}

inline bool weight_heads_ok(const CtxView& c, int32_t n) { return n == 1 || n == c.model->num_kv_heads; }

struct PagedLayout {
  size_t first, lse2, rec_ml, rec_acc, scores, total;
  int64_t score_stride;
};
inline int32_t paged_passes(int32_t group) { return (group + 15) / 16; }
// Width of an output row: the head's, or the latent's.
inline int32_t paged_out_dim(const CtxView& c) { return c.model->kind == PIC_KIND_MLA ? c.model->rope_offset : c.model->head_dim; }
inline int64_t paged_max_parts(int32_t v_heads, int head_dim) {
  return std::max<int64_t>(1, static_cast<int64_t>(kPagedMaxSms) * paged_ranges_per_sm(head_dim) / v_heads);
}
inline PagedLayout paged_layout(const CtxView& c, int64_t n_req, int64_t q_heads, int64_t max_len, bool weights) {
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
inline bool paged_heads_ok(const CtxView& c, int32_t num_q_heads) {
  return num_q_heads > 0 && num_q_heads % c.model->num_kv_heads == 0;
}
// What one call takes: sizes beyond it would overflow the kernels' counts (and a workspace's size).
inline bool paged_size_ok(int64_t n_req, int64_t num_q_heads) {
  return num_q_heads <= kPagedMaxHeads && n_req * num_q_heads <= std::numeric_limits<int32_t>::max() / 2;
}

}  // namespace entry
}  // namespace pic
