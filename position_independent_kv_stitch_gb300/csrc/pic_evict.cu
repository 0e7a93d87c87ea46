// Evicts cached tokens by accumulated attention weight (sm_103a).
//
// Per layer, request and weight head (all KV heads share one, or each has its
// own), a sequence longer than the budget keeps its first n_first tokens, its
// last n_recent, and of the tokens between the heaviest that fit, equal
// weights to the lower slot.  The kept tokens slide down, in order, to slots
// 0 .. budget - 1; with `renumber` a key that moved from slot s to j is turned
// by R(j - s), so that the cache is again a sequence of consecutive positions.
//
// Two launches:
//   * k_evict_select, one CTA per (layer, request, weight head): the weight of
//     the last token that fits is found by radix selection over the weights'
//     bits (four passes of 8 bits, counts in shared memory), then one ordered
//     pass writes the kept slots, ascending.
//   * k_evict_move, one CTA per (layer, request, KV head) and tensor: moves the
//     rows in place.  Rank j lands on slot j <= its own, so a tile of ranks
//     may be read long before the tiles below it are written, and may be
//     written once every thread of the CTA has read it: tiles are read one
//     ahead, with one barrier between a tile's reads and its writes.  Kept tokens
//     before the first evicted one are already in place and not touched.
// Bound: HBM (moved rows once in and once out) for large evictions, the
// latency of the passes over the weights for small ones.
#include <cfloat>

#include "pic_decode.h"
#include "pic_device.cuh"
#include "pic_paged.cuh"

namespace pic {
namespace {

using namespace dev;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;

// Order of the weights as unsigned integers: NaN lowest, -0 equal to 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) != 0 ? ~u : (u | 0x80000000u);
}

// Sum of v over the CTA's threads before this one, and over all of them.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += up;
  }
  __syncthreads();   // warp_sums is free
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) {
    const int s = warp_sums[i];
    before += i < warp ? s : 0;
    total += s;
  }
  return before + incl - v;
}

__global__ void __launch_bounds__(kSelThreads) k_evict_select(const __grid_constant__ EvictParams P) {
  __shared__ int s_hist[256];
  __shared__ int s_warp[kSelWarps];
  __shared__ int s_pick[2];
  __shared__ int s_first_moved;
  const int64_t unit = blockIdx.x;
  const int wh = static_cast<int>(unit % P.weight_heads);
  const int r = static_cast<int>(unit / P.weight_heads % P.n_req);
  const int64_t layer = unit / P.weight_heads / P.n_req;
  int32_t* kept = P.kept + unit * P.budget;
  const int len = __ldg(P.lens + r);
  const int tid = threadIdx.x;

  // a request whose length or blocks are not legal keeps all it has
  bool bad = len < 0 || len > P.max_len;
  if (bad) {
    if (tid == 0) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_BAD_LENGTH));
  } else {
    const int blocks = (len + P.paged.block_size - 1) / P.paged.block_size;
    bool mine = false;
    for (int b = tid; b < blocks; b += kSelThreads) {
      const int32_t block = __ldg(P.paged.tables + static_cast<int64_t>(r) * P.paged.max_blocks + b);
      if (block < 0 || block >= P.paged.num_cache_blocks) {
        mine = true;
        raise_block(P.status, r, b * P.paged.block_size);
      }
    }
    bad = __syncthreads_or(mine);
  }
  if (tid == 0 && layer == 0 && wh == 0) P.next_lens[r] = bad || len <= P.budget ? len : P.budget;
  if (bad || len <= P.budget) {
    for (int j = tid; j < P.budget; j += kSelThreads) kept[j] = !bad && j < len ? j : -1;
    if (tid == 0) P.units[unit] = EvictUnit{0, 0};
    return;
  }

  const uint8_t* wl = reinterpret_cast<const uint8_t*>(P.weights) + layer * P.weights_ls;
  auto key_of = [&](int slot) -> uint32_t {
    const int64_t row = paged_row(P.paged, r, slot);
    const int64_t block = row / P.paged.block_size, at = row - block * P.paged.block_size;
    return weight_key(*(reinterpret_cast<const float*>(wl) + (block * P.weight_heads + wh) * P.paged.block_size + at));
  };
  const int lo = P.n_first, hi = len - P.n_recent;     // candidates: slots [lo, hi)
  const int want = P.budget - P.n_first - P.n_recent;  // how many of them stay; fewer than hi - lo
  uint32_t border = 0xffffffffu;                       // key of the last one that stays
  int ties = 0;                                        // candidates of that key that stay
  if (want > 0) {
    uint32_t prefix = 0, mask = 0;
    int left = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) s_hist[i] = 0;
      __syncthreads();
      for (int s = lo + tid; s < hi; s += kSelThreads) {
        const uint32_t k = key_of(s);
        if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & 255u], 1);
      }
      __syncthreads();
      // digits from the top: the one in which the count reaches `left`
      int total;
      const int n = tid < 256 ? s_hist[255 - tid] : 0;
      const int above = block_scan(n, s_warp, total);
      if (tid < 256 && above < left && above + n >= left) {
        s_pick[0] = 255 - tid;
        s_pick[1] = left - above;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(s_pick[0]) << shift;
      mask |= 255u << shift;
      left = s_pick[1];
      __syncthreads();
    }
    border = prefix;
    ties = left;
  }
  if (tid == 0) s_first_moved = P.budget;
  int n_kept = 0, n_ties = 0;
  for (int base = 0; base < len; base += kSelThreads) {
    const int s = base + tid;
    const bool cand = s >= lo && s < hi;
    const uint32_t k = cand && want > 0 ? key_of(s) : 0u;
    const bool tie = cand && want > 0 && k == border;
    int total;
    const int ties_before = n_ties + block_scan(tie ? 1 : 0, s_warp, total);
    n_ties += total;
    const bool keep = s < len && (!cand || (want > 0 && (k > border || (tie && ties_before < ties))));
    const int rank = n_kept + block_scan(keep ? 1 : 0, s_warp, total);
    n_kept += total;
    if (keep) {
      kept[rank] = s;
      if (rank != s) atomicMin(&s_first_moved, rank);
    }
  }
  __syncthreads();
  if (tid == 0) P.units[unit] = EvictUnit{P.budget, s_first_moved};
}

constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 4;    // items in flight per thread and tile

// grid.x: (layer, request, KV head); grid.y: 0 keys, 1 values, last: the weights.
template <int PAIRING>
__global__ void __launch_bounds__(kMoveThreads) k_evict_move(const __grid_constant__ EvictParams P, int tensors) {
  constexpr bool NEOX = PAIRING == kNeox;
  const int64_t unit = blockIdx.x;
  const int h = static_cast<int>(unit % P.kv_heads);
  const int r = static_cast<int>(unit / P.kv_heads % P.n_req);
  const int64_t layer = unit / P.kv_heads / P.n_req;
  const int wh = P.weight_heads == 1 ? 0 : h;
  const int which = blockIdx.y;
  const int64_t wu = (layer * P.n_req + r) * P.weight_heads + wh;
  if (unit % P.kv_heads == 0 && layer == 0 && which == 0 && threadIdx.x == 0) P.new_lens[r] = P.next_lens[r];
  const EvictUnit u = P.units[wu];
  if (u.first_moved >= u.n_keep) return;
  const int32_t* kept = P.kept + wu * P.budget;
  const int bs = P.paged.block_size;

  if (which == tensors) {   // the weights move with their tokens
    if (h >= P.weight_heads) return;
    float* wl = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(P.weights) + layer * P.weights_ls);
    auto at = [&](int slot) -> float* {
      const int64_t row = paged_row(P.paged, r, slot), block = row / bs;
      return wl + (block * P.weight_heads + wh) * bs + (row - block * bs);
    };
    for (int base = u.first_moved; base < u.n_keep; base += kMoveThreads * kMoveBatch) {
      float x[kMoveBatch];
#pragma unroll
      for (int i = 0; i < kMoveBatch; ++i) {
        const int j = base + i * kMoveThreads + threadIdx.x;
        if (j < u.n_keep) x[i] = *at(kept[j]);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMoveBatch; ++i) {
        const int j = base + i * kMoveThreads + threadIdx.x;
        if (j < u.n_keep) *at(j) = x[i];
      }
    }
    return;
  }

  // A row is cut into items of two 16-byte chunks, one per thread: a turned
  // item holds both members of its 8 pairs.
  uint8_t* cache = (which == 0 ? P.k_cache : P.v_cache) + layer * P.cache_ls + static_cast<int64_t>(h) * P.head_bytes;
  const int64_t row_bytes = static_cast<int64_t>(P.kv_heads) * P.head_bytes;
  const int items = P.head_bytes / 32;
  const int rows = kMoveThreads / items;              // rows one pass of the CTA covers
  const int my_row = threadIdx.x / items, item = threadIdx.x - my_row * items;
  const bool idle = my_row >= rows;
  const bool turns = which == 0 && P.renumber && item < P.rope_items;
  const int c0 = 8 * item;                            // first frequency of a turned item
  int off_a, off_b;
  if (which == 0 && item < P.rope_items) {
    off_a = P.rope_off + (NEOX ? item : 2 * item) * 16;
    off_b = P.rope_off + (NEOX ? item + P.rope_items : 2 * item + 1) * 16;
  } else {  // copied items; MLA rows hold their latent before the rope slice
    const int k = which == 0 ? item - P.rope_items : item;
    off_a = k * 32;
    off_b = off_a + 16;
  }
  const int tile = rows * kMoveBatch;
  uint4 a[2][kMoveBatch], b[2][kMoveBatch];
  int src[2][kMoveBatch];
  auto read = [&](int base, uint4 (&xa)[kMoveBatch], uint4 (&xb)[kMoveBatch], int (&xs)[kMoveBatch]) {
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      const int j = base + i * rows + my_row;
      xs[i] = -1;
      if (idle || j >= u.n_keep) continue;
      xs[i] = kept[j];
      const uint8_t* p = cache + paged_row(P.paged, r, xs[i]) * row_bytes;
      xa[i] = *reinterpret_cast<const uint4*>(p + off_a);
      xb[i] = *reinterpret_cast<const uint4*>(p + off_b);
    }
  };
  auto write = [&](int base, uint4 (&xa)[kMoveBatch], uint4 (&xb)[kMoveBatch], int (&xs)[kMoveBatch]) {
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      if (xs[i] < 0) continue;
      const int j = base + i * rows + my_row;
      if (turns && xs[i] != j) {
        float c[8], s[8];
#pragma unroll
        for (int f = 0; f < 8; ++f) shift_cossin(j - xs[i], P.freq.turns[c0 + f], c[f], s[f]);
        if (NEOX) {
          rotate_neox(xa[i], xb[i], c, s);
        } else {
          rotate_interleaved(xa[i], c, s);
          rotate_interleaved(xb[i], c + 4, s + 4);
        }
      }
      uint8_t* p = cache + paged_row(P.paged, r, j) * row_bytes;
      *reinterpret_cast<uint4*>(p + off_a) = xa[i];
      *reinterpret_cast<uint4*>(p + off_b) = xb[i];
    }
  };
  read(u.first_moved, a[0], b[0], src[0]);
  for (int base = u.first_moved; base < u.n_keep; base += 2 * tile) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int at = base + x * tile;
      if (at >= u.n_keep) break;
      read(at + tile, a[x ^ 1], b[x ^ 1], src[x ^ 1]);
      __syncthreads();   // the tile's rows are in registers everywhere
      write(at, a[x], b[x], src[x]);
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int pairing, int, cudaStream_t s) {
  const int64_t units = static_cast<int64_t>(p.layers) * p.n_req;
  k_evict_select<<<static_cast<unsigned>(units * p.weight_heads), kSelThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int tensors = p.v_cache != nullptr ? 2 : 1;
  const dim3 grid(static_cast<unsigned>(units * p.kv_heads), tensors + 1);
  if (pairing == kNeox) k_evict_move<kNeox><<<grid, kMoveThreads, 0, s>>>(p, tensors);
  else k_evict_move<kInterleaved><<<grid, kMoveThreads, 0, s>>>(p, tensors);
  return cudaGetLastError();
}

}  // namespace pic
