// Evicts cached tokens by accumulated attention weight (sm_103a).
//
// Per layer, request and weight head (all KV heads share one, or each has its
// own), a sequence longer than the budget keeps its first n_first tokens, its
// last n_recent, and of the tokens between the heaviest that fit, equal
// weights to the lower slot.  The kept tokens slide down, in order, to slots
// 0 .. budget - 1; with `renumber` a key that moved from slot s to j is turned
// by R(j - s), so that the cache is again a sequence of consecutive positions.
//
// Two launches.  (The second is no programmatic dependent of the first: its CTAs
// live long, and those placed early would crowd the few SMs the first leaves
// free.)
//
// k_evict_select, one CTA per (layer, request, weight head).  The weights are
// read once and kept in shared memory as sort keys (those past its size are read
// again from L2); only -0 and NaNs do not come back from their keys.
// The weight of the last token that fits is found by radix selection over the
// weights' bits, from the top: 11, 11 and 10 bits, counted in shared memory.
// Every warp takes a contiguous run of slots; a sweep counts what surely stays in
// each and lists the members of the border's top digit, and the lower digits
// are looked for in that list (in all weights, should it overflow).  After a
// scan over the warps a last sweep writes the kept slots, in order and without
// further barriers; the weights follow from shared memory.
//
// k_evict_move, in place: one CTA per slice (32 bytes to whole rows) of the
// kept rows of one tensor, which it walks in order.  Rank j lands on slot j,
// never above its own slot, so rows may be read any time before, and a tile may
// be written once the CTA has read it: the next tile's rows and the list of the
// one after are on their way while a tile is written, with one barrier each.
// Slices share no byte, so CTAs never wait for one another; how finely rows
// are sliced is chosen so that the slices fill the GPU.  (Tiles of whole rows
// dealt to all CTAs by tickets, each waiting for the lower tiles to be read,
// moved 3.4-4.7 TB/s: a chain of five round trips to memory per tile.)  Kept
// tokens before the first evicted one are in place already.
//
// Measured on fresh weights (GB300): 32k -> 4k tokens in 16 layers of 8 heads, each
// head its own set, keys turned, 136 us (selection 28; 559 MB, 4.1 TB/s); 12 of
// 16 sequences cut to 2k in 8 layers, heads together, 240 us (1.61 GB, 6.7 TB/s);
// MLA, 16k -> 8k, 3 sequences, 16 layers 209 us (910 MB, 4.4 TB/s); 2,064 -> 2,048
// in one layer 11.2 us.
#include "pic_decode.h"
#include "pic_device.cuh"
#include "pic_paged.cuh"

namespace pic {
namespace {

using namespace dev;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kSelList = 2048;

// Order of the weights as unsigned integers: NaN lowest, -0 equal to 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) != 0 ? ~u : (u | 0x80000000u);
}
// The weight of a key, for all but those of lossy().
__device__ __forceinline__ float key_weight(uint32_t k) {
  return __uint_as_float(k == 0u ? 0x7fffffffu : ((k & 0x80000000u) != 0 ? k ^ 0x80000000u : ~k));
}
// Whether a weight cannot be had back from its key: -0, which counts as 0, and NaN.
__device__ __forceinline__ bool lossy(float w) { return w != w || __float_as_uint(w) == 0x80000000u; }
// Bits i of 4 with i < n.
__device__ __forceinline__ uint32_t below(int n) { return 0xfu >> (4 - min(max(n, 0), 4)); }

// Sum of v over the CTA's threads before this one.
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
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
  int s = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += up;
  }
  const int before = __shfl_sync(kFull, s, warp) - warp_sums[warp];
  return before + incl - v;
}

__global__ void __launch_bounds__(kSelThreads) k_evict_select(const __grid_constant__ EvictParams P) {
  extern __shared__ __align__(16) uint32_t s_key[];   // keys of the first slots' weights
  __shared__ int s_hist[kBins];
  __shared__ int s_warp[kSelWarps];
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  __shared__ int s_pick[2];
  __shared__ uint2 s_list[kSelList];   // keys of the border's top digit, and the warps whose runs they lie in
  __shared__ int s_listed;
  __shared__ int s_first_moved;
  static_assert(kSelWarps == 32, "one lane per warp in the scans");
  const int64_t unit = blockIdx.x;
  const int wh = static_cast<int>(unit % P.weight_heads);
  const int r = static_cast<int>(unit / P.weight_heads % P.n_req);
  const int64_t layer = unit / P.weight_heads / P.n_req;
  int32_t* kept = P.kept + unit * P.budget;
  const int len = __ldg(P.lens + r);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = P.paged.block_size;

  // a request whose length or blocks are not legal keeps all it has
  bool bad = len < 0 || len > P.max_len;
  if (bad) {
    if (tid == 0) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_BAD_LENGTH));
  } else {
    const int blocks = (len + bs - 1) / bs;
    bool mine = false;
    for (int b = tid; b < blocks; b += kSelThreads) {
      const int32_t block = __ldg(P.paged.tables + static_cast<int64_t>(r) * P.paged.max_blocks + b);
      if (block < 0 || block >= P.paged.num_cache_blocks) {
        mine = true;
        raise_block(P.status, r, b * bs);
      }
    }
    bad = __syncthreads_or(mine);
  }
  const bool cut = !bad && len > P.budget;
  if (tid == 0 && layer == 0 && wh == 0) P.next_lens[r] = cut ? P.budget : len;
  if (!cut) {
    for (int j = tid; j < P.budget; j += kSelThreads) kept[j] = !bad && j < len ? j : -1;
    if (tid == 0) P.units[unit] = EvictUnit{0, 0};
    return;
  }

  float* wl = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(P.weights) + layer * P.weights_ls);
  auto at = [&](int slot) -> float* {
    const int b = block_of(P.paged, slot);
    const int64_t block = __ldg(P.paged.tables + static_cast<int64_t>(r) * P.paged.max_blocks + b);
    return wl + (block * P.weight_heads + wh) * bs + (slot - b * bs);
  };
  const int cached = min(len, P.sel_cap);   // slots whose keys are in shared memory
  // the keys of slots s .. s + 3 (0 past the end; s a multiple of 4)
  auto load4 = [&](int s, uint32_t (&k)[4]) {
    if (s + 4 <= cached) {
      const uint4 x = *reinterpret_cast<const uint4*>(s_key + s);
      k[0] = x.x, k[1] = x.y, k[2] = x.z, k[3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = s + i >= len ? 0u : (s + i < cached ? s_key[s + i] : weight_key(__ldcg(at(s + i))));
    }
  };
  const int lo = P.n_first, hi = len - P.n_recent;     // candidates: slots [lo, hi)
  const int want = P.budget - P.n_first - P.n_recent;  // how many of them stay; fewer than hi - lo
  for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
  if (tid == 0) s_first_moved = P.budget;
  if (tid == 0) s_listed = 0;
  __syncthreads();
  // The weights come in, and the top digits of the candidates' keys are counted.
  // Four neighbouring slots lie together when blocks hold a multiple of four.
  const bool vec = (bs & 3) == 0 && ((reinterpret_cast<uintptr_t>(P.weights) | static_cast<uintptr_t>(P.weights_ls)) & 15) == 0;
  auto count_top = [&](uint32_t key) { atomicAdd(&s_hist[key >> 21], 1); };
  auto is_cand = [&](int s) { return s >= lo && s < hi; };
  bool lost = false;   // a weight that has to be moved from memory
  if (vec) {
#pragma unroll 4
    for (int s = 4 * tid; s < cached; s += 4 * kSelThreads) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(at(s)));
      const uint4 k = make_uint4(weight_key(x.x), weight_key(x.y), weight_key(x.z), weight_key(x.w));
      *reinterpret_cast<uint4*>(s_key + s) = k;
      lost |= lossy(x.x) || lossy(x.y) || lossy(x.z) || lossy(x.w);
      const uint32_t cand = below(hi - s) & ~below(lo - s);
      if (cand & 1u) count_top(k.x);
      if (cand & 2u) count_top(k.y);
      if (cand & 4u) count_top(k.z);
      if (cand & 8u) count_top(k.w);
    }
  } else {
#pragma unroll 4
    for (int s = tid; s < cached; s += kSelThreads) {
      const float w = __ldcg(at(s));
      const uint32_t k = weight_key(w);
      s_key[s] = k;
      lost |= lossy(w);
      if (is_cand(s)) count_top(k);
    }
  }
  for (int s = cached + tid; s < len; s += kSelThreads)
    if (is_cand(s)) count_top(weight_key(__ldcg(at(s))));
  const bool from_keys = __syncthreads_or(lost) == 0;

  // The digit in which the count from the top reaches `left`, two digits a
  // thread; what is left within it.  The counts return to 0.
  auto pick = [&](int& left) -> uint32_t {
    const int d = kBins - 1 - 2 * tid;
    const int n0 = s_hist[d], n1 = s_hist[d - 1];
    const int above = block_scan(n0 + n1, s_warp);
    if (above < left && above + n0 + n1 >= left) {
      const bool first = above + n0 >= left;
      s_pick[0] = first ? d : d - 1;
      s_pick[1] = left - above - (first ? 0 : n0);
    }
    s_hist[d] = s_hist[d - 1] = 0;
    __syncthreads();
    left = s_pick[1];
    return static_cast<uint32_t>(s_pick[0]);
  };
  // Every warp's run of slots, 128 a step, four neighbours a lane.  Per lane:
  // bits of the slots that stay whatever happens (their key is above `top`, or
  // they are no candidates), and of those whose key lies in [base, top].
  const int run = (len + kSelThreads * 4 - 1) / (kSelThreads * 4) * 128;
  const int begin = min(len, warp * run), end = min(len, begin + run);
  auto classify = [&](int s, uint32_t base, uint32_t top, uint32_t& stays, uint32_t& tie, uint32_t (&key)[4]) {
    load4(s, key);
    uint32_t ge = 0, gt = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ge |= key[i] >= base ? 1u << i : 0u;
      gt |= key[i] > top ? 1u << i : 0u;
    }
    const uint32_t in = below(end - s), cand = below(hi - s) & ~below(lo - s);
    stays = in & (gt | ~cand);
    tie = in & cand & ge & ~gt;
  };
  // Counts this warp's run against a border, the keys [base, top]; lists its members when asked to.
  auto count_run = [&](uint32_t base, uint32_t top, bool list) {
    int mine = 0, mine_ties = 0;
    for (int s0 = begin; s0 < end; s0 += 128) {
      uint32_t stays, tie, key[4];
      classify(s0 + 4 * lane, base, top, stays, tie, key);
      mine += __popc(stays);
      mine_ties += __popc(tie);
      if (list && tie != 0) {   // few: in no order
        int at_list = atomicAdd(&s_listed, __popc(tie));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((tie >> i) & 1u) {
            if (at_list < kSelList) s_list[at_list] = make_uint2(key[i], warp);
            ++at_list;
          }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mine += __shfl_xor_sync(kFull, mine, o);
      mine_ties += __shfl_xor_sync(kFull, mine_ties, o);
    }
    if (lane == 0) {
      s_gt[warp] = mine;
      s_eq[warp] = mine_ties;
    }
    __syncthreads();
  };

  uint32_t border = 0xffffffffu;  // key of the last candidate that stays
  int ties = 0;                   // candidates of that key that stay
  if (want == 0) {
    count_run(border, border, false);   // no key is that high
  } else {
    int left = want;
    border = pick(left);
    count_run(border << 21, border << 21 | 0x1fffffu, true);
    const bool listed = s_listed <= kSelList;
    // the two lower digits: over the list, or over everything when too many share the top digit
#pragma unroll
    for (int pass = 1; pass < 3; ++pass) {
      const int shift = pass == 1 ? 10 : 0, bits = pass == 1 ? 11 : 10;
      const uint32_t digits = (1u << bits) - 1u;
      if (listed) {
        for (int i = tid; i < s_listed; i += kSelThreads) {
          const uint32_t k = s_list[i].x;
          if ((k >> (shift + bits)) == border) atomicAdd(&s_hist[(k >> shift) & digits], 1);
        }
      } else {
#pragma unroll 2
        for (int s = 4 * tid; s < hi; s += 4 * kSelThreads) {
          uint32_t k[4];
          load4(s, k);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (is_cand(s + i) && (k[i] >> (shift + bits)) == border) atomicAdd(&s_hist[(k[i] >> shift) & digits], 1);
        }
      }
      __syncthreads();
      const uint32_t digit = pick(left);
      border = border << bits | digit;
    }
    ties = left;
    if (listed) {   // the counts of the runs, from the list's members
      if (lane == 0) s_eq[warp] = 0;
      __syncthreads();
      for (int i = tid; i < s_listed; i += kSelThreads) {
        const uint2 x = s_list[i];
        if (x.x > border) atomicAdd(&s_gt[x.y], 1);
        else if (x.x == border) atomicAdd(&s_eq[x.y], 1);
      }
      __syncthreads();
    } else {
      count_run(border, border, false);
    }
  }
  int gt_before = lane < warp ? s_gt[lane] : 0, eq_before = lane < warp ? s_eq[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt_before += __shfl_xor_sync(kFull, gt_before, o);
    eq_before += __shfl_xor_sync(kFull, eq_before, o);
  }
  int first_out = len;   // first evicted slot of this lane's
  for (int s0 = begin; s0 < end; s0 += 128) {
    const int s = s0 + 4 * lane;
    uint32_t stays, tie, key[4];
    classify(s, border, border, stays, tie, key);
    const int n = __popc(stays) | __popc(tie) << 16;   // 128 of each at most
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    int gt = gt_before + ((incl - n) & 0xffff), eq = eq_before + ((incl - n) >> 16);
    uint32_t out = below(end - s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool is_tie = (tie >> i) & 1u, keep = ((stays >> i) & 1u) || (is_tie && eq < ties);
      if (keep) {
        kept[gt + min(eq, ties)] = s + i;
        out ^= 1u << i;
      }
      gt += (stays >> i) & 1u;
      eq += is_tie ? 1 : 0;
    }
    if (out != 0) first_out = min(first_out, s + __ffs(out) - 1);
    const int all = __shfl_sync(kFull, incl, 31);
    gt_before += all & 0xffff;
    eq_before += all >> 16;
  }
  if (first_out < len) atomicMin(&s_first_moved, first_out);
  __syncthreads();
  if (tid == 0) P.units[unit] = EvictUnit{P.budget, s_first_moved};
  // the weights move with their tokens (kept[] is this CTA's own, written above)
  if (cached == len && from_keys) {
    for (int j = s_first_moved + tid; j < P.budget; j += kSelThreads) *at(j) = key_weight(s_key[kept[j]]);
    return;
  }
  // some are only in memory as they were: in order, a tile's reads before its writes
  for (int base = s_first_moved; base < P.budget; base += kSelThreads) {
    const int j = base + tid;
    float x = 0.0f;
    if (j < P.budget) {
      const int s = kept[j];
      x = s < cached && from_keys ? key_weight(s_key[s]) : __ldcg(at(s));
    }
    // the barrier takes a value made of the loaded one: every load has arrived
    __syncthreads_or(__float_as_uint(x) == 0x7fc12345u);
    if (j < P.budget) *at(j) = x;
  }
}

constexpr int kMoveThreads = kEvictMoveThreads;
constexpr int kMoveCtas = kEvictMoveCtas;
constexpr int kMoveBatch = 1;    // items per thread and tile
constexpr int kMoveStages = 3;   // tiles in shared memory, most of them on their way
// Threads x CTAs per SM x stages, on the three large cases above (us; with the
// hardware's sine and cosine, which are less exact than turn_cossin2's): 384 x 4 x 3
// 126 / 241 / 197; 256 x 4 x 5 130 / 259 / 206, 256 x 5 x 4 130 / 243 / 204, 320 x 4 x 4
// 126 / 249 / 197, 384 x 4 x 4 131 / 244 / 204, 512 x 3 x 3 148 / 242 / 241.  Three tiles of
// 12 KB each of four CTAs cover the latency; the slices follow from the threads.
constexpr int kMoveSmem = kMoveStages * kMoveBatch * kMoveThreads * (2 * 16 + 4);

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int PAIRING, bool TURN>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) k_evict_move(const __grid_constant__ EvictParams P) {
  constexpr bool NEOX = PAIRING == kNeox;
  // stream = ((layer, request), tensor, piece of the heads, slice of the piece)
  const int64_t stream = blockIdx.x;
  const int slice = static_cast<int>(stream % P.slices);
  const int piece = static_cast<int>(stream / P.slices % P.pieces);
  const int tensor = static_cast<int>(stream / P.slices / P.pieces % P.tensors);
  const int64_t lr = stream / P.slices / P.pieces / P.tensors;
  const int r = static_cast<int>(lr % P.n_req);
  const int64_t layer = lr / P.n_req;
  const int tid = threadIdx.x;
  if (layer == 0 && tensor == 0 && piece == 0 && slice == 0 && tid == 0) P.new_lens[r] = P.next_lens[r];
  const int64_t wu = lr * P.weight_heads + (P.weight_heads == 1 ? 0 : piece);
  const EvictUnit u = P.units[wu];
  if (u.first_moved >= u.n_keep) return;
  const int32_t* kept = P.kept + wu * P.budget;

  // A row's slice is cut into items of two 16-byte chunks, one per thread, that
  // lie half a head apart (in the latent of an MLA row: half a latent), so that
  // neighbouring threads cover whole sectors and a neox item holds both
  // members of its 8 pairs.
  const int per_pass = kMoveThreads / P.slice_items;   // rows one pass of the CTA covers
  const int my_row = tid / P.slice_items;
  const bool idle = my_row >= per_pass;
  const int item = slice * P.slice_items + tid - my_row * P.slice_items;   // within the piece
  const int h = item / P.head_items, in_head = item - h * P.head_items;
  const bool rope = tensor == 0 && in_head < P.rope_items;
  const int run = tensor != 0 || rope ? P.rope_items : P.head_items - P.rope_items;   // items (GQA: the head's) between the two chunks
  const int off_a = h * P.head_bytes + (rope ? P.rope_off + in_head * 16 : (tensor == 0 ? in_head - P.rope_items : in_head) * 16);
  const int off_b = off_a + run * 16;
  uint8_t* cache = (tensor == 0 ? P.k_cache : P.v_cache) + layer * P.cache_ls +
                   static_cast<int64_t>(piece) * P.piece_heads * P.head_bytes;
  const int64_t row_bytes = static_cast<int64_t>(P.kv_heads) * P.head_bytes;
  // Rows on their way wait in shared memory, each thread's items in places of
  // its own: what a thread reads back it copied in itself, and the barrier
  // only orders the CTA's reads of a tile before its writes.
  extern __shared__ __align__(16) uint4 s_ring[];   // [stage][item][2][thread], then the slots [stage][item][thread]
  int* s_slot = reinterpret_cast<int*>(s_ring + kMoveStages * kMoveBatch * 2 * kMoveThreads);
  __shared__ float4 s_freq[TURN ? kMaxFreqs / 2 : 1];
  if (TURN) {
    if (tid < kMaxFreqs) put_freq(s_freq, tid, P.freq.turns[tid]);
    __syncthreads();
  }
  auto place = [&](int stage, int i) { return stage * kMoveBatch + i; };
  auto load_slots = [&](int base, int (&slot)[kMoveBatch]) {
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      const int j = base + i * per_pass + my_row;
      slot[i] = !idle && j < u.n_keep ? __ldcg(kept + j) : -1;
    }
  };
  // A slot's block (the selection has checked the table).  Kept raw until its
  // row is needed: arithmetic on a load that has not arrived stops the warp.
  const int32_t* table = P.paged.tables + static_cast<int64_t>(r) * P.paged.max_blocks;
  const int bs = P.paged.block_size;
  auto load_blocks = [&](const int (&slot)[kMoveBatch], int (&block)[kMoveBatch]) {
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) block[i] = slot[i] >= 0 ? __ldg(table + block_of(P.paged, slot[i])) : 0;
  };
  auto load_dst_blocks = [&](int base, int (&block)[kMoveBatch]) {
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      const int j = base + i * per_pass + my_row;
      block[i] = j < u.n_keep ? __ldg(table + block_of(P.paged, j)) : 0;
    }
  };
  auto row_at = [&](int block, int slot) -> uint8_t* {
    return cache + (static_cast<int64_t>(block) * bs + (slot - block_of(P.paged, slot) * bs)) * row_bytes;
  };
  auto fetch = [&](int stage, const int (&slot)[kMoveBatch], const int (&block)[kMoveBatch]) {
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      if (slot[i] >= 0) {
        const uint8_t* p = row_at(block[i], slot[i]);
        cp_async16(s_ring + place(stage, i) * 2 * kMoveThreads + tid, p + off_a);
        cp_async16(s_ring + (place(stage, i) * 2 + 1) * kMoveThreads + tid, p + off_b);
      }
      s_slot[place(stage, i) * kMoveThreads + tid] = slot[i];
    }
    cp_commit();
  };
  // The kept list runs two tiles ahead of the fetches, the table lookups of
  // source and destination one ahead of their use.
  const int tile = per_pass * kMoveBatch;
  int slots[2][kMoveBatch], from[2][kMoveBatch], to[2][kMoveBatch];
  {
    int s[kMoveStages - 1][kMoveBatch], f[kMoveStages - 1][kMoveBatch];
#pragma unroll
    for (int k = 0; k < kMoveStages - 1; ++k) load_slots(u.first_moved + k * tile, s[k]);
    load_slots(u.first_moved + (kMoveStages - 1) * tile, slots[0]);
    load_slots(u.first_moved + kMoveStages * tile, slots[1]);
    load_dst_blocks(u.first_moved, to[0]);
#pragma unroll
    for (int k = 0; k < kMoveStages - 1; ++k) load_blocks(s[k], f[k]);
    load_blocks(slots[0], from[0]);
#pragma unroll
    for (int k = 0; k < kMoveStages - 1; ++k) fetch(k, s[k], f[k]);
  }
  int stage = 0;
  for (int base0 = u.first_moved; base0 < u.n_keep; base0 += 2 * tile) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int base = base0 + x * tile;
      if (base >= u.n_keep) break;
      fetch(stage == 0 ? kMoveStages - 1 : stage - 1, slots[x], from[x]);
      load_slots(base + (kMoveStages + 1) * tile, slots[x]);
      load_blocks(slots[x ^ 1], from[x ^ 1]);
      load_dst_blocks(base + tile, to[x ^ 1]);
      cp_wait<kMoveStages - 1>();
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMoveBatch; ++i) {
        const int slot = s_slot[place(stage, i) * kMoveThreads + tid];
        if (slot < 0) continue;
        const int j = base + i * per_pass + my_row;
        uint4 a = s_ring[place(stage, i) * 2 * kMoveThreads + tid], b = s_ring[(place(stage, i) * 2 + 1) * kMoveThreads + tid];
        if (TURN && rope && slot != j) {
          const float2 shift = make_float2(static_cast<float>(j - slot), static_cast<float>(j - slot));
          // Pairs of frequencies.  All first and then the rotation for neox, word by
          // word for interleaved: 136 us (evict_prompt) and 209 (evict_latent); the
          // other way about 149 and 219.
          if (NEOX) {
            float c[8], s[8];
#pragma unroll
            for (int f = 0; f < 4; ++f) turn_cossin2(shift, s_freq[4 * in_head + f], c + 2 * f, s + 2 * f);
            rotate_neox(a, b, c, s);
          } else {   // 2 i .. of the first chunk, 2 (i + run) .. of the second
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              float c[2], s[2];
              turn_cossin2(shift, s_freq[2 * (in_head + (f < 2 ? 0 : run)) + (f & 1)], c, s);
              uint4& v = f < 2 ? a : b;
              rotate_interleaved_word(word(v, 2 * (f & 1)), c[0], s[0]);
              rotate_interleaved_word(word(v, 2 * (f & 1) + 1), c[1], s[1]);
            }
          }
        }
        uint8_t* p = row_at(to[x][i], j);
        *reinterpret_cast<uint4*>(p + off_a) = a;
        *reinterpret_cast<uint4*>(p + off_b) = b;
      }
      stage = stage + 1 == kMoveStages ? 0 : stage + 1;
    }
  }
  cp_wait<0>();
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int pairing, cudaStream_t s) {
  const int64_t lr = static_cast<int64_t>(p.layers) * p.n_req;
  const int smem = p.sel_cap * static_cast<int>(sizeof(float));
  static std::atomic<uint32_t> select_done{0}, move_done[3] = {{0}, {0}, {0}};
  cudaError_t e = allow_smem(k_evict_select, kEvictCachedSlots * static_cast<int>(sizeof(float)), select_done);
  if (e != cudaSuccess) return e;
  k_evict_select<<<static_cast<unsigned>(lr * p.weight_heads), kSelThreads, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int variant = p.renumber == 0 ? 0 : (pairing == kNeox ? 1 : 2);
  auto move = variant == 0 ? k_evict_move<kNeox, false> : (variant == 1 ? k_evict_move<kNeox, true> : k_evict_move<kInterleaved, true>);
  e = allow_smem(move, kMoveSmem, move_done[variant]);
  if (e != cudaSuccess) return e;
  move<<<static_cast<unsigned>(lr * p.tensors * p.pieces * p.slices), kMoveThreads, kMoveSmem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace pic
