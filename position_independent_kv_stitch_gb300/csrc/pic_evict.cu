// Evicts cached tokens by accumulated attention weight (sm_103a).
//
// Per layer, request and weight head (all KV heads share one, or each has its
// own), a sequence longer than the budget keeps its first n_first tokens, its
// last n_recent, and of the tokens between the heaviest that fit, equal
// weights to the lower slot.  The kept tokens slide down, in order, to slots
// 0 .. budget - 1; with `renumber` a key that moved from slot s to j is turned
// by R(j - s), so that the cache is again a sequence of consecutive positions.
//
// Two launches, the second a programmatic dependent of the first:
//
// k_evict_select, one CTA per (layer, request, weight head).  The weights are
// read once into shared memory (those past its size are read again from L2).
// The weight of the last token that fits is found by radix selection over the
// weights' bits, from the top: 11, 11 and 10 bits, counted in shared memory.
// Then every warp takes a contiguous run of slots, counts what it keeps, and
// after a scan over the warps writes its kept slots and their weights, in
// order and without further barriers.
//
// k_evict_move, one CTA per tile of kept rows (16 KB) of one tensor, in place.
// Rank j lands on slot j, never above its own slot, so a tile may be written
// once every lower tile of its unit has been read, and reading never has to
// wait.  CTAs take tiles by a ticket, lowest tiles of all units first: a tile's
// lower neighbours were taken earlier, by CTAs that are running, and the
// wait for their "read" flags ends whatever the number of resident CTAs (it
// is bounded all the same).  So one sequence is moved by as many CTAs as it
// has tiles.  Kept tokens before the first evicted one are in place already.
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

// Order of the weights as unsigned integers: NaN lowest, -0 equal to 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) != 0 ? ~u : (u | 0x80000000u);
}

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
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ float s_w[];   // weights of slots [0, cap)
  __shared__ int s_hist[kBins];
  __shared__ int s_warp[kSelWarps];
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  __shared__ int s_pick[2];
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

  // the move's flags and ticket start at 0
  for (int64_t i = unit * kSelThreads + tid; i < P.n_flags; i += static_cast<int64_t>(gridDim.x) * kSelThreads) P.flags[i] = 0;

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
  if (tid == 0 && layer == 0 && wh == 0) P.next_lens[r] = bad || len <= P.budget ? len : P.budget;
  if (bad || len <= P.budget) {
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
  const int cap = P.sel_cap;
  auto weight_of = [&](int slot) -> float { return slot < cap ? s_w[slot] : __ldcg(at(slot)); };
  const int lo = P.n_first, hi = len - P.n_recent;     // candidates: slots [lo, hi)
  const int want = P.budget - P.n_first - P.n_recent;  // how many of them stay; fewer than hi - lo
  for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
  if (tid == 0) s_first_moved = P.budget;
#pragma unroll 4
  for (int s = tid; s < min(len, cap); s += kSelThreads) s_w[s] = __ldcg(at(s));
  __syncthreads();

  uint32_t border = 0xffffffffu;  // key of the last candidate that stays
  int ties = 0;                   // candidates of that key that stay
  if (want > 0) {
    uint32_t prefix = 0, mask = 0;
    int left = want;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t digits = pass == 2 ? 1023u : 2047u;
      for (int s = lo + tid; s < hi; s += kSelThreads) {
        const uint32_t k = weight_key(weight_of(s));
        if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & digits], 1);
      }
      __syncthreads();
      // two digits a thread, from the top: the one in which the count reaches `left`
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
      prefix |= static_cast<uint32_t>(s_pick[0]) << shift;
      mask |= digits << shift;
      left = s_pick[1];
    }
    border = prefix;
    ties = left;
  }

  // every warp's run of slots, a multiple of 32
  const int run = (len + kSelThreads - 1) / kSelThreads * 32;
  const int begin = min(len, warp * run), end = min(len, begin + run);
  auto classify = [&](int s, bool& stays, bool& tie) {
    const bool cand = s >= lo && s < hi;
    const uint32_t k = cand && want > 0 ? weight_key(weight_of(s)) : 0u;
    tie = cand && want > 0 && k == border;
    stays = s < end && (!cand || (want > 0 && k > border));
  };
  int gt = 0, eq = 0;
  for (int s0 = begin; s0 < end; s0 += 32) {
    bool stays, tie;
    classify(s0 + lane, stays, tie);
    gt += __popc(__ballot_sync(kFull, stays));
    eq += __popc(__ballot_sync(kFull, tie && s0 + lane < end));
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  int gt_before = lane < warp ? s_gt[lane] : 0, eq_before = lane < warp ? s_eq[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt_before += __shfl_xor_sync(kFull, gt_before, o);
    eq_before += __shfl_xor_sync(kFull, eq_before, o);
  }
  const bool all_cached = len <= cap;
  const unsigned below = (1u << lane) - 1u;
  int first_out = len;   // first evicted slot of this run
  for (int s0 = begin; s0 < end; s0 += 32) {
    const int s = s0 + lane;
    bool stays, tie;
    classify(s, stays, tie);
    tie = tie && s < end;
    const unsigned gts = __ballot_sync(kFull, stays), eqs = __ballot_sync(kFull, tie);
    const int eq_mine = eq_before + __popc(eqs & below);
    const bool keep = stays || (tie && eq_mine < ties);
    const int rank = gt_before + __popc(gts & below) + min(eq_mine, ties);
    if (keep) {
      kept[rank] = s;
      if (all_cached && rank != s) *at(rank) = s_w[s];
    }
    const unsigned out = __ballot_sync(kFull, !keep && s < end);
    if (out != 0 && first_out == len) first_out = s0 + __ffs(out) - 1;
    gt_before += __popc(gts);
    eq_before += __popc(eqs);
  }
  if (lane == 0 && first_out < len) atomicMin(&s_first_moved, first_out);
  __syncthreads();
  if (tid == 0) P.units[unit] = EvictUnit{P.budget, s_first_moved};
  if (all_cached) return;
  // some weights are only in memory: move them in order, a tile's reads before its writes
  for (int base = s_first_moved; base < P.budget; base += kSelThreads) {
    const int j = base + tid;
    float x = 0.0f;
    if (j < P.budget) x = weight_of(kept[j]);
    // the barrier takes a value made of the loaded one: every load has arrived
    __syncthreads_or(__float_as_uint(x) == 0x7fc12345u);
    if (j < P.budget) *at(j) = x;
  }
}

constexpr int kMoveThreads = 128;
constexpr int kMoveBatch = kEvictTileItems / kMoveThreads;  // items in flight per thread
constexpr uint32_t kMaxPolls = 1u << 20;

// cos / sin of a whole-position shift: the exact reduction of shift_cossin,
// then the hardware's sine and cosine, whose absolute error on [-pi, pi] is
// below 2^-21: far inside the rounding to bf16 that follows, at a fifth of the
// instructions (a moved key has a shift of its own, so nothing is shared).
__device__ __forceinline__ void shift_cossin_fast(float d, float2 f, float& c, float& s) {
  const float p = __fmul_rn(d, f.x);
  const float e = __fmaf_rn(d, f.x, -p);
  const float r = __fsub_rn(p, rintf(p));
  const float t = 6.283185307179586f * __fadd_rn(r, __fmaf_rn(d, f.y, e));
  c = __cosf(t);
  s = __sinf(t);
}

template <int PAIRING>
__global__ void __launch_bounds__(kMoveThreads, 8) k_evict_move(const __grid_constant__ EvictParams P) {
  constexpr bool NEOX = PAIRING == kNeox;
  __shared__ int64_t s_ticket;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) s_ticket = static_cast<int64_t>(atomicAdd(P.flags, 1u));
  __syncthreads();
  // ticket = tile * units + unit; unit = ((layer, request), tensor, piece)
  const int64_t units = static_cast<int64_t>(P.layers) * P.n_req * P.tensors * P.pieces;
  const int64_t unit = s_ticket % units;
  const int tile = static_cast<int>(s_ticket / units);
  const int piece = static_cast<int>(unit % P.pieces);
  const int tensor = static_cast<int>(unit / P.pieces % P.tensors);
  const int64_t lr = unit / P.pieces / P.tensors;
  const int r = static_cast<int>(lr % P.n_req);
  const int64_t layer = lr / P.n_req;
  if (tile == 0 && layer == 0 && tensor == 0 && piece == 0 && threadIdx.x == 0) P.new_lens[r] = P.next_lens[r];
  const int64_t wu = lr * P.weight_heads + (P.weight_heads == 1 ? 0 : piece);
  const EvictUnit u = P.units[wu];
  const int base = u.first_moved + tile * P.tile_rows;   // first rank of the tile
  if (base >= u.n_keep) return;
  const int32_t* kept = P.kept + wu * P.budget;
  uint32_t* flags = P.flags + 1 + unit * P.tiles;

  const int h0 = piece * P.piece_heads;
  const int items = min(P.piece_heads, P.kv_heads - h0) * P.head_items;   // 32-byte items of a row
  uint8_t* cache = (tensor == 0 ? P.k_cache : P.v_cache) + layer * P.cache_ls + static_cast<int64_t>(h0) * P.head_bytes;
  const int64_t row_bytes = static_cast<int64_t>(P.kv_heads) * P.head_bytes;
  const int rows = min(P.tile_rows, u.n_keep - base);

  // An item is two 16-byte chunks; a key item of the rope slice holds both
  // members of its 8 pairs.  off_a / off_b: its place in the piece's row.
  auto chunks = [&](int item, int& off_a, int& off_b, int& freq) {
    const int h = item / P.head_items, i = item - h * P.head_items;
    const int ho = h * P.head_bytes;
    freq = -1;
    if (tensor == 0 && i < P.rope_items) {
      off_a = ho + P.rope_off + (NEOX ? i : 2 * i) * 16;
      off_b = ho + P.rope_off + (NEOX ? i + P.rope_items : 2 * i + 1) * 16;
      freq = 8 * i;
    } else {   // copied; MLA rows hold their latent before the rope slice
      off_a = ho + (tensor == 0 ? i - P.rope_items : i) * 32;
      off_b = off_a + 16;
    }
  };
  uint4 a[kMoveBatch], b[kMoveBatch];
  int src[kMoveBatch];
  uint32_t seen = 0;
#pragma unroll
  for (int x = 0; x < kMoveBatch; ++x) {
    const int e = x * kMoveThreads + threadIdx.x, row = e / items;
    src[x] = row < rows ? __ldcg(kept + base + row) : -1;
  }
#pragma unroll
  for (int x = 0; x < kMoveBatch; ++x) {
    if (src[x] < 0) continue;
    const int e = x * kMoveThreads + threadIdx.x;
    int off_a, off_b, freq;
    chunks(e % items, off_a, off_b, freq);
    const uint8_t* p = cache + paged_row(P.paged, r, src[x]) * row_bytes;
    a[x] = __ldcg(reinterpret_cast<const uint4*>(p + off_a));
    b[x] = __ldcg(reinterpret_cast<const uint4*>(p + off_b));
  }
#pragma unroll
  for (int x = 0; x < kMoveBatch; ++x)
    if (src[x] >= 0) seen ^= a[x].x ^ b[x].x;
  // the barrier takes a value made of the loaded ones: every load of the CTA has arrived
  __syncthreads_or(seen == 0x7fc12345u);
  if (threadIdx.x == 0)
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(flags + tile), "r"(1u) : "memory");
  // every lower tile of the unit has been read
  bool timeout = false;
  for (int t = threadIdx.x; t < tile; t += kMoveThreads) {
    uint32_t done = 0;
    for (uint32_t n = 0; n < kMaxPolls && done == 0; ++n)
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(done) : "l"(flags + t) : "memory");
    timeout |= done == 0;
  }
  if (__syncthreads_or(timeout)) {
    if (threadIdx.x == 0) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_TIMEOUT));
    return;
  }
#pragma unroll
  for (int x = 0; x < kMoveBatch; ++x) {
    if (src[x] < 0) continue;
    const int e = x * kMoveThreads + threadIdx.x;
    const int j = base + e / items;
    int off_a, off_b, freq;
    chunks(e % items, off_a, off_b, freq);
    if (P.renumber && freq >= 0 && src[x] != j) {
      float c[8], s[8];
#pragma unroll
      for (int f = 0; f < 8; ++f) shift_cossin_fast(static_cast<float>(j - src[x]), P.freq.turns[freq + f], c[f], s[f]);
      if (NEOX) {
        rotate_neox(a[x], b[x], c, s);
      } else {
        rotate_interleaved(a[x], c, s);
        rotate_interleaved(b[x], c + 4, s + 4);
      }
    }
    uint8_t* p = cache + paged_row(P.paged, r, j) * row_bytes;
    *reinterpret_cast<uint4*>(p + off_a) = a[x];
    *reinterpret_cast<uint4*>(p + off_b) = b[x];
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int pairing, cudaStream_t s) {
  const int64_t lr = static_cast<int64_t>(p.layers) * p.n_req;
  const int smem = p.sel_cap * static_cast<int>(sizeof(float));
  cudaError_t e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k_evict_select<<<static_cast<unsigned>(lr * p.weight_heads), kSelThreads, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(lr * p.tensors * p.pieces * p.tiles));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return pairing == kNeox ? cudaLaunchKernelEx(&cfg, k_evict_move<kNeox>, p)
                          : cudaLaunchKernelEx(&cfg, k_evict_move<kInterleaved>, p);
}

}  // namespace pic
