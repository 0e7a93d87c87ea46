// Block tables and token lists from request lengths (sm_103a): the step of a
// serving loop that gives every new token its place in the paged cache.
//
// With have = ceil(len / block_size) and want = ceil((len + grow) / block_size):
// requests that shrink put blocks [want, have) of their table on the pile of free
// blocks, in order; then those that grow take theirs from its top, in order,
// while it lasts.  Token i of request r gets slot len + i.
//
// Everything follows from prefix sums over the requests.  A CTA of 1,024 threads sums
// them itself, 1,024 at a time, and lists its own part of the tokens; blocks and
// tokens are dealt to threads one by one, each finding its request by halving
// (a thread per request, walking its blocks, took 85 us where requests of 1,000 slots end).
// Where there are many tokens, the first CTA moves the blocks and the others list them;
// the new lengths, when they are the inputs' own memory, are written by the CTA whose
// ticket is the last, when all have read.
// Bound: for a decode step the launch and a chain of dependent reads (counts, sums,
// table, pile); for prompts the stores of 12 bytes a token.
// Measured (GB300): a decode step of 64 requests 6.3 us; 256 prompts of 128k token rows 12.0 us.
#include "pic_decode.h"
#include "pic_paged.cuh"

namespace pic {
namespace {

using namespace dev;

constexpr int kMapThreads = 1024, kMapWarps = kMapThreads / 32;
constexpr int kMapTokensPerCta = 2048;   // more CTAs beyond this
constexpr unsigned kFull = 0xffffffffu;

// What a request adds to the sums: blocks it gives back, token rows, blocks it needs.
struct Counts {
  int64_t back, rows, need;
};
__device__ __forceinline__ Counts operator+(const Counts& a, const Counts& b) {
  return Counts{a.back + b.back, a.rows + b.rows, a.need + b.need};
}
__device__ __forceinline__ Counts shfl_up(const Counts& v, int o) {
  return Counts{__shfl_up_sync(kFull, v.back, o), __shfl_up_sync(kFull, v.rows, o), __shfl_up_sync(kFull, v.need, o)};
}
__device__ __forceinline__ Counts shfl(const Counts& v, int lane) {
  return Counts{__shfl_sync(kFull, v.back, lane), __shfl_sync(kFull, v.rows, lane), __shfl_sync(kFull, v.need, lane)};
}
__device__ __forceinline__ Counts warp_scan(Counts v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Counts up = shfl_up(v, o);
    if (lane >= o) v = v + up;
  }
  return v;
}

struct MapShared {
  Counts warp[kMapWarps];
  int64_t best[kMapWarps];
  // a sweep's lists: the first element of each request, and one past the last request's
  int64_t back[kMapThreads + 1], rows[kMapThreads + 1], need[kMapThreads + 1];
  int from[kMapThreads];            // column of the first block that goes; -1: none does
  int to[kMapThreads];              // column of the first block that comes; -1: none does
  int len[kMapThreads];             // length; -1: gets no slots
  int shift[kMapThreads];
  uint32_t ticket;
};

// Inclusive sums over the CTA; `total` of all.
__device__ __forceinline__ Counts block_scan(Counts v, MapShared& S, Counts& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_scan(v, lane);
  __syncthreads();   // S.warp is free
  if (lane == 31) S.warp[warp] = v;
  __syncthreads();
  const Counts w = warp_scan(S.warp[lane], lane);
  if (warp > 0) v = v + shfl(w, warp - 1);
  total = shfl(w, 31);
  return v;
}
__device__ __forceinline__ int64_t block_max(int64_t v, MapShared& S) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) S.best[threadIdx.x >> 5] = v;
  __syncthreads();
  v = S.best[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
// The request (of the sweep's n) that element e belongs to: first[x] <= e < first[x + 1].
__device__ __forceinline__ int owner(const int64_t* first, int n, int64_t e) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= e) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct Request {
  int64_t len, grow;
  int have, want;
  bool legal;
  __device__ __forceinline__ Counts counts() const {
    return Counts{legal && grow < 0 ? have - want : 0, grow > 0 ? grow : 0, legal && grow > 0 ? want - have : 0};
  }
};
__device__ __forceinline__ Request read_request(const MapParams& P, int r, bool raise) {
  Request q{0, 0, 0, 0, true};
  if (r >= P.n_req) return q;
  q.len = __ldcg(P.lens + r);
  q.grow = __ldcg(P.grow + r);
  const int64_t to = q.len + q.grow;
  q.legal = q.len >= 0 && q.len <= P.max_len && to >= 0 && to <= P.max_len;
  if (!q.legal) {
    if (raise) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_BAD_LENGTH));
    return q;
  }
  // (below 2^32: no 64-bit division)
  const uint32_t bs = static_cast<uint32_t>(P.block_size);
  q.have = static_cast<int>((static_cast<uint32_t>(q.len) + bs - 1) / bs);
  q.want = static_cast<int>((static_cast<uint32_t>(to) + bs - 1) / bs);
  return q;
}

// Blocks of a sweep's requests (from r0 on, n of them) that go onto the pile, whose place `base` is their first.
__device__ __forceinline__ void move_back(const MapParams& P, const MapShared& S, int r0, int n, int64_t total, int64_t base) {
  for (int64_t e = threadIdx.x; e < total; e += kMapThreads) {
    const int x = owner(S.back, n, e);
    if (S.from[x] < 0) continue;
    const int column = S.from[x] + static_cast<int>(e - S.back[x]);
    const int32_t block = __ldcg(P.tables + static_cast<int64_t>(r0 + x) * P.max_blocks + column);
    if (block < 0 || block >= P.num_blocks) raise_block(P.status, r0 + x, column * P.block_size);
    P.free_blocks[base + e] = block;
  }
}

// TOKENS: lists token rows [row0, row1).  STATE: moves blocks, writes offsets, and tells of what is wrong.
// lens: writes the new lengths and the new count of free blocks.
template <bool TOKENS, bool STATE>
__device__ __forceinline__ void map_step(const MapParams& P, int64_t n_free, int64_t row0, int64_t row1, bool lens, MapShared& S) {
  constexpr bool raise = STATE;
  const int tid = threadIdx.x;
  const bool one = P.n_req <= kMapThreads;   // one sweep: read and summed once
  int64_t given = 0;                         // blocks given back that had room on the pile
  if (!one) {
    // all that is given back comes before anything that is taken
    int64_t base = 0;
    for (int r0 = 0; r0 < P.n_req; r0 += kMapThreads) {
      const Request q = read_request(P, r0 + tid, raise);
      Counts c = q.counts(), total;
      const int64_t back = c.back;
      c = block_scan(Counts{back, 0, 0}, S, total);
      if (total.back == 0) continue;
      const bool fits = n_free + base + c.back <= P.num_blocks;
      if (back > 0 && !fits && raise) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_CAPACITY));
      if (STATE) {
        S.back[tid + 1] = c.back;
        if (tid == 0) S.back[0] = 0;
        S.from[tid] = back > 0 && fits ? q.want : -1;
        __syncthreads();
        move_back(P, S, r0, min(kMapThreads, P.n_req - r0), total.back, n_free + base);
      }
      given = max(given, n_free + base + total.back <= P.num_blocks ? base + total.back : block_max(fits ? base + c.back : 0, S));
      base += total.back;
    }
    __threadfence_block();
  }
  Counts base{0, 0, 0};   // of the requests before this sweep
  int64_t taken = 0;
  for (int r0 = 0; r0 < P.n_req; r0 += kMapThreads) {
    const int r = r0 + tid, n = min(kMapThreads, P.n_req - r0);
    const Request q = read_request(P, r, raise && one);
    const Counts mine = q.counts();
    Counts total;
    const Counts c = base + block_scan(mine, S, total);
    const bool room = n_free + c.back <= P.num_blocks;   // (also false behind a request whose blocks had none)
    if (one) {
      if (mine.back > 0 && !room && raise) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_CAPACITY));
      given = n_free + total.back <= P.num_blocks ? total.back : block_max(room ? c.back : 0, S);
    }
    const int64_t pile = n_free + given;
    const bool fits = c.rows <= P.n_tokens;
    const bool ok = q.legal && (mine.back == 0 || room) && (q.grow <= 0 || fits) && (mine.need == 0 || c.need <= pile);
    if (TOKENS || STATE) {
      __syncthreads();   // the last sweep's lists have been read
      S.back[tid + 1] = c.back - base.back;
      S.rows[tid + 1] = c.rows;
      S.need[tid + 1] = c.need - base.need;
      if (tid == 0) {
        S.back[0] = S.need[0] = 0;
        S.rows[0] = base.rows;
      }
      S.from[tid] = mine.back > 0 && ok ? q.want : -1;
      S.to[tid] = mine.need > 0 && ok ? q.have : -1;
      S.len[tid] = ok ? static_cast<int>(q.len) : -1;
      S.shift[tid] = TOKENS && P.shift != nullptr && r < P.n_req ? __ldcg(P.shift + r) : 0;
      __syncthreads();
    }
    if (STATE && r < P.n_req) {
      if ((q.grow > 0 && !fits) || (mine.need > 0 && c.need > pile)) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_CAPACITY));
      P.indptr[r + 1] = static_cast<int32_t>(min(c.rows, static_cast<int64_t>(P.n_tokens)));
    }
    if (lens && r < P.n_req) P.new_lens[r] = static_cast<int32_t>(ok ? q.len + q.grow : q.len);
    if (STATE && one && total.back > 0) {
      move_back(P, S, r0, n, total.back, n_free);
      __threadfence_block();
      __syncthreads();   // blocks put on the pile may be taken again
    }
    if (TOKENS) {
      const int64_t stop = min(row1, base.rows + total.rows);
      for (int64_t i = max(row0, base.rows) + tid; i < stop; i += kMapThreads) {
        const int x = owner(S.rows, n, i);
        const int slot = S.len[x] < 0 ? -1 : S.len[x] + static_cast<int>(i - S.rows[x]);
        P.req[i] = r0 + x;
        P.slot[i] = slot;
        if (P.pos != nullptr)
          P.pos[i] = slot < 0 ? 0 : static_cast<int32_t>(static_cast<uint32_t>(slot) + static_cast<uint32_t>(S.shift[x]));
      }
    }
    if (STATE && total.need > 0) {
      // granted requests come first among those that need blocks: the elements up to the pile's end
      const int64_t stop = min(total.need, pile - base.need);
      for (int64_t e = tid; e < stop; e += kMapThreads) {
        const int x = owner(S.need, n, e);
        if (S.to[x] < 0) continue;
        const int column = S.to[x] + static_cast<int>(e - S.need[x]);
        const int32_t block = __ldcg(P.free_blocks + (pile - 1 - base.need - e));
        if (block < 0 || block >= P.num_blocks) raise_block(P.status, r0 + x, column * P.block_size);
        P.tables[static_cast<int64_t>(r0 + x) * P.max_blocks + column] = block;
      }
    }
    // taken so far: the largest sum that was granted
    if (lens && total.need > 0) taken = max(taken, block_max(ok && mine.need > 0 ? c.need : 0, S));
    base = base + total;
  }
  if (TOKENS) {   // padding behind the last request's tokens
    for (int64_t i = max(row0, base.rows) + tid; i < row1; i += kMapThreads) {
      P.req[i] = 0;
      P.slot[i] = -1;
      if (P.pos != nullptr) P.pos[i] = 0;
    }
  }
  if (STATE && tid == 0) P.indptr[0] = 0;
  if (lens && tid == 0) *P.new_n_free = static_cast<int32_t>(n_free + given - taken);
}

__global__ void __launch_bounds__(kMapThreads) k_map_tokens(const __grid_constant__ MapParams P) {
  __shared__ MapShared S;
  int64_t n_free = __ldcg(P.n_free);
  if (n_free < 0 || n_free > P.num_blocks) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_BAD_LENGTH));
    n_free = 0;
  }
  if (gridDim.x == 1) {
    __syncthreads();   // every thread has the count, which the step may write
    map_step<true, true>(P, n_free, 0, P.n_tokens, true, S);
    return;
  }
  // The first CTA moves the blocks, which no other reads; the others list the tokens.  Lengths and
  // the count that are written over what all read are left to the CTA whose ticket is the last.
  const bool in_place = P.new_lens == P.lens || P.new_n_free == P.n_free;
  if (blockIdx.x == 0) {
    map_step<false, true>(P, n_free, 0, 0, !in_place, S);
  } else {
    const int64_t part = blockIdx.x - 1, parts = gridDim.x - 1;
    map_step<true, false>(P, n_free, P.n_tokens * part / parts, P.n_tokens * (part + 1) / parts, false, S);
  }
  if (!in_place) return;
  __syncthreads();     // this CTA has read its inputs
  if (threadIdx.x == 0) {
    __threadfence();
    S.ticket = atomicAdd(P.ticket, 1u);
    __threadfence();
  }
  __syncthreads();
  if (S.ticket != gridDim.x - 1) return;
  if (threadIdx.x == 0) *P.ticket = 0;
  map_step<false, false>(P, n_free, 0, 0, true, S);
}

}  // namespace

cudaError_t launch_map(const MapParams& p, int sm_count, cudaStream_t s) {
  const int64_t parts = (static_cast<int64_t>(p.n_tokens) + kMapTokensPerCta - 1) / kMapTokensPerCta;
  const unsigned grid = static_cast<unsigned>(parts <= 1 ? 1 : 1 + (parts >= sm_count ? sm_count - 1 : parts));
  k_map_tokens<<<grid, kMapThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace pic
