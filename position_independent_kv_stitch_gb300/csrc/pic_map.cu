// Block tables and token lists from request lengths (sm_103a): the step of a
// serving loop that gives every new token its place in the paged cache.
//
// With have = ceil(len / block_size) and want = ceil((len + grow) / block_size):
// requests that shrink put blocks [want, have) of their table on the pile of free
// blocks, in order; then those that grow take theirs from its top, in order,
// while it lasts.  Token i of request r gets slot len + i.
//
// Everything follows from prefix sums over the requests.  Bound: for a decode
// step a launch and a chain of five dependent reads (counts, sums, table,
// pile, stores); for prompts the stores of 12 bytes a token.  A CTA of 1,024 threads
// sums all requests itself, 1,024 at a time, and lists its own part of the tokens; the
// CTA whose ticket is the last, when all have read the inputs, moves the blocks and
// writes the new lengths, which may be the inputs' own memory.
#include "pic_decode.h"
#include "pic_paged.cuh"

namespace pic {
namespace {

using namespace dev;

constexpr int kMapThreads = 1024, kMapWarps = kMapThreads / 32;
constexpr int kMapTokensPerCta = 4096;   // more CTAs beyond this
constexpr unsigned kFull = 0xffffffffu;

// Sums over the CTA: `v` becomes the inclusive prefix sum, the return value is the total.
__device__ __forceinline__ int64_t block_scan(int64_t& v, int64_t* s_warp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += up;
  }
  __syncthreads();   // s_warp is free
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int64_t w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(kFull, w, o);
    if (lane >= o) w += up;
  }
  if (warp > 0) v += __shfl_sync(kFull, w, warp - 1);
  return __shfl_sync(kFull, w, 31);
}

struct Request {
  int64_t len, grow;
  int have, want;
  bool legal;
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
  q.have = static_cast<int>((q.len + P.block_size - 1) / P.block_size);
  q.want = static_cast<int>((to + P.block_size - 1) / P.block_size);
  return q;
}

struct MapShared {
  int64_t warp[kMapWarps];
  int64_t start[kMapThreads + 1];   // first token row of each request of the sweep
  int len[kMapThreads];             // its length; -1: gets no slots
  int shift[kMapThreads];
  uint32_t ticket;
};

// Blocks given back: the count, and with MOVE the blocks themselves; `full`: not all had room.
template <bool MOVE>
__device__ __forceinline__ int64_t give_back(const MapParams& P, int64_t n_free, MapShared& S, bool raise, bool& full) {
  int64_t base = 0;   // blocks of the requests before this sweep
  int64_t given = 0;  // of those, the ones that found room on the pile
  for (int r0 = 0; r0 < P.n_req; r0 += kMapThreads) {
    const int r = r0 + static_cast<int>(threadIdx.x);
    const Request q = read_request(P, r, raise);
    const int64_t n = q.legal && q.grow < 0 ? q.have - q.want : 0;
    int64_t at = n;
    const int64_t total = block_scan(at, S.warp);
    at += base;       // one past this request's last
    if (n > 0) {
      if (n_free + at > P.num_blocks) {
        if (raise) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_CAPACITY));
      } else if (MOVE) {
        const int32_t* from = P.tables + static_cast<int64_t>(r) * P.max_blocks + q.want;
        for (int64_t i = 0; i < n; ++i) {
          const int32_t block = __ldcg(from + i);
          if (block < 0 || block >= P.num_blocks) raise_block(P.status, r, (q.want + static_cast<int>(i)) * P.block_size);
          P.free_blocks[n_free + at - n + i] = block;
        }
      }
    }
    // what fits: requests in order, up to the first whose blocks do not
    const int64_t fits = n > 0 && n_free + at <= P.num_blocks ? at : 0;
    int64_t best = fits;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(kFull, best, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) S.warp[threadIdx.x >> 5] = best;
    __syncthreads();
    best = S.warp[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(kFull, best, o));
    given = max(given, best);
    base += total;
  }
  full = n_free + base > P.num_blocks;
  return given;
}

// Grants in request order (full: also whether a shrinking request's blocks had room).  TOKENS: lists rows [row0, row1); STATE: moves blocks, writes lengths and offsets.
template <bool TOKENS, bool STATE>
__device__ __forceinline__ void grant(const MapParams& P, int64_t n_free, int64_t pile, bool full, int64_t row0, int64_t row1,
                                      MapShared& S) {
  int64_t rows = 0, asked = 0, backed = 0, taken = 0;   // of the requests before this sweep
  for (int r0 = 0; r0 < P.n_req; r0 += kMapThreads) {
    const int r = r0 + static_cast<int>(threadIdx.x);
    const Request q = read_request(P, r, false);
    const int64_t n = q.grow > 0 ? q.grow : 0;
    const int64_t need = q.legal && q.grow > 0 ? q.want - q.have : 0;
    int64_t end = n, top = need;
    const int64_t all_rows = block_scan(end, S.warp), all_need = block_scan(top, S.warp);
    end += rows;
    top += asked;
    const bool fits = end <= P.n_tokens;
    bool ok = q.legal && (q.grow <= 0 || fits) && (need == 0 || top <= pile);
    if (full) {
      const int64_t n_back = q.legal && q.grow < 0 ? q.have - q.want : 0;
      int64_t at = n_back;
      const int64_t all_back = block_scan(at, S.warp);
      if (n_back > 0 && n_free + backed + at > P.num_blocks) ok = false;
      backed += all_back;
    }
    if (STATE && r < P.n_req) {
      if (!fits || !(need == 0 || top <= pile)) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_CAPACITY));
      P.indptr[r + 1] = static_cast<int32_t>(min(end, static_cast<int64_t>(P.n_tokens)));
      P.new_lens[r] = static_cast<int32_t>(ok ? q.len + q.grow : q.len);
      if (ok && need > 0) {
        int32_t* to = P.tables + static_cast<int64_t>(r) * P.max_blocks + q.have;
        const int64_t first = top - need;   // blocks asked for before this request's
        for (int64_t i = 0; i < need; ++i) {
          const int32_t block = __ldcg(P.free_blocks + (pile - 1 - first - i));
          if (block < 0 || block >= P.num_blocks) raise_block(P.status, r, (q.have + static_cast<int>(i)) * P.block_size);
          to[i] = block;
        }
      }
    }
    if (TOKENS) {
      __syncthreads();   // the last sweep's lists have been read
      S.start[threadIdx.x + 1] = end;
      if (threadIdx.x == 0) S.start[0] = rows;
      S.len[threadIdx.x] = ok && r < P.n_req ? static_cast<int>(q.len) : -1;
      S.shift[threadIdx.x] = P.shift != nullptr && r < P.n_req ? __ldcg(P.shift + r) : 0;
      __syncthreads();
      const int64_t stop = min(row1, rows + all_rows);
      for (int64_t i = max(row0, rows) + threadIdx.x; i < stop; i += kMapThreads) {
        int lo = 0, hi = kMapThreads;   // start[lo] <= i < start[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (S.start[mid] <= i) lo = mid;
          else hi = mid;
        }
        const int slot = S.len[lo] < 0 ? -1 : S.len[lo] + static_cast<int>(i - S.start[lo]);
        P.req[i] = r0 + lo;
        P.slot[i] = slot;
        if (P.pos != nullptr)
          P.pos[i] = slot < 0 ? 0 : static_cast<int32_t>(static_cast<uint32_t>(slot) + static_cast<uint32_t>(S.shift[lo]));
      }
    }
    if (STATE) {
      // blocks taken so far: the largest sum that was granted
      int64_t mine = ok && need > 0 ? top : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mine = max(mine, __shfl_xor_sync(kFull, mine, o));
      __syncthreads();
      if ((threadIdx.x & 31) == 0) S.warp[threadIdx.x >> 5] = mine;
      __syncthreads();
      mine = S.warp[threadIdx.x & 31];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mine = max(mine, __shfl_xor_sync(kFull, mine, o));
      taken = max(taken, mine);
    }
    rows += all_rows;
    asked += all_need;
  }
  if (TOKENS) {   // padding behind the last request's tokens
    for (int64_t i = max(row0, rows) + threadIdx.x; i < row1; i += kMapThreads) {
      P.req[i] = 0;
      P.slot[i] = -1;
      if (P.pos != nullptr) P.pos[i] = 0;
    }
  }
  if (STATE && threadIdx.x == 0) {
    P.indptr[0] = 0;
    *P.new_n_free = static_cast<int32_t>(pile - taken);
  }
}

__global__ void __launch_bounds__(kMapThreads) k_map_tokens(const __grid_constant__ MapParams P) {
  __shared__ MapShared S;
  int64_t n_free = __ldcg(P.n_free);
  if (n_free < 0 || n_free > P.num_blocks) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_BAD_LENGTH));
    n_free = 0;
  }
  bool full;
  if (gridDim.x == 1) {
    const int64_t given = give_back<true>(P, n_free, S, true, full);
    __threadfence_block();
    __syncthreads();   // blocks put on the pile may be taken again
    grant<true, true>(P, n_free, n_free + given, full, 0, P.n_tokens, S);
    return;
  }
  const int64_t row0 = static_cast<int64_t>(P.n_tokens) * blockIdx.x / gridDim.x;
  const int64_t row1 = static_cast<int64_t>(P.n_tokens) * (blockIdx.x + 1) / gridDim.x;
  const int64_t given = give_back<false>(P, n_free, S, blockIdx.x == 0, full);
  grant<true, false>(P, n_free, n_free + given, full, row0, row1, S);
  __syncthreads();     // this CTA has read its inputs
  if (threadIdx.x == 0) {
    __threadfence();
    S.ticket = atomicAdd(P.ticket, 1u);
    __threadfence();
  }
  __syncthreads();
  if (S.ticket != gridDim.x - 1) return;
  if (threadIdx.x == 0) *P.ticket = 0;
  give_back<true>(P, n_free, S, false, full);
  __threadfence_block();
  __syncthreads();
  grant<false, true>(P, n_free, n_free + given, full, 0, 0, S);
}

}  // namespace

cudaError_t launch_map(const MapParams& p, int sm_count, cudaStream_t s) {
  const int64_t parts = (static_cast<int64_t>(p.n_tokens) + kMapTokensPerCta - 1) / kMapTokensPerCta;
  const unsigned grid = static_cast<unsigned>(parts < 1 ? 1 : (parts > sm_count ? sm_count : parts));
  k_map_tokens<<<grid, kMapThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace pic
