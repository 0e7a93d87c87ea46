// Attention of one new token per request over its paged cache (GQA, sm_103a),
// with lengths read on the device: the decode step of a context that grows.
//
//   s_t = scale * q . k_t,  p = softmax(s) over slots [0, len),
//   out = sum_t p_t v_t,  lse = log sum_t exp(s_t),
//   and, when weights are kept: w[slot t] += sum over the query heads p_t.
//
// Every cached row is read once, so HBM bounds the step.  The cache is cut
// along its length: all requests' tiles (16 slots of one request) form one
// list, and each warp takes a contiguous, equally long range of it for one
// KV head, whatever the requests' lengths are.  A warp keeps a running
// maximum, sum and weighted values for the query heads of its KV head (online
// softmax) and leaves one record per request it crosses; a second kernel
// joins the records.  Range p and request r cross at most once and both only
// grow along the list, so record p + r is unique without any bookkeeping.
//
// Warps work alone: each streams its rows through its own ring in shared
// memory with cp.async (16 bytes a lane, rows past the end filled with zeros)
// and no barrier joins warps.  A CTA's warps hold adjacent KV heads of the same
// rows, so the rows of a token are read together.
//
// Products: S = Q K^T and O += P V on mma.sync m16n8k16 (bf16 in, fp32
// accumulate).  A tile has one row per query head of a KV head, 1 to 16 of
// them: tcgen05's 64 or 128 rows would be mostly padding, and the step waits for
// memory.  K and V enter as stored; P is an fp32 value and is split into bf16
// hi + lo parts (a third part when the output is fp32), each a product of its
// own, so P keeps 16 (24) significant bits.  With up to 8 query heads the hi and
// lo parts share one product, in rows g and g + 8.
#include <algorithm>
#include <cfloat>

#include <cuda_bf16.h>

#include "pic_decode.h"
#include "pic_device.cuh"
#include "pic_paged.cuh"

namespace pic {
namespace {

using namespace dev;

constexpr unsigned kFull = 0xffffffffu;
constexpr int TT = kPagedTile;
constexpr float kLn2 = 0.69314718055994531f;

__host__ __device__ constexpr int paged_stages(int D) { return D <= 64 ? 6 : (D <= 128 ? 3 : 2); }
__host__ __device__ constexpr int paged_warps(int D) { return D <= 128 ? kPagedWarps : kPagedWarps * 3 / 4; }
__host__ __device__ constexpr int stage_bytes(int D) { return 2 * TT * D * 2; }

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (x, y) as a bf16 pair, and what the pair leaves out
__device__ __forceinline__ uint32_t take_bf16(float& x, float& y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const float2 f = __bfloat1622float2(h);
  x -= f.x;
  y -= f.y;
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A request's legal length, 0 for one outside [0, max_len] (which is raised).
__device__ __forceinline__ int legal_len(int len, int max_len, uint32_t* status, bool raise) {
  if (len >= 0 && len <= max_len) return len;
  if (raise) atomicOr(status, static_cast<uint32_t>(PIC_DEV_BAD_LENGTH));
  return 0;
}

// The tile list all kernels share: request r owns ceil(len / 16) tiles, in
// order; range p of n holds tiles [T p / n, T (p + 1) / n).
struct TileList {
  int64_t total;   // T
  int64_t parts;   // n: fewer than P.parts when there are few tiles
  __device__ int64_t begin(int64_t p) const { return total * p / parts; }
};
__device__ __forceinline__ int tiles_of(const PagedParams& P, int r, bool raise) {
  return (legal_len(__ldg(P.lens + r), P.max_len, P.status, raise) + TT - 1) / TT;
}
__device__ __forceinline__ TileList tile_list(const PagedParams& P, int lane, bool raise) {
  int64_t n = 0;
  for (int r = lane; r < P.n_req; r += 32) n += tiles_of(P, r, raise);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(kFull, n, o);
  TileList L;
  L.total = n;
  const int64_t want = (n + kPagedMinTiles - 1) / kPagedMinTiles;
  L.parts = want < P.parts ? (want < 1 ? 1 : want) : P.parts;
  return L;
}
// The request that holds tile t of the list, and its first tile (warp-wide;
// t below the total).
__device__ __forceinline__ void find_tile(const PagedParams& P, int64_t t, int lane, int& req, int64_t& first) {
  int64_t base = 0;
  for (int r0 = 0; r0 < P.n_req; r0 += 32) {
    const int r = r0 + lane;
    int64_t n = r < P.n_req ? tiles_of(P, r, false) : 0;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned hit = __ballot_sync(kFull, base + incl > t);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      req = r0 + src;
      first = base + __shfl_sync(kFull, incl - n, src);
      return;
    }
    base += __shfl_sync(kFull, incl, 31);
  }
  req = P.n_req;
  first = base;
}
// First tile of request r (warp-wide).
__device__ __forceinline__ int64_t first_tile(const PagedParams& P, int r, int lane) {
  int64_t n = 0;
  for (int i = lane; i < r; i += 32) n += tiles_of(P, i, false);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(kFull, n, o);
  return n;
}

// A place in the list: tile `tile` of request `req`.
struct Place {
  int req, tile, len;
  int64_t first;   // the request's first tile in the list
};
__device__ __forceinline__ void advance(const PagedParams& P, Place& x) {
  if (x.req >= P.n_req) return;   // past the list
  const int n = (x.len + TT - 1) / TT;
  if (++x.tile < n) return;
  x.first += n;
  x.tile = 0;
  do {
    ++x.req;
    x.len = x.req < P.n_req ? legal_len(__ldg(P.lens + x.req), P.max_len, P.status, false) : 0;
  } while (x.len == 0 && x.req < P.n_req);
}

// WIDE: 9 to 16 query heads per warp, one per row of the products; else up to
// 8, in rows 0-7 (rows 8-15 carry the lo parts of P).  F32: fp32 output.
template <int D, bool WIDE, bool F32>
__global__ void __launch_bounds__(32 * paged_warps(D), 1) k_paged_attend(const __grid_constant__ PagedParams P) {
  constexpr int KS = D / 16, NT = D / 8, CH = D / 8;  // k-steps, output n-tiles, 16-byte chunks of a row
  constexpr int NS = paged_stages(D);
  constexpr int ROWS = 32 / CH > 0 ? 32 / CH : 1;     // rows one warp-wide copy covers
  constexpr int COPIES = TT * CH / 32;                // warp-wide copies of a K (or V) tile
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + warp * NS * stage_bytes(D);
  const int64_t w = static_cast<int64_t>(blockIdx.x) * paged_warps(D) + warp;
  const int vh = static_cast<int>(w % P.v_heads);
  const int64_t part = w / P.v_heads;
  const TileList L = tile_list(P, lane, w == 0);
  if (part >= L.parts || L.total == 0) return;
  const int64_t t_begin = L.begin(part), t_end = L.begin(part + 1);
  if (t_begin >= t_end) return;

  const int hk = vh / P.passes;
  const int g0 = (vh % P.passes) * 16;                       // first query head of the pass within the group
  const int n_heads = min(16, P.group - g0);
  const int hq0 = hk * P.group + g0;
  const int g = lane >> 2, tq = lane & 3;

  Place load;
  find_tile(P, t_begin, lane, load.req, load.first);
  load.tile = static_cast<int>(t_begin - load.first);
  load.len = load.req < P.n_req ? legal_len(__ldg(P.lens + load.req), P.max_len, P.status, false) : 0;
  Place cur = load;
  int64_t t_load = t_begin;

  // this lane's cache row of a tile (lane t: slot t % 16), -1 past the end or for a bad block
  auto row_of = [&](const Place& x) -> int {
    const int slot = x.tile * TT + (lane & (TT - 1));
    if (slot >= x.len) return -1;
    const int64_t row = paged_row(P.paged, x.req, slot);
    if (row < 0 && lane < TT) raise_block(P.status, x.req, slot);
    return static_cast<int>(row);   // below 2^31 (checked when the context was made)
  };
  auto issue = [&](int stage, int row) {
    const uint32_t k_dst = ring + stage * stage_bytes(D), v_dst = k_dst + TT * D * 2;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int r = CH >= 32 ? i : i * ROWS + lane / CH, c = lane % CH;
      const int src_row = __shfl_sync(kFull, row, r);
      const bool live = src_row >= 0;
      const int64_t off = static_cast<int64_t>(live ? src_row : 0) * P.row_bytes + hk * D * 2 + c * 16;
      const uint32_t dst = r * D * 2 + ((c ^ (r & 7)) << 4);
      cp_async16_zfill(k_dst + dst, P.k_cache + off, live);
      cp_async16_zfill(v_dst + dst, P.v_cache + off, live);
    }
  };

  // fill the ring but for one stage; the rows of the next tile are looked up one tile ahead
  unsigned live_ring[NS];
  int next_row = row_of(load);
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) {
    live_ring[i] = 0;
    if (t_load < t_end) {
      live_ring[i] = __ballot_sync(kFull, next_row >= 0);
      issue(i, next_row);
      ++t_load;
      if (t_load < t_end) {
        advance(P, load);
        next_row = row_of(load);
      }
    }
    cp_commit();
  }
  live_ring[NS - 1] = 0;

  uint32_t qa[KS][4];
  float o[NT][4];
  float m_run[2], l_run[2];
  // ldmatrix addresses of this lane, before the swizzle
  const int mi = lane >> 3, ri = lane & 7;
  const int k_row = ri + ((mi & 2) ? 8 : 0), v_row = ri + ((mi & 1) ? 8 : 0);
  bool opened = false;

  int64_t t = t_begin;
  while (t < t_end) {
#pragma unroll
    for (int st = 0; st < NS; ++st) {
      if (t >= t_end) break;
      // the stage freed by the previous tile takes the next one
      {
        const int fs = st == 0 ? NS - 1 : st - 1;
        live_ring[fs] = 0;
        if (t_load < t_end) {
          live_ring[fs] = __ballot_sync(kFull, next_row >= 0);
          issue(fs, next_row);
          ++t_load;
          if (t_load < t_end) {
            advance(P, load);
            next_row = row_of(load);
          }
        }
        cp_commit();
      }
      if (!opened) {
        opened = true;
        m_run[0] = m_run[1] = -FLT_MAX;
        l_run[0] = l_run[1] = 0.0f;
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        const uint8_t* qp = P.q + cur.req * P.q_stride + static_cast<int64_t>(hq0) * D * 2;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int h = g + (x & 1) * 8, d = kk * 16 + (x >> 1) * 8 + 2 * tq;
            qa[kk][x] = (WIDE || (x & 1) == 0) && h < n_heads
                            ? __ldg(reinterpret_cast<const uint32_t*>(qp + (h * D + d) * 2))
                            : 0u;
          }
        }
      }
      cp_wait<NS - 1>();
      __syncwarp();
      const uint32_t kb = ring + st * stage_bytes(D), vb = kb + TT * D * 2;
      // ---- scores of the tile's 16 slots
      float s0[4] = {}, s1[4] = {};
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        uint32_t b[4];
        ldsm4(kb + k_row * D * 2 + (((2 * kk + (mi & 1)) ^ (k_row & 7)) << 4), b);
        mma(s0, qa[kk], b[0], b[1]);
        mma(s1, qa[kk], b[2], b[3]);
      }
      // [row half][slot 2tq, 2tq + 1, 8 + 2tq, 9 + 2tq]
      float sc[2][4] = {{s0[0], s0[1], s1[0], s1[1]}, {s0[2], s0[3], s1[2], s1[3]}};
      const unsigned live = live_ring[st];
      float p[2][4];
      float alpha[2] = {1.0f, 1.0f};
#pragma unroll
      for (int hf = 0; hf < (WIDE ? 2 : 1); ++hf) {
        float mt = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int slot = (i < 2 ? 0 : 8) + 2 * tq + (i & 1);
          sc[hf][i] = (live >> slot) & 1u ? sc[hf][i] * P.scale_log2 : -INFINITY;
          mt = fmaxf(mt, sc[hf][i]);
        }
        mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, 1));
        mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, 2));
        const float m_new = fmaxf(m_run[hf], mt);
        alpha[hf] = exp2f(m_run[hf] - m_new);
        m_run[hf] = m_new;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[hf][i] = exp2f(sc[hf][i] - m_new);
        l_run[hf] = l_run[hf] * alpha[hf] + ((p[hf][0] + p[hf][1]) + (p[hf][2] + p[hf][3]));
        if (P.scores != nullptr && g + 8 * hf < n_heads) {
          float* sp = P.scores + static_cast<int64_t>(hq0 + g + 8 * hf) * P.score_stride + t * TT + 2 * tq;
          *reinterpret_cast<float2*>(sp) = make_float2(sc[hf][0], sc[hf][1]);
          *reinterpret_cast<float2*>(sp + 8) = make_float2(sc[hf][2], sc[hf][3]);
        }
      }
      // the running maximum soon stays: most tiles leave the sums as they are
      if (!__all_sync(kFull, alpha[0] == 1.0f && alpha[1] == 1.0f)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][0] *= alpha[0];
          o[j][1] *= alpha[0];
          o[j][2] *= alpha[WIDE ? 1 : 0];
          o[j][3] *= alpha[WIDE ? 1 : 0];
        }
      }
      // ---- O += P V, P in bf16 parts
      uint32_t pa[3][4];
      if (WIDE) {
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          pa[x][0] = take_bf16(p[0][0], p[0][1]);
          pa[x][1] = take_bf16(p[1][0], p[1][1]);
          pa[x][2] = take_bf16(p[0][2], p[0][3]);
          pa[x][3] = take_bf16(p[1][2], p[1][3]);
        }
      } else {
        pa[0][0] = take_bf16(p[0][0], p[0][1]);
        pa[0][2] = take_bf16(p[0][2], p[0][3]);
        pa[0][1] = take_bf16(p[0][0], p[0][1]);
        pa[0][3] = take_bf16(p[0][2], p[0][3]);
        pa[1][0] = take_bf16(p[0][0], p[0][1]);
        pa[1][2] = take_bf16(p[0][2], p[0][3]);
        pa[1][1] = pa[1][3] = 0u;
      }
      constexpr int NP = (WIDE ? 2 : 1) + (F32 ? 1 : 0);
#pragma unroll
      for (int j = 0; j < NT; j += 2) {
        uint32_t b[4];
        ldsm4_t(vb + v_row * D * 2 + (((j + (mi >> 1)) ^ (v_row & 7)) << 4), b);
        if (F32) {
          // the tensor cores round sums towards zero: over a long range that
          // would show in fp32, so each tile's product is added here instead
          float y0[4] = {}, y1[4] = {};
#pragma unroll
          for (int x = 0; x < NP; ++x) {
            mma(y0, pa[x], b[0], b[1]);
            mma(y1, pa[x], b[2], b[3]);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            o[j][x] += y0[x];
            o[j + 1][x] += y1[x];
          }
        } else {
#pragma unroll
          for (int x = 0; x < NP; ++x) {
            mma(o[j], pa[x], b[0], b[1]);
            mma(o[j + 1], pa[x], b[2], b[3]);
          }
        }
      }
      __syncwarp();   // every lane has read the stage before it is refilled
      ++t;
      const int n_tiles = (cur.len + TT - 1) / TT;
      if (cur.tile + 1 == n_tiles || t == t_end) {
        // ---- the record of this range and request
        const int64_t rec = part + cur.req;
#pragma unroll
        for (int hf = 0; hf < (WIDE ? 2 : 1); ++hf) {
          float l = l_run[hf];
          l += __shfl_xor_sync(kFull, l, 1);
          l += __shfl_xor_sync(kFull, l, 2);
          const int h = g + 8 * hf;
          if (h < n_heads) {
            float* acc = P.rec_acc + (rec * P.q_heads + hq0 + h) * D;
#pragma unroll
            for (int j = 0; j < NT; ++j)
              *reinterpret_cast<float2*>(acc + 8 * j + 2 * tq) =
                  WIDE ? make_float2(o[j][2 * hf], o[j][2 * hf + 1])
                       : make_float2(o[j][0] + o[j][2], o[j][1] + o[j][3]);
            if (tq == 0) P.rec_ml[rec * P.q_heads + hq0 + h] = make_float2(m_run[hf], l);
          }
        }
        opened = false;
      }
      if (t < t_end) advance(P, cur);
    }
  }
}

// One CTA per (request, query head): joins the records of its ranges.  The
// warps take the records in turn, a lane D / 32 neighbouring dims of each, and
// add up their sums in warp order at the end.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinRecords = 512;   // record weights held in shared memory at a time

__device__ __forceinline__ float block_reduce(float v, bool is_max, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(kFull, v, o);
    v = is_max ? fmaxf(v, w) : v + w;
  }
  __syncthreads();   // red is free
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) v = is_max ? fmaxf(v, red[w]) : v + red[w];
  return v;
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(const __grid_constant__ PagedParams P) {
  constexpr int V = D / 32;   // dims of a lane
  __shared__ int64_t s_first;
  __shared__ TileList s_list;
  __shared__ float s_red[kJoinWarps];
  __shared__ float s_e[kJoinRecords];
  __shared__ float s_acc[kJoinWarps][D];
  asm volatile("griddepcontrol.launch_dependents;");
  const int r = blockIdx.x, hq = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) {
    const TileList L = tile_list(P, lane, false);
    const int64_t f = first_tile(P, r, lane);
    if (lane == 0) {
      s_list = L;
      s_first = f;
    }
  }
  const int n = tiles_of(P, r, false);
  __syncthreads();
  int64_t rec0 = 0;   // the request's first record
  int recs = 0;
  if (n > 0) {
    const TileList L = s_list;
    // the range of tile t is the largest p with begin(p) <= t
    const int64_t p0 = ((s_first + 1) * L.parts - 1) / L.total;
    recs = static_cast<int>(((s_first + n) * L.parts - 1) / L.total - p0 + 1);
    rec0 = p0 + r;
  }
  // everything above came from the caller's lengths; the records are the previous kernel's
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float2* ml = P.rec_ml + rec0 * P.q_heads + hq;
  const float* acc_in = P.rec_acc + (rec0 * P.q_heads + hq) * D;
  float mx = -FLT_MAX;
  for (int k = threadIdx.x; k < recs; k += kJoinThreads) mx = fmaxf(mx, ml[static_cast<int64_t>(k) * P.q_heads].x);
  const float M = block_reduce(mx, true, s_red);
  float part = 0.0f;
  float acc[V] = {};
  for (int k0 = 0; k0 < recs; k0 += kJoinRecords) {
    const int m = min(kJoinRecords, recs - k0);
    __syncthreads();   // s_e is free
    for (int k = threadIdx.x; k < m; k += kJoinThreads) {
      const float2 x = ml[static_cast<int64_t>(k0 + k) * P.q_heads];
      const float e = exp2f(x.x - M);
      s_e[k] = e;
      part += e * x.y;
    }
    __syncthreads();
#pragma unroll 4
    for (int k = warp; k < m; k += kJoinWarps) {
      const float e = s_e[k];
      const float* a = acc_in + static_cast<int64_t>(k0 + k) * P.q_heads * D + lane * V;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += e * a[i];
    }
  }
  const float sum = block_reduce(part, false, s_red);
#pragma unroll
  for (int i = 0; i < V; ++i) s_acc[warp][lane * V + i] = acc[i];
  __syncthreads();
  const int64_t out_at = (static_cast<int64_t>(r) * P.q_heads + hq) * D;
  for (int d = threadIdx.x; d < D; d += kJoinThreads) {
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) x += s_acc[w][d];
    const float v = n > 0 ? x / sum : 0.0f;
    if (P.out_bf16) static_cast<__nv_bfloat16*>(P.out)[out_at + d] = __float2bfloat16_rn(v);
    else static_cast<float*>(P.out)[out_at + d] = v;
  }
  if (threadIdx.x == 0) {
    const float l2 = n > 0 ? M + log2f(sum) : -INFINITY;
    if (P.lse != nullptr) P.lse[static_cast<int64_t>(r) * P.q_heads + hq] = l2 * kLn2;
    if (P.lse2 != nullptr) P.lse2[static_cast<int64_t>(r) * P.q_heads + hq] = l2;
  }
}

// Adds each slot's attention weight: a warp takes a run of tiles for one
// weight head, half a warp a tile, one lane a slot; the query heads are summed
// in order (no atomics: a slot belongs to one lane).  A lane looks up four
// slots, then loads their scores and old weights together: the step is a
// chain of two memory round trips, not bandwidth, so few of them count.
constexpr int kWeightThreads = 256;
constexpr int kWeightCtas = 6;      // per SM
constexpr int kWeightBatch = 4;

__global__ void __launch_bounds__(kWeightThreads, kWeightCtas) k_paged_weights(const __grid_constant__ PagedParams P) {
  const int lane = threadIdx.x & 31, half = lane >> 4, sl = lane & (TT - 1);
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kWeightThreads / 32) + (threadIdx.x >> 5);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kWeightThreads / 32) / P.weight_heads;
  const int wh = static_cast<int>(w % P.weight_heads);
  const int64_t part = w / P.weight_heads;
  if (part >= warps) return;
  const TileList L = tile_list(P, lane, false);
  const int64_t t_begin = L.total * part / warps, t_end = L.total * (part + 1) / warps;
  if (t_begin >= t_end) return;
  const int heads = P.q_heads / P.weight_heads;   // query heads of a weight head
  Place x;
  find_tile(P, t_begin, lane, x.req, x.first);
  x.tile = static_cast<int>(t_begin - x.first);
  x.len = legal_len(__ldg(P.lens + x.req), P.max_len, P.status, false);
  if (half != 0) advance(P, x);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int64_t t = t_begin + half; t < t_end; t += 2 * kWeightBatch) {
    int64_t at[kWeightBatch];
    int req[kWeightBatch];
#pragma unroll
    for (int u = 0; u < kWeightBatch; ++u) {
      at[u] = -1;
      req[u] = x.req;
      if (t + 2 * u >= t_end) continue;
      const int slot = x.tile * TT + sl;
      if (slot < x.len) {
        const int b = block_of(P.paged, slot);
        const int32_t block = __ldg(P.paged.tables + static_cast<int64_t>(x.req) * P.paged.max_blocks + b);
        if (block >= 0 && block < P.paged.num_cache_blocks)
          at[u] = (static_cast<int64_t>(block) * P.weight_heads + wh) * P.paged.block_size + (slot - b * P.paged.block_size);
      }
      advance(P, x);
      advance(P, x);
    }
    float old[kWeightBatch], sum[kWeightBatch];
#pragma unroll
    for (int u = 0; u < kWeightBatch; ++u) {
      sum[u] = 0.0f;
      if (at[u] >= 0) old[u] = P.weights[at[u]];
    }
    const float* sc = P.scores + wh * heads * P.score_stride + t * TT + sl;
#pragma unroll 2
    for (int h = 0; h < heads; ++h, sc += P.score_stride) {
#pragma unroll
      for (int u = 0; u < kWeightBatch; ++u)
        if (at[u] >= 0)
          sum[u] += exp2f(__ldcs(sc + 2 * u * TT) - P.lse2[static_cast<int64_t>(req[u]) * P.q_heads + wh * heads + h]);
    }
#pragma unroll
    for (int u = 0; u < kWeightBatch; ++u)
      if (at[u] >= 0) P.weights[at[u]] = old[u] + sum[u];
  }
}

// A kernel launched as a programmatic dependent of the one before it.
template <typename Kern>
cudaError_t launch_after(Kern kern, dim3 grid, int threads, const PagedParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D, bool WIDE, bool F32>
cudaError_t launch_attend_d(const PagedParams& p, int grid, cudaStream_t s) {
  auto kern = k_paged_attend<D, WIDE, F32>;
  const int smem = static_cast<int>(paged_smem(D));
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, 32 * paged_warps(D), smem, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const PagedParams& p, int grid, int sm_count, cudaStream_t s) {
  const bool wide = p.group > 8;
  cudaError_t e;
  if (wide) e = p.out_bf16 ? launch_attend_d<D, true, false>(p, grid, s) : launch_attend_d<D, true, true>(p, grid, s);
  else e = p.out_bf16 ? launch_attend_d<D, false, false>(p, grid, s) : launch_attend_d<D, false, true>(p, grid, s);
  if (e != cudaSuccess) return e;
  e = launch_after(k_paged_join<D>, dim3(p.n_req, p.q_heads), kJoinThreads, p, s);
  if (e != cudaSuccess || p.weights == nullptr) return e;
  const int need = (p.weight_heads + kWeightThreads / 32 - 1) / (kWeightThreads / 32);
  return launch_after(k_paged_weights, dim3(std::max(sm_count * kWeightCtas, need)), kWeightThreads, p, s);
}

}  // namespace

size_t paged_smem(int head_dim) {
  return static_cast<size_t>(paged_warps(head_dim)) * paged_stages(head_dim) * stage_bytes(head_dim);
}

int paged_warps_per_cta(int head_dim) { return paged_warps(head_dim); }

cudaError_t launch_paged(const PagedParams& p, int head_dim, int grid, int sm_count, cudaStream_t s) {
  if (head_dim == 64) return launch_d<64>(p, grid, sm_count, s);
  if (head_dim == 128) return launch_d<128>(p, grid, sm_count, s);
  return launch_d<256>(p, grid, sm_count, s);
}

}  // namespace pic
