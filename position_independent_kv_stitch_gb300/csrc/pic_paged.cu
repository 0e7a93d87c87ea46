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
// softmax) and leaves one record per request it crosses.  Range p and request
// r cross at most once and both only grow along the list, so record p + r is
// unique without any bookkeeping.  Later kernels (programmatic dependents) join
// the records into the outputs and add each slot's weight from the scores kept
// meanwhile.  One cooperative kernel with a grid barrier instead took 13.0 us
// against 11.0 for one request of 777 slots, and its eight warps per SM were
// too few for the weights.
//
// Warps work alone: each streams its rows through its own ring in shared
// memory with cp.async (16 bytes a lane, rows past the end filled with zeros)
// and no barrier joins warps.  A CTA's warps hold adjacent KV heads of the same
// rows, so the rows of a token are read together.
//
// Products: S = Q K^T and O += P V on mma.sync m16n8k16 (bf16 in, fp32
// accumulate).  A tile has one row per query head of a KV head, 1 to 16 of
// them: tcgen05's 64 or 128 rows would be mostly padding, and the step waits for
// memory.  (32 to 128 heads over latent rows would fill such a tile; they too are
// done here 16 at a time, see k_paged_latent.)  K and V enter as stored; P is an
// fp32 value and is split into bf16 hi + lo parts (a third part when the output is
// fp32), each a product of its own, so P keeps 16 (24) significant bits.  With up to
// 8 query heads the hi and lo parts share one product, in rows g and g + 8.
//
// Measured (GB300, 32 query over 8 KV heads of 128 dims, blocks of 16): 64
// requests of 16,384 slots, fp32 out, 622-643 us (6.7-6.9 TB/s of rows); 64 of
// 1-8,192 with weights 229 us (without 196: 6.6 TB/s); one of 131,071 with
// weights 106 us (without 91: 5.9 TB/s); one of 777 8.4-9.5 us; 3,000 of 64 77 us.
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

// Warps and ring depth: as many warps as the registers of the running values
// allow, and the ring that then fits.  Measured (bf16 out, no weights, GB/s): 64
// dims 12 x 4 5,490 (8 x 6 4,510, 16 x 2 5,570 with spills), 128 dims 8 x 3
// 6,780 (12 x 2 6,560, 6 x 4 6,570), 256 dims 4 x 3 5,100 (6 x 2 4,900).  At 256
// dims all 255 registers are used and 24 to 180 bytes a thread spilled; with 16
// query heads, whose running values are 256 registers' worth, that leaves 3,200 to 3,900.
__host__ __device__ constexpr int paged_warps(int D) { return D <= 64 ? 12 : (D <= 128 ? 8 : 4); }
__host__ __device__ constexpr int paged_stages(int D) { return D <= 64 ? 4 : 3; }
__host__ __device__ constexpr int stage_bytes(int D) { return 2 * TT * D * 2; }
// Scores leave a warp several tiles at a time, one bulk copy per head.
__host__ __device__ constexpr int score_tiles(int D, bool wide) { return (wide ? 2 : 4) * (D <= 64 ? 1 : 2); }
__host__ __device__ constexpr int score_pitch(int D, bool wide) { return score_tiles(D, wide) * TT + 4; }  // floats, bank-shifted
__host__ __device__ constexpr int score_stage(int D, bool wide) { return (wide ? 16 : 8) * score_pitch(D, wide); }

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool live, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void bulk_wait_read_all() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
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
// 2^x to 2 units in the last place; results below 2^-126 become 0
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
__device__ __forceinline__ int64_t parts_of(const PagedParams& P, int64_t total) {   // at least a tile each
  return total < P.parts ? (total < 1 ? 1 : total) : P.parts;
}
__device__ __forceinline__ TileList tile_list(const PagedParams& P, int lane, bool raise) {
  int64_t n = 0;
  for (int r = lane; r < P.n_req; r += 32) n += tiles_of(P, r, raise);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(kFull, n, o);
  TileList L;
  L.total = n;
  L.parts = parts_of(P, n);
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
// Leaves the first tiles of the requests that begin in tiles [t, t_end) of the
// list to the joins (warp-wide; t is in request r, whose first tile is `base`).
__device__ __forceinline__ void leave_first_tiles(const PagedParams& P, int64_t t, int64_t t_end, int r, int64_t base, int lane) {
  for (; r < P.n_req && base < t_end; r += 32) {
    const int64_t n = r + lane < P.n_req ? tiles_of(P, r + lane, false) : 0;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    const int64_t at = base + incl - n;
    if (n > 0 && at >= t && at < t_end) P.first[r + lane] = at;
    base += __shfl_sync(kFull, incl, 31);
  }
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
__device__ __forceinline__ void attend_range(const PagedParams& P, const TileList& L, int64_t w, uint8_t* smem) {
  constexpr int KS = D / 16, NT = D / 8, CH = D / 8;  // k-steps, output n-tiles, 16-byte chunks of a row
  constexpr int NS = paged_stages(D);
  constexpr int ROWS = 32 / CH > 0 ? 32 / CH : 1;     // rows one warp-wide copy covers
  constexpr int COPIES = TT * CH / 32;                // warp-wide copies of a K (or V) tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + warp * NS * stage_bytes(D);
  const int vh = static_cast<int>(w % P.v_heads);
  const int64_t part = w / P.v_heads;
  if (part >= L.parts || L.total == 0) return;
  const int64_t t_begin = L.begin(part), t_end = L.begin(part + 1);
  if (t_begin >= t_end) return;

  const int hk = vh / P.passes;
  const int g0 = (vh % P.passes) * 16;                       // first query head of the pass within the group
  const int n_heads = min(16, P.group - g0);
  const int hq0 = hk * P.group + g0;
  const int g = lane >> 2, tq = lane & 3;
  // the rows pass through L2 once (groups of more than 16 heads: once a pass, by
  // warps side by side); the scores, read again at the end, may stay
  uint64_t stream_once;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(stream_once));

  Place load;
  find_tile(P, t_begin, lane, load.req, load.first);
  if (P.first != nullptr && vh == 0) leave_first_tiles(P, t_begin, t_end, load.req, load.first, lane);
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
      cp_async16_zfill(k_dst + dst, P.k_cache + off, live, stream_once);
      cp_async16_zfill(v_dst + dst, P.v_cache + off, live, stream_once);
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
  float* stage = reinterpret_cast<float*>(smem + paged_warps(D) * NS * stage_bytes(D)) + warp * score_stage(D, WIDE);
  int n_staged = 0;   // tiles whose scores wait in the stage

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
      if (P.scores != nullptr && n_staged == 0) {
        bulk_wait_read_all();   // the stage has been copied out
        __syncwarp();
      }
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
        alpha[hf] = ex2(m_run[hf] - m_new);
        m_run[hf] = m_new;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[hf][i] = ex2(sc[hf][i] - m_new);
        l_run[hf] = l_run[hf] * alpha[hf] + ((p[hf][0] + p[hf][1]) + (p[hf][2] + p[hf][3]));
        if (P.scores != nullptr && g + 8 * hf < n_heads) {
          float* sp = stage + (g + 8 * hf) * score_pitch(D, WIDE) + n_staged * TT + 2 * tq;
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
          // would show in fp32 (1e-5 of the result over 16,384 slots; bf16 rounds
          // by 2e-3), so each tile's product is added here instead
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
      if (P.scores != nullptr && (++n_staged == score_tiles(D, WIDE) || t == t_end)) {
        // the staged tiles, one bulk copy a head
        fence_proxy_async_smem();
        __syncwarp();
        if (lane < n_heads)
          bulk_store(P.scores + (hq0 + lane) * P.score_stride + (t - n_staged) * TT, stage + lane * score_pitch(D, WIDE),
                     n_staged * TT * sizeof(float));
        bulk_commit();
        n_staged = 0;
      }
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
  bulk_wait_all();
}

template <int D, bool WIDE, bool F32>
__global__ void __launch_bounds__(32 * paged_warps(D), 1) k_paged_attend(const __grid_constant__ PagedParams P) {
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(128) uint8_t smem[];
  const TileList L = tile_list(P, threadIdx.x & 31, blockIdx.x == 0 && threadIdx.x < 32);
  if (P.first != nullptr && blockIdx.x == 0 && threadIdx.x == 0) P.first[P.n_req] = L.total;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * paged_warps(D);
  // one range each; more only when there are more heads than warps
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * paged_warps(D) + (threadIdx.x >> 5);
       w < static_cast<int64_t>(P.parts) * P.v_heads; w += warps)
    attend_range<D, WIDE, F32>(P, L, w, smem);
}

// ---- MLA: latent rows
//
// Every query head reads the same rows (512 latent dims and a 64-dim rope key,
// the latent also the value), so a CTA takes a range for 16 heads (more heads:
// more passes, whose CTAs read the same rows side by side) and works on it
// together, 32 slots of one request a step, the next step's rows on their way:
//   * warp w scores slots 16 (w / 4) .. + 15 over a quarter of the 576 dims (9
//     k-steps, whose query fragments stay in registers); the quarters meet in
//     shared memory;
//   * sixteen threads a head add them, keep the running maximum and sum (two
//     scores each) and leave P in bf16 parts, as above;
//   * warp w adds latent dims 64 w .. 64 w + 63 of every head.
// The three barriers of a step come between these; two CTAs per SM cover each
// other's.  Bound: the chain of a step's three parts and mma.sync's rate (400
// products a step of 37 KB; 600 TFLOP/s measured for mma.sync alone).  104 bytes a
// thread are spilled with fp32 output, 28 with bf16.
// Measured: 64 requests of 8,192 slots, 16 heads, 132 us (4.6 TB/s of
// rows; fp32 out 159); 128 heads 927 us (158 TFLOP/s of useful products, ten times the
// time of the rows or the products alone: eight passes of 16 heads; products of
// 64 or 128 heads on tcgen05, over tiles found from the lengths as here, are not built).
constexpr int kLatDims = 512, kLatRow = 576;
constexpr int kLatRowBytes = kLatRow * 2, kLatChunks = kLatRowBytes / 16;
constexpr int kLatHeads = 16;
constexpr int kLatSlots = 32, kLatTiles = kLatSlots / TT;   // of a step
constexpr int kLatThreads = 256;
constexpr int kLatSteps = kLatRow / 16 / 4;   // k-steps of a quarter
constexpr int kLatCtas = 2;              // per SM
constexpr int kLatPitch = 80;            // bytes of a head's P: eight rows in distinct banks
constexpr int kLatScorePitch = kLatSlots + 4;
constexpr int kLatRowPitch = kLatRowBytes + 16;   // an odd number of 16-byte chunks: eight rows in distinct banks
struct LatSmem {
  alignas(128) uint8_t kv[2][kLatSlots][kLatRowPitch];
  alignas(16) uint8_t q[kLatHeads][kLatRowPitch];
  alignas(16) uint8_t p[3][kLatHeads][kLatPitch];
  alignas(16) float s[4][kLatHeads][kLatScorePitch];   // scores over each quarter of the dims
  float alpha[kLatHeads];
  uint8_t live[2][kLatSlots];
};

template <bool F32>
__global__ void __launch_bounds__(kLatThreads, kLatCtas) k_paged_latent(const __grid_constant__ PagedParams P) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int NP = F32 ? 3 : 2, NT = kLatDims / 8 / 8;   // parts of P, output n-tiles of a warp
  extern __shared__ __align__(128) uint8_t smem[];
  LatSmem& S = *reinterpret_cast<LatSmem*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const int a_row = (lane & 7) + ((lane >> 3) & 1) * 8;    // ldmatrix row of a 16-row operand
  const int my_row = tid >> 3;                             // eight threads copy a row
  const int my_head = tid >> 4, my_slot = (tid & 15) * 2;  // sixteen threads weigh a head's slots
  const int quarter = warp & 3, col = (warp >> 2) * 16;    // this warp's part of the scores
  // ldmatrix addresses (stage 0): queries; keys as two n-tiles of 8 slots, both
  // halves of a k-step; the latent dims of this warp as value rows; P
  const uint32_t q_at = smem_u32(S.q[a_row]) + (2 * quarter * kLatSteps + (lane >> 4)) * 16;
  const uint32_t k_at = smem_u32(S.kv[0][col + (lane & 7) + (lane >> 4) * 8]) + (2 * quarter * kLatSteps + ((lane >> 3) & 1)) * 16;
  const uint32_t v_at = smem_u32(S.kv[0][a_row]) + (warp * NT + (lane >> 4)) * 16;
  const uint32_t p_at = smem_u32(S.p[0][a_row]) + (lane >> 4) * 16;
  const uint32_t row_at = smem_u32(S.kv[0][my_row]) + (tid & 7) * 16;
  constexpr uint32_t kStage = kLatSlots * kLatRowPitch;
  const TileList L = tile_list(P, lane, blockIdx.x == 0 && warp == 0);
  uint64_t policy;   // rows that no other CTA reads pass through L2 first-out
  if (P.passes == 1) asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  else asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
  if (P.first != nullptr && blockIdx.x == 0 && tid == 0) P.first[P.n_req] = L.total;

  for (int64_t w = blockIdx.x; w < static_cast<int64_t>(P.parts) * P.v_heads; w += gridDim.x) {
    const int hq0 = static_cast<int>(w % P.v_heads) * kLatHeads, n_heads = min(kLatHeads, P.q_heads - hq0);
    const int64_t part = w / P.v_heads;
    if (part >= L.parts || L.total == 0) continue;
    const int64_t t_end = L.begin(part + 1);
    int64_t t = L.begin(part), first;
    int r;
    find_tile(P, t, lane, r, first);
    if (P.first != nullptr && hq0 == 0 && warp == 0) leave_first_tiles(P, t, t_end, r, first, lane);
    // the range, request by request: slots [s0, s_end) of request r, in tiles up to slot s_pad
    for (; t < t_end; ++r) {
      const int len = legal_len(__ldg(P.lens + r), P.max_len, P.status, false);
      const int n_tiles = (len + TT - 1) / TT;
      const int s0 = static_cast<int>(t - first) * TT;
      const int s_pad = static_cast<int>(min(t_end - first, static_cast<int64_t>(n_tiles))) * TT, s_end = min(s_pad, len);
      if (s0 < s_pad) {
        const int64_t score_at = t * TT - s0;   // a slot's place in the scores
        // The block of this thread's slot, looked up a step ahead and looked at
        // only when its row is asked for: a warp stops where it touches a load
        // that has not arrived.
        const int32_t* table = P.paged.tables + static_cast<int64_t>(r) * P.paged.max_blocks;
        auto block_at = [&](int step_slot) {
          const int slot = step_slot + my_row;
          return slot < s_end ? __ldg(table + block_of(P.paged, slot)) : -1;
        };
        auto issue = [&](int stage, int step_slot, int block) {
          const int slot = step_slot + my_row;
          const bool live = block >= 0 && block < P.paged.num_cache_blocks;
          if (!live && slot < s_end && (tid & 7) == 0) raise_block(P.status, r, slot);
          const int64_t row = live ? static_cast<int64_t>(block) * P.paged.block_size + (slot - block_of(P.paged, slot) * P.paged.block_size) : 0;
          const uint8_t* src = P.k_cache + row * kLatRowBytes + (tid & 7) * 16;
#pragma unroll
          for (int i = 0; i < kLatChunks / 8; ++i)
            cp_async16_zfill(row_at + stage * kStage + i * 128, src + i * 128, live, policy);
          if ((tid & 7) == 0) S.live[stage][my_row] = live;
        };
        __syncthreads();   // shared memory is free
        issue(0, s0, block_at(s0));
        cp_commit();
        int next_block = block_at(s0 + kLatSlots);
        const uint8_t* qp = P.q + r * P.q_stride + static_cast<int64_t>(hq0) * kLatRowBytes;
        for (int i = tid; i < kLatHeads * kLatChunks; i += kLatThreads) {
          const int h = i / kLatChunks, c = i - h * kLatChunks;
          *reinterpret_cast<uint4*>(S.q[h] + c * 16) =
              h < n_heads ? __ldg(reinterpret_cast<const uint4*>(qp + i * 16)) : make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
        uint32_t qf[kLatSteps][4];
#pragma unroll
        for (int kk = 0; kk < kLatSteps; ++kk) ldsm4(q_at + kk * 32, qf[kk]);
        float o[NT][4], m_run = -FLT_MAX, l_run = 0.0f;
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        int stage = 0;
        for (int slot0 = s0; slot0 < s_pad; slot0 += kLatSlots, stage ^= 1) {
          cp_wait<0>();
          __syncthreads();   // the step's rows are in place; the other stage is free
          if (slot0 + kLatSlots < s_pad) issue(stage ^ 1, slot0 + kLatSlots, next_block);
          cp_commit();
          next_block = block_at(slot0 + 2 * kLatSlots);
          const uint32_t off = stage * kStage;
          // ---- scores of 16 slots over a quarter of the dims
          {
            float s0a[4] = {}, s1a[4] = {};
#pragma unroll
            for (int kk = 0; kk < kLatSteps; ++kk) {
              uint32_t b[4];
              ldsm4(k_at + off + kk * 32, b);
              mma(s0a, qf[kk], b[0], b[1]);
              mma(s1a, qf[kk], b[2], b[3]);
            }
            float* sp = &S.s[quarter][g][col + 2 * tq];
            *reinterpret_cast<float2*>(sp) = make_float2(s0a[0], s0a[1]);
            *reinterpret_cast<float2*>(sp + 8) = make_float2(s1a[0], s1a[1]);
            sp += 8 * kLatScorePitch;
            *reinterpret_cast<float2*>(sp) = make_float2(s0a[2], s0a[3]);
            *reinterpret_cast<float2*>(sp + 8) = make_float2(s1a[2], s1a[3]);
          }
          __syncthreads();   // all quarters of the scores
          {
            float2 x = *reinterpret_cast<const float2*>(&S.s[0][my_head][my_slot]);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
              const float2 y = *reinterpret_cast<const float2*>(&S.s[i][my_head][my_slot]);
              x.x += y.x;
              x.y += y.y;
            }
            const uint16_t live = *reinterpret_cast<const uint16_t*>(&S.live[stage][my_slot]);
            const float sc0 = (live & 0xff) != 0 ? x.x * P.scale_log2 : -INFINITY;
            const float sc1 = (live >> 8) != 0 ? x.y * P.scale_log2 : -INFINITY;
            if (P.scores != nullptr && my_head < n_heads && slot0 + my_slot < s_pad)
              *reinterpret_cast<float2*>(P.scores + (hq0 + my_head) * P.score_stride + score_at + slot0 + my_slot) =
                  make_float2(sc0, sc1);
            float m = fmaxf(sc0, sc1);
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
            m = fmaxf(m_run, m);
            const float alpha = ex2(m_run - m);
            m_run = m;
            float p0 = ex2(sc0 - m), p1 = ex2(sc1 - m);
            l_run = l_run * alpha + (p0 + p1);
#pragma unroll
            for (int i = 0; i < NP; ++i) *reinterpret_cast<uint32_t*>(&S.p[i][my_head][my_slot * 2]) = take_bf16(p0, p1);
            if ((tid & 15) == 0) S.alpha[my_head] = alpha;
          }
          __syncthreads();   // P is in place
          // ---- this warp's 64 latent dims of every head
          const float a0 = S.alpha[g], a1 = S.alpha[g + 8];
          if (!__all_sync(kFull, a0 == 1.0f && a1 == 1.0f)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              o[j][0] *= a0;
              o[j][1] *= a0;
              o[j][2] *= a1;
              o[j][3] *= a1;
            }
          }
          uint32_t a[NP][kLatTiles][4];
#pragma unroll
          for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int ks = 0; ks < kLatTiles; ++ks) ldsm4(p_at + i * kLatHeads * kLatPitch + ks * 32, a[i][ks]);
#pragma unroll
          for (int j = 0; j < NT; j += 2) {
            float y0[4] = {}, y1[4] = {};
#pragma unroll
            for (int ks = 0; ks < kLatTiles; ++ks) {
              uint32_t b[4];
              ldsm4_t(v_at + off + ks * 16 * kLatRowPitch + j * 16, b);
#pragma unroll
              for (int i = 0; i < NP; ++i) {
                if (F32) {   // added outside the tensor cores, as above
                  mma(y0, a[i][ks], b[0], b[1]);
                  mma(y1, a[i][ks], b[2], b[3]);
                } else {
                  mma(o[j], a[i][ks], b[0], b[1]);
                  mma(o[j + 1], a[i][ks], b[2], b[3]);
                }
              }
            }
            if (F32) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[j][e] += y0[e];
                o[j + 1][e] += y1[e];
              }
            }
          }
        }
        cp_wait<0>();
        // ---- the record of this range and request
        const int64_t rec = (part + r) * P.q_heads + hq0;
        float l = l_run;
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) l += __shfl_xor_sync(kFull, l, d);
        if ((tid & 15) == 0 && my_head < n_heads) P.rec_ml[rec + my_head] = make_float2(m_run, l);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int h = g + 8 * hf;
          if (h >= n_heads) continue;
          float* acc = P.rec_acc + (rec + h) * kLatDims + warp * 64 + 2 * tq;
#pragma unroll
          for (int j = 0; j < NT; ++j) *reinterpret_cast<float2*>(acc + 8 * j) = make_float2(o[j][2 * hf], o[j][2 * hf + 1]);
        }
      }
      first += n_tiles;
      t = max(t, min(first, t_end));
    }
  }
}

// ---- the join
constexpr int kFinishThreads = 256;
constexpr int kFinishWarps = kFinishThreads / 32;
constexpr int kFinishWeightCtas = 2;   // per SM, of 3 that fit: the joins run beside them

// The records of request r: the ranges that cross its n tiles (first: its
// first tile in the list).
struct Records {
  int64_t first;
  int count;
};
__device__ __forceinline__ Records records_of(const TileList& L, int64_t first, int n, int r) {
  Records x{0, 0};
  if (n > 0) {
    // the range of tile t is the largest p with begin(p) <= t
    const int64_t p0 = ((first + 1) * L.parts - 1) / L.total;
    x.count = static_cast<int>(((first + n) * L.parts - 1) / L.total - p0 + 1);
    x.first = p0 + r;
  }
  return x;
}
// The same for a join, which waits here for the kernel that wrote the records.
// Of few requests the lengths are walked again, before the wait; of many
// (P.first set) the attention kernel has left what is needed in the workspace:
// the total, and the first tile of each request that has any.
__device__ __forceinline__ Records join_records(const PagedParams& P, const TileList& walked, int r, int lane) {
  const int n = tiles_of(P, r, false);
  Records x;
  if (P.first == nullptr) {
    x = records_of(walked, first_tile(P, r, lane), n, r);
    asm volatile("griddepcontrol.wait;" ::: "memory");
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    TileList L;
    L.total = __ldcg(P.first + P.n_req);
    L.parts = parts_of(P, L.total);
    x = records_of(L, n > 0 ? __ldcg(P.first + r) : 0, n, r);
  }
  return x;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float2 load_ml(const PagedParams& P, const Records& x, int k, int hq) {
  return __ldcg(P.rec_ml + (x.first + k) * P.q_heads + hq);
}
// Largest running maximum of a query head's records, and the sum of their
// sums brought to it (warp-wide).
__device__ __forceinline__ void join_stats(const PagedParams& P, const Records& x, int hq, int lane, float& M, float& sum) {
  float m = -FLT_MAX, s = 0.0f;
  for (int k = lane; k < x.count; k += 32) {
    const float2 ml = load_ml(P, x, k, hq);
    const float up = fmaxf(m, ml.x);
    s = s * ex2(m - up) + ml.y * ex2(ml.x - up);
    m = up;
  }
  M = warp_max(m);
  sum = warp_sum(s * ex2(m - M));
}
// sum of the records k = begin, begin + step, ... of a query head, lane: dims lane V .. lane V + V - 1
template <int D>
__device__ __forceinline__ void join_values(const PagedParams& P, const Records& x, int hq, int lane, float M, int begin,
                                            int step, float (&acc)[D / 32]) {
  constexpr int V = D / 32;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll (V > 8 ? 2 : 8)
  for (int k = begin; k < x.count; k += step) {
    const float e = ex2(load_ml(P, x, k, hq).x - M);
    const float* a = P.rec_acc + ((x.first + k) * P.q_heads + hq) * D + lane * V;
    float v[V];
    if constexpr (V == 2) {
      const float2 y = __ldcg(reinterpret_cast<const float2*>(a));
      v[0] = y.x, v[1] = y.y;
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(a + i));
        v[i] = y.x, v[i + 1] = y.y, v[i + 2] = y.z, v[i + 3] = y.w;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += e * v[i];
  }
}
__device__ __forceinline__ void store_out(const PagedParams& P, int64_t at, float v) {
  if (P.out_bf16) static_cast<__nv_bfloat16*>(P.out)[at] = __float2bfloat16_rn(v);
  else static_cast<float*>(P.out)[at] = v;
}

// out and lse of (request, query head) `task`, by one warp or (ALL) by all
// warps of the CTA, which share the records.
template <int D, bool ALL>
__device__ __forceinline__ void join_output(const PagedParams& P, const Records& x, int r, int hq, float* part) {
  constexpr int V = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float M, sum, acc[V];
  join_stats(P, x, hq, lane, M, sum);
  join_values<D>(P, x, hq, lane, M, ALL ? warp : 0, ALL ? kFinishWarps : 1, acc);
  const int64_t task = static_cast<int64_t>(r) * P.q_heads + hq;
  if (ALL) {
#pragma unroll
    for (int i = 0; i < V; ++i) part[warp * D + lane * V + i] = acc[i];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kFinishThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kFinishWarps; ++w) v += part[w * D + d];
      store_out(P, task * D + d, sum == 0.0f ? 0.0f : v / sum);   // nothing attended: 0
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) store_out(P, task * D + lane * V + i, sum == 0.0f ? 0.0f : acc[i] / sum);
  }
  if (P.lse != nullptr && lane == 0 && (warp == 0 || !ALL)) P.lse[task] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * kLn2;
}

// Adds each slot's attention weight: a warp takes a run of tiles for one
// weight head, four lanes a tile, a lane four slots (one 16-byte load of each
// head's scores), and no atomics are needed: one warp has all heads of a slot,
// and their order follows from the lengths alone.  Few warps wait for long
// latencies here, so every load of a step is issued unconditionally (places past
// the run are read again from its last tile and dropped) and 16 tiles are in
// flight.  Where a run has fewer tiles, 2, 4 or 8 groups of four lanes share a
// tile's heads (at least four each) and add their sums: one weight for 128 heads
// of one request of 1,000 slots 22 us (one group: 60), one for 64 heads of 32,768
// slots 44 us (73).
constexpr int kWeightBatch = 2;

// Tiles [begin, end) of the list for weight head wh; the first tile of request
// r, which holds `begin`, is `first`.
struct WeightRun {
  int64_t begin, end, first;
  int r, wh;
};
// Part w / weight_heads of `all` equal parts (warp-wide; from the lengths alone).
__device__ __forceinline__ WeightRun weight_run(const PagedParams& P, const TileList& L, int64_t w, int64_t all, int lane) {
  WeightRun x;
  const int64_t part = w / P.weight_heads;
  x.wh = static_cast<int>(w - part * P.weight_heads);
  x.begin = L.total * part / all;
  x.end = L.total * (part + 1) / all;
  x.r = 0;
  x.first = 0;
  if (x.begin < x.end) find_tile(P, x.begin, lane, x.r, x.first);
  return x;
}
__device__ __forceinline__ void add_weights(const PagedParams& P, const WeightRun& run) {
  const int lane = threadIdx.x & 31, c = (lane & 3) * 4;
  const int wh = run.wh;
  const int64_t t_begin = run.begin, t_end = run.end;
  const int heads = P.q_heads / P.weight_heads;   // query heads of a weight head
  const int hq0 = wh * heads;
  const int bs = P.paged.block_size;
  const bool vec = (bs & 3) == 0 && (reinterpret_cast<uintptr_t>(P.weights) & 15) == 0;  // a lane's slots lie together
  const float* scores = P.scores + hq0 * P.score_stride + c;
  int r = run.r;
  int64_t first = run.first;
  for (int64_t t0 = t_begin; t0 < t_end;) {
    const int len = legal_len(__ldg(P.lens + r), P.max_len, P.status, false);
    const int n = (len + TT - 1) / TT;
    const int64_t piece = min(t_end, first + n);   // tiles [t0, piece) are of request r
    if (t0 < piece) {
      const float* lse2 = P.lse2 + static_cast<int64_t>(r) * P.q_heads + hq0;
      const int32_t* table = P.paged.tables + static_cast<int64_t>(r) * P.paged.max_blocks;
      // element of a slot's weight, -1 for a block outside the cache
      auto place = [&](int slot) -> int64_t {
        const int b = block_of(P.paged, slot);
        const int32_t block = __ldg(table + b);
        return block >= 0 && block < P.paged.num_cache_blocks
                   ? (static_cast<int64_t>(block) * P.weight_heads + wh) * bs + (slot - b * bs)
                   : -1;
      };
      int split = 1;   // quads that share a tile's heads
      while (split < 8 && 2 * split * (piece - t0) <= 8 * kWeightBatch && 8 * split <= heads) split *= 2;
      const int step = 8 / split, quad = (lane >> 2) / split, sub = (lane >> 2) % split;
      for (int64_t t = t0 + quad; t - quad < piece; t += step * kWeightBatch) {
        int64_t at[kWeightBatch], tile[kWeightBatch];
        int slot[kWeightBatch];
        float4 sum[kWeightBatch], old[kWeightBatch];
#pragma unroll
        for (int u = 0; u < kWeightBatch; ++u) {
          const bool mine = t + step * u < piece;
          tile[u] = mine ? t + step * u : piece - 1;
          slot[u] = static_cast<int>(tile[u] - first) * TT + c;
          at[u] = place(min(slot[u], len - 1));
          if (!mine || slot[u] >= len) at[u] = -1;
          sum[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        if (vec) {
#pragma unroll
          for (int u = 0; u < kWeightBatch; ++u)
            old[u] = __ldcg(reinterpret_cast<const float4*>(P.weights + (at[u] < 0 ? 0 : at[u])));
        }
#pragma unroll 4
        for (int h = sub; h < heads; h += split) {
          const float l2 = __ldcg(lse2 + h);
#pragma unroll
          for (int u = 0; u < kWeightBatch; ++u) {
            const float4 s = __ldcg(reinterpret_cast<const float4*>(scores + h * P.score_stride + tile[u] * TT));
            sum[u].x += ex2(s.x - l2);
            sum[u].y += ex2(s.y - l2);
            sum[u].z += ex2(s.z - l2);
            sum[u].w += ex2(s.w - l2);
          }
        }
        for (int o = 4; o < 4 * split; o *= 2) {
#pragma unroll
          for (int u = 0; u < kWeightBatch; ++u) {
            sum[u].x += __shfl_xor_sync(kFull, sum[u].x, o);
            sum[u].y += __shfl_xor_sync(kFull, sum[u].y, o);
            sum[u].z += __shfl_xor_sync(kFull, sum[u].z, o);
            sum[u].w += __shfl_xor_sync(kFull, sum[u].w, o);
          }
        }
        if (sub != 0) continue;
#pragma unroll
        for (int u = 0; u < kWeightBatch; ++u) {
          if (vec && at[u] >= 0 && slot[u] + 4 <= len) {
            *reinterpret_cast<float4*>(P.weights + at[u]) =
                make_float4(old[u].x + sum[u].x, old[u].y + sum[u].y, old[u].z + sum[u].z, old[u].w + sum[u].w);
          } else if (t + step * u < piece) {
            const float x[4] = {sum[u].x, sum[u].y, sum[u].z, sum[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (slot[u] + i >= len) continue;
              const int64_t e = place(slot[u] + i);
              if (e >= 0) P.weights[e] += x[i];
            }
          }
        }
      }
    }
    t0 = max(t0, piece);
    first += n;
    ++r;
  }
}

// One warp per (request, query head): its log-sum-exp in log2 units, for the
// weights (their warps are many: each joining the records itself took 5 us
// longer on one request of 128k slots).
__global__ void __launch_bounds__(kFinishThreads) k_paged_lse(const __grid_constant__ PagedParams P) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kFinishWarps + (threadIdx.x >> 5);
  const int r = static_cast<int>(task / P.q_heads), hq = static_cast<int>(task % P.q_heads);
  if (r >= P.n_req) return;
  const Records x = join_records(P, P.first == nullptr ? tile_list(P, lane, false) : TileList{0, 1}, r, lane);
  float M, sum;
  join_stats(P, x, hq, lane, M, sum);
  if (lane == 0) P.lse2[task] = sum == 0.0f ? INFINITY : M + log2f(sum);   // nothing attended: every share 0
}

// The first CTAs add the weights (the longer part); the others join the
// records into the outputs: one CTA per (request, query head) while these are
// few (few requests, each cut into many ranges), else one warp for each.
template <int D>
__global__ void __launch_bounds__(kFinishThreads, 3) k_paged_finish(const __grid_constant__ PagedParams P) {
  __shared__ float s_part[kFinishWarps * D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = static_cast<int>(blockIdx.x) - P.weight_ctas;
  const TileList L = P.first == nullptr || block < 0 ? tile_list(P, lane, false) : TileList{0, 1};
  if (block >= 0) {
    const bool all = P.join_wide != 0;
    const int64_t task = all ? block : static_cast<int64_t>(block) * kFinishWarps + warp;
    const int r = static_cast<int>(task / P.q_heads), hq = static_cast<int>(task % P.q_heads);
    if (r >= P.n_req) return;
    const Records x = join_records(P, L, r, lane);
    if (all) join_output<D, true>(P, x, r, hq, s_part);
    else join_output<D, false>(P, x, r, hq, s_part);
    return;
  }
  const int64_t warps = static_cast<int64_t>(P.weight_ctas) * kFinishWarps;
  const int64_t all = warps / P.weight_heads > 0 ? warps / P.weight_heads : 1;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kFinishWarps + warp; w < all * P.weight_heads; w += warps) {
    const WeightRun run = weight_run(P, L, w, all, lane);
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the scores and log-sum-exps; at once when it has been passed
    add_weights(P, run);
  }
}

// A kernel launched as a programmatic dependent of the one before it.
cudaError_t launch_after(void (*kern)(PagedParams), unsigned grid, const PagedParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFinishThreads);
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
  constexpr int smem = paged_warps(D) * (paged_stages(D) * stage_bytes(D) + score_stage(D, WIDE) * static_cast<int>(sizeof(float)));
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::atomic<uint32_t> done{0};
  const cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  kern<<<grid, 32 * paged_warps(D), smem, s>>>(p);
  return cudaGetLastError();
}

template <bool F32>
cudaError_t launch_latent(const PagedParams& p, int sm_count, cudaStream_t s) {
  auto kern = k_paged_latent<F32>;
  constexpr int smem = sizeof(LatSmem);
  static_assert(kLatCtas * (smem + 1024) <= 228 * 1024, "shared memory");
  static std::atomic<uint32_t> done{0};
  const cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  kern<<<sm_count * kLatCtas, kLatThreads, smem, s>>>(p);
  return cudaGetLastError();
}

// The kernels after the attention: D is the width of an output row.
template <int D>
cudaError_t launch_join(PagedParams p, int sm_count, cudaStream_t s) {
  const int64_t tasks = static_cast<int64_t>(p.n_req) * p.q_heads;
  p.join_wide = tasks <= 2 * sm_count;
  p.weight_ctas = p.weights != nullptr ? kFinishWeightCtas * sm_count : 0;
  const int64_t join_ctas = p.join_wide ? tasks : (tasks + kFinishWarps - 1) / kFinishWarps;
  if (p.weights != nullptr) {
    const cudaError_t e = launch_after(k_paged_lse, static_cast<unsigned>((tasks + kFinishWarps - 1) / kFinishWarps), p, s);
    if (e != cudaSuccess) return e;
  }
  return launch_after(k_paged_finish<D>, static_cast<unsigned>(p.weight_ctas + join_ctas), p, s);
}

template <int D>
cudaError_t launch_d(const PagedParams& p, int sm_count, cudaStream_t s) {
  const int grid = sm_count;   // one CTA per SM: its rings fill shared memory
  cudaError_t e;
  if (p.group > 8) e = p.out_bf16 ? launch_attend_d<D, true, false>(p, grid, s) : launch_attend_d<D, true, true>(p, grid, s);
  else e = p.out_bf16 ? launch_attend_d<D, false, false>(p, grid, s) : launch_attend_d<D, false, true>(p, grid, s);
  return e != cudaSuccess ? e : launch_join<D>(p, sm_count, s);
}

}  // namespace

int paged_ranges_per_sm(int head_dim) { return head_dim == kLatRow ? kLatCtas : paged_warps(head_dim); }

cudaError_t launch_paged(const PagedParams& p, int head_dim, int sm_count, cudaStream_t s) {
  if (head_dim == kLatRow) {
    const cudaError_t e = p.out_bf16 ? launch_latent<false>(p, sm_count, s) : launch_latent<true>(p, sm_count, s);
    return e != cudaSuccess ? e : launch_join<kLatDims>(p, sm_count, s);
  }
  if (head_dim == 64) return launch_d<64>(p, sm_count, s);
  if (head_dim == 128) return launch_d<128>(p, sm_count, s);
  return launch_d<256>(p, sm_count, s);
}

}  // namespace pic
