// Attention of many query rows over the paged cache on the fifth-generation
// tensor cores (tcgen05 with TMEM accumulators, TMA tensor copies), sm_103a:
// prompts, chunked prompts, the tokens recomputed after a stitch, and all
// requests' queries over the prefix they share.
//
//   s_it = scale * q_i . k_t where row i sees slot t (else -inf),
//   out_i = sum_t p_it v_t,  p_i = softmax(s_i),  lse_i = log sum_t exp(s_it).
//
// Rows are (token, query head) pairs of one request and KV head, in the order of
// tokens; a CTA takes 256 of them (two tiles of 128) or 128 (one: heads of 256 dims, and
// calls of few rows, see tile_shape_of in pic_serve.cpp) and walks the slots that some of them see, 128 (64) at a time: from the lowest window's
// start to the highest slot, then the first n_first.  One pass, with a running maximum and
// sum.  Where there are too few row blocks for the SMs, a block's slots are
// dealt to several CTAs, which leave records (O, max, sum) that a later kernel joins.
//
// Warps by role, per step of K and V tiles in a shared ring:
//   * two producer warps look up the blocks of the step's slots and
//     copy them with TMA, a whole block of all dims at a time: the cache is mapped as
//     [head][8-row group][64-dim plane][8 rows][64 dims], so that a copy lands as rows of 128
//     swizzled bytes in groups of 8, whichever blocks follow each other.  (A block size that is
//     no multiple of 8 goes by 4, 2 or 1 rows and one plane at a time.)
//   * a warp per tile issues its products: S = Q K^T, M = 128 rows, N = slots, and
//     O += P V with P read from TMEM and V as an MN-major operand;
//   * eight warps per tile, two threads per row: read S from TMEM, mask, raise the
//     maximum when a score passes it by more than 2^8 (O and the sum are then rescaled, which
//     after the first steps hardly happens), write P = exp2(s - m) as bf16 over S, in one part
//     or in two.
// Two tiles take turns: while one is in its softmax, the tensor cores work on the other's.
// (One tile: the next step's S is made ahead.  At 256 dims O alone takes half of TMEM.)
//
// P is rounded to bf16 (2^-8 of each weight, where the output's own rounding is 2^-8 of
// their sum), unnormalised: between 2^-8 and 2^8 at the maximum.  So it is for the tokens of
// requests.  Over a shared prefix (PARTS = 2) P keeps 16 bits, as in the row-by-row kernel that
// attends to the rest of the same rows: what the rounding leaves, a second bf16 part, fills the
// other half of S's columns and is multiplied with the same rows of V, half as many products
// again.  Measured: a prefix of 32k slots beside 1-2,048 of their own for 64 requests 93 us a
// call with one part, 98 with two, 256 requests over 2,003 slots 125 and 128; but a prompt of 8,192
// tokens in a window of 4,096, which the products bound, 307 with one, 405 with two (errors against 64
// bits 2.2e-3 and 1.6e-3, the latter the output's own rounding), so tokens have one.
// Sums, maxima and O are fp32.  Masked scores are replaced, so what K holds there does not matter; V's
// rows that no row of the CTA sees are zeroed in shared memory before the product.
//
// Bound by the chain of a step (products, scores read, maximum, exponentials, P seen by the
// issuing warp), about 2,900 cycles for both tiles where the products alone are 2,060, and by 6 us in which a CTA
// starts and ends (one tile 5).  256 rows, since two tiles are what registers, TMEM and shared memory hold and one would leave the
// tensor cores idle during its softmax; steps of 128 slots, since S of both tiles and O fill TMEM.
// Measured (GB300, 32 query over 8 KV heads of 128 dims, blocks of 16): a prompt of 8,192
// tokens in a window of 4,096, 291 us (1.42 PFLOP/s of visible pairs); of 4,096, all visible, 103 (1.33); heads of 64 dims
// 86 (0.80), of 256 104 (1.32); the recomputed heads of 4 requests of 16k slots, 164 us.
// Every wait is bounded: one that runs out raises PIC_DEV_TIMEOUT, tells the other
// roles to stop, and the CTA frees its TMEM before it leaves.
#include <cfloat>

#include <cuda_bf16.h>

#include "pic_decode.h"
#include "pic_device.cuh"
#include "pic_paged.cuh"
#include "pic_tc.cuh"

namespace pic {
namespace {

using namespace dev;

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLazy = 8.0f;   // log2 units a maximum may be passed by before O is rescaled
constexpr int kProducers = 2;
constexpr uint32_t kTmemCols = 512, kOCol = 256;

template <int D, int TILES>
struct Cfg {
  static constexpr int NQ = TILES;                     // tiles of rows
  static constexpr int BN = tile_slots(D);             // slots of a step
  static constexpr int PL = D / 64;                    // 64-dim planes
  static constexpr int kStage = BN * D * 2;            // K or V of a step
  static constexpr int kStages = D == 64 ? 8 : (D == 128 && NQ == 1 ? 6 : 5);
  static constexpr int kQTile = kTileRows * D * 2;
  // Warps 0 and 1 issue the products, one for each tile: a wait, even for what has happened, and an
  // issue each take their time, and one warp could not keep the tensor cores busy (382 us
  // for a prompt of 8,192 tokens in a window of 4,096).  As the oldest of their schedulers they are not kept
  // waiting by the softmax warps' arithmetic either (398 as the youngest).
  static constexpr int kProducer0 = 2;
  static constexpr int kSoftmax0 = kProducer0 + kProducers;   // a multiple of 4: warp w reads TMEM lanes 32 (w % 4) ..
  static constexpr int kSoftmaxWarps = 8 * NQ;
  static constexpr int kThreads = 32 * (kSoftmax0 + kSoftmaxWarps);   // 640 (384): 96 (168) registers a thread
  static_assert(kSoftmax0 % 4 == 0, "TMEM lane quadrants");
  // shared memory, from a 1024-byte aligned base
  static constexpr int kRing = NQ * kQTile;
  static constexpr int kBars = kRing + kStages * kStage;
  // full[kStages] empty[kStages] s_full[2] p_full[2] o_full[2] pv_done done[2] q_full[2] turn[2]
  static constexpr int kNumBars = 2 * kStages + 13;
  static constexpr int kTop = kBars + kNumBars * 8;             // float [rows]: a row's maximum, between its two threads
  static constexpr int kMisc = kTop + 4 * NQ * kTileRows;       // TMEM slot, abort flag, int [2][warps]
  static constexpr int kTotal = kMisc + 16 + 2 * 4 * (kThreads / 32);
  static constexpr int kAlloc = kTotal + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  static_assert(NQ * D + kOCol <= kTmemCols && 2 * BN <= static_cast<int>(kOCol), "TMEM columns");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two fp32 operations at once.  (Written out: through the header's float2 functions a step's
// exponentials took 646 cycles a warp where these take 431.)
__device__ __forceinline__ uint64_t pair64(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t r) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// (x, y) as a bf16 pair, x in the low half
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// a box of 8-row groups of all planes, and one of rows of one plane
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int group, int head, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(head), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// Joins the softmax warps (PER threads a tile), at named barrier 15: whether any thread's flag is set.
template <int PER>
__device__ __forceinline__ bool softmax_any(int tiles, bool flag) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.or.pred q, 15, %1, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(PER * tiles), "r"(flag ? 1u : 0u)
      : "memory");
  return r != 0;
}

// Joins the two warps that share rows, at named barrier `id`: whether any thread's flag is set.
__device__ __forceinline__ bool pair_any(uint32_t id, bool flag) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(flag ? 1u : 0u)
      : "memory");
  return r != 0;
}

// the low n bits of a word (n anything)
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? kFull : (1u << n) - 1u); }

// The rows of a CTA.
struct Work {
  int table;      // row of the block tables
  int token0;     // first token of its request
  int n_rows;     // rows of its request (one KV head)
  int row0;       // first of the CTA's
};
// What a step covers, and what the rows of the CTA see.
struct Slots {
  int lo, hi;          // slots lo .. hi of some window (hi < lo: nothing is seen)
  int n_first;         // slots below are seen by every row behind them
  // steps over the window, and after them over the first slots where those are apart
  // (the few scores of the first would be a poor first maximum)
  int base;            // first slot of the window's steps
  int steps_w, steps;
  int whole_lo, whole_hi;   // a step that begins between these is seen whole by every row
  __device__ __forceinline__ int next_slot(int t, int j, int bn) const { return j == steps_w ? 0 : t + bn; }
  __device__ __forceinline__ int first_slot(int j, int bn) const { return j < steps_w ? base + j * bn : (j - steps_w) * bn; }
  __device__ __forceinline__ bool some(int a, int b) const {   // whether any of slots [a, b) is seen by a row
    return a <= hi && (b > lo || a < n_first);
  }
  __device__ __forceinline__ bool seen(int t) const { return t <= hi && (t >= lo || t < n_first); }
  __device__ __forceinline__ bool all_seen(int a, int b) const {   // whether some row sees each of [a, b)
    return b - 1 <= hi && (a >= lo || b <= n_first || n_first >= lo);
  }
};

// Finds row block `index` of one KV head, the last of the last request first (the
// longest of a prompt, so that the short ones fill the gaps at the end); warp-wide.
template <int RC>
__device__ __forceinline__ bool find_rows(const TileParams& P, int64_t index, int lane, Work& w) {
  if (P.indptr == nullptr) {
    const int n = P.n_tokens * P.group, blocks = (n + RC - 1) / RC;
    if (index >= blocks) return false;
    w = Work{0, 0, n, static_cast<int>(blocks - 1 - index) * RC};
    return true;
  }
  int64_t base = 0;
  for (int i0 = 0; i0 < P.n_req; i0 += 32) {
    const int r = P.n_req - 1 - (i0 + lane);
    int begin = 0, rows = 0;
    if (r >= 0) {
      begin = min(max(__ldg(P.indptr + r), 0), P.n_tokens);
      const int count = min(max(__ldg(P.indptr + r + 1), begin), P.n_tokens) - begin;
      rows = count >= P.least ? count * P.group : 0;
    }
    const int blocks = (rows + RC - 1) / RC;
    int64_t incl = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned hit = __ballot_sync(kFull, base + incl > index);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      const int k = static_cast<int>(index - base - __shfl_sync(kFull, incl - blocks, src));
      w.table = P.n_req - 1 - (i0 + src);
      w.token0 = __shfl_sync(kFull, begin, src);
      w.n_rows = __shfl_sync(kFull, rows, src);
      w.row0 = (__shfl_sync(kFull, blocks, src) - 1 - k) * RC;
      return true;
    }
    base += __shfl_sync(kFull, incl, 31);
  }
  return false;
}

// Slot of a token's row, -1: it sees nothing.
__device__ __forceinline__ int row_slot(const TileParams& P, int token, bool raise) {
  if (P.indptr == nullptr) {
    int len = __ldg(P.lens + token), prefix = __ldg(P.prefix_len);
    // (lengths and prefix are raised by the kernel that reads the requests' own slots)
    if (len < 0 || len > P.max_len) len = 0;
    if (prefix < 0 || prefix > P.capacity) prefix = 0;
    return min(len, prefix) - 1;
  }
  const int s = __ldg(P.slot + token);
  if (s >= P.capacity) {
    if (raise) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_BAD_LENGTH));
    return -1;
  }
  return s < 0 ? -1 : s;
}

template <int D, int TILES, bool WIDE_BOX, int PARTS>
__global__ void __launch_bounds__(Cfg<D, TILES>::kThreads, 1) k_attend_tile(const __grid_constant__ TileParams P,
                                                                     const __grid_constant__ TileMaps maps) {
  using C = Cfg<D, TILES>;
  constexpr int NQ = C::NQ, BN = C::BN, PL = C::PL, RC = NQ * kTileRows;
  constexpr uint32_t kIdS = idesc(128, BN, 0), kIdPV = idesc(128, D, 0, 1);
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base_u32 = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t* full = bars;                        // a stage's rows landed
  uint64_t* empty = full + C::kStages;          // the products that read it finished
  uint64_t* s_full = empty + C::kStages;        // S is made (by buffer, as below)
  uint64_t* p_full = s_full + 2;                // P is written
  uint64_t* o_full = p_full + 2;                // a tile's O is complete
  uint64_t* pv_done = o_full + 2;               // (256 dims) a step's value product finished
  uint64_t* done = pv_done + 1;                 // an issuer's products all finished
  uint64_t* q_full = done + 2;                  // a tile's queries are in place
  uint64_t* turn = q_full + 2;                    // a tile's products of a step may be issued
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);
  int* s_range = reinterpret_cast<int*>(smem + C::kMisc + 16);   // [2][warps]

  // (the warp's number from one lane, and the range below from reductions: what is known to be the same in all lanes
  // is kept beside their 96 registers, which a step's scores need; 303 us for a prompt of 8,192 tokens else, 291 so)
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  const uint32_t unit = blockIdx.x / static_cast<uint32_t>(P.splits);
  const int split = static_cast<int>(blockIdx.x - unit * P.splits);
  const int hk = static_cast<int>(unit % static_cast<uint32_t>(P.kv_heads));
  if (P.indptr != nullptr && blockIdx.x == 0 && warp == 0) {   // offsets that are not non-decreasing inside [0, n_tokens]
    bool bad = false;
    for (int r = lane; r <= P.n_req; r += 32) {
      const int at = __ldg(P.indptr + r), before = r > 0 ? __ldg(P.indptr + r - 1) : 0;
      bad |= at < before || at > P.n_tokens;
    }
    if (bad) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_BAD_LENGTH));
  }
  Work w{};
  if (!find_rows<RC>(P, unit / static_cast<uint32_t>(P.kv_heads), lane, w)) return;   // the same in every warp

  const int tiles = NQ == 2 && w.row0 + kTileRows >= w.n_rows ? 1 : NQ;   // tiles with rows

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], kProducers);   // each warp announces its own copies
      mbar_init(&empty[i], tiles);           // each tile's products have read it
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(pv_done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&done[i], 1);
      mbar_init(&q_full[i], 8);
      mbar_init(&turn[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (tid < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tid == 0 ? &maps.k : &maps.v)) : "memory");
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // this thread's row (softmax warps)
  const int my_tile = (warp - C::kSoftmax0) >> 3, my_half = ((warp - C::kSoftmax0) >> 2) & 1;
  const int my_row = w.row0 + my_tile * kTileRows + 32 * (warp & 3) + lane;
  const bool has_row = warp >= C::kSoftmax0 && my_row < w.n_rows;
  const int my_token = w.token0 + (has_row ? my_row / P.group : 0);
  const int my_head = hk * P.group + (has_row ? my_row % P.group : 0);
  const int my_slot = has_row ? row_slot(P, my_token, hk == 0 && split == 0) : -1;
  if (warp >= C::kSoftmax0 && my_tile < tiles) {
    // The queries of the warp's rows (16 of a quadrant's 32 each), as rows of 128 swizzled bytes, one 64-dim
    // plane after the other; asked for once the slots are known, which the first copies of K wait for.  Lanes share rows here and where results leave (a row a
    // lane is 32 lines an instruction: it took 6,000 cycles).
    constexpr int CH = D / 8, RW = 32 / CH;   // chunks of a row, rows of an instruction
    const int64_t mine = has_row ? my_token * P.q_stride + static_cast<int64_t>(my_head) * D * 2 : -1;
    const int c = lane % CH, sub = lane / CH;
    const uint32_t to = base_u32 + my_tile * C::kQTile + (c >> 3) * (kTileRows * 128);
#pragma unroll 8
    for (int r0 = 16 * my_half; r0 < 16 * my_half + 16; r0 += RW) {
      const int64_t from = __shfl_sync(kFull, mine, r0 + sub);
      const int r = 32 * (warp & 3) + r0 + sub;
      cp_async16_zfill(to + r * 128 + (((c & 7) ^ (r & 7)) << 4), P.q + (from >= 0 ? from : 0) + c * 16, from >= 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  {
    const int lo = __reduce_min_sync(kFull, my_slot >= 0 ? my_slot : INT32_MAX), hi = __reduce_max_sync(kFull, my_slot);
    if (lane == 0) {
      s_range[warp] = lo;
      s_range[C::kThreads / 32 + warp] = hi;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  Slots S;
  {
    const bool one = lane >= C::kSoftmax0 && lane < C::kThreads / 32;
    const int lo = __reduce_min_sync(kFull, one ? s_range[lane] : INT32_MAX);
    const int hi = __reduce_max_sync(kFull, one ? s_range[C::kThreads / 32 + lane] : -1);
    S.hi = hi;
    S.lo = P.window > 0 && hi >= 0 ? max(0, lo + 1 - P.window) : 0;
    S.n_first = min(P.n_first, S.lo);
    // the first slots apart from the window, where steps over them end before it
    const int steps_a = (S.n_first + BN - 1) / BN;
    const int lo_box = S.lo & -P.box;   // boxes are powers of two
    const bool apart = S.n_first > 0 && static_cast<int64_t>(steps_a) * BN < lo_box;
    S.base = apart || S.n_first == 0 ? lo_box : 0;
    S.steps_w = hi < 0 ? 0 : (hi - S.base) / BN + 1;
    S.steps = S.steps_w + (apart ? steps_a : 0);
    S.whole_lo = P.window > 0 ? max(0, hi + 1 - P.window) : 0;
    S.whole_hi = lo == INT32_MAX ? -1 : lo + 1 - BN;
  }
  // this CTA's part of the steps
  int j_begin = 0, n = S.steps;
  if (P.splits > 1) {
    const int each = S.steps / P.splits, rest = S.steps - each * P.splits;
    j_begin = each * split + min(split, rest);
    n = each + (split < rest ? 1 : 0);
  }
  auto fail = [&]() {
    atomicOr(P.status, kDevTimeout);
    *abort_flag = 1;
  };

  if (warp >= C::kProducer0 && warp < C::kSoftmax0 && n > 0) {
    // -------------------------------------------------------------- producers
    const int prod = warp - C::kProducer0;
    const int32_t* table = P.paged.tables + static_cast<int64_t>(w.table) * P.paged.max_blocks;
    const int boxes = BN / P.box;
    const int copies = WIDE_BOX ? boxes : boxes * PL;   // of K, and of V, dealt to the warps
    const uint32_t bytes = P.box * (WIDE_BOX ? D : 64) * 2;
    const uint32_t my_bytes = ((copies + kProducers - 1 - prod) / kProducers) * bytes;
    // Block of a slot whose box (slots [first, last)) some row sees, else -1; looked at only when its copy is
    // issued, as a warp stops where it touches a load that has not arrived.
    auto block_at = [&](int slot, int first, int last) { return S.some(first, last) ? __ldg(table + block_of(P.paged, slot)) : -1; };
    // cache row of a slot in that block, cache_rows: nothing is read (nobody sees it, or its block is bad)
    auto row_in = [&](int32_t block, int slot) -> int {
      if (block < 0 || block >= P.paged.num_cache_blocks) return P.cache_rows;
      return block * P.paged.block_size + (slot - block_of(P.paged, slot) * P.paged.block_size);
    };
    const int c0 = kProducers * lane + prod;   // this lane's first copy
    auto copy_slot = [&](int i, int c) { return S.first_slot(j_begin + i, BN) + (WIDE_BOX ? c : c / PL) * P.box; };
    auto copy_block = [&](int i, int c) {
      const int t = copy_slot(i, c);
      return block_at(t, t, t + P.box);
    };
    bool ok = true;
    int issued = 0, st = 0;
    uint32_t round = 0;   // parity of the ring's round
    int32_t next = c0 < copies ? copy_block(0, c0) : -1;
    for (int i = 0; i < n; ++i) {
      const int32_t block0 = next;
#pragma unroll
      for (int x = 0; x < 2; ++x) {   // K, then V
        const int fill = 2 * i + x;
        if (fill >= C::kStages) ok = wait_or_abort(&empty[st], round ^ 1, abort_flag, kMaxSpins);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], my_bytes);
        __syncwarp();
        const CUtensorMap* map = x == 0 ? &maps.k : &maps.v;
        const uint32_t dst = base_u32 + C::kRing + st * C::kStage;
        for (int c = c0; c < copies; c += 32 * kProducers) {
          const int row = row_in(c == c0 ? block0 : copy_block(i, c), copy_slot(i, c));
          if constexpr (WIDE_BOX) {
            tma_load_5d(dst + c * bytes, map, row >> 3, hk, &full[st]);
          } else {
            const int box = c / PL, plane = c - box * PL, at = box * P.box;
            tma_load_3d(dst + (at >> 3) * (PL * 1024) + plane * 1024 + (at & 7) * 128, map, 64 * plane, hk, row, &full[st]);
          }
        }
        issued = fill + 1;
        if (++st == C::kStages) {
          st = 0;
          round ^= 1;
        }
      }
      if (!ok) {
        if (lane == 0) fail();
        break;
      }
      if (i + 1 < n && c0 < copies) next = copy_block(i + 1, c0);
    }
    if (!ok && lane == 0) {
      // wait (bounded) for the copies in flight
      for (int fill = max(0, issued - C::kStages); fill < issued; ++fill)
        mbar_wait_bounded(&full[fill % C::kStages], (fill / C::kStages) & 1, 1024);
    }
  } else if (warp < tiles && n > 0) {
    // --------------------------------------------------------------- products
    const int q = warp;
    // Descriptors are stepped in their low words (addresses in 16 bytes, which stay below
    // 2^14): the high words are constants.
    const auto desc = [](uint32_t lo, uint64_t like) {
      uint64_t d;
      asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(static_cast<uint32_t>(like >> 32)));
      return d;
    };
    constexpr uint32_t kStep = C::kStage >> 4;
    const uint64_t dq = sdesc(base_u32, 16, 1024), dk = sdesc(base_u32 + C::kRing, 16, PL * 1024),
                   dv = sdesc(base_u32 + C::kRing, 1024, PL * 1024);
    bool ok = true;
    auto ready = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(kFull, wait_or_abort(bar, parity, abort_flag, kMaxSpins));
      return ok;
    };
    // a place in the ring
    struct Ring {
      uint32_t stage, parity;
      __device__ __forceinline__ void next() {   // two fills on: K to K, V to V
        stage += 2;
        if (stage >= C::kStages) {
          stage -= C::kStages;
          parity ^= 1;
        }
      }
    };
    auto score = [&](int buf, uint32_t stage) {   // S = Q K^T
      const uint32_t a = static_cast<uint32_t>(dq) + q * (C::kQTile >> 4), b = static_cast<uint32_t>(dk) + stage * kStep;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        tc_mma_elect(tmem + buf * BN, desc(a + (((ks >> 2) * (kTileRows * 128) + (ks & 3) * 32) >> 4), dq),
                     desc(b + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), dk), kIdS, ks > 0);
      tc_commit_elect(&s_full[buf]);
    };
    auto value = [&](int buf, uint32_t stage, bool first) {   // O += P V (both parts of P over the same rows of V)
      const uint32_t b = static_cast<uint32_t>(dv) + stage * kStep;
#pragma unroll
      for (int ks = 0; ks < BN / 16; ++ks) {
        const uint64_t v = desc(b + ((ks * 2 * PL * 1024) >> 4), dv);
        tc_mma_tmem_a_elect(tmem + kOCol + q * D, tmem + buf * BN + 8 * ks, v, kIdPV, !first || ks > 0);
        if constexpr (PARTS == 2) tc_mma_tmem_a_elect(tmem + kOCol + q * D, tmem + buf * BN + BN / 2 + 8 * ks, v, kIdPV, true);
      }
    };
    // V of step i has landed, and its rows that no row of the CTA sees are zeros (both tiles'
    // warps write the same)
    auto wait_v = [&](int t0, const Ring& r) {
      if (!ready(&full[r.stage], r.parity)) return false;
      if (!S.all_seen(t0, t0 + BN)) {
        uint8_t* v = smem + C::kRing + r.stage * C::kStage;
        for (int x = lane; x < BN * PL * 8; x += 32) {
          const int row = x / (PL * 8), part = x % (PL * 8);
          if (!S.seen(t0 + row))
            *reinterpret_cast<uint4*>(v + (row >> 3) * (PL * 1024) + (part >> 3) * 1024 + (row & 7) * 128 + (part & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      return true;
    };
    int t0 = S.first_slot(j_begin, BN);
    Ring rk{0, 0}, rv{1, 0};   // of K of the step whose scores come next, of V of the current step
    if (ready(&q_full[q], 0) && ready(&full[0], 0)) {
      tc_fence_after();
      score(NQ == 2 ? q : 0, 0);
      tc_commit_elect(&empty[0]);
      rk.next();
      for (int i = 0; i < n; ++i) {
        const bool more = i + 1 < n;
        const int buf = NQ == 2 ? q : i & 1;
        const uint32_t parity = (NQ == 2 ? i : i >> 1) & 1;
        // (what has landed long ago is looked at before what is waited for)
        if (!wait_v(t0, rv) || (more && !ready(&full[rk.stage], rk.parity))) break;
        if (NQ == 1 && more) {
          tc_fence_after();
          score((i + 1) & 1, rk.stage);
          tc_commit_elect(&empty[rk.stage]);
        }
        // The tiles take turns, so that one's products run during the other's softmax (each going its own
        // way, both were soon in step, and both units idle half of the time: 394 us).
        if (tiles == 2 && (q == 1 || i > 0) && !ready(&turn[q], (q == 1 ? i : i - 1) & 1)) break;
        if (!ready(&p_full[buf], parity)) break;
        tc_fence_after();
        value(buf, rv.stage, i == 0);
        if (NQ == 2 && more) score(buf, rk.stage);
        if (tiles == 2 && lane == 0) mbar_arrive(&turn[q ^ 1]);
        if (NQ == 2 && more) tc_commit_elect(&empty[rk.stage]);
        tc_commit_elect(&empty[rv.stage]);
        if (NQ == 1) tc_commit_elect(pv_done);
        if (!more) tc_commit_elect(&o_full[q]);
        rk.next();
        rv.next();
        t0 = S.next_slot(t0, j_begin + i + 1, BN);
      }
    }
    if (!ok && lane == 0) fail();
    tc_commit_elect(&done[q]);
    mbar_wait_bounded(&done[q], 0);
  } else if (warp >= C::kSoftmax0 && my_tile < tiles) {
    // ---------------------------------------------------------------- softmax
    const int q = my_tile;
    const int at = has_row ? my_token * P.q_heads + my_head : -1;   // row of the outputs, below 2^30
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (n > 0) {
      if (P.sign <= 0) {   // queries of a negative scale enter negated, of scale 0 as zeros
        __syncwarp();
        for (int r0 = 16 * my_half; r0 < 16 * my_half + 16; ++r0) {
          const int r = 32 * (warp & 3) + r0;
          for (int c = lane; c < D / 8; c += 32) {
            uint4* x = reinterpret_cast<uint4*>(smem + q * C::kQTile + (c >> 3) * (kTileRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            uint4 v = *x;
#pragma unroll
            for (int e = 0; e < 4; ++e) word(v, e) = P.sign < 0 ? word(v, e) ^ 0x80008000u : 0u;
            *x = v;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[q]);
    }
    // Two threads share a row, with half of a step's slots each.  They hold the row's maximum alike, and meet once a
    // step to learn whether either must raise it.
    constexpr int HN = BN / 2, HW = HN / 32;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t o_at = tl + kOCol + q * D;
    const uint32_t pair = 1 + 4 * q + (warp & 3);   // named barrier of the two warps
    float* s_top = reinterpret_cast<float*>(smem + C::kTop) + q * kTileRows + 32 * (warp & 3) + lane;
    const float scale = P.scale_log2;
    // Blocks outside the cache among those that some row sees: looked for once, all softmax warps together,
    // so that steps need not ask (where there are any, each step does).
    const int32_t* table = P.paged.tables + static_cast<int64_t>(w.table) * P.paged.max_blocks;
    bool bad = false;
    {
      const int bs = P.paged.block_size, x0 = (warp - C::kSoftmax0) * 32 + lane, stride = 256 * tiles;
      for (int part = 0; part < 2; ++part) {
        // the CTA's steps over the window, then those over the first slots
        const int ja = part == 0 ? j_begin : max(j_begin, S.steps_w), jb = part == 0 ? min(j_begin + n, S.steps_w) : j_begin + n;
        if (ja >= jb) continue;
        const int t = S.first_slot(ja, BN);
        const int end = part == 0 ? min(S.hi + 1, t + (jb - ja) * BN) : min(S.n_first, t + (jb - ja) * BN);
        const int b0 = block_of(P.paged, t), b1 = end > t ? block_of(P.paged, end - 1) : b0 - 1;
        for (int b = b0 + x0; b <= b1; b += stride) {
          if (!S.some(b * bs, b * bs + min(bs, S.hi + 1 - b * bs))) continue;   // (b * bs <= hi: no overflow)
          const int32_t block = __ldg(table + b);
          if (block < 0 || block >= P.paged.num_cache_blocks) {
            raise_block(P.status, P.indptr == nullptr ? kPrefixTable : w.table, b * bs);
            bad = true;
          }
        }
      }
      bad = softmax_any<32 * 8>(tiles, bad);
    }
    float m_run = -FLT_MAX, l_run = 0.0f;
    bool ok = true;
    int t0 = S.first_slot(j_begin, BN);
    for (int i = 0; i < n; ++i) {
      const int buf = NQ == 2 ? q : i & 1;
      const uint32_t parity = (NQ == 2 ? i : i >> 1) & 1;
      // what this row sees of the step, before its scores are there
      const bool masked = bad || t0 < S.whole_lo || t0 > S.whole_hi;
      uint32_t mask[HW];
      if (masked) {
        // slots t <= my_slot that are in the window or among the first, in blocks of the cache
        const int my_lo = P.window > 0 ? max(0, my_slot + 1 - P.window) : 0;   // its window's first
#pragma unroll
        for (int x = 0; x < HW; ++x) {
          const int t = t0 + 32 * (my_half * HW + x);
          mask[x] = low_bits(my_slot + 1 - t) & (~low_bits(my_lo - t) | low_bits(P.n_first - t));
          if (bad) {
            const int32_t block = S.seen(t + lane) ? __ldg(table + block_of(P.paged, t + lane)) : 0;
            mask[x] &= __ballot_sync(kFull, block >= 0 && block < P.paged.num_cache_blocks);
          }
        }
      }
      ok = __all_sync(kFull, ok && wait_or_abort(&s_full[buf], parity, abort_flag, kMaxSpins));
      // (a wait that ran out in one warp of a pair ends both, where they meet)
      tc_fence_after();
      const uint32_t s_at = tl + buf * BN + my_half * HN;
      float s[HN];
#pragma unroll
      for (int c = 0; c < HN; c += 32) tmem_ld32(s_at + c, s + c);
      tmem_wait_ld();
      if (masked) {
#pragma unroll
        for (int x = 0; x < HN; ++x) s[x] = (mask[x / 32] >> (x & 31)) & 1u ? s[x] : -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int x = 4; x < HN - 4; x += 8) {
#pragma unroll
        for (int y = 0; y < 4; ++y) mx[y] = max3(mx[y], s[x + 2 * y], s[x + 2 * y + 1]);
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) mx[y] = fmaxf(mx[y], s[HN - 4 + y]);
      const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * scale;
      if (pair_any(pair, !ok || i == 0 || top > m_run + kLazy)) {
        // the second half's maximum goes to the first, which decides
        if (my_half == 1) *s_top = ok ? top : INFINITY;
        pair_any(pair, false);
        if (my_half == 0) {
          const float both = fmaxf(top, *s_top);
          *s_top = i == 0 ? fmaxf(both, -FLT_MAX) : (both > m_run + kLazy ? both : m_run);
        }
        if (pair_any(pair, !ok)) {
          ok = false;
          break;
        }
        const float m_new = *s_top;
        const float alpha = ex2(m_run - m_new);
        m_run = m_new;
        l_run *= alpha;
        if (i > 0) {
          if (NQ == 1) {
            ok = __all_sync(kFull, wait_or_abort(pv_done, (i - 1) & 1, abort_flag, kMaxSpins));
            tc_fence_after();
          }
#pragma unroll 1
          for (int c = my_half * (D / 2); c < (my_half + 1) * (D / 2); c += 16) {
            float o[16];
            tmem_ld16(o_at + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] *= alpha;
            tmem_st16(o_at + c, o);
          }
        }
      }
      const uint64_t sc = pair64(scale, scale), neg = pair64(-m_run, -m_run);
      uint64_t part[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < HN; c += 32) {
        uint32_t p[16], rest[PARTS == 2 ? 16 : 1];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 y = unpair(fma2(pair64(s[c + 2 * e], s[c + 2 * e + 1]), sc, neg));
          y.x = ex2(y.x);
          y.y = ex2(y.y);
          part[e & 1] = add2(part[e & 1], pair64(y.x, y.y));
          p[e] = pack2(y.x, y.y);
          if constexpr (PARTS == 2) rest[e] = pack2(y.x - bf_lo(p[e]), y.y - bf_hi(p[e]));   // (exact differences)
        }
        // (over scores that both threads of the row have read)
        tmem_st16u(tl + buf * BN + (my_half * HN + c) / 2, p);
        if constexpr (PARTS == 2) tmem_st16u(tl + buf * BN + BN / 2 + (my_half * HN + c) / 2, rest);
      }
      const float2 sum = unpair(add2(part[0], part[1]));
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[buf]);
      l_run += sum.x + sum.y;
      t0 = S.next_slot(t0, j_begin + i + 1, BN);
    }
    if (!ok && lane == 0) fail();
    // ---- the output, or this part's record
    const bool direct = P.rec_acc == nullptr;
    if (n > 0 && ok) {
      ok = __all_sync(kFull, wait_or_abort(&o_full[q], 0, abort_flag, kMaxSpins));
      if (!ok && lane == 0) fail();
      tc_fence_after();
    }
    // 4 KB of the queries' memory for each warp (64 dims: each pair), of which every product has been made
    uint8_t* stage = smem + q * C::kQTile + (D == 64 ? (warp & 3) * 4096 : ((warp & 3) * 2 + my_half) * 4096);
    ok = !pair_any(pair, !ok);
    {
      // the row's sum: both halves'
      float* x = reinterpret_cast<float*>(smem + q * C::kQTile + (warp & 3) * (D == 64 ? 4096 : 8192));
      x[32 * my_half + lane] = l_run;
      pair_any(pair, false);
      l_run = x[lane] + x[32 + lane];
      if (my_slot < 0) l_run = 0.0f;   // a row that sees nothing
      pair_any(pair, false);
    }
    if (ok) {
      // 128 bytes of each of the warp's rows at a time
      const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
      uint8_t* out = direct ? static_cast<uint8_t*>(P.out)
                            : reinterpret_cast<uint8_t*>(P.rec_acc + static_cast<int64_t>(split) * P.n_tokens * P.q_heads * D);
      const int64_t pitch = D * (direct ? 2 : 4);
      const int mine = direct || l_run != 0.0f ? at : -1;   // nothing is kept beside a sum of 0
      const int width = direct ? 64 : 32, halves = D == 64 ? 1 : 2;
      const auto send = [&](int c) {
        __syncwarp();
        uint4 y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = 4 * k + (lane >> 3);
          y[k] = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = __shfl_sync(kFull, mine, 4 * k + (lane >> 3));
          if (row >= 0) *reinterpret_cast<uint4*>(out + row * pitch + c * (direct ? 2 : 4) + (lane & 7) * 16) = y[k];
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int c = my_half < halves ? my_half * width : D; c < D; c += halves * width) {
        float o[32];
        if (direct) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (n > 0) {
              tmem_ld32(o_at + c + 32 * h, o);
              tmem_wait_ld();
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint4 y = make_uint4(0, 0, 0, 0);
              if (l_run != 0.0f) {
#pragma unroll
                for (int e = 0; e < 4; ++e) word(y, e) = pack2(o[8 * x + 2 * e] * inv, o[8 * x + 2 * e + 1] * inv);
              }
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * h + x) ^ (lane & 7)) << 4)) = y;
            }
          }
        } else {
          if (n > 0) {
            tmem_ld32(o_at + c, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int x = 0; x < 8; ++x)
            *reinterpret_cast<float4*>(stage + lane * 128 + ((x ^ (lane & 7)) << 4)) =
                make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
        send(c);
      }
      if (at >= 0 && my_half == 0) {
        if (!direct) P.rec_ml[static_cast<int64_t>(split) * P.n_tokens * P.q_heads + at] = make_float2(l_run == 0.0f ? -FLT_MAX : m_run, l_run);
        else if (P.lse != nullptr) P.lse[at] = l_run == 0.0f ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// One warp per (token, query head): joins the parts of a row's slots.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_tile_join(const __grid_constant__ TileParams P) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int64_t rows = static_cast<int64_t>(P.n_tokens) * P.q_heads;
  if (task < rows) {
    // rows of the requests that the tiles took
    const int token = static_cast<int>(task / P.q_heads);
    bool mine = token >= __ldg(P.indptr) && token < __ldg(P.indptr + P.n_req);
    if (mine) {
      int lo = 0, hi = P.n_req;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(P.indptr + mid) <= token) lo = mid;
        else hi = mid;
      }
      mine = __ldg(P.indptr + lo + 1) - __ldg(P.indptr + lo) >= P.least;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (mine) {
      float m = -FLT_MAX, sum = 0.0f, acc[V];
      for (int k = lane; k < P.splits; k += 32) m = fmaxf(m, __ldcg(P.rec_ml + k * rows + task).x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
#pragma unroll
      for (int x = 0; x < V; ++x) acc[x] = 0.0f;
#pragma unroll 4
      for (int k = 0; k < P.splits; ++k) {
        const float2 ml = __ldcg(P.rec_ml + k * rows + task);
        if (ml.y == 0.0f) continue;   // nothing was written beside it
        const float e = ex2(ml.x - m);
        sum += ml.y * e;
        const float* a = P.rec_acc + (k * rows + task) * D + lane * V;
#pragma unroll
        for (int x = 0; x < V; x += 2) {
          const float2 y = __ldcg(reinterpret_cast<const float2*>(a + x));
          acc[x] += e * y.x;
          acc[x + 1] += e * y.y;
        }
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(P.out) + task * D + lane * V);
#pragma unroll
      for (int x = 0; x < V; x += 2) to[x / 2] = bf_pack(acc[x] * inv, acc[x + 1] * inv);
      if (P.lse != nullptr && lane == 0) P.lse[task] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
    }
  }
}

template <int D, int TILES, bool WIDE_BOX, int PARTS>
cudaError_t launch_box(const TileParams& p, const TileMaps& maps, cudaStream_t s) {
  auto kern = k_attend_tile<D, TILES, WIDE_BOX, PARTS>;
  static std::atomic<uint32_t> done{0};
  const cudaError_t e = allow_smem(kern, Cfg<D, TILES>::kAlloc, done);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.blocks) * p.kv_heads * p.splits);
  kern<<<grid, Cfg<D, TILES>::kThreads, Cfg<D, TILES>::kAlloc, s>>>(p, maps);
  return cudaGetLastError();
}
template <int D, int TILES, bool WIDE_BOX>
cudaError_t launch_parts(const TileParams& p, const TileMaps& maps, cudaStream_t s) {
  return p.indptr == nullptr ? launch_box<D, TILES, WIDE_BOX, 2>(p, maps, s) : launch_box<D, TILES, WIDE_BOX, 1>(p, maps, s);
}
template <int D, int TILES>
cudaError_t launch_d(const TileParams& p, const TileMaps& maps, cudaStream_t s) {
  return p.box >= 8 ? launch_parts<D, TILES, true>(p, maps, s) : launch_parts<D, TILES, false>(p, maps, s);
}
template <int D>
cudaError_t launch_join_d(const TileParams& p, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(p.n_tokens) * p.q_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tile_join<D>, p);
}

}  // namespace

cudaError_t launch_tile(const TileParams& p, const TileMaps& maps, int head_dim, cudaStream_t s) {
  if (head_dim == 64) return p.tiles == 2 ? launch_d<64, 2>(p, maps, s) : launch_d<64, 1>(p, maps, s);
  if (head_dim == 128) return p.tiles == 2 ? launch_d<128, 2>(p, maps, s) : launch_d<128, 1>(p, maps, s);
  return launch_d<256, 1>(p, maps, s);
}
cudaError_t launch_tile_join(const TileParams& p, int head_dim, cudaStream_t s) {
  if (head_dim == 64) return launch_join_d<64>(p, s);
  if (head_dim == 128) return launch_join_d<128>(p, s);
  return launch_join_d<256>(p, s);
}

}  // namespace pic
