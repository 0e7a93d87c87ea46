// Writes new tokens into the paged cache, with their rotary positions applied
// (sm_103a): decode tokens, the tokens recomputed at chunk heads, and image or
// video tokens whose positions have several axes.
//
// Frequency f of a head turns its pair (x_a, x_b) by the angle
// pos[axis(f)] * theta_f.  Queries are turned into q_out, keys on their way
// into their cache slot; values and the latent part of MLA rows are copied.
//
// Bound: HBM for many tokens (every byte is read once and written once), the
// launch and one memory round trip for a decode step.  A warp takes one token
// and a run of its heads: 2^lph_shift lanes share a head, each lane turns
// eight frequencies (32 bytes), so its eight cos / sin pairs serve every head
// of the run and stay in registers.  Copies are warps of their own.
#include "pic_decode.h"
#include "pic_device.cuh"
#include "pic_paged.cuh"

namespace pic {
namespace {

using namespace dev;

constexpr int kWriteThreads = 128;
constexpr int kRotBatch = 4;    // heads in flight per lane
constexpr int kCopyBatch = 8;   // 16-byte chunks in flight per lane

template <int PAIRING>
__global__ void __launch_bounds__(kWriteThreads) k_write_tokens(const __grid_constant__ WriteParams P) {
  constexpr bool NEOX = PAIRING == kNeox;
  const int lane = threadIdx.x & 31;
  const int tasks = P.rot_parts + P.copy_parts;
  const int64_t n_tasks = static_cast<int64_t>(P.n_tokens) * tasks;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kWriteThreads / 32);
  const int row_bytes = P.kv_heads * P.head_bytes;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * (kWriteThreads / 32) + (threadIdx.x >> 5); task < n_tasks;
       task += step) {
    const int tok = static_cast<int>(task / tasks), part = static_cast<int>(task % tasks);
    // the token's positions and cache row (the same in every lane)
    int pos[PIC_MAX_AXES];
    bool bad_pos = false;
#pragma unroll
    for (int a = 0; a < PIC_MAX_AXES; ++a) {
      pos[a] = a < P.n_axes ? __ldg(P.pos + static_cast<int64_t>(a) * P.n_tokens + tok) : 0;
      bad_pos |= pos[a] > PIC_MAX_ABS_DELTA || pos[a] < -PIC_MAX_ABS_DELTA;
    }
    int64_t row = -1;
    if (P.kv_heads > 0) {
      const int slot = __ldg(P.slot + tok);
      if (slot >= 0) {
        const int req = __ldg(P.req + tok);
        row = req >= 0 && req < P.paged.n_tables ? paged_row(P.paged, req, slot) : -1;
        if (row < 0 && lane == 0) raise_block(P.status, req, slot);
      }
    }
    if (bad_pos) {
      if (lane == 0) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_BAD_POS));
      continue;
    }
    if (part < P.rot_parts) {
      const int lph = 1 << P.lph_shift;
      const int j = lane & (lph - 1), sub = lane >> P.lph_shift, hpi = 32 >> P.lph_shift;
      // this lane's 8 frequencies: neox pairs chunk j with chunk j + lph,
      // interleaved turns the pairs of chunks 2j and 2j + 1
      float c[8], s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int f = 8 * j + i;
        const int a = P.axis[f];
        int p = pos[0];
#pragma unroll
        for (int x = 1; x < PIC_MAX_AXES; ++x) p = a == x ? pos[x] : p;
        shift_cossin(p, P.freq.turns[f], c[i], s[i]);
      }
      const int off_a = P.rope_off + (NEOX ? j : 2 * j) * 16;
      const int off_b = P.rope_off + (NEOX ? j + lph : 2 * j + 1) * 16;
      const int heads = P.q_heads + (row >= 0 ? P.kv_heads : 0);
      const int h_begin = part * P.rot_iters * hpi + sub;
      const int h_end = min(heads, (part + 1) * P.rot_iters * hpi);
      for (int h0 = h_begin; h0 < h_end; h0 += kRotBatch * hpi) {
        uint4 a[kRotBatch], b[kRotBatch];
#pragma unroll
        for (int u = 0; u < kRotBatch; ++u) {
          const int h = h0 + u * hpi;
          if (h >= h_end) continue;
          const uint8_t* src = h < P.q_heads ? P.q + tok * P.q_stride + static_cast<int64_t>(h) * P.head_bytes
                                             : P.k + tok * P.k_stride + static_cast<int64_t>(h - P.q_heads) * P.head_bytes;
          a[u] = *reinterpret_cast<const uint4*>(src + off_a);
          b[u] = *reinterpret_cast<const uint4*>(src + off_b);
        }
#pragma unroll
        for (int u = 0; u < kRotBatch; ++u) {
          const int h = h0 + u * hpi;
          if (h >= h_end) continue;
          if (NEOX) {
            rotate_neox(a[u], b[u], c, s);
          } else {
            rotate_interleaved(a[u], c, s);
            rotate_interleaved(b[u], c + 4, s + 4);
          }
          uint8_t* dst = h < P.q_heads ? P.q_out + tok * P.q_out_stride + static_cast<int64_t>(h) * P.head_bytes
                                       : P.k_cache + row * row_bytes + static_cast<int64_t>(h - P.q_heads) * P.head_bytes;
          *reinterpret_cast<uint4*>(dst + off_a) = a[u];
          *reinterpret_cast<uint4*>(dst + off_b) = b[u];
        }
      }
      continue;
    }
    // copies: the query heads' latent chunks, then the key row's, then the value row
    const int nq = P.q_heads * P.q_copy_chunks;
    const int nk = row >= 0 ? P.k_copy_chunks : 0;
    const int nv = row >= 0 && P.v != nullptr ? row_bytes / 16 : 0;
    const int n = nq + nk + nv;
    const int first = (part - P.rot_parts) * 32 * kCopyBatch + lane;
    uint4 x[kCopyBatch];
    uint8_t* to[kCopyBatch];
#pragma unroll
    for (int u = 0; u < kCopyBatch; ++u) {
      int i = first + u * 32;
      to[u] = nullptr;
      if (i >= n) continue;
      const uint8_t* from;
      if (i < nq) {
        const int h = i / P.q_copy_chunks, o = (i % P.q_copy_chunks) * 16;
        from = P.q + tok * P.q_stride + static_cast<int64_t>(h) * P.head_bytes + o;
        to[u] = P.q_out + tok * P.q_out_stride + static_cast<int64_t>(h) * P.head_bytes + o;
      } else if (i < nq + nk) {
        from = P.k + tok * P.k_stride + (i - nq) * 16;
        to[u] = P.k_cache + row * row_bytes + (i - nq) * 16;
      } else {
        from = P.v + tok * P.v_stride + (i - nq - nk) * 16;
        to[u] = P.v_cache + row * row_bytes + (i - nq - nk) * 16;
      }
      x[u] = *reinterpret_cast<const uint4*>(from);
    }
#pragma unroll
    for (int u = 0; u < kCopyBatch; ++u)
      if (to[u] != nullptr) *reinterpret_cast<uint4*>(to[u]) = x[u];
    if (P.weights != nullptr && row >= 0 && part == P.rot_parts) {
      const int64_t block = row / P.paged.block_size, at = row % P.paged.block_size;
      for (int h = lane; h < P.weight_heads; h += 32)
        P.weights[(block * P.weight_heads + h) * P.paged.block_size + at] = 0.0f;
    }
  }
}

}  // namespace

cudaError_t launch_write(const WriteParams& p, int pairing, int sm_count, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(p.n_tokens) * (p.rot_parts + p.copy_parts);
  const int64_t ctas = (warps + kWriteThreads / 32 - 1) / (kWriteThreads / 32);
  const int64_t cap = static_cast<int64_t>(sm_count) * 16;
  const int grid = static_cast<int>(ctas < cap ? ctas : cap);
  if (pairing == kNeox) k_write_tokens<kNeox><<<grid, kWriteThreads, 0, s>>>(p);
  else k_write_tokens<kInterleaved><<<grid, kWriteThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace pic
