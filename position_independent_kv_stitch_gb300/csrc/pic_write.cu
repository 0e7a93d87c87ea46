// Writes new tokens into the paged cache, with their rotary positions applied
// (sm_103a): decode tokens, the tokens recomputed at chunk heads, and image or
// video tokens whose positions have several axes.
//
// Frequency f of a head turns its pair (x_a, x_b) by the angle
// pos[axis(f)] * theta_f.  Queries are turned into q_out, keys on their way
// into their cache slot; values and the latent part of MLA rows are copied.
//
// Bound: HBM for many tokens (every byte is read once and written once), the
// launch and one chain of memory round trips for a decode step.  A warp takes
// one token and a run of its heads: 2^lph_shift lanes share a head, each lane
// turns eight frequencies (32 bytes), so its eight cos / sin pairs serve every
// head of the run and stay in registers.  Copies (values, latents) are warps of
// their own.  Rows are asked for before anything they do not depend on, and
// positions, slots and blocks are looked at after that.
// Measured (GB300, 32 + 8 heads of 128 dims): 16,384 tokens of three axes 61.0 us,
// 403 MB at 6.6 TB/s; 64 tokens 2.9 us; one token 2.7 us.  MLA, 16 query heads,
// 2,048 tokens: 16.0 us, 5.0 TB/s.
#include "pic_decode.h"
#include "pic_device.cuh"
#include "pic_paged.cuh"

namespace pic {
namespace {

using namespace dev;

constexpr int kWriteThreads = 128;
constexpr int kWriteWarps = kWriteThreads / 32;
constexpr int kRotBatch = 2;    // heads in flight per lane
constexpr int kCopyBatch = 8;   // 16-byte chunks in flight per lane
constexpr int kLatentChunks = 512 * 2 / 16;   // 16-byte chunks of a latent (pic_create admits no other width)

template <int PAIRING>
__global__ void __launch_bounds__(kWriteThreads, 6) k_write_tokens(const __grid_constant__ WriteParams P) {
  constexpr bool NEOX = PAIRING == kNeox;
  __shared__ float4 s_freq[kWriteWarps][kMaxFreqs / 2];   // lanes read eight of their own
  __shared__ __align__(8) uint8_t s_axis[kWriteWarps][kMaxFreqs];
  const int lane = threadIdx.x & 31;
  const int tasks = P.rot_parts + P.copy_parts;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kWriteWarps + (threadIdx.x >> 5);
  const int row_bytes = P.kv_heads * P.head_bytes;
  const int tok = static_cast<int>(task / tasks), part = static_cast<int>(task - static_cast<int64_t>(tok) * tasks);
  if (tok < P.n_tokens) {
    // The token's positions and block (the same in every lane).  What is loaded
    // here is first used after the rows have been asked for: a warp stops where
    // it touches a load that has not arrived.
    int pos[PIC_MAX_AXES];
#pragma unroll
    for (int a = 0; a < PIC_MAX_AXES; ++a)
      pos[a] = a < P.n_axes ? __ldg(P.pos + static_cast<int64_t>(a) * P.n_tokens + tok) : 0;
    int slot = -1, req = 0;
    if (P.kv_heads > 0) {
      slot = __ldg(P.slot + tok);
      req = __ldg(P.req + tok);
    }
    // cache row of the token, -1: not written (padding, or a bad place, which is raised)
    auto find_row = [&]() -> int64_t {
      if (slot < 0) return -1;
      const int64_t row = req >= 0 && req < P.paged.n_tables ? paged_row(P.paged, req, slot) : -1;
      if (row < 0 && lane == 0) raise_block(P.status, req, slot);
      return row;
    };
    auto bad_position = [&]() {
      bool bad = false;
#pragma unroll
      for (int a = 0; a < PIC_MAX_AXES; ++a) bad |= pos[a] > PIC_MAX_ABS_DELTA || pos[a] < -PIC_MAX_ABS_DELTA;
      if (bad && lane == 0) atomicOr(P.status, static_cast<uint32_t>(PIC_DEV_BAD_POS));
      return bad;
    };
    if (part < P.rot_parts) {
      const int lph = 1 << P.lph_shift;
      const int j = lane & (lph - 1), sub = lane >> P.lph_shift, hpi = 32 >> P.lph_shift;
      const int off_a = P.rope_off + (NEOX ? j : 2 * j) * 16;
      const int off_b = P.rope_off + (NEOX ? j + lph : 2 * j + 1) * 16;
      const int h_begin = part * P.rot_iters * hpi + sub;
      const int h_end = min(P.q_heads + P.kv_heads, (part + 1) * P.rot_iters * hpi);
      const uint8_t* qs = P.q + tok * P.q_stride;
      const uint8_t* ks = P.k + tok * P.k_stride - static_cast<int64_t>(P.q_heads) * P.head_bytes;
      uint4 a[2][kRotBatch], b[2][kRotBatch];
      auto load = [&](int h0, uint4 (&xa)[kRotBatch], uint4 (&xb)[kRotBatch]) {
#pragma unroll
        for (int u = 0; u < kRotBatch; ++u) {
          const int h = h0 + u * hpi;
          if (h >= h_end) continue;
          const uint8_t* src = (h < P.q_heads ? qs : ks) + static_cast<int64_t>(h) * P.head_bytes;
          xa[u] = *reinterpret_cast<const uint4*>(src + off_a);
          xb[u] = *reinterpret_cast<const uint4*>(src + off_b);
        }
      };
      load(h_begin, a[0], b[0]);
      float4* freq = s_freq[threadIdx.x >> 5];
      uint8_t* axis = s_axis[threadIdx.x >> 5];
      for (int i = lane; i < 8 * lph; i += 32) {
        put_freq(freq, i, P.freq.turns[i]);
        axis[i] = P.axis[i];
      }
      __syncwarp();
      if (bad_position()) return;
      const int64_t row = find_row();
      // this lane's 8 frequencies: neox pairs chunk j with chunk j + lph,
      // interleaved turns the pairs of chunks 2j and 2j + 1
      float c[8], s[8];
      const uint2 axes = *reinterpret_cast<const uint2*>(axis + 8 * j);
      auto position = [&](int i) {
        const int x = ((i < 4 ? axes.x : axes.y) >> (8 * (i & 3))) & 255u;
        int p = pos[0];
#pragma unroll
        for (int y = 1; y < PIC_MAX_AXES; ++y) p = x == y ? pos[y] : p;
        return static_cast<float>(p);   // exact for |p| < 2^24
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) turn_cossin2(make_float2(position(2 * i), position(2 * i + 1)), freq[4 * j + i], c + 2 * i, s + 2 * i);
      uint8_t* qd = P.q_out + tok * P.q_out_stride;
      uint8_t* kd = P.k_cache + row * row_bytes - static_cast<int64_t>(P.q_heads) * P.head_bytes;
      const int step = kRotBatch * hpi;
      for (int h0 = h_begin; h0 < h_end; h0 += 2 * step) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          load(h0 + (x + 1) * step, a[x ^ 1], b[x ^ 1]);
#pragma unroll
          for (int u = 0; u < kRotBatch; ++u) {
            const int h = h0 + x * step + u * hpi;
            if (h >= h_end || (h >= P.q_heads && row < 0)) continue;
            if (NEOX) {
              rotate_neox(a[x][u], b[x][u], c, s);
            } else {
              rotate_interleaved(a[x][u], c, s);
              rotate_interleaved(b[x][u], c + 4, s + 4);
            }
            uint8_t* dst = (h < P.q_heads ? qd : kd) + static_cast<int64_t>(h) * P.head_bytes;
            *reinterpret_cast<uint4*>(dst + off_a) = a[x][u];
            *reinterpret_cast<uint4*>(dst + off_b) = b[x][u];
          }
        }
      }
      return;
    }
    // copies: the query heads' latent chunks, then the key row's, then the value row
    const int nq = P.q_heads * P.q_copy_chunks, nk = P.k_copy_chunks;
    const int n = nq + nk + (P.v != nullptr ? row_bytes / 16 : 0);
    const int first = (part - P.rot_parts) * 32 * kCopyBatch + lane;
    uint4 x[kCopyBatch];
#pragma unroll
    for (int u = 0; u < kCopyBatch; ++u) {
      const int i = first + u * 32;
      if (i >= n) continue;
      const uint8_t* from;
      if (i < nq) from = P.q + tok * P.q_stride + static_cast<int64_t>(i / kLatentChunks) * P.head_bytes + (i % kLatentChunks) * 16;
      else if (i < nq + nk) from = P.k + tok * P.k_stride + (i - nq) * 16;
      else from = P.v + tok * P.v_stride + (i - nq - nk) * 16;
      x[u] = *reinterpret_cast<const uint4*>(from);
    }
    if (bad_position()) return;
    const int64_t row = find_row();
#pragma unroll
    for (int u = 0; u < kCopyBatch; ++u) {
      const int i = first + u * 32;
      if (i >= n || (i >= nq && row < 0)) continue;
      uint8_t* to;
      if (i < nq) to = P.q_out + tok * P.q_out_stride + static_cast<int64_t>(i / kLatentChunks) * P.head_bytes + (i % kLatentChunks) * 16;
      else if (i < nq + nk) to = P.k_cache + row * row_bytes + (i - nq) * 16;
      else to = P.v_cache + row * row_bytes + (i - nq - nk) * 16;
      *reinterpret_cast<uint4*>(to) = x[u];
    }
    if (P.weights != nullptr && row >= 0 && part == P.rot_parts) {
      const int64_t block = row / P.paged.block_size, at = row % P.paged.block_size;
      for (int h = lane; h < P.weight_heads; h += 32)
        P.weights[(block * P.weight_heads + h) * P.paged.block_size + at] = 0.0f;
    }
  }
}

}  // namespace

cudaError_t launch_write(const WriteParams& p, int pairing, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(p.n_tokens) * (p.rot_parts + p.copy_parts);
  const unsigned grid = static_cast<unsigned>((warps + kWriteWarps - 1) / kWriteWarps);
  if (pairing == kNeox) k_write_tokens<kNeox><<<grid, kWriteThreads, 0, s>>>(p);
  else k_write_tokens<kInterleaved><<<grid, kWriteThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace pic
