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
// With norms (pic_write_normed_tokens) a head x is first replaced by
// x / sqrt(mean(x^2) + eps) * w.  The lanes that turn a head hold all of it, so the sum of
// its squares is joined by 2 to 4 shuffles between its load and its rotation, all
// in fp32, and a value is rounded once.  The weights lie in shared memory as fp32:
// in registers they would be 32 more, for q and k.  The latent of an MLA row is
// normalised by a warp of its own, two chunks a lane.
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
// heads in flight per lane (with norms one, at two more CTAs per SM: 86 us for 16,384 tokens against 90)
__host__ __device__ constexpr int rot_batch(bool norm) { return norm ? 1 : 2; }
constexpr int kCopyBatch = 8;   // 16-byte chunks in flight per lane
constexpr int kLatentChunks = 512 * 2 / 16;   // 16-byte chunks of a latent (pic_create admits no other width)

constexpr int kNormDims = 256;   // of the widest head that is normalised whole

// Eight weights of a norm, from element 8 i on, as they multiply.
__device__ __forceinline__ void norm_weights(const WriteParams& P, const uint8_t* w, int i, float* out) {
  if (P.norm_f32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w) + 2 * i), b = __ldg(reinterpret_cast<const float4*>(w) + 2 * i + 1);
    out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w;
    out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
  } else {
    uint4 a = __ldg(reinterpret_cast<const uint4*>(w) + i);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      out[2 * x] = bf_lo(word(a, x));
      out[2 * x + 1] = bf_hi(word(a, x));
    }
  }
#pragma unroll
  for (int x = 0; x < 8; ++x) out[x] += P.norm_offset;
}
__device__ __forceinline__ float sum_squares(uint4 v) {
  float s = 0.0f;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const float2 y = bf_pair(word(v, x));
    s = __fmaf_rn(y.x, y.x, __fmaf_rn(y.y, y.y, s));
  }
  return s;
}

template <int PAIRING, bool NORM>
__global__ void __launch_bounds__(kWriteThreads, NORM ? 8 : 6) k_write_tokens(const __grid_constant__ WriteParams P) {
  constexpr bool NEOX = PAIRING == kNeox;
  __shared__ float4 s_freq[kWriteWarps][kMaxFreqs / 2];   // lanes read eight of their own
  __shared__ __align__(8) uint8_t s_axis[kWriteWarps][kMaxFreqs];
  const int lane = threadIdx.x & 31;
  __shared__ __align__(16) float s_norm[NORM ? kWriteWarps : 1][NORM ? 2 : 1][NORM ? kNormDims : 4];   // weights of q and k
  const int tasks = P.rot_parts + P.copy_parts + (NORM ? P.latent_norm : 0);
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
      constexpr int kRotBatch = rot_batch(NORM);
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
      float(*norm)[NORM ? kNormDims : 4] = s_norm[NORM ? threadIdx.x >> 5 : 0];
      if constexpr (NORM) {
        // (MLA: heads as they are, its latent has a warp of its own)
        for (int i = lane; i < 4 * lph && P.latent_norm == 0; i += 32) {
          const int kind = i / (2 * lph), chunk = i - kind * 2 * lph;
          const uint8_t* w = kind == 0 ? P.q_norm : P.k_norm;
          if (w != nullptr) norm_weights(P, w, chunk, &norm[kind][8 * chunk]);
        }
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
      // (with norms all lanes leave the loop together: they meet in shuffles)
      for (int h0 = h_begin; (NORM ? h0 - sub : h0) < h_end; h0 += 2 * step) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          load(h0 + (x + 1) * step, a[x ^ 1], b[x ^ 1]);
#pragma unroll
          for (int u = 0; u < kRotBatch; ++u) {
            const int h = h0 + x * step + u * hpi;
            if constexpr (NORM) {
              // (every lane takes part in the shuffles; a head past the end is not stored)
              const int kind = h < P.q_heads ? 0 : 1;
              const bool normed = P.latent_norm == 0 && (kind == 0 ? P.q_norm : P.k_norm) != nullptr;
              float sum = h < h_end ? sum_squares(a[x][u]) + sum_squares(b[x][u]) : 0.0f;
              for (int o = 1; o < lph; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
              if (h >= h_end || (h >= P.q_heads && row < 0)) continue;
              if (normed) {
                const float r = rsqrtf(sum / static_cast<float>(16 * lph) + P.norm_eps);
                const float* wa = &norm[kind][8 * (NEOX ? j : 2 * j)];
                const float* wb = &norm[kind][8 * (NEOX ? j + lph : 2 * j + 1)];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 ya = bf_pair(word(a[x][u], e)), yb = bf_pair(word(b[x][u], e));
                  const float a0 = ya.x * r * wa[2 * e], a1 = ya.y * r * wa[2 * e + 1];
                  const float b0 = yb.x * r * wb[2 * e], b1 = yb.y * r * wb[2 * e + 1];
                  if (NEOX) {   // pairs (a, b) of frequencies 2 e and 2 e + 1
                    const float c0 = c[2 * e], c1 = c[2 * e + 1], s0 = s[2 * e], s1 = s[2 * e + 1];
                    word(a[x][u], e) = bf_pack(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
                    word(b[x][u], e) = bf_pack(a0 * s0 + b0 * c0, a1 * s1 + b1 * c1);
                  } else {      // pairs (a0, a1) of frequency e, (b0, b1) of 4 + e
                    word(a[x][u], e) = bf_pack(a0 * c[e] - a1 * s[e], a0 * s[e] + a1 * c[e]);
                    word(b[x][u], e) = bf_pack(b0 * c[4 + e] - b1 * s[4 + e], b0 * s[4 + e] + b1 * c[4 + e]);
                  }
                }
                uint8_t* dst = (h < P.q_heads ? qd : kd) + static_cast<int64_t>(h) * P.head_bytes;
                *reinterpret_cast<uint4*>(dst + off_a) = a[x][u];
                *reinterpret_cast<uint4*>(dst + off_b) = b[x][u];
                continue;
              }
            }
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
    auto clear_weights = [&](int64_t row) {
      const int64_t block = row / P.paged.block_size, at = row % P.paged.block_size;
      for (int h = lane; h < P.weight_heads; h += 32)
        P.weights[(block * P.weight_heads + h) * P.paged.block_size + at] = 0.0f;
    };
    if constexpr (NORM) {
      if (part == P.rot_parts + P.copy_parts) {   // the latent of the key row
        const uint4* from = reinterpret_cast<const uint4*>(P.k + tok * P.k_stride);
        uint4 v[2] = {from[lane], from[lane + 32]};
        float w[2][8];
        norm_weights(P, P.k_norm, lane, w[0]);
        norm_weights(P, P.k_norm, lane + 32, w[1]);
        float sum = sum_squares(v[0]) + sum_squares(v[1]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrtf(sum * (1.0f / (8 * kLatentChunks)) + P.norm_eps);
        if (bad_position()) return;
        const int64_t row = find_row();
        if (row < 0) return;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = bf_pair(word(v[x], e));
            word(v[x], e) = bf_pack(y.x * r * w[x][2 * e], y.y * r * w[x][2 * e + 1]);
          }
          reinterpret_cast<uint4*>(P.k_cache + row * row_bytes)[lane + 32 * x] = v[x];
        }
        if (P.weights != nullptr && P.copy_parts == 0) clear_weights(row);
        return;
      }
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
    if (P.weights != nullptr && row >= 0 && part == P.rot_parts) clear_weights(row);
  }
}

}  // namespace

namespace {
template <bool NORM>
cudaError_t launch(const WriteParams& p, int pairing, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(p.n_tokens) * (p.rot_parts + p.copy_parts + p.latent_norm);
  const unsigned grid = static_cast<unsigned>((warps + kWriteWarps - 1) / kWriteWarps);
  if (pairing == kNeox) k_write_tokens<kNeox, NORM><<<grid, kWriteThreads, 0, s>>>(p);
  else k_write_tokens<kInterleaved, NORM><<<grid, kWriteThreads, 0, s>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_write(const WriteParams& p, int pairing, cudaStream_t s) { return launch<false>(p, pairing, s); }
cudaError_t launch_write_normed(const WriteParams& p, int pairing, cudaStream_t s) { return launch<true>(p, pairing, s); }

}  // namespace pic
