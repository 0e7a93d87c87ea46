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
// in fp32, and a value is rounded once.  The weights lie in shared memory as fp32, in the
// order in which lanes read them: in registers they would be 32 more, for q and k.  The
// latent of an MLA row is normalised by a warp of its own, two chunks a lane.
// Measured (GB300, 32 + 8 heads of 128 dims): 16,384 tokens of three axes 61.0 us,
// 403 MB at 6.6 TB/s; 64 tokens 2.9 us; one token 2.7 us.  MLA, 16 query heads,
// 2,048 tokens: 16.0 us, 5.0 TB/s.  With norms: 16,384 tokens of one axis 78 us (5.2 TB/s),
// where shuffles, weights and the products with them keep the loads apart; one token 4.9 us;
// MLA, 2,048 tokens: 16.7 us.
#include "pic_decode.h"
#include "pic_device.cuh"
#include "pic_paged.cuh"

namespace pic {
namespace {

using namespace dev;

constexpr int kWriteThreads = 128;
constexpr int kWriteWarps = kWriteThreads / 32;
// heads in flight per lane; with norms one and the next, at two more CTAs per SM (16,384 tokens: 78 us, six CTAs 82)
__host__ __device__ constexpr int rot_batch(bool norm) { return norm ? 1 : 2; }
constexpr int kCopyBatch = 8;   // 16-byte chunks in flight per lane
constexpr int kLatentChunks = 512 * 2 / 16;   // 16-byte chunks of a latent (pic_create admits no other width)

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
// Packed fp32 arithmetic, written out.
__device__ __forceinline__ uint64_t pair64(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
// a pair of fp32 values as bf16
__device__ __forceinline__ uint32_t pack64(uint64_t v) {
  const float2 f = unpair(v);
  return bf_pack(f.x, f.y);
}
__device__ __forceinline__ float sum_squares(uint4 v, uint4 w) {
  uint64_t s = 0, t = 0;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint64_t y = pair64(bf_lo(word(v, x)), bf_hi(word(v, x))), z = pair64(bf_lo(word(w, x)), bf_hi(word(w, x)));
    s = fma2(y, y, s);
    t = fma2(z, z, t);
  }
  const float2 a = unpair(s), b = unpair(t);
  return (a.x + a.y) + (b.x + b.y);
}

template <int PAIRING, bool NORM>
__global__ void __launch_bounds__(kWriteThreads, NORM ? 8 : 6) k_write_tokens(const __grid_constant__ WriteParams P) {
  constexpr bool NEOX = PAIRING == kNeox;
  __shared__ float4 s_freq[kWriteWarps][kMaxFreqs / 2];   // lanes read eight of their own
  __shared__ __align__(8) uint8_t s_axis[kWriteWarps][kMaxFreqs];
  const int lane = threadIdx.x & 31;
  // weights of q and k as lanes read them: parts 0, 1 the first chunk of a lane, 2, 3 the second (16 lanes at most)
  __shared__ float4 s_norm[NORM ? kWriteWarps : 1][NORM ? 2 : 1][4][NORM ? 16 : 1];
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
      float4(*norm)[4][NORM ? 16 : 1] = s_norm[NORM ? threadIdx.x >> 5 : 0];
      if constexpr (NORM) {
        // (MLA: heads as they are, its latent has a warp of its own)
        for (int i = lane; i < 4 * lph; i += 32) {
          const int kind = i / (2 * lph), chunk = i - kind * 2 * lph;
          const uint8_t* w = P.latent_norm != 0 ? nullptr : (kind == 0 ? P.q_norm : P.k_norm);
          float x[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
          if (w != nullptr) norm_weights(P, w, chunk, x);
          const int at = NEOX ? chunk & (lph - 1) : chunk >> 1, part = NEOX ? 2 * (chunk >> P.lph_shift) : 2 * (chunk & 1);
          norm[kind][part][at] = make_float4(x[0], x[1], x[2], x[3]);
          norm[kind][part + 1][at] = make_float4(x[4], x[5], x[6], x[7]);
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
      if constexpr (NORM) {
        // one head at a time, the next one on its way; two elements at a time; heads that have no norm as with weights
        // and factor 1 (one path: the second was in the way of the first's instructions)
        const float inv_dims = 1.0f / (16 * lph);
        // (all lanes leave the loop together: they meet in shuffles)
#pragma unroll 1
        for (int h = h_begin; h - sub < h_end; h += hpi) {
          load(h + hpi, a[1], b[1]);
          const int kind = h < P.q_heads ? 0 : 1;
          float sum = h < h_end ? sum_squares(a[0][0], b[0][0]) : 0.0f;
#pragma unroll
          for (int o = 1; o < 16; o <<= 1)
            if (o < lph) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (h < h_end && (kind == 0 || row >= 0)) {
            const bool normed = P.latent_norm == 0 && (kind == 0 ? P.q_norm : P.k_norm) != nullptr;
            const float r = normed ? rsqrtf(sum * inv_dims + P.norm_eps) : 1.0f;
            const uint64_t rr = pair64(r, r);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 fa = norm[kind][e >> 1][j], fb = norm[kind][2 + (e >> 1)][j];
              const uint32_t va = word(a[0][0], e), vb = word(b[0][0], e);
              const uint64_t xa = mul2(mul2(pair64(bf_lo(va), bf_hi(va)), rr), (e & 1) ? pair64(fa.z, fa.w) : pair64(fa.x, fa.y));
              const uint64_t xb = mul2(mul2(pair64(bf_lo(vb), bf_hi(vb)), rr), (e & 1) ? pair64(fb.z, fb.w) : pair64(fb.x, fb.y));
              if (NEOX) {   // pairs (a, b) of frequencies 2 e and 2 e + 1
                const uint64_t cc = pair64(c[2 * e], c[2 * e + 1]), ss = pair64(s[2 * e], s[2 * e + 1]);
                word(a[0][0], e) = pack64(fma2(xa, cc, mul2(xb, ss ^ 0x8000000080000000ull)));
                word(b[0][0], e) = pack64(fma2(xa, ss, mul2(xb, cc)));
              } else {      // pairs within a word: of frequency e, and 4 + e
                const float2 ya = unpair(xa), yb = unpair(xb);
                word(a[0][0], e) = bf_pack(ya.x * c[e] - ya.y * s[e], ya.x * s[e] + ya.y * c[e]);
                word(b[0][0], e) = bf_pack(yb.x * c[4 + e] - yb.y * s[4 + e], yb.x * s[4 + e] + yb.y * c[4 + e]);
              }
            }
            uint8_t* dst = (kind == 0 ? qd : kd) + static_cast<int64_t>(h) * P.head_bytes;
            *reinterpret_cast<uint4*>(dst + off_a) = a[0][0];
            *reinterpret_cast<uint4*>(dst + off_b) = b[0][0];
          }
          a[0][0] = a[1][0];
          b[0][0] = b[1][0];
        }
        return;
      }
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
        float sum = sum_squares(v[0], v[1]);
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
