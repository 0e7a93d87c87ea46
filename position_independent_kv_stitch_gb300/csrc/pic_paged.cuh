// Device helpers of the decode-loop operators: block-table lookups with their
// bounds check, and the errors they raise.
#pragma once

#include "pic_decode.h"
#include "pic_device.cuh"

namespace pic {
namespace dev {

// Block of a slot (0 <= slot): slot / block_size, as a product (no branch and no
// division, whatever the size).
__device__ __forceinline__ int block_of(const PagedView& v, int slot) {
  return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(slot)) * v.block_mul >> v.block_shift);
}

// Absolute cache row of a request's slot, -1 when the table has no such slot
// or names a block outside the cache.
__device__ __forceinline__ int64_t paged_row(const PagedView& v, int req, int slot) {
  const int b = block_of(v, slot);
  if (b >= v.max_blocks) return -1;
  const int32_t block = __ldg(v.tables + static_cast<int64_t>(req) * v.max_blocks + b);
  if (block < 0 || block >= v.num_cache_blocks) return -1;
  return static_cast<int64_t>(block) * v.block_size + (slot - b * v.block_size);
}

// The frequencies of a head in shared memory, two in a float4: (hi, hi, lo, lo),
// as turn_cossin2 takes them.
__device__ __forceinline__ void put_freq(float4* table, int i, float2 turns) {
  float* at = reinterpret_cast<float*>(table + (i >> 1)) + (i & 1);
  at[0] = turns.x;
  at[2] = turns.y;
}
// cos / sin of pos * theta for two frequencies at once, in packed fp32 arithmetic
// (these operators turn every token by angles of its own).  The angle is reduced
// as in shift_cossin, and further to t + k / 2 turns with |t| <= 1/4; then, with
// a = sqrt(2) sin(pi t) and b = sqrt(2) cos(pi t),
//   sin(2 pi t) = a b,  cos(2 pi t) = 1 - a a,  both negated where k is odd.
// a / t and b are polynomials in t^2, fitted for the least largest error over
// |t| <= 1/4 (2^-28 and 2^-25 of the value).  In fp32 the sine and cosine are off by
// 2^-21.5 at most (root mean square 2^-24), and where the angle is below an eighth turn
// by 2^-21.7 of themselves, so that an element that is small beside its partner
// keeps bf16's precision.  (The hardware's sine and cosine, of absolute error
// 2^-21, left sines of 1e-5 off by up to 4 %.)
__device__ __forceinline__ void turn_cossin2(float2 pos, float4 freq, float* c, float* s) {
  constexpr float kRound = 12582912.0f;   // 1.5 * 2^23: added, leaves an integer in the low bits
  const auto both = [](float x) { return make_float2(x, x); };
  const float2 hi = make_float2(freq.x, freq.y), lo = make_float2(freq.z, freq.w), neg = make_float2(-pos.x, -pos.y);
  const float2 p = __fmul2_rn(pos, hi);
  const float2 e = __ffma2_rn(neg, hi, p);                                            // p - pos * hi, exact
  const float2 r = __ffma2_rn(p, both(-1.0f), make_float2(rintf(p.x), rintf(p.y)));   // exact
  const float2 turn = __fadd2_rn(r, __ffma2_rn(neg, lo, e));                          // of the other sign, whole turns dropped
  const float2 k = __ffma2_rn(turn, both(2.0f), both(kRound));
  const float2 t = __ffma2_rn(__fadd2_rn(k, both(-kRound)), both(-0.5f), turn);       // exact
  const float2 u = __fmul2_rn(t, t);
  float2 a = __ffma2_rn(both(0.832989037f), u, both(-3.60590672f));
  a = __ffma2_rn(a, u, both(7.30824232f));
  a = __fmul2_rn(t, __ffma2_rn(a, u, both(-4.44288301f)));
  float2 b = __ffma2_rn(both(-1.84626889f), u, both(5.73819876f));
  b = __ffma2_rn(b, u, both(-6.97884226f));
  b = __ffma2_rn(b, u, both(1.41421354f));
  const float2 sn = __fmul2_rn(a, b);
  const uint32_t odd_x = __float_as_uint(k.x) << 31, odd_y = __float_as_uint(k.y) << 31;
  c[0] = __uint_as_float(__float_as_uint(__fmaf_rn(-a.x, a.x, 1.0f)) ^ odd_x);
  s[0] = __uint_as_float(__float_as_uint(sn.x) ^ odd_x);
  c[1] = __uint_as_float(__float_as_uint(__fmaf_rn(-a.y, a.y, 1.0f)) ^ odd_y);
  s[1] = __uint_as_float(__float_as_uint(sn.y) ^ odd_y);
}

// The status word and, beside it, where the last bad block was met (WsHeader).
__device__ __forceinline__ void raise_block(uint32_t* status, int req, int slot) {
  atomicOr(status, static_cast<uint32_t>(PIC_DEV_BAD_BLOCK));
  status[1] = static_cast<uint32_t>(req);
  status[2] = static_cast<uint32_t>(slot);
}

}  // namespace dev
}  // namespace pic
