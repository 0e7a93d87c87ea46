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

// cos / sin of pos * theta with the exact reduction of shift_cossin, then the
// hardware's sine and cosine: their absolute error on [-pi, pi] is below 2^-21,
// far inside the rounding to bf16 that follows here, at a fifth of the
// instructions of sincospif (these operators turn every token by angles of its own).
__device__ __forceinline__ void turn_cossin(float pos, float2 f, float& c, float& s) {
  const float p = __fmul_rn(pos, f.x);
  const float e = __fmaf_rn(pos, f.x, -p);
  const float r = __fsub_rn(p, rintf(p));
  const float t = 6.283185307179586f * __fadd_rn(r, __fmaf_rn(pos, f.y, e));
  c = __cosf(t);
  s = __sinf(t);
}

// The status word and, beside it, where the last bad block was met (WsHeader).
__device__ __forceinline__ void raise_block(uint32_t* status, int req, int slot) {
  atomicOr(status, static_cast<uint32_t>(PIC_DEV_BAD_BLOCK));
  status[1] = static_cast<uint32_t>(req);
  status[2] = static_cast<uint32_t>(slot);
}

}  // namespace dev
}  // namespace pic
