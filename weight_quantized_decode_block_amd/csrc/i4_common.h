// What the kernels of products with 4-bit integer weights share.
//
// w[n,k] = (q[n,k] - z[n,k/group]) * s[n,k/group], q a code of 0 .. 15, z a
// zero point (8 where none are given), s FP16 or BF16, group 32, 64 or 128.
// Codes lie in tiles of 16 rows x 128 k of 1024 bytes, in the matrix operand's
// order: lane (n, g) = (lane % 16, lane / 16) has the 16 bytes at 16 * lane, and
// dword j of them is k = 32 j + 8 g .. + 7 of row n.  Nibbles p and p + 4 of a
// dword are elements 2p and 2p + 1, so that one shift and one mask give a pair.
// Scales and zero points lie either
//   in tiles: a tile's are [16 rows][128/group], one piece of memory too, or
//   row by row ([N][K/group], as a checkpoint has them): a load then touches a line for each
//     of 16 rows.
// A call says which (I4Operands::by_row).
#pragma once

#include "mx_common.h"
#include "wqd_internal.h"

namespace wqd {

constexpr uint32_t kI4Tile = 1024;  // bytes of 16 rows x 128 k

// 8 codes as BF16 values 16 + q (exact: q are the upper four fraction bits of
// [16, 32)): eight integer instructions and no conversion, where the compiler does not
// know the constants and keeps them in registers.  16 is taken back with the sum of
// the activations.
constexpr uint32_t kI4BiasMask = 0x00780078u, kI4BiasBase = 0x41804180u;
__device__ __forceinline__ bf16x8_t i4_biased(uint32_t w, uint32_t mask, uint32_t base) {
  const u32x4_t x = {(w << 3 & mask) | base, (w >> 1 & mask) | base, (w >> 5 & mask) | base, (w >> 9 & mask) | base};
  return __builtin_bit_cast(bf16x8_t, x);
}
constexpr float kI4Bias = 16.0f;

// A scale's value.  Both readings are formed and one is taken: the compiler
// makes a branch of it otherwise, which no load and no matrix instruction crosses.
__device__ __forceinline__ float i4_scale(uint32_t bits, bool bf) {
  float b = __uint_as_float(bits << 16), h = (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  asm volatile("" : "+v"(b), "+v"(h));
  return bf ? b : h;
}

// The scales (zero points) of a row of a tile: NG of them, one load.  Rows are SROW scales and ZROW zero points
// apart.
template <int NG>
struct I4Groups {
  uint32_t s[NG == 4 ? 2 : 1], z;
};
template <int NG, bool ZEROS, int SROW = NG, int ZROW = NG>
__device__ __forceinline__ I4Groups<NG> i4_load_groups(const uint16_t *s, const uint8_t *z, uint32_t row) {
  I4Groups<NG> r;
  s += row * SROW;
  z += row * ZROW;
  if constexpr (NG == 4) {
    const u32x2_t v = *reinterpret_cast<const u32x2_t *>(s);
    r.s[0] = v.x;
    r.s[1] = v.y;
  } else if constexpr (NG == 2) {
    r.s[0] = *reinterpret_cast<const uint32_t *>(s);
  } else {
    r.s[0] = *s;
  }
  if constexpr (!ZEROS)
    r.z = 0x08080808u;
  else if constexpr (NG == 4)
    r.z = *reinterpret_cast<const uint32_t *>(z);
  else if constexpr (NG == 2)
    r.z = *reinterpret_cast<const uint16_t *>(z);
  else
    r.z = *z;
  return r;
}
template <int NG>
__device__ __forceinline__ float i4_scale_of(const I4Groups<NG> &x, int i, bool bf) {
  return i4_scale(x.s[i >> 1] >> (16 * (i & 1)) & 0xffffu, bf);
}
template <int NG>
__device__ __forceinline__ float i4_zero_of(const I4Groups<NG> &x, int i) {
  return (float)(x.z >> (8 * i) & 255u);
}

// The rows of chunk number `chunk` when every expert's list is cut into chunks
// of CHUNK rows: its expert, the place of its first row in `order` and how many
// they are; false past the last one.  All lanes of a wave call it.  Places are
// held to the pairs that there are, whatever the lists say.
template <uint32_t CHUNK>
__device__ __forceinline__ bool i4_find_chunk(const int32_t *offsets, uint32_t E, uint32_t pairs, uint32_t chunk,
                                              uint32_t lane, uint32_t &expert, uint32_t &first, uint32_t &rows) {
  uint32_t before = 0;
  for (uint32_t e0 = 0; e0 < E; e0 += 64u) {
    const uint32_t e = e0 + lane;
    uint32_t lo = 0, hi = 0;
    if (e < E) {
      lo = (uint32_t)offsets[e];
      hi = (uint32_t)offsets[e + 1u];
    }
    lo = lo < pairs ? lo : pairs;
    hi = hi < pairs ? hi : pairs;
    const uint32_t count = hi > lo ? hi - lo : 0u, chunks = (count + CHUNK - 1u) / CHUNK;
    uint32_t sum = chunks;
#pragma unroll
    for (uint32_t d = 1; d < 64; d *= 2) {
      const uint32_t v = (uint32_t)__shfl_up((int)sum, d);
      sum += lane >= d ? v : 0u;
    }
    const uint32_t total = (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
    if (chunk - before < total) {
      const uint32_t l = (uint32_t)__builtin_ctzll(__ballot(sum > chunk - before));
      const uint32_t c = chunk - before - (uint32_t)__builtin_amdgcn_readlane((int)(sum - chunks), (int)l);
      const uint32_t left = (uint32_t)__builtin_amdgcn_readlane((int)count, (int)l) - c * CHUNK;
      expert = e0 + l;
      first = (uint32_t)__builtin_amdgcn_readlane((int)lo, (int)l) + c * CHUNK;
      rows = left < CHUNK ? left : CHUNK;
      return true;
    }
    before += total;
  }
  return false;
}

// How many chunks there are.
template <uint32_t CHUNK>
__device__ __forceinline__ uint32_t i4_count_chunks(const int32_t *offsets, uint32_t E, uint32_t pairs, uint32_t lane) {
  uint32_t sum = 0;
  for (uint32_t e = lane; e < E; e += 64u) {
    uint32_t lo = (uint32_t)offsets[e], hi = (uint32_t)offsets[e + 1u];
    lo = lo < pairs ? lo : pairs;
    hi = hi < pairs ? hi : pairs;
    sum += ((hi > lo ? hi - lo : 0u) + CHUNK - 1u) / CHUNK;
  }
#pragma unroll
  for (uint32_t d = 1; d < 64; d *= 2) sum += (uint32_t)__shfl_xor((int)sum, d);
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)sum);
}

// Chunks that lists of `pairs` pairs over E experts are cut into, at most.
inline uint64_t i4_chunks(uint64_t pairs, uint32_t E, uint32_t chunk) {
  const uint64_t busy = pairs < E ? pairs : E;
  return (pairs + busy * (chunk - 1u)) / chunk;
}

}  // namespace wqd
