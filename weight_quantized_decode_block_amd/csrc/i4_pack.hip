// Layout of 4-bit integer weights for gfx950 (MI355X): rows of codes, two a
// byte, to the tiles that the products read (i4_common.h).  Done once per
// matrix.  A thread gathers the 16 bytes of one lane of a tile from four dwords
// of its row, and a scale and a zero point, where they are to be in tiles too; rows past the
// matrix are written as zeros.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "i4_common.h"
#include "mx_product.h"

namespace wqd {
namespace {

// Nibbles e0 .. e7 of a dword to the order e0 e2 e4 e6 e1 e3 e5 e7
__device__ __forceinline__ uint32_t halves(uint32_t w) {
  auto even = [](uint32_t x) {  // nibbles 0, 2, 4, 6 to 16 bits
    x &= 0x0f0f0f0fu;
    x = (x | x >> 4) & 0x00ff00ffu;
    return (x | x >> 8) & 0xffffu;
  };
  return even(w) | even(w >> 4) << 16;
}

__global__ __launch_bounds__(256) void i4_pack_kernel(const uint32_t *__restrict__ Q, const uint16_t *__restrict__ S,
                                                      const uint8_t *__restrict__ Z, I4Matrix to, uint32_t N, uint32_t K,
                                                      uint32_t groups, uint64_t first, uint64_t pieces) {
  const uint64_t x = first + (uint64_t)blockIdx.x * 256u + threadIdx.x;
  if (x >= pieces) return;
  const uint32_t kt = K >> 7, tiles = (N + 15u) >> 4, lane = (uint32_t)x & 63u, n = lane & 15u, g = lane >> 4;
  const uint64_t tile = x >> 6, row_tile = tile / kt, e = row_tile / tiles;
  const uint32_t t = (uint32_t)(tile - row_tile * kt), row = (uint32_t)(row_tile - e * tiles) * 16u + n;
  const uint64_t from = (e * N + row) * kt + t;
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (row < N) {
    const uint32_t *q = Q + from * 16u + g;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) v[j] = halves(q[4u * j]);
  }
  reinterpret_cast<u32x4_t *>(const_cast<uint8_t *>(to.W))[x] = v;
  if (g < groups) {  // lane (n, g): group g of row n
    const uint64_t at = (tile * 16u + n) * groups + g;
    if (S) const_cast<uint16_t *>(to.S)[at] = row < N ? S[from * groups + g] : (uint16_t)0;
    if (Z) const_cast<uint8_t *>(to.Z)[at] = row < N ? Z[from * groups + g] : (uint8_t)0;
  }
}

}  // namespace

hipError_t launch_i4_pack(const void *Q, const I4Matrix &to, const void *S, const void *Z, uint32_t N, uint32_t K,
                          uint32_t group, uint32_t count, hipStream_t stream) {
  const uint64_t pieces = (uint64_t)count * ((N + 15u) / 16u) * (K / 128u) * 64u, most = (uint64_t)mx_max_grid(256) * 256u;
  for (uint64_t first = 0; first < pieces; first += most) {
    const uint64_t left = pieces - first < most ? pieces - first : most;
    hipLaunchKernelGGL(i4_pack_kernel, dim3((uint32_t)((left + 255u) / 256u)), dim3(256), 0, stream,
                       static_cast<const uint32_t *>(Q), static_cast<const uint16_t *>(S), static_cast<const uint8_t *>(Z), to, N, K,
                       128u / group, first, pieces);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace wqd
