// Products with 4-bit integer weights for few rows, for gfx950 (MI355X):
//
//   C[m,n] = bf16( sum_k a[m,k] w[n,k] ),  w[n,k] = (q[n,k] - z[n,k/group]) s[n,k/group],
//
// with two weight matrices silu of the first times the second, and the same
// for the rows that a router gave to each of many matrices.  The weights' bytes
// bound it: each is read once.
//
//   * sum over a group of a (q - z) = sum a (16 + q) - (16 + z) sum a: the codes
//     enter the BF16 matrix instruction as 16 + q (i4_biased), a second one
//     against ones gives the activations' sum in the same lanes, and the group's
//     scale meets both in fp32.  All products are exact, sums are fp32.
//   * A workgroup of 8 waves owns 16 weight rows (of both matrices in the gated
//     form) and up to MMAX activation rows; a wave has an eighth of K to itself, as
//     consecutive tiles of 16 x 128 codes, which come in whole KB in the matrix
//     operand's order.  Its activations come in row order and turn in LDS that is
//     the wave's own.  The waves meet once, to add their sums in wave order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/wqd.h"
#include "i4_common.h"
#include "mx_product.h"
#include "wqd_internal.h"

namespace wqd {
namespace {

constexpr int NW = 8;  // waves of a workgroup

// Where a workgroup's rows come from.
constexpr int kDense = 0;  // rows m0 ..
constexpr int kLists = 1;  // rows of one expert's list
constexpr int kPairs = 2;  // one row, of one token and slot
constexpr int kSum = 3;    // one token's slots, one after another, weighted and added

template <int MMAX, bool GATED, int NG, bool ZEROS, int ROWS, int DEPTH>
__global__ __launch_bounds__(64 * NW) void i4_skinny_kernel(I4Operands op) {
  constexpr int MT = (MMAX + 15) / 16, G = GATED ? 2 : 1, SA = (MMAX + 3) / 4;
  constexpr uint32_t kLanes = MMAX <= 4 ? 16 : 64;  // lanes that end with rows below MMAX
  constexpr uint32_t kARegion = MMAX * 256, kParts = NW * G * MT * kLanes * 16;
  constexpr uint32_t kLds = NW * kARegion > kParts ? NW * kARegion : kParts;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];

  const uint32_t tid = threadIdx.x, lane = tid & 63u, r = lane & 15u, g = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t tiles = (op.N + 15u) >> 4, kt = op.K >> 7, pairs = op.T * op.top_k;

  // which rows and which matrix
  uint32_t block = blockIdx.x, tile, first = 0, rows = 1, expert = 0;
  if constexpr (ROWS == kDense) {
    const uint32_t chunks = (op.M + MMAX - 1u) / MMAX;
    tile = block / chunks;
    first = (block - tile * chunks) * MMAX;
    rows = op.M - first < (uint32_t)MMAX ? op.M - first : (uint32_t)MMAX;
  } else if constexpr (ROWS == kLists) {
    const uint32_t chunk = block / tiles;
    tile = block - chunk * tiles;
    if (!i4_find_chunk<MMAX>(op, chunk, lane, expert, first, rows)) return;
  } else {
    first = block / tiles;  // pair, or token
    tile = block - first * tiles;
    if constexpr (ROWS == kPairs) {
      expert = (uint32_t)op.ids[first];
      if (expert >= op.E) return;
    }
  }
  // the row of A that row m of this workgroup multiplies, and the row it writes
  auto pair_of = [&](uint32_t m) __attribute__((always_inline)) {
    if constexpr (ROWS == kLists) {
      const uint32_t p = (uint32_t)op.order[first + (m < rows ? m : rows - 1u)];
      return p < pairs ? p : 0u;
    } else {
      return first;
    }
  };
  auto source = [&](uint32_t m) __attribute__((always_inline)) {
    if constexpr (ROWS == kDense) return first + (m < rows ? m : rows - 1u);
    return GATED ? pair_of(m) / op.top_k : pair_of(m);
  };

  // this wave's tiles: of one row of tiles, or of all slots' after another
  const uint32_t total = ROWS == kSum ? kt * op.top_k : kt;
  const uint32_t u0 = (uint32_t)((uint64_t)total * wave / NW), u1 = (uint32_t)((uint64_t)total * (wave + 1u) / NW);
  const uint32_t n = tile * 16u + r, nn = n < op.N ? n : op.N - 1u;
  const uint32_t srow = op.K / (128u / NG), scale_at = (nn - tile * 16u) * srow;

  const u32x4_t *arow[SA];  // of each 16-byte piece that this lane brings
#pragma unroll
  for (int i = 0; i < SA; ++i)
    arow[i] = reinterpret_cast<const u32x4_t *>(op.A + (uint64_t)(ROWS == kSum ? 0u : source(i * 4u + g)) * op.lda) + r;
  struct Step {
    u32x4_t w[G], a[SA];
    I4Groups<NG> s[G];
    float weight;
    uint32_t here;
  };
  auto load = [&](uint32_t u) __attribute__((always_inline)) {
    Step x;
    uint32_t t = u < u1 ? u : u1 - 1u, e = expert;
    uint64_t a0 = 0;
    x.here = 1u;
    x.weight = 1.0f;
    if constexpr (ROWS == kSum) {
      const uint32_t slot = t / kt, p = first * op.top_k + slot;
      t -= slot * kt;
      e = (uint32_t)__builtin_amdgcn_readfirstlane(op.ids[p]);
      x.here = e < op.E;
      e = x.here ? e : 0u;
      x.weight = op.weights[p];
      a0 = (uint64_t)p * op.lda / 8u;
    }
    // an offset that the compiler cannot follow from step to step: it would keep a pointer for every request in flight
    asm volatile("" : "+s"(t));
    const uint64_t wt = (((uint64_t)e * tiles + tile) * kt + t) * kI4Tile;
    const uint64_t st = ((uint64_t)e * op.N + tile * 16u) * srow + t * NG;
#pragma unroll
    for (int m = 0; m < G; ++m) {
      const I4Matrix &mat = m ? op.up : op.w;
      x.w[m] = *reinterpret_cast<const u32x4_t *>(mat.W + wt + lane * 16u);
      x.s[m] = i4_load_groups<NG, ZEROS>(mat.S + st, mat.Z + st, scale_at);
    }
#pragma unroll
    for (int i = 0; i < SA; ++i) x.a[i] = arow[i][a0 + t * 16u];
    return x;
  };

  f32x4_t acc[G][MT];
#pragma unroll
  for (int m = 0; m < G; ++m)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[m][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  uint8_t *mine = lds + wave * kARegion;
  const bool bf = op.scale_bf16;
  const u32x4_t one = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
  const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, one);
  auto compute = [&](Step x) __attribute__((always_inline)) {
    if (ROWS == kSum && !x.here) return;
    // conversions stay with their own step: of several steps at once they would take twice the registers
#pragma unroll
    for (int m = 0; m < G; ++m) asm volatile("" : "+v"(x.w[m]));
    // Piece p of row m lies in slot p ^ (m % 16): the sixteen lanes that a
    // 16-byte LDS read serves together meet all 64 banks.
#pragma unroll
    for (int i = 0; i < SA; ++i) {
      const uint32_t m = i * 4u + g;
      if (MMAX % 4 == 0 || m < (uint32_t)MMAX) *reinterpret_cast<u32x4_t *>(mine + m * 256u + (r ^ (m & 15u)) * 16u) = x.a[i];
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const uint32_t m = i * 16u + (r & (MMAX < 16 ? MMAX - 1u : 15u));
      bf16x8_t a[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        a[j] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t *>(mine + m * 256u + ((4u * j + g) ^ (m & 15u)) * 16u));
      f32x4_t sum[NG];
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        sum[q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = q * 4 / NG; j < (q + 1) * 4 / NG; ++j)
          sum[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], ones, sum[q], 0, 0, 0);
      }
#pragma unroll
      for (int t = 0; t < G; ++t)
#pragma unroll
        for (int q = 0; q < NG; ++q) {
          f32x4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = q * 4 / NG; j < (q + 1) * 4 / NG; ++j)
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], i4_biased(x.w[t][j]), p, 0, 0, 0);
          const float s = i4_scale_of(x.s[t], q, bf) * (ROWS == kSum ? x.weight : 1.0f);
          const float z = -kI4Bias - i4_zero_of(x.s[t], q);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[t][i][c] = __builtin_fmaf(s, __builtin_fmaf(z, sum[q][c], p[c]), acc[t][i][c]);
        }
    }
  };

  if (u0 < u1) {
    Step ring[DEPTH];
    mx_unroll<0, DEPTH>([&](auto d) __attribute__((always_inline)) { ring[decltype(d)::value] = load(u0 + decltype(d)::value); });
    uint32_t u = u0;
    // whole rounds of the ring, so that the compiler's waits count the requests in flight
    while (u + DEPTH < u1) {
      mx_unroll<0, DEPTH>([&](auto d) __attribute__((always_inline)) {
        constexpr int D = decltype(d)::value;
        compute(ring[D]);
        ring[D] = load(u + D + DEPTH);
        __builtin_amdgcn_sched_barrier(0);  // steps side by side would take twice the registers
      });
      u += DEPTH;
    }
    mx_unroll<0, DEPTH>([&](auto d) __attribute__((always_inline)) {
      if (u + decltype(d)::value < u1) compute(ring[decltype(d)::value]);
      __builtin_amdgcn_sched_barrier(0);
    });
  }

  __syncthreads();
  f32x4_t *part = reinterpret_cast<f32x4_t *>(lds);
  if (lane < kLanes) {
#pragma unroll
    for (int t = 0; t < G; ++t)
#pragma unroll
      for (int i = 0; i < MT; ++i) part[((wave * G + t) * MT + i) * kLanes + lane] = acc[t][i];
  }
  __syncthreads();
  for (uint32_t x = tid; x < kLanes * MT; x += 64u * NW) {
    const uint32_t l = x % kLanes, i = x / kLanes;
    f32x4_t c[G];
#pragma unroll
    for (int t = 0; t < G; ++t) {
      c[t] = part[(t * MT + i) * kLanes + l];
#pragma unroll
      for (uint32_t w = 1; w < NW; ++w) c[t] += part[((w * G + t) * MT + i) * kLanes + l];
    }
    const uint32_t col = tile * 16u + (l & 15u);
    if (col >= op.N) continue;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      const uint32_t m = i * 16u + 4u * (l >> 4) + j;
      if (m >= rows) continue;
      const uint64_t at = (uint64_t)(ROWS == kDense || ROWS == kSum ? first + m : pair_of(m)) * op.ldc + col;
      if constexpr (GATED) {
        op.C[at] = (uint16_t)bf16x2_rne(silu_times(c[0][j], c[1][j]), 0.0f);
      } else if constexpr (ROWS == kLists) {
        op.Y[(uint64_t)pair_of(m) * op.N + col] = c[0][j];
      } else {
        op.C[at] = (uint16_t)bf16x2_rne(c[0][j], 0.0f);
      }
    }
  }
}

template <int MMAX, bool GATED, int NG, int ROWS, int DEPTH>
hipError_t launch_zeros(const I4Operands &op, uint32_t grid, hipStream_t stream) {
  if (op.w.Z)
    hipLaunchKernelGGL((i4_skinny_kernel<MMAX, GATED, NG, true, ROWS, DEPTH>), dim3(grid), dim3(64 * NW), 0, stream, op);
  else
    hipLaunchKernelGGL((i4_skinny_kernel<MMAX, GATED, NG, false, ROWS, DEPTH>), dim3(grid), dim3(64 * NW), 0, stream, op);
  return hipGetLastError();
}

template <int MMAX, bool GATED, int ROWS, int DEPTH>
hipError_t launch_cfg(const I4Operands &op, uint32_t grid, hipStream_t stream) {
  if (op.group == 128u) return launch_zeros<MMAX, GATED, 1, ROWS, DEPTH>(op, grid, stream);
  if (op.group == 64u) return launch_zeros<MMAX, GATED, 2, ROWS, DEPTH>(op, grid, stream);
  return launch_zeros<MMAX, GATED, 4, ROWS, DEPTH>(op, grid, stream);
}

template <int MMAX, bool GATED, int DEPTH>
hipError_t launch_dense(const I4Operands &op, hipStream_t stream) {
  const uint32_t tiles = (op.N + 15u) / 16u, rows = mx_max_grid(64 * NW) / tiles * MMAX;
  for (uint32_t m = 0; m < op.M; m += rows) {
    I4Operands part = op;
    part.A = op.A + (uint64_t)m * op.lda;
    part.C = op.C + (uint64_t)m * op.ldc;
    part.M = op.M - m < rows ? op.M - m : rows;
    const hipError_t e = launch_cfg<MMAX, GATED, kDense, DEPTH>(part, tiles * ((part.M + MMAX - 1u) / MMAX), stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool GATED>
hipError_t launch_rows(const I4Operands &op, hipStream_t stream) {
  if (op.M <= 4u) return launch_dense<4, GATED, 4>(op, stream);
  if (op.M <= 8u) return launch_dense<8, GATED, 3>(op, stream);
  return launch_dense<16, GATED, 2>(op, stream);
}

}  // namespace

hipError_t launch_i4_skinny(const I4Operands &op, bool gated, hipStream_t stream) {
  return gated ? launch_rows<true>(op, stream) : launch_rows<false>(op, stream);
}

uint64_t i4_experts_grid(const I4Operands &op) {
  const uint64_t pairs = (uint64_t)op.T * op.top_k, tiles = (op.N + 15u) / 16u;
  if (!op.order) return tiles * (op.gated ? pairs : op.T);
  return tiles * i4_chunks(pairs, op.E, 16u);
}

uint64_t i4_experts_max_grid() { return mx_max_grid(64 * NW); }

hipError_t launch_i4_experts_skinny(const I4Operands &op, hipStream_t stream) {
  const uint32_t grid = (uint32_t)i4_experts_grid(op);
  if (op.order) return op.gated ? launch_cfg<16, true, kLists, 2>(op, grid, stream) : launch_cfg<16, false, kLists, 2>(op, grid, stream);
  return op.gated ? launch_cfg<4, true, kPairs, 4>(op, grid, stream) : launch_cfg<4, false, kSum, 4>(op, grid, stream);
}

}  // namespace wqd
