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
//   * A wave owns NT tiles of 16 weight rows (gated: of both matrices) and up to MMAX
//     activation rows, and of K an eighth (with experts also a half, a quarter, a
//     sixteenth): consecutive tiles of 16 x 128 codes, which come in whole KB in the
//     matrix operand's order.  Its activations come in row order and turn in LDS that is
//     the wave's own.  The waves meet once, to add their sums in wave order: no atomics,
//     and no second launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/wqd.h"
#include "i4_common.h"
#include "mx_product.h"
#include "wqd_internal.h"

namespace wqd {
namespace {

// Waves of a workgroup, but for kSum.  4 or 16 are slower at most sizes (1 x 5120, K = 5120 6.0 us, with 16 waves 7.9,
// with 4 7.3).
constexpr int kWaves = 8;

// Where a workgroup's rows come from.
constexpr int kDense = 0;  // rows m0 ..
constexpr int kLists = 1;  // rows of one expert's list
constexpr int kPairs = 2;  // one row, of one token and slot
constexpr int kSum = 3;    // one token's slots, one after another, weighted and added

// What is not needed before the first loads.
struct Rest {
  const uint8_t *ZU;
  uint16_t *C;
  float *Y;
  const int32_t *ids, *order, *offsets;
  const float *weights;
  uint32_t ldc, scale_bf16, top_k, E;
  uint32_t chunk;  // the first of this launch
};

// BY_ROW: scales and zero points row by row: 16 lanes then touch 16 lines for them at each step, where those of a tile are
// one or two (1 x 5120, K = 5120 6.0 us, in tiles 5.7; 16 x 5120, K = 17408 in groups of 64 with zero points 23.7 and
// 15.9; 33 tokens' last products 27.2 and 23.0).
// NT: 16-row weight tiles of a wave (of either matrix).  KS of the NW waves share K; NW / KS
// such groups stand side by side.  DEPTH: steps in flight.  The arguments up to SU are in
// registers when a wave starts.  M: rows, or tokens.
template <int NW, int MMAX, int NT, int KS, int DEPTH, bool GATED, int NG, bool ZEROS, bool BY_ROW, int ROWS>
__global__ __launch_bounds__(64 * NW) void i4_skinny_kernel(const uint8_t *__restrict__ W, const uint16_t *__restrict__ S,
                                                            const uint16_t *__restrict__ A, uint32_t K, uint32_t N,
                                                            uint32_t M, uint32_t lda, const uint8_t *__restrict__ Z,
                                                            const uint8_t *__restrict__ WU, const uint16_t *__restrict__ SU,
                                                            Rest op) {
  constexpr int MT = (MMAX + 15) / 16, G = GATED ? 2 : 1, WT = NT * G, SA = (MMAX + 3) / 4;
  constexpr uint32_t kLanes = MMAX <= 4 ? 16 : 64;  // lanes that end with rows below MMAX
  constexpr uint32_t kARegion = MMAX * 256, kParts = NW * WT * MT * kLanes * 16;
  constexpr uint32_t kLds = NW * kARegion > kParts ? NW * kARegion : kParts;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];

  const uint32_t tid = threadIdx.x, lane = tid & 63u, r = lane & 15u, g = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t tiles = (N + 15u) >> 4, kt = K >> 7, ks = wave % KS;
  const uint32_t tile0 = blockIdx.x * (NW / KS * NT), tile = tile0 + wave / KS * NT;  // of the workgroup, of this wave

  // which rows and which matrix
  uint32_t first = blockIdx.y, rows = 1, expert = 0;  // first: row, place in the lists, pair or token
  if constexpr (ROWS == kDense) {
    first *= MMAX;
    rows = M - first < (uint32_t)MMAX ? M - first : (uint32_t)MMAX;
  } else if constexpr (ROWS == kLists) {
    if (!i4_find_chunk<MMAX>(op.offsets, op.E, M * op.top_k, op.chunk + blockIdx.y, lane, expert, first, rows)) return;
  } else if constexpr (ROWS == kPairs) {
    expert = (uint32_t)op.ids[first];
    if (expert >= op.E) return;
  }
  // pair of row m of this workgroup, and the row of A that it multiplies
  auto pair_of = [&](uint32_t m) __attribute__((always_inline)) {
    if constexpr (ROWS == kLists) {
      const uint32_t p = (uint32_t)op.order[first + (m < rows ? m : rows - 1u)];
      return p < M * op.top_k ? p : 0u;
    } else {
      return first;
    }
  };
  auto source = [&](uint32_t m) __attribute__((always_inline)) {
    if constexpr (ROWS == kDense) return first + (m < rows ? m : rows - 1u);
    if constexpr (ROWS == kSum) return 0u;
    return GATED ? pair_of(m) / op.top_k : pair_of(m);
  };

  // this wave's steps: the tiles of a row of tiles, or of all slots' after another
  const uint32_t total = ROWS == kSum ? kt * op.top_k : kt;
  const uint32_t u0 = total * ks / KS, u1 = total * (ks + 1u) / KS;

  const u32x4_t *arow[SA];  // of each 16-byte piece that this lane brings
#pragma unroll
  for (int i = 0; i < SA; ++i) arow[i] = reinterpret_cast<const u32x4_t *>(A + (uint64_t)source(i * 4u + g) * lda) + r;
  struct Step {
    u32x4_t w[WT], a[SA];
    I4Groups<NG> s[WT];
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
      a0 = (uint64_t)p * lda / 8u;
    }
    // an offset that the compiler cannot follow from step to step: it would keep a pointer for every request in flight
    asm volatile("" : "+s"(t));
#pragma unroll
    for (int j = 0; j < WT; ++j) {
      const uint32_t row = tile + j / G < tiles ? tile + j / G : tiles - 1u;
      const uint64_t at = ((uint64_t)e * tiles + row) * kt + t;
      const bool up = GATED && (j & 1);
      // this step's scales of the tile's first row, and by how many steps' this lane's come later: of a row that there is
      const uint64_t group = (BY_ROW ? ((uint64_t)e * N + row * 16u) * kt + t : at * 16u) * NG;
      uint32_t own = r;
      if constexpr (BY_ROW) {
        uint32_t last = (N - 1u - row * 16u) * kt;
        asm volatile("" : "+s"(last));  // formed here: kept from step to step they would not fit the registers
        own = r * kt < last ? r * kt : last;
        if (MMAX > 16) __builtin_amdgcn_sched_barrier(0);  // and of several tiles at once neither
      }
      x.w[j] = *reinterpret_cast<const u32x4_t *>((up ? WU : W) + at * kI4Tile + lane * 16u);
      x.s[j] = i4_load_groups<NG, ZEROS>((up ? SU : S) + group, (up ? op.ZU : Z) + group, own);
    }
#pragma unroll
    for (int i = 0; i < SA; ++i) x.a[i] = arow[i][a0 + t * 16u];
    return x;
  };

  f32x4_t acc[WT][MT];
#pragma unroll
  for (int t = 0; t < WT; ++t)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[t][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  uint8_t *mine = lds + wave * kARegion;
  uint32_t mask = kI4BiasMask, base = kI4BiasBase;
  asm volatile("" : "+s"(mask), "+v"(base));
  const u32x4_t one = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
  const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, one);
  auto compute = [&](Step x) __attribute__((always_inline)) {
    if (ROWS == kSum && !x.here) return;
    // conversions stay with their own step: of several steps at once they would take twice the registers
#pragma unroll
    for (int t = 0; t < WT; ++t) asm volatile("" : "+v"(x.w[t]));
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
      for (int t = 0; t < WT; ++t)
#pragma unroll
        for (int q = 0; q < NG; ++q) {
          f32x4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = q * 4 / NG; j < (q + 1) * 4 / NG; ++j)
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], i4_biased(x.w[t][j], mask, base), p, 0, 0, 0);
          const float s = i4_scale_of(x.s[t], q, op.scale_bf16) * (ROWS == kSum ? x.weight : 1.0f);
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
    // Whole rounds of the ring without a branch, so that the compiler's waits count the requests in flight; those
    // past the last step ask for it once more (with a branch around each 1 x 5120, K = 5120 6.4 instead of 6.0 us).
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
    for (int t = 0; t < WT; ++t)
#pragma unroll
      for (int i = 0; i < MT; ++i) part[((wave * WT + t) * MT + i) * kLanes + lane] = acc[t][i];
  }
  __syncthreads();
  for (uint32_t x = tid; x < kLanes * MT * NT * (NW / KS); x += 64u * NW) {
    const uint32_t l = x % kLanes, i = x / kLanes % MT, at = x / (kLanes * MT), t = at % NT, w0 = at / NT * KS;
    f32x4_t c[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      c[h] = part[((w0 * WT + t * G + h) * MT + i) * kLanes + l];
#pragma unroll
      for (uint32_t w = 1; w < KS; ++w) c[h] += part[(((w0 + w) * WT + t * G + h) * MT + i) * kLanes + l];
    }
    const uint32_t col = (tile0 + at) * 16u + (l & 15u);
    if (col >= N) continue;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      const uint32_t m = i * 16u + 4u * (l >> 4) + j;
      if (m >= rows) continue;
      if constexpr (ROWS == kLists && !GATED) {
        op.Y[(uint64_t)pair_of(m) * N + col] = c[0][j];
      } else {
        const float y = GATED ? silu_times(c[0][j], c[G - 1][j]) : c[0][j];
        op.C[(uint64_t)(ROWS == kLists ? pair_of(m) : first + m) * op.ldc + col] = (uint16_t)bf16x2_rne(y, 0.0f);
      }
    }
  }
}

template <int MMAX, int NT, int KS, int DEPTH, bool GATED, int NG, bool ZEROS, bool BY_ROW, int ROWS>
hipError_t launch_kernel(const I4Operands &op, uint32_t count, uint32_t chunk, hipStream_t stream) {
  constexpr int NW = KS > kWaves ? KS : kWaves;
  constexpr uint32_t kCols = 16 * NT * (NW / KS);
  const Rest rest = {op.up.Z, op.C, op.Y, op.ids, op.order, op.offsets, op.weights, op.ldc, op.scale_bf16, op.top_k, op.E, chunk};
  hipLaunchKernelGGL((i4_skinny_kernel<NW, MMAX, NT, KS, DEPTH, GATED, NG, ZEROS, BY_ROW, ROWS>), dim3((op.N + kCols - 1u) / kCols, count),
                     dim3(64 * NW), 0, stream, op.w.W, op.w.S, op.A, op.K, op.N, ROWS == kDense ? op.M : op.T, op.lda, op.w.Z,
                     op.up.W, op.up.S, rest);
  return hipGetLastError();
}

template <int MMAX, int NT, int KS, int DEPTH, bool GATED, int NG, int ROWS>
hipError_t launch_group(const I4Operands &op, uint32_t count, uint32_t chunk, hipStream_t stream) {
  if (op.by_row)
    return op.w.Z ? launch_kernel<MMAX, NT, KS, DEPTH, GATED, NG, true, true, ROWS>(op, count, chunk, stream)
                  : launch_kernel<MMAX, NT, KS, DEPTH, GATED, NG, false, true, ROWS>(op, count, chunk, stream);
  return op.w.Z ? launch_kernel<MMAX, NT, KS, DEPTH, GATED, NG, true, false, ROWS>(op, count, chunk, stream)
                : launch_kernel<MMAX, NT, KS, DEPTH, GATED, NG, false, false, ROWS>(op, count, chunk, stream);
}

// `count`: chunks, pairs or tokens, the grid's second dimension; `chunk`: the first of them, of chunks
template <int MMAX, int NT, int KS, int DEPTH, bool GATED, int ROWS>
hipError_t launch_cfg(const I4Operands &op, uint32_t count, hipStream_t stream, uint32_t chunk = 0) {
  if (op.group == 128u) return launch_group<MMAX, NT, KS, DEPTH, GATED, 1, ROWS>(op, count, chunk, stream);
  if (op.group == 64u) return launch_group<MMAX, NT, KS, DEPTH, GATED, 2, ROWS>(op, count, chunk, stream);
  return launch_group<MMAX, NT, KS, DEPTH, GATED, 4, ROWS>(op, count, chunk, stream);
}

// Chunks (pairs, tokens) of one launch: the grid's second dimension holds 65535, and all its threads are half of 2^32
// at most.
uint32_t most_of(const I4Operands &op) {
  const uint32_t fit = mx_max_grid(64 * 16) / ((op.N + 15u) / 16u);
  return fit < 65535u ? fit : 65535u;
}

template <int MMAX, int NT, int DEPTH, bool GATED>
hipError_t launch_dense(const I4Operands &op, hipStream_t stream) {
  const uint32_t rows = most_of(op) * MMAX;
  for (uint32_t m = 0; m < op.M; m += rows) {
    I4Operands part = op;
    part.A = op.A + (uint64_t)m * op.lda;
    part.C = op.C + (uint64_t)m * op.ldc;
    part.M = op.M - m < rows ? op.M - m : rows;
    const hipError_t e = launch_cfg<MMAX, NT, kWaves, DEPTH, GATED, kDense>(part, (part.M + MMAX - 1u) / MMAX, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Steps in flight: two.  More keep further workgroups off the compute unit by their registers (1 x 5120, K = 5120 6.0
// us, with three 6.3, with four 6.4).
template <bool GATED>
hipError_t launch_rows(const I4Operands &op, bool wide, hipStream_t stream) {
  constexpr int kTwo = GATED ? 1 : 2;
  if (op.M <= 4u) return launch_dense<4, 1, 2, GATED>(op, stream);
  if (op.M <= 8u) return launch_dense<8, kTwo, 2, GATED>(op, stream);
  if (!wide) return launch_dense<16, kTwo, 2, GATED>(op, stream);
  return launch_dense<32, 2 * kTwo, 1, GATED>(op, stream);
}

}  // namespace

hipError_t launch_i4_skinny(const I4Operands &op, bool wide, hipStream_t stream) {
  return op.gated ? launch_rows<true>(op, wide, stream) : launch_rows<false>(op, wide, stream);
}

bool i4_experts_skinny_fit(const I4Operands &op) {
  const uint64_t pairs = (uint64_t)op.T * op.top_k;
  return (op.order ? i4_chunks(pairs, op.E, 16u) : (op.gated ? pairs : op.T)) <= most_of(op);
}

// With lists two waves share K and four such pairs stand side by side: with all eight on K a wave has a step or two,
// and a workgroup's start (its expert, its rows, their first values) takes longer than its work (33 tokens of 8 of 64
// experts, 2048 outputs, K = 1024 72 -> 27 us with two weight tiles for a wave, gated 1024 outputs, K = 2048 49 -> 33).
// Without, a workgroup has one row: four waves on K below 4096 (1 token, K = 2048 5.8 -> 5.5 us), eight from there on (K = 5120
// 7.8 -> 5.4); and a token's sum takes sixteen where its workgroups leave compute units idle (1 token, 2048 outputs 7.5
// -> 6.2 us).
hipError_t launch_i4_experts_skinny(const I4Operands &op, hipStream_t stream) {
  const uint32_t pairs = op.T * op.top_k;
  if (op.order) {
    const uint32_t chunks = (uint32_t)i4_chunks(pairs, op.E, 16u), most = most_of(op);
    for (uint32_t c = 0; c < chunks; c += most) {
      const uint32_t count = chunks - c < most ? chunks - c : most;
      const hipError_t e = op.gated ? launch_cfg<16, 1, 2, 2, true, kLists>(op, count, stream, c)
                                    : launch_cfg<16, 2, 2, 2, false, kLists>(op, count, stream, c);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  if (op.gated)
    return op.K < 4096u ? launch_cfg<4, 1, 4, 2, true, kPairs>(op, pairs, stream) : launch_cfg<4, 1, 8, 2, true, kPairs>(op, pairs, stream);
  return (uint64_t)((op.N + 15u) / 16u) * op.T <= 256u ? launch_cfg<4, 1, 16, 2, false, kSum>(op, op.T, stream)
                                                      : launch_cfg<4, 1, 8, 1, false, kSum>(op, op.T, stream);
}

}  // namespace wqd
