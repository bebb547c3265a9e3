// Products with MXFP4 weights for few rows, for gfx950 (MI355X):
//
//   C[m,n] = bf16( sum_k a[m,k] w[n,k] ),  or with two weight matrices
//   C[m,n] = bf16( silu(sum_k a[m,k] wg[n,k]) * sum_k a[m,k] wu[n,k] ),
//
// a in BF16, MXFP8 or MXFP4 and w in MXFP4 (scale per 32 k on both sides),
// all sums in fp32.  The weights' bytes bound it: each is read once.
//
// A workgroup of 8 waves owns 16 * NT weight rows (of both matrices in the
// gated form) and up to MMAX activation rows, and walks K in segments of 1024:
// wave w takes the segment's w-th 128-k step, and the waves' partial tiles are
// added in LDS, in wave order, at the end.
//   * A wave loads its own step's weights, DEPTH segments ahead, four
//     neighbouring lanes the four 16-byte pieces of a row, and turns them through
//     a KB of LDS of its own into the matrix operand's order: lane (r, g) =
//     (lane % 16, lane / 16) takes k block g (32 codes) of row r.  Loaded in that
//     order at once (neighbours in different rows) the weights come at a quarter
//     of the rate.
//   * Everything else of a segment, the activations and both sides' scale
//     bytes, goes through LDS (two buffers, one barrier per segment), loaded
//     in whole 16-byte pieces and dwords and DEPTH segments ahead in registers.
//     Loaded by each lane for itself, as the weights are, these small pieces
//     cost as many vector-memory instructions as the weights several times
//     over, and those bound the kernel.
//   * MXFP8 and MXFP4 activations: v_mfma_scale_f32_16x16x128_f8f6f4 takes the
//     codes and scale bytes as they are, the weights as its first operand.  It
//     wants 4-bit k = 32g .. 32g+31 from lane group g, and of 8-bit values
//     k = 16g .. 16g+15 and 64+16g .. 64+16g+15; the scale byte is that of
//     k block g on either side.
//   * BF16 activations: the codes become BF16 pairs, scaled in the conversion
//     (exact: two significand bits and a power of two), and instruction j of
//     four 16x16x32 ones takes k = 32g + 8j .. 32g + 8j + 7 of both sides.
// Requests past the last step or row fall outside the buffer and come back as
// zeros, which add nothing.  A lane ends with 4 consecutive n of one m.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/wqd.h"
#include "mx_common.h"
#include "mx_product.h"
#include "wqd_internal.h"

namespace wqd {
namespace {

constexpr uint32_t kPastEnd = 0x80000000u;
// Waves of a workgroup, and segments in flight: 4 or 16 waves, and 1, 3 or 4
// segments, were all slower where this was chosen, 8 x 5120, K = 17408, MXFP8
// (12.2 us now).
constexpr int NW = 8, DEPTH = 2;

// Bytes of an activation row in a step.
template <MxFormat FMT>
constexpr uint32_t kStepBytes = FMT == MxFormat::kBf16 ? 256 : (FMT == MxFormat::kFp8 ? 128 : 64);

// Place of 16-byte piece p of activation row m.  BF16: the row's k block of 32
// is four pieces, so pieces 4 apart are read together; rows 4-11 turn them among
// places 0-7 and the others among 8-15.
template <MxFormat FMT>
__device__ __forceinline__ uint32_t act_piece(uint32_t m, uint32_t p) {
  if constexpr (FMT != MxFormat::kBf16) return p;
  const uint32_t r = m & 15u;
  return p ^ (r < 4u ? r + 8u : (r < 12u ? r - 4u : r));
}

template <MxFormat FMT, int MMAX, int NT, bool GATED>
__global__ __launch_bounds__(64 * NW) void mx_skinny_kernel(const uint8_t *__restrict__ W,
                                                             const uint8_t *__restrict__ WS,
                                                             const uint8_t *__restrict__ A, uint32_t K, uint32_t M,
                                                             uint32_t N, uint32_t lda, const uint8_t *__restrict__ AS,
                                                             const uint8_t *__restrict__ WU,
                                                             const uint8_t *__restrict__ WUS, MxOut out) {
  constexpr int MT = (MMAX + 15) / 16, G = GATED ? 2 : 1, WT = NT * G;  // 16-row tiles: activations, matrices, weights
  constexpr bool kActScales = FMT != MxFormat::kBf16;
  constexpr uint32_t kWaves = NW, kThreads = 64 * NW;
  constexpr uint32_t kRowBytes = NW * kStepBytes<FMT>;                     // of a segment's activation row
  constexpr uint32_t kScaleBytes = 4 * NW, kScalePitch = kScaleBytes + 4;  // of a segment's scale row
  // A 16-byte LDS read serves lanes 0-3, 12-15, 20-27 (then 4-11, 16-19, 28-31)
  // together: rows 0-3 and 12-15 of one piece and 4-11 of the next k block's.
  // Quantised rows 32 bytes longer than the segment, and BF16 rows with their
  // pieces' places turned by the row (act_piece), then meet all 64 banks: 16 x
  // 17408, K = 5120, MXFP8 16.6 -> 16.3 us against rows 16 bytes longer.
  constexpr uint32_t kPitch = kRowBytes + (FMT == MxFormat::kBf16 ? 0 : 32), kPieces = kRowBytes / 16;
  constexpr uint32_t kARegion = MMAX * kPitch;
  constexpr uint32_t kWsRows = 16 * WT, kScaleRows = kWsRows + (kActScales ? MMAX : 0);  // kScalePitch each
  constexpr uint32_t kBuffer = (kARegion + kScaleRows * kScalePitch + 15) / 16 * 16;
  constexpr int SA = (MMAX * kPieces + kThreads - 1) / kThreads, SS = (kScaleRows + 63) / 64;
  constexpr uint32_t kParts = kWaves * WT * MT * 1024;
  constexpr uint32_t kTurn = 2 * kBuffer;  // each wave's own KB per weight tile
  constexpr uint32_t kLds = kTurn + NW * WT * 1024 > kParts ? kTurn + NW * WT * 1024 : kParts;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];

  const uint32_t tid = threadIdx.x, lane = tid & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t r = lane & 15u, g = lane >> 4;
  const uint32_t chunks = (M + MMAX - 1u) / MMAX;
  const uint32_t tile = blockIdx.x / chunks;
  const uint32_t n0 = tile * 16u * NT, m0 = (blockIdx.x - tile * chunks) * MMAX;
  const uint32_t nb = K >> 5, steps = K >> 7, nseg = (steps + NW - 1u) / NW, wpitch = K >> 1;
  const uint32_t nrows = N - n0 < 16u * NT ? N - n0 : 16u * NT;
  const uint32_t mrows = M - m0 < (uint32_t)MMAX ? M - m0 : (uint32_t)MMAX;
  const uint32_t apitch = act_bytes<FMT>(lda), arow = act_bytes<FMT>(K);

  const __amdgpu_buffer_rsrc_t ar = rows_rsrc(A, m0, mrows, apitch, arow);
  const __amdgpu_buffer_rsrc_t wr = rows_rsrc(W, n0, nrows, wpitch, wpitch);
  const __amdgpu_buffer_rsrc_t ur = rows_rsrc(GATED ? WU : W, n0, nrows, wpitch, wpitch);

  // scale rows of this wave's staging slots: weight rows (gated: 16 of the gate
  // matrix, 16 of the up matrix, ...), then activation rows, 64 / NW per slot, so
  // a slot's matrix is the same for the wave.  soff: this lane's first byte, or
  // past the end.
  __amdgpu_buffer_rsrc_t sr[SS];
  uint32_t soff[SS];
#pragma unroll
  for (int u = 0; u < SS; ++u) {
    constexpr uint32_t kRows = 64 / NW, kSlots = 16 / kRows;  // rows of a slot, slots of a tile
    const uint32_t slot = wave + (uint32_t)u * kWaves, t = slot / kSlots;
    const bool act = kActScales && t >= (uint32_t)WT;
    const uint8_t *p = act ? AS : (GATED && (t & 1u) ? WUS : WS);
    const uint32_t rows = act ? mrows : (t < (uint32_t)WT ? nrows : 0u);
    const uint32_t row = (act ? slot * kRows - kWsRows : t / G * 16u + slot % kSlots * kRows) + lane / NW;
    sr[u] = rows_rsrc(p, act ? m0 : n0, rows > 0u ? rows : 1u, nb, nb);
    soff[u] = row < rows ? row * nb + lane % NW * 4u : kPastEnd;
  }
  const uint32_t sbyte = lane % NW * 4u;

  // weights of segment i for this lane: tile t of each matrix
  struct WSeg {
    u32x4_t v[WT];
  };
  auto load_w = [&](uint32_t i) __attribute__((always_inline)) {
    WSeg x;
    const uint32_t s = i * NW + wave;
    const bool in = s < steps;
#pragma unroll
    for (int t = 0; t < WT; ++t) {
      const uint32_t o = in ? ((uint32_t)(t / G) * 16u + (lane >> 2)) * wpitch + s * 64u + (lane & 3u) * 16u : kPastEnd;
      x.v[t] = __builtin_amdgcn_raw_buffer_load_b128(GATED && (t & 1) ? ur : wr, o, 0, 0);
    }
    return x;
  };
  // staged pieces of segment i for this thread
  struct SSeg {
    u32x4_t a[SA];
    uint32_t s[SS];
  };
  auto load_s = [&](uint32_t i) __attribute__((always_inline)) {
    SSeg x;
#pragma unroll
    for (int u = 0; u < SA; ++u) {
      const uint32_t p = tid + (uint32_t)u * kThreads, m = p / kPieces;
      const uint32_t b = i * kRowBytes + (p % kPieces) * 16u;  // byte of the row
      x.a[u] = __builtin_amdgcn_raw_buffer_load_b128(ar, m < mrows && b < arow ? m * apitch + b : kPastEnd, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < SS; ++u) {
      const uint32_t b = i * kScaleBytes;
      x.s[u] = __builtin_amdgcn_raw_buffer_load_b32(sr[u], b + sbyte < nb ? soff[u] + b : kPastEnd, 0, 0);
    }
    return x;
  };
  auto store_s = [&](const SSeg &x, uint32_t buf) __attribute__((always_inline)) {
    uint8_t *p0 = lds + buf * kBuffer;
#pragma unroll
    for (int u = 0; u < SA; ++u) {
      const uint32_t p = tid + (uint32_t)u * kThreads, m = p / kPieces;
      if (m < (uint32_t)MMAX)
        *reinterpret_cast<u32x4_t *>(p0 + m * kPitch + act_piece<FMT>(m, p % kPieces) * 16u) = x.a[u];
    }
#pragma unroll
    for (int u = 0; u < SS; ++u) {
      const uint32_t p = tid + (uint32_t)u * kThreads;
      if (p < kScaleRows * NW)
        *reinterpret_cast<uint32_t *>(p0 + kARegion + p / NW * kScalePitch + p % NW * 4u) = x.s[u];
    }
  };

  f32x4_t acc[WT][MT];
#pragma unroll
  for (int t = 0; t < WT; ++t)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[t][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  auto compute = [&](const WSeg &x, uint32_t buf) __attribute__((always_inline)) {
    const uint8_t *p0 = lds + buf * kBuffer, *ps = p0 + kARegion + wave * 4u + g;
    uint8_t *turn = lds + kTurn + wave * (WT * 1024u);
#pragma unroll
    for (int t = 0; t < WT; ++t)
      *reinterpret_cast<u32x4_t *>(turn + t * 1024 + unit_byte(lane >> 2, lane & 3u)) = x.v[t];
    WeightCodes w[WT];
#pragma unroll
    for (int t = 0; t < WT; ++t) {
      w[t].v = *reinterpret_cast<const u32x4_t *>(turn + t * 1024 + unit_byte(r, g));
      w[t].s = ps[(t * 16u + r) * kScalePitch];
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      // rows past the last staged one repeat row MMAX - 1: their outputs are not stored
      const uint32_t m = MMAX % 16 == 0 ? j * 16u + r : (j * 16u + r < MMAX ? j * 16u + r : MMAX - 1u);
      const uint8_t *pa = p0 + m * kPitch;
      ActRegs<FMT> a;
      if constexpr (FMT == MxFormat::kBf16) {
#pragma unroll
        for (uint32_t h = 0; h < 4; ++h)
          a.v[h] = *reinterpret_cast<const u32x4_t *>(pa + act_piece<FMT>(m, wave * 16u + g * 4u + h) * 16u);
      } else {
        a.v[0] = *reinterpret_cast<const u32x4_t *>(pa + wave * kStepBytes<FMT> + g * 16u);
        if constexpr (FMT == MxFormat::kFp8)
          a.v[1] = *reinterpret_cast<const u32x4_t *>(pa + wave * 128u + 64u + g * 16u);
        a.s = ps[(kWsRows + m) * kScalePitch];
      }
#pragma unroll
      for (int t = 0; t < WT; ++t) acc[t][j] = mx_mfma<FMT>(WeightRegs<FMT>(w[t]), a, acc[t][j]);
    }
  };

  // segment i + 1 is written to LDS while segment i is computed, so the staged
  // pieces' ring is one ahead of the weights'
  SSeg first = load_s(0), sring[DEPTH];
  WSeg wring[DEPTH];
  mx_unroll<0, DEPTH>([&](auto d) __attribute__((always_inline)) {
    wring[decltype(d)::value] = load_w(decltype(d)::value);
    sring[decltype(d)::value] = load_s(decltype(d)::value + 1);
  });
  store_s(first, 0);
  uint32_t i = 0;
  auto segment = [&](auto d, auto more) __attribute__((always_inline)) {
    constexpr int D = decltype(d)::value;
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's LDS accesses
    __builtin_amdgcn_s_barrier();
    compute(wring[D], i & 1u);
    store_s(sring[D], (i + 1u) & 1u);
    if constexpr (decltype(more)::value) {
      wring[D] = load_w(i + DEPTH);
      sring[D] = load_s(i + 1u + DEPTH);
    }
    ++i;
  };
  // whole rounds of the ring without a branch, so that the compiler's waits
  // count the requests in flight exactly; the rest requests nothing
  while (i + DEPTH <= nseg)
    mx_unroll<0, DEPTH>([&](auto d) __attribute__((always_inline)) { segment(d, std::true_type{}); });
  mx_unroll<0, DEPTH>([&](auto d) __attribute__((always_inline)) {
    if (i < nseg) segment(d, std::false_type{});
  });

  __syncthreads();
  f32x4_t *part = reinterpret_cast<f32x4_t *>(lds);
#pragma unroll
  for (int t = 0; t < WT; ++t)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[((wave * WT + t) * MT + j) * 64u + lane] = acc[t][j];
  __syncthreads();
  for (uint32_t x = tid; x < 64u * NT * MT; x += kThreads) {
    const uint32_t l = x & 63u, j = (x >> 6) % MT, t = (x >> 6) / MT;
    f32x4_t c = part[(t * G * MT + j) * 64u + l];
#pragma unroll
    for (uint32_t w = 1; w < kWaves; ++w) c += part[((w * WT + t * G) * MT + j) * 64u + l];
    if constexpr (GATED) {
      f32x4_t u = part[((t * G + 1) * MT + j) * 64u + l];
#pragma unroll
      for (uint32_t w = 1; w < kWaves; ++w) u += part[((w * WT + t * G + 1) * MT + j) * 64u + l];
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = silu_times(c[e], u[e]);
    }
    const uint32_t m = m0 + 16u * j + (l & 15u), n = n0 + 16u * t + 4u * (l >> 4);
    if (m < m0 + mrows) store4(out, N, m, n, c);
  }
}

template <MxFormat FMT, int MMAX, int NT, bool GATED>
hipError_t launch_cfg(const MxOperands &op, hipStream_t stream) {
  const uint32_t tiles = (op.N + 16u * NT - 1u) / (16u * NT);
  constexpr uint32_t kMaxGrid = mx_max_grid(64 * NW);
  static_assert(kMaxGrid >= WQD_MX_MAX_ROWS / (16u * NT), "a launch holds the widest chunk of rows");
  const uint32_t rows = kMaxGrid / tiles * MMAX;
  for (uint32_t m = 0; m < op.M; m += rows) {
    const MxOperands part = mx_rows(op, FMT, m, rows);
    const uint32_t chunks = (part.M + MMAX - 1u) / MMAX;
    hipLaunchKernelGGL((mx_skinny_kernel<FMT, MMAX, NT, GATED>), dim3(tiles * chunks), dim3(64 * NW), 0, stream,
                       static_cast<const uint8_t *>(part.W), static_cast<const uint8_t *>(part.WS),
                       static_cast<const uint8_t *>(part.A), part.K, part.M, part.N, part.lda,
                       static_cast<const uint8_t *>(part.AS), static_cast<const uint8_t *>(part.WU),
                       static_cast<const uint8_t *>(part.WUS), part.out);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Activation rows of a workgroup: the least of 2, 4, 8, 16 and 32 that hold M
// (32 at a time above).  Rows that are not there are staged and multiplied all
// the same: 1 x 5120, K = 5120, BF16 5.6 us with 2 rows, 8.4 with 16.
// Weight rows: 16, and from 9 activation rows on 32, over which the activations'
// pass through LDS is shared (16 rows: 5120 outputs, K = 17408, BF16 30.1 -> 23.3
// us; 17408 outputs, K = 5120, MXFP8 17.5 -> 16.5).  The gated form already has
// two matrices' 16 rows; twice that is slower (30.4 against 28.0 us).
template <MxFormat FMT, bool GATED>
hipError_t launch_fmt(const MxOperands &op, hipStream_t stream) {
  constexpr int kWide = GATED ? 1 : 2;
  if (op.M <= 2u) return launch_cfg<FMT, 2, 1, GATED>(op, stream);
  if (op.M <= 4u) return launch_cfg<FMT, 4, 1, GATED>(op, stream);
  if (op.M <= 8u) return launch_cfg<FMT, 8, 1, GATED>(op, stream);
  if (op.M <= 16u) return launch_cfg<FMT, 16, kWide, GATED>(op, stream);
  return launch_cfg<FMT, 32, kWide, GATED>(op, stream);
}

}  // namespace

hipError_t launch_mx_skinny(const MxOperands &op, MxFormat fmt, bool gated, hipStream_t stream) {
  switch (fmt) {
    case MxFormat::kBf16:
      return gated ? launch_fmt<MxFormat::kBf16, true>(op, stream) : launch_fmt<MxFormat::kBf16, false>(op, stream);
    case MxFormat::kFp8:
      return gated ? launch_fmt<MxFormat::kFp8, true>(op, stream) : launch_fmt<MxFormat::kFp8, false>(op, stream);
    default:
      return gated ? launch_fmt<MxFormat::kFp4, true>(op, stream) : launch_fmt<MxFormat::kFp4, false>(op, stream);
  }
}

}  // namespace wqd
