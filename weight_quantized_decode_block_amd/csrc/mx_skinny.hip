// Products with MXFP4 weights for few rows, for gfx950 (MI355X):
//
//   C[m,n] = bf16( sum_k a[m,k] w[n,k] ),  or with two weight matrices
//   C[m,n] = bf16( silu(sum_k a[m,k] wg[n,k]) * sum_k a[m,k] wu[n,k] ),
//
// a in BF16, MXFP8 or MXFP4 and w in MXFP4 (scale per 32 k on both sides),
// all sums in fp32.  The weights' bytes bound it: each is read once.
//
// A workgroup of 8 waves owns 16 weight rows (of both matrices in the gated
// form) and 16 * MT activation rows; its waves take the 128-k steps in turn and
// add their partial tiles in LDS, in wave order, at the end.  In a step lane
// (r, g) = (lane % 16, lane / 16) loads the 16 bytes of weight block g (32
// codes) of row r straight from memory and its scale byte:
//   * MXFP8 and MXFP4 activations: v_mfma_scale_f32_16x16x128_f8f6f4 takes the
//     codes and scale bytes as they are, the weights as its first operand.  It
//     wants 4-bit k = 32g .. 32g+31 from lane group g, and of 8-bit values
//     k = 16g .. 16g+15 and 64+16g .. 64+16g+15; the scale byte is that of
//     k block g on either side.
//   * BF16 activations: the codes become BF16 pairs, scaled in the conversion
//     (exact: two significand bits and a power of two), and instruction j of
//     four 16x16x32 ones takes k = 32g + 8j .. 32g + 8j + 7 of both sides.
// A lane keeps DEPTH steps in flight in registers; requests past the last step
// or row fall outside the buffer and come back as zeros, which add nothing.
// The result is 4 consecutive n of one m per lane.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_common.h"
#include "mx_product.h"
#include "wqd_internal.h"

namespace wqd {
namespace {

constexpr uint32_t kWaves = 8;
constexpr uint32_t kThreads = 64 * kWaves;
constexpr uint32_t kPastEnd = 0x80000000u;

template <MxFormat FMT, int MT>
struct StepRegs {
  u32x4_t w, wu;         // 32 weight codes of this lane's block (wu: up matrix)
  uint32_t ws, wus;      // their scale bytes
  ActRegs<FMT> a[MT];
};

template <MxFormat FMT, int MT, bool GATED, int DEPTH>
__global__ __launch_bounds__(kThreads) void mx_skinny_kernel(MxOperands op) {
  __shared__ f32x4_t part[GATED ? 2 : 1][kWaves][MT][64];
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = lane & 15u, g = lane >> 4;
  const uint32_t chunks = (op.M + 16u * MT - 1u) / (16u * MT);
  const uint32_t tile = blockIdx.x / chunks;
  const uint32_t n0 = tile * 16u, m0 = (blockIdx.x - tile * chunks) * (16u * MT);
  const uint32_t nb = op.K >> 5, steps = op.K >> 7;
  const uint32_t nrows = op.N - n0 < 16u ? op.N - n0 : 16u;
  const uint32_t mrows = op.M - m0 < 16u * MT ? op.M - m0 : 16u * MT;

  const __amdgpu_buffer_rsrc_t wr = rows_rsrc(op.W, n0, nrows, op.K >> 1, op.K >> 1);
  const __amdgpu_buffer_rsrc_t wsr = rows_rsrc(op.WS, n0, nrows, nb, nb);
  const __amdgpu_buffer_rsrc_t ur = rows_rsrc(GATED ? op.WU : op.W, n0, nrows, op.K >> 1, op.K >> 1);
  const __amdgpu_buffer_rsrc_t usr = rows_rsrc(GATED ? op.WUS : op.WS, n0, nrows, nb, nb);
  const uint32_t apitch = act_bytes<FMT>(op.lda), arow = act_bytes<FMT>(op.K);
  const __amdgpu_buffer_rsrc_t ar = rows_rsrc(op.A, m0, mrows, apitch, arow);
  const __amdgpu_buffer_rsrc_t asr = rows_rsrc(FMT == MxFormat::kBf16 ? op.A : op.AS, m0, mrows, nb, nb);

  auto load = [&](uint32_t s) __attribute__((always_inline)) {
    StepRegs<FMT, MT> x;
    const bool in = s < steps;
    const uint32_t wo = in ? r * (op.K >> 1) + s * 64u + g * 16u : kPastEnd;
    const uint32_t so = in ? r * nb + s * 4u + g : kPastEnd;
    x.w = __builtin_amdgcn_raw_buffer_load_b128(wr, wo, 0, 0);
    x.ws = __builtin_amdgcn_raw_buffer_load_b8(wsr, so, 0, 0);
    if constexpr (GATED) {
      x.wu = __builtin_amdgcn_raw_buffer_load_b128(ur, wo, 0, 0);
      x.wus = __builtin_amdgcn_raw_buffer_load_b8(usr, so, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint32_t m = 16u * t + r;
      // rows past the last one have an offset of their own past the end: the
      // pitch may be wider than the row
      const bool ok = in && m < mrows;
      const uint32_t ao = m * apitch;
      if constexpr (FMT == MxFormat::kBf16) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x.a[t].v[j] = __builtin_amdgcn_raw_buffer_load_b128(ar, ok ? ao + s * 256u + g * 64u + 16u * j : kPastEnd, 0, 0);
      } else {
        if constexpr (FMT == MxFormat::kFp8) {
          x.a[t].v[0] = __builtin_amdgcn_raw_buffer_load_b128(ar, ok ? ao + s * 128u + g * 16u : kPastEnd, 0, 0);
          x.a[t].v[1] = __builtin_amdgcn_raw_buffer_load_b128(ar, ok ? ao + s * 128u + 64u + g * 16u : kPastEnd, 0, 0);
        } else {
          x.a[t].v[0] = __builtin_amdgcn_raw_buffer_load_b128(ar, ok ? ao + s * 64u + g * 16u : kPastEnd, 0, 0);
        }
        x.a[t].s = __builtin_amdgcn_raw_buffer_load_b8(asr, ok ? m * nb + s * 4u + g : kPastEnd, 0, 0);
      }
    }
    return x;
  };

  f32x4_t acc[MT], accu[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = accu[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  StepRegs<FMT, MT> ring[DEPTH];
  uint32_t next = wave;
  mx_unroll<0, DEPTH>([&](auto d) __attribute__((always_inline)) {
    ring[decltype(d)::value] = load(next);
    next += kWaves;
  });
  const uint32_t mine = steps > wave ? (steps - wave + kWaves - 1u) / kWaves : 0u;
  for (uint32_t i = 0; i < mine; i += DEPTH)
    mx_unroll<0, DEPTH>([&](auto d) __attribute__((always_inline)) {
      StepRegs<FMT, MT> &x = ring[decltype(d)::value];
      WeightRegs<FMT> w(x.w, x.ws), wu;
      if constexpr (GATED) wu = WeightRegs<FMT>(x.wu, x.wus);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        acc[t] = mx_mfma<FMT>(w, x.a[t], acc[t]);
        if constexpr (GATED) accu[t] = mx_mfma<FMT>(wu, x.a[t], accu[t]);
      }
      x = load(next);
      next += kWaves;
    });

#pragma unroll
  for (int t = 0; t < MT; ++t) {
    part[0][wave][t][lane] = acc[t];
    if constexpr (GATED) part[1][wave][t][lane] = accu[t];
  }
  __syncthreads();
  for (uint32_t x = threadIdx.x; x < 64u * MT; x += kThreads) {
    const uint32_t t = x >> 6, l = x & 63u;
    f32x4_t c = part[0][0][t][l];
#pragma unroll
    for (uint32_t w = 1; w < kWaves; ++w) c += part[0][w][t][l];
    if constexpr (GATED) {
      f32x4_t u = part[1][0][t][l];
#pragma unroll
      for (uint32_t w = 1; w < kWaves; ++w) u += part[1][w][t][l];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = silu_times(c[i], u[i]);
    }
    const uint32_t m = m0 + 16u * t + (l & 15u), n = n0 + 4u * (l >> 4);
    if (m < op.M) store4(op, m, n, c);
  }
}

template <MxFormat FMT, int MT, bool GATED, int DEPTH>
hipError_t launch_cfg(const MxOperands &op, hipStream_t stream) {
  const uint32_t tiles = (op.N + 15u) / 16u;
  const uint32_t rows = kMxMaxGrid / tiles * 16u * MT;  // N <= 2^24, so at least one chunk
  for (uint32_t m = 0; m < op.M; m += rows) {
    const MxOperands part = mx_rows(op, FMT, m, rows);
    const uint32_t chunks = (part.M + 16u * MT - 1u) / (16u * MT);
    hipLaunchKernelGGL((mx_skinny_kernel<FMT, MT, GATED, DEPTH>), dim3(tiles * chunks), dim3(kThreads), 0, stream, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <MxFormat FMT, bool GATED>
hipError_t launch_fmt(const MxOperands &op, hipStream_t stream) {
  if (op.M <= 16u) return launch_cfg<FMT, 1, GATED, 4>(op, stream);
  if (op.M <= 32u) return launch_cfg<FMT, 2, GATED, 2>(op, stream);
  return launch_cfg<FMT, 4, GATED, FMT == MxFormat::kBf16 ? 1 : 2>(op, stream);
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
