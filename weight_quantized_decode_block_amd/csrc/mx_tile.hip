// Products with MXFP4 weights for many rows, for gfx950 (MI355X): the
// operations of mx_skinny.hip, bound by the matrix instructions.
//
// A workgroup of 8 waves owns BM x BN outputs (in the gated form BN / 2
// outputs of both matrices) and walks K in steps of 128.  Each wave owns a
// (BM / WM) x (BN / WN) part as 16 x 16 tiles: the weights are the matrix
// instruction's rows, the activations its columns, so a lane ends with four
// consecutive n of one m.
//
//   * Staging.  A step's codes go straight from memory to LDS (16 bytes per
//     lane, no registers), PRE steps ahead of their use, into NBUF = PRE + 1
//     buffers.  The unit is 16 rows x 64 bytes in one instruction.  Four
//     neighbouring lanes bring the four 16-byte pieces of a row: with the lanes
//     in a matrix operand's own order (neighbours in different rows) the same
//     transfers run at a quarter of the rate (37 instead of 120 to 146 GB/s per
//     compute unit from L2).  Piece p of row r lies in slot p ^ (r / 4) of the
//     row, so the 16 lanes that read one piece of 16 rows meet all 64 banks.
//     Rows past the matrix repeat its last row; their outputs are not stored.
//   * Scales.  16 bytes per row cover four steps; they are staged the same way
//     one group of four steps ahead.  A wave reads them once per group and
//     turns them so that byte t of a lane's register is its k block in step t,
//     which the matrix instruction's byte select takes directly.
//   * One barrier per step: before it a wave waits for its own transfers of the
//     step (later ones stay in flight) and for its LDS reads; after it the
//     buffer of the step before is free.
//   * Workgroups are dealt to the 8 XCDs in contiguous runs of tiles, and tiles
//     run down four tile rows before the next tile column, so the workgroups
//     that share an L2 at one time share rows of both operands.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_common.h"
#include "mx_product.h"
#include "wqd_internal.h"

namespace wqd {
namespace {

constexpr uint32_t kUnit = 1024;  // 16 rows x 64 bytes

template <MxFormat FMT>
constexpr uint32_t kActUnits = FMT == MxFormat::kBf16 ? 4 : (FMT == MxFormat::kFp8 ? 2 : 1);  // per 16 rows and step

typedef uint32_t rsrc_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ rsrc_t bytes_rsrc(const void *p, uint64_t offset, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p) + offset;
  const rsrc_t r = {(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a),
                    (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xffffu),
                    (uint32_t)__builtin_amdgcn_readfirstlane(bytes), 0x00020000u};
  return r;
}

// 16 bytes per lane from voff of the buffer to LDS byte `lds` + 16 * lane.
// The transfer has no destination registers; it is waited for by count
// (step_barrier), which the compiler's own waits could not do per buffer.
__device__ __forceinline__ void copy_to_lds(uint32_t lds, rsrc_t r, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(r)
               : "memory");
}

// Wait until at most N of this wave's transfers are in flight and its LDS
// reads have returned, then meet the other waves.
template <int N>
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// KS: groups of waves that take the steps in turn and add their sums at the
// end.  PP: the two halves of the waves, one of each per SIMD, run half a step
// apart, one reading LDS while the other has the matrix unit.
template <MxFormat FMT, int BM, int BN, int WM, int WN, int KS, int PRE, bool PP, bool GATED>
__global__ __launch_bounds__(64 * WM * WN * KS) void mx_tile_kernel(MxOperands op) {
  static_assert(!PP || (KS == 1 && WM * WN == 8), "two waves per SIMD");
  constexpr uint32_t kGroupWaves = WM * WN, kWaves = kGroupWaves * KS;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int NBUF = PRE + 1;
  constexpr uint32_t kWUnits = BN / 16, kAUnits = BM / 16 * kActUnits<FMT>;
  constexpr uint32_t kStep = (kWUnits + kAUnits) * kUnit, kStage = KS * kStep;
  static_assert(kWUnits % kGroupWaves == 0, "a wave's weight units are all of one matrix");
  constexpr int WU = kWUnits / kGroupWaves, AU = (kAUnits + kGroupWaves - 1) / kGroupWaves, ND = WU + AU;
  constexpr bool kActScales = FMT != MxFormat::kBf16;
  constexpr uint32_t kScaleRows = BN + (kActScales ? (BM + 63) / 64 * 64 : 0);  // whole transfers of 64 rows
  constexpr uint32_t kScaleStage = kScaleRows * 16;
  static_assert(BN % 64 == 0 && kScaleRows <= 64 * kWaves, "at most one scale transfer per wave");
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // NBUF stages, two scale stages
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t all_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t ks = KS == 1 ? 0u : all_wave / kGroupWaves, wave = all_wave - ks * kGroupWaves;
  const uint32_t r = lane & 15u, g = lane >> 4;
  constexpr uint32_t BNO = GATED ? BN / 2 : BN;  // outputs per tile row

  // tile of this workgroup
  const uint32_t tm = (op.M + BM - 1u) / BM, tn = (op.N + BNO - 1u) / BNO;
  const uint32_t total = tm * tn, xcd = blockIdx.x & 7u, q8 = total >> 3, rem = total & 7u;
  const uint32_t id = xcd * q8 + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
  const uint32_t band = id / (4u * tn), in_band = id - band * 4u * tn;
  const uint32_t band_rows = tm - band * 4u < 4u ? tm - band * 4u : 4u;
  const uint32_t col = in_band / band_rows;
  const uint32_t m0 = (band * 4u + in_band - col * band_rows) * BM, n0 = col * BNO;
  const uint32_t mlast = (op.M - m0 < (uint32_t)BM ? op.M - m0 : (uint32_t)BM) - 1u;
  const uint32_t nlast = (op.N - n0 < BNO ? op.N - n0 : BNO) - 1u;

  const uint32_t steps = op.K >> 7, nb = op.K >> 5, wpitch = op.K >> 1, apitch = act_bytes<FMT>(op.lda);
  const uint32_t stages = (steps + KS - 1u) / KS;

  // transfers of this wave for its group's step: weight units wave, wave +
  // kGroupWaves, ... and activation units likewise (where they do not come out
  // even, some are brought twice: every wave then has as many transfers in
  // flight as the waits count).  Gated: even units are the gate matrix, odd ones
  // the up matrix.
  const bool up = GATED && (wave & 1u);
  const rsrc_t wr = bytes_rsrc(up ? op.WU : op.W, (uint64_t)n0 * wpitch, (nlast + 1u) * wpitch);
  const rsrc_t ar = bytes_rsrc(op.A, (uint64_t)m0 * apitch, mlast * apitch + act_bytes<FMT>(op.K));
  const uint32_t lrow = lane >> 2, lpiece = ((lane & 3u) ^ (lane >> 4)) * 16u;  // this lane's row and piece of a unit
  uint32_t woff[WU], aoff[AU];
#pragma unroll
  for (int i = 0; i < WU; ++i) {
    const uint32_t u = wave + kGroupWaves * i;
    const uint32_t row = (GATED ? u >> 1 : u) * 16u + lrow;
    woff[i] = (row < nlast ? row : nlast) * wpitch + lpiece;
  }
#pragma unroll
  for (int i = 0; i < AU; ++i) {
    const uint32_t u = (wave + kGroupWaves * i) % kAUnits;
    const uint32_t row = u / kActUnits<FMT> * 16u + lrow;
    aoff[i] = (row < mlast ? row : mlast) * apitch + (u % kActUnits<FMT>) * 64u + lpiece;
  }
  // scale rows 64 w .. 64 w + 63 of wave w: weights (gated: gate, then up), then activations
  const uint32_t srow = all_wave * 64u + lane;
  const bool s_act = all_wave * 64u >= (uint32_t)BN, s_up = GATED && !s_act && all_wave * 64u >= BNO;
  const bool s_any = all_wave * 64u < kScaleRows;
  const rsrc_t sr = s_act ? bytes_rsrc(op.AS, (uint64_t)m0 * nb, (mlast + 1u) * nb)
                          : bytes_rsrc(s_up ? op.WUS : op.WS, (uint64_t)n0 * nb, (nlast + 1u) * nb);
  const uint32_t s_in = s_act ? srow - BN : (s_up ? srow - BNO : srow);
  const uint32_t s_last = s_act ? mlast : nlast;
  const uint32_t soff = (s_in < s_last ? s_in : s_last) * nb;

  auto issue = [&](uint32_t stage, uint32_t buf) __attribute__((always_inline)) {
    uint32_t s = stage * KS + ks;
    if (KS > 1) s = s < steps ? s : steps - 1u;  // a step too many is brought but not computed
    const uint32_t base = lds0 + buf * kStage + ks * kStep;
#pragma unroll
    for (int i = 0; i < WU; ++i) copy_to_lds(base + (wave + i * kGroupWaves) * kUnit, wr, woff[i] + s * 64u);
#pragma unroll
    for (int i = 0; i < AU; ++i)
      copy_to_lds(base + (kWUnits + (wave + kGroupWaves * i) % kAUnits) * kUnit, ar, aoff[i] + s * 64u * kActUnits<FMT>);
  };
  // the 16 scale bytes from step 4q on, or the row's last 16 where fewer are left (nb >= 16)
  auto issue_scales = [&](uint32_t q) __attribute__((always_inline)) {
    const uint32_t at = 16u * q + 16u <= nb ? 16u * q : nb - 16u;
    if (s_any) copy_to_lds(lds0 + NBUF * kStage + (q & 1u) * kScaleStage + all_wave * kUnit, sr, soff + at);
  };

  const uint32_t wm = wave / WN, wn = wave % WN;  // this wave's part of the tile
  f32x4_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // byte g of each of four dwords, as one register
  const uint32_t pick = 0x0c0c0000u | (g + 4u) << 8 | g;
  uint32_t wsc[NT], asc[kActScales ? MT : 1];
  auto turn = [&](u32x4_t d, uint32_t shift) __attribute__((always_inline)) {
    const uint32_t lo = __builtin_amdgcn_perm(d.y, d.x, pick), hi = __builtin_amdgcn_perm(d.w, d.z, pick);
    return (lo | hi << 16) >> shift;
  };
  auto read_scales = [&](uint32_t q) __attribute__((always_inline)) {
    const uint8_t *p = lds + NBUF * kStage + (q & 1u) * kScaleStage;
    // 8 bits a step, 4 bytes a step; a wave group's first step is byte 0
    const uint32_t shift = (16u * q + 16u <= nb ? 0u : (16u * q + 16u - nb) * 2u) + 8u * ks;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint32_t t = wn * NT + i;
      const uint32_t row = (GATED ? (t & 1u) * BNO + (t >> 1) * 16u : t * 16u) + r;
      wsc[i] = turn(*reinterpret_cast<const u32x4_t *>(p + row * 16u), shift);
    }
    if constexpr (kActScales) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
        asc[j] = turn(*reinterpret_cast<const u32x4_t *>(p + (BN + (wm * MT + j) * 16u + r) * 16u), shift);
    }
  };

  // operands of a step from LDS, and the products on them; T: the scales' byte
  const uint32_t mine = r * 64u + (g ^ (r >> 2)) * 16u;  // piece g of row r of a unit
  auto read_w = [&](uint32_t buf, auto T, WeightRegs<FMT> (&w)[NT]) __attribute__((always_inline)) {
    constexpr int t = decltype(T)::value;
    const uint8_t *p = lds + buf * kStage + ks * kStep + wn * NT * kUnit + mine;
#pragma unroll
    for (int i = 0; i < NT; ++i)
      w[i] = WeightRegs<FMT>(*reinterpret_cast<const u32x4_t *>(p + i * kUnit),
                             kActScales ? wsc[i] : (wsc[i] >> (8 * t)) & 255u);
  };
  auto read_a = [&](uint32_t buf, int j) __attribute__((always_inline)) {
    const uint8_t *p = lds + buf * kStage + ks * kStep + (kWUnits + wm * MT * kActUnits<FMT>) * kUnit;
    ActRegs<FMT> a;
    if constexpr (FMT == MxFormat::kBf16) {
#pragma unroll
      for (uint32_t h = 0; h < 4; ++h)  // k 32g .. 32g + 31 are the four pieces of unit g
        a.v[h] = *reinterpret_cast<const u32x4_t *>(p + (j * 4 + g) * kUnit + r * 64u + (h ^ (r >> 2)) * 16u);
    } else {
#pragma unroll
      for (uint32_t h = 0; h < kActUnits<FMT>; ++h)
        a.v[h] = *reinterpret_cast<const u32x4_t *>(p + (j * kActUnits<FMT> + h) * kUnit + mine);
      a.s = asc[j];
    }
    return a;
  };

  issue_scales(0);
  mx_unroll<0, PRE>([&](auto d) __attribute__((always_inline)) {
    constexpr uint32_t s = decltype(d)::value;
    if (s < stages) issue(s, s);
  });
  uint32_t buf = 0;
  constexpr int kGroup = 4 / KS;  // stages per group of four steps
  if constexpr (PP) {
    // Stage s has arrived for everybody before the barrier that ends the read
    // half of stage s - 1; the second half of the waves starts one barrier late.
    if (PRE <= stages)
      step_barrier<(PRE - 1) * ND>();
    else
      step_barrier<0>();
    if (wave >= 4u) __builtin_amdgcn_s_barrier();
    for (uint32_t s0 = 0; s0 < stages; s0 += kGroup) {
      mx_unroll<0, kGroup>([&](auto T) __attribute__((always_inline)) {
        constexpr int t = decltype(T)::value;
        const uint32_t s = s0 + t;
        if (s < stages) {
          if constexpr (t == 0) {
            read_scales(s0 / kGroup);
            __builtin_amdgcn_sched_barrier(0);  // their registers are free again before the operands' are taken
          }
          WeightRegs<FMT> w[NT];
          ActRegs<FMT> a[MT];
          read_w(buf, T, w);
#pragma unroll
          for (int j = 0; j < MT; ++j) a[j] = read_a(buf, j);
          if constexpr (t == 0) {
            if (s0 + kGroup < stages) issue_scales(s0 / kGroup + 1u);
          }
          if (s + PRE < stages) {
            issue(s + PRE, buf == 0 ? NBUF - 1 : buf - 1);
            step_barrier<(PRE - 1) * ND>();
          } else {
            step_barrier<0>();
          }
          __builtin_amdgcn_sched_barrier(0);
          __builtin_amdgcn_s_setprio(1);
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[i][j] = mx_mfma<FMT, t>(w[i], a[j], acc[i][j]);
          __builtin_amdgcn_s_setprio(0);
          __builtin_amdgcn_sched_barrier(0);
          __builtin_amdgcn_s_barrier();
          buf = buf + 1u == (uint32_t)NBUF ? 0u : buf + 1u;
        }
      });
    }
    if (wave < 4u) __builtin_amdgcn_s_barrier();
  } else {
    for (uint32_t s0 = 0; s0 < stages; s0 += kGroup) {
      mx_unroll<0, kGroup>([&](auto T) __attribute__((always_inline)) {
        constexpr int t = decltype(T)::value;
        const uint32_t s = s0 + t;
        if (s < stages) {
          // the transfers of stages s + 1 .. s + PRE - 1 may still be in flight
          // (at a group's start no more than a group's, so that its scales have arrived)
          if (s + PRE <= stages)
            step_barrier<(t == 0 && PRE - 1 > kGroup ? kGroup : PRE - 1) * ND>();
          else
            step_barrier<0>();
          if constexpr (t == 0) {
            read_scales(s0 / kGroup);
            if (s0 + kGroup < stages) issue_scales(s0 / kGroup + 1u);
          }
          if (s + PRE < stages) issue(s + PRE, buf == 0 ? NBUF - 1 : buf - 1);
          if (KS == 1 || s * KS + ks < steps) {
            WeightRegs<FMT> w[NT];
            read_w(buf, std::integral_constant<int, t * KS>{}, w);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              const ActRegs<FMT> a = read_a(buf, j);
#pragma unroll
              for (int i = 0; i < NT; ++i) acc[i][j] = mx_mfma<FMT, t * KS>(w[i], a, acc[i][j]);
            }
          }
          buf = buf + 1u == (uint32_t)NBUF ? 0u : buf + 1u;
        }
      });
    }
  }

  if constexpr (KS > 1) {  // the groups' sums, in order, onto the first group's
    static_assert((KS - 1) * BM * BN * 4 <= NBUF * kStage, "partial sums fit the stages");
    step_barrier<0>();
    f32x4_t *part = reinterpret_cast<f32x4_t *>(lds);
    if (ks > 0u) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) part[(((all_wave - kGroupWaves) * NT + i) * MT + j) * 64u + lane] = acc[i][j];
    }
    step_barrier<0>();
    if (ks > 0u) return;
#pragma unroll
    for (int k = 1; k < KS; ++k)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] += part[((((k - 1) * kGroupWaves + wave) * NT + i) * MT + j) * 64u + lane];
  }

  // the lane again, so that nothing of it stays in registers through the loop
  const uint32_t l = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)), ln = (l >> 4) * 4u;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const uint32_t m = m0 + (wm * MT + j) * 16u + (l & 15u);
    if constexpr (GATED) {
#pragma unroll
      for (int i = 0; i < NT; i += 2) {
        f32x4_t c;
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = silu_times(acc[i][j][e], acc[i + 1][j][e]);
        const uint32_t n = n0 + (wn * NT + i) * 8u + ln;
        if (m < op.M) store4(op.out, op.N, m, n, c);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint32_t n = n0 + (wn * NT + i) * 16u + ln;
        if (m < op.M) store4(op.out, op.N, m, n, acc[i][j]);
      }
    }
  }
}

template <MxFormat FMT, int BM, int BN, int WM, int WN, int KS, int PRE, bool PP, bool GATED>
hipError_t launch_cfg(const MxOperands &op, hipStream_t stream) {
  constexpr auto kern = mx_tile_kernel<FMT, BM, BN, WM, WN, KS, PRE, PP, GATED>;
  constexpr uint32_t kLds = (PRE + 1) * KS * (BN / 16 + BM / 16 * kActUnits<FMT>) * kUnit +
                            2 * (BN + (FMT == MxFormat::kBf16 ? 0 : (BM + 63) / 64 * 64)) * 16;
  static_assert(kLds <= 160 * 1024, "one workgroup's LDS");
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  if (attr != hipSuccess) return attr;
  const uint32_t bno = GATED ? BN / 2 : BN;
  const uint32_t tn = (op.N + bno - 1u) / bno;
  const uint32_t rows = kMxMaxGrid / tn * BM;  // a launch holds fewer than 2^32 threads
  for (uint32_t m = 0; m < op.M; m += rows) {
    const MxOperands part = mx_rows(op, FMT, m, rows);
    const uint32_t grid = tn * ((part.M + BM - 1u) / BM);
    hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * WM * WN * KS), kLds, stream, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <MxFormat FMT, bool GATED>
hipError_t launch_fmt(const MxOperands &op, hipStream_t stream) {
  if constexpr (FMT == MxFormat::kBf16)
    return launch_cfg<FMT, 128, 256, 2, 4, 1, 2, true, GATED>(op, stream);
  else if constexpr (FMT == MxFormat::kFp8)
    return launch_cfg<FMT, 256, 256, 4, 2, 1, 2, true, GATED>(op, stream);
  else
    return launch_cfg<FMT, 256, 256, 4, 2, 1, 3, true, GATED>(op, stream);
}

}  // namespace

bool mx_tile_supports(const MxOperands &op) { return op.K >= 512u; }

hipError_t launch_mx_tile(const MxOperands &op, MxFormat fmt, bool gated, hipStream_t stream) {
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
