// Products with MXFP4 weights for many rows, for gfx950 (MI355X): the
// operations of mx_skinny.hip, bound by the matrix instructions.
//
// A workgroup owns BM x BN outputs (in the gated form BN / 2 outputs of both
// matrices) and walks K in steps of 128.  Each wave owns a (BM / WM) x (BN / WN)
// part as 16 x 16 tiles: the weights are the matrix instruction's rows, the
// activations its columns, so a lane ends with four consecutive n of one m.
//
//   * Staging.  Codes go straight from memory to LDS (16 bytes per lane, no
//     registers), PRE stages ahead of their use, into PRE + 1 buffers.  A
//     transfer is 16 rows x 64 bytes, four neighbouring lanes the four pieces of
//     a row: with the lanes in a matrix operand's own order (neighbours in
//     different rows) the same transfers run at a quarter of the rate (37
//     instead of 120 to 146 GB/s per compute unit from L2).  4-bit codes of one
//     step are half a 128-byte line per row; where a stage is two steps they are
//     brought together, 8 rows x 128 bytes a transfer (transfers alone 95
//     instead of 54 GB/s per compute unit, 128 x 128 tiles of 4-bit codes on
//     both sides 435 -> 377 ns a step).  Rows past the matrix repeat its last
//     row; their outputs are not stored.
//   * Scales.  16 bytes per row cover four steps; they are staged the same way
//     one group of four steps ahead (of K below 512, whose rows of scales are
//     shorter, before the first step).  A wave reads them once per group and
//     turns them so that byte t of a lane's register is its k block in step t,
//     which the matrix instruction's byte select takes directly.
//   * A wave waits for its own transfers of a stage (later ones stay in flight)
//     and for its LDS reads before the barrier that opens the stage; after it
//     the buffer of the stage before is free.
//   * Large tiles run the two halves of the waves half a step apart (kHalves):
//     4096 x 17408, K = 5120, MXFP8 380 -> 312 us; 1000 x 5120, K = 17408, BF16
//     207 -> 188.  Small tiles, bound by the latency of a step, give the steps
//     in turn to two groups of waves (KS = 2): tiles of 64 x 64 over 64 x 5120, K =
//     5120, MXFP8 14.8 -> 9.7 us; the narrowest ones, 64 x 32, which serve that
//     size now, to four (MXFP8 and MXFP4; of 64 x 64 four are no faster than two).
//   * BF16 activations: the weights are converted between the matrix
//     instructions that use them, and 8 waves side by side in n convert each
//     weight once (the conversions, 7.5 cycles each, otherwise cost as much as
//     half the matrix instructions).
//   * Workgroups are dealt to the 8 XCDs in contiguous runs of tiles, and tiles
//     run down four tile rows before the next tile column, so the workgroups
//     that share an L2 at one time share rows of both operands.
//
// What bounds it: with all compute units on random operands the chip lowers its
// clock (matrix instructions alone reach 4.3 PFLOP/s on FP4 x FP8, 8 on FP4 x
// FP4, 2.1 on BF16); 4096 x 17408, K = 5120, MXFP8 runs at 2.53 PFLOP/s, 4096 x
// 5120, K = 5120, MXFP4 at 3.0, 1000 x 5120, K = 17408, BF16 at 1.17.  64 rows are
// bound by the latency of their steps (64 x 5120, K = 17408: matrix units 12 to 19
// % busy, weights read at 1.2 to 2.7 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/wqd.h"
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
// (step_barrier), which the compiler's own waits could not do per buffer.  The
// LDS address is in m0, which the compiler sets, so that it knows what m0 holds;
// the transfer wants one instruction between.
__device__ __forceinline__ void copy_to_lds(uint32_t lds, rsrc_t r, uint32_t voff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(voff), "s"(r) : "memory");
}

// Wait until at most N of this wave's transfers are in flight and its LDS
// reads have returned, then meet the other waves.
template <int N>
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// KS: groups of waves that take the steps in turn and add their sums at the
// end.  MODE:
constexpr int kPlain = 0;   // read a step's operands, multiply
constexpr int kHalves = 1;  // the two halves of the waves, one of each per SIMD, run half a step apart:
                            // one reads LDS while the other has the matrix unit
constexpr int kPair = 2;    // MXFP4 activations: a stage is two steps, which one barrier serves

// LDS of a workgroup: PRE + 1 stages of all groups' (kPair: two) steps, and
// two stages of scales, whose rows are the weights' (gated: of either matrix),
// then the activations', in whole transfers of 64.
template <int BN, bool GATED>
constexpr uint32_t kMatScaleRows = (BN / (GATED ? 2 : 1) + 63) / 64 * 64;  // of one weight matrix
template <MxFormat FMT, int BM, int BN, bool GATED>
constexpr uint32_t kAllScaleRows = kMatScaleRows<BN, GATED> * (GATED ? 2 : 1) +
                                   (FMT == MxFormat::kBf16 ? 0 : (BM + 63) / 64 * 64);
template <MxFormat FMT, int BM, int BN, int KS, int MODE>
constexpr uint32_t kStageBytes = (MODE == kPair ? 2 : KS) * (BN / 16 + BM / 16 * kActUnits<FMT>) * kUnit;

template <MxFormat FMT, int BM, int BN, int KS, int PRE, int MODE, bool GATED>
constexpr uint32_t lds_bytes() {
  return (PRE + 1) * kStageBytes<FMT, BM, BN, KS, MODE> + 2 * kAllScaleRows<FMT, BM, BN, GATED> * 16;
}

// SHORT: K below the four steps that scales are staged in.  A kernel of its own:
// with the choice made inside it, the schedule of the others changes (1000 x 5120,
// K = 17408, BF16 150 -> 152 us).
template <MxFormat FMT, int BM, int BN, int WM, int WN, int KS, int PRE, int MODE, bool GATED, bool SHORT>
__global__ __launch_bounds__(64 * WM * WN * KS) void mx_tile_kernel(MxOperands op) {
  static_assert(MODE != kHalves || (KS == 1 && WM * WN == 8), "two waves per SIMD");
  constexpr uint32_t kGroupWaves = WM * WN, kWaves = kGroupWaves * KS;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int NBUF = PRE + 1;
  constexpr bool kTwo = MODE == kPair;  // a stage is two steps of every wave
  static_assert(!kTwo || (FMT == MxFormat::kFp4 && KS == 1), "4-bit codes on both sides");
  static_assert(KS == 1 || KS == 2 || KS == 4, "a group of four scale bytes is whole stages");
  // 4-bit codes of a stage's two steps come in units of 8 rows x 128 bytes,
  // which all waves share; others in units of 16 rows x 64 bytes per step.
  constexpr bool kLineW = kTwo || KS >= 2, kLineA = kLineW && FMT == MxFormat::kFp4;
  constexpr uint32_t kPairs = KS == 4 ? 2 : 1, kPairWaves = kWaves / kPairs;  // pairs of steps in a stage of lines
  constexpr uint32_t kWWaves = kLineW ? kPairWaves : kGroupWaves, kAWaves = kLineA ? kPairWaves : kGroupWaves;
  constexpr uint32_t kWUnits = BN / (kLineW ? 8 : 16), kAUnits = kLineA ? BM / 8 : BM / 16 * kActUnits<FMT>;
  constexpr uint32_t kStage = (kPairs * kWUnits + (kLineA ? kPairs : KS) * kAUnits) * kUnit;
  static_assert((kStage == kStageBytes<FMT, BM, BN, KS, MODE>));
  static_assert(!GATED || (kWUnits % 4 == 0 && kWWaves % 4 == 0 && NT % 2 == 0),
                "units of the two matrices alternate");
  static_assert(!kLineW || (kWaves % 2 == 0 && kWUnits % 2 == 0 && kAUnits % 2 == 0),
                "a wave's units are one half of the row tiles");
  constexpr int WU = (kWUnits + kWWaves - 1) / kWWaves, AU = (kAUnits + kAWaves - 1) / kAWaves, ND = WU + AU;
  constexpr bool kActScales = FMT != MxFormat::kBf16;
  constexpr uint32_t kMatRows = kMatScaleRows<BN, GATED>, kWsRows = kMatRows * (GATED ? 2 : 1);
  constexpr uint32_t kScaleRows = kAllScaleRows<FMT, BM, BN, GATED>;
  constexpr uint32_t kScaleStage = kScaleRows * 16;
  constexpr int SN = (kScaleRows / 64 + kWaves - 1) / kWaves;  // scale transfers per wave
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
  constexpr uint32_t kSteps = kTwo ? 2 : KS;  // of a stage
  const uint32_t stages = (steps + kSteps - 1u) / kSteps;

  // Transfers of this wave: weight units ww, ww + kWWaves, ... and activation
  // units likewise (where they do not come out even, some are brought twice, the
  // same bytes to the same place: every wave then has as many transfers in
  // flight as the waits count).  Gated: 16-row tiles are of the gate and the up
  // matrix in turn, and a wave's units all of one.
  const uint32_t pair = kPairs == 1 ? 0u : all_wave / kPairWaves, line_wave = all_wave - pair * kPairWaves;
  const uint32_t ww = kLineW ? line_wave : wave, aw = kLineA ? line_wave : wave;
  const bool up = GATED && (kLineW ? ww >> 1 & 1u : ww & 1u);
  const rsrc_t wr = bytes_rsrc(up ? op.WU : op.W, (uint64_t)n0 * wpitch, (nlast + 1u) * wpitch);
  const rsrc_t ar = bytes_rsrc(op.A, (uint64_t)m0 * apitch, mlast * apitch + act_bytes<FMT>(op.K));
  // this lane's row of a 16-row tile and piece of the row
  const uint32_t line_w = (ww & 1u) * 8u + (lane >> 3), line_a = (aw & 1u) * 8u + (lane >> 3);
  const uint32_t wrow = kLineW ? line_w : lane >> 2, arow = kLineA ? line_a : lane >> 2;
  const uint32_t wpiece = (kLineW ? (lane & 7u) ^ pair_turn(wrow) : (lane & 3u) ^ unit_turn(wrow)) * 16u;
  const uint32_t apiece = (kLineA ? (lane & 7u) ^ pair_turn(arow) : (lane & 3u) ^ unit_turn(arow)) * 16u;
  uint32_t woff[WU], aoff[AU];
#pragma unroll
  for (int i = 0; i < WU; ++i) {
    const uint32_t u = (ww + kWWaves * i) % kWUnits;
    const uint32_t row = u / (kLineW ? 2u : 1u) / (GATED ? 2u : 1u) * 16u + wrow;
    woff[i] = (row < nlast ? row : nlast) * wpitch + (kLineW ? 0u : wpiece);
  }
#pragma unroll
  for (int i = 0; i < AU; ++i) {
    const uint32_t u = (aw + kAWaves * i) % kAUnits;
    const uint32_t row = u / (kLineA ? 2u : kActUnits<FMT>) * 16u + arow;
    aoff[i] = (row < mlast ? row : mlast) * apitch + (kLineA ? 0u : (u % kActUnits<FMT>) * 64u + apiece);
  }
  // scale rows 64 p .. 64 p + 63 in transfer p, waves in turn: weights (gated: gate, then up), then activations
  rsrc_t sr[SN];
  uint32_t soff[SN];
#pragma unroll
  for (int i = 0; i < SN; ++i) {
    const uint32_t row = (all_wave + (uint32_t)i * kWaves) * 64u;
    const bool act = row >= kWsRows, s_up = GATED && !act && row >= kMatRows;
    sr[i] = act ? bytes_rsrc(op.AS, (uint64_t)m0 * nb, (mlast + 1u) * nb)
                : bytes_rsrc(s_up ? op.WUS : op.WS, (uint64_t)n0 * nb, (nlast + 1u) * nb);
    const uint32_t in = row - (act ? kWsRows : (s_up ? kMatRows : 0u)) + lane, last = act ? mlast : nlast;
    soff[i] = (in < last ? in : last) * nb;
  }

  // of a stage: its weights (a pair's after the other's), then its activations (of pairs or steps)
  constexpr uint32_t kABase = kPairs * kWUnits * kUnit;
  const uint32_t w_group = kPairs == 1 ? 0u : (ks >> 1) * kWUnits * kUnit;  // that this wave multiplies
  const uint32_t a_group = kABase + (kLineA ? (kPairs == 1 ? 0u : (ks >> 1)) : ks) * kAUnits * kUnit;
  const uint32_t w_put = pair * kWUnits * kUnit;  // that this wave brings
  const uint32_t a_put = kLineA ? kABase + pair * kAUnits * kUnit : a_group;
  auto issue = [&](uint32_t stage, uint32_t buf) __attribute__((always_inline)) {
    const uint32_t base = lds0 + buf * kStage;
    // where the last stage lacks its second step, what is brought of the first
    // one serves for it; it is not multiplied
    const uint32_t s = stage * KS + ks < steps ? stage * KS + ks : steps - 1u;
    const uint32_t last = (steps - 1u) >> 1, sp = kPairs == 1 ? stage : (stage * 2u + pair < last ? stage * 2u + pair : last);
    const bool whole = sp * 2u + 1u < steps;
    const uint32_t kw = kLineW ? sp * 128u + (whole ? wpiece : wpiece & 48u) : s * 64u;
    const uint32_t ka = kLineA ? sp * 128u + (whole ? apiece : apiece & 48u) : s * 64u * kActUnits<FMT>;
#pragma unroll
    for (int i = 0; i < WU; ++i) copy_to_lds(base + w_put + (ww + i * kWWaves) % kWUnits * kUnit, wr, woff[i] + kw);
#pragma unroll
    for (int i = 0; i < AU; ++i) copy_to_lds(base + a_put + (aw + i * kAWaves) % kAUnits * kUnit, ar, aoff[i] + ka);
  };
  // the 16 scale bytes from step 4q on, or the row's last 16 where fewer are left (nb >= 16)
  auto issue_scales = [&](uint32_t q) __attribute__((always_inline)) {
    const uint32_t at = 16u * q + 16u <= nb ? 16u * q : nb - 16u;
#pragma unroll
    for (int i = 0; i < SN; ++i) {
      const uint32_t p = all_wave + (uint32_t)i * kWaves;
      if (p < kScaleRows / 64u) copy_to_lds(lds0 + NBUF * kStage + (q & 1u) * kScaleStage + p * kUnit, sr[i], soff[i] + at);
    }
  };

  // the same of rows of 4, 8 or 12 bytes: step by step through registers, to the
  // end of their 16
  [[maybe_unused]] auto put_short_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < SN; ++i) {
      const uint32_t p = all_wave + (uint32_t)i * kWaves;
      if (p >= kScaleRows / 64u) continue;
      const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc(
          reinterpret_cast<void *>((uint64_t)sr[i].y << 32 | sr[i].x), (short)0, (int)sr[i].z, 0x00020000);
      uint32_t *to = reinterpret_cast<uint32_t *>(lds + NBUF * kStage + p * kUnit + lane * 16u) + 4u - steps;
      for (uint32_t t = 0; t < steps; ++t) to[t] = __builtin_amdgcn_raw_buffer_load_b32(from, soff[i] + 4u * t, 0, 0);
    }
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
    return (lo | hi << 16) >> (shift & 31u);  // 32 and more only for a group without a step there
  };
  auto read_scales = [&](uint32_t q) __attribute__((always_inline)) {
    const uint8_t *p = lds + NBUF * kStage + (q & 1u) * kScaleStage;
    // 8 bits a step, 4 bytes a step; a wave group's first step is byte 0
    const uint32_t shift = (16u * q + 16u <= nb ? 0u : (16u * q + 16u - nb) * 2u) + 8u * ks;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint32_t t = wn * NT + i;
      const uint32_t row = (GATED ? (t & 1u) * kMatRows + (t >> 1) * 16u : t * 16u) + r;
      wsc[i] = turn(*reinterpret_cast<const u32x4_t *>(p + row * 16u), shift);
    }
    if constexpr (kActScales) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
        asc[j] = turn(*reinterpret_cast<const u32x4_t *>(p + (kWsRows + (wm * MT + j) * 16u + r) * 16u), shift);
    }
  };

  // operands of a step from LDS; h: which of a stage's two steps
  const uint32_t mine = unit_byte(r, g);  // piece g of row r of a unit
  auto line_byte = [&](uint32_t h) __attribute__((always_inline)) { return r * 128u + ((h * 4u + g) ^ pair_turn(r)) * 16u; };
  auto read_w = [&](uint32_t buf, uint32_t h, WeightCodes (&w)[NT]) __attribute__((always_inline)) {
    constexpr uint32_t kTile = (kLineW ? 2 : 1) * kUnit;  // 16 rows
    const uint8_t *p = lds + buf * kStage + w_group + wn * NT * kTile + (kLineW ? line_byte(h) : mine);
#pragma unroll
    for (int i = 0; i < NT; ++i) w[i] = {*reinterpret_cast<const u32x4_t *>(p + i * kTile), wsc[i]};
  };
  auto read_a = [&](uint32_t buf, uint32_t h, int j) __attribute__((always_inline)) {
    constexpr uint32_t kTile = (kLineA ? 2 : kActUnits<FMT>) * kUnit;
    const uint8_t *p = lds + buf * kStage + a_group + (wm * MT + j) * kTile;
    ActRegs<FMT> a;
    if constexpr (FMT == MxFormat::kBf16) {
#pragma unroll
      for (uint32_t x = 0; x < 4; ++x)  // k 32g .. 32g + 31 are the four pieces of unit g
        a.v[x] = *reinterpret_cast<const u32x4_t *>(p + g * kUnit + unit_byte(r, x));
    } else if constexpr (kLineA) {
      a.v[0] = *reinterpret_cast<const u32x4_t *>(p + line_byte(h));
      a.s = asc[j];
    } else {
#pragma unroll
      for (uint32_t x = 0; x < kActUnits<FMT>; ++x) a.v[x] = *reinterpret_cast<const u32x4_t *>(p + x * kUnit + mine);
      a.s = asc[j];
    }
    return a;
  };

  if constexpr (SHORT)
    put_short_scales();
  else
    issue_scales(0);
  mx_unroll<0, PRE>([&](auto d) __attribute__((always_inline)) {
    constexpr uint32_t s = decltype(d)::value;
    if (s < stages) issue(s, s);
  });
  uint32_t buf = 0;
  constexpr int kGroup = 4 / KS;  // stages per group of four steps
  if constexpr (MODE == kHalves) {
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
          WeightCodes w[NT];
          ActRegs<FMT> a[MT];
          read_w(buf, 0u, w);
#pragma unroll
          for (int j = 0; j < MT; ++j) a[j] = read_a(buf, 0u, j);
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
          for (int i = 0; i < NT; ++i) {
            const WeightRegs<FMT, t> x(w[i]);
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = mx_mfma<FMT, t>(x, a[j], acc[i][j]);
          }
          __builtin_amdgcn_s_setprio(0);
          __builtin_amdgcn_sched_barrier(0);
          __builtin_amdgcn_s_barrier();
          buf = buf + 1u == (uint32_t)NBUF ? 0u : buf + 1u;
        }
      });
    }
    if (wave < 4u) __builtin_amdgcn_s_barrier();
  } else if constexpr (MODE == kPair) {
    for (uint32_t s0 = 0; s0 < stages; s0 += 2u) {
      mx_unroll<0, 2>([&](auto T) __attribute__((always_inline)) {
        constexpr int t = decltype(T)::value;
        const uint32_t s = s0 + t;
        if (s < stages) {
          if (s + PRE <= stages)
            step_barrier<(PRE - 1) * ND>();
          else
            step_barrier<0>();
          if constexpr (t == 0) {
            read_scales(s0 / 2u);
            if (s0 + 2u < stages) issue_scales(s0 / 2u + 1u);
          }
          if (s + PRE < stages) issue(s + PRE, buf == 0 ? NBUF - 1 : buf - 1);
          mx_unroll<0, 2>([&](auto H) __attribute__((always_inline)) {
            constexpr int h = decltype(H)::value;
            if (h == 0 || s * 2u + 1u < steps) {
              WeightCodes w[NT];
              ActRegs<FMT> a[MT];
#pragma unroll
              for (int j = 0; j < MT; ++j) a[j] = read_a(buf, h, j);
              read_w(buf, h, w);
#pragma unroll
              for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                  acc[i][j] = mx_mfma<FMT, t * 2 + h>(WeightRegs<FMT, t * 2 + h>(w[i]), a[j], acc[i][j]);
            }
          });
          buf = buf + 1u == (uint32_t)NBUF ? 0u : buf + 1u;
        }
      });
    }
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
            WeightCodes w[NT];
            read_w(buf, ks & 1u, w);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              const ActRegs<FMT> a = read_a(buf, ks & 1u, j);
#pragma unroll
              for (int i = 0; i < NT; ++i) acc[i][j] = mx_mfma<FMT, t * KS>(WeightRegs<FMT, t * KS>(w[i]), a, acc[i][j]);
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
  const uint32_t l = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)), lm = l & 15u, ln = (l >> 4) * 4u;
  constexpr int NO = GATED ? NT / 2 : NT;  // 16-column output tiles of this wave
  const uint32_t mw = m0 + wm * MT * 16u, nw = n0 + wn * NO * 16u;
  auto output = [&](int i, int j) __attribute__((always_inline)) {
    if constexpr (GATED) {
      f32x4_t c;
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = silu_times(acc[2 * i][j][e], acc[2 * i + 1][j][e]);
      return c;
    } else {
      return acc[i][j];
    }
  };
  // A lane holds 4 columns of a row: written as they are, an instruction covers
  // 32 bytes of 16 rows.  Large tiles inside the matrix go through LDS, each
  // wave's part on its own, and leave in whole row pieces of 16 bytes per lane.
  if constexpr (KS == 1) {
    constexpr uint32_t kRow = NO * 32 + 16, kPieces = NO * 2, kPart = MT * 16 * kRow;  // bytes, 16-byte pieces of a row
    static_assert(kPart % 16 == 0 && kWaves * kPart <= lds_bytes<FMT, BM, BN, KS, PRE, MODE, GATED>(), "outputs fit in LDS");
    if (op.out.wide >= 2u && n0 + BNO <= op.N) {
      step_barrier<0>();  // everybody has read the last stage
      uint8_t *part = lds + wave * kPart;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < NO; ++i) {
          const f32x4_t c = output(i, j);
          *reinterpret_cast<u32x2_t *>(part + (j * 16u + lm) * kRow + i * 32u + ln * 2u) =
              u32x2_t{bf16x2_rne(c[0], c[1]), bf16x2_rne(c[2], c[3])};
        }
#pragma unroll
      for (uint32_t p = 0; p < (MT * 16u * kPieces + 63u) / 64u; ++p) {
        const uint32_t x = p * 64u + l, row = x / kPieces, piece = x % kPieces;
        if ((MT * 16u * kPieces % 64u == 0u || x < MT * 16u * kPieces) && mw + row < op.M)
          *reinterpret_cast<u32x4_t *>(op.out.C + (uint64_t)(mw + row) * op.out.ldc + nw + piece * 8u) =
              *reinterpret_cast<const u32x4_t *>(part + row * kRow + piece * 16u);
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < NO; ++i)
      if (mw + j * 16u + lm < op.M) store4(op.out, op.N, mw + j * 16u + lm, nw + i * 16u + ln, output(i, j));
}

// Lets a kernel use all of a compute unit's LDS on the current device, once per device.
hipError_t allow_lds(const void *kern, std::atomic<uint64_t> &ready) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (ready.load(std::memory_order_relaxed) & bit)) return hipSuccess;
  e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  if (e == hipSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <MxFormat FMT, int BM, int BN, int WM, int WN, int KS, int PRE, int MODE, bool GATED>
hipError_t launch_cfg(const MxOperands &op, hipStream_t stream) {
  const bool short_k = op.K < 512u;
  const auto kern = short_k ? mx_tile_kernel<FMT, BM, BN, WM, WN, KS, PRE, MODE, GATED, true>
                            : mx_tile_kernel<FMT, BM, BN, WM, WN, KS, PRE, MODE, GATED, false>;
  constexpr uint32_t kLds = lds_bytes<FMT, BM, BN, KS, PRE, MODE, GATED>();
  static_assert(kLds <= 160 * 1024, "one workgroup's LDS");
  static std::atomic<uint64_t> ready[2];  // devices on which the kernel may use that much LDS
  const hipError_t attr = allow_lds(reinterpret_cast<const void *>(kern), ready[short_k]);
  if (attr != hipSuccess) return attr;
  const uint32_t bno = GATED ? BN / 2 : BN;
  const uint32_t tn = (op.N + bno - 1u) / bno;
  constexpr uint32_t kMaxGrid = mx_max_grid(64 * WM * WN * KS);
  static_assert(kMaxGrid >= WQD_MX_MAX_ROWS / (GATED ? BN / 2 : BN), "a launch holds the widest row of tiles");
  const uint32_t rows = kMaxGrid / tn * BM;
  for (uint32_t m = 0; m < op.M; m += rows) {
    const MxOperands part = mx_rows(op, FMT, m, rows);
    const uint32_t grid = tn * ((part.M + BM - 1u) / BM);
    hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * WM * WN * KS), kLds, stream, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// What a configuration takes per 128-k step, in ns: the first round of tiles
// over the compute units, and every further one; `share` workgroups fit one
// compute unit, so a further round comes in that many parts.  Measured at
// K = 5120 with 256, 512 and 1024 tiles (MI355X, weights from memory).
struct Cost {
  uint32_t bm, bn;  // outputs of a tile
  uint32_t first, more, share;
};

// The kernel for few rows works in tiles of 32 x 32 (gated: 16) and splits K
// eight ways, so it is ahead while its tiles do not fill the chip: 400 x 512
// outputs, K = 5120, MXFP8 7.7 us against 10.8 with 64 x 64 tiles, 800 x 512
// 14.5 against 11.1.  While 64 x 64 tiles leave compute units idle, 64 x 32 ones
// on twice as many read the weights faster: 64 x 5120, K = 17408, MXFP4 35.6 ->
// 24.8 us, MXFP8 41.8 -> 34.1, BF16 55.1 -> 46.6; gated 64 x 8192, K = 5120, MXFP8
// 22.2 -> 18.0; with two rounds of them 128 x 5120, K = 5120, MXFP8 11.2 with
// 64 x 64 tiles against 16.7.  Larger tiles cost less per output (MXFP8: 64 x 64 51 ns
// per 1000 outputs and step, 128 x 128 29, 256 x 256 24) and lose by rounds
// that they do not fill: 4096 x 5120, K = 5120, MXFP4, is 320 tiles of
// 256 x 256 (two rounds, 94 us) and 1280 of 128 x 128, two to a compute unit
// (five half rounds, 72 us); 1000 x 5120, K = 17408, MXFP8 one round of
// 128 x 160 (98 us) or of 80 tiles of 256 x 256 (160 us).  So the configuration
// of the least estimated time is taken.
template <MxFormat FMT, bool GATED>
struct Costs;
template <>
struct Costs<MxFormat::kBf16, false> {
  static constexpr Cost v[] = {{32, 32, 258, 240, 1},     {64, 32, 390, 390, 1},     {64, 64, 461, 420, 1},
                               {96, 256, 1364, 1310, 1}, {128, 192, 1435, 1350, 1}, {128, 256, 1777, 1620, 1}};
};
template <>
struct Costs<MxFormat::kBf16, true> {
  static constexpr Cost v[] = {{32, 16, 258, 240, 1}, {64, 32, 444, 410, 1}, {64, 64, 638, 610, 1},
                               {96, 128, 1364, 1310, 1}, {128, 128, 1777, 1620, 1}};
};
template <>
struct Costs<MxFormat::kFp8, false> {
  static constexpr Cost v[] = {{32, 32, 175, 160, 1},     {64, 32, 210, 160, 1},     {64, 64, 260, 210, 2},
                               {128, 128, 649, 470, 2},   {128, 160, 779, 690, 1},   {256, 160, 1191, 1100, 1},
                               {256, 224, 1509, 1430, 1}, {256, 256, 1685, 1590, 1}};
};
template <>
struct Costs<MxFormat::kFp8, true> {
  static constexpr Cost v[] = {{32, 16, 175, 160, 1}, {64, 32, 335, 300, 1},     {64, 64, 430, 400, 1},
                               {128, 64, 649, 470, 2}, {192, 128, 1373, 1250, 1}, {256, 128, 1685, 1590, 1}};
};
template <>
struct Costs<MxFormat::kFp4, false> {
  static constexpr Cost v[] = {{32, 32, 140, 115, 1},  {64, 32, 143, 150, 2},    {64, 64, 206, 172, 2},
                               {128, 128, 509, 377, 2}, {256, 192, 1064, 983, 1}, {256, 256, 1289, 1230, 1}};
};
template <>
struct Costs<MxFormat::kFp4, true> {
  static constexpr Cost v[] = {{32, 16, 140, 115, 1}, {64, 32, 230, 160, 1},    {64, 64, 331, 285, 2},
                               {128, 64, 509, 377, 2}, {192, 128, 1076, 987, 1}, {256, 128, 1289, 1230, 1}};
};

uint64_t cost_of(const Cost &c, const MxOperands &op, uint32_t cus) {
  const uint64_t tiles = (uint64_t)((op.M + c.bm - 1u) / c.bm) * ((op.N + c.bn - 1u) / c.bn);
  const uint64_t parts = (tiles * c.share + cus - 1u) / cus;  // of a round
  return c.first + (parts > c.share ? (parts - c.share) * c.more / c.share : 0u);
}

// The index of the least cost; 0, the kernel for few rows, up to 32 rows (its
// own row tiles).  The costs of a step serve K below 512 too, where the few-row
// kernel leaves five to seven of its eight waves without a step: from 33 x 512 to
// 4096 x 17408 outputs the choice was never more than 5 % behind it, and ahead
// wherever it takes tiles (64 x 5120, K = 256, BF16 9.5 -> 4.2 us; 4096 x 17408
// 1035 -> 80, MXFP8 719 -> 58, MXFP4 349 -> 48).
template <MxFormat FMT, bool GATED>
uint32_t pick(const MxOperands &op, uint32_t cus) {
  using C = Costs<FMT, GATED>;
  if (op.M <= 32u) return 0u;
  uint32_t best = 0;
  for (uint32_t i = 1; i < sizeof(C::v) / sizeof(Cost); ++i)
    if (cost_of(C::v[i], op, cus) < cost_of(C::v[best], op, cus)) best = i;
  return best;
}

template <MxFormat FMT, bool GATED>
hipError_t launch_fmt(const MxOperands &op, uint32_t cus, hipStream_t stream) {
  const uint32_t i = pick<FMT, GATED>(op, cus);
  if (i == 0u) return launch_mx_skinny(op, FMT, GATED, stream);
  // The waves of a 64 x 32 tile's group: two for plain products of codes (64 x
  // 5120, K = 17408, MXFP4 24.7 us, with four 27.0; MXFP8 34.0 either way), four
  // where a wave has more to convert or multiply (BF16 64 x 5120, K = 5120 14.2 us,
  // with two 15.3; gated MXFP4 64 x 8192 14.7, with two 15.2).
  if constexpr (FMT == MxFormat::kBf16 && GATED) {
    if (i == 1u) return launch_cfg<FMT, 64, 64, 2, 2, 2, 2, kPlain, GATED>(op, stream);
    if (i == 2u) return launch_cfg<FMT, 64, 128, 1, 4, 2, 1, kPlain, GATED>(op, stream);
    if (i == 3u) return launch_cfg<FMT, 96, 256, 1, 8, 1, 2, kHalves, GATED>(op, stream);
    return launch_cfg<FMT, 128, 256, 1, 8, 1, 2, kHalves, GATED>(op, stream);
  } else if constexpr (FMT == MxFormat::kBf16) {
    if (i == 1u) return launch_cfg<FMT, 64, 32, 4, 1, 2, 2, kPlain, GATED>(op, stream);
    if (i == 2u) return launch_cfg<FMT, 64, 64, 2, 2, 2, 2, kPlain, GATED>(op, stream);
    if (i == 3u) return launch_cfg<FMT, 96, 256, 1, 8, 1, 2, kHalves, GATED>(op, stream);
    if (i == 4u) return launch_cfg<FMT, 128, 192, 2, 4, 1, 2, kHalves, GATED>(op, stream);
    return launch_cfg<FMT, 128, 256, 1, 8, 1, 2, kHalves, GATED>(op, stream);
  } else if constexpr (FMT == MxFormat::kFp4 && GATED) {
    if (i == 1u) return launch_cfg<FMT, 64, 64, 4, 1, 4, 2, kPlain, GATED>(op, stream);
    if (i == 2u) return launch_cfg<FMT, 64, 128, 2, 2, 2, 2, kPlain, GATED>(op, stream);
    if (i == 3u) return launch_cfg<FMT, 128, 128, 4, 2, 1, 1, kPair, GATED>(op, stream);
    if (i == 4u) return launch_cfg<FMT, 192, 256, 4, 2, 1, 1, kPair, GATED>(op, stream);
    return launch_cfg<FMT, 256, 256, 4, 2, 1, 1, kPair, GATED>(op, stream);
  } else if constexpr (FMT == MxFormat::kFp4) {
    if (i == 1u) return launch_cfg<FMT, 64, 32, 2, 1, 4, 2, kPlain, GATED>(op, stream);
    if (i == 2u) return launch_cfg<FMT, 64, 64, 2, 2, 2, 2, kPlain, GATED>(op, stream);
    if (i == 3u) return launch_cfg<FMT, 128, 128, 4, 2, 1, 1, kPair, GATED>(op, stream);
    if (i == 4u) return launch_cfg<FMT, 256, 192, 4, 2, 1, 1, kPair, GATED>(op, stream);
    return launch_cfg<FMT, 256, 256, 4, 2, 1, 1, kPair, GATED>(op, stream);
  } else if constexpr (GATED) {
    if (i == 1u) return launch_cfg<FMT, 64, 64, 4, 1, 4, 2, kPlain, GATED>(op, stream);
    if (i == 2u) return launch_cfg<FMT, 64, 128, 2, 2, 2, 2, kPlain, GATED>(op, stream);
    if (i == 3u) return launch_cfg<FMT, 128, 128, 4, 2, 1, 2, kHalves, GATED>(op, stream);
    if (i == 4u) return launch_cfg<FMT, 192, 256, 4, 2, 1, 2, kHalves, GATED>(op, stream);
    return launch_cfg<FMT, 256, 256, 4, 2, 1, 2, kHalves, GATED>(op, stream);
  } else {
    if (i == 1u) return launch_cfg<FMT, 64, 32, 2, 1, 4, 2, kPlain, GATED>(op, stream);
    if (i == 2u) return launch_cfg<FMT, 64, 64, 2, 2, 2, 2, kPlain, GATED>(op, stream);
    if (i == 3u) return launch_cfg<FMT, 128, 128, 4, 2, 1, 2, kHalves, GATED>(op, stream);
    if (i == 4u) return launch_cfg<FMT, 128, 160, 4, 2, 1, 2, kHalves, GATED>(op, stream);
    if (i == 5u) return launch_cfg<FMT, 256, 160, 4, 2, 1, 2, kHalves, GATED>(op, stream);
    if (i == 6u) return launch_cfg<FMT, 256, 224, 4, 2, 1, 2, kHalves, GATED>(op, stream);
    return launch_cfg<FMT, 256, 256, 4, 2, 1, 2, kHalves, GATED>(op, stream);
  }
}

// Compute units of the current device, asked for once per device.
hipError_t compute_units(uint32_t &cus) {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 64) n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    e = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    n = n > 0 ? n : 1;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  }
  cus = (uint32_t)n;
  return hipSuccess;
}

}  // namespace

hipError_t launch_mx_product(const MxOperands &op, MxFormat fmt, bool gated, hipStream_t stream) {
  uint32_t cus = 1;
  const hipError_t e = compute_units(cus);
  if (e != hipSuccess) return e;
  switch (fmt) {
    case MxFormat::kBf16:
      return gated ? launch_fmt<MxFormat::kBf16, true>(op, cus, stream) : launch_fmt<MxFormat::kBf16, false>(op, cus, stream);
    case MxFormat::kFp8:
      return gated ? launch_fmt<MxFormat::kFp8, true>(op, cus, stream) : launch_fmt<MxFormat::kFp8, false>(op, cus, stream);
    default:
      return gated ? launch_fmt<MxFormat::kFp4, true>(op, cus, stream) : launch_fmt<MxFormat::kFp4, false>(op, cus, stream);
  }
}

}  // namespace wqd
