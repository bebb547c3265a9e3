// Products with 4-bit integer weights for many rows, for gfx950 (MI355X): the
// operations of i4_skinny.hip, bound by the matrix instructions and by what feeds
// them.
//
// A workgroup of 8 waves owns BM rows and 256 weight rows (in the gated form
// 128 of both matrices) and walks K in steps of 128.  With 64 rows the waves stand side
// by side in n: each converts its own weights only, and all read all activations.  With
// 128 they are four in n and two in m, which share a SIMD and convert the same weights.
//
//   * Staging.  Activations, codes, scales and zero points go straight from memory to
//     LDS, two steps ahead of their use, into the third of three stages; a wave asks for
//     an eighth of each.  Codes lie in the matrix operand's order, so a lane reads back
//     what its neighbours brought in whole KB.  Rows past the last one repeat it; their
//     outputs are not stored.
//   * Codes become BF16 values 16 + q by two integer instructions a pair (i4_biased), a
//     chunk of 16 k ahead of the matrix instructions that take them.  16 + z goes with the
//     sums of the activations: without zero points a group's sums start at -24 times them, with
//     zero points at -(16 + z) times them, a product of rank one by a matrix instruction, for
//     which a sum is split into three BF16 values (exact).  Each wave forms those of 16 rows for
//     all, by matrix instructions against ones, a step ahead.
//   * All instructions of both waves of a SIMD share its issue: beside a 32 x 32 x 16
//     matrix instruction (32 cycles) there is room for six others of its wave, beside a 16
//     x 16 x 32 one for two.  Hence 32 x 32, and no more than two instructions for a pair of
//     codes.  Of a step of 128 rows (1.45 us on 160 compute units) the matrix instructions
//     take 0.9 at the highest clock.
//     Where all compute units work the clock falls to about 2 GHz: 4096 x 5120, K = 5120 208 - 214
//     us, 1.0 PFLOP/s, 16384 x 2048, K = 4096 267 us, 1.03.
//   * The sums of a group are a matrix accumulator of their own, which the scale
//     adds to the output's, all in fp32.  What is rounded in them are sums of a (16 + q) and their
//     remainder after (16 + z) times those of a, which may be a few times the sum that is meant.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/wqd.h"
#include "i4_common.h"
#include "mx_product.h"
#include "wqd_internal.h"

namespace wqd {
namespace {

constexpr uint32_t kWaves = 8;

typedef uint32_t rsrc_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ rsrc_t bytes_rsrc(const void *p, uint64_t offset, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p) + offset;
  const rsrc_t r = {(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a),
                    (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xffffu),
                    (uint32_t)__builtin_amdgcn_readfirstlane(bytes), 0x00020000u};
  return r;
}

// 16 bytes per lane from voff of the buffer to LDS byte `lds` + 16 * lane.  The
// transfer has no destination registers; it is waited for by count.
__device__ __forceinline__ void copy16_to_lds(uint32_t lds, rsrc_t r, uint32_t voff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(voff), "s"(r) : "memory");
}
// BYTES (4, 2 or 1, in multiples of which voff is) for each of the first LANES lanes, where all 64 are
// active, to LDS byte `lds` + 4 * lane; fewer than 4 are followed by zeros.
template <int LANES, int BYTES = 4>
__device__ __forceinline__ void copy_to_lds(uint32_t lds, rsrc_t r, uint32_t voff) {
  constexpr uint64_t lanes = (1ull << LANES) - 1ull;
  if constexpr (BYTES == 4)
    asm volatile("s_mov_b64 exec, %3\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds\n\ts_mov_b64 exec, -1"
                 :
                 : "{m0}"(lds), "v"(voff), "s"(r), "s"(lanes)
                 : "memory");
  else if constexpr (BYTES == 2)
    asm volatile("s_mov_b64 exec, %3\n\ts_nop 0\n\tbuffer_load_ushort %1, %2, 0 offen lds\n\ts_mov_b64 exec, -1"
                 :
                 : "{m0}"(lds), "v"(voff), "s"(r), "s"(lanes)
                 : "memory");
  else
    asm volatile("s_mov_b64 exec, %3\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, 0 offen lds\n\ts_mov_b64 exec, -1"
                 :
                 : "{m0}"(lds), "v"(voff), "s"(r), "s"(lanes)
                 : "memory");
}

// Wait until at most N of this wave's transfers are in flight and its LDS
// reads have returned, then meet the other waves.
template <int N>
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

constexpr int kDense = 0;  // rows m0 ..
constexpr int kLists = 1;  // rows of one expert's list

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// LDS of a stage: activations, and of 16 weight tiles the codes, 128 bytes of
// scales and 64 of zero points (this step's and what follows them)
// and the sums of the activations of each group; and three stages
constexpr uint32_t NBUF = 3;
template <int BM, int NG, bool ZEROS>
constexpr uint32_t kStage = BM * 256 + 16 * (kI4Tile + 128 + (ZEROS ? 64 : 0)) + NG * BM * (ZEROS && NG <= 2 ? 8 : 4);
// and which pairs the rows are
template <int BM, int NG, bool ZEROS>
constexpr uint32_t kLdsBytes = NBUF * kStage<BM, NG, ZEROS> + BM * 4;

// WM: waves side by side in m; 8 / WM in n.  BY_ROW: scales and zero points row by row; a transfer takes what a step
// needs of each of 16 rows (4096 x 5120, K = 5120 212 us, in tiles 208; gated 500 x 17408, K = 5120 with zero points 210 and 205).
template <int BM, int WM, bool GATED, int NG, bool ZEROS, bool BY_ROW, int ROWS>
__global__ __launch_bounds__(64 * kWaves) void i4_tile_kernel(I4Operands op, uint32_t tm) {
  static_assert(BM <= 128, "a wave forms the sums of 16 rows");
  constexpr int MT = BM / WM / 32, NS = WM, AU = BM / 32;  // 32 x 32 tiles of a wave; its transfers of activations
  constexpr int ND = AU + (ZEROS ? 6 : 4);                  // transfers of a wave and step
  constexpr uint32_t BNT = GATED ? 8 : 16;                  // 16-column tiles of the output
  // Zero points by a matrix instruction (16 + z times the sums of the activations, before a group's products; 1000 x
  // 5120, K = 17408 229 -> 217 us, 4096 x 5120, K = 5120 in groups of 64 273 -> 268) or, with groups of 32, for which the
  // sums in three parts do not fit LDS, by a second multiply-add of the fold
  constexpr bool kOuter = ZEROS && NG <= 2, kFolded = ZEROS && NG > 2;
  constexpr uint32_t kW = BM * 256, kS = kW + 16 * kI4Tile, kZ = kS + 16 * 128, kSum = kZ + (ZEROS ? 16 * 64 : 0);
  constexpr uint32_t kBuf = kStage<BM, NG, ZEROS>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

  const uint32_t lane = threadIdx.x & 63u, n5 = lane & 31u, kk = lane >> 5, r = lane & 15u, g = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t wm = wave / (kWaves / WM), wn = wave % (kWaves / WM);
  const uint32_t tiles = (op.N + 15u) >> 4, kt = op.K >> 7, tn = (tiles + BNT - 1u) / BNT;

  // Tile of this workgroup: the 8 XCDs, which take workgroups in turn, get
  // contiguous runs, and tiles run down four rows before the next column.  Of lists
  // the grid has more than there are, which would all be the last XCDs'.
  if constexpr (ROWS == kLists) {
    const uint32_t chunks = i4_count_chunks<BM>(op.offsets, op.E, op.T * op.top_k, lane);
    tm = chunks < tm ? chunks : tm;
    if (blockIdx.x >= tm * tn) return;
  }
  const uint32_t total = tm * tn, xcd = blockIdx.x & 7u, q8 = total >> 3, rem = total & 7u;
  const uint32_t id = xcd * q8 + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
  const uint32_t band = id / (4u * tn), in_band = id - band * 4u * tn;
  const uint32_t band_rows = tm - band * 4u < 4u ? tm - band * 4u : 4u;
  const uint32_t col = in_band / band_rows, chunk = band * 4u + in_band - col * band_rows;

  uint32_t first = chunk * BM, rows, expert = 0;
  if constexpr (ROWS == kDense) {
    rows = op.M - first < (uint32_t)BM ? op.M - first : (uint32_t)BM;
  } else {
    if (!i4_find_chunk<BM>(op.offsets, op.E, op.T * op.top_k, chunk, lane, expert, first, rows)) return;
  }
  uint32_t *const pair_of = reinterpret_cast<uint32_t *>(lds + NBUF * kBuf);
  if constexpr (ROWS == kLists) {
    if (threadIdx.x < (uint32_t)BM) {
      const uint32_t p = (uint32_t)op.order[first + (threadIdx.x < rows ? threadIdx.x : rows - 1u)];
      pair_of[threadIdx.x] = p < op.T * op.top_k ? p : 0u;
    }
    __syncthreads();
  }

  // Activations: units of 4 rows x 256 bytes; slot x of row m has piece x ^ (m % 16), so
  // that the sixteen lanes that an LDS read serves together meet all 64 banks.
  const uint32_t pitch = op.lda * 2u;
  const rsrc_t ar = ROWS == kDense ? bytes_rsrc(op.A, (uint64_t)first * pitch, (rows - 1u) * pitch + op.K * 2u)
                                   : bytes_rsrc(op.A, 0, ((GATED ? op.T : op.T * op.top_k) - 1u) * pitch + op.K * 2u);
  uint32_t aoff[AU];
#pragma unroll
  for (int i = 0; i < AU; ++i) {
    const uint32_t m = (wave + i * kWaves) * 4u + g;
    const uint32_t row = ROWS == kDense ? (m < rows ? m : rows - 1u) : (GATED ? pair_of[m] / op.top_k : pair_of[m]);
    aoff[i] = row * pitch + (r ^ (m & 15u)) * 16u;
  }
  // the two weight tiles that this wave brings (gated: one of either matrix)
  rsrc_t wr[2], sr[2], zr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const I4Matrix &m = GATED && i ? op.up : op.w;
    const uint32_t t = col * BNT + (GATED ? wave : wave * 2u + i);
    const uint64_t at = ((uint64_t)expert * tiles + (t < tiles ? t : tiles - 1u)) * kt;
    wr[i] = bytes_rsrc(m.W, at * kI4Tile, kt * kI4Tile);
    // the tile's scales: its row of tiles', or the rows that there are
    const uint32_t row = (t < tiles ? t : tiles - 1u) * 16u, left = op.N - row;
    const uint64_t groups = BY_ROW ? ((uint64_t)expert * op.N + row) * kt * NG : at * (16u * NG);
    const uint32_t count = (BY_ROW && left < 16u ? left : 16u) * kt * NG;
    sr[i] = bytes_rsrc(m.S, groups * 2u, count * 2u);
    if constexpr (ZEROS) zr[i] = bytes_rsrc(m.Z, groups, count);
  }
  // Row by row a lane brings its row's piece, 4 bytes at most: rows of scales lie kSRow and of zero points kZRow
  // elements apart in LDS then
  constexpr int kSRow = BY_ROW && NG == 1 ? 2 : NG, kZRow = BY_ROW ? 4 : NG;
  constexpr int kSBytes = NG == 1 ? 2 : 4, kZBytes = NG;
  const uint32_t srow = NG == 4 ? (lane >> 1) * (kt * 8u) + (lane & 1u) * 4u : lane * (kt * (2u * NG)), zrow = lane * (kt * NG);
  // Transfer i of step s to its stage.  Past the last step it comes once more.
  // Scales and zero points beyond a tile's are read as zeros and not used.
  auto issue = [&](int i, uint32_t s, uint32_t stage) __attribute__((always_inline)) {
    const uint32_t t = s < kt ? s : kt - 1u, h = (i - AU) & 1, to = lds0 + stage;
    if (i < AU)
      copy16_to_lds(to + (wave + i * kWaves) * 1024u, ar, aoff[i] + t * 256u);
    else if (i < AU + 2)
      copy16_to_lds(to + kW + (wave * 2u + h) * kI4Tile, wr[h], t * kI4Tile + lane * 16u);
    else if (i < AU + 4) {
      if constexpr (BY_ROW)
        copy_to_lds<NG == 4 ? 32 : 16, kSBytes>(to + kS + (wave * 2u + h) * 128u, sr[h], t * (2u * NG) + srow);
      else
        copy_to_lds<32>(to + kS + (wave * 2u + h) * 128u, sr[h], t * (32u * NG) + lane * 4u);
    } else if constexpr (BY_ROW)
      copy_to_lds<16, kZBytes>(to + kZ + (wave * 2u + h) * 64u, zr[h], t * NG + zrow);
    else
      copy_to_lds<16>(to + kZ + (wave * 2u + h) * 64u, zr[h], t * (16u * NG) + lane * 4u);
  };

  f32x16_t acc[MT][NS];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[j][i][e] = 0.0f;

  // A step's weights of this lane's columns (n5 of each 32): the 16 bytes of chunks
  // (k = 16 c + 8 kk ..) of even and odd c, scales, zero points
  struct Codes {
    u32x4_t w[NS][2];
    I4Groups<NG> s[NS];
  };
  uint32_t mask = kI4BiasMask, base = kI4BiasBase;
  asm volatile("" : "+s"(mask), "+v"(base));
  auto read_codes = [&](uint32_t stage) __attribute__((always_inline)) {
    Codes x;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const uint32_t t = (wn * NS + i) * 2u + (n5 >> 4);
      const uint8_t *p = lds + stage;
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h)
        x.w[i][h] = *reinterpret_cast<const u32x4_t *>(p + kW + t * kI4Tile + (2u * h + kk) * 256u + r * 16u);
      x.s[i] = i4_load_groups<NG, ZEROS, kSRow, kZRow>(reinterpret_cast<const uint16_t *>(p + kS + t * 128u), p + kZ + t * 64u, r);
    }
    return x;
  };
  bf16x8_t a[2][MT], b[2][NS];  // of chunk c in place c % 2
  auto read_a = [&](uint32_t stage, int c) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
      a[c & 1][j] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t *>(
          lds + stage + (wm * (MT * 32u) + j * 32u + n5) * 256u + ((2u * c + kk) ^ r) * 16u));
  };
  auto convert = [&](const Codes &x, int c) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      b[c & 1][i] = i4_biased(x.w[i][c & 1][c >> 1], mask, base);
      asm volatile("" : "+v"(b[c & 1][i]));  // here, not where it is used
    }
  };
  // The sums of the activations of a step's groups (without zero points times -24), of
  // 16 rows by this wave (of fewer rows two waves write the same): read, multiply, write
  const uint32_t sum_rows = wave % (BM / 16);
  u32x4_t sum_a[4];
  f32x4_t sum_t[NG];
  auto sums_read = [&](uint32_t stage) __attribute__((always_inline)) {
#pragma unroll
    for (uint32_t x = 0; x < 4; ++x)
      sum_a[x] = *reinterpret_cast<const u32x4_t *>(lds + stage + (sum_rows * 16u + r) * 256u + ((4u * x + g) ^ r) * 16u);
  };
  auto sums_form = [&]() __attribute__((always_inline)) {
    const u32x4_t one = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      sum_t[q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = q * 4 / NG; x < (q + 1) * 4 / NG; ++x)
        sum_t[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, sum_a[x]), __builtin_bit_cast(bf16x8_t, one),
                                                           sum_t[q], 0, 0, 0);
    }
  };
  auto sums_write = [&](uint32_t stage) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NG; ++q)  // the sixteen lanes of a row group hold and write the same
      *reinterpret_cast<f32x4_t *>(lds + stage + kSum + (q * BM + sum_rows * 16u + g * 4u) * 4u) =
          ZEROS ? sum_t[q] : sum_t[q] * (-kI4Bias - 8.0f);
  };
  // The same as three BF16 values, whose sum it is bit for bit; four lanes write a row each
  auto sums_split = [&](uint32_t stage) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      const float lo = r & 1u ? sum_t[q][1] : sum_t[q][0], hi = r & 1u ? sum_t[q][3] : sum_t[q][2], v = r & 2u ? hi : lo;
      const uint32_t first = __float_as_uint(v) & 0xffff0000u;
      const float rest = v - __uint_as_float(first);
      const uint32_t second = __float_as_uint(rest) & 0xffff0000u;
      const uint32_t third = __float_as_uint(rest - __uint_as_float(second)) >> 16;
      if (r < 4u)
        *reinterpret_cast<u32x2_t *>(lds + stage + kSum + (q * BM + sum_rows * 16u + g * 4u + r) * 8u) = u32x2_t{first >> 16 | second, third};
    }
  };
  // Their products with -(16 + z) of tile (j, i): the lower lanes' k have z, the upper ones' 16
  auto outer = [&](const u32x2_t &v, const Codes &x, int q, int i) __attribute__((always_inline)) {
    const uint32_t z = kk ? __float_as_uint(-kI4Bias) >> 16 : __float_as_uint(-i4_zero_of(x.s[i], q)) >> 16;
    const u32x4_t left = {v.x, v.y, 0u, 0u}, right = {z << 16 | z, z, 0u, 0u};
    const f32x16_t none = {};
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, left), __builtin_bit_cast(bf16x8_t, right), none, 0, 0, 0);
  };
  // rows 8 (e / 4) + 4 kk + e % 4 of tile j, as a lane's outputs have them
  auto sums_of = [&](uint32_t stage, int q, int j) __attribute__((always_inline)) {
    f32x16_t t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4_t x = *reinterpret_cast<const f32x4_t *>(lds + stage + kSum + (q * BM + wm * (MT * 32u) + j * 32u + i * 8u + kk * 4u) * 4u);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[4 * i + e] = x[e];
    }
    return t;
  };

  // The group that is being multiplied, and the scales and zero points of its columns: it
  // joins the outputs when the next one begins.
  f32x16_t t[MT][NS];
  float scale[NS], zero[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    scale[i] = zero[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) t[j][i][e] = 0.0f;
  }
  auto fold = [&](int j, int i, const f32x16_t &z) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      acc[j][i][e] = __builtin_fmaf(scale[i], kFolded ? __builtin_fmaf(zero[i], z[e], t[j][i][e]) : t[j][i][e], acc[j][i][e]);
    asm volatile("" : "+v"(acc[j][i]));
  };
  Codes even;
  auto step = [&](uint32_t s, uint32_t prev, uint32_t cur, uint32_t nxt, const Codes &x, Codes &after) __attribute__((always_inline)) {
    step_barrier<0>();
    Codes y;
    mx_unroll<0, 8>([&](auto C) __attribute__((always_inline)) {
      constexpr int c = decltype(C)::value, q = c * NG / 8;
      constexpr bool kFirst = c * NG % 8 == 0;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        f32x16_t from = {}, z = {};
        if constexpr (kFirst && kFolded) z = sums_of(c == 0 ? prev : cur, (q + NG - 1) % NG, j);
        if constexpr (kFirst && !ZEROS) from = sums_of(cur, q, j);
        u32x2_t sum = {};
        if constexpr (kFirst && kOuter)
          sum = *reinterpret_cast<const u32x2_t *>(lds + cur + kSum + (q * BM + wm * (MT * 32u) + j * 32u + n5) * 8u);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          if constexpr (kFirst) fold(j, i, z);
          if constexpr (kFirst && kFolded) {
#pragma unroll
            for (int e = 0; e < 16; ++e) from[e] = 0.0f;
          }
          if constexpr (kFirst && kOuter) {
            from = outer(sum, x, q, i);
            asm volatile("" : "+v"(from));
            if (i == NS - 1) __builtin_amdgcn_sched_barrier(0);  // later ones take registers that are still held
          }
          t[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[c & 1][j], b[c & 1][i], kFirst ? from : t[j][i], 0, 0, 0);
        }
      }
      if constexpr (kFirst) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          scale[i] = i4_scale_of(x.s[i], q, op.scale_bf16);
          zero[i] = -kI4Bias - i4_zero_of(x.s[i], q);
        }
      }
      read_a(c < 7 ? cur : nxt, (c + 1) % 8);
      if constexpr (c == 5) y = read_codes(nxt);
      convert(c < 7 ? x : y, (c + 1) % 8);
      if constexpr (c == 2) sums_read(nxt);
      if constexpr (c == 3) sums_form();
      if constexpr (c == 5 && kOuter) sums_split(nxt);
      if constexpr (c == 5 && !kOuter) sums_write(nxt);
      // a matrix instruction and others in turn
      if constexpr (!kFirst) {
        mx_unroll<0, MT * NS>([&](auto) __attribute__((always_inline)) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
        });
      }
      __builtin_amdgcn_sched_barrier(0);
      // a share of the next transfers: all at once they hold up what follows
#pragma unroll
      for (int i = 0; i < ND; ++i)
        if (i * 4 / ND == c) issue(i, s + 2u, prev);
    });
    after = y;
  };

#pragma unroll
  for (int i = 0; i < ND; ++i) issue(i, 0u, 0u);
#pragma unroll
  for (int i = 0; i < ND; ++i) issue(i, 1u, kBuf);
  step_barrier<ND>();
  sums_read(0u);
  sums_form();
  if constexpr (kOuter) sums_split(0u);
  else sums_write(0u);
  if constexpr (kFolded) {  // "the step before" has sums of zero
    for (uint32_t i = threadIdx.x; i < NG * BM; i += 64u * kWaves) *reinterpret_cast<float *>(lds + 2u * kBuf + kSum + i * 4u) = 0.0f;
  }
  even = read_codes(0u);
  read_a(0u, 0);
  convert(even, 0);
  uint32_t prev = 2 * kBuf, cur = 0, nxt = kBuf;
  auto turn = [&]() __attribute__((always_inline)) {
    const uint32_t free = prev;
    prev = cur;
    cur = nxt;
    nxt = free;
  };
  if ((WM == 2 && (ROWS == kLists || ZEROS)) && wm * (MT * 32u) >= rows) {
    // Rows that are none of this wave's: it brings its share and forms its sums only, and leaves the SIMD to the
    // other one there (512 tokens of 8 of 64 experts, 2048 outputs, K = 1024 56.1 -> 53 us, 300 x 17408, K = 5120 with
    // zero points 77 -> 71.5).  Without lists and zero points the second loop costs more than it gives where tiles
    // are full (1000 x 5120, K = 5120 64.2 -> 67.7; 300 x 17408, K = 5120 74.8 -> 68.9).
    for (uint32_t s = 0; s < kt; ++s) {
      step_barrier<0>();
      sums_read(nxt);
      sums_form();
      if constexpr (kOuter) sums_split(nxt);
      else sums_write(nxt);
#pragma unroll
      for (int i = 0; i < ND; ++i) issue(i, s + 2u, prev);
      const uint32_t free = prev;
      prev = cur;
      cur = nxt;
      nxt = free;
    }
  } else if constexpr (NG == 1 || (NG == 2 && !ZEROS)) {
    // Two steps an iteration: then no sums are copied from the registers that one step leaves
    // them in to those that the next expects (1000 x 5120, K = 17408: 225 -> 202 us; 1000 x
    // 5120, K = 5120 71.5 -> 64.5).  In groups of 32, and with zero points in groups of 64, the registers no
    // longer suffice.
    Codes odd;
    uint32_t s = 0;
    for (; s + 1u < kt; s += 2u) {
      step(s, prev, cur, nxt, even, odd);
      turn();
      step(s + 1u, prev, cur, nxt, odd, even);
      turn();
    }
    if (s < kt) {
      step(s, prev, cur, nxt, even, odd);
      turn();
    }
  } else {
    for (uint32_t s = 0; s < kt; ++s) {
      step(s, prev, cur, nxt, even, even);
      const uint32_t free = prev;
      prev = cur;
      cur = nxt;
      nxt = free;
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    f32x16_t z = {};
    if constexpr (kFolded) z = sums_of(prev, NG - 1, j);
#pragma unroll
    for (int i = 0; i < NS; ++i) fold(j, i, z);
  }
  step_barrier<0>();  // nothing is in flight

  if constexpr (ROWS == kLists && !GATED) {  // 128 bytes of a row each half wave
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (uint32_t e = 0; e < 16; ++e) {
        const uint32_t m = (wm * MT + j) * 32u + 8u * (e >> 2) + 4u * kk + (e & 3u);
        float *y = op.Y + (uint64_t)pair_of[m] * op.N;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const uint32_t c = col * (BNT * 16u) + (wn * NS + i) * 32u + n5;
          if (m < rows && c < op.N) y[c] = acc[j][i][e];
        }
      }
  } else {
    // Through LDS, to leave in whole pieces of 16 bytes.  Rows 16 bytes longer than their values.
    constexpr uint32_t kCols = BNT * 16, kRow = kCols * 2 + 16, kPieces = kCols / 8;
    static_assert(BM * kRow <= NBUF * kBuf, "outputs fit in the stages");
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (uint32_t e = 0; e < 16; ++e) {
        const uint32_t m = (wm * MT + j) * 32u + 8u * (e >> 2) + 4u * kk + (e & 3u);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          float y = acc[j][i][e];
          if constexpr (GATED) y = silu_times(y, __shfl_xor(y, 16));  // the up matrix's column is 16 lanes on
          const uint32_t c = GATED ? (wn * NS + i) * 16u + r : (wn * NS + i) * 32u + n5;
          if (!GATED || n5 < 16u) *reinterpret_cast<uint16_t *>(lds + m * kRow + c * 2u) = (uint16_t)bf16x2_rne(y, 0.0f);
        }
      }
    __syncthreads();
    const bool wide = (reinterpret_cast<uint64_t>(op.C) & 15u) == 0u && op.ldc % 8u == 0u;
    for (uint32_t x = threadIdx.x; x < rows * kPieces; x += 64u * kWaves) {
      const uint32_t m = x / kPieces, n = col * kCols + x % kPieces * 8u;
      if (n >= op.N) continue;
      const uint8_t *from = lds + m * kRow + x % kPieces * 16u;
      uint16_t *to = op.C + (uint64_t)(ROWS == kDense ? first + m : pair_of[m]) * op.ldc + n;
      if (wide && n + 8u <= op.N) {
        *reinterpret_cast<u32x4_t *>(to) = *reinterpret_cast<const u32x4_t *>(from);
      } else {
        for (uint32_t i = 0; i < 8u && n + i < op.N; ++i) to[i] = reinterpret_cast<const uint16_t *>(from)[i];
      }
    }
  }
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

template <int BM, int WM, bool GATED, int NG, bool ZEROS, bool BY_ROW, int ROWS>
hipError_t launch_kernel(const I4Operands &op, uint32_t tm, hipStream_t stream) {
  const auto kern = i4_tile_kernel<BM, WM, GATED, NG, ZEROS, BY_ROW, ROWS>;
  constexpr uint32_t kLds = kLdsBytes<BM, NG, ZEROS>;
  static_assert(kLds <= 160 * 1024, "one workgroup's LDS");
  static std::atomic<uint64_t> ready;  // devices on which the kernel may use that much LDS
  const hipError_t attr = allow_lds(reinterpret_cast<const void *>(kern), ready);
  if (attr != hipSuccess) return attr;
  constexpr uint32_t kCols = kWaves * 16 * (GATED ? 1 : 2);
  hipLaunchKernelGGL(kern, dim3(tm * ((op.N + kCols - 1u) / kCols)), dim3(64 * kWaves), kLds, stream, op, tm);
  return hipGetLastError();
}

template <int BM, int WM, bool GATED, int NG, int ROWS>
hipError_t launch_group(const I4Operands &op, uint32_t tm, hipStream_t stream) {
  if (op.by_row)
    return op.w.Z ? launch_kernel<BM, WM, GATED, NG, true, true, ROWS>(op, tm, stream)
                  : launch_kernel<BM, WM, GATED, NG, false, true, ROWS>(op, tm, stream);
  return op.w.Z ? launch_kernel<BM, WM, GATED, NG, true, false, ROWS>(op, tm, stream)
                : launch_kernel<BM, WM, GATED, NG, false, false, ROWS>(op, tm, stream);
}

template <int BM, int WM, bool GATED, int ROWS>
hipError_t launch_cfg(const I4Operands &op, uint32_t tm, hipStream_t stream) {
  if (op.group == 128u) return launch_group<BM, WM, GATED, 1, ROWS>(op, tm, stream);
  if (op.group == 64u) return launch_group<BM, WM, GATED, 2, ROWS>(op, tm, stream);
  return launch_group<BM, WM, GATED, 4, ROWS>(op, tm, stream);
}

template <int BM, int WM, bool GATED>
hipError_t launch_dense(const I4Operands &op, hipStream_t stream) {
  constexpr uint32_t kCols = kWaves * 16 * (GATED ? 1 : 2);
  const uint32_t rows = mx_max_grid(64 * kWaves) / ((op.N + kCols - 1u) / kCols) * BM;
  for (uint32_t m = 0; m < op.M; m += rows) {
    I4Operands part = op;
    part.A = op.A + (uint64_t)m * op.lda;
    part.C = op.C + (uint64_t)m * op.ldc;
    part.M = op.M - m < rows ? op.M - m : rows;
    const hipError_t e = launch_cfg<BM, WM, GATED, kDense>(part, (part.M + BM - 1u) / BM, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// What a way to multiply takes, in ns: one round of its tiles over 256 compute units (`first` and
// `first_step` for each 128 k), and every further one.  Measured at 24 to 1024 rows times 512, 5120 and 17408 outputs,
// K = 512 to 17408 (MI355X, weights from memory).  Several full rounds, where the clock falls, take up to a third longer than
// these say (4096 x 4096, K = 5120 160 us, here 127).
struct Cost {
  uint32_t bm, bn;  // outputs of a tile, half as many in the gated form
  uint32_t first, first_step, more, more_step;
};
constexpr Cost kCosts[] = {{16, 32, 3000, 70, 600, 88}, {32, 64, 3200, 220, 0, 230}, {64, 256, 3500, 1190, 1500, 1190},
                           {128, 256, 5000, 1490, 3000, 1490}};

// The same with lists, whose tiles first find their expert and rows: 64 to 2048 tokens of 8 of 64 experts, 2048 outputs,
// K = 1024, and gated 1024 outputs, K = 2048.
constexpr Cost kListCosts[] = {{16, 128, 8000, 330, 1300, 330}, {64, 256, 8000, 1190, 6000, 1190}, {128, 256, 10000, 1540, 12000, 1540}};

uint64_t cost_of(const Cost &c, uint64_t tiles, uint32_t steps) {
  const uint64_t rounds = (tiles + 255u) / 256u;
  return c.first + c.first_step * steps + (rounds > 1u ? (rounds - 1u) * (c.more + (uint64_t)c.more_step * steps) : 0u);
}

// The least cost and its index; chunks(bm): tiles of bm rows.
struct Choice {
  uint32_t way;
  uint64_t cost;
};
template <uint32_t COUNT, typename F>
Choice least(const Cost (&costs)[COUNT], const I4Operands &op, F &&chunks) {
  const uint32_t n = op.gated ? 2u * op.N : op.N;
  Choice best = {0u, ~0ull};
  for (uint32_t i = 0; i < COUNT; ++i) {
    const uint64_t x = cost_of(costs[i], chunks(costs[i].bm) * ((n + costs[i].bn - 1u) / costs[i].bn), op.K >> 7);
    if (x < best.cost) best = {i, x};
  }
  return best;
}

Choice least_product(const I4Operands &op) {
  if (op.M <= 16u) return {0u, 0u};
  return least(kCosts, op, [&](uint32_t bm) { return (uint64_t)((op.M + bm - 1u) / bm); });
}

hipError_t launch_way(const I4Operands &op, uint32_t way, hipStream_t stream) {
  if (way < 2u) return launch_i4_skinny(op, way == 1u, stream);
  if (way == 2u) return op.gated ? launch_dense<64, 1, true>(op, stream) : launch_dense<64, 1, false>(op, stream);
  return op.gated ? launch_dense<128, 2, true>(op, stream) : launch_dense<128, 2, false>(op, stream);
}

// Outputs from n on (a whole number of weight tiles): rows of scales in tiles and row by row are as long
I4Matrix from_row(const I4Matrix &m, const I4Operands &op, uint32_t n) {
  const uint64_t values = (uint64_t)n * op.K;
  return {m.W ? m.W + values / 2u : nullptr, m.S ? m.S + values / op.group : nullptr, m.Z ? m.Z + values / op.group : nullptr};
}

}  // namespace

// 0 and 1 are the kernel for few rows, which splits K eight ways over the waves of a tile: in chunks of 16 rows, and of 32
// with twice the weight rows, where its activations pass through fewer workgroups (96 x 5120, K = 5120 17.3 -> 12.3 us).
// Tiles cost less per output and wait for each of their steps: 256 x 5120, K = 5120 30.5 us in chunks, 51 in tiles of 64
// rows and 70 of 128; 1024 rows 143 in chunks of 16, 103 and 65 in tiles.
//
// A last round of tiles that leaves most compute units idle costs as much as a full one.  Where it is less, only as many
// outputs as fill whole rounds are left to the tiles, and the others get the way that is best for them, in a
// launch of their own (gated 500 x 17408, K = 5120 248 -> 205 us, 256 rows 153 -> 101; 2000 x 5120, K = 5120 138 -> 124).
hipError_t launch_i4_product(const I4Operands &op, hipStream_t stream) {
  const Choice whole = least_product(op);
  if (whole.way >= 2u) {
    const Cost &c = kCosts[whole.way];
    const uint32_t each = op.gated ? c.bn / 2u : c.bn, tn = (op.N + each - 1u) / each;
    const uint64_t tm = (op.M + c.bm - 1u) / c.bm, cols = tm * tn / 256u * 256u / tm;
    if (cols > 0u && cols < tn) {
      I4Operands first = op, rest = op;
      first.N = (uint32_t)cols * each;
      rest.N = op.N - first.N;
      rest.w = from_row(op.w, op, first.N);
      rest.up = from_row(op.up, op, first.N);
      rest.C = op.C + first.N;
      const Choice then = least_product(rest);
      if (cost_of(c, tm * cols, op.K >> 7) + then.cost < whole.cost) {
        const hipError_t e = launch_way(first, whole.way, stream);
        return e == hipSuccess ? launch_way(rest, then.way, stream) : e;
      }
    }
  }
  return launch_way(op, whole.way, stream);
}

// Whether one launch of tiles of bm rows holds the lists' products.  Rows of more than 4 GB are beyond its offsets.
static bool i4_tiles_fit(const I4Operands &op, uint32_t bm) {
  const uint32_t pairs = op.T * op.top_k, cols = kWaves * 16 * (op.gated ? 1 : 2);
  return (uint64_t)(op.gated ? op.T : pairs) * op.lda * 2u < 1ull << 32 &&
         i4_chunks(pairs, op.E, bm) * ((op.N + cols - 1u) / cols) <= mx_max_grid(64 * kWaves);
}

// With lists the few-row kernel takes what no launch of tiles holds, in several launches if need be.
bool i4_experts_fit(const I4Operands &op) {
  return op.order ? (uint64_t)op.T * op.top_k * op.N <= WQD_MOE_MAX_VALUES : i4_experts_skinny_fit(op);
}

// The lists' lengths are on the GPU: every expert is taken to have the mean of rows, and a quarter of them a chunk more.
hipError_t launch_i4_experts(const I4Operands &op, hipStream_t stream) {
  const uint32_t pairs = op.T * op.top_k, busy = pairs < op.E ? pairs : op.E;
  uint32_t way = 0;
  if (op.order && i4_tiles_fit(op, 128u)) {
    way = least(kListCosts, op, [&](uint32_t bm) {
            const uint64_t chunks = pairs / bm + busy / 4u;
            return chunks > busy ? chunks : (uint64_t)busy;
          }).way;
    if ((way == 0u && !i4_experts_skinny_fit(op)) || (way == 1u && !i4_tiles_fit(op, 64u))) way = 2u;
  }
  if (way == 0u) return launch_i4_experts_skinny(op, stream);
  const uint32_t chunks = (uint32_t)i4_chunks(pairs, op.E, way == 1u ? 64u : 128u);
  if (way == 1u) return op.gated ? launch_cfg<64, 1, true, kLists>(op, chunks, stream) : launch_cfg<64, 1, false, kLists>(op, chunks, stream);
  return op.gated ? launch_cfg<128, 2, true, kLists>(op, chunks, stream) : launch_cfg<128, 2, false, kLists>(op, chunks, stream);
}

}  // namespace wqd
