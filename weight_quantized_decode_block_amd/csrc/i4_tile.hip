// Products with 4-bit integer weights for many rows, for gfx950 (MI355X): the
// operations of i4_skinny.hip, bound by the matrix instructions and by what feeds
// them.
//
// A workgroup of 8 waves owns BM rows and 128 NT weight rows (in the gated form
// 64 NT of both matrices) and walks K in steps of 128.  The waves stand side by side
// in n, so each converts its own weights only, once; all of them read all activations.
//
//   * Staging.  Activations, codes, scales and zero points go straight from memory to
//     LDS, PRE steps ahead of their use, into PRE + 1 buffers; a wave waits for its
//     own transfers by count.  Codes lie in the matrix operand's order, so a lane
//     reads back what its neighbours brought in whole KB.  Rows past the last one
//     repeat it; their outputs are not stored.
//   * Codes become the BF16 values of q - z (exact: integers of at most 8 bits):
//     1024 + q as FP16 by two integer instructions a pair, minus 1024 + z by
//     a mixed multiply-add each, and a conversion for two.  A step's codes are converted
//     between the matrix instructions of the step before.
//   * The sums of a group are a matrix accumulator of their own, which the scale
//     adds to the output's in fp32: nothing but the output is rounded.
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

// 16 (or 4) bytes per lane from voff of the buffer to LDS byte `lds` + 16 (4) *
// lane.  The transfer has no destination registers; it is waited for by count.
__device__ __forceinline__ void copy16_to_lds(uint32_t lds, rsrc_t r, uint32_t voff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(voff), "s"(r) : "memory");
}
__device__ __forceinline__ void copy4_to_lds(uint32_t lds, rsrc_t r, uint32_t voff) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(voff), "s"(r) : "memory");
}

// Wait until at most N of this wave's transfers are in flight and its LDS
// reads have returned, then meet the other waves.
template <int N>
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

constexpr int kDense = 0;  // rows m0 ..
constexpr int kLists = 1;  // rows of one expert's list

// LDS of a stage: activations, codes, scales, zero points (of each wave: NT tiles')
template <int BM, int NT, int NG, bool ZEROS>
constexpr uint32_t kStage = BM * 256 + kWaves * NT * (kI4Tile + 32 * NG + (ZEROS ? 16 * NG : 0));
template <int BM, int NT, int NG, bool ZEROS, int PRE>
constexpr uint32_t kLdsBytes = (PRE + 1) * kStage<BM, NT, NG, ZEROS>;

// What the conversion keeps in registers: a mask and 1024 twice as FP16, for one
// instruction that masks and sets, and a one that the compiler does not see, so
// that a mixed multiply-add widens and subtracts at once.
struct Constants {
  uint32_t mask, base;
  float one;
};

// 8 codes as the BF16 values of q - z; minus: -(1024 + z)
__device__ __forceinline__ bf16x8_t i4_values(uint32_t w, float minus, const Constants &k) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2_t x = __builtin_bit_cast(f16x2_t, (w >> (4 * i) & k.mask) | k.base);
    v[i] = bf16x2_rne(__builtin_fmaf((float)x.x, k.one, minus), __builtin_fmaf((float)x.y, k.one, minus));
  }
  return __builtin_bit_cast(bf16x8_t, v);
}

template <int BM, int NT, bool GATED, int NG, bool ZEROS, int ROWS, int PRE>
__global__ __launch_bounds__(64 * kWaves) void i4_tile_kernel(I4Operands op, uint32_t tm) {
  static_assert(!GATED || NT == 2, "a wave has a tile of either matrix");
  constexpr int MT = BM / 16, AU = BM / 32, NBUF = PRE + 1;
  constexpr int ND = AU + NT * (ZEROS ? 3 : 2);  // transfers of a wave and step
  constexpr uint32_t BNT = kWaves * NT / (GATED ? 2 : 1);  // 16-column tiles of the output
  constexpr uint32_t kW = BM * 256, kS = kW + kWaves * NT * kI4Tile, kZ = kS + kWaves * NT * 32 * NG;
  constexpr uint32_t kBuf = kStage<BM, NT, NG, ZEROS>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

  const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, g = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tiles = (op.N + 15u) >> 4, kt = op.K >> 7, tn = (tiles + BNT - 1u) / BNT;

  // Tile of this workgroup: the 8 XCDs, which take workgroups in turn, get
  // contiguous runs, and tiles run down four rows before the next column.
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
  auto pair_of = [&](uint32_t m) __attribute__((always_inline)) {
    const uint32_t p = (uint32_t)op.order[first + (m < rows ? m : rows - 1u)];
    return p < op.T * op.top_k ? p : 0u;
  };

  // Activations: units of 4 rows x 256 bytes; slot x of row m has piece x ^ (m % 16), so
  // that the sixteen lanes that an LDS read serves together meet all 64 banks.
  const uint32_t pitch = op.lda * 2u;
  const rsrc_t ar = ROWS == kDense ? bytes_rsrc(op.A, (uint64_t)first * pitch, (rows - 1u) * pitch + op.K * 2u)
                                   : bytes_rsrc(op.A, 0, ((GATED ? op.T : op.T * op.top_k) - 1u) * pitch + op.K * 2u);
  uint32_t aoff[AU];
#pragma unroll
  for (int i = 0; i < AU; ++i) {
    const uint32_t m = (wave + i * kWaves) * 4u + g;
    const uint32_t row = ROWS == kDense ? (m < rows ? m : rows - 1u) : (GATED ? pair_of(m) / op.top_k : pair_of(m));
    aoff[i] = row * pitch + (r ^ (m & 15u)) * 16u;
  }
  // this wave's weight tiles (gated: one of either matrix)
  const uint32_t t0 = col * BNT + (GATED ? wave : wave * NT);
  rsrc_t wr[NT], sr[NT], zr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const I4Matrix &m = GATED && i ? op.up : op.w;
    const uint32_t t = t0 + (GATED ? 0u : i);
    const uint64_t at = ((uint64_t)expert * tiles + (t < tiles ? t : tiles - 1u)) * kt;
    wr[i] = bytes_rsrc(m.W, at * kI4Tile, kt * kI4Tile);
    sr[i] = bytes_rsrc(m.S, at * (32u * NG), kt * (32u * NG));
    if constexpr (ZEROS) zr[i] = bytes_rsrc(m.Z, at * (16u * NG), kt * (16u * NG));
  }
  const uint32_t put_w = kW + wave * NT * kI4Tile, put_s = kS + wave * NT * (32 * NG), put_z = kZ + wave * NT * (16 * NG);
  auto issue_a = [&](uint32_t s) __attribute__((always_inline)) {
    const uint32_t base = lds0 + s % NBUF * kBuf, k = (s < kt ? s : kt - 1u) * 256u;
#pragma unroll
    for (int i = 0; i < AU; ++i) copy16_to_lds(base + (wave + i * kWaves) * 1024u, ar, aoff[i] + k);
  };
  auto issue_w = [&](uint32_t s) __attribute__((always_inline)) {
    const uint32_t base = lds0 + s % NBUF * kBuf, t = s < kt ? s : kt - 1u;
#pragma unroll
    for (int i = 0; i < NT; ++i) copy16_to_lds(base + put_w + i * kI4Tile, wr[i], t * kI4Tile + lane * 16u);
    if (lane < 8u * NG) {
#pragma unroll
      for (int i = 0; i < NT; ++i) copy4_to_lds(base + put_s + i * 32 * NG, sr[i], t * (32u * NG) + lane * 4u);
    }
    if constexpr (ZEROS) {
      if (lane < 4u * NG) {
#pragma unroll
        for (int i = 0; i < NT; ++i) copy4_to_lds(base + put_z + i * 16 * NG, zr[i], t * (16u * NG) + lane * 4u);
      }
    }
  };

  f32x4_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // A step's weights: values and scales
  struct Weights {
    bf16x8_t v[NT][4];
    float s[NT][NG];
  };
  struct Codes {
    u32x4_t w[NT];
    I4Groups<NG> s[NT];
  };
  Constants k = {0x000f000fu, 0x64006400u, 1.0f};
  asm volatile("" : "+s"(k.mask), "+v"(k.base), "+v"(k.one));
  auto read_codes = [&](uint32_t s) __attribute__((always_inline)) {
    const uint8_t *p = lds + s % NBUF * kBuf;
    Codes c;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      c.w[i] = *reinterpret_cast<const u32x4_t *>(p + put_w + i * kI4Tile + lane * 16u);
      c.s[i] = i4_load_groups<NG, ZEROS>(reinterpret_cast<const uint16_t *>(p + put_s + i * 32 * NG), p + put_z + i * 16 * NG, r);
    }
    return c;
  };
  // dword d (0 .. 3) of tile i
  auto convert = [&](const Codes &c, int i, int d, Weights &w) __attribute__((always_inline)) {
    w.v[i][d] = i4_values(c.w[i][d], -1024.0f - i4_zero_of(c.s[i], d * NG / 4), k);
    asm volatile("" : "+v"(w.v[i][d]));  // here, not where it is used
    if (d * NG % 4 == 0) w.s[i][d * NG / 4] = i4_scale_of(c.s[i], d * NG / 4, op.scale_bf16);
  };
  // The sums of the last group that was multiplied, and their scales: they join the
  // output's while the matrix instructions of the next one run.
  f32x4_t last[NT];
  float last_s[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    last[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    last_s[i] = 0.0f;
  }
  struct Rows {
    bf16x8_t v[4];
  };
  auto fold = [&](int j) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(last_s[i], last[i][e], acc[i][j][e]);
      asm volatile("" : "+v"(acc[i][j]));  // here, not where it is used
    }
  };
  auto step = [&](uint32_t s, const Weights &w, Weights &next) __attribute__((always_inline)) {
    step_barrier<(PRE - 1) * ND>();
    issue_a(s + PRE);
    issue_w(s + PRE + 1);
    const Codes c = read_codes(s + 1);
    const uint8_t *p = lds + s % NBUF * kBuf;
    auto read_a = [&](int j) __attribute__((always_inline)) {
      Rows a;
#pragma unroll
      for (uint32_t x = 0; x < 4; ++x)
        a.v[x] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t *>(p + (j * 16u + r) * 256u + ((4u * x + g) ^ r) * 16u));
      return a;
    };
    Rows a[2];
    a[0] = read_a(0);
    mx_unroll<0, MT>([&](auto J) __attribute__((always_inline)) {
      constexpr int j = decltype(J)::value;
      if constexpr (j + 1 < MT) a[(j + 1) & 1] = read_a(j + 1);
      mx_unroll<0, NG>([&](auto Q) __attribute__((always_inline)) {
        constexpr int q = decltype(Q)::value;
        f32x4_t t[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) t[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = q * 4 / NG; x < (q + 1) * 4 / NG; ++x)
#pragma unroll
          for (int i = 0; i < NT; ++i) t[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j & 1].v[x], w.v[i][x], t[i], 0, 0, 0);
        fold(q > 0 ? j : (j + MT - 1) % MT);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          last[i] = t[i];
          last_s[i] = w.s[i][q];
        }
      });
#pragma unroll
      for (int x = j * NT * 4 / MT; x < (j + 1) * NT * 4 / MT; ++x) convert(c, x / 4, x % 4, next);
      // matrix instructions and the others in turn
      constexpr int kOther = (8 * NG * NT / 2 + 20 * NT * 4 / MT) / (4 * NT) + 1;
      __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
      mx_unroll<0, 4 * NT>([&](auto) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, kOther, 0);
      });
      __builtin_amdgcn_sched_barrier(0);  // without it the registers of several rounds do not fit
    });
  };

  issue_w(0);
  mx_unroll<0, PRE>([&](auto d) __attribute__((always_inline)) {
    issue_a(decltype(d)::value);
    issue_w(decltype(d)::value + 1);
  });
  Weights even, odd;
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(PRE * ND) : "memory");
  {
    const Codes c = read_codes(0);
#pragma unroll
    for (int x = 0; x < NT * 4; ++x) convert(c, x / 4, x % 4, even);
  }
  uint32_t s = 0;
  for (; s + 1u < kt; s += 2u) {
    step(s, even, odd);
    step(s + 1u, odd, even);
  }
  if (s < kt) step(s, even, odd);
  fold(MT - 1);
  step_barrier<0>();  // nothing is in flight, and everybody has read the last stage

  const uint32_t n = r;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
      const uint32_t m = j * 16u + 4u * g + e;
      if (m >= rows) continue;
      const uint64_t row = ROWS == kDense ? first + m : pair_of(m);
#pragma unroll
      for (int i = 0; i < (GATED ? 1 : NT); ++i) {
        const uint32_t c = (t0 + i) * 16u + n;
        if (c >= op.N) continue;
        if constexpr (ROWS == kLists && !GATED) {
          op.Y[row * op.N + c] = acc[i][j][e];
        } else {
          const float y = GATED ? silu_times(acc[0][j][e], acc[NT - 1][j][e]) : acc[i][j][e];
          op.C[row * op.ldc + c] = (uint16_t)bf16x2_rne(y, 0.0f);
        }
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

template <int BM, int NT, bool GATED, int NG, bool ZEROS, int ROWS, int PRE>
hipError_t launch_kernel(const I4Operands &op, uint32_t tm, hipStream_t stream) {
  const auto kern = i4_tile_kernel<BM, NT, GATED, NG, ZEROS, ROWS, PRE>;
  constexpr uint32_t kLds = kLdsBytes<BM, NT, NG, ZEROS, PRE>;
  static_assert(kLds <= 160 * 1024, "one workgroup's LDS");
  static std::atomic<uint64_t> ready;  // devices on which the kernel may use that much LDS
  const hipError_t attr = allow_lds(reinterpret_cast<const void *>(kern), ready);
  if (attr != hipSuccess) return attr;
  constexpr uint32_t kCols = kWaves * NT * 16 / (GATED ? 2 : 1);
  hipLaunchKernelGGL(kern, dim3(tm * ((op.N + kCols - 1u) / kCols)), dim3(64 * kWaves), kLds, stream, op, tm);
  return hipGetLastError();
}

template <int BM, int NT, bool GATED, int ROWS, int PRE>
hipError_t launch_cfg(const I4Operands &op, uint32_t tm, hipStream_t stream) {
  const bool z = op.w.Z != nullptr;
  if (op.group == 128u)
    return z ? launch_kernel<BM, NT, GATED, 1, true, ROWS, PRE>(op, tm, stream) : launch_kernel<BM, NT, GATED, 1, false, ROWS, PRE>(op, tm, stream);
  if (op.group == 64u)
    return z ? launch_kernel<BM, NT, GATED, 2, true, ROWS, PRE>(op, tm, stream) : launch_kernel<BM, NT, GATED, 2, false, ROWS, PRE>(op, tm, stream);
  return z ? launch_kernel<BM, NT, GATED, 4, true, ROWS, PRE>(op, tm, stream) : launch_kernel<BM, NT, GATED, 4, false, ROWS, PRE>(op, tm, stream);
}

template <int BM, int NT, bool GATED, int PRE>
hipError_t launch_dense(const I4Operands &op, hipStream_t stream) {
  constexpr uint32_t kCols = kWaves * NT * 16 / (GATED ? 2 : 1);
  const uint32_t rows = mx_max_grid(64 * kWaves) / ((op.N + kCols - 1u) / kCols) * BM;
  for (uint32_t m = 0; m < op.M; m += rows) {
    I4Operands part = op;
    part.A = op.A + (uint64_t)m * op.lda;
    part.C = op.C + (uint64_t)m * op.ldc;
    part.M = op.M - m < rows ? op.M - m : rows;
    const hipError_t e = launch_cfg<BM, NT, GATED, kDense, PRE>(part, (part.M + BM - 1u) / BM, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_i4_product(const I4Operands &op, hipStream_t stream) {
  if (op.M <= 64u) return launch_i4_skinny(op, op.gated, stream);
  return op.gated ? launch_dense<128, 2, true, 1>(op, stream) : launch_dense<128, 2, false, 1>(op, stream);
}

hipError_t launch_i4_experts(const I4Operands &op, hipStream_t stream) {
  const uint32_t pairs = op.T * op.top_k;
  if (!op.order || pairs / op.E < 48u || (uint64_t)(op.gated ? op.T : pairs) * op.lda * 2u >= 1ull << 32)
    return launch_i4_experts_skinny(op, stream);
  const uint32_t chunks = (uint32_t)i4_chunks(pairs, op.E, 128u);
  return op.gated ? launch_cfg<128, 2, true, kLists, 1>(op, chunks, stream) : launch_cfg<128, 2, false, kLists, 1>(op, chunks, stream);
}

}  // namespace wqd
