// Microscaled quantisation and its inverse, and the residual addition with a
// root-mean-square norm whose rows leave in 8 bits, for gfx950 (MI355X).
//
// Quantisation of a block of 32 values x: s = max(floor(log2 max|x|) - emax,
// -127) + 127 with emax 2 (E2M1) or 8 (E4M3), codes = x / 2^(s-127) rounded to
// nearest even and saturated; a block that holds an infinity or NaN has s =
// 255 and codes 0.  The division is a multiplication by a power of two, so a
// code is the correctly rounded one.
//
// All three kernels move a few bytes per value and compute little: memory
// bounds them.  A lane holds 8 consecutive values (16 bytes of BF16), a block
// is four neighbouring lanes, and its maximum two DPP steps: no LDS, and every
// load and store of a wave is one contiguous piece.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/wqd.h"
#include "mx_common.h"
#include "wqd_internal.h"

namespace wqd {
namespace {

constexpr uint32_t kThreads = 256;

struct Bf16 {
  static constexpr uint32_t kBytes = 2;
};
struct Fp16 {
  static constexpr uint32_t kBytes = 2;
};
struct Fp32 {
  static constexpr uint32_t kBytes = 4;
};

__device__ __forceinline__ void bf16x8_to_f32(const u32x4_t &w, float (&v)[8]) {
  v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}

// STREAM: 16-bit values of a call larger than the caches (launches of two
// groups per thread) pass them by; codes do not, as their reader comes next.
// 17408 x 5120 BF16 to 4 bits and back 93 -> 72 us.  FP32 values, 32 bytes per
// lane in two pieces, do not (back from 4 bits 101 us, streamed 144).
template <bool STREAM>
__device__ __forceinline__ u32x4_t load16(const uint8_t *p) {
  const u32x4_t *q = reinterpret_cast<const u32x4_t *>(p);
  if constexpr (STREAM) return __builtin_nontemporal_load(q);
  return *q;
}
template <bool STREAM>
__device__ __forceinline__ void store16(uint8_t *p, const u32x4_t &v) {
  u32x4_t *q = reinterpret_cast<u32x4_t *>(p);
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

template <typename T, bool STREAM = false>
__device__ __forceinline__ void load8(const uint8_t *p, float (&v)[8]) {
  const u32x4_t w = load16<STREAM>(p);
  if constexpr (std::is_same_v<T, Bf16>) {
    bf16x8_to_f32(w, v);
  } else if constexpr (std::is_same_v<T, Fp16>) {
    typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
    const f16x8_t h = __builtin_bit_cast(f16x8_t, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  } else {
    const u32x4_t w2 = load16<STREAM>(p + 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(w[i]);
      v[4 + i] = __uint_as_float(w2[i]);
    }
  }
}

template <typename T, bool STREAM = false>
__device__ __forceinline__ void store8(uint8_t *p, const float (&v)[8]) {
  if constexpr (std::is_same_v<T, Fp32>) {
    const u32x4_t a = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    const u32x4_t b = {__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    store16<STREAM>(p, a);
    store16<STREAM>(p + 16, b);
  } else if constexpr (std::is_same_v<T, Fp16>) {
    typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
    f16x8_t h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
    store16<STREAM>(p, __builtin_bit_cast(u32x4_t, h));
  } else {
    const u32x4_t w = {bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])};
    store16<STREAM>(p, w);
  }
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    m = m > b ? m : b;
  }
  return m;
}

// Quantise this lane's 8 values of a block and store its codes and, from the
// block's first lane, its scale byte; `grp` counts groups of 8 values from the
// start of the (contiguous) code and scale arrays.
template <bool FP4>
__device__ __forceinline__ void quantize_store(float (&v)[8], uint8_t *Q, uint8_t *S, uint64_t grp, bool live) {
  const uint32_t s = mx_scale_byte<FP4 ? kFp4Emax : kFp8Emax>(max_of_4_lanes(amax8(v)));
  const float inv = mx_inverse(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = s == 255u ? 0.0f : v[i] * inv;
  if (!live) return;
  if constexpr (FP4)
    *reinterpret_cast<uint32_t *>(Q + grp * 4u) = fp4x8(v);
  else
    *reinterpret_cast<u32x2_t *>(Q + grp * 8u) = fp8x8(v);
  if ((grp & 3u) == 0u) S[grp >> 2] = (uint8_t)s;
}

// The groups of 8 values are counted through all rows (row, then column);
// workgroup b owns groups [b * 256 * G, ...), its threads every 256th.  Rows
// are a multiple of four groups, so a block's four lanes are of one row.
template <int G>
struct Walk {
  uint64_t first;  // this thread's first group
  uint32_t row0, col;
  uint32_t gpr;  // groups per row
  __device__ __forceinline__ Walk(uint32_t K) : gpr(K >> 3) {
    const uint64_t base = (uint64_t)blockIdx.x * (kThreads * G);
    const uint64_t r = base / gpr;  // uniform: once per workgroup
    row0 = (uint32_t)r;
    col = (uint32_t)(base - r * gpr) + threadIdx.x;
    first = base + threadIdx.x;
  }
  __device__ __forceinline__ void at(int u, uint32_t &row, uint32_t &c) const {
    const uint32_t x = col + (uint32_t)u * kThreads;
    const uint32_t dr = x / gpr;
    row = row0 + dr;
    c = x - dr * gpr;
  }
};

template <typename T, bool FP4, int G>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const uint8_t *__restrict__ X, uint8_t *__restrict__ Q,
                                                            uint8_t *__restrict__ S, uint64_t groups, uint32_t K,
                                                            uint32_t ldx) {
  const Walk<G> walk(K);
  float v[G][8];
#pragma unroll
  for (int u = 0; u < G; ++u) {
    if (walk.first + (uint32_t)u * kThreads < groups) {
      uint32_t row, c;
      walk.at(u, row, c);
      load8<T, (G > 1 && T::kBytes == 2)>(X + ((uint64_t)row * ldx + 8u * c) * T::kBytes, v[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
    }
  }
#pragma unroll
  for (int u = 0; u < G; ++u) {
    const uint64_t grp = walk.first + (uint32_t)u * kThreads;
    quantize_store<FP4>(v[u], Q, S, grp, grp < groups);
  }
}

template <typename T, bool FP4, int G>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t *__restrict__ Q,
                                                              const uint8_t *__restrict__ S, uint8_t *__restrict__ Y,
                                                              uint64_t groups, uint32_t K, uint32_t ldy) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const Walk<G> walk(K);
  u32x2_t q[G];
  uint32_t s[G];
#pragma unroll
  for (int u = 0; u < G; ++u) {
    const uint64_t grp = walk.first + (uint32_t)u * kThreads;
    if (grp < groups) {
      if constexpr (FP4)
        q[u].x = *reinterpret_cast<const uint32_t *>(Q + grp * 4u);
      else
        q[u] = *reinterpret_cast<const u32x2_t *>(Q + grp * 8u);
      s[u] = S[grp >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < G; ++u) {
    if (walk.first + (uint32_t)u * kThreads >= groups) continue;
    f32x2_t p[4];
    if constexpr (FP4) {
      p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.0f, 0);
      p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.0f, 1);
      p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.0f, 2);
      p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.0f, 3);
    } else {
      p[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u].x, false);
      p[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u].x, true);
      p[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u].y, false);
      p[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u].y, true);
    }
    const float f = e8m0_value(s[u]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i >> 1][i & 1] * f;
    uint32_t row, c;
    walk.at(u, row, c);
    store8<T, (G > 1 && T::kBytes == 2)>(Y + ((uint64_t)row * ldy + 8u * c) * T::kBytes, v);
  }
}

// Groups per thread: two loads in flight per lane where there is work for it on
// every compute unit (17408 x 5120 to 4 bits 40 us; four 49), one where the call
// is small and latency counts.
constexpr uint64_t kManyGroups = 256ull * 4 * 4 * kThreads;

template <typename T, bool FP4>
hipError_t quantize_as(const void *X, void *Q, void *S, uint32_t M, uint32_t K, uint32_t ldx, hipStream_t stream) {
  const uint64_t groups = (uint64_t)M * (K >> 3);
  const int g = groups >= kManyGroups ? 2 : 1;
  const uint32_t grid = (uint32_t)((groups + kThreads * g - 1) / (kThreads * g));
  if (g == 2)
    hipLaunchKernelGGL((quantize_kernel<T, FP4, 2>), dim3(grid), dim3(kThreads), 0, stream,
                       static_cast<const uint8_t *>(X), static_cast<uint8_t *>(Q), static_cast<uint8_t *>(S), groups, K,
                       ldx);
  else
    hipLaunchKernelGGL((quantize_kernel<T, FP4, 1>), dim3(grid), dim3(kThreads), 0, stream,
                       static_cast<const uint8_t *>(X), static_cast<uint8_t *>(Q), static_cast<uint8_t *>(S), groups, K,
                       ldx);
  return hipGetLastError();
}

template <typename T, bool FP4>
hipError_t dequantize_as(const void *Q, const void *S, void *Y, uint32_t M, uint32_t K, uint32_t ldy, hipStream_t stream) {
  const uint64_t groups = (uint64_t)M * (K >> 3);
  const int g = groups >= kManyGroups ? 2 : 1;
  const uint32_t grid = (uint32_t)((groups + kThreads * g - 1) / (kThreads * g));
  if (g == 2)
    hipLaunchKernelGGL((dequantize_kernel<T, FP4, 2>), dim3(grid), dim3(kThreads), 0, stream,
                       static_cast<const uint8_t *>(Q), static_cast<const uint8_t *>(S), static_cast<uint8_t *>(Y), groups,
                       K, ldy);
  else
    hipLaunchKernelGGL((dequantize_kernel<T, FP4, 1>), dim3(grid), dim3(kThreads), 0, stream,
                       static_cast<const uint8_t *>(Q), static_cast<const uint8_t *>(S), static_cast<uint8_t *>(Y), groups,
                       K, ldy);
  return hipGetLastError();
}

// ------------------------------------------------------------------- norm
// One workgroup per row; a thread keeps its NCH groups of 8 values in
// registers between the sum of squares and the scaling, so the row is read
// once.  h is rounded to BF16 before the sum: the norm is that of the residual
// stream as the next layer reads it.  The sum and the products are held in 64
// bits and y is rounded to fp32 once: the squares of BF16 values leave fp32's
// range at either end, and in 32 bits the kernel is no faster (4096 x 5120 31.3
// against 30.5 us), as memory bounds it (147 MB, 4.8 TB/s).
constexpr uint32_t kNormMaxThreads = 1024;

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
  return x;
}

template <int NCH>
__global__ __launch_bounds__(kNormMaxThreads) void add_rmsnorm_kernel(const uint8_t *X, const uint8_t *R,
                                                                      const uint8_t *__restrict__ G, uint8_t *H,
                                                                      uint8_t *__restrict__ Y, uint8_t *__restrict__ Q,
                                                                      uint8_t *__restrict__ S, uint32_t K, uint32_t ldx,
                                                                      uint32_t ldr, float eps) {
  __shared__ double part[kNormMaxThreads / 64];
  const uint32_t row = blockIdx.x, tid = threadIdx.x, nt = blockDim.x;
  const uint32_t gpr = K >> 3;
  const uint8_t *x = X + (uint64_t)row * ldx * 2u;
  u32x4_t h[NCH], g[NCH];
  double sum = 0.0;
#pragma unroll
  for (int u = 0; u < NCH; ++u) {
    const uint32_t c = tid + (uint32_t)u * nt;
    h[u] = u32x4_t{0u, 0u, 0u, 0u};
    g[u] = u32x4_t{0u, 0u, 0u, 0u};
    if (c < gpr) {
      h[u] = *reinterpret_cast<const u32x4_t *>(x + 16u * c);
      g[u] = *reinterpret_cast<const u32x4_t *>(G + 16u * c);
    }
  }
  if (R) {  // uniform
    u32x4_t r[NCH];
#pragma unroll
    for (int u = 0; u < NCH; ++u) {
      const uint32_t c = tid + (uint32_t)u * nt;
      r[u] = u32x4_t{0u, 0u, 0u, 0u};
      if (c < gpr) r[u] = *reinterpret_cast<const u32x4_t *>(R + (uint64_t)row * ldr * 2u + 16u * c);
    }
#pragma unroll
    for (int u = 0; u < NCH; ++u) {
      const uint32_t c = tid + (uint32_t)u * nt;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[u][i] = bf16x2_rne(bf16_lo(h[u][i]) + bf16_lo(r[u][i]), bf16_hi(h[u][i]) + bf16_hi(r[u][i]));
      if (c < gpr) *reinterpret_cast<u32x4_t *>(H + (uint64_t)row * ldr * 2u + 16u * c) = h[u];
    }
  }
#pragma unroll
  for (int u = 0; u < NCH; ++u) {
    float v[8];
    bf16x8_to_f32(h[u], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)v[i], (double)v[i], sum);
  }
  sum = wave_sum(sum);
  if ((tid & 63u) == 0u) part[tid >> 6] = sum;
  __syncthreads();
  sum = 0.0;
  for (uint32_t w = 0; w < (nt >> 6); ++w) sum += part[w];
  const double inv = 1.0 / __builtin_sqrt(sum / (double)K + (double)eps);
#pragma unroll
  for (int u = 0; u < NCH; ++u) {
    const uint32_t c = tid + (uint32_t)u * nt;
    float v[8], w[8];
    bf16x8_to_f32(h[u], v);
    bf16x8_to_f32(g[u], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)((double)v[i] * inv * (double)w[i]);
    const uint64_t grp = (uint64_t)row * gpr + c;
    if (Y && c < gpr) store8<Bf16>(Y + grp * 16u, v);
    quantize_store<false>(v, Q, S, grp, c < gpr);
  }
}

template <int NCH>
hipError_t norm_as(const void *X, const void *R, const void *G, void *H, void *Y, void *Q, void *S, uint32_t M,
                   uint32_t K, uint32_t ldx, uint32_t ldr, float eps, hipStream_t stream) {
  const uint32_t per_thread = ((K >> 3) + NCH - 1) / NCH;
  const uint32_t threads = (per_thread + 63u) / 64u * 64u;
  hipLaunchKernelGGL((add_rmsnorm_kernel<NCH>), dim3(M), dim3(threads), 0, stream, static_cast<const uint8_t *>(X),
                     static_cast<const uint8_t *>(R), static_cast<const uint8_t *>(G), static_cast<uint8_t *>(H),
                     static_cast<uint8_t *>(Y), static_cast<uint8_t *>(Q), static_cast<uint8_t *>(S), K, ldx, ldr, eps);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const void *X, uint32_t type, void *Q, void *S, bool fp4, uint32_t M, uint32_t K,
                              uint32_t ldx, hipStream_t stream) {
  if (type == WQD_TYPE_BF16)
    return fp4 ? quantize_as<Bf16, true>(X, Q, S, M, K, ldx, stream)
               : quantize_as<Bf16, false>(X, Q, S, M, K, ldx, stream);
  if (type == WQD_TYPE_FP16)
    return fp4 ? quantize_as<Fp16, true>(X, Q, S, M, K, ldx, stream)
               : quantize_as<Fp16, false>(X, Q, S, M, K, ldx, stream);
  return fp4 ? quantize_as<Fp32, true>(X, Q, S, M, K, ldx, stream)
             : quantize_as<Fp32, false>(X, Q, S, M, K, ldx, stream);
}

hipError_t launch_mx_dequantize(const void *Q, const void *S, bool fp4, void *Y, uint32_t type, uint32_t M, uint32_t K,
                                uint32_t ldy, hipStream_t stream) {
  if (type == WQD_TYPE_BF16)
    return fp4 ? dequantize_as<Bf16, true>(Q, S, Y, M, K, ldy, stream)
               : dequantize_as<Bf16, false>(Q, S, Y, M, K, ldy, stream);
  if (type == WQD_TYPE_FP16)
    return fp4 ? dequantize_as<Fp16, true>(Q, S, Y, M, K, ldy, stream)
               : dequantize_as<Fp16, false>(Q, S, Y, M, K, ldy, stream);
  return fp4 ? dequantize_as<Fp32, true>(Q, S, Y, M, K, ldy, stream)
             : dequantize_as<Fp32, false>(Q, S, Y, M, K, ldy, stream);
}

hipError_t launch_add_rmsnorm_mx8(const void *X, const void *R, const void *G, void *H, void *Y, void *Q, void *S,
                                  uint32_t M, uint32_t K, uint32_t ldx, uint32_t ldr, float eps, hipStream_t stream) {
  // Few rows want one group per thread (one row of 5120 3.2 us, with two 3.4;
  // 256 rows 4.0, 4.3); from 1024 rows on two keep more loads in flight (1024
  // rows 9.7 -> 9.2 us, 8192 rows 58 -> 54, without a residual 4096 22 -> 17).
  const uint32_t gpr = K >> 3;
  if (gpr <= kNormMaxThreads && M < 1024u) return norm_as<1>(X, R, G, H, Y, Q, S, M, K, ldx, ldr, eps, stream);
  if (gpr <= 2 * kNormMaxThreads) return norm_as<2>(X, R, G, H, Y, Q, S, M, K, ldx, ldr, eps, stream);
  return norm_as<4>(X, R, G, H, Y, Q, S, M, K, ldx, ldr, eps, stream);
}

}  // namespace wqd
