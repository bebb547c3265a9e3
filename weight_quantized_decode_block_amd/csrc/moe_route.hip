// A router's choice of experts, the experts' lists of tokens and the weighted
// sum of the experts' outputs, for gfx950 (MI355X).
//
// Choice (moe_route_kernel): a wave takes a token; lane l holds experts l V ..
// l V + V - 1, so the lowest lane among equals has the lowest expert.  Scores
// and what is chosen by (score + bias) are 64-bit: a rounding to fewer bits would
// swap experts whose values differ by less.  The top_k rounds are a maximum over
// the wave each (DPP steps, no LDS).
//
// Lists (moe_lists_kernel): a workgroup per expert counts the pairs of all
// lower experts, which is where its own list begins, and writes its pairs in
// ascending order; no atomics, no second launch, no workspace.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/wqd.h"
#include "i4_common.h"
#include "mx_product.h"

namespace wqd {
namespace {

constexpr double kNone = -__builtin_huge_val();

template <int CTRL, int ROWS>
__device__ __forceinline__ double from_lane(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
  const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp((int)lo, (int)lo, CTRL, ROWS, 0xF, false);
  const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp((int)hi, (int)hi, CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)h << 32 | l);
}
__device__ __forceinline__ double read_lane(double x, uint32_t lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t l = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, (int)lane);
  const uint32_t h = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), (int)lane);
  return __builtin_bit_cast(double, (uint64_t)h << 32 | l);
}
// Largest value of a wave, none of them NaN
__device__ __forceinline__ double wave_max(double x) {
  x = __builtin_fmax(x, from_lane<0x111, 0xF>(x));  // from 1, 2, 4 and 8 lanes below in a row of 16
  x = __builtin_fmax(x, from_lane<0x112, 0xF>(x));
  x = __builtin_fmax(x, from_lane<0x114, 0xF>(x));
  x = __builtin_fmax(x, from_lane<0x118, 0xF>(x));
  x = __builtin_fmax(x, from_lane<0x142, 0xA>(x));  // the last lane of a row to the next row
  x = __builtin_fmax(x, from_lane<0x143, 0xC>(x));  // lane 31 to the upper half
  return read_lane(x, 63u);
}
// Sum over a wave, the same in every lane
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
  return x;
}

// Expert v of a lane, or the last one for those past it
template <int V>
__device__ __forceinline__ uint32_t held(uint32_t lane, int v, uint32_t E) {
  const uint32_t e = lane * V + v;
  return e < E ? e : E - 1u;
}

template <int V>
__global__ __launch_bounds__(256) void moe_route_kernel(MoeRoute op) {
  extern __shared__ __attribute__((aligned(16))) double shared[];  // of a choice by groups: each wave's values
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t t = blockIdx.x * 4u + wave;
  if (t >= op.T) return;  // no barriers below

  // An expert whose logit is NaN or minus infinity, or whose bias is, is never chosen.
  // All values are asked for before one is used, and without a branch between.
  double p[V], key[V];
  double top = kNone;
  uint32_t bits[V];
  float bias[V];
  const uint64_t row = (uint64_t)t * op.ld;
  if (op.type == WQD_TYPE_FP32) {
#pragma unroll
    for (int v = 0; v < V; ++v) bits[v] = static_cast<const uint32_t *>(op.logits)[row + held<V>(lane, v, op.E)];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) bits[v] = static_cast<const uint16_t *>(op.logits)[row + held<V>(lane, v, op.E)];
  }
  if (op.bias) {
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = op.bias[held<V>(lane, v, op.E)];
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float half = (float)__builtin_bit_cast(_Float16, (uint16_t)bits[v]);
    float x = op.type == WQD_TYPE_FP32 ? __uint_as_float(bits[v]) : op.type == WQD_TYPE_BF16 ? __uint_as_float(bits[v] << 16) : half;
    if (lane * V + v >= op.E) x = __builtin_nanf("");
    x = x > 3.402823466e38f ? 3.402823466e38f : x;  // an infinity is the largest value
    key[v] = x > -__builtin_inff() ? (double)x : kNone;
    top = __builtin_fmax(top, key[v]);
  }
  top = wave_max(top);
  if (op.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = 1.0 / (1.0 + exp(-key[v]));
  } else {
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = key[v] > kNone ? exp(key[v] - top) : 0.0;
      sum += p[v];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = p[v] / sum;
  }
  // Without a bias the order is that of the logits.
  if (op.bias) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t e = lane * V + v;
      const double b = e < op.E ? (double)bias[v] : kNone;
      key[v] = key[v] > kNone && b > kNone ? p[v] + b : kNone;
    }
  }

  if (op.groups > 1u) {
    // The groups of the largest sums of their group_top largest values; a lane takes a group.
    const uint32_t size = op.E / op.groups;
    double *mine = shared + wave * op.E;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t e = lane * V + v;
      if (e < op.E) mine[e] = op.bias || op.group_top == 1u || !(key[v] > kNone) ? key[v] : p[v];
    }
    double first = kNone, second = kNone;
    if (lane < op.groups) {
      for (uint32_t i = 0; i < size; ++i) {
        const double x = mine[lane * size + i];
        second = __builtin_fmax(second, __builtin_fmin(first, x));
        first = __builtin_fmax(first, x);
      }
    }
    const double score = op.group_top == 2u && second > kNone ? first + second : first;
    uint32_t ahead = 0;
    for (uint32_t i = 0; i < op.groups; ++i) {
      const double x = read_lane(score, i);
      ahead += x > score || (x == score && i < lane) ? 1u : 0u;
    }
    const uint64_t in = __ballot(lane < op.groups && ahead < op.top_groups);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t e = lane * V + v;
      if (e < op.E && !(in >> (e / size) & 1u)) key[v] = kNone;
    }
  }

  uint32_t taken = 0, id = ~0u;  // this lane's experts that are taken; the choice of slot `lane`
  double weight = 0.0, sum = 0.0;
  for (uint32_t s = 0; s < op.top_k; ++s) {
    double best = kNone, score = 0.0;
    uint32_t at = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!(taken >> v & 1u) && key[v] > best) {
        best = key[v];
        score = p[v];
        at = v;
      }
    const double m = wave_max(best);
    if (!(m > kNone)) break;
    const uint32_t l = (uint32_t)__builtin_ctzll(__ballot(best == m));
    const uint32_t e = (uint32_t)__builtin_amdgcn_readlane((int)at, (int)l) + l * V;
    const double w = read_lane(score, l);
    if (lane == l) taken |= 1u << at;
    if (lane == s) {
      id = e;
      weight = w;
    }
    sum += w;
  }
  if (lane < op.top_k) {
    if (op.renormalize) weight = sum > 0.0 ? weight / sum : 0.0;
    op.ids[(uint64_t)t * op.top_k + lane] = (int32_t)id;
    op.weights[(uint64_t)t * op.top_k + lane] = (float)(weight * (double)op.scale);
  }
}

template <int V>
hipError_t launch_route(const MoeRoute &op, hipStream_t stream) {
  hipLaunchKernelGGL((moe_route_kernel<V>), dim3((op.T + 3u) / 4u), dim3(256), op.groups > 1u ? 4u * op.E * 8u : 0u, stream, op);
  return hipGetLastError();
}

// kBatch loads of 256 pairs of a wave in flight: up to 32768 pairs are read once only (4096 tokens of 8 of 64 experts 6.5 us,
// 1 token 3.5), beyond that twice (8192 tokens 11.6).  Every workgroup counts all pairs, so that the work grows as pairs
// times experts: 8192 tokens of 8 of 512 experts 19.7 us, 131072 of 256 197.
constexpr uint32_t kListWaves = 16, kBatch = 8;

typedef uint32_t ids_t __attribute__((ext_vector_type(4), aligned(4)));

// Workgroup e < E writes expert e's list; workgroup E the lists' end and what is behind it.
__global__ __launch_bounds__(64 * kListWaves) void moe_lists_kernel(const int32_t *__restrict__ ids, int32_t *__restrict__ order,
                                                                    int32_t *__restrict__ offsets, uint32_t pairs, uint32_t E) {
  __shared__ uint32_t counts[2][kListWaves];
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), e = blockIdx.x;
  // each wave its own stretch of pairs, in whole rounds of 256: four neighbours a lane
  const uint32_t each = ((pairs + 255u) / 256u + kListWaves - 1u) / kListWaves * 256u;
  const uint32_t from = wave * each < pairs ? wave * each : pairs, to = pairs - from < each ? pairs : from + each;
  uint32_t id[kBatch][4];
  auto load = [&](uint32_t i0) __attribute__((always_inline)) {
#pragma unroll
    for (uint32_t b = 0; b < kBatch; ++b) {
      const uint32_t p = i0 + b * 256u + lane * 4u;
      ids_t v = {~0u, ~0u, ~0u, ~0u};
      if (p + 3u < to) {
        v = *reinterpret_cast<const ids_t *>(ids + p);
      } else {
#pragma unroll
        for (uint32_t j = 0; j < 3; ++j)
          if (p + j < to) v[j] = (uint32_t)ids[p + j];
      }
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) id[b][j] = v[j];
    }
  };
  uint32_t below = 0, own = 0;
  for (uint32_t i0 = from; i0 < to; i0 += 256u * kBatch) {
    load(i0);
#pragma unroll
    for (uint32_t b = 0; b < kBatch; ++b) {
      if (i0 + b * 256u >= to) break;
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) {
        below += (uint32_t)__builtin_popcountll(__ballot(id[b][j] < e));
        own += (uint32_t)__builtin_popcountll(__ballot(id[b][j] == e));
      }
    }
  }
  if (lane == 0u) {
    counts[0][wave] = below;
    counts[1][wave] = own;
  }
  __syncthreads();
  uint32_t start = 0, place = 0;
  for (uint32_t w = 0; w < kListWaves; ++w) {
    start += counts[0][w];
    place += w < wave ? counts[1][w] : 0u;
  }
  if (threadIdx.x == 0u) offsets[e] = (int32_t)start;
  if (e == E) {
    for (uint32_t i = start + threadIdx.x; i < pairs; i += 64u * kListWaves) order[i] = -1;
    return;
  }
  place += start;
  for (uint32_t i0 = from; i0 < to; i0 += 256u * kBatch) {
    if (each > 256u * kBatch) load(i0);
#pragma unroll
    for (uint32_t b = 0; b < kBatch; ++b) {
      if (i0 + b * 256u >= to) break;
      uint32_t before = 0, count = 0;
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) {
        const uint64_t set = __ballot(id[b][j] == e);
        before = __builtin_amdgcn_mbcnt_hi((uint32_t)(set >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)set, before));
        count += (uint32_t)__builtin_popcountll(set);
      }
      int32_t *to_list = order + place + before;
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        if (id[b][j] == e) *to_list++ = (int32_t)(i0 + b * 256u + lane * 4u + j);
      place += count;
    }
  }
}

// A thread adds four columns of a token's rows in slot order; slots without an
// expert of these are passed over.  Rows of kSlots slots are in flight at once (33 tokens of
// 8 slots, 2048 columns: with the products 27.0 -> 25.2 us; 2048 tokens: the same, 28
// us for 142 MB).
constexpr uint32_t kSlots = 8;

__global__ __launch_bounds__(256) void moe_combine_kernel(I4Operands op, uint64_t from) {
  const uint32_t pieces = (op.N + 3u) / 4u;
  const uint64_t x = from + (uint64_t)blockIdx.x * 256u + threadIdx.x;
  const uint32_t t = (uint32_t)(x / pieces), n = (uint32_t)(x - (uint64_t)t * pieces) * 4u;
  if (x >= (uint64_t)op.T * pieces) return;
  const bool whole = op.N % 4u == 0u;
  f32x4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t s0 = 0; s0 < op.top_k; s0 += kSlots) {
    bool here[kSlots];
    float w[kSlots];
    f32x4_t y[kSlots];
#pragma unroll
    for (uint32_t i = 0; i < kSlots; ++i) {
      const uint32_t s = s0 + i < op.top_k ? s0 + i : op.top_k - 1u, p = t * op.top_k + s;
      here[i] = s0 + i < op.top_k && (uint32_t)op.ids[p] < op.E;
      w[i] = op.weights[p];
    }
#pragma unroll
    for (uint32_t i = 0; i < kSlots; ++i) {
      y[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      const float *row = op.Y + (uint64_t)(t * op.top_k + s0 + i) * op.N + n;
      if (here[i] && whole) y[i] = *reinterpret_cast<const f32x4_t *>(row);
      if (here[i] && !whole) {
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
          if (n + j < op.N) y[i][j] = row[j];
      }
    }
#pragma unroll
    for (uint32_t i = 0; i < kSlots; ++i)
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) c[j] = here[i] ? __builtin_fmaf(w[i], y[i][j], c[j]) : c[j];
  }
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j)
    if (n + j < op.N) op.C[(uint64_t)t * op.ldc + n + j] = (uint16_t)bf16x2_rne(c[j], 0.0f);
}

}  // namespace

hipError_t launch_moe_route(const MoeRoute &op, hipStream_t stream) {
  if (op.E <= 64u) return launch_route<1>(op, stream);
  if (op.E <= 128u) return launch_route<2>(op, stream);
  if (op.E <= 256u) return launch_route<4>(op, stream);
  if (op.E <= 512u) return launch_route<8>(op, stream);
  return launch_route<16>(op, stream);
}

hipError_t launch_moe_lists(const int32_t *ids, int32_t *order, int32_t *offsets, uint32_t pairs, uint32_t E,
                            hipStream_t stream) {
  hipLaunchKernelGGL(moe_lists_kernel, dim3(E + 1u), dim3(64 * kListWaves), 0, stream, ids, order, offsets, pairs, E);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const I4Operands &op, hipStream_t stream) {
  const uint64_t threads = (uint64_t)op.T * ((op.N + 3u) / 4u), most = (uint64_t)mx_max_grid(256) * 256u;
  for (uint64_t from = 0; from < threads; from += most) {
    const uint64_t left = threads - from < most ? threads - from : most;
    hipLaunchKernelGGL(moe_combine_kernel, dim3((uint32_t)((left + 255u) / 256u)), dim3(256), 0, stream, op, from);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace wqd
