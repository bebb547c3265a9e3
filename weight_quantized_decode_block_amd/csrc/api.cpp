// C-ABI layer of libwqd.so: argument validation, Q2_0 row chunking, device
// checks and launch dispatch.  Every check runs before the first HIP call, so
// argument errors are reported the same way on a machine without a GPU.
//
// Behaviour follows page "gemv_q2_vec.rs" (q2_0_gemv_vec launcher; the
// batched launcher's Q2_BATCHM_MAX_M chunking, batchm_row_chunks and
// batchm_launch_chunks) and page "w8a16_gemm_m16.rs" (the checks of
// w8a16_gemm_m16 and its _n64 and _strided variants).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <atomic>

#include "../../include/wqd.h"
#include "wqd_internal.h"

namespace {

thread_local char g_last_error[512] = "";

int fail(int code, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return code;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// 0 = not yet checked, 1 = gfx950, 2 = other architecture.  Written once
// per device (racing writers store the same value), read without a lock.
constexpr int kMaxDevices = 64;
std::atomic<int> g_dev_state[kMaxDevices];

// Confirms a current HIP device exists and is a gfx950 part (the only code
// object this library carries).
int check_device(const char *fn) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return fail(WQD_ENODEV, "%s: no usable HIP device (%s)", fn, hipGetErrorString(e));
  }
  if (dev >= kMaxDevices) return fail(WQD_ENODEV, "%s: device index %d too large", fn, dev);
  int state = g_dev_state[dev].load(std::memory_order_acquire);
  if (state == 0) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return fail(WQD_EHIP, "%s: hipGetDeviceProperties: %s", fn, hipGetErrorString(e));
    state = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_dev_state[dev].store(state, std::memory_order_release);
  }
  if (state != 1)
    return fail(WQD_EUNSUPPORTED, "%s: device %d is not gfx950 (this library carries gfx950 code only)", fn, dev);
  return WQD_OK;
}

// Q2_0 matrix-core row tiers (include/wqd.h, WQD_Q2_0_TIER_WIDTHS): widths 1
// and 8 are the base tiers, 2, 4 and 6 the exact-row tiers.
constexpr uint32_t kTierWidths[WQD_Q2_0_TIER_COUNT] = WQD_Q2_0_TIER_WIDTHS;
constexpr bool kTierExact[WQD_Q2_0_TIER_COUNT] = {false, true, true, true, false};
constexpr uint32_t kTiersCompiled = (1u << WQD_Q2_0_TIER_COUNT) - 1u;

// Kernel for Q2_0, chosen from N and K only (never M), so batched rows stay
// bit-identical to M=1 rows: the matrix-core kernels when K is a multiple of
// 256 from 1024 up and the weights are under 2^31 bytes, on the row tier
// q2_0_tier_width(m), else the vector-ALU kernel.  The two families differ
// from each other only by fp32 rounding order; every matrix-core kernel and
// tier gives the same bits.  The presence of WQD_Q2_0_VALU (any value; read
// once per process) forces the vector-ALU kernel everywhere, for A/B runs.
hipError_t launch_q2_0(const void *A, const void *B, void *C, uint32_t N, uint32_t K, uint32_t m,
                       hipStream_t stream) {
  static const bool valu = std::getenv("WQD_Q2_0_VALU") != nullptr;
  const uint32_t width = q2_0_tier_width(m);
  if (!valu && width != 0 && wqd::q2_0_pairs_supports(N, K))
    return wqd::launch_q2_0_pairs(A, B, C, N, K, m, width, stream);
  return wqd::launch_q2_0_valu(A, B, C, N, K, m, stream);
}

int check_launch(const char *fn, hipError_t e) {
  if (e == hipSuccess) e = hipGetLastError();
  if (e != hipSuccess) return fail(WQD_EHIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return WQD_OK;
}

int validate_q2_0(const char *fn, const void *A, const void *B, void *C, uint32_t N,
                  uint32_t K, uint32_t group) {
  if (!A || !B || !C) return fail(WQD_ENULL, "%s: A, B and C must be non-NULL", fn);
  if (group != WQD_Q2_0_GROUP) return fail(WQD_EINVAL, "%s: group=%u, only 128 is supported", fn, group);
  if (N == 0) return fail(WQD_EINVAL, "%s: N must be >= 1", fn);
  if (K == 0 || K % WQD_Q2_0_GROUP != 0) return fail(WQD_EINVAL, "%s: K=%u is not a positive multiple of 128", fn, K);
  if (K > WQD_Q2_0_MAX_K) return fail(WQD_EUNSUPPORTED, "%s: K=%u above %u", fn, K, (unsigned)WQD_Q2_0_MAX_K);
  if (!aligned(A, 16)) return fail(WQD_EALIGN, "%s: A must be 16-byte aligned", fn);
  if (!aligned(B, 4)) return fail(WQD_EALIGN, "%s: B must be 4-byte aligned", fn);
  if (!aligned(C, 2)) return fail(WQD_EALIGN, "%s: C must be 2-byte aligned", fn);
  return WQD_OK;
}

// Checks shared by the three W8A16 entry points (page "w8a16_gemm_m16.rs":
// 1 <= m <= 16, K a multiple of 128).
int validate_w8a16(const char *fn, const void *A, const void *W, const float *S, void *C, uint32_t M,
                   uint32_t N, uint32_t K) {
  if (!A || !W || !S || !C) return fail(WQD_ENULL, "%s: A, W, S and C must be non-NULL", fn);
  if (M < 1 || M > WQD_W8A16_MAX_M) return fail(WQD_EINVAL, "%s: m=%u outside 1..16 (the M tile)", fn, M);
  if (K == 0 || K % WQD_W8A16_BLOCK != 0)
    return fail(WQD_EINVAL, "%s: K=%u is not a positive multiple of 128 (block-scale granularity)", fn, K);
  if (N == 0) return fail(WQD_EINVAL, "%s: N must be >= 1", fn);
  if (!aligned(A, 16)) return fail(WQD_EALIGN, "%s: A must be 16-byte aligned", fn);
  if (!aligned(W, 16)) return fail(WQD_EALIGN, "%s: W must be 16-byte aligned", fn);
  if (!aligned(S, 4)) return fail(WQD_EALIGN, "%s: S must be 4-byte aligned", fn);
  if (!aligned(C, 2)) return fail(WQD_EALIGN, "%s: C must be 2-byte aligned", fn);
  return WQD_OK;
}

// Row pitches of the strided entry points (page "w8a16_gemm_m16.rs", doc of
// w8a16_gemm_m16_strided): each covers its row, the activation pitch keeps
// rows 16-byte aligned, and the strided span fits 32-bit element offsets.
int validate_pitches(const char *fn, uint32_t M, uint32_t N, uint32_t K, uint32_t a_row_stride,
                     uint32_t c_row_stride) {
  if (a_row_stride < K || c_row_stride < N)
    return fail(WQD_EINVAL, "%s: row pitches must cover the rows (a_row_stride=%u < K=%u or c_row_stride=%u < N=%u)",
                fn, a_row_stride, K, c_row_stride, N);
  if (a_row_stride % 8 != 0)
    return fail(WQD_EINVAL, "%s: a_row_stride=%u is not a multiple of 8 (16-byte activation rows)", fn, a_row_stride);
  if (static_cast<uint64_t>(M - 1) * a_row_stride + K > 0xFFFFFFFFull ||
      static_cast<uint64_t>(M - 1) * c_row_stride + N > 0xFFFFFFFFull)
    return fail(WQD_EINVAL, "%s: row pitches too large (the strided span exceeds 2^32 elements)", fn);
  return WQD_OK;
}

// Rows of a microscaled quantisation or its inverse: the values' type and
// pitch, the format, and sizes that one launch covers.
int validate_mx_rows(const char *fn, const void *V, const char *v_name, uint32_t type, const void *Q, const void *S,
                     uint32_t format, uint32_t M, uint32_t K, uint32_t row_stride) {
  if (M && (!V || !Q || !S)) return fail(WQD_ENULL, "%s: %s, Q and S must be non-NULL", fn, v_name);
  if (type != WQD_TYPE_BF16 && type != WQD_TYPE_FP16 && type != WQD_TYPE_FP32)
    return fail(WQD_EINVAL, "%s: type %u of %s is not BF16, FP16 or FP32", fn, type, v_name);
  if (format != WQD_MXFP4 && format != WQD_MXFP8)
    return fail(WQD_EINVAL, "%s: format %u is neither MXFP4 nor MXFP8", fn, format);
  if (K == 0 || K % WQD_MX_BLOCK != 0) return fail(WQD_EINVAL, "%s: K=%u is not a positive multiple of 32", fn, K);
  if (K > WQD_Q2_0_MAX_K) return fail(WQD_EUNSUPPORTED, "%s: K=%u above %u", fn, K, (unsigned)WQD_Q2_0_MAX_K);
  const uint32_t piece = type == WQD_TYPE_FP32 ? 4u : 8u;
  if (row_stride < K || row_stride % piece != 0)
    return fail(WQD_EINVAL, "%s: row stride %u must be at least K=%u and a multiple of %u (16-byte rows)", fn,
                row_stride, K, piece);
  if (static_cast<uint64_t>(M) * K > WQD_MX_MAX_VALUES)
    return fail(WQD_EUNSUPPORTED, "%s: %u rows of %u values are too many for one call", fn, M, K);
  if (!aligned(V, 16)) return fail(WQD_EALIGN, "%s: %s must be 16-byte aligned", fn, v_name);
  if (!aligned(Q, 16)) return fail(WQD_EALIGN, "%s: Q must be 16-byte aligned", fn);
  return WQD_OK;
}

// One product or gated pair of products with MXFP4 weights: checks, then the
// kernel.  A BF16 call has no activation scales; a quantised one has pitch K.
int run_mx_product(const char *fn, wqd::MxOperands op, wqd::MxFormat fmt, bool gated, hipStream_t stream) {
  const bool bf16 = fmt == wqd::MxFormat::kBf16;
  if (!op.W || !op.WS || (gated && (!op.WU || !op.WUS)) || (op.M && (!op.A || !op.out.C || (!bf16 && !op.AS))))
    return fail(WQD_ENULL, "%s: operands must be non-NULL", fn);
  if (op.N == 0) return fail(WQD_EINVAL, "%s: N must be >= 1", fn);
  if (op.K == 0 || op.K % 128u != 0) return fail(WQD_EINVAL, "%s: K=%u is not a positive multiple of 128", fn, op.K);
  if (op.K > WQD_MX_MAX_K) return fail(WQD_EUNSUPPORTED, "%s: K=%u above %u", fn, op.K, (unsigned)WQD_MX_MAX_K);
  if (op.lda < op.K || op.out.ldc < op.N)
    return fail(WQD_EINVAL, "%s: row strides must cover the rows (a_row_stride=%u < K=%u or c_row_stride=%u < N=%u)",
                fn, op.lda, op.K, op.out.ldc, op.N);
  if (op.lda % 8u != 0)
    return fail(WQD_EINVAL, "%s: a_row_stride=%u is not a multiple of 8 (16-byte activation rows)", fn, op.lda);
  if (op.lda > WQD_MX_MAX_STRIDE)
    return fail(WQD_EUNSUPPORTED, "%s: a_row_stride=%u above %u", fn, op.lda, (unsigned)WQD_MX_MAX_STRIDE);
  if (op.M > WQD_MX_MAX_ROWS || op.N > WQD_MX_MAX_ROWS)
    return fail(WQD_EUNSUPPORTED, "%s: M=%u or N=%u above %u", fn, op.M, op.N, (unsigned)WQD_MX_MAX_ROWS);
  if (!aligned(op.A, 16)) return fail(WQD_EALIGN, "%s: A must be 16-byte aligned", fn);
  if (!aligned(op.W, 16) || !aligned(op.WU, 16)) return fail(WQD_EALIGN, "%s: weights must be 16-byte aligned", fn);
  if (!aligned(op.AS, 4) || !aligned(op.WS, 4) || !aligned(op.WUS, 4))
    return fail(WQD_EALIGN, "%s: scales must be 4-byte aligned", fn);
  if (!aligned(op.out.C, 2)) return fail(WQD_EALIGN, "%s: C must be 2-byte aligned", fn);
  if (op.M == 0) return WQD_OK;  // no rows: nothing to launch
  if (int rc = check_device(fn)) return rc;
  op.out.wide = aligned(op.out.C, 16) && op.out.ldc % 8u == 0 ? 2u : (aligned(op.out.C, 8) && op.out.ldc % 4u == 0 ? 1u : 0u);
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_mx_product(op, fmt, gated, stream));
}

wqd::MxOperands mx_operands(const void *A, const void *AS, const void *W, const void *WS, const void *WU,
                            const void *WUS, void *C, uint32_t M, uint32_t N, uint32_t K, uint32_t lda, uint32_t ldc) {
  return {A, AS, W, WS, WU, WUS, M, N, K, lda, {static_cast<uint16_t *>(C), ldc, 0u}};
}

// Checks shared by the products with 4-bit integer weights: matrices (`both`:
// two of them), their scales and zero points, and what the kernels' sizes assume.
int validate_i4(const char *fn, const wqd::I4Operands &op, bool both, uint32_t scales) {
  const uint32_t scale_type = scales & ~(uint32_t)WQD_I4_BY_ROW;
  if (!op.w.W || !op.w.S || (both && (!op.up.W || !op.up.S)))
    return fail(WQD_ENULL, "%s: weights and scales must be non-NULL", fn);
  if (both && !op.w.Z != !op.up.Z)
    return fail(WQD_ENULL, "%s: zero points of both matrices must be given or be NULL", fn);
  if (op.N == 0) return fail(WQD_EINVAL, "%s: N must be >= 1", fn);
  if (op.K == 0 || op.K % 128u != 0) return fail(WQD_EINVAL, "%s: K=%u is not a positive multiple of 128", fn, op.K);
  if (op.group != 32u && op.group != 64u && op.group != 128u)
    return fail(WQD_EINVAL, "%s: group=%u is not 32, 64 or 128", fn, op.group);
  if (scale_type != WQD_TYPE_FP16 && scale_type != WQD_TYPE_BF16)
    return fail(WQD_EINVAL, "%s: scale type %u is neither FP16 nor BF16", fn, scale_type);
  if (op.K > WQD_MX_MAX_K) return fail(WQD_EUNSUPPORTED, "%s: K=%u above %u", fn, op.K, (unsigned)WQD_MX_MAX_K);
  if (op.N > WQD_MX_MAX_ROWS) return fail(WQD_EUNSUPPORTED, "%s: N=%u above %u", fn, op.N, (unsigned)WQD_MX_MAX_ROWS);
  if (op.lda < op.K || op.ldc < op.N)
    return fail(WQD_EINVAL, "%s: row strides must cover the rows (%u < K=%u or %u < N=%u)", fn, op.lda, op.K, op.ldc, op.N);
  if (op.lda % 8u != 0)
    return fail(WQD_EINVAL, "%s: a_row_stride=%u is not a multiple of 8 (16-byte activation rows)", fn, op.lda);
  if (op.lda > WQD_MX_MAX_STRIDE)
    return fail(WQD_EUNSUPPORTED, "%s: a_row_stride=%u above %u", fn, op.lda, (unsigned)WQD_MX_MAX_STRIDE);
  if (!aligned(op.A, 16)) return fail(WQD_EALIGN, "%s: activations must be 16-byte aligned", fn);
  if (!aligned(op.w.W, 16) || !aligned(op.up.W, 16)) return fail(WQD_EALIGN, "%s: weights must be 16-byte aligned", fn);
  // row by row what a row has for 128 k is one load
  const uint32_t sa = op.by_row ? 256u / op.group : 16u, za = op.by_row ? 128u / op.group : 16u;
  if (!aligned(op.w.S, sa) || !aligned(op.up.S, sa)) return fail(WQD_EALIGN, "%s: scales must be %u-byte aligned", fn, sa);
  if (!aligned(op.w.Z, za) || !aligned(op.up.Z, za))
    return fail(WQD_EALIGN, "%s: zero points must be %u-byte aligned", fn, za);
  if (!aligned(op.C, 2)) return fail(WQD_EALIGN, "%s: C must be 2-byte aligned", fn);
  return WQD_OK;
}

int run_i4_product(const char *fn, const wqd::I4Operands &op, uint32_t scales, hipStream_t stream) {
  if (op.M && (!op.A || !op.C)) return fail(WQD_ENULL, "%s: A and C must be non-NULL", fn);
  if (int rc = validate_i4(fn, op, op.gated, scales)) return rc;
  if (op.M > WQD_MX_MAX_ROWS) return fail(WQD_EUNSUPPORTED, "%s: M=%u above %u", fn, op.M, (unsigned)WQD_MX_MAX_ROWS);
  if (op.M == 0) return WQD_OK;  // no rows: nothing to launch
  if (int rc = check_device(fn)) return rc;
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_i4_product(op, stream));
}

// Sizes of a routed call.
int validate_routes(const char *fn, uint32_t T, uint32_t top_k, uint32_t E) {
  if (E == 0 || E > WQD_MOE_MAX_EXPERTS)
    return fail(WQD_EINVAL, "%s: E=%u is not from 1 to %u", fn, E, (unsigned)WQD_MOE_MAX_EXPERTS);
  if (top_k == 0 || top_k > E || top_k > WQD_MOE_MAX_TOP_K)
    return fail(WQD_EINVAL, "%s: top_k=%u is not from 1 to E=%u and %u", fn, top_k, E, (unsigned)WQD_MOE_MAX_TOP_K);
  if ((uint64_t)T * top_k > WQD_MOE_MAX_PAIRS)
    return fail(WQD_EUNSUPPORTED, "%s: T=%u tokens with top_k=%u are too many for one call", fn, T, top_k);
  return WQD_OK;
}

int run_i4_experts(const char *fn, const wqd::I4Operands &op, uint32_t scales, hipStream_t stream) {
  if (op.T && (!op.A || !op.C || !op.ids || (!op.gated && !op.weights)))
    return fail(WQD_ENULL, "%s: activations, ids, weights and outputs must be non-NULL", fn);
  if (op.T && !op.order != !op.offsets) return fail(WQD_ENULL, "%s: order and offsets must both be given or both be NULL", fn);
  if (op.T && !op.gated && op.order && !op.Y) return fail(WQD_ENULL, "%s: Y must be non-NULL where lists are given", fn);
  if (int rc = validate_routes(fn, op.T, op.top_k, op.E)) return rc;
  if (int rc = validate_i4(fn, op, op.gated, scales)) return rc;
  if (!aligned(op.ids, 4) || !aligned(op.order, 4) || !aligned(op.offsets, 4) || !aligned(op.weights, 4))
    return fail(WQD_EALIGN, "%s: ids, weights and lists must be 4-byte aligned", fn);
  if (!aligned(op.Y, 16)) return fail(WQD_EALIGN, "%s: Y must be 16-byte aligned", fn);
  if (op.T == 0) return WQD_OK;
  if (!wqd::i4_experts_fit(op))
    return fail(WQD_EUNSUPPORTED, "%s: T=%u tokens of top_k=%u experts times N=%u are too many for one call", fn, op.T, op.top_k, op.N);
  if (int rc = check_device(fn)) return rc;
  (void)hipGetLastError();
  if (int rc = check_launch(fn, wqd::launch_i4_experts(op, stream))) return rc;
  return !op.gated && op.order ? check_launch(fn, wqd::launch_moe_combine(op, stream)) : WQD_OK;
}

// How the scales of a call come (WQD_TYPE_* and WQD_I4_BY_ROW).
void set_scales(wqd::I4Operands &op, uint32_t scales) {
  op.scale_bf16 = (scales & ~(uint32_t)WQD_I4_BY_ROW) == WQD_TYPE_BF16;
  op.by_row = scales & WQD_I4_BY_ROW;
}

wqd::I4Matrix i4_matrix(const void *W, const void *S, const void *Z) {
  return {static_cast<const uint8_t *>(W), static_cast<const uint16_t *>(S), static_cast<const uint8_t *>(Z)};
}

// 16-row tiles per workgroup in w8a16_gemm_m16_n64: 64 weight rows each.
constexpr uint32_t kN64Band = 4;

}  // namespace

extern "C" {

const char *wqd_last_error(void) { return g_last_error; }

int q2_0_select_tier(uint32_t m, uint32_t present_mask, int exact_m) {
  if (m == 0) return -1;
  for (int i = 0; i < WQD_Q2_0_TIER_COUNT; ++i)
    if (kTierWidths[i] >= m && ((present_mask >> i) & 1u) && (exact_m || !kTierExact[i])) return i;
  return -1;
}

int q2_0_exact_m_tiers_enabled(void) {
  static const int on = std::getenv("WQD_NO_EXACT_M_TIERS") == nullptr ? 1 : 0;
  return on;
}

uint32_t q2_0_tier_width(uint32_t m) {
  const int i = q2_0_select_tier(m, kTiersCompiled, q2_0_exact_m_tiers_enabled());
  return i < 0 ? 0u : kTierWidths[i];
}

size_t q2_0_packed_bytes(uint32_t N, uint32_t K) {
  if (K % WQD_Q2_0_GROUP != 0) return 0;
  return static_cast<size_t>(N) * (K / WQD_Q2_0_GROUP) * WQD_Q2_0_BLOCK_BYTES;
}

uint32_t q2_0_batchm_chunks(uint32_t M, uint32_t K, uint32_t N, uint64_t *out3, uint32_t cap) {
  uint32_t count = 0;
  for (uint32_t r0 = 0; r0 < M; r0 += WQD_Q2_0_BATCHM_MAX_M, ++count) {
    uint32_t rows = (M - r0) < WQD_Q2_0_BATCHM_MAX_M ? (M - r0) : WQD_Q2_0_BATCHM_MAX_M;
    if (out3 && count < cap) {
      out3[3 * count + 0] = static_cast<uint64_t>(r0) * K * 2;
      out3[3 * count + 1] = static_cast<uint64_t>(r0) * N * 2;
      out3[3 * count + 2] = rows;
    }
  }
  return count;
}

int q2_0_gemv(const void *A, const void *B, void *C, uint32_t N, uint32_t K, uint32_t group,
              hipStream_t stream) {
  static const char fn[] = "q2_0_gemv";
  int rc = validate_q2_0(fn, A, B, C, N, K, group);
  if (rc) return rc;
  if ((rc = check_device(fn))) return rc;
  (void)hipGetLastError();
  return check_launch(fn, launch_q2_0(A, B, C, N, K, 1, stream));
}

int q2_0_gemv_batchm(const void *A, const void *B, void *C, uint32_t N, uint32_t K,
                     uint32_t group, uint32_t M, hipStream_t stream) {
  static const char fn[] = "q2_0_gemv_batchm";
  int rc = validate_q2_0(fn, A, B, C, N, K, group);
  if (rc) return rc;
  if (M == 0) return WQD_OK;  // no rows: nothing to launch
  if ((rc = check_device(fn))) return rc;
  (void)hipGetLastError();
  const char *a = static_cast<const char *>(A);
  char *c = static_cast<char *>(C);
  for (uint32_t r0 = 0; r0 < M; r0 += WQD_Q2_0_BATCHM_MAX_M) {
    uint32_t rows = (M - r0) < WQD_Q2_0_BATCHM_MAX_M ? (M - r0) : WQD_Q2_0_BATCHM_MAX_M;
    rc = check_launch(fn, launch_q2_0(a + static_cast<size_t>(r0) * K * 2, B,
                                           c + static_cast<size_t>(r0) * N * 2, N, K, rows, stream));
    if (rc) return rc;
  }
  return WQD_OK;
}

int w8a16_gemm_m16(const void *A, const void *W, const float *S, void *C, uint32_t M, uint32_t N,
                   uint32_t K, hipStream_t stream) {
  static const char fn[] = "w8a16_gemm_m16";
  int rc = validate_w8a16(fn, A, W, S, C, M, N, K);
  if (rc) return rc;
  if ((rc = check_device(fn))) return rc;
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_w8a16_m16(A, W, S, C, M, N, K, K, N, 0, stream));
}

int w8a16_gemm_m16_n64(const void *A, const void *W, const float *S, void *C, uint32_t M, uint32_t N,
                       uint32_t K, hipStream_t stream) {
  static const char fn[] = "w8a16_gemm_m16_n64";
  int rc = validate_w8a16(fn, A, W, S, C, M, N, K);
  if (rc) return rc;
  if ((rc = check_device(fn))) return rc;
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_w8a16_m16(A, W, S, C, M, N, K, K, N, kN64Band, stream));
}

int w8a16_gemm_m16_strided(const void *A, const void *W, const float *S, void *C, uint32_t M, uint32_t N,
                           uint32_t K, uint32_t a_row_stride, uint32_t c_row_stride, hipStream_t stream) {
  static const char fn[] = "w8a16_gemm_m16_strided";
  int rc = validate_w8a16(fn, A, W, S, C, M, N, K);
  if (rc) return rc;
  if ((rc = validate_pitches(fn, M, N, K, a_row_stride, c_row_stride))) return rc;
  if ((rc = check_device(fn))) return rc;
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_w8a16_m16(A, W, S, C, M, N, K, a_row_stride, c_row_stride, 0, stream));
}

int w8a16_gemv_batch16_strided(const void *A, const void *W, const float *S, void *C, uint32_t M, uint32_t N,
                               uint32_t K, uint32_t a_row_stride, uint32_t c_row_stride, hipStream_t stream) {
  static const char fn[] = "w8a16_gemv_batch16_strided";
  int rc = validate_w8a16(fn, A, W, S, C, M, N, K);
  if (rc) return rc;
  if ((rc = validate_pitches(fn, M, N, K, a_row_stride, c_row_stride))) return rc;
  const uint32_t rows = wqd::w8a16_gemv_rows_per_launch(K);
  if (rows == 0)
    return fail(WQD_EUNSUPPORTED, "%s: K=%u above 81920 (one activation row must fit in LDS)", fn, K);
  if ((rc = check_device(fn))) return rc;
  (void)hipGetLastError();
  const uint16_t *a = static_cast<const uint16_t *>(A);
  uint16_t *c = static_cast<uint16_t *>(C);
  for (uint32_t r0 = 0; r0 < M; r0 += rows) {
    const uint32_t m = (M - r0) < rows ? (M - r0) : rows;
    rc = check_launch(fn, wqd::launch_w8a16_gemv(a + static_cast<size_t>(r0) * a_row_stride, W, S,
                                                 c + static_cast<size_t>(r0) * c_row_stride, m, N, K,
                                                 a_row_stride, c_row_stride, stream));
    if (rc) return rc;
  }
  return WQD_OK;
}

int w8a16_gemv_batch16(const void *A, const void *W, const float *S, void *C, uint32_t M, uint32_t N, uint32_t K,
                       hipStream_t stream) {
  return w8a16_gemv_batch16_strided(A, W, S, C, M, N, K, K, N, stream);
}

int mx_quantize(const void *X, uint32_t x_type, void *Q, void *S, uint32_t format, uint32_t M, uint32_t K,
                uint32_t x_row_stride, hipStream_t stream) {
  static const char fn[] = "mx_quantize";
  int rc = validate_mx_rows(fn, X, "X", x_type, Q, S, format, M, K, x_row_stride);
  if (rc) return rc;
  if (M == 0) return WQD_OK;  // no rows: nothing to launch
  if ((rc = check_device(fn))) return rc;
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_mx_quantize(X, x_type, Q, S, format == WQD_MXFP4, M, K, x_row_stride, stream));
}

int mx_dequantize(const void *Q, const void *S, uint32_t format, void *Y, uint32_t y_type, uint32_t M, uint32_t K,
                  uint32_t y_row_stride, hipStream_t stream) {
  static const char fn[] = "mx_dequantize";
  int rc = validate_mx_rows(fn, Y, "Y", y_type, Q, S, format, M, K, y_row_stride);
  if (rc) return rc;
  if (M == 0) return WQD_OK;
  if ((rc = check_device(fn))) return rc;
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_mx_dequantize(Q, S, format == WQD_MXFP4, Y, y_type, M, K, y_row_stride, stream));
}

int add_rmsnorm_mx8(const void *X, const void *R, const void *G, void *H, void *Y, void *Q, void *S, uint32_t M,
                    uint32_t K, uint32_t x_row_stride, uint32_t r_row_stride, float eps, hipStream_t stream) {
  static const char fn[] = "add_rmsnorm_mx8";
  if (!G || (M && (!X || !Q || !S))) return fail(WQD_ENULL, "%s: X, G, Q and S must be non-NULL", fn);
  if (!R != !H) return fail(WQD_ENULL, "%s: R and H must both be given or both be NULL", fn);
  if (K == 0 || K % WQD_MX_BLOCK != 0) return fail(WQD_EINVAL, "%s: K=%u is not a positive multiple of 32", fn, K);
  if (K > WQD_MX_NORM_MAX_K) return fail(WQD_EUNSUPPORTED, "%s: K=%u above %u", fn, K, (unsigned)WQD_MX_NORM_MAX_K);
  if (M > WQD_MX_NORM_MAX_M) return fail(WQD_EUNSUPPORTED, "%s: M=%u rows are too many for one call", fn, M);
  if (x_row_stride < K || x_row_stride % 8u != 0 || (R && (r_row_stride < K || r_row_stride % 8u != 0)))
    return fail(WQD_EINVAL, "%s: row strides %u, %u must be at least K=%u and multiples of 8 (16-byte rows)", fn,
                x_row_stride, r_row_stride, K);
  if (M && H == X && x_row_stride != r_row_stride)
    return fail(WQD_EINVAL, "%s: H may be X only where their row strides are equal (%u, %u)", fn, x_row_stride,
                r_row_stride);
  if (!std::isfinite(eps) || eps < 0.0f) return fail(WQD_EINVAL, "%s: eps must be finite and not negative", fn);
  if (!aligned(X, 16) || !aligned(R, 16) || !aligned(G, 16) || !aligned(H, 16) || !aligned(Y, 16) || !aligned(Q, 16))
    return fail(WQD_EALIGN, "%s: X, R, G, H, Y and Q must be 16-byte aligned", fn);
  if (M == 0) return WQD_OK;
  if (int rc = check_device(fn)) return rc;
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_add_rmsnorm_mx8(X, R, G, H, Y, Q, S, M, K, x_row_stride, r_row_stride, eps, stream));
}

int w4a16_gemm(const void *A, const void *W, const void *WS, void *C, uint32_t M, uint32_t N, uint32_t K,
               uint32_t a_row_stride, uint32_t c_row_stride, hipStream_t stream) {
  return run_mx_product("w4a16_gemm", mx_operands(A, nullptr, W, WS, nullptr, nullptr, C, M, N, K, a_row_stride, c_row_stride),
                        wqd::MxFormat::kBf16, false, stream);
}

int w4a8_gemm(const void *A, const void *AS, const void *W, const void *WS, void *C, uint32_t M, uint32_t N, uint32_t K,
              uint32_t c_row_stride, hipStream_t stream) {
  return run_mx_product("w4a8_gemm", mx_operands(A, AS, W, WS, nullptr, nullptr, C, M, N, K, K, c_row_stride),
                        wqd::MxFormat::kFp8, false, stream);
}

int w4a4_gemm(const void *A, const void *AS, const void *W, const void *WS, void *C, uint32_t M, uint32_t N, uint32_t K,
              uint32_t c_row_stride, hipStream_t stream) {
  return run_mx_product("w4a4_gemm", mx_operands(A, AS, W, WS, nullptr, nullptr, C, M, N, K, K, c_row_stride),
                        wqd::MxFormat::kFp4, false, stream);
}

int w4a16_gated(const void *A, const void *WG, const void *WGS, const void *WU, const void *WUS, void *C, uint32_t M,
                uint32_t N, uint32_t K, uint32_t a_row_stride, uint32_t c_row_stride, hipStream_t stream) {
  return run_mx_product("w4a16_gated", mx_operands(A, nullptr, WG, WGS, WU, WUS, C, M, N, K, a_row_stride, c_row_stride),
                        wqd::MxFormat::kBf16, true, stream);
}

int w4a8_gated(const void *A, const void *AS, const void *WG, const void *WGS, const void *WU, const void *WUS, void *C,
               uint32_t M, uint32_t N, uint32_t K, uint32_t c_row_stride, hipStream_t stream) {
  return run_mx_product("w4a8_gated", mx_operands(A, AS, WG, WGS, WU, WUS, C, M, N, K, K, c_row_stride),
                        wqd::MxFormat::kFp8, true, stream);
}

int w4a4_gated(const void *A, const void *AS, const void *WG, const void *WGS, const void *WU, const void *WUS, void *C,
               uint32_t M, uint32_t N, uint32_t K, uint32_t c_row_stride, hipStream_t stream) {
  return run_mx_product("w4a4_gated", mx_operands(A, AS, WG, WGS, WU, WUS, C, M, N, K, K, c_row_stride),
                        wqd::MxFormat::kFp4, true, stream);
}

int i4_pack(const void *Q, const void *S, const void *Z, void *W, void *WS, void *WZ, uint32_t N, uint32_t K,
            uint32_t group, uint32_t count, hipStream_t stream) {
  static const char fn[] = "i4_pack";
  if (count && (!Q || !W)) return fail(WQD_ENULL, "%s: Q and W must be non-NULL", fn);
  if (count && !S != !WS) return fail(WQD_ENULL, "%s: S and WS must both be non-NULL or both be NULL", fn);
  if (count && !Z != !WZ) return fail(WQD_ENULL, "%s: Z and WZ must both be given or both be NULL", fn);
  if (N == 0) return fail(WQD_EINVAL, "%s: N must be >= 1", fn);
  if (K == 0 || K % 128u != 0) return fail(WQD_EINVAL, "%s: K=%u is not a positive multiple of 128", fn, K);
  if (group != 32u && group != 64u && group != 128u)
    return fail(WQD_EINVAL, "%s: group=%u is not 32, 64 or 128", fn, group);
  if (K > WQD_MX_MAX_K) return fail(WQD_EUNSUPPORTED, "%s: K=%u above %u", fn, K, (unsigned)WQD_MX_MAX_K);
  if (N > WQD_MX_MAX_ROWS) return fail(WQD_EUNSUPPORTED, "%s: N=%u above %u", fn, N, (unsigned)WQD_MX_MAX_ROWS);
  if (count > WQD_MOE_MAX_EXPERTS)
    return fail(WQD_EUNSUPPORTED, "%s: count=%u above %u", fn, count, (unsigned)WQD_MOE_MAX_EXPERTS);
  if (!aligned(Q, 4) || !aligned(S, 2)) return fail(WQD_EALIGN, "%s: Q must be 4-byte and S 2-byte aligned", fn);
  if (!aligned(W, 16) || !aligned(WS, 16) || !aligned(WZ, 16))
    return fail(WQD_EALIGN, "%s: W, WS and WZ must be 16-byte aligned", fn);
  if (count == 0) return WQD_OK;
  if (int rc = check_device(fn)) return rc;
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_i4_pack(Q, i4_matrix(static_cast<uint8_t *>(W), WS, WZ), S, Z, N, K, group, count, stream));
}

uint32_t i4_packed_rows(uint32_t N) { return N > WQD_MX_MAX_ROWS ? 0u : (N + 15u) / 16u * 16u; }

int i4a16_gemm(const void *A, const void *W, const void *WS, const void *WZ, void *C, uint32_t M, uint32_t N, uint32_t K,
               uint32_t group, uint32_t scale_type, uint32_t a_row_stride, uint32_t c_row_stride, hipStream_t stream) {
  wqd::I4Operands op = {};
  op.A = static_cast<const uint16_t *>(A);
  op.w = i4_matrix(W, WS, WZ);
  op.C = static_cast<uint16_t *>(C);
  op.M = M, op.N = N, op.K = K, op.lda = a_row_stride, op.ldc = c_row_stride, op.group = group;
  set_scales(op, scale_type);
  return run_i4_product("i4a16_gemm", op, scale_type, stream);
}

int i4a16_gated(const void *A, const void *WG, const void *WGS, const void *WGZ, const void *WU, const void *WUS,
                const void *WUZ, void *C, uint32_t M, uint32_t N, uint32_t K, uint32_t group, uint32_t scale_type,
                uint32_t a_row_stride, uint32_t c_row_stride, hipStream_t stream) {
  wqd::I4Operands op = {};
  op.A = static_cast<const uint16_t *>(A);
  op.w = i4_matrix(WG, WGS, WGZ);
  op.up = i4_matrix(WU, WUS, WUZ);
  op.C = static_cast<uint16_t *>(C);
  op.M = M, op.N = N, op.K = K, op.lda = a_row_stride, op.ldc = c_row_stride, op.group = group;
  set_scales(op, scale_type);
  op.gated = true;
  return run_i4_product("i4a16_gated", op, scale_type, stream);
}

int moe_route(const void *logits, uint32_t logits_type, const float *bias, int32_t *ids, float *weights, uint32_t T,
              uint32_t E, uint32_t top_k, uint32_t row_stride, uint32_t scoring, uint32_t groups, uint32_t top_groups,
              uint32_t group_top, int renormalize, float scale, hipStream_t stream) {
  static const char fn[] = "moe_route";
  if (T && (!logits || !ids || !weights)) return fail(WQD_ENULL, "%s: logits, ids and weights must be non-NULL", fn);
  if (int rc = validate_routes(fn, T, top_k, E)) return rc;
  if (logits_type != WQD_TYPE_BF16 && logits_type != WQD_TYPE_FP16 && logits_type != WQD_TYPE_FP32)
    return fail(WQD_EINVAL, "%s: type %u of the logits is not BF16, FP16 or FP32", fn, logits_type);
  if (scoring != WQD_MOE_SOFTMAX && scoring != WQD_MOE_SIGMOID)
    return fail(WQD_EINVAL, "%s: scoring %u is neither softmax nor sigmoid", fn, scoring);
  if (row_stride < E) return fail(WQD_EINVAL, "%s: row_stride=%u below E=%u", fn, row_stride, E);
  if (groups == 0 || groups > 64u || E % groups != 0)
    return fail(WQD_EINVAL, "%s: groups=%u is not from 1 to 64 or does not divide E=%u", fn, groups, E);
  if (top_groups == 0 || top_groups > groups || top_k > top_groups * (E / groups))
    return fail(WQD_EINVAL, "%s: top_groups=%u of %u groups do not hold top_k=%u experts", fn, top_groups, groups, top_k);
  if (group_top != 1u && group_top != 2u) return fail(WQD_EINVAL, "%s: group_top=%u is neither 1 nor 2", fn, group_top);
  if (!std::isfinite(scale)) return fail(WQD_EINVAL, "%s: scale must be finite", fn);
  const uintptr_t size = logits_type == WQD_TYPE_FP32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return fail(WQD_EALIGN, "%s: operands must be aligned to their elements", fn);
  if (T == 0) return WQD_OK;
  if (int rc = check_device(fn)) return rc;
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_moe_route({logits, bias, ids, weights, logits_type, T, E, top_k, row_stride,
                                                 scoring == WQD_MOE_SIGMOID ? 1u : 0u, groups, top_groups, group_top,
                                                 renormalize ? 1u : 0u, scale}, stream));
}

int moe_lists(const int32_t *ids, int32_t *order, int32_t *offsets, uint32_t T, uint32_t top_k, uint32_t E,
              hipStream_t stream) {
  static const char fn[] = "moe_lists";
  if (!offsets || (T && (!ids || !order))) return fail(WQD_ENULL, "%s: ids, order and offsets must be non-NULL", fn);
  if (int rc = validate_routes(fn, T, top_k, E)) return rc;
  if (!aligned(ids, 4) || !aligned(order, 4) || !aligned(offsets, 4))
    return fail(WQD_EALIGN, "%s: ids, order and offsets must be 4-byte aligned", fn);
  if (int rc = check_device(fn)) return rc;
  (void)hipGetLastError();
  return check_launch(fn, wqd::launch_moe_lists(ids, order, offsets, T * top_k, E, stream));
}

int i4a16_experts_gated(const void *A, const int32_t *ids, const int32_t *order, const int32_t *offsets, const void *WG,
                        const void *WGS, const void *WGZ, const void *WU, const void *WUS, const void *WUZ, void *H,
                        uint32_t T, uint32_t top_k, uint32_t E, uint32_t N, uint32_t K, uint32_t group,
                        uint32_t scale_type, uint32_t a_row_stride, hipStream_t stream) {
  wqd::I4Operands op = {};
  op.A = static_cast<const uint16_t *>(A);
  op.w = i4_matrix(WG, WGS, WGZ);
  op.up = i4_matrix(WU, WUS, WUZ);
  op.C = static_cast<uint16_t *>(H);
  op.ids = ids, op.order = order, op.offsets = offsets;
  op.N = N, op.K = K, op.lda = a_row_stride, op.ldc = N, op.group = group;
  set_scales(op, scale_type);
  op.T = T, op.top_k = top_k, op.E = E;
  op.gated = true;
  return run_i4_experts("i4a16_experts_gated", op, scale_type, stream);
}

int i4a16_experts_down(const void *H, const int32_t *ids, const float *weights, const int32_t *order,
                       const int32_t *offsets, const void *W, const void *WS, const void *WZ, float *Y, void *C,
                       uint32_t T, uint32_t top_k, uint32_t E, uint32_t N, uint32_t K, uint32_t group,
                       uint32_t scale_type, uint32_t c_row_stride, hipStream_t stream) {
  wqd::I4Operands op = {};
  op.A = static_cast<const uint16_t *>(H);
  op.w = i4_matrix(W, WS, WZ);
  op.C = static_cast<uint16_t *>(C);
  op.Y = Y;
  op.ids = ids, op.order = order, op.offsets = offsets, op.weights = weights;
  op.N = N, op.K = K, op.lda = K, op.ldc = c_row_stride, op.group = group;
  set_scales(op, scale_type);
  op.T = T, op.top_k = top_k, op.E = E;
  return run_i4_experts("i4a16_experts_down", op, scale_type, stream);
}

}  // extern "C"
