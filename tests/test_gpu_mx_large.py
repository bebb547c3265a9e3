"""The microscaled operators where offsets pass 32 bits: more than 2^32 bytes and
more than 2^32 elements from an operand's start to its end, and products that take
several launches.  Operands are mostly pitch or zero codes, so that little of the
memory is touched; what is there is checked as in test_gpu_mx.py."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from parity import dev_u16, dev_u8, host_u16, requires_gpu
from test_gpu_mx import ACTS, FORMATS, check_norm, same
from weight_quantized_decode_block_amd import inputs as gen
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]

PITCH = 2 ** 21 + 8  # elements; 2050 rows of it reach past 2^32 of them
ROWS = 2050


def pitched(rows, pitch, t, width, fill):
    """A buffer of rows `pitch` apart, of which the first `width` columns hold `fill`."""
    b = torch.empty(rows * pitch, dtype=t, device="cuda").view(rows, pitch)
    b[:, :width] = fill
    return b


@pytest.mark.parametrize("fmt,t", [("mxfp4", torch.bfloat16), ("mxfp8", torch.float32), ("mxfp8", torch.float16)])
def test_quantize_and_back_far_rows(fmt, t):
    K = 96
    x = torch.randn(ROWS, K, generator=torch.Generator().manual_seed(5)).to(t)
    X = pitched(ROWS, PITCH, t, K + 8, float("nan"))
    X[:, :K] = x.cuda()
    Q = torch.zeros(ROWS, K // 2 if fmt == "mxfp4" else K, dtype=torch.uint8, device="cuda")
    S = torch.zeros(ROWS, K // 32, dtype=torch.uint8, device="cuda")
    wqd.mx_quantize(X, Q, S, fmt, ROWS, K, x_row_stride=PITCH)
    q, s = ref.quantize(x.double().numpy(), fmt)
    assert same(Q.cpu().numpy(), q) and same(S.cpu().numpy(), s)
    X[:, :K + 8] = 7.0
    wqd.mx_dequantize(Q, S, X, fmt, ROWS, K, y_row_stride=PITCH)
    assert same(X[:, :K].double().cpu().numpy(), ref.values(q, s, fmt)) and bool((X[:, K:K + 8] == 7.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_and_back_many_values(fmt):
    """2^32 values and more in one call, in the launch of two groups per thread."""
    K, M = 4128, 1040500
    X = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(6))
    Q = torch.empty(M, K // 2 if fmt == "mxfp4" else K, dtype=torch.uint8, device="cuda")
    S = torch.empty(M, K // 32, dtype=torch.uint8, device="cuda")
    wqd.mx_quantize(X, Q, S, fmt, M, K)
    at = torch.from_numpy(np.r_[0:20, 520000:520020, 1040380:1040500]).cuda()
    q, s = ref.quantize(X[at].double().cpu().numpy(), fmt)
    assert same(Q[at].cpu().numpy(), q) and same(S[at].cpu().numpy(), s)
    X.zero_()
    wqd.mx_dequantize(Q, S, X, fmt, M, K)
    assert same(X[at].double().cpu().numpy(), ref.values(q, s, fmt))


@pytest.mark.parametrize("residual", [True, False])
def test_norm_far_rows(residual):
    K = 160
    r = gen.rng(971, 1)
    x, h, g = (gen.bf16_bits(f * r.standard_normal(n)) for f, n in ((1, (ROWS, K)), (4, (ROWS, K)), (1, K)))
    X = pitched(ROWS, PITCH, torch.int16, K, dev_u16(x))
    R = pitched(ROWS, PITCH + 8, torch.int16, K, dev_u16(h)) if residual else None
    Q = torch.zeros(ROWS, K, dtype=torch.uint8, device="cuda")
    S = torch.zeros(ROWS, K // 32, dtype=torch.uint8, device="cuda")
    Y = torch.zeros(ROWS, K, dtype=torch.int16, device="cuda")
    wqd.add_rmsnorm_mx8(X, R, dev_u16(g), R, Y, Q, S, ROWS, K, 1e-6, x_row_stride=PITCH, r_row_stride=PITCH + 8)
    got = (host_u16(R[:, :K].contiguous()) if residual else None, host_u16(Y), Q.cpu().numpy(), S.cpu().numpy())
    assert check_norm(x, h if residual else None, g, ROWS, K, 1e-6, got).all()


@pytest.mark.parametrize("N,K", [(70, 128), (600, 512)])
def test_product_far_rows(N, K):
    """BF16 rows of the largest pitch and outputs of a larger one: the few-row
    kernel, and tiles of 64 x 64."""
    M, lda, ldc = 2100, 2 ** 21, 2 ** 21 + 3
    a, _ = ref.exact_activations(1, M, K, "bf16")
    w, ws = ref.weights(2, N, K)
    A = pitched(M, lda, torch.int16, K + 8, 0x7FC1)
    A[:, :K] = dev_u16(a)
    C = pitched(M, ldc, torch.int16, N + 3, 77)
    wqd.w4a16_gemm(A, dev_u8(w), dev_u8(ws), C, M, N, K, a_row_stride=lda, c_row_stride=ldc)
    c = host_u16(C[:, :N + 3].contiguous())
    want = ref.bf16(ref.act_values(a, None, "bf16") @ ref.values(w, ws, "mxfp4").T)
    assert np.array_equal(gen.bf16_values(c[:, :N]).astype(np.float64), want) and (c[:, N:] == 77).all()


def ends(rows, K, per_byte, seed):
    """Code rows of zeros but for the first and last 256 values, on the host and the GPU."""
    r = gen.rng(972, seed)
    n = 512 // per_byte
    host = r.integers(0, 256, (rows, n), np.uint8)
    if per_byte == 1:
        host &= 0xBF  # below 2 in magnitude
    dev = torch.zeros(rows, K // per_byte, dtype=torch.uint8, device="cuda")
    dev[:, :n // 2], dev[:, -n // 2:] = dev_u8(host[:, :n // 2]), dev_u8(host[:, n // 2:])
    return host, dev


@pytest.mark.parametrize("fmt,M,N", [("mxfp8", 4200, 20), ("mxfp8", 8300, 20), ("mxfp4", 8300, 20), ("bf16", 40, 9000), ("bf16", 2, 9000),
                                     ("mxfp8", 40, 9000), ("mxfp4", 2, 9000)])
def test_product_long_rows(fmt, M, N):
    """K of 2^20: activation codes or weights of more than 2^32 bytes, in both
    kernels.  The sums are exact: 512 products, multiples of 1/32 up to 36."""
    K = 2 ** 20
    one = lambda n: torch.full((n, K // 32), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    w, W = ends(N, K, 2, N)
    C = torch.zeros(M, N, dtype=torch.int16, device="cuda")
    if fmt == "bf16":
        bits, _ = ref.exact_activations(M, M, 512, "bf16")
        A = torch.zeros(M, K, dtype=torch.int16, device="cuda")
        A[:, :256], A[:, -256:] = dev_u16(bits[:, :256]), dev_u16(bits[:, 256:])
        av = ref.act_values(bits, None, "bf16")
        wqd.w4a16_gemm(A, W, one(N), C, M, N, K)
    else:
        a, A = ends(M, K, 1 if fmt == "mxfp8" else 2, M)
        av = ref.code_values(a, fmt)
        if fmt == "mxfp8":  # steps of 1/16, which the instruction's grid keeps
            av = np.trunc(av * 16) / 16
            codes = ref.nearest_codes(np.abs(av), ref.E4M3) | np.where(av < 0, 128, 0)
            A[:, :256], A[:, -256:] = dev_u8(codes[:, :256]), dev_u8(codes[:, 256:])
        call = wqd.w4a8_gemm if fmt == "mxfp8" else wqd.w4a4_gemm
        call(A, one(M), W, one(N), C, M, N, K)
    want = ref.bf16(av @ ref.code_values(w, "mxfp4").T)
    assert np.array_equal(gen.bf16_values(host_u16(C)).astype(np.float64), want)


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_products_of_several_launches(fmt, gated):
    """2^24 outputs a row: the few-row kernel takes 256 rows a launch (gated 128),
    and the outputs are 10 GB."""
    M, N, K = 300, 2 ** 24, 128
    a, s = ref.exact_activations(7, M, K, fmt)
    g = torch.Generator("cuda").manual_seed(8)
    mats = []
    for _ in range(2 if gated else 1):
        mats += [torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g),
                 torch.randint(119, 122, (N, K // 32), dtype=torch.uint8, device="cuda", generator=g)]
    C = torch.empty(M, N, dtype=torch.int16, device="cuda")
    kind = "gated" if gated else "gemm"
    if fmt == "bf16":
        getattr(wqd, "w4a16_" + kind)(dev_u16(a), *mats, C, M, N, K)
    else:
        getattr(wqd, f"w4a{fmt[-1]}_{kind}")(dev_u8(a), dev_u8(s), *mats, C, M, N, K)
    cols = np.r_[0:40, gen.rng(973, 1).integers(0, N, 200), N - 40:N]
    at = torch.from_numpy(cols).cuda()
    c = gen.bf16_values(host_u16(C[:, at])).astype(np.float64)
    av = ref.act_values(a, s, fmt)
    sums = [av @ ref.values(q[at].cpu().numpy(), e[at].cpu().numpy(), "mxfp4").T for q, e in zip(mats[::2], mats[1::2])]
    if not gated:
        assert np.array_equal(c, ref.bf16(sums[0]))
    else:
        want = ref.silu(sums[0]) * sums[1]
        e = 2.0 ** -19 * np.abs(want)  # the activation's (test_gpu_mx_gates.py); the sums are exact
        assert (np.abs(c - want) <= 2.0 ** -8 * (np.abs(want) + e) + e + 2.0 ** -134).all()
