"""The microscaled operators' paths that sizes choose, each at sizes that take it
(test_mx_paths.py checks on the CPU that every one is taken)."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from parity import dev_u8, requires_gpu
from test_gpu_mx import ACTS, FORMATS, TYPES, check_gated, check_norm, norm_gpu, product_gpu, quantize_gpu, same, sums
from test_gpu_mx_precision import cut_sums_gpu
from weight_quantized_decode_block_amd import inputs as gen
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]

# tiles of 64 x 64 of a gated pair from MXFP8 rows: ragged and whole outputs, whole and part groups of steps
GATED_64 = [(100, 5120, 640), (128, 8192, 896), (161, 4099, 1152), (65, 5123, 512)]
# every height of the few-row kernel, alone and with a row to spare
FEW = [(1, 33, 256), (2, 1, 128), (3, 47, 1152), (4, 80, 512), (5, 31, 640), (8, 65, 2176), (9, 48, 384), (16, 100, 1280),
       (17, 36, 128), (31, 129, 640), (32, 64, 1024)]
# K below the four steps that the tile kernel stages scales in, many rows: some of
# the few-row kernel, and below all tiles
SHORT = [(m, n, k) for k in (128, 256, 384) for m, n in ((33, 300), (130, 1029), (520, 77))]
# tiles that few shapes of test_gpu_mx.py take
LARGE = [(130, 16944, 640), (386, 16494, 640), (481, 10790, 640), (646, 13726, 640), (771, 15271, 640)]
SHORT_TILES = [(m, n, k) for i, (m, n) in enumerate([(33, 4164), (65, 5123), (100, 5121), (130, 16408), (257, 13829), (385, 12515),
                                                     (386, 16494), (481, 10790), (528, 16458), (781, 14341)])
               for k in ((128, 384), (256, 128, 384))[i % 2]]
# few outputs, many rows and the other way round
THIN = [(1, 1, 128), (700, 1, 640), (130, 3, 512), (1, 9999, 128), (2049, 17, 896)]


def exact_product(fmt, M, N, K, pads):
    a, s = ref.exact_activations(M + N, M, K, fmt)
    w, ws = ref.weights(K + N, N, K)
    want = ref.bf16(sums(ref.act_values(a, s, fmt), ref.values(w, ws, "mxfp4"), exact=True)[0])
    for pad, shift in pads:
        c = product_gpu(fmt, a, s, (w, ws), N, K, lda_pad=8, ldc_pad=pad, shift=shift)
        assert np.array_equal(gen.bf16_values(c).astype(np.float64), want)


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M,N,K", FEW + SHORT + SHORT_TILES + LARGE + THIN)
def test_products(fmt, M, N, K):
    exact_product(fmt, M, N, K, ((0, 0), (-N % 4, 0), (1, 1)))


def check_pair(fmt, M, N, K, ldc_pad, shift):
    """check_gated, whose operands these are; of MXFP8 rows against sums of the
    products as the instruction cuts them (test_gpu_mx_precision.py).  What is cut is
    up to 7 * 2^-12 of a group's largest product, which fp32's K * 2^-24 does not
    cover where K is small; with the cut sums all that is left is the fp32 additions
    of K / 8 groups and 8 partial sums, a step of the magnitudes each, and the
    activation, 2^-19."""
    if fmt != "mxfp8":
        return check_gated(fmt, M, N, K, ldc_pad, shift)
    a, s = ref.activations(M + 1, M, K, fmt)
    g, u = ref.weights(2 * N, N, K, spread=5), ref.weights(2 * N + 1, N, K, spread=5)
    c = gen.bf16_values(product_gpu(fmt, a, s, (*g, *u), N, K, 8, ldc_pad, shift)).astype(np.float64)
    (gate, gm), (up, um) = cut_sums_gpu(a, s, *g), cut_sums_gpu(a, s, *u)
    want = ref.silu(gate) * up
    eg, eu = ((K / 8 + 8) * 2.0 ** -23 * m for m in (gm, um))
    e = 1.1 * eg * (np.abs(up) + eu) + np.abs(ref.silu(gate)) * eu + 2.0 ** -19 * np.abs(want)
    assert (np.abs(c - want) <= 2.0 ** -8 * (np.abs(want) + e) + e + 2.0 ** -134).all()


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M,N,K", FEW + SHORT + SHORT_TILES + LARGE + THIN)
def test_gated_pairs(fmt, M, N, K):
    check_pair(fmt, M, N, K, 0, 0)
    check_pair(fmt, M, N, K, -N % 4 + 1, 1)


@pytest.mark.parametrize("M,N,K", GATED_64)
def test_gated_64(M, N, K):
    for pad in (N % 3, -N % 8):
        check_pair("mxfp8", M, N, K, pad, 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("M,K,pad", [(2500, 4256, 40), (2048, 4096, 0), (2049, 4128, 8), (8193, 1056, 0), (262147, 32, 8)])
def test_large_quantize_and_back(fmt, t, M, K, pad):
    """Two groups per thread (from 8.4 million values on), streamed where they have
    16 bits; last workgroups whole and in part; the second case is on the border."""
    g = torch.Generator().manual_seed(M)
    x = (torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-8, 9, (M, 1), generator=g).float())).to(TYPES[t])
    q, s = quantize_gpu(x, fmt, K, pad)
    rq, rs = ref.quantize(x.double().numpy(), fmt)
    assert same(s, rs) and same(q, rq)
    Y = torch.full((M, K + pad), 7.0, dtype=TYPES[t], device="cuda")
    wqd.mx_dequantize(dev_u8(q), dev_u8(s), Y, fmt, M, K, y_row_stride=K + pad)
    Y = Y.cpu()
    v = torch.from_numpy(ref.values(q, s, fmt)).to(torch.float32).to(TYPES[t])  # exact in fp32, then one rounding
    assert torch.equal(Y[:, :K], v) and bool((Y[:, K:] == 7.0).all())


def norm_codes(X, R, G, K, eps):
    """The norm in 64 bits, rounded to fp32 once: (fp32 rows, 64-bit rows)."""
    h = gen.bf16_values(X)
    if R is not None:
        h = gen.bf16_values(gen.bf16_bits(h + gen.bf16_values(R)))
    h = h.astype(np.float64)
    y = h / np.sqrt((h * h).sum(-1, keepdims=True) / K + eps) * gen.bf16_values(G).astype(np.float64)
    with np.errstate(over="ignore"):
        return y.astype(np.float32), y


def check_rounded_once(X, R, G, K, eps, got):
    """Codes, scales and BF16 rows are those of y rounded to fp32 once.  64-bit
    sums of K squares, in either order, and the few steps after them are at most
    K + 10 roundings of 2^-53 off, less than 2^-36 (K <= 2^15).  Rounding keeps
    order, so every code lies between those of y (1 - 2^-36) and y (1 + 2^-36),
    each rounded to fp32 first; nearly all are both's."""
    _, y, q, s = got
    _, want = norm_codes(X, R, G, K, eps)
    sides = []
    for f in (1 - 2.0 ** -36, 1 + 2.0 ** -36):
        with np.errstate(over="ignore"):
            v = (want * f).astype(np.float32).astype(np.float64)
        sides.append((ref.quantize(v, "mxfp8"), gen.bf16_bits(v)))
    ((q0, s0), y0), ((q1, s1), y1) = sides
    low = np.repeat(s == s0, 32, -1) & (q == q0)
    high = np.repeat(s == s1, 32, -1) & (q == q1)
    assert (low | high).all() and ((s == s0) | (s == s1)).all()
    assert (low & high).mean() > 0.999
    if y is not None:
        assert ((y == y0) | (y == y1)).all() and ((y == y0) & (y == y1)).mean() > 0.999


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("M,K", [(1023, 160), (1024, 32), (1024, 5120), (1030, 160), (1030, 8192), (1025, 8224), (5, 5120), (3, 17408)])
def test_norm_rounds_once(M, K, residual):
    """Either side of 1024 rows and of 8192 and 16384 values, where the groups per
    thread change."""
    r = gen.rng(981, M, K)
    X = gen.bf16_bits(r.standard_normal((M, K)))
    R = gen.bf16_bits(8 * r.standard_normal((M, K))) if residual else None
    G = gen.bf16_bits(1 + 0.2 * r.standard_normal(K))
    got = norm_gpu(X, R, G, M, K, 1e-6, 8, 16 if residual else 0)
    assert check_norm(X, R, G, M, K, 1e-6, got).all()
    check_rounded_once(X, R, G, K, 1e-6, got)


@pytest.mark.parametrize("M", [4, 1028])
def test_norm_of_far_values(M):
    """Rows whose squares leave fp32 at either end: around 1e25, 1e-25, 1e38, and
    one of subnormals beside a single large value."""
    K = 320
    r = gen.rng(982, M)
    x = r.standard_normal((M, K)) * np.array([1e25, 1e-25, 1e37, 1e-38])[np.arange(M) % 4, None]
    x[3::4, 7] = 1e30
    X, G = gen.bf16_bits(x), gen.bf16_bits(1 + 0.2 * r.standard_normal(K))
    for eps in (0.0, 1e-6):
        got = norm_gpu(X, None, G, M, K, eps)
        check_rounded_once(X, None, G, K, eps, got)


@pytest.mark.parametrize("M,N", [(2, 16), (64, 6000)])
@pytest.mark.parametrize("fmt", ACTS)
def test_weights_beyond_bf16(fmt, M, N):
    """Scale bytes 253 and 254 over every code, activations of 2^-100: quantised
    ones give the finite products, BF16 ones take weights of 2^128 and more as
    infinities."""
    K = 512
    w, ws = np.zeros((N, K // 2), np.uint8), np.full((N, K // 32), 127, np.uint8)
    w[:, 16] = np.arange(N) % 8  # k 32
    ws[:, 1] = np.where(np.arange(N) % 16 < 8, 253, 254)
    if fmt == "bf16":
        a, s = np.zeros((M, K)), None
        a[:, 32] = 2.0 ** -100
        a = gen.bf16_bits(a)
    else:
        a = np.zeros((M, K if fmt == "mxfp8" else K // 2), np.uint8)
        a[:, 32 if fmt == "mxfp8" else 16] = 0x38 if fmt == "mxfp8" else 2
        s = np.full((M, K // 32), 27, np.uint8)
    c = gen.bf16_values(product_gpu(fmt, a, s, (w, ws), N, K)).astype(np.float64)
    v = ref.values(w, ws, "mxfp4")[:, 32]
    want = np.where(v >= 2.0 ** 128, np.inf, v * 2.0 ** -100) if fmt == "bf16" else v * 2.0 ** -100
    assert np.array_equal(c, np.resize(want, (M, N)))
