"""GPU tests of the microscaled operators against their definitions in 64 bits
(mx_reference), through the C ABI.

Quantisation and its inverse are exact.  Tolerances of the others:
  * products: fp32 sums of K exact products (4-bit times 4- or 8-bit or BF16
    significands fit 24 bits) are within K * 2^-24 * sum |a w| of the exact sum
    in any order; the store adds half a BF16 step, 2^-8 of the value.  Where
    every partial sum is exact in fp32 the outputs equal the rounded exact sums.
    (On MXFP8 the matrix instruction first cuts the products of 8 consecutive k
    to the grid of the largest, test_gpu_mx_precision.py; normal values under a
    scale per 32 stay within the bound above.)
  * gated: the two sums as above; |silu'| <= 1.1; silu itself within 2^-16 of the
    result (test_gpu_mx_gates.py holds it to 2^-19, far gates included); then the
    store.
  * norm: y is computed in 64 bits and rounded to fp32 once, 2^-24; check_norm's
    2^-18 leaves room for 32-bit sums (test_gpu_mx_paths.py holds it to the one
    rounding).
"""
import numpy as np
import pytest
import torch

import mx_reference as ref
from parity import CANARY, dev_u8, dev_u16, host_u16, requires_gpu
from weight_quantized_decode_block_amd import inputs as gen
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]

FORMATS = ["mxfp4", "mxfp8"]
ACTS = ["bf16", "mxfp8", "mxfp4"]
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FILL = 0xA5


def same(a, b):
    return np.array_equal(np.asarray(a), np.asarray(b), equal_nan=np.asarray(a).dtype.kind == "f")


# ------------------------------------------------------------ quantisation
def quantize_gpu(x: torch.Tensor, fmt, K, pad=0):
    """Codes and scales of the rows of a host tensor, placed in a wider buffer
    (padding of NaN) when pad > 0; the bytes behind the outputs stay as they were."""
    M = x.shape[0]
    wide = torch.full((M, K + pad), float("nan"), dtype=x.dtype)
    wide[:, :K] = x
    nq = M * K // 2 if fmt == "mxfp4" else M * K
    Q = torch.full((nq + 64,), FILL, dtype=torch.uint8, device="cuda")
    S = torch.full((M * K // 32 + 64,), FILL, dtype=torch.uint8, device="cuda")
    wqd.mx_quantize(wide.cuda(), Q, S, fmt, M, K, x_row_stride=K + pad)
    torch.cuda.synchronize()
    q, s = Q.cpu().numpy(), S.cpu().numpy()
    assert (q[nq:] == FILL).all() and (s[M * K // 32:] == FILL).all()
    return q[:nq].reshape(M, -1), s[: M * K // 32].reshape(M, -1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("M,K,pad", [(1, 32, 0), (3, 96, 8), (33, 160, 40), (257, 1056, 0), (1000, 5120, 0), (2500, 4256, 8)])
def test_quantize_exact(fmt, t, M, K, pad):
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-30, 14, (M, K // 32), generator=g).float())
         .repeat_interleave(32, 1)).clamp(-60000, 60000).to(TYPES[t])
    q, s = quantize_gpu(x, fmt, K, pad)
    rq, rs = ref.quantize(x.double().numpy(), fmt)
    assert same(s, rs) and same(q, rq)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_quantize_every_16_bit_pattern(fmt, t):
    """All 65536 patterns (subnormals, infinities, NaN, both zeros), neighbours
    together and shuffled, and each finite one as its block's only value."""
    p = np.arange(65536, dtype=np.uint16)
    shuffled = gen.rng(953, 1).permutation(p)
    alone = np.zeros((65536, 32), np.uint16)
    alone[p, p % 32] = p
    for bits in (p.reshape(-1, 64), shuffled.reshape(-1, 64), alone):
        x = torch.from_numpy(bits.view(np.int16).copy()).view(TYPES[t])
        q, s = quantize_gpu(x, fmt, bits.shape[1])
        rq, rs = ref.quantize(x.double().numpy(), fmt)
        assert same(s, rs) and same(q, rq)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_fp32_borders(fmt):
    """fp32 values at, just below and just above every rounding border, at
    scales from the smallest subnormal's to the largest."""
    grid = ref.GRID[fmt]
    mid = (grid[1:] + grid[:-1]) / 2
    around = np.concatenate([np.float32(mid), np.nextafter(np.float32(mid), np.float32(0)),
                             np.nextafter(np.float32(mid), np.float32(1e9)), np.float32(grid)])
    around = np.concatenate([around, -around])
    n = -(-len(around) // 31) * 31
    block = np.zeros((n // 31, 32), np.float32)
    block[:, 1:] = np.resize(around, n).reshape(-1, 31)
    block[:, 0] = grid[-1]  # keeps the block's scale
    rows = [block * np.float32(2.0 ** e) for e in (0, -100, -126, -140, 100, 119)]
    rows.append(np.float32([[3.4028235e38] + [1e38] * 31, [1e-45] * 32, [np.inf] + [1.0] * 31, [-np.inf] + [1.0] * 31]))
    x = np.concatenate(rows)
    q, s = quantize_gpu(torch.from_numpy(x), fmt, 32)
    rq, rs = ref.quantize(x.astype(np.float64), fmt)
    assert same(s, rs) and same(q, rq)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("t", list(TYPES))
def test_dequantize_every_code_and_scale(fmt, t):
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
    q = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    if fmt == "mxfp4":
        q = q[:, :128]
        q = np.concatenate([q, q ^ 0x80])
        s = np.concatenate([s, s])
    M, K = q.shape[0], 256
    Y = torch.full((M, K + 8), 7.0, dtype=TYPES[t], device="cuda")
    wqd.mx_dequantize(dev_u8(q), dev_u8(s), Y, fmt, M, K, y_row_stride=K + 8)
    torch.cuda.synchronize()
    v = ref.values(q, s, fmt)
    want = ref.bf16(v) if t == "bf16" else torch.from_numpy(v).to(torch.float32).to(TYPES[t]).double().numpy()
    assert same(Y[:, :K].double().cpu().numpy(), want)
    assert (Y[:, K:] == 7.0).all()


# -------------------------------------------------------------------- norm
def norm_gpu(X, R, G, M, K, eps, px=0, pr=0, alias=None, want_y=True):
    def rows(a, pad):
        b = np.full((M, K + pad), 0x7FC1, np.uint16)
        b[:, :K] = a
        return dev_u16(b)
    Xd, Rd = rows(X, px), rows(R, pr) if R is not None else None
    H = None
    if R is not None:
        H = {"R": Rd, "X": Xd}.get(alias)
        if H is None:
            H = torch.full((M, K + pr), CANARY, dtype=torch.int16, device="cuda")
    Y = torch.full((M * K + 64,), CANARY, dtype=torch.int16, device="cuda") if want_y else None
    Q = torch.full((M * K + 64,), FILL, dtype=torch.uint8, device="cuda")
    S = torch.full((M * K // 32 + 64,), FILL, dtype=torch.uint8, device="cuda")
    wqd.add_rmsnorm_mx8(Xd, Rd, dev_u16(G), H, Y, Q, S, M, K, eps, x_row_stride=K + px, r_row_stride=K + pr)
    torch.cuda.synchronize()
    q, s = Q.cpu().numpy(), S.cpu().numpy()
    assert (q[M * K:] == FILL).all() and (s[M * K // 32:] == FILL).all()
    y = host_u16(Y) if want_y else None
    assert y is None or (y[M * K:] == CANARY).all()
    h = host_u16(H).reshape(M, -1) if H is not None else None
    if h is not None and pr:
        assert (h[:, K:] == (CANARY if alias is None else 0x7FC1)).all()
    return (h[:, :K] if h is not None else None, y[:M * K].reshape(M, K) if want_y else None,
            q[:M * K].reshape(M, K), s[:M * K // 32].reshape(M, K // 32))


def check_norm(X, R, G, M, K, eps, got):
    h, y, q, s = got
    hv = gen.bf16_values(X)
    if R is not None:
        hv = hv + gen.bf16_values(R)  # fp32
        assert np.array_equal(h, gen.bf16_bits(hv))
        hv = gen.bf16_values(gen.bf16_bits(hv))
    hv = hv.astype(np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        want = hv / np.sqrt((hv * hv).mean(-1, keepdims=True) + eps) * gen.bf16_values(G).astype(np.float64)
    good = np.isfinite(want).all(-1)
    d = 2.0 ** -18
    if y is not None:
        yv = gen.bf16_values(y).astype(np.float64)
        assert (np.abs(yv - want)[good] <= (2.0 ** -8 * (1 + d) + d) * np.abs(want)[good] + 2.0 ** -133).all()
    want, q, s = want[good], q[good], s[good].astype(np.int64)
    amax = np.abs(want).reshape(len(want), -1, 32).max(-1)
    lo, hi = (np.where(amax > 0, np.maximum(np.frexp(amax * f)[1] - 1 - 8, -127), -127) + 127 for f in (1 - d, 1 + d))
    assert ((s >= lo) & (s <= hi)).all()
    v = want * np.repeat(np.ldexp(1.0, 127 - s), 32, -1)
    c = ref.code_values(q, "mxfp8")
    near = np.minimum(np.abs(v), 448.0)
    half = np.maximum(2.0 ** -10, np.ldexp(1.0, np.frexp(np.maximum(near, 2.0 ** -30))[1] - 1 - 4))
    assert (np.abs(c - np.sign(v) * near) <= half + 2 * d * near).all()
    assert not np.isnan(c).any()
    return good


@pytest.mark.parametrize("M,K,residual,px,pr,alias,want_y", [
    (1, 5120, True, 0, 0, None, False), (1, 32, True, 0, 0, "R", True), (3, 160, False, 0, 0, None, True),
    (257, 5120, True, 8, 16, None, True), (7, 8192, True, 0, 0, "X", True), (5, 8224, True, 8, 8, "X", False),
    (129, 1056, False, 24, 0, None, False), (4, 17408, True, 0, 64, "R", True), (2, 32768, True, 0, 0, None, True),
    (2, 16416, False, 8, 0, None, True),
])
def test_norm(M, K, residual, px, pr, alias, want_y):
    r = gen.rng(954, M, K)
    X = gen.bf16_bits(r.standard_normal((M, K)))
    R = gen.bf16_bits(8 * r.standard_normal((M, K))) if residual else None
    G = gen.bf16_bits(1 + 0.2 * r.standard_normal(K))
    assert check_norm(X, R, G, M, K, 1e-6, norm_gpu(X, R, G, M, K, 1e-6, px, pr, alias, want_y)).all()


def test_norm_special_rows():
    """A zero row, rows with an infinity or NaN (which touch no other row),
    tiny and huge rows, and a zero eps."""
    M, K = 7, 320
    r = gen.rng(955, 1)
    x = r.standard_normal((M, K))
    x[0] = 0
    x[1, 5], x[2, 300] = np.inf, np.nan
    x[3] *= 1e-30
    x[4] *= 1e15
    X, G = gen.bf16_bits(x), gen.bf16_bits(np.ones(K))
    h, y, q, s = norm_gpu(X, None, G, M, K, 1e-6)
    good = check_norm(X, None, G, M, K, 1e-6, (h, y, q, s))
    assert list(good) == [True, False, False, True, True, True, True]
    assert not q[0].any() and not s[0].any() and not y[0].any()
    # an infinity makes the mean infinite: x / inf = 0, and NaN where x is infinite; a NaN spreads to its row
    assert s[1, 0] == 255 and not s[1, 1:].any() and (s[2] == 255).all()
    h, y, q, s = norm_gpu(X[3:], None, G, 4, K, 0.0)
    assert check_norm(X[3:], None, G, 4, K, 0.0, (h, y, q, s)).sum() >= 3


# ---------------------------------------------------------------- products
def product_gpu(fmt, a, s, mats, N, K, lda_pad=0, ldc_pad=0, shift=0, extra=1, stream=None):
    """C bits [M, N]; checks that padding, rows past M and what lies before a
    shifted C keep their canary."""
    M = a.shape[0]
    ldc = N + ldc_pad
    C = torch.full((shift + (M + extra) * ldc,), CANARY, dtype=torch.int16, device="cuda")
    view = C[shift:]
    mats = [dev_u8(x) if isinstance(x, np.ndarray) else x for x in mats]
    kind = "gated" if len(mats) == 4 else "gemm"
    if fmt == "bf16":
        wide = np.full((M, K + lda_pad), 0x7FC1, np.uint16)
        wide[:, :K] = a
        getattr(wqd, "w4a16_" + kind)(dev_u16(wide), *mats, view, M, N, K, a_row_stride=K + lda_pad, c_row_stride=ldc, stream=stream)
    else:
        getattr(wqd, f"w4a{fmt[-1]}_{kind}")(dev_u8(a), dev_u8(s), *mats, view, M, N, K, c_row_stride=ldc, stream=stream)
    torch.cuda.synchronize()
    c = host_u16(C)
    assert (c[:shift] == CANARY).all()
    c = c[shift:].reshape(M + extra, ldc)
    assert (c[M:] == CANARY).all() and (c[:, N:] == CANARY).all()
    return c[:M, :N]


def sums(av, wv, exact=False):
    """(exact sums, sums of magnitudes) by fp64 products on the GPU."""
    A, W = torch.from_numpy(av).cuda(), torch.from_numpy(wv).cuda()
    return (A @ W.T).cpu().numpy(), None if exact else (A.abs() @ W.abs().T).cpu().numpy()


SHAPES = [(1, 16, 128), (1, 5120, 1024), (2, 17, 256), (15, 129, 384), (16, 64, 640), (17, 255, 1152), (33, 300, 512),
          (64, 48, 2048), (65, 130, 896), (77, 513, 5120), (128, 256, 1024), (129, 257, 1536), (200, 1000, 768),
          (256, 512, 1280), (300, 259, 2176), (513, 771, 640), (1030, 520, 1024)]


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_exact_sums(fmt, M, N, K):
    """Where every partial sum is exact in fp32, the outputs are the rounded
    exact sums: |a w| <= 8 * 6 * 2^-6 in steps of 2^-11 (a in steps of 1/4, w of
    1/2 * 2^-8), so 17408 of them stay below 2^24 steps."""
    a, s = ref.exact_activations(M + N, M, K, fmt)
    w, ws = ref.weights(K + N, N, K)
    c = product_gpu(fmt, a, s, (w, ws), N, K)
    want, _ = sums(ref.act_values(a, s, fmt), ref.values(w, ws, "mxfp4"), exact=True)
    assert np.array_equal(gen.bf16_values(c).astype(np.float64), ref.bf16(want))


# The tile sizes are chosen by M, N and the format (csrc/mx_tile.hip, Costs): with 256 compute units these
# outputs, those of NARROW below and of test_gpu_mx_paths.py meet every one of them, for products and gated
# pairs of each format (test_mx_paths.py checks that), with ragged last tiles; the K have 4, 5, 6, 7 and 9
# steps of 128, so the last group of four is full and partial, pairs whole and half.
MANY = [(33, 4164, 640), (65, 12493, 512), (65, 16714, 896), (67, 8321, 1152), (98, 16549, 768), (130, 16408, 640),
        (132, 13672, 512), (257, 13829, 896), (293, 16391, 640), (385, 12515, 1152), (397, 16447, 640),
        (482, 10850, 768), (528, 16458, 512), (645, 16512, 896), (781, 14341, 640)]


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M,N,K", MANY)
def test_many_outputs_exact_sums(fmt, M, N, K):
    a, s = ref.exact_activations(M + N, M, K, fmt)
    w, ws = ref.weights(K + N, N, K)
    want = ref.bf16(sums(ref.act_values(a, s, fmt), ref.values(w, ws, "mxfp4"), exact=True)[0])
    for pad, shift in ((N % 3, M % 2), (-N % 8, 0)):  # outputs at any alignment, and whole 16-byte pieces
        c = product_gpu(fmt, a, s, (w, ws), N, K, lda_pad=8, ldc_pad=pad, shift=shift)
        assert np.array_equal(gen.bf16_values(c).astype(np.float64), want)


def check_product(c, want, mag, K):
    e = K * 2.0 ** -24 * mag
    d = np.abs(gen.bf16_values(c).astype(np.float64) - want)
    assert (d <= 2.0 ** -8 * (np.abs(want) + e) + e).all(), float((d / (np.abs(want) + 1e-30)).max())


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M,N,K,lda_pad,ldc_pad,shift", [
    (1, 300, 5120, 8, 3, 0), (9, 77, 17408, 0, 0, 1), (40, 250, 2176, 64, 6, 2), (130, 300, 1152, 8, 5, 4),
    (300, 517, 2048, 0, 3, 3), (500, 256, 5120, 16, 0, 0)])
def test_product_random(fmt, M, N, K, lda_pad, ldc_pad, shift):
    """Random operands, strided rows (NaN in the padding), outputs at every alignment."""
    a, s = ref.activations(M, M, K, fmt)
    w, ws = ref.weights(N, N, K, spread=12)
    c = product_gpu(fmt, a, s, (w, ws), N, K, lda_pad, ldc_pad, shift)
    want, mag = sums(ref.act_values(a, s, fmt), ref.values(w, ws, "mxfp4"))
    check_product(c, want, mag, K)


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M,N,K,ldc_pad,shift", [(1, 1000, 1024, 0, 0), (5, 17, 384, 3, 1), (16, 128, 5120, 0, 0), (33, 130, 640, 2, 2),
                                                 (64, 64, 1024, 0, 0), (129, 257, 1280, 1, 0), (300, 384, 2048, 0, 0), (520, 129, 896, 7, 3)])
def test_gated(fmt, M, N, K, ldc_pad, shift):
    check_gated(fmt, M, N, K, ldc_pad, shift)


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M,N,K", MANY)
def test_gated_many_outputs(fmt, M, N, K):
    for ldc_pad in (N % 3, -N % 8):
        check_gated(fmt, M, N, K, ldc_pad, 0)


def check_gated(fmt, M, N, K, ldc_pad, shift):
    a, s = ref.activations(M + 1, M, K, fmt)
    g, gs = ref.weights(2 * N, N, K, spread=5)
    u, us = ref.weights(2 * N + 1, N, K, spread=5)
    c = product_gpu(fmt, a, s, (g, gs, u, us), N, K, 8, ldc_pad, shift)
    av = ref.act_values(a, s, fmt)
    gw, gm = sums(av, ref.values(g, gs, "mxfp4"))
    uw, um = sums(av, ref.values(u, us, "mxfp4"))
    want = ref.silu(gw) * uw
    eg, eu = K * 2.0 ** -24 * gm, K * 2.0 ** -24 * um
    e = 1.1 * eg * (np.abs(uw) + eu) + np.abs(ref.silu(gw)) * eu + 2.0 ** -16 * np.abs(want)
    d = np.abs(gen.bf16_values(c).astype(np.float64) - want)
    assert (d <= 2.0 ** -8 * (np.abs(want) + e) + e + 2.0 ** -133).all()


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M", [20, 300])
def test_bad_values_stay_in_their_rows(fmt, M):
    """A NaN activation (BF16) or a scale of 255 spoils its own row or column only."""
    N, K = 330, 1024
    a, s = ref.exact_activations(3, M, K, fmt)
    w, ws = ref.weights(4, N, K)
    clean = product_gpu(fmt, a, s, (w, ws), N, K)
    a, ws = a.copy(), ws.copy()
    if fmt == "bf16":
        a[M - 2, 517] = 0x7FC0
    else:
        s = s.copy()
        s[M - 2, 16] = 255
    ws[N - 3, 31] = 255
    c = product_gpu(fmt, a, s, (w, ws), N, K)
    v = gen.bf16_values(c)
    assert np.isnan(v[M - 2]).all() and np.isnan(v[:, N - 3]).all()
    keep = np.ones((M, N), bool)
    keep[M - 2], keep[:, N - 3] = False, False
    assert np.array_equal(c[keep], clean[keep])


@pytest.mark.parametrize("fmt", ACTS)
def test_extreme_scales(fmt):
    """Weight scales from 2^-127 up, activations that bring the sums back to
    ordinary size: subnormal weights and scales are not flushed."""
    M, N, K = 18, 40, 256
    r = gen.rng(956, 1)
    w = r.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
    ws = np.repeat(np.arange(N, dtype=np.uint8)[:, None], K // 32, 1)
    if fmt == "bf16":
        a, s = gen.bf16_bits(np.ldexp(r.integers(-8, 9, size=(M, K)), 110)), None
    else:
        a, s = ref.exact_activations(6, M, K, fmt)
        s = np.full_like(s, 127 + 110)
    c = product_gpu(fmt, a, s, (w, ws), N, K)
    want, mag = sums(ref.act_values(a, s, fmt), ref.values(w, ws, "mxfp4"))
    check_product(c, want, mag, K)


@pytest.mark.parametrize("M", [1, 48, 300])
def test_other_stream_and_repeated_calls(M):
    """On a stream of its own, and the same bits from call to call."""
    N, K = 700, 2048
    w, ws = ref.weights(8, N, K, spread=12)
    st = torch.cuda.Stream()
    for fmt in ACTS:
        a, s = ref.activations(9, M, K, fmt)
        first = product_gpu(fmt, a, s, (w, ws), N, K)
        with torch.cuda.stream(st):
            assert np.array_equal(product_gpu(fmt, a, s, (w, ws), N, K), first)
        st.synchronize()
        assert np.array_equal(product_gpu(fmt, a, s, (w, ws), N, K, stream=st), first)


# ------------------------------------------------------- a block of a decode step
class Block:
    """A feed-forward block: residual addition and norm, gate and up, down."""

    def __init__(self, M, D, F, down="bf16"):
        self.M, self.D, self.F, self.down = M, D, F, down
        self.host = [ref.weights(i + 20, n, k, spread=4) for i, (n, k) in enumerate(((F, D), (F, D), (D, F)))]
        self.w = [(dev_u8(q), dev_u8(s)) for q, s in self.host]
        self.g = gen.bf16_bits(1 + 0.1 * gen.rng(957, 1).standard_normal(D))
        self.G = dev_u16(self.g)
        i16 = lambda *n: torch.zeros(n, dtype=torch.int16, device="cuda")  # noqa: E731
        u8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.X, self.R, self.H = i16(M, D), i16(M, D), i16(M, D)
        self.Q, self.S, self.A, self.C = u8(M, D), u8(M, D // 32), i16(M, F), i16(M, D)
        self.AQ, self.AS = u8(M, F), u8(M, F // 32)

    def set(self, seed):
        r = gen.rng(958, seed)
        self.x = gen.bf16_bits(r.standard_normal((self.M, self.D)))
        self.r = gen.bf16_bits(4 * r.standard_normal((self.M, self.D)))
        self.X.copy_(dev_u16(self.x))
        self.R.copy_(dev_u16(self.r))

    def run(self):
        M, D, F = self.M, self.D, self.F
        (gq, gs), (uq, us), (dq, ds) = self.w
        wqd.add_rmsnorm_mx8(self.X, self.R, self.G, self.H, None, self.Q, self.S, M, D, 1e-6)
        wqd.w4a8_gated(self.Q, self.S, gq, gs, uq, us, self.A, M, F, D)
        if self.down == "bf16":
            wqd.w4a16_gemm(self.A, dq, ds, self.C, M, D, F)
        else:
            wqd.mx_quantize(self.A.view(torch.bfloat16), self.AQ, self.AS, "mxfp8", M, F)
            wqd.w4a8_gemm(self.AQ, self.AS, dq, ds, self.C, M, D, F)

    def outputs(self):
        torch.cuda.synchronize()
        return [host_u16(self.H), self.Q.cpu().numpy(), self.S.cpu().numpy(), host_u16(self.A), host_u16(self.C)]


@pytest.mark.parametrize("M,down", [(1, "bf16"), (9, "mxfp8"), (150, "mxfp8"), (300, "bf16")])
def test_feed_forward_block(M, down):
    """The operators one after another, each checked on what the one before it
    really gave."""
    b = Block(M, 640, 1152, down)
    b.set(1)
    b.run()
    h, q, s, act, c = b.outputs()
    assert check_norm(b.x, b.r, b.g, M, b.D, 1e-6, (h, None, q, s)).all()
    mats = [ref.values(*w, "mxfp4") for w in b.host]
    av = ref.values(q, s, "mxfp8")
    (gw, gm), (uw, um) = sums(av, mats[0]), sums(av, mats[1])
    want = ref.silu(gw) * uw
    e = b.D * 2.0 ** -24 * (1.1 * gm * (np.abs(uw) + 1) + np.abs(ref.silu(gw)) * um) + 2.0 ** -16 * np.abs(want)
    assert (np.abs(gen.bf16_values(act) - want) <= 2.0 ** -8 * (np.abs(want) + e) + e).all()
    av = gen.bf16_values(act).astype(np.float64)
    if down == "mxfp8":
        q, s = ref.quantize(av, "mxfp8")
        assert same(b.AQ.cpu().numpy(), q) and same(b.AS.cpu().numpy(), s)
        av = ref.values(q, s, "mxfp8")
    check_product(c, *sums(av, mats[2]), b.F)


@pytest.mark.parametrize("M", [1, 150])
def test_block_captured_and_replayed(M):
    """Two blocks captured into graphs, replayed in turn on new inputs with
    eager work of the same blocks in between: every replay gives the eager bits."""
    blocks = [Block(M, 640, 1152, d) for d in ("bf16", "mxfp8")]
    for b in blocks:
        b.set(0)
        b.run()
    torch.cuda.synchronize()
    graphs = []
    for b in blocks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run()
        graphs.append(g)
    for seed in range(1, 5):
        for b, g in zip(blocks, graphs):
            b.set(seed)
            b.run()
            eager = b.outputs()
            for t in (b.H, b.Q, b.S, b.A, b.C):
                t.zero_()
            g.replay()
            assert all(np.array_equal(x, y) for x, y in zip(b.outputs(), eager))


def test_binding_checks_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros(4, 32, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="fewer"):
        wqd.mx_quantize(x, q, s[:3].clone(), "mxfp4", 4, 64)
    with pytest.raises(ValueError, match="fewer"):
        wqd.mx_quantize(x, q, s, "mxfp8", 4, 64)
    with pytest.raises(ValueError, match="fewer"):
        wqd.mx_quantize(x, q, s, "mxfp4", 4, 64, x_row_stride=72)
    with pytest.raises(ValueError, match="2-byte"):
        wqd.w4a16_gemm(x.float(), q, s, x, 4, 4, 64)
    with pytest.raises(ValueError, match="1-byte"):
        wqd.mx_dequantize(q, s.half(), x, "mxfp4", 4, 64)
    with pytest.raises(ValueError, match="contiguous"):
        wqd.mx_quantize(x.t(), q, s, "mxfp4", 4, 64)
    with pytest.raises(ValueError, match="current GPU"):
        wqd.mx_quantize(x.cpu(), q, s, "mxfp4", 4, 64)
    with pytest.raises(wqd.WqdError) as e:
        wqd.mx_quantize(x, q, s, "mxfp4", 4, 48)
    assert e.value.code == wqd.WQD_EINVAL
    wqd.mx_quantize(x, q, s, "mxfp4", 4, 64)


def test_binding_checks_views():
    """A view's rows have to lie as far apart as the call reads them."""
    wide = torch.randn(6, 96, device="cuda").bfloat16()
    x = wide[:, :64]
    q, s = torch.zeros(6, 32, dtype=torch.uint8, device="cuda"), torch.zeros(6, 2, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="rows are not 64"):
        wqd.mx_quantize(x, q, s, "mxfp4", 6, 64)
    with pytest.raises(ValueError, match="rows are not 32"):
        wqd.mx_quantize(x, torch.zeros(6, 48, dtype=torch.uint8, device="cuda")[:, :32], s, "mxfp4", 6, 64, x_row_stride=96)
    with pytest.raises(ValueError, match="rows are not 96"):
        wqd.mx_quantize(x[:1].expand(6, 64), q, s, "mxfp4", 6, 64, x_row_stride=96)
    wqd.mx_quantize(x, q, s, "mxfp4", 6, 64, x_row_stride=96)
    want = ref.quantize(x.double().cpu().numpy(), "mxfp4")
    assert same(q.cpu().numpy(), want[0]) and same(s.cpu().numpy(), want[1])
    wqd.mx_quantize(wide.view(2, 3, 96)[:, :, :64], q, s, "mxfp4", 6, 64, x_row_stride=96)
    assert same(q.cpu().numpy(), want[0])


def test_empty_tensors():
    x, q, s = (torch.zeros(0, n, dtype=t, device="cuda") for n, t in ((128, torch.bfloat16), (128, torch.uint8), (4, torch.uint8)))
    w, ws = torch.zeros(16, 64, dtype=torch.uint8, device="cuda"), torch.zeros(16, 4, dtype=torch.uint8, device="cuda")
    c, g = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda"), torch.zeros(128, dtype=torch.bfloat16, device="cuda")
    wqd.mx_quantize(x, q, s, "mxfp8", 0, 128)
    wqd.mx_dequantize(q, s, x, "mxfp8", 0, 128)
    wqd.add_rmsnorm_mx8(x, x, g, x, x, q, s, 0, 128, 1e-6)
    wqd.w4a16_gemm(x, w, ws, c, 0, 16, 128)
    wqd.w4a8_gated(q, s, w, ws, w, ws, c, 0, 16, 128)


# tiles of 64 x 32 outputs, four groups of waves: whole and part stages of four steps
NARROW = [(40, 7001, 1152), (47, 5130, 512), (61, 7170, 640), (100, 2100, 896), (128, 4096, 768)]


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M,N,K", NARROW)
def test_narrow_tiles_exact_sums(fmt, M, N, K):
    test_many_outputs_exact_sums(fmt, M, N, K)


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M,N,K", NARROW)
def test_gated_narrow_tiles(fmt, M, N, K):
    test_gated_many_outputs(fmt, M, N, K)
