"""Host-side tests of the microscaled operators: refusals (before any HIP
call), empty calls, and the binding's own checks.  Nothing is launched."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from weight_quantized_decode_block_amd import wqd

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced
P = FAKE


@pytest.fixture(scope="module")
def L():
    return wqd.lib()


QUANT = dict(X=P, type=0, Q=P, S=P, format=4, M=2, K=64, ld=64)


@pytest.mark.parametrize("change,code,frag", [
    (dict(X=None), wqd.WQD_ENULL, "non-NULL"), (dict(Q=None), wqd.WQD_ENULL, "non-NULL"),
    (dict(S=None), wqd.WQD_ENULL, "non-NULL"), (dict(type=3), wqd.WQD_EINVAL, "type"),
    (dict(format=5), wqd.WQD_EINVAL, "format"), (dict(K=0), wqd.WQD_EINVAL, "multiple of 32"),
    (dict(K=48), wqd.WQD_EINVAL, "multiple of 32"), (dict(ld=56), wqd.WQD_EINVAL, "row stride"),
    (dict(ld=68), wqd.WQD_EINVAL, "row stride"), (dict(type=2, ld=66), wqd.WQD_EINVAL, "row stride"),
    (dict(X=P + 8), wqd.WQD_EALIGN, "16-byte"), (dict(Q=P + 8), wqd.WQD_EALIGN, "Q must"),
    (dict(K=(1 << 24) + 32, ld=(1 << 24) + 32), wqd.WQD_EUNSUPPORTED, "above"),
    (dict(M=1 << 31, K=64), wqd.WQD_EUNSUPPORTED, "too many"),
])
@pytest.mark.parametrize("fn", ["mx_quantize", "mx_dequantize"])
def test_rows_refusals(L, fn, change, code, frag):
    a = QUANT | change
    if fn == "mx_quantize":
        rc = L.mx_quantize(a["X"], a["type"], a["Q"], a["S"], a["format"], a["M"], a["K"], a["ld"], None)
    else:
        rc = L.mx_dequantize(a["Q"], a["S"], a["format"], a["X"], a["type"], a["M"], a["K"], a["ld"], None)
    assert rc == code and frag in wqd.last_error() and fn in wqd.last_error()


NORM = dict(X=P, R=P, G=P, H=P, Y=P, Q=P, S=P, M=2, K=64, lx=64, lr=64, eps=1e-6)


@pytest.mark.parametrize("change,code,frag", [
    (dict(X=None), wqd.WQD_ENULL, "non-NULL"), (dict(G=None), wqd.WQD_ENULL, "non-NULL"),
    (dict(Q=None), wqd.WQD_ENULL, "non-NULL"), (dict(S=None), wqd.WQD_ENULL, "non-NULL"),
    (dict(R=None), wqd.WQD_ENULL, "both"), (dict(H=None), wqd.WQD_ENULL, "both"),
    (dict(K=0), wqd.WQD_EINVAL, "multiple of 32"), (dict(K=40), wqd.WQD_EINVAL, "multiple of 32"),
    (dict(K=32800, lx=32800, lr=32800), wqd.WQD_EUNSUPPORTED, "above"),
    (dict(M=(1 << 21) + 1), wqd.WQD_EUNSUPPORTED, "too many"),
    (dict(lx=56), wqd.WQD_EINVAL, "row strides"), (dict(lr=68), wqd.WQD_EINVAL, "row strides"),
    (dict(H=P, R=P + 64, lr=72), wqd.WQD_EINVAL, "H may be X"),
    (dict(eps=-1e-6), wqd.WQD_EINVAL, "eps"), (dict(eps=float("nan")), wqd.WQD_EINVAL, "eps"),
    (dict(eps=float("inf")), wqd.WQD_EINVAL, "eps"),
    (dict(Y=P + 2), wqd.WQD_EALIGN, "16-byte"), (dict(G=P + 2), wqd.WQD_EALIGN, "16-byte"),
])
def test_norm_refusals(L, change, code, frag):
    a = NORM | change
    assert L.add_rmsnorm_mx8(*a.values(), None) == code and frag in wqd.last_error()


PROD = dict(A=P, AS=P, W=P, WS=P, WU=P, WUS=P, C=P, M=3, N=17, K=256, lda=256, ldc=17)


def product(L, fn, a):
    bf16, gated = "a16" in fn, "gated" in fn
    args = [a["A"]] + ([] if bf16 else [a["AS"]]) + [a["W"], a["WS"]] + ([a["WU"], a["WUS"]] if gated else [])
    args += [a["C"], a["M"], a["N"], a["K"]] + ([a["lda"]] if bf16 else []) + [a["ldc"]]
    return getattr(L, fn)(*args, None)


PRODUCTS = ["w4a16_gemm", "w4a8_gemm", "w4a4_gemm", "w4a16_gated", "w4a8_gated", "w4a4_gated"]


@pytest.mark.parametrize("change,code,frag", [
    (dict(A=None), wqd.WQD_ENULL, "non-NULL"), (dict(W=None), wqd.WQD_ENULL, "non-NULL"),
    (dict(WS=None), wqd.WQD_ENULL, "non-NULL"), (dict(C=None), wqd.WQD_ENULL, "non-NULL"),
    (dict(N=0), wqd.WQD_EINVAL, "N must"), (dict(K=0), wqd.WQD_EINVAL, "multiple of 128"),
    (dict(K=192), wqd.WQD_EINVAL, "multiple of 128"), (dict(ldc=16), wqd.WQD_EINVAL, "cover"),
    (dict(K=(1 << 20) + 128, lda=(1 << 20) + 128), wqd.WQD_EUNSUPPORTED, "above"),
    (dict(M=(1 << 24) + 1), wqd.WQD_EUNSUPPORTED, "above"),
    (dict(N=(1 << 24) + 1, ldc=(1 << 24) + 1), wqd.WQD_EUNSUPPORTED, "above"),
    (dict(A=P + 8), wqd.WQD_EALIGN, "A must"), (dict(W=P + 8), wqd.WQD_EALIGN, "weights"),
    (dict(WS=P + 2), wqd.WQD_EALIGN, "scales"), (dict(C=P + 1), wqd.WQD_EALIGN, "C must"),
])
@pytest.mark.parametrize("fn", PRODUCTS)
def test_product_refusals(L, fn, change, code, frag):
    rc = product(L, fn, PROD | change)
    assert rc == code and frag in wqd.last_error() and fn in wqd.last_error()


@pytest.mark.parametrize("fn,change,code,frag", [
    ("w4a16_gemm", dict(lda=248), wqd.WQD_EINVAL, "cover"), ("w4a16_gated", dict(lda=260), wqd.WQD_EINVAL, "multiple of 8"),
    ("w4a16_gemm", dict(lda=(1 << 21) + 8), wqd.WQD_EUNSUPPORTED, "a_row_stride"),
    ("w4a8_gemm", dict(AS=None), wqd.WQD_ENULL, "non-NULL"), ("w4a4_gated", dict(AS=P + 1), wqd.WQD_EALIGN, "scales"),
    ("w4a8_gated", dict(WU=None), wqd.WQD_ENULL, "non-NULL"), ("w4a16_gated", dict(WUS=None), wqd.WQD_ENULL, "non-NULL"),
    ("w4a4_gated", dict(WU=P + 4), wqd.WQD_EALIGN, "weights"), ("w4a8_gated", dict(WUS=P + 2), wqd.WQD_EALIGN, "scales"),
])
def test_refusals_of_one_form(L, fn, change, code, frag):
    assert product(L, fn, PROD | change) == code and frag in wqd.last_error()


def test_no_rows_is_a_noop(L):
    for fn in PRODUCTS:
        assert product(L, fn, PROD | dict(M=0)) == wqd.WQD_OK
    assert L.mx_quantize(P, 0, P, P, 4, 0, 64, 64, None) == wqd.WQD_OK
    assert L.mx_dequantize(P, P, 8, P, 2, 0, 64, 64, None) == wqd.WQD_OK
    assert L.add_rmsnorm_mx8(P, P, P, P, P, P, P, 0, 64, 64, 64, 1e-6, None) == wqd.WQD_OK


def test_no_rows_need_no_rows_memory(L):
    """An empty tensor's address is NULL."""
    for fn in PRODUCTS:
        assert product(L, fn, PROD | dict(M=0, A=None, AS=None, C=None)) == wqd.WQD_OK
        assert product(L, fn, PROD | dict(M=0, W=None)) == wqd.WQD_ENULL
    assert L.mx_quantize(None, 0, None, None, 4, 0, 64, 64, None) == wqd.WQD_OK
    assert L.mx_dequantize(None, None, 8, None, 2, 0, 64, 64, None) == wqd.WQD_OK
    assert L.add_rmsnorm_mx8(None, None, P, None, None, None, None, 0, 64, 64, 72, 1e-6, None) == wqd.WQD_OK


def test_rows_of_a_view():
    t = torch.zeros(4, 6, 40)
    assert wqd._rows_apart(t[:, :, :32], 40) and not wqd._rows_apart(t[:, :, :32], 32)
    assert not wqd._rows_apart(t[:, :3, :32], 40)  # a gap between the leading dimension's rows
    assert wqd._rows_apart(t[:, 0, :32], 240) and wqd._rows_apart(t[:1, :3, :32], 40)
    assert wqd._rows_apart(t[0, :1, :32], 7) and wqd._rows_apart(t[0, 0], 7)  # one row


def test_valid_calls_reach_the_device_check(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for fn in PRODUCTS:
        assert product(L, fn, PROD) in (wqd.WQD_ENODEV, wqd.WQD_EHIP)
    assert L.add_rmsnorm_mx8(*(NORM | dict(R=None, H=None, Y=None, lr=0)).values(), None) in (wqd.WQD_ENODEV, wqd.WQD_EHIP)


def test_binding_refuses_host_tensors_and_unknown_formats():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current GPU"):
        wqd.mx_quantize(x, P, P, "mxfp4", 2, 64)
    with pytest.raises(ValueError, match="format"):
        wqd.mx_quantize(P, P, P, "fp4", 2, 64)
    with pytest.raises(ValueError, match="BF16, FP16 or FP32"):
        wqd.mx_quantize(x.double(), P, P, "mxfp4", 2, 64)
    with pytest.raises(ValueError, match="2\\^32"):
        wqd.w4a8_gemm(P, P, P, P, P, -1, 16, 128)
    with pytest.raises(ValueError, match="2\\^32"):
        wqd.mx_dequantize(P, P, P, "mxfp8", 1 << 32, 64)


# ------------------------------------------------ the reference of the GPU tests
def test_reference_codecs_against_torch():
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b)
    e4 = t.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(ref.code_values(b, "mxfp8"), nan=-1), np.nan_to_num(e4, nan=-1))
    e8 = t.view(torch.float8_e8m0fnu).double().numpy()
    assert np.array_equal(ref.scale_values(b)[:255], e8[:255]) and np.isnan(e8[255])
    x = np.concatenate((np.linspace(-470, 470, 20001), np.ldexp(1.0, np.arange(-12, 9)), np.ldexp(1.5, np.arange(-14, 8))))
    c = ref.nearest_codes(np.abs(x), ref.E4M3)
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).double().abs().numpy()
    keep = np.clip(x, -448, 448).astype(np.float32) == np.clip(x, -448, 448)  # torch goes through fp32
    assert np.array_equal(ref.E4M3[c][keep], want[keep])


def test_reference_bf16_against_torch():
    x = np.concatenate((np.random.default_rng(5).standard_normal(4096) * 10.0 ** np.arange(4096 / 128).repeat(128) / 1e18,
                        [0.0, 2.0 ** -133, 1.5 * 2.0 ** -133, 2.0 ** -134, 3.4e38, 3.39e38])).astype(np.float32)
    assert np.array_equal(ref.bf16(x), torch.from_numpy(x).bfloat16().double().numpy())


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_reference_quantiser_closed_forms(fmt):
    """Ties, saturation, a zero block, a subnormal block and a block with a NaN."""
    x = np.zeros((7, 32))
    top = ref.GRID[fmt][-1]
    x[0, :8] = [top, 0.25, -0.75, 1.25, 1.75, 2.5, 3.5, -5.0]
    # 6 * 1.3 = 7.8 < 8 keeps the scale and saturates; 448 * 1.3 = 582.4 >= 512 has the next
    # scale, where 291.2 lies between 288 and 320
    x[1, :2] = [top * 1.3, -top * 1.3]
    x[6, :2] = [top * 1.1, -top * 1.1]  # 6.6 and 492.8: saturate
    x[3, 0] = 2.0 ** -149
    x[4, 3] = np.nan
    x[5, :2] = [-2.0 ** -10 * top, -0.0]
    q, s = ref.quantize(x, fmt)
    assert list(s[:, 0]) == [127, 127 if fmt == "mxfp4" else 128, 0, 0, 255, 117, 127]
    v = ref.values(q, s, fmt)
    if fmt == "mxfp4":
        assert list(v[0, :8]) == [6, 0, -1, 1, 2, 2, 4, -4]
        assert q[5, 0] == 0x8F  # both signs kept: -6 and -0
    assert v[1, 0] == -v[1, 1] == (6 if fmt == "mxfp4" else 576) and v[6, 0] == top and v[6, 1] == -top
    assert not v[2].any() and np.isnan(v[4]).all()
    assert v[3, 0] == 0 and v[5, 0] == x[5, 0]
