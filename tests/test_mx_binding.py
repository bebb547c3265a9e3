"""The binding's checks of tensor operands, on the CPU: refusals come before the
library is called, and calls that pass them reach it (a stand-in that records its
arguments)."""
import pytest
import torch

from weight_quantized_decode_block_amd import wqd

BF, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
M, N, K = 4, 16, 128


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return wqd.WQD_OK
        return call


@pytest.fixture
def library(monkeypatch):
    """Host tensors count as the current GPU's, and no library call is made."""
    wqd._here(0)  # the types' table is filled
    monkeypatch.setattr(wqd, "_raw_device", lambda: -1)
    monkeypatch.setattr(wqd, "_raw_stream", lambda device: None)
    fake = Library()
    monkeypatch.setattr(wqd, "_lib", fake)
    return fake


def z(*shape, t=U8):
    return torch.zeros(*shape, dtype=t)


def operands():
    """Tensors of every call, by name."""
    bits = {"mxfp4": 2, "mxfp8": 1}
    calls = {}
    for fmt in bits:
        q, s = z(M, K // bits[fmt]), z(M, K // 32)
        calls["mx_quantize " + fmt] = dict(X=z(M, K, t=BF), Q=q, S=s, fmt=fmt, M=M, K=K)
        calls["mx_dequantize " + fmt] = dict(Q=q, S=s, Y=z(M, K, t=F32), fmt=fmt, M=M, K=K)
    rows = lambda: z(M, K, t=BF)  # noqa: E731
    calls["add_rmsnorm_mx8"] = dict(X=rows(), R=rows(), G=z(K, t=BF), H=rows(), Y=rows(), Q=z(M, K), S=z(M, K // 32), M=M, K=K, eps=1e-6)
    for fmt, a in (("16", rows()), ("8", z(M, K)), ("4", z(M, K // 2))):
        act = dict(A=a) | ({} if fmt == "16" else dict(AS=z(M, K // 32)))
        c = dict(C=z(M, N, t=BF), M=M, N=N, K=K)
        w, ws = z(N, K // 2), z(N, K // 32)
        calls[f"w4a{fmt}_gemm"] = act | dict(W=w, WS=ws) | c
        calls[f"w4a{fmt}_gated"] = act | dict(WG=w, WGS=ws, WU=w, WUS=ws) | c
    return calls


def run(name, a):
    getattr(wqd, name.split()[0])(**a)


CALLS = list(operands())


def kinds(name):
    """(operand, its own type, types of the same size that it must not have)."""
    for k, x in operands()[name].items():
        if not torch.is_tensor(x) or (name.startswith("mx_") and k in "XY"):
            continue
        if x.dtype == BF:
            yield k, BF, (F16,)
        elif k.endswith("S"):
            yield k, torch.float8_e8m0fnu, (torch.bool, torch.float8_e4m3fn, torch.float8_e5m2)
        elif k.startswith("W") or name.startswith("w4a4") or name.endswith("mxfp4"):
            yield k, torch.float4_e2m1fn_x2, (torch.bool, torch.float8_e4m3fn, torch.float8_e8m0fnu)
        else:
            yield k, torch.float8_e4m3fn, (torch.bool, torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float4_e2m1fn_x2)


@pytest.mark.parametrize("name", CALLS)
def test_types(library, name):
    """An operand of its own type or of integers of its size passes; one of another
    type of the same size would be read as what it is not, and is refused."""
    run(name, operands()[name])
    for k, own, other in kinds(name):
        plain = (torch.int16, torch.uint16) if own is BF else (U8, torch.int8)
        for t in (own, *plain):
            run(name, operands()[name] | {k: operands()[name][k].view(t)})
        before = len(library.calls)
        for t in other:
            with pytest.raises(ValueError, match=f"{k} must have {own.itemsize}-byte elements of type .*not {str(t)[6:]}"):
                run(name, operands()[name] | {k: operands()[name][k].view(t)})
        with pytest.raises(ValueError, match="elements of type"):
            run(name, operands()[name] | {k: operands()[name][k].float() if own is BF else operands()[name][k].half()})
        assert len(library.calls) == before


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_values_tell_their_type(library, fmt):
    for t, number in ((BF, wqd.TYPE_BF16), (F16, wqd.TYPE_FP16), (F32, wqd.TYPE_FP32)):
        run("mx_quantize", operands()["mx_quantize " + fmt] | dict(X=z(M, K, t=t)))
        assert library.calls[-1][1][1] == number
        run("mx_dequantize", operands()["mx_dequantize " + fmt] | dict(Y=z(M, K, t=t)))
        assert library.calls[-1][1][4] == number
    for t in (torch.int16, torch.float64):
        with pytest.raises(ValueError, match="BF16, FP16 or FP32"):
            run("mx_quantize", operands()["mx_quantize " + fmt] | dict(X=z(M, K, t=t)))
