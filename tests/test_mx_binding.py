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
    wqd._here("", 0)  # the types' table is filled
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


def pitched(name):
    """(operand, argument that gives its pitch) of the operands that have one."""
    if name.startswith("mx_quantize"):
        yield "X", "x_row_stride"
    elif name.startswith("mx_dequantize"):
        yield "Y", "y_row_stride"
    elif name.startswith("add"):
        yield from (("X", "x_row_stride"), ("R", "r_row_stride"), ("H", "r_row_stride"))
    else:
        yield "C", "c_row_stride"
        if "a16" in name:
            yield "A", "a_row_stride"


@pytest.mark.parametrize("name", CALLS)
def test_rows_of_wider_tensors(library, name):
    """A wider tensor passes with its pitch and is refused without it, whether
    whole or as a view of the rows; so is one of twice the width."""
    own = operands()[name]
    given = dict(pitched(name))
    for k, x in own.items():
        if not torch.is_tensor(x) or x.dim() < 2:
            continue
        width = x.shape[1]
        for extra in (8, width):
            wide = torch.zeros(x.shape[0], width + extra, dtype=x.dtype)
            before = len(library.calls)
            for t in (wide, wide[:, :width]):
                with pytest.raises(ValueError, match=f"{k}'s rows are not {width} elements apart"):
                    run(name, own | {k: t})
            assert len(library.calls) == before
            if k in given and not (name.startswith("add") and k != "X"):
                run(name, own | {k: wide, given[k]: width + extra})
                run(name, own | {k: wide[:, :width], given[k]: width + extra})
    if name.startswith("add"):
        wide = torch.zeros(M, K + 8, dtype=BF)
        run(name, own | dict(R=wide, H=wide, r_row_stride=K + 8))


@pytest.mark.parametrize("name", CALLS)
def test_other_shapes_of_the_same_memory(library, name):
    """Flat tensors and ones larger than the call reaches, rows in several
    dimensions or in parts, more rows than the call has, and one row of any width."""
    own = operands()[name]
    one = own | dict(M=1)
    for k, x in own.items():
        if not torch.is_tensor(x) or x.dim() < 2:
            continue
        rows, width = x.shape
        more = torch.zeros(2 * rows, width, dtype=x.dtype)
        run(name, own | {k: x.reshape(-1)})
        run(name, own | {k: more.reshape(-1)[: rows * width + 8]})
        run(name, own | {k: more})
        run(name, own | {k: more.reshape(2, rows, width)})
        run(name, own | {k: x.reshape(rows, 2, -1)})
        run(name, own | {k: more.reshape(1, -1)})
        run(name, own | {k: x.reshape(rows // 2, 2 * width)})  # just as large
        if not k.startswith("W"):
            run(name, one | {k: torch.zeros(rows, width + 8, dtype=x.dtype)})
    assert len(library.calls) > 0


@pytest.mark.parametrize("name", CALLS)
def test_part_blocks(library, name):
    """A K that is not whole blocks has the library's status, whatever the tensors."""
    for k in (0, 1, 48, K + 8):
        with pytest.raises(wqd.WqdError, match="multiple of 32") as e:
            run(name, operands()[name] | dict(K=k))
        assert e.value.code == wqd.WQD_EINVAL
    assert not library.calls


@pytest.mark.parametrize("name", CALLS)
def test_streams(library, monkeypatch, name):
    """A stream of another GPU would run the call there, on this one's memory."""
    class Stream:
        def __init__(self, gpu):
            self.device, self.cuda_stream = torch.device("cuda", gpu), 4096 + gpu
    monkeypatch.setattr(wqd, "_raw_device", lambda: 1)
    monkeypatch.setattr(wqd, "_raw_stream", lambda device: 512 + device)
    addresses = {k: 1 << 20 if torch.is_tensor(x) else x for k, x in operands()[name].items()}
    bare = type("Bare", (), {"cuda_stream": 99})()
    for stream, number in ((None, 513), (Stream(1), 4097), (77, 77), (bare, 99)):
        run(name, addresses | dict(stream=stream))
        assert library.calls[-1][1][-1] == number
    with pytest.raises(ValueError, match="stream is not the current GPU's"):
        run(name, addresses | dict(stream=Stream(0)))
    assert len(library.calls) == 4
