"""The binding's checks of the operands of the 4-bit integer products, the router and
the experts, on the CPU: refusals come before the library is called, and calls that
pass them reach it."""
import pytest
import torch

from test_mx_binding import BF, F16, F32, U8, library, z  # noqa: F401  (library: a fixture)
from weight_quantized_decode_block_amd import wqd

I32 = torch.int32
M, N, K, G = 4, 20, 256, 64
T, E, P = 3, 8, 2  # tokens, experts, slots
PAD = 32  # rows of a laid-out matrix


def weights(n=1, scales=F16):
    return z(n * PAD * K // 2), z(n * PAD * K // G, t=scales), z(n * PAD * K // G)


def operands():
    act = dict(A=z(M, K, t=BF), C=z(M, N, t=BF), M=M, N=N, K=K, group=G)
    routed = dict(ids=z(T, P, t=I32), T=T, top_k=P, E=E)
    lists = dict(order=z(T * P, t=I32), offsets=z(E + 1, t=I32))
    experts = routed | lists | dict(N=N, K=K, group=G)
    named = lambda w, *names: dict(zip(names, w))  # noqa: E731
    pair = lambda n=1: named(weights(n), "WG", "WGS", "WGZ") | named(weights(n), "WU", "WUS", "WUZ")  # noqa: E731
    return {
        "i4_pack": dict(Q=z(N, K // 2), S=z(N, K // G, t=F16), Z=z(N, K // G), N=N, K=K, group=G) | named(weights(), "W", "WS", "WZ"),
        "i4a16_gemm": act | named(weights(), "W", "WS", "WZ"),
        "i4a16_gated": act | pair(),
        "moe_route": dict(logits=z(T, E, t=F32), bias=z(E, t=F32), ids=z(T, P, t=I32), weights=z(T, P, t=F32), T=T, E=E, top_k=P),
        "moe_lists": routed | lists,
        "i4a16_experts_gated": experts | dict(A=z(T, K, t=BF), H=z(T * P, N, t=BF)) | pair(E),
        "i4a16_experts_down": experts | dict(H=z(T * P, K, t=BF), weights=z(T, P, t=F32), Y=z(T * P, N, t=F32), C=z(T, N, t=BF))
                              | named(weights(E), "W", "WS", "WZ"),
    }


CALLS = list(operands())


def run(name, a):
    getattr(wqd, name)(**a)


def tensors(name):
    return [(k, x) for k, x in operands()[name].items() if torch.is_tensor(x)]


@pytest.mark.parametrize("name", CALLS)
def test_types(library, name):  # noqa: F811
    """Operands pass in their own type and are refused in another of the same size, and of another size."""
    run(name, operands()[name])
    for k, x in tensors(name):
        if k in ("S", "WS", "WGS", "WUS", "logits"):
            continue
        same, other = {U8: (torch.bool, F32), BF: (F16, F32), I32: (F32, torch.int64), F32: (I32, BF)}[x.dtype]
        before = len(library.calls)
        with pytest.raises(ValueError, match=f"{k} must have {x.dtype.itemsize}-byte elements of type"):
            run(name, operands()[name] | {k: x.view(same)})
        with pytest.raises(ValueError, match="elements of type"):
            run(name, operands()[name] | {k: x.to(other)})
        assert len(library.calls) == before


def test_scales_tell_their_type(library):  # noqa: F811
    for name, at, scales in (("i4a16_gemm", 9, ("WS",)), ("i4a16_gated", 12, ("WGS", "WUS")), ("i4a16_experts_gated", 17, ("WGS", "WUS")),
                             ("i4a16_experts_down", 16, ("WS",))):
        own = operands()[name]
        for t, number in ((F16, wqd.TYPE_FP16), (BF, wqd.TYPE_BF16)):
            run(name, own | {k: own[k].to(t) for k in scales})
            assert library.calls[-1][1][at] == number
            run(name, own | {k: 4096 for k in scales} | dict(scale_type=number))
            assert library.calls[-1][1][at] == number
        run(name, own | {k: 4096 for k in scales})
        assert library.calls[-1][1][at] == wqd.TYPE_FP16
        before = len(library.calls)
        for bad in ({scales[0]: own[scales[0]].view(torch.int16)}, dict(scale_type=wqd.TYPE_BF16), {scales[-1]: own[scales[-1]].float()}):
            with pytest.raises(ValueError):
                run(name, own | bad)
        if len(scales) == 2:
            with pytest.raises(ValueError, match="scales must all be"):
                run(name, own | {scales[1]: own[scales[1]].to(BF)})
        assert len(library.calls) == before
    own = operands()["i4_pack"]
    run("i4_pack", own | dict(S=own["S"].to(BF), WS=own["WS"].to(BF)))
    with pytest.raises(ValueError, match="S and WS must have the same type"):
        run("i4_pack", own | dict(S=own["S"].to(BF)))


def test_logits_tell_their_type(library):  # noqa: F811
    own = operands()["moe_route"]
    for t, number in ((BF, wqd.TYPE_BF16), (F16, wqd.TYPE_FP16), (F32, wqd.TYPE_FP32)):
        run("moe_route", own | dict(logits=own["logits"].to(t)))
        assert library.calls[-1][1][1] == number
    with pytest.raises(ValueError, match="BF16, FP16 or FP32"):
        run("moe_route", own | dict(logits=own["logits"].double()))
    for scoring, number in (("softmax", 0), ("sigmoid", 1), (1, 1)):
        run("moe_route", own | dict(scoring=scoring))
        assert library.calls[-1][1][9] == number
    for scoring in ("relu", 2, None, ["softmax"]):
        with pytest.raises(ValueError, match="neither 'softmax' nor 'sigmoid'"):
            run("moe_route", own | dict(scoring=scoring))


@pytest.mark.parametrize("name", CALLS)
def test_memory_that_is_too_short(library, name):  # noqa: F811
    """An operand one element, or row, short of what the call reaches is refused."""
    for k, x in tensors(name):
        before = len(library.calls)
        with pytest.raises(ValueError, match=k):
            run(name, operands()[name] | {k: x[:-1].clone()})
        assert len(library.calls) == before


@pytest.mark.parametrize("name", CALLS)
def test_another_gpu_s_tensor(library, name, monkeypatch):  # noqa: F811
    monkeypatch.setattr(wqd, "_raw_device", lambda: 0)
    for k, x in tensors(name):
        with pytest.raises(ValueError, match="is not on the current GPU"):
            run(name, {n: 4096 if torch.is_tensor(v) and n != k else v for n, v in operands()[name].items()})
    assert not library.calls


@pytest.mark.parametrize("name", CALLS)
def test_rows_that_are_not_where_the_call_takes_them(library, name):  # noqa: F811
    """Rows of a wider buffer pass with their stride where the call has one, and are refused without it; a transposed
    matrix is refused."""
    pitch = {"A": "a_row_stride", "C": "c_row_stride", "logits": "row_stride"}
    own = operands()[name]
    for k, x in tensors(name):
        if x.dim() != 2:
            continue
        wide = torch.zeros(x.shape[0], x.shape[1] + 8, dtype=x.dtype)
        before = len(library.calls)
        for bad in (wide[:, :x.shape[1]], torch.zeros(x.shape[1], x.shape[0], dtype=x.dtype).t()):
            with pytest.raises(ValueError, match=k):
                run(name, own | {k: bad})
        assert len(library.calls) == before
        if k in pitch:
            for good in (wide, wide[:, :x.shape[1]]):
                run(name, own | {k: good, pitch[k]: wide.shape[1]})
            assert len(library.calls) == before + 2


@pytest.mark.parametrize("name", CALLS)
def test_sizes(library, name):  # noqa: F811
    own = operands()[name]
    for k, x in own.items():
        if isinstance(x, int):
            for bad in (-1, 1 << 32):
                with pytest.raises((ValueError, wqd.WqdError)):
                    run(name, own | {k: bad})
    if "group" in own:
        for bad in (0, 48, 256):
            with pytest.raises(wqd.WqdError, match="is not 32, 64 or 128"):
                run(name, own | dict(group=bad))
        for bad in (0, 64, 200):
            with pytest.raises(wqd.WqdError, match="is not a positive multiple of 128"):
                run(name, own | dict(K=bad))
    assert not library.calls


def test_optional_operands(library):  # noqa: F811
    """Zero points, a bias, lists and their scratch may be absent; addresses are taken as they are."""
    for name, absent in (("i4_pack", ("Z", "WZ")), ("i4a16_gemm", ("WZ",)), ("i4a16_gated", ("WGZ", "WUZ")), ("moe_route", ("bias",)),
                         ("i4a16_experts_gated", ("order", "offsets")), ("i4a16_experts_down", ("order", "offsets", "Y"))):
        run(name, operands()[name] | {k: None for k in absent})
    for name in CALLS:
        run(name, {k: 4096 if torch.is_tensor(x) else x for k, x in operands()[name].items()})
    assert len(library.calls) == 6 + len(CALLS)
