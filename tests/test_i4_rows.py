"""Scales and zero points row by row or in tiles, on the CPU: a call tells the library which of the two its tensors'
shapes say, and shapes that say neither, or both, are refused before the library is called."""
import pytest
import torch

from test_i4_abi import EALIGN, EINVAL, ENULL, PRODUCTS, P, refused
from test_i4_binding import BF, E, F16, G, K, M, N, PAD, T, U8, library, operands, run, z  # noqa: F401  (library: a fixture)
from weight_quantized_decode_block_amd import wqd

AT = {"i4a16_gemm": 9, "i4a16_gated": 12, "i4a16_experts_gated": 17, "i4a16_experts_down": 16}  # scale_type's place
GROUPS = {"i4a16_gemm": ("WS", "WZ"), "i4a16_gated": ("WGS", "WGZ", "WUS", "WUZ"), "i4a16_experts_gated": ("WGS", "WGZ", "WUS", "WUZ"),
          "i4a16_experts_down": ("WS", "WZ")}


def count(name):
    return E if "experts" in name else 1


def rows(name, n=N, t=F16):
    """Every scale and zero point of a call, row by row."""
    e = count(name)
    return {k: z(e, n, K // G, t=t if k[-1] == "S" else U8) for k in GROUPS[name]}


def tiles(name, n=PAD, t=F16):
    return {k: z(count(name), n // 16, K // 128, 16, 128 // G, t=t if k[-1] == "S" else U8) for k in GROUPS[name]}


@pytest.mark.parametrize("n", [N, 32])  # with 32 rows both layouts are as many bytes
@pytest.mark.parametrize("name", list(AT))
def test_the_shape_tells_the_layout(library, name, n):  # noqa: F811
    own = operands()[name] | {k: x for k, x in dict(N=n, C=z(max(M, T), n, t=BF), H=z(T * 2, n, t=BF), Y=z(T * 2, n, t=torch.float32)).items()
                              if k in operands()[name] and not (k == "H" and name.endswith("down"))}
    if n == PAD and name.endswith("down"):
        own["H"] = operands()[name]["H"]
    for t, number in ((F16, wqd.TYPE_FP16), (BF, wqd.TYPE_BF16)):
        by_row, in_tiles = rows(name, n, t), tiles(name, t=t)
        for given in ({}, dict(scale_type=number), dict(scale_type=number | wqd.I4_BY_ROW)):
            run(name, own | by_row | given)
            assert library.calls[-1][1][AT[name]] == number | wqd.I4_BY_ROW == number | 0x100
        flat = {k: x.flatten(0, 1) for k, x in by_row.items()}  # the experts' rows one after another
        run(name, own | flat)
        assert library.calls[-1][1][AT[name]] == number | wqd.I4_BY_ROW
        for same in (in_tiles, {k: x.flatten() for k, x in in_tiles.items()}, {k: x.flatten(1) for k, x in in_tiles.items()}):
            for given in ({}, dict(scale_type=number)):
                run(name, own | same | given)
                assert library.calls[-1][1][AT[name]] == number
        before = len(library.calls)
        with pytest.raises(ValueError, match="by row"):
            run(name, own | in_tiles | dict(scale_type=number | wqd.I4_BY_ROW))
        for k in by_row:  # one of them unlike the others
            for a, b in ((by_row, in_tiles), (in_tiles, by_row)):
                with pytest.raises(ValueError, match="all lie row by row or all in tiles"):
                    run(name, own | a | {k: b[k]})
        assert len(library.calls) == before


@pytest.mark.parametrize("name", list(AT))
def test_shapes_that_are_neither(library, name):  # noqa: F811
    own, e, g = operands()[name], count(name), K // G
    for shape in ((e, g, N), (e, g, PAD), (e, PAD // 16, g, 16), (e, N, K // 32), (e, N, 1), (e, N // 2, 2 * g), (e, PAD // 16, K // 128, 128 // G, 16)):
        for k in GROUPS[name]:
            with pytest.raises(ValueError, match=f"{k} of shape .* is neither row by row"):
                run(name, own | {k: z(*shape, t=own[k].dtype)})
    if e > 1:  # experts that are not N rows apart
        for shape in ((e, PAD, g), (e * PAD, g), (e, N + 1, g)):
            with pytest.raises(ValueError, match="is neither row by row"):
                run(name, own | {k: z(*shape, t=own[k].dtype) for k in GROUPS[name]})
    assert not library.calls


@pytest.mark.parametrize("shape,E,N,K,group,by_row", [
    ((1, 64, 16), 1, 64, 2048, 128, True), ((64, 16), 1, 64, 2048, 128, True), ((80, 16), 1, 70, 2048, 128, True),
    ((1, 4, 16, 16), 1, 64, 2048, 128, None), ((4, 16, 16), 1, 64, 2048, 128, None),  # [row tile][group][row], [row tile][row][group]
    ((1, 4, 16, 16, 1), 1, 64, 2048, 128, False), ((16, 16, 1), 1, 16, 2048, 128, False), ((16, 64), 1, 64, 2048, 128, None),
    ((3, 64, 16), 3, 64, 2048, 128, True), ((192, 16), 3, 64, 2048, 128, True), ((3, 80, 16), 3, 70, 2048, 128, None), ((240, 16), 3, 70, 2048, 128, None),
    ((3, 1024), 3, 64, 2048, 128, False), ((4096,), 4, 64, 2048, 128, False), ((3, 70, 4), 3, 70, 128, 32, True), ((3, 5, 1, 16, 4), 3, 70, 128, 32, False),
])
def test_shapes(shape, E, N, K, group, by_row):
    assert wqd._i4_by_row(torch.Size(shape), E, N, K, group) is by_row


@pytest.mark.parametrize("name", list(AT))
def test_rows_that_are_too_few_or_elsewhere(library, name):  # noqa: F811
    own, by_row = operands()[name], rows(name)
    for k, x in by_row.items():
        short = z(1, N - 1, K // G, t=x.dtype) if count(name) == 1 else z(E - 1, N, K // G, t=x.dtype)
        apart = z(count(name), N, K // G + 4, t=x.dtype)[..., :K // G]
        for bad in (short, apart, x.view(count(name), K // G, N).transpose(1, 2)):
            with pytest.raises(ValueError, match=k):
                run(name, own | by_row | {k: bad})
    assert not library.calls


@pytest.mark.parametrize("name", list(AT))
def test_addresses_say_which(library, name):  # noqa: F811
    own = operands()[name]
    run(name, own | {k: 4096 for k in GROUPS[name]} | dict(scale_type=wqd.TYPE_BF16 | wqd.I4_BY_ROW))
    assert library.calls[-1][1][AT[name]] == wqd.TYPE_BF16 | wqd.I4_BY_ROW
    one = rows(name)
    run(name, own | {k: 4096 for k in GROUPS[name]} | {GROUPS[name][-1]: one[GROUPS[name][-1]]})
    assert library.calls[-1][1][AT[name]] == wqd.TYPE_FP16 | wqd.I4_BY_ROW


def test_pack_writes_tiles_only(library):  # noqa: F811
    """What it writes must not look like rows to the products."""
    own = operands()["i4_pack"]
    for k in ("WS", "WZ"):
        x = own[k]
        for bad in (x.view(PAD, K // G), x.view(1, PAD, K // G), x.view(K // G, PAD)):
            with pytest.raises(ValueError, match=f"{k} of shape .* is not in tiles"):
                run("i4_pack", own | {k: bad})
    assert not library.calls
    run("i4_pack", own | dict(WS=own["WS"].view(1, 2, K // 128, 16, 128 // G), WZ=own["WZ"].view(2, K // 128, 16, 128 // G)))
    assert len(library.calls) == 1


@pytest.mark.parametrize("fn", PRODUCTS)
def test_the_library_checks_rows(fn):
    """Row by row a row's scales of 128 k are one load, and so are its zero points: that much alignment, and no more."""
    row = wqd.I4_BY_ROW
    for group, scales, zeros in ((128, 2, 1), (64, 4, 2), (32, 8, 4)):
        refused(fn, dict(t=1 | row, group=group, WS=P + scales // 2), EALIGN, f"scales must be {scales}-byte aligned")
        if zeros > 1:
            refused(fn, dict(t=1 | row, group=group, WZ=P + zeros // 2), EALIGN, f"zero points must be {zeros}-byte aligned")
        # past its alignment the next check refuses
        refused(fn, dict(t=1 | row, group=group, WS=P + scales, WZ=P + zeros) | ({"C": P + 1} if "gemm" in fn or fn == "i4a16_gated" else {"ids": P + 1}),
                EALIGN, "C must" if "gemm" in fn or fn == "i4a16_gated" else "ids")
    for t in (2 | row, 3 | row, 0x200, 0x300, row << 1):
        refused(fn, dict(t=t), EINVAL, "scale type")


def test_pack_of_codes_alone(library):  # noqa: F811
    run("i4_pack", operands()["i4_pack"] | dict(S=None, Z=None, WS=None, WZ=None))
    assert [library.calls[-1][1][i] for i in (1, 2, 4, 5)] == [None] * 4


@pytest.mark.parametrize("change", [dict(S=None), dict(WS=None), dict(S=None, Z=None, WZ=None), dict(WS=None, Z=None, WZ=None)])
def test_pack_of_half_the_scales(change):
    refused("i4_pack", change, ENULL, "S and WS must both be non-NULL")
