"""Host-side tests of the products with 4-bit integer weights and the routed
block: refusals (before any HIP call) and empty calls.  Nothing is launched."""
import pytest

from weight_quantized_decode_block_amd import wqd

P = 0x7F0000000000  # 16-byte aligned, never dereferenced
OK, EINVAL, ENULL, EALIGN, EUNSUPPORTED = wqd.WQD_OK, wqd.WQD_EINVAL, wqd.WQD_ENULL, wqd.WQD_EALIGN, wqd.WQD_EUNSUPPORTED

PACK = dict(Q=P, S=P, Z=P, W=P, WS=P, WZ=P, N=17, K=256, group=64, count=2)
GEMM = dict(A=P, W=P, WS=P, WZ=P, C=P, M=3, N=17, K=256, group=64, t=1, lda=256, ldc=17)
GATED = dict(A=P, W=P, WS=P, WZ=P, WU=P, WUS=P, WUZ=P, C=P, M=3, N=17, K=256, group=64, t=1, lda=256, ldc=17)
ROUTE = dict(logits=P, t=2, bias=P, ids=P, weights=P, T=5, E=64, top_k=4, ld=64, scoring=0, groups=8, top_groups=2, group_top=2, renorm=1, scale=1.0)
LISTS = dict(ids=P, order=P, offsets=P, T=5, top_k=4, E=64)
XGATED = dict(A=P, ids=P, order=P, offsets=P, W=P, WS=P, WZ=P, WU=P, WUS=P, WUZ=P, H=P, T=5, top_k=4, E=64, N=17, K=256, group=64, t=1, lda=256)
XDOWN = dict(H=P, ids=P, weights=P, order=P, offsets=P, W=P, WS=P, WZ=P, Y=P, C=P, T=5, top_k=4, E=64, N=17, K=256, group=64, t=1, ldc=17)
CALLS = {"i4_pack": PACK, "i4a16_gemm": GEMM, "i4a16_gated": GATED, "moe_route": ROUTE, "moe_lists": LISTS, "i4a16_experts_gated": XGATED,
         "i4a16_experts_down": XDOWN}
PRODUCTS = ["i4a16_gemm", "i4a16_gated", "i4a16_experts_gated", "i4a16_experts_down"]
EXPERTS = PRODUCTS[2:]


def call(fn, change=None):
    return getattr(wqd.lib(), fn)(*(CALLS[fn] | (change or {})).values(), None)


def refused(fn, change, code, frag):
    assert call(fn, change) == code and frag in wqd.last_error() and fn in wqd.last_error(), wqd.last_error()


@pytest.mark.parametrize("fn", PRODUCTS)
@pytest.mark.parametrize("change,code,frag", [
    (dict(W=None), ENULL, "non-NULL"), (dict(WS=None), ENULL, "non-NULL"), (dict(N=0, ldc=0), EINVAL, "N must"),
    (dict(K=0), EINVAL, "multiple of 128"), (dict(K=192), EINVAL, "multiple of 128"), (dict(group=16), EINVAL, "group"),
    (dict(group=256), EINVAL, "group"), (dict(t=2), EINVAL, "scale type"), (dict(t=3), EINVAL, "scale type"),
    (dict(K=(1 << 20) + 128, lda=(1 << 20) + 128), EUNSUPPORTED, "above"), (dict(N=(1 << 24) + 1, ldc=(1 << 24) + 1), EUNSUPPORTED, "above"),
    (dict(W=P + 8), EALIGN, "weights"), (dict(WS=P + 8), EALIGN, "scales"), (dict(WZ=P + 8), EALIGN, "zero points"),
])
def test_product_refusals(fn, change, code, frag):
    refused(fn, {k: v for k, v in change.items() if k in CALLS[fn]}, code, frag)


@pytest.mark.parametrize("fn,change,code,frag", [
    ("i4a16_gemm", dict(A=None), ENULL, "A and C"), ("i4a16_gated", dict(C=None), ENULL, "A and C"),
    ("i4a16_gemm", dict(A=P + 8), EALIGN, "16-byte"), ("i4a16_gemm", dict(C=P + 1), EALIGN, "C must"),
    ("i4a16_gemm", dict(lda=248), EINVAL, "cover"), ("i4a16_gemm", dict(ldc=16), EINVAL, "cover"), ("i4a16_gated", dict(lda=260), EINVAL, "multiple of 8"),
    ("i4a16_gemm", dict(lda=(1 << 21) + 8), EUNSUPPORTED, "a_row_stride"), ("i4a16_gemm", dict(M=(1 << 24) + 1), EUNSUPPORTED, "above"),
    ("i4a16_gated", dict(WU=None), ENULL, "non-NULL"), ("i4a16_gated", dict(WUS=None), ENULL, "non-NULL"), ("i4a16_gated", dict(WUZ=None), ENULL, "both"),
    ("i4a16_gated", dict(WZ=None), ENULL, "both"), ("i4a16_gated", dict(WU=P + 4), EALIGN, "weights"), ("i4a16_gated", dict(WUS=P + 2), EALIGN, "scales"),
    ("i4a16_gated", dict(WUZ=P + 1), EALIGN, "zero points"), ("i4a16_experts_gated", dict(WUZ=None), ENULL, "both"),
    ("i4_pack", dict(Q=None), ENULL, "non-NULL"), ("i4_pack", dict(W=None), ENULL, "non-NULL"), ("i4_pack", dict(N=0), EINVAL, "N must"),
    ("i4_pack", dict(K=64), EINVAL, "multiple of 128"), ("i4_pack", dict(count=1025), EUNSUPPORTED, "count"), ("i4_pack", dict(Q=P + 2), EALIGN, "Q must"),
    ("i4_pack", dict(W=P + 8), EALIGN, "16-byte"), ("i4_pack", dict(WS=P + 8), EALIGN, "16-byte"), ("i4_pack", dict(WZ=P + 8), EALIGN, "16-byte"),
    ("i4_pack", dict(S=None), ENULL, "non-NULL"), ("i4_pack", dict(WS=None), ENULL, "non-NULL"), ("i4_pack", dict(Z=None), ENULL, "both"),
    ("i4_pack", dict(WZ=None), ENULL, "both"), ("i4_pack", dict(group=96), EINVAL, "group"), ("i4_pack", dict(S=P + 1), EALIGN, "2-byte"), ("i4_pack", dict(K=(1 << 20) + 128), EUNSUPPORTED, "above"), ("i4_pack", dict(N=(1 << 24) + 1), EUNSUPPORTED, "above"),
])
def test_refusals_of_one_form(fn, change, code, frag):
    refused(fn, change, code, frag)


@pytest.mark.parametrize("fn", ["moe_route", "moe_lists", *EXPERTS])
@pytest.mark.parametrize("change,code,frag", [
    (dict(E=0), EINVAL, "E="), (dict(E=1025), EINVAL, "E="), (dict(top_k=0), EINVAL, "top_k"), (dict(top_k=65), EINVAL, "top_k"),
    (dict(top_k=33), EINVAL, "top_k"), (dict(E=3), EINVAL, "top_k"), (dict(T=(1 << 22) + 1), EUNSUPPORTED, "too many"), (dict(ids=None), ENULL, "non-NULL"),
    (dict(ids=P + 2), EALIGN, "aligned"),
])
def test_routed_sizes(fn, change, code, frag):
    refused(fn, change, code, frag)


@pytest.mark.parametrize("change,code,frag", [
    (dict(logits=None), ENULL, "non-NULL"), (dict(weights=None), ENULL, "non-NULL"), (dict(t=3), EINVAL, "type"), (dict(scoring=2), EINVAL, "scoring"),
    (dict(ld=63), EINVAL, "row_stride"), (dict(groups=0), EINVAL, "groups"), (dict(groups=7), EINVAL, "groups"), (dict(groups=128, E=128, ld=128), EINVAL, "groups"),
    (dict(top_groups=0), EINVAL, "top_groups"), (dict(top_groups=9), EINVAL, "top_groups"), (dict(top_groups=1, top_k=9), EINVAL, "top_groups"),
    (dict(group_top=0), EINVAL, "group_top"), (dict(group_top=3), EINVAL, "group_top"), (dict(scale=float("nan")), EINVAL, "scale"),
    (dict(scale=float("inf")), EINVAL, "scale"), (dict(logits=P + 2), EALIGN, "aligned"), (dict(bias=P + 1), EALIGN, "aligned"), (dict(weights=P + 2), EALIGN, "aligned"),
])
def test_route_refusals(change, code, frag):
    refused("moe_route", change, code, frag)


@pytest.mark.parametrize("fn,change,code,frag", [
    ("moe_lists", dict(order=None), ENULL, "non-NULL"), ("moe_lists", dict(offsets=None), ENULL, "non-NULL"), ("moe_lists", dict(order=P + 1), EALIGN, "aligned"),
    ("i4a16_experts_gated", dict(order=None), ENULL, "both"), ("i4a16_experts_down", dict(offsets=None), ENULL, "both"),
    ("i4a16_experts_gated", dict(H=None), ENULL, "non-NULL"), ("i4a16_experts_gated", dict(A=None), ENULL, "non-NULL"),
    ("i4a16_experts_gated", dict(lda=128), EINVAL, "cover"), ("i4a16_experts_down", dict(ldc=16), EINVAL, "cover"),
    ("i4a16_experts_down", dict(weights=None), ENULL, "non-NULL"), ("i4a16_experts_down", dict(Y=None), ENULL, "Y must"),
    ("i4a16_experts_down", dict(Y=P + 8), EALIGN, "Y must"), ("i4a16_experts_down", dict(H=P + 8), EALIGN, "16-byte"),
    ("i4a16_experts_down", dict(offsets=P + 2), EALIGN, "aligned"), ("i4a16_experts_down", dict(weights=P + 2), EALIGN, "aligned"),
    ("i4a16_experts_gated", dict(T=1 << 20, top_k=16, N=1 << 20), EUNSUPPORTED, "too many"),
])
def test_experts_refusals(fn, change, code, frag):
    refused(fn, change, code, frag)


def test_nothing_to_do():
    """No rows, no tokens, no matrices: nothing is launched, and what holds them may be NULL; the rest is checked."""
    assert call("i4_pack", dict(count=0, Q=None, S=None, Z=None, W=None, WS=None, WZ=None)) == OK
    for fn in PRODUCTS[:2]:
        assert call(fn, dict(M=0, A=None, C=None)) == OK
        assert call(fn, dict(M=0, W=None)) == ENULL
    assert call("moe_route", dict(T=0, logits=None, ids=None, weights=None)) == OK
    assert call("moe_route", dict(T=0, groups=7)) == EINVAL
    assert call("i4a16_experts_gated", dict(T=0, A=None, ids=None, order=None, offsets=None, H=None)) == OK
    assert call("i4a16_experts_down", dict(T=0, H=None, ids=None, weights=None, Y=None, C=None)) == OK
    assert call("i4a16_experts_down", dict(T=0, group=48)) == EINVAL


def test_packed_rows():
    assert [wqd.i4_packed_rows(n) for n in (1, 16, 17, 1 << 24)] == [16, 16, 32, 1 << 24]
