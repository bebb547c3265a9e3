"""Routed calls with lists at the sizes where launches and 32-bit offsets end, on the CPU: what the header allows passes
every check (and ends at the missing GPU), and what is beyond it is refused."""
import pytest
import torch

from test_i4_abi import CALLS, EXPERTS, EUNSUPPORTED, call, refused
from weight_quantized_decode_block_amd import wqd


@pytest.mark.skipif(torch.cuda.is_available(), reason="the operands are no memory")
@pytest.mark.parametrize("fn,sizes", [
    # rows of 4 GB and more, and more than 65535 chunks of 16 of them
    ("i4a16_experts_down", dict(T=131072, top_k=8, E=64, K=2048, N=64)), ("i4a16_experts_down", dict(T=1 << 20, top_k=16, E=16, K=128, N=1)),
    ("i4a16_experts_down", dict(T=16384, top_k=8, E=64, K=16384, N=5120)),
    ("i4a16_experts_gated", dict(T=1 << 20, top_k=1, E=4, K=2048, N=16)), ("i4a16_experts_gated", dict(T=1 << 24, top_k=1, E=1, K=128, N=16384)),
    # the most outputs
    ("i4a16_experts_gated", dict(T=1 << 20, top_k=16, E=32, K=128, N=1 << 14)), ("i4a16_experts_down", dict(T=1 << 19, top_k=32, E=32, K=128, N=1 << 14)),
    ("i4a16_experts_gated", dict(T=1 << 14, top_k=1, E=32, K=128, N=1 << 24)),
])
def test_what_the_header_allows(fn, sizes):
    more = {k: v for k, v in dict(lda=sizes["K"], ldc=sizes["N"]).items() if k in CALLS[fn]}
    assert call(fn, sizes | more) == wqd.WQD_ENODEV, wqd.last_error()


@pytest.mark.parametrize("fn", EXPERTS)
@pytest.mark.parametrize("T,top_k,N", [(1 << 20, 16, (1 << 14) + 1), (1 << 14, 1, (1 << 24)), (1 << 15, 2, (1 << 24) - 1)])
def test_more_outputs_than_there_may_be(fn, T, top_k, N):
    T += T * top_k * N == 1 << 38
    refused(fn, dict(T=T, top_k=top_k, N=N) | ({"ldc": N} if "ldc" in CALLS[fn] else {}), EUNSUPPORTED, "too many")


def test_without_lists_launches_are_the_limit():
    few = dict(order=None, offsets=None)
    refused("i4a16_experts_gated", few | dict(T=65536, top_k=1), EUNSUPPORTED, "too many")
    refused("i4a16_experts_down", few | dict(T=65536, top_k=1), EUNSUPPORTED, "too many")
    refused("i4a16_experts_gated", few | dict(T=(1 << 21) // 320 + 1, top_k=1, N=5120), EUNSUPPORTED, "too many")
