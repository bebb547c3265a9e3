"""Routed calls with lists at the sizes where launches and 32-bit offsets end, on the CPU: what the header allows passes
every check (and ends at the missing GPU), and what is beyond it is refused."""
import pytest
import torch

import test_gpu_i4_lists as gpu_lists
import test_gpu_i4_paths as gpu_paths
import test_gpu_i4_range as gpu_range
import test_gpu_moe as gpu_moe
import test_i4_paths as paths
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


# ---------------------------------------------------- the kernels that lists take
def fit(T, E, top_k, N, lda, gated, bm):
    """Chunks of bm rows that a call may have, and whether a launch of tiles of them holds it."""
    pairs, busy = T * top_k, min(T * top_k, E)
    chunks = (pairs + busy * (bm - 1)) // bm
    return chunks, (T if gated else pairs) * lda * 2 < 1 << 32 and chunks * -(-N // (128 if gated else 256)) <= 1 << 22


def launch(T, E, top_k, N, K, gated, lda=None):
    """(kernel, launches) of a call with lists: 0 the one for few rows, 1 and 2 tiles of 64 and 128 rows."""
    lda, pairs, busy = lda or K, T * top_k, min(T * top_k, E)
    most = min((1 << 21) // -(-N // 16), 65535)
    launches = -(-fit(T, E, top_k, N, lda, gated, 16)[0] // most)
    if not fit(T, E, top_k, N, lda, gated, 128)[1]:
        return 0, launches
    way = paths.cheapest(paths.costs("kListCosts"), lambda bm: max(pairs // bm + busy // 4, busy), N, K, gated)[0]
    if way == 0 and launches > 1 or way == 1 and not fit(T, E, top_k, N, lda, gated, 64)[1]:
        way = 2
    return way, launches if way == 0 else 1


def test_the_tests_take_the_kernels_that_they_name():
    for gated in (False, True):
        for sizes, ways in ((gpu_lists.ROUTED, (0, 1, 2)), (gpu_range.ROUTED, (0, 0, 1, 2))):
            assert [launch(*x, gated) for x in sizes] == [(w, 1) for w in ways]
        taken = {launch(*x, gated) for x in gpu_paths.LISTS + gpu_moe.EXPERTS}
        assert taken == {(0, 1), (1, 1), (2, 1)}  # what the costs say, always
        assert launch(200000, 8, 8, 24, 128, gated) == (2, 1)  # more chunks than a launch for few rows holds
    assert launch(131072, 64, 8, 64, 2048, False) == (0, 2) and launch(1 << 20, 300, 1, 17, 2048, False) == (0, 2)
    assert launch(1100000, 6, 1, 32, 256, True, lda=2048) == (0, 2)
    assert {launch(T, 16, 4, 384, 256, True)[0] for T in (600, 2000, 8000)} == {1, 2}
    assert {launch(T, 16, 4, 256, 384, False)[0] for T in (600, 2000, 8000)} == {0, 1, 2}
    product = {i: paths.product(paths.costs("kCosts"), *x, False) for i, x in enumerate(gpu_range.SIZES)}
    assert product == {0: (0,), 1: (0,), 2: (0,), 3: (1,), 4: (1,), 5: (2,), 6: (3,)}
