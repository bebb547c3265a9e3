"""Every kernel for 4-bit integer weights that the sizes of a call can choose is chosen
by some test: the choice of csrc/i4_tile.hip, repeated here from its tables of costs."""
import os
import re

import pytest

import test_gpu_i4 as base
import test_gpu_i4_paths as paths
import test_gpu_moe as moe
from weight_quantized_decode_block_amd import build as hip_build

SOURCE = open(os.path.join(hip_build.CSRC, "i4_tile.hip")).read()


def costs(name):
    body = re.search(rf"constexpr Cost {name}\[\] = \{{(.*?)\}};", SOURCE, re.S).group(1)
    return [tuple(int(x) for x in m) for m in re.findall(r"\{(\d+), (\d+), (\d+), (\d+), (\d+), (\d+)\}", body)]


def cost(c, tiles, steps):
    bm, bn, first, first_step, more, more_step = c
    return first + first_step * steps + max(-(-tiles // 256) - 1, 0) * (more + more_step * steps)


def cheapest(table, chunks, N, K, gated):
    """(index, cost) of the kernel for all outputs."""
    n = 2 * N if gated else N
    return min((cost(c, chunks(c[0]) * -(-n // c[1]), K // 128), i) for i, c in enumerate(table))[::-1]


def product(table, M, N, K, gated):
    """The kernels of a product: one, or that of whole rounds and that of the last outputs."""
    if M <= 16:
        return (0,)
    rows = lambda bm: -(-M // bm)  # noqa: E731
    way, whole = cheapest(table, rows, N, K, gated)
    bm, bn = table[way][:2]
    each = bn // 2 if gated else bn
    cols = rows(bm) * -(-N // each) // 256 * 256 // rows(bm)
    if way >= 2 and 0 < cols < -(-N // each):
        then, rest = cheapest(table, rows, N - cols * each, K, gated)
        if cost(table[way], rows(bm) * cols, K // 128) + rest < whole:
            return way, then
    return (way,)


@pytest.mark.parametrize("gated", [False, True])
def test_every_product_is_tested(gated):
    table = costs("kCosts")
    assert [c[0] for c in table] == [16, 32, 64, 128]
    taken = {i: [] for i in range(4)}
    for M, N, K in (paths.GATED if gated else paths.PRODUCT) + base.SIZES:
        ways = product(table, M, N, K, gated)
        assert len(ways) == 1
        taken[ways[0]].append((M, N, K))
    for i, sizes in taken.items():
        assert any(M % table[i][0] and N % table[i][1] for M, N, _ in sizes), (table[i], sizes)
        assert {1, 0} == {K // 128 % 2 for _, _, K in sizes} and (i == 0 or 128 in [K for _, _, K in sizes]), (table[i], sizes)
    assert {1, 2, 4, 7, 11, 16} <= {M for M, _, _ in base.SIZES}  # heights 4, 8 and 16 of the kernel for few rows


@pytest.mark.parametrize("gated", [False, True])
def test_every_kernel_for_the_last_outputs_is_tested(gated):
    sizes = paths.GATED_SPLIT if gated else paths.PRODUCT_SPLIT
    assert {product(costs("kCosts"), *x, gated) for x in sizes} == {(3, 0), (3, 1), (3, 2)}
    assert not gated or product(costs("kCosts"), *paths.GATED_LARGE[0], True) == (2, 1)


@pytest.mark.parametrize("gated", [False, True])
def test_every_product_of_lists_is_tested(gated):
    table = costs("kListCosts")
    taken = {i: [] for i in range(3)}
    for T, E, top_k, N, K in paths.LISTS + moe.EXPERTS:
        pairs = T * top_k
        busy = min(pairs, E)
        taken[cheapest(table, lambda bm: max(pairs // bm + busy // 4, busy), N, K, gated)[0]].append((T, E, top_k, N, K))
    for i, sizes in taken.items():
        assert len(sizes) >= 2 or (i == 2 and sizes), (table[i], sizes)


def test_every_split_without_lists_is_tested():
    """Four or eight waves on K of a pair; sixteen or eight on a token's sum."""
    assert {K < 4096 for _, _, _, _, K in moe.EXPERTS + [(0, 0, 0, 0, 131072)]} == {True, False}
    assert {-(-N // 16) * T <= 256 for T, _, _, N, _ in moe.EXPERTS} == {True, False}
