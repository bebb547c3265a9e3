"""Every kernel that the sizes of a call can choose is chosen by some test: the
choice of csrc/mx_tile.hip, repeated here from its table of costs."""
import os
import re

import pytest

import test_gpu_mx as base
import test_gpu_mx_paths as paths
from weight_quantized_decode_block_amd import build as hip_build

UNITS = 256  # compute units of an MI355X
SOURCE = open(os.path.join(hip_build.CSRC, "mx_tile.hip")).read()
FMT = {"bf16": "kBf16", "mxfp8": "kFp8", "mxfp4": "kFp4"}


def costs(fmt, gated):
    """(bm, bn, first, more, share) of each kernel; the first is the few-row one."""
    body = re.search(rf"struct Costs<MxFormat::{FMT[fmt]}, {str(gated).lower()}> \{{(.*?)\n\}};", SOURCE, re.S).group(1)
    return [tuple(int(x) for x in m) for m in re.findall(r"\{(\d+), (\d+), (\d+), (\d+), (\d+)\}", body)]


def pick(table, M, N, K):
    if M <= 32:
        return 0

    def cost(c):
        bm, bn, first, more, share = c
        parts = -(-(-(-M // bm) * -(-N // bn)) * share // UNITS)
        return first + (parts - share) * more // share if parts > share else first
    return min(range(len(table)), key=lambda i: cost(table[i]))


def launches(fmt, gated):
    """Kernels that the dispatch has for a format, the few-row one among them."""
    text = SOURCE[SOURCE.index("hipError_t launch_fmt"):]
    text = text[:text.index("\n}\n")]
    order = [("bf16", True), ("bf16", False), ("mxfp4", True), ("mxfp4", False), ("mxfp8", True), ("mxfp8", False)]
    parts = re.split(r"if constexpr \(|\} else \{", text)
    return 1 + parts[1 + order.index((fmt, gated))].count("launch_cfg<")


def shapes_of(gated):
    both = base.MANY + base.NARROW + paths.FEW + paths.SHORT + paths.SHORT_TILES + paths.LARGE + paths.THIN
    if not gated:
        return {f: both + base.SHAPES for f in FMT}
    return {f: both + (paths.GATED_64 if f == "mxfp8" else []) for f in FMT}


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", list(FMT))
def test_every_kernel_is_tested(fmt, gated):
    table = costs(fmt, gated)
    assert len(table) == launches(fmt, gated) >= 5
    taken = {i: [] for i in range(len(table))}
    for M, N, K in shapes_of(gated)[fmt]:
        taken[pick(table, M, N, K)].append((M, N, K))
    for i, shapes in taken.items():
        tile = table[i][:2]
        assert len(shapes) >= 2, (fmt, gated, tile, shapes)
        if i:  # outputs in part tiles; a last group of four steps in part
            assert any(M % tile[0] and N % tile[1] for M, N, _ in shapes), (fmt, gated, tile, shapes)
            assert any(K // 128 % 4 for _, _, K in shapes if K > 512), (fmt, gated, tile, shapes)
            assert {128, 384} <= {K for _, _, K in shapes}, (fmt, gated, tile, shapes)


def test_every_height_of_the_few_row_kernel_is_tested():
    source = open(os.path.join(hip_build.CSRC, "mx_skinny.hip")).read()
    heights = [int(x) for x in re.findall(r"op\.M <= (\d+)u\) return launch_cfg<FMT, \1,", source)]
    assert heights == [2, 4, 8, 16]
    rows = [M for M, _, _ in paths.FEW]
    for low, high in zip([0] + heights, heights + [32]):
        assert high in rows and any(low < M < high for M in rows)


def test_both_launches_of_the_row_operators_are_tested():
    source = open(os.path.join(hip_build.CSRC, "mx_quant.hip")).read()
    assert "kManyGroups = 256ull * 4 * 4 * kThreads" in source and "kThreads = 256;" in source
    border = 256 * 4 * 4 * 256 * 8
    sizes = [m * k for m, k, _ in next(x for x in paths.test_large_quantize_and_back.pytestmark if x.args[0] == "M,K,pad").args[1]]
    assert border in sizes and any(s > border for s in sizes) and any(s % 4096 for s in sizes)
    norm = next(x for x in paths.test_norm_rounds_once.pytestmark if x.args[0] == "M,K").args[1]
    assert "gpr <= kNormMaxThreads && M < 1024u" in source and "kNormMaxThreads = 1024" in source
    assert {(M < 1024, K <= 8192, K <= 16384) for M, K in norm} >= {(True, True, True), (False, True, True), (False, False, True), (True, False, False)}
