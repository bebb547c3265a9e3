"""GPU tests of the products with 4-bit integer weights at the ends of what activations may be: the largest for which the
header promises finite outputs, and rows that are not finite, on every kernel that sizes choose."""
import pytest
import torch

import i4_reference as ref
import test_gpu_moe as moe
from parity import requires_gpu
from test_gpu_i4 import BF, out, untouched
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]

# the kernel for few rows of 4, 8 and 16, chunks of 32 rows, tiles of 64 and of 128 rows
SIZES = [(1, 40, 256), (6, 40, 256), (12, 40, 256), (97, 5120, 128), (300, 1000, 256), (5864, 385, 256), (5471, 898, 256)]


@pytest.mark.parametrize("top", [15, 255])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_the_largest_activations(M, N, K, group, top):
    """All of one sign, a step below 2^116 with zero points up to 15 and below 2^112 with any.  A group's sums have 8 bits of the
    activation, 7 of the count and 9 of 16 + z: exact in fp32, and so are the outputs before they are rounded."""
    w = ref.Weights(ref.generator(91, M, group), 1, N, K, group, True, "fp16")
    w.codes[:, ::3], w.codes[:, 1::3] = 0, 15
    w.z[:] = top
    w.z[:, N // 2:] = 0
    w.s[:] = 2.0 ** -14
    A = torch.full((M, K), (2.0 - 2.0 ** -7) * 2.0 ** (115 if top == 15 else 111), dtype=BF)
    A[1::2] *= -1.0
    C = out(M, N, N)
    wqd.i4a16_gemm(A.cuda(), *w.operands(), C, M, N, K, group)
    want = (A[:2].double() @ w.values()[0].T).to(BF)
    assert bool(torch.isfinite(want).all()) and torch.equal(C[:M].cpu(), want[torch.arange(M) % 2]) and untouched(C, M, N)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_groups_whose_scores_are_equal_in_64_bits(scoring):
    """Logits of 800 and more: sigmoids are all 1, and softmax has zeros.  Without a bias the largest logit decides between groups
    (group_top 1), and between experts; the sum of two scores leaves equal groups to the lowest index."""
    x = torch.full((1, 16), -900.0)
    x[0, [1, 6, 9, 10, 14]] = torch.tensor([800.0, 850.0, 900.0, 2.0, 1700.0])
    one, _ = moe.route(x, None, 2, scoring=scoring, groups=4, top_groups=2, group_top=1)
    two, _ = moe.route(x, None, 2, scoring=scoring, groups=4, top_groups=2, group_top=2)
    assert one.tolist() == [[14, 9]]  # groups 3 and 2
    # softmax: group 3 and, of those with zeros, 0; sigmoid: group 2 with 1 + 0.88 and, of those with 1 + 0, 0
    assert two.tolist() == ([[14, 1]] if scoring == "softmax" else [[9, 1]])
    for group_top in (1, 2):
        moe.check_route(x, None, 2, scoring=scoring, groups=4, top_groups=2, group_top=group_top)


def both(fn, operands, into, a, at, bad):
    """Outputs of rows a and of the same with `bad` at a[at]."""
    got = []
    for x in (a, a.clone()):
        if got:
            x[at] = bad
        C = into()
        fn(x, *operands, C)
        got.append(C)
    return got


BAD = [float("inf"), -float("inf"), float("nan")]
CONFIGS = [(32, True), (64, False), (64, True), (128, False), (128, True)]


@pytest.mark.parametrize("group,zeros", CONFIGS)
@pytest.mark.parametrize("M,N,K", SIZES[3:])
def test_rows_that_are_not_finite_stay_alone(M, N, K, group, zeros):
    """A row with an infinity or NaN has no finite output, and the other rows' bits are as they were."""
    g = ref.generator(92, M)
    wg, wu = (ref.Weights(g, 1, N, K, group, zeros, "fp16").operands() for _ in range(2))
    a = torch.randn(M, K, generator=g).to(BF).cuda()
    for i, bad in enumerate(BAD):
        at = (0, M // 2, M - 1)[i]
        keep = torch.arange(M) != at
        for fn, w in ((lambda x, *o: wqd.i4a16_gemm(x, *o, M, N, K, group), wg), (lambda x, *o: wqd.i4a16_gated(x, *o, M, N, K, group), wg + wu)):
            C, D = both(fn, w, lambda: out(M, N, N), a, (at, 100 + i), bad)
            assert not bool(torch.isfinite(D[at]).any()) and bool(torch.isfinite(C[:M]).all())
            assert torch.equal(C[:M].cpu()[keep], D[:M].cpu()[keep]) and untouched(D, M, N)


# (T, E, top_k, N, K): the kernel for few rows, tiles of 64 and of 128 rows
ROUTED = [(1, 4, 2, 40, 256), (20, 4, 2, 40, 256), (2000, 4, 2, 257, 128), (2000, 5, 3, 513, 640)]


@pytest.mark.parametrize("group,zeros", CONFIGS)
@pytest.mark.parametrize("T,E,top_k,N,K", ROUTED)
def test_routed_rows_that_are_not_finite_stay_alone(T, E, top_k, N, K, group, zeros):
    """A token with an infinity or NaN reaches its own pairs' rows alone, and a pair's row its own token's outputs."""
    g = ref.generator(93, T)
    wg, wu, wd = (ref.Weights(g, E, N, K, group, zeros, "fp16").operands() for _ in range(3))
    ids = torch.stack([torch.randperm(E, generator=g)[:top_k] for _ in range(T)]).to(torch.int32).cuda()
    weights = (torch.rand(T, top_k, generator=g) + 0.1).cuda()
    order, offsets = torch.empty(T * top_k, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    wqd.moe_lists(ids, order, offsets, T, top_k, E)
    a, h = torch.randn(T, K, generator=g).to(BF).cuda(), torch.randn(T * top_k, K, generator=g).to(BF).cuda()
    for lists in ((None, None), (order, offsets)) if T < 100 else ((order, offsets),):
        Y = torch.empty(T * top_k, N, device="cuda")
        for i, bad in enumerate(BAD):
            t = (0, T // 2, T - 1)[i]
            C, D = both(lambda x, *o: wqd.i4a16_experts_gated(x, ids, *lists, *o, T, top_k, E, N, K, group), wg + wu,
                        lambda: out(T * top_k, N, N), a, (t, 100 + i), bad)
            hit = torch.arange(T * top_k) // top_k == t
            assert not bool(torch.isfinite(D[:-1].cpu()[hit]).any()) and torch.equal(C[:-1].cpu()[~hit], D[:-1].cpu()[~hit])
            assert bool(torch.isfinite(C).all()) and untouched(D, T * top_k, N)
            C, D = both(lambda x, *o: wqd.i4a16_experts_down(x, ids, weights, *lists, *o[:3], Y, o[3], T, top_k, E, N, K, group), wd,
                        lambda: out(T, N, N), h, (t * top_k + top_k - 1, 100 + i), bad)
            hit = torch.arange(T) == t
            assert not bool(torch.isfinite(D[:-1].cpu()[hit]).any()) and torch.equal(C[:-1].cpu()[~hit], D[:-1].cpu()[~hit])
            assert bool(torch.isfinite(C).all()) and untouched(D, T, N)
