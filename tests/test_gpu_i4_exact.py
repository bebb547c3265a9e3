"""GPU tests of the products with 4-bit integer weights where every sum is exact, at the lengths of K that are split over the waves
many steps each: no error of sums widens the tolerance, so that a step, a group or a wave's share that is lost shows
(test_i4_exact.py checks on the CPU that it would)."""
import pytest
import torch

import i4_reference as ref
from parity import requires_gpu
from test_gpu_i4 import BF, SIZES, out, untouched
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]

EXACT = SIZES + [(M, N, K) for K in (5120, 17408) for M, N in ((1, 100), (4, 130), (8, 129), (16, 257), (33, 100))]
CONFIGS = [(128, False, "fp16"), (64, True, "bf16"), (32, True, "fp16"), (128, True, "fp16")]


def inputs(seed, M, N, K, group, zeros, scale, count=1):
    """Activations of -8 .. 8 and scales of 2^-9 .. 2^-11: in units of 2^-11 a sum is below 17408 * 8 * 15 * 4 < 2^23 in magnitude, and a
    group's sums of a (16 + q) below 128 * 8 * 31: exact in fp32, added in any order."""
    g = ref.generator(seed, M, N, K, group)
    ws = [ref.Weights(g, 1, N, K, group, zeros, scale, exact=True) for _ in range(count)]
    for w in ws:
        w.s *= 2.0 ** -5
    return ws, torch.randint(-8, 9, (M, K), generator=g).to(BF)


def sums(a, w):
    return a.double() @ w.values()[0].T


def gated(gate, up):
    """silu(gate) * up of exact sums, and how far the output may be: the activation's own error and the rounding."""
    want, err = ref.gated(gate, up, torch.zeros_like(gate), torch.zeros_like(up))
    return want, ref.stored(want, err)


@pytest.mark.parametrize("group,zeros,scale", CONFIGS)
@pytest.mark.parametrize("M,N,K", EXACT)
def test_product(M, N, K, group, zeros, scale):
    (w,), a = inputs(101, M, N, K, group, zeros, scale)
    want = sums(a, w).to(BF)
    for operands in (w.operands(), (w.operands()[0], w.s.cuda(), w.z.cuda() if zeros else None)):
        C = out(M, N, N)
        wqd.i4a16_gemm(a.cuda(), *operands, C, M, N, K, group)
        assert torch.equal(C[:M].cpu(), want) and untouched(C, M, N)


@pytest.mark.parametrize("group,zeros,scale", CONFIGS)
@pytest.mark.parametrize("M,N,K", EXACT)
def test_gated(M, N, K, group, zeros, scale):
    (wg, wu), a = inputs(102, M, N, K, group, zeros, scale, 2)
    want, bound = gated(sums(a, wg), sums(a, wu))
    C = out(M, N, N)
    wqd.i4a16_gated(a.cuda(), *wg.operands(), *wu.operands(), C, M, N, K, group)
    assert bool(((C[:M].cpu().double() - want).abs() <= bound).all()) and untouched(C, M, N)


# (T, E, top_k, N, K)
ROUTED = [(1, 4, 2, 40, 5120), (3, 8, 2, 130, 4096), (40, 4, 2, 65, 5120), (300, 3, 2, 129, 2048), (2000, 5, 3, 200, 1152)]


@pytest.mark.parametrize("group,zeros,scale", CONFIGS)
@pytest.mark.parametrize("T,E,top_k,N,K", ROUTED)
def test_experts(T, E, top_k, N, K, group, zeros, scale):
    g = ref.generator(103, T, E, N, K)
    wg, wu = (ref.Weights(g, E, N, K, group, zeros, scale, exact=True) for _ in range(2))
    for w in (wg, wu):
        w.s *= 2.0 ** -5
    a = torch.randint(-8, 9, (T, K), generator=g).to(BF)
    ids = torch.stack([torch.randperm(E, generator=g)[:top_k] for _ in range(T)]).to(torch.int32)
    lists = tuple(x.cuda() for x in ref.lists(ids, E))
    flat, rows = ids.flatten().long(), a.repeat_interleave(top_k, 0).double()
    gate, up = (torch.empty(T * top_k, N, dtype=torch.float64) for _ in range(2))
    for e in range(E):
        at = flat == e
        gate[at], up[at] = rows[at] @ wg.values()[e].T, rows[at] @ wu.values()[e].T
    want, bound = gated(gate, up)
    for order, offsets in ((None, None), lists) if T < 1000 else (lists,):
        H = out(T * top_k, N, N)
        wqd.i4a16_experts_gated(a.cuda(), ids.cuda(), order, offsets, *wg.operands(), *wu.operands(), H, T, top_k, E, N, K, group)
        assert bool(((H[:-1].cpu().double() - want).abs() <= bound).all()) and untouched(H, T * top_k, N)
