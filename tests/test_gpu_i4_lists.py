"""GPU tests of routed calls with lists where launches and 32-bit offsets end, and over lists that are not moe_lists'."""
import pytest
import torch

import i4_reference as ref
import test_gpu_moe as moe
from parity import requires_gpu
from test_gpu_i4 import BF, out, untouched
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.mark.parametrize("T,E,top_k,N,K,group", [(131072, 64, 8, 64, 2048, 128), (1 << 20, 300, 1, 17, 2048, 64)])
def test_last_products_of_4_gb_of_rows(T, E, top_k, N, K, group):
    """More than 65535 chunks of 16 rows, which only the kernel for few rows can reach: several launches."""
    g = torch.Generator(device="cuda")
    g.manual_seed(81)
    pairs = T * top_k
    w = ref.Weights(ref.generator(82, T), E, N, K, group, True, "bf16", exact=True)
    h = torch.randint(-8, 9, (pairs, K), generator=g, device="cuda", dtype=torch.int8).to(BF)
    assert h.nbytes >= 1 << 32 and pairs > 16 * 65535
    ids = torch.randint(-1, E, (T, top_k), generator=g, device="cuda", dtype=torch.int32)
    weights = torch.exp2(-torch.randint(0, 3, (T, top_k), generator=g, device="cuda").float())
    order, offsets = torch.empty(pairs, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    wqd.moe_lists(ids, order, offsets, T, top_k, E)
    C, Y = out(T, N, N), torch.full((pairs, N), float("nan"), device="cuda")
    wqd.i4a16_experts_down(h, ids, weights, order, offsets, *w.operands(), Y, C, T, top_k, E, N, K, group)
    some = torch.cat((torch.arange(64), torch.randperm(T, generator=ref.generator(83))[:400], torch.arange(T - 64, T))).unique()
    at = (some.unsqueeze(1) * top_k + torch.arange(top_k)).flatten()
    y, _, here = moe.pair_products(h[at.cuda()].cpu(), w, ids.cpu().flatten()[at], E)
    want = (y * (weights.cpu()[some].double().flatten() * here).unsqueeze(1)).view(-1, top_k, N).sum(1).to(BF)
    assert torch.equal(C.cpu()[some], want) and untouched(C, T, N)
    assert bool(torch.isfinite(C).all())


def test_gated_products_of_4_gb_of_rows():
    T, E, N, K, lda, group = 1100000, 6, 32, 256, 2048, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(84)
    wg, wu = (ref.Weights(ref.generator(85, i), E, N, K, group, True, "fp16") for i in range(2))
    A = torch.full((T, lda), float("nan"), dtype=BF, device="cuda")
    A[:, :K] = torch.randn(T, K, generator=g, device="cuda").to(BF)
    ids = torch.randint(0, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    order, offsets = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    wqd.moe_lists(ids, order, offsets, T, 1, E)
    H = out(T, N, N)
    wqd.i4a16_experts_gated(A, ids, order, offsets, *wg.operands(), *wu.operands(), H, T, 1, E, N, K, group, a_row_stride=lda)
    some = torch.cat((torch.arange(64), torch.randperm(T, generator=ref.generator(86))[:1000], torch.arange(T - 64, T))).unique()
    a, flat = A[some.cuda(), :K].cpu(), ids.cpu().flatten()[some]
    gate, eg, _ = moe.pair_products(a, wg, flat, E)
    up, eu, _ = moe.pair_products(a, wu, flat, E)
    want, err = ref.gated(gate, up, eg, eu)
    assert bool(((H.cpu()[some].double() - want).abs() <= ref.stored(want, err)).all()) and untouched(H, T, N)
    assert bool(torch.isfinite(H).all())


# (T, E, top_k, N, K): the kernel for few rows, tiles of 64 and of 128 rows
ROUTED = [(40, 8, 2, 65, 640), (2000, 4, 2, 257, 128), (2000, 5, 3, 513, 640)]


@pytest.mark.parametrize("T,E,top_k,N,K", ROUTED)
def test_lists_that_point_elsewhere_stay_inside(T, E, top_k, N, K):
    """Lists that are not moe_lists' of any ids are read and written within the operands all the same, in every kernel."""
    g, pairs, group, guard = ref.generator(87, T), T * top_k, 64, 64
    wg, wu, wd = (ref.Weights(g, E, N, K, group, True, "fp16").operands() for _ in range(3))
    ids = moe.choice(g, T, E, top_k).cuda()
    a, h = torch.randn(T, K, generator=g).to(BF).cuda(), torch.randn(pairs, K, generator=g).to(BF).cuda()
    weights = torch.rand(T, top_k, generator=g).cuda()
    some = torch.randint(-(1 << 31), (1 << 31) - 1, (pairs,), generator=g)
    for offsets in ([0] + [pairs] * E, [pairs] * (E + 1), [-1] * (E + 1), [1 << 30, -5, 3, pairs + 1, 100, 7, 0, -(1 << 31), 1 << 30][:E + 1],
                    [0, pairs] * (E // 2 + 1)):
        for order in (torch.full((pairs,), 1 << 30), torch.full((pairs,), -1), torch.full((pairs,), pairs - 1), some):
            lists = order.to(torch.int32).cuda(), torch.tensor(offsets[:E + 1], dtype=torch.int32).cuda()
            H = torch.full((pairs + 2 * guard, N), moe.CANARY, dtype=BF, device="cuda")
            Y = torch.full((pairs + 2 * guard, N), moe.CANARY, device="cuda")
            C = torch.full((T + 2 * guard, N), moe.CANARY, dtype=BF, device="cuda")
            wqd.i4a16_experts_gated(a, ids, *lists, *wg, *wu, H[guard:-guard], T, top_k, E, N, K, group)
            wqd.i4a16_experts_down(h, ids, weights, *lists, *wd, Y[guard:-guard], C[guard:-guard], T, top_k, E, N, K, group)
            for x in (H, Y, C):
                assert bool((x[:guard] == moe.CANARY).all() and (x[-guard:] == moe.CANARY).all())


@pytest.mark.parametrize("T", [600, 2000, 8000])
def test_routed_block_in_tiles(T):
    """As for few tokens: eagerly, captured and replayed, each step against its definition."""
    moe.test_routed_block(T)
