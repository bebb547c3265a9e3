"""GPU tests of the products with scales and zero points row by row: against the definition in 64 bits (i4_reference)
and, on every path that sizes choose, bit for bit against the same weights in tiles."""
import pytest
import torch

import i4_reference as ref
import test_gpu_i4_paths as paths
import test_gpu_moe as moe
from parity import requires_gpu
from test_gpu_i4 import BF, CANARY, out, rows, untouched
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]


def by_row(w):
    """Operands of ref.Weights with its scales and zero points as they are."""
    return ref.laid_out(w.codes).cuda(), w.s.cuda(), None if w.z is None else w.z.cuda()


@pytest.mark.parametrize("scale", ["fp16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (1, 96, 1152), (3, 17, 256), (5, 1, 1152), (8, 32, 2176), (16, 48, 1024), (23, 65, 640), (40, 130, 512),
                                   (130, 257, 256), (300, 1000, 256), (1000, 500, 384)])
def test_product_exact(M, N, K, group, zeros, scale):
    """Integers times powers of two: every sum is exact in fp32, so the outputs are the rounded exact sums."""
    g = ref.generator(61, M, N, K, group)
    w = ref.Weights(g, 1, N, K, group, zeros, scale, exact=True)
    a, A = rows(g, M, K, exact=True)
    C = out(M, N, N)
    wqd.i4a16_gemm(A, *by_row(w), C, M, N, K, group)
    assert torch.equal(C[:M].cpu(), (a.double() @ w.values()[0].T).to(BF)) and untouched(C, M, N)


class Pair:
    """The same random matrices with scales and zero points in both layouts, made on the GPU.  What follows the rows in memory
    are NaN and 255."""

    def __init__(self, seed, E, N, K, group, zeros, scale):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        R, t, k = wqd.i4_packed_rows(N), ref.SCALES[scale], K // group
        codes = torch.randint(0, 256, (E, R * K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = ((torch.rand(E, N, k, generator=g, device="cuda") + 0.5) * K ** -0.5).to(t)
        z = torch.randint(0, 16, (E, N, k), generator=g, device="cuda", dtype=torch.uint8) if zeros else None

        def tiles(x, fill):
            wide = torch.full((E, R, k), fill, dtype=x.dtype, device="cuda")
            wide[:, :N] = x
            return wide.view(E, R // 16, 16, K // 128, 128 // group).transpose(2, 3).contiguous()

        def rows(x, fill):
            memory = torch.full((x.numel() + 64 * k,), fill, dtype=x.dtype, device="cuda")
            memory[:x.numel()] = x.flatten()
            return memory[:x.numel()].view(x.shape)

        self.rows = codes, rows(s, float("nan")), rows(z, 255) if zeros else None
        self.tiles = codes, tiles(s, 0), tiles(z, 0) if zeros else None


FEW = [(1, 5120, 5120), (2, 333, 17408), (4, 1000, 384), (7, 513, 5120), (11, 512, 4992), (16, 129, 17408), (17, 257, 1024), (45, 5119, 5120)]


@pytest.mark.parametrize("group,zeros,scale", paths.CONFIGS)
@pytest.mark.parametrize("M,N,K", FEW + paths.PRODUCT + paths.PRODUCT_SPLIT)
def test_product_as_with_tiles(M, N, K, group, zeros, scale):
    w = Pair(62 + M, 1, N, K, group, zeros, scale)
    A = torch.randn(M, K, device="cuda").to(BF)
    C, D = out(M, N, N), out(M, N, N)
    wqd.i4a16_gemm(A, *w.tiles, C, M, N, K, group)
    wqd.i4a16_gemm(A, *w.rows, D, M, N, K, group)
    assert torch.equal(C, D) and bool(torch.isfinite(D).all()) and bool((D[:M] != 0).any())


@pytest.mark.parametrize("group,zeros,scale", paths.CONFIGS)
@pytest.mark.parametrize("M,N,K", FEW + paths.GATED + paths.GATED_SPLIT + paths.GATED_LARGE)
def test_gated_as_with_tiles(M, N, K, group, zeros, scale):
    gate, up = Pair(63 + M, 1, N, K, group, zeros, scale), Pair(64 + M, 1, N, K, group, zeros, scale)
    A = torch.randn(M, K, device="cuda").to(BF)
    C, D = out(M, N, N), out(M, N, N)
    wqd.i4a16_gated(A, *gate.tiles, *up.tiles, C, M, N, K, group)
    wqd.i4a16_gated(A, *gate.rows, *up.rows, D, M, N, K, group)
    assert torch.equal(C, D) and bool(torch.isfinite(D).all()) and bool((D[:M] != 0).any())


@pytest.mark.parametrize("group,zeros,scale", paths.CONFIGS)
@pytest.mark.parametrize("T,E,top_k,N,K", moe.EXPERTS + paths.LISTS + [(2, 4, 2, 40, 4096)])
def test_experts_as_with_tiles(T, E, top_k, N, K, group, zeros, scale):
    """With lists and without, the gated and the last products."""
    g = ref.generator(65, T, E, N, K)
    ids = moe.choice(g, T, E, top_k)
    gate, up, down = (Pair(66 + i, E, N, K, group, zeros, scale) for i in range(3))
    a, h = torch.randn(T, K, generator=g).to(BF).cuda(), torch.randn(T * top_k, K, generator=g).to(BF).cuda()
    weights = torch.rand(T, top_k, generator=g).cuda()
    for order, offsets in ((None, None), moe.lists_of(ids, E)):
        got = []
        for how in ("tiles", "rows"):
            H, C, Y = out(T * top_k, N, N), out(T, N, N), torch.full((T * top_k, N), float("nan"), device="cuda")
            G, U, W = (getattr(w, how) for w in (gate, up, down))
            wqd.i4a16_experts_gated(a, ids.cuda(), order, offsets, *G, *U, H, T, top_k, E, N, K, group)
            wqd.i4a16_experts_down(h, ids.cuda(), weights, order, offsets, *W, Y, C, T, top_k, E, N, K, group)
            got.append((H, C))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert bool(torch.isfinite(got[1][0]).all()) and bool((got[1][1] != 0).any()) and untouched(got[1][1], T, N)


@pytest.mark.parametrize("group,zeros,scale", [(128, True, "fp16"), (64, True, "bf16"), (32, False, "fp16")])
@pytest.mark.parametrize("T,E,top_k,N,K", [(2, 4, 2, 17, 256), (33, 8, 2, 65, 640), (300, 3, 2, 300, 512)])
def test_experts_exact(T, E, top_k, N, K, group, zeros, scale):
    """The last products of exact sums, each slot weighted by a power of two: the outputs are the rounded exact sums."""
    g = ref.generator(67, T, E, N, K)
    ids = moe.choice(g, T, E, top_k)
    w = ref.Weights(g, E, N, K, group, zeros, scale, exact=True)
    h = torch.randint(-8, 9, (T * top_k, K), generator=g).to(BF)
    weights = torch.exp2(-torch.randint(0, 3, (T, top_k), generator=g).float())
    y, _, here = moe.pair_products(h, w, ids, E)
    want = (y * (weights.double().flatten() * here).unsqueeze(1)).view(T, top_k, N).sum(1).to(BF)
    for order, offsets in ((None, None), moe.lists_of(ids, E)):
        C, Y = out(T, N, N), torch.full((T * top_k, N), float("nan"), device="cuda")
        wqd.i4a16_experts_down(h.cuda(), ids.cuda(), weights.cuda(), order, offsets, *by_row(w), Y, C, T, top_k, E, N, K, group)
        assert torch.equal(C[:T].cpu(), want) and untouched(C, T, N)


@pytest.mark.parametrize("E,N,K,group", [(1, 1, 128, 128), (3, 17, 384, 32), (2, 100, 1152, 64)])
def test_pack_of_codes_alone(E, N, K, group):
    w = ref.Weights(ref.generator(73, E, N, K), E, N, K, group, True, "fp16", exact=True)
    W = torch.full((E * wqd.i4_packed_rows(N) * K // 2 + 32,), 0xA5, dtype=torch.uint8, device="cuda")
    wqd.i4_pack(ref.rows_of_pairs(w.codes).cuda(), None, None, W, None, None, N, K, group, E)
    assert torch.equal(W[:-32].cpu(), ref.laid_out(w.codes).flatten()) and bool((W[-32:] == 0xA5).all())
    a, A = rows(ref.generator(74, N), 3, K, exact=True)
    C = out(3, N, N)
    wqd.i4a16_gemm(A, W[:-32], w.s.cuda(), w.z.cuda(), C, 3, N, K, group)
    assert torch.equal(C[:3].cpu(), (a.double() @ w.values()[0].T).to(BF)) and untouched(C, 3, N)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_every_scale_of_a_slice(M):
    """Rows that begin anywhere: scales and zero points of rows 1 .. of a larger matrix, aligned to their own loads only."""
    N, K = 40, 384
    for group in (128, 64, 32):
        w = ref.Weights(ref.generator(68, M, group), 1, N, K, group, True, "fp16", exact=True)
        s, z = (torch.cat((x[:, :1], x), 1).cuda()[:, 1:] for x in (w.s, w.z))
        assert s.data_ptr() % 16 or z.data_ptr() % 16
        a, A = rows(ref.generator(69, M), M, K, exact=True)
        C = out(M, N, N)
        wqd.i4a16_gemm(A, ref.laid_out(w.codes).cuda(), s, z, C, M, N, K, group)
        assert torch.equal(C[:M].cpu(), (a.double() @ w.values()[0].T).to(BF)) and untouched(C, M, N)


@pytest.mark.parametrize("T", [1, 40, 1000])
def test_scales_beyond_4_gb(T):
    """The last of 33 matrices, 4.4 GB of scales in all: few rows, chunks and tiles.  Only its last 16 rows are not zeros."""
    E, N, K, group = 33, 8192, 262144, 32
    g = ref.generator(70, T)
    last = ref.Weights(g, 1, 16, K, group, False, "fp16")
    last.s[:] = 2.0 ** -6  # |sum a (q - 8)| <= 2^22 of these units: exact
    W = ref.laid_out(last.codes).cuda()
    codes = torch.zeros(E * N * K // 2, dtype=torch.uint8, device="cuda")
    codes[-W.numel():] = W.flatten()
    scales = torch.zeros(E, N, K // group, dtype=torch.float16, device="cuda")
    scales[-1, -16:] = 2.0 ** -6
    assert scales.nbytes > 1 << 32
    A = torch.randint(-2, 3, (T, K), generator=g).to(BF).cuda()
    ids = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
    order, offsets = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    wqd.moe_lists(ids, order, offsets, T, 1, E)
    want = (A.double() @ last.values()[0].T.cuda()).to(BF)
    for lists in ((None, None), (order, offsets)) if T < 100 else ((order, offsets),):
        C, Y = out(T, N, N), torch.empty(T, N, device="cuda")
        wqd.i4a16_experts_down(A, ids, torch.ones(T, 1, device="cuda"), *lists, codes, scales, None, Y, C, T, 1, E, N, K, group)
        assert torch.equal(C[:T, -16:], want) and bool((C[:T, :-16] == 0).all()) and untouched(C, T, N)


@pytest.mark.parametrize("M", [1, 6, 50, 700])
def test_graph_replays(M):
    """Captured calls give the eager results, replay after replay, also on new inputs in the same places."""
    N, K, group = 200, 384, 64
    gate, up = Pair(71, 1, N, K, group, True, "fp16"), Pair(72, 1, N, K, group, True, "fp16")
    A, C, D = torch.randn(M, K, device="cuda").to(BF), out(M, N, N), out(M, N, N)

    def calls():
        wqd.i4a16_gemm(A, *gate.rows, C, M, N, K, group)
        wqd.i4a16_gated(A, *gate.rows, *up.rows, D, M, N, K, group)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        calls()
    for _ in range(4):
        A.copy_(torch.randn(M, K, device="cuda").to(BF))
        C.fill_(CANARY), D.fill_(CANARY)
        graph.replay()
        torch.cuda.synchronize()
        got = C.clone(), D.clone()
        calls()
        assert torch.equal(got[0], C) and torch.equal(got[1], D)
