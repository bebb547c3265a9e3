"""The products with 4-bit integer weights on every path that sizes choose, each at
sizes that take it (test_i4_paths.py checks on the CPU that every one is taken), and
at sizes where offsets pass 32 bits."""
import pytest
import torch

import i4_reference as ref
import test_gpu_moe as moe
from parity import requires_gpu
from test_gpu_i4 import BF, CANARY, out, rows, untouched
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]

CONFIGS = [(group, zeros, "bf16" if (group == 64) == zeros else "fp16") for group in (32, 64, 128) for zeros in (False, True)]
# (M, N, K): tiles of 128 rows for whole rounds and the last outputs in chunks of 16, of 32 rows and tiles of 64
PRODUCT_SPLIT = [(8248, 1808, 640), (4368, 1991, 640), (5435, 1747, 640)]
GATED_SPLIT = [(3883, 2052, 384), (6211, 771, 384), (6793, 710, 384)]
# tiles of 64 rows for whole rounds, and a prompt's
GATED_LARGE = [(165, 16774, 5120), (500, 17408, 5120)]
# chunks of 32 rows, tiles of 64 and of 128 rows; one to five steps
PRODUCT = [(97, 5120, 128), (300, 1000, 256), (1000, 500, 384), (7043, 385, 128), (5864, 385, 256), (5864, 385, 640), (7698, 898, 128),
           (5471, 898, 256), (4947, 898, 384), (4685, 841, 640)]
GATED = [(97, 5120, 128), (300, 1000, 256), (1000, 500, 384), (4554, 328, 128), (4554, 271, 256), (4554, 271, 640), (5733, 613, 128),
         (7436, 328, 256), (5733, 385, 384), (5078, 385, 640)]
# (T, E, top_k, N, K)
LISTS = [(2000, 4, 2, 257, 128), (900, 4, 2, 700, 384), (3000, 3, 2, 300, 256), (6000, 3, 1, 300, 128), (1500, 16, 4, 640, 128),
         (2000, 5, 3, 513, 640)]


@pytest.mark.parametrize("group,zeros,scale", CONFIGS)
@pytest.mark.parametrize("M,N,K", PRODUCT + PRODUCT_SPLIT)
def test_product_exact(M, N, K, group, zeros, scale):
    """Integers times powers of two: every sum is exact in fp32, so the outputs are the rounded exact sums."""
    g = ref.generator(41, M, N, K, group)
    w = ref.Weights(g, 1, N, K, group, zeros, scale, exact=True)
    lda, ldc = K + 8 * (M % 3), N + 8 - N % 8 + M % 2  # whole 16-byte rows for even M only
    a, A = rows(g, M, K, lda, exact=True)
    C = out(M, N, ldc)
    wqd.i4a16_gemm(A, *w.operands(), C, M, N, K, group, a_row_stride=lda, c_row_stride=ldc)
    assert torch.equal(C[:M, :N].cpu(), (a.double() @ w.values()[0].T).to(BF)) and untouched(C, M, N)


@pytest.mark.parametrize("group,zeros,scale", CONFIGS)
@pytest.mark.parametrize("M,N,K", GATED + GATED_SPLIT)
def test_gated(M, N, K, group, zeros, scale):
    g = ref.generator(42, M, N, K, group)
    wg, wu = ref.Weights(g, 1, N, K, group, zeros, scale), ref.Weights(g, 1, N, K, group, zeros, scale)
    a, A = rows(g, M, K)
    C = out(M, N, N)
    wqd.i4a16_gated(A, *wg.operands(), *wu.operands(), C, M, N, K, group)
    sums = [(a.double() @ w.values()[0].T, ref.sum_error(a.double().abs() @ w.size()[0].T, K)) for w in (wg, wu)]
    want, err = ref.gated(sums[0][0], sums[1][0], sums[0][1], sums[1][1])
    assert bool(((C[:M].cpu().double() - want).abs() <= ref.stored(want, err)).all()) and untouched(C, M, N)


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("M,N,K", GATED_LARGE)
def test_gated_by_parts(M, N, K, group):
    """Bit for bit as its parts of 1040 outputs, which take other kernels: all sums are exact."""
    g = torch.Generator(device="cuda")
    g.manual_seed(51)
    R = wqd.i4_packed_rows(N)

    def weights():
        codes = torch.randint(0, 256, (R, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = torch.exp2(-torch.randint(6, 9, (R, K // group), generator=g, device="cuda").float()).half()
        return codes, s, torch.randint(0, 16, (R, K // group), generator=g, device="cuda", dtype=torch.uint8)

    G, U = weights(), weights()
    A = torch.randint(-2, 3, (M, K), generator=g, device="cuda").to(BF)
    C, D = out(M, N, N), out(M, N, N)
    wqd.i4a16_gated(A, *G, *U, C, M, N, K, group)
    for n in range(0, N, 1040):
        m = min(1040, N - n)
        part = lambda x: x[n:n + wqd.i4_packed_rows(m)]  # noqa: E731
        wqd.i4a16_gated(A, *map(part, G), *map(part, U), D[:, n:], M, m, K, group, c_row_stride=N)
    assert torch.equal(C, D) and untouched(C, M, N) and bool((C[:M] != 0).any())


@pytest.mark.parametrize("M", [3, 40, 150])
def test_the_most_outputs(M):
    """2^24 outputs, the most there may be: bit for bit as parts of them."""
    N, K, group = 1 << 24, 128, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(52)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.exp2(-torch.randint(6, 9, (N, K // group), generator=g, device="cuda").float()).bfloat16()
    A = torch.randint(-2, 3, (M, K), generator=g, device="cuda").to(BF)
    C = torch.full((M, N), CANARY, dtype=BF, device="cuda")
    wqd.i4a16_gemm(A, codes, s, None, C, M, N, K, group)
    D = out(M, 512, 512)
    for n in (0, 1 << 20, (1 << 23) + 16, (1 << 24) - 4096 - 256, (1 << 24) - 512):
        wqd.i4a16_gemm(A, codes[n:n + 512], s[n:n + 512], None, D, M, 512, K, group)
        assert torch.equal(C[:, n:n + 512], D[:M])
    assert not bool((C == CANARY).any())


@pytest.mark.parametrize("group,zeros,scale", CONFIGS)
@pytest.mark.parametrize("T,E,top_k,N,K", LISTS)
def test_experts(T, E, top_k, N, K, group, zeros, scale):
    moe.test_experts_gated(T, E, top_k, N, K, group, zeros, scale)
    moe.test_experts_down(T, E, top_k, N, K, group, zeros, scale)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T", [40, 3000])
def test_one_expert_has_all(T, zeros):
    """Every token at the same expert, the others without any: bit for bit as one dense product."""
    E, N, K, group = 6, 300, 256, 64
    g = ref.generator(43, T)
    wg, wu = (ref.Weights(g, E, N, K, group, zeros, "bf16", exact=True) for _ in range(2))
    one = ref.Weights(g, 1, N, K, group, zeros, "bf16", exact=True), ref.Weights(g, 1, N, K, group, zeros, "bf16", exact=True)
    for w, v in zip((wg, wu), one):
        v.codes, v.s, v.z = w.codes[4:5], w.s[4:5], None if w.z is None else w.z[4:5]
    _, A = rows(g, T, K, exact=True)
    ids = torch.full((T, 1), 4, dtype=torch.int32).cuda()
    order, offsets = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    wqd.moe_lists(ids, order, offsets, T, 1, E)
    want = out(T, N, N)
    wqd.i4a16_gated(A, *one[0].operands(), *one[1].operands(), want, T, N, K, group)
    for lists in ((None, None), (order, offsets)):
        H = out(T, N, N)
        wqd.i4a16_experts_gated(A, ids, *lists, *wg.operands(), *wu.operands(), H, T, 1, E, N, K, group)
        assert torch.equal(H, want)


def test_more_pairs_than_a_launch_of_few_rows_holds():
    T, E, top_k, N, K, group = 200000, 8, 8, 24, 128, 128
    g = ref.generator(44)
    wg, wu = (ref.Weights(g, E, N, K, group, True, "fp16") for _ in range(2))
    wd = ref.Weights(g, E, N, K, group, False, "fp16")
    ids = torch.randint(-1, E, (T, top_k), generator=g, dtype=torch.int32)
    a, A = rows(g, T, K)
    order, offsets = torch.empty(T * top_k, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    wqd.moe_lists(ids.cuda(), order, offsets, T, top_k, E)
    flat = ids.flatten()
    by = torch.sort(flat, stable=True)[1][int((flat < 0).sum()):].to(torch.int32)
    assert torch.equal(order.cpu()[:len(by)], by) and bool((order[len(by):] == -1).all())
    H = out(T * top_k, N, N)
    wqd.i4a16_experts_gated(A, ids.cuda(), order, offsets, *wg.operands(), *wu.operands(), H, T, top_k, E, N, K, group)
    some = torch.randperm(T, generator=g)[:500].sort()[0]
    pairs = (some.unsqueeze(1) * top_k + torch.arange(top_k)).flatten()
    x = a[some].repeat_interleave(top_k, 0)
    gate, eg, here = moe.pair_products(x, wg, flat[pairs], E)
    up, eu, _ = moe.pair_products(x, wu, flat[pairs], E)
    want, err = ref.gated(gate, up, eg, eu)
    got = H.cpu()[pairs].double()
    assert bool((got[~here] == CANARY).all()) and bool(((got - want).abs() <= ref.stored(want, err))[here].all())
    h = torch.randn(T * top_k, K, generator=g).to(BF)
    weights = torch.rand(T, top_k, generator=g)
    C, Y = out(T, N, N), torch.full((T * top_k, N), float("nan"), device="cuda")
    wqd.i4a16_experts_down(h.cuda(), ids.cuda(), weights.cuda(), order, offsets, *wd.operands(), Y, C, T, top_k, E, N, K, group)
    y, err, here = moe.pair_products(h[pairs], wd, flat[pairs], E)
    s = (weights[some].double().flatten() * here).unsqueeze(1)
    want, err = ((v.view(-1, top_k, N).sum(1)) for v in (s * y, s * err + (top_k + 2) * 2.0 ** -23 * s * (y.abs() + err)))
    assert bool(((C.cpu()[some].double() - want).abs() <= ref.stored(want, err)).all()) and untouched(C, T, N)


@pytest.mark.parametrize("T", [1, 3, 1000])
def test_experts_beyond_4_gb(T):
    """The last of nine matrices, 4.8 GB in all: few rows, chunks and tiles.  Only its last 16 rows are not zeros."""
    E, N, K, group = 9, 8192, 131072, 128
    g = ref.generator(45, T)
    last = ref.Weights(g, 1, 16, K, group, False, "fp16")
    last.s[:] = 2.0 ** -6  # |sum a (q - 8)| <= 2^21 of these units: exact
    W, S, _ = last.operands()
    codes, scales = (torch.zeros(E * N * K // n, dtype=t, device="cuda") for n, t in ((2, torch.uint8), (group, torch.float16)))
    codes[-W.numel():], scales[-S.numel():] = W.flatten(), S.flatten()
    A = torch.randint(-2, 3, (T, K), generator=g).to(BF).cuda()
    ids = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
    order, offsets = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    wqd.moe_lists(ids, order, offsets, T, 1, E)
    want = (A.double() @ last.values()[0].T.cuda()).to(BF)
    up = torch.full_like(scales, 2.0 ** -12)  # the up matrix: codes of the gate's
    for lists in ((None, None), (order, offsets)) if T < 100 else ((order, offsets),):
        C, Y = out(T, N, N), torch.empty(T, N, device="cuda")
        wqd.i4a16_experts_down(A, ids, torch.ones(T, 1, device="cuda"), *lists, codes, scales, None, Y, C, T, 1, E, N, K, group)
        assert torch.equal(C[:T, -16:], want) and bool((C[:T, :-16] == 0).all()) and untouched(C, T, N)
        H = out(T, N, N)
        wqd.i4a16_experts_gated(A, ids, *lists, codes, scales, None, codes, up, None, H, T, 1, E, N, K, group)
        u = A.double() @ last.values()[0].T.cuda()
        y = ref.silu(u) * (u * 2.0 ** -6)
        assert bool(((H[:T, -16:].double() - y).abs() <= ref.stored(y, 2.0 ** -16 * y.abs())).all()) and bool((H[:T, :-16] == 0).all())


@pytest.mark.parametrize("M,N,K,lda,ldc", [(1100, 64, 128, 1 << 21, 1 << 21), (7043, 385, 128, 1 << 19, 1 << 19), (7698, 898, 128, 1 << 19, 1000)])
def test_rows_beyond_4_gb(M, N, K, lda, ldc):
    g = ref.generator(46, M)
    w = ref.Weights(g, 1, N, K, 64, True, "bf16", exact=True)
    a = torch.randint(-8, 9, (M, K), generator=g).to(BF)
    A = torch.full((M, lda), float("nan"), dtype=BF, device="cuda")
    A[:, :K] = a.cuda()
    C = torch.full((M, ldc), CANARY, dtype=BF, device="cuda")
    wqd.i4a16_gemm(A, *w.operands(), C, M, N, K, 64, a_row_stride=lda, c_row_stride=ldc)
    assert torch.equal(C[:, :N].cpu(), (a.double() @ w.values()[0].T).to(BF)) and bool((C[:, N:] == CANARY).all())


def test_listed_rows_beyond_4_gb():
    T, E, N, K, lda = 2100, 2, 600, 128, 1 << 20
    g = ref.generator(47)
    wg, wu = (ref.Weights(g, E, N, K, 128, False, "fp16") for _ in range(2))
    a = torch.randn(T, K, generator=g).to(BF)
    A = torch.full((T, lda), float("nan"), dtype=BF, device="cuda")
    A[:, :K] = a.cuda()
    ids = torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32)
    order, offsets = moe.lists_of(ids, E)
    gate, eg, _ = moe.pair_products(a, wg, ids, E)
    up, eu, _ = moe.pair_products(a, wu, ids, E)
    want, err = ref.gated(gate, up, eg, eu)
    H = out(T, N, N)
    wqd.i4a16_experts_gated(A, ids.cuda(), order, offsets, *wg.operands(), *wu.operands(), H, T, 1, E, N, K, 128, a_row_stride=lda)
    assert bool(((H[:T].cpu().double() - want).abs() <= ref.stored(want, err)).all()) and untouched(H, T, N)


@pytest.mark.parametrize("M,N,K", [(3, 700, 1024), (700, 777, 384), (5864, 385, 256), (4947, 898, 384)])
def test_two_streams_at_once(M, N, K):
    """Calls of two streams on the same weights and activations, twenty of each in flight: the same bits from all."""
    g = ref.generator(48, M)
    w = ref.Weights(g, 1, N, K, 128, True, "fp16").operands()
    _, A = rows(g, M, K)
    want = out(M, N, N)
    wqd.i4a16_gemm(A, *w, want, M, N, K, 128)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [[out(M, N, N) for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for s, cs in zip(streams, outs):
            wqd.i4a16_gemm(A, *w, cs[i], M, N, K, 128, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for cs in outs for c in cs)


@pytest.mark.parametrize("T", [30, 3000])
def test_two_routed_blocks_at_once(T):
    """Two captured blocks that share weights and inputs, each with its own lists and scratch, replayed side by side."""
    E, top_k, D, F, group = 4, 2, 256, 384, 64
    g = ref.generator(49, T)
    wg, wu, wd = (ref.Weights(g, E, *n, group, True, "fp16").operands() for n in ((F, D), (F, D), (D, F)))
    _, x = rows(g, T, D)
    logits = torch.randn(T, E, generator=g).cuda()

    class Block:
        def __init__(self):
            i32 = dict(dtype=torch.int32, device="cuda")
            self.ids, self.weights = torch.empty(T, top_k, **i32), torch.empty(T, top_k, device="cuda")
            self.order, self.offsets = torch.empty(T * top_k, **i32), torch.empty(E + 1, **i32)
            self.H, self.Y = torch.empty(T * top_k, F, dtype=BF, device="cuda"), torch.empty(T * top_k, D, device="cuda")
            self.C = torch.empty(T, D, dtype=BF, device="cuda")

        def run(self):
            wqd.moe_route(logits, None, self.ids, self.weights, T, E, top_k)
            wqd.moe_lists(self.ids, self.order, self.offsets, T, top_k, E)
            wqd.i4a16_experts_gated(x, self.ids, self.order, self.offsets, *wg, *wu, self.H, T, top_k, E, F, D, group)
            wqd.i4a16_experts_down(self.H, self.ids, self.weights, self.order, self.offsets, *wd, self.Y, self.C, T, top_k, E, D, F, group)

    first, blocks = Block(), (Block(), Block())
    first.run()
    graphs = []
    for b in blocks:
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            b.run()
        graphs.append((graph, stream))
    for _ in range(3):
        for b in blocks:
            b.C.fill_(CANARY), b.Y.fill_(CANARY), b.H.fill_(CANARY)
        torch.cuda.synchronize()
        for graph, stream in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b.C, first.C) and torch.equal(b.H, first.H) for b in blocks)
