"""GPU tests of the products with 4-bit integer weights against their definition
in 64 bits (i4_reference, which derives the tolerances)."""
import pytest
import torch

import i4_reference as ref
from parity import requires_gpu
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]

BF = torch.bfloat16
CANARY = 768.0  # a BF16 value


def rows(g, M, K, lda=None, exact=False):
    """BF16 activations on the CPU and, in rows lda apart with NaN between, on the GPU."""
    a = torch.randint(-8, 9, (M, K), generator=g).to(BF) if exact else torch.randn(M, K, generator=g).to(BF)
    wide = torch.full((M, lda or K), float("nan"), dtype=BF)
    wide[:, :K] = a
    return a, wide.cuda()


def out(M, N, ldc):
    return torch.full((M + 1, ldc), CANARY, dtype=BF, device="cuda")


def untouched(C, M, N):
    C = C.cpu().float()
    return bool((C[M:] == CANARY).all() and (C[:M, N:] == CANARY).all())


@pytest.mark.parametrize("scale,zeros", [("fp16", True), ("bf16", False)])
@pytest.mark.parametrize("E,N,K,group", [(1, 1, 128, 128), (1, 16, 256, 64), (3, 17, 384, 32), (2, 100, 1152, 64), (5, 33, 128, 128)])
def test_pack(E, N, K, group, scale, zeros):
    w = ref.Weights(ref.generator(E, N, K), E, N, K, group, zeros, scale)
    n = E * wqd.i4_packed_rows(N) * K
    W = torch.full((n // 2 + 32,), 0xA5, dtype=torch.uint8, device="cuda")
    S = torch.full((n // group + 32,), CANARY, dtype=w.s.dtype, device="cuda")
    Z = torch.full((n // group + 32,), 0xA5, dtype=torch.uint8, device="cuda") if zeros else None
    wqd.i4_pack(ref.rows_of_pairs(w.codes).cuda(), w.s.cuda(), w.z.cuda() if zeros else None, W, S, Z, N, K, group, E)
    for got, want, size, fill in zip((W, S, Z), w.operands("cpu"), (n // 2, n // group, n // group), (0xA5, CANARY, 0xA5)):
        if want is not None:
            assert torch.equal(got[:size].cpu(), want.flatten()) and bool((got[size:] == fill).all())


@pytest.mark.parametrize("scale", ["fp16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (1, 100, 1152), (3, 17, 256), (5, 1, 1152), (8, 33, 2176), (16, 48, 1024), (23, 65, 640),
                                   (40, 130, 512), (130, 257, 256)])
def test_product_exact(M, N, K, group, zeros, scale):
    """Integers times powers of two: every sum is exact in fp32, so the outputs are the rounded exact sums."""
    g = ref.generator(1, M, N, K, group)
    w = ref.Weights(g, 1, N, K, group, zeros, scale, exact=True)
    a, A = rows(g, M, K, exact=True)
    C = out(M, N, N)
    wqd.i4a16_gemm(A, *w.operands(), C, M, N, K, group)
    assert torch.equal(C[:M].cpu(), (a.double() @ w.values()[0].T).to(BF)) and untouched(C, M, N)


SIZES = [(1, 5120, 5120), (2, 333, 17408), (4, 1000, 384), (7, 513, 5120), (11, 512, 4992), (16, 129, 17408), (17, 257, 1024), (32, 640, 2048),
         (33, 100, 5120), (64, 512, 1024), (65, 300, 1152), (200, 777, 640), (513, 384, 1280)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("group,zeros,scale", [(128, False, "fp16"), (64, True, "bf16"), (32, True, "fp16")])
def test_product(M, N, K, group, zeros, scale):
    g = ref.generator(2, M, N, K, group)
    w = ref.Weights(g, 1, N, K, group, zeros, scale)
    lda, ldc = K + 8 * (M % 3), N + M % 4
    a, A = rows(g, M, K, lda)
    C = out(M, N, ldc)
    wqd.i4a16_gemm(A, *w.operands(), C, M, N, K, group, a_row_stride=lda, c_row_stride=ldc)
    want = a.double() @ w.values()[0].T
    bound = ref.stored(want, ref.sum_error(a.double().abs() @ w.size()[0].T, K))
    assert bool(((C[:M, :N].cpu().double() - want).abs() <= bound).all()) and untouched(C, M, N)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("group,zeros,scale", [(128, True, "fp16"), (64, False, "bf16"), (32, False, "fp16")])
def test_gated(M, N, K, group, zeros, scale):
    g = ref.generator(3, M, N, K, group)
    wg, wu = ref.Weights(g, 1, N, K, group, zeros, scale), ref.Weights(g, 1, N, K, group, zeros, scale)
    a, A = rows(g, M, K)
    ldc = N + 8 * (M % 2)
    C = out(M, N, ldc)
    wqd.i4a16_gated(A, *wg.operands(), *wu.operands(), C, M, N, K, group, c_row_stride=ldc)
    sums = [(a.double() @ w.values()[0].T, ref.sum_error(a.double().abs() @ w.size()[0].T, K)) for w in (wg, wu)]
    want, err = ref.gated(sums[0][0], sums[1][0], sums[0][1], sums[1][1])
    assert bool(((C[:M, :N].cpu().double() - want).abs() <= ref.stored(want, err)).all()) and untouched(C, M, N)


def test_every_code_zero_point_and_scale():
    """All codes against all zero points, and scales at the ends of their range (subnormal, largest, zero, negative)."""
    K, group, N = 128, 32, 512
    for name, t in ref.SCALES.items():
        s = torch.tensor([0.0, torch.finfo(t).tiny, torch.finfo(t).tiny / 64, 1.0, -2.0, 60000.0, -0.0, 1 / 3], dtype=torch.float64).to(t)
        w = ref.Weights(ref.generator(4), 1, N, K, group, True, name)
        w.codes = (torch.arange(N * K) % 16).view(1, N, K).to(torch.uint8)
        w.z = (torch.arange(N * K // group) % 256).view(1, N, K // group).to(torch.uint8)
        w.s = s[torch.arange(N * K // group) // 256 % len(s)].view(1, N, K // group)
        for M in (1, 40):
            A = torch.zeros(M, K, dtype=BF)
            for m in range(M):
                A[m, (m * 37) % K] = 1.0 + (m % 5)
            C = out(M, N, N)
            wqd.i4a16_gemm(A.cuda(), *w.operands(), C, M, N, K, group)
            want = A.double() @ w.values()[0].T  # one product each: exact in fp32, rounded once
            assert torch.equal(C[:M].cpu(), want.float().to(BF))


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("M", [1, 9, 70])
def test_rows_that_are_not_finite_stay_alone(M, bad):
    N, K, group = 96, 512, 64
    g = ref.generator(5, M)
    w = ref.Weights(g, 1, N, K, group, True, "fp16")
    a, A = rows(g, M, K)
    C, D = out(M, N, N), out(M, N, N)
    W = w.operands()
    wqd.i4a16_gemm(A, *W, C, M, N, K, group)
    A[M // 2, 200] = bad
    wqd.i4a16_gemm(A, *W, D, M, N, K, group)
    assert not bool(torch.isfinite(D[M // 2]).any())
    keep = torch.arange(M) != M // 2
    assert torch.equal(C[:M].cpu()[keep], D[:M].cpu()[keep])


@pytest.mark.parametrize("M,K", [(1, 1024), (6, 1024), (16, 256), (50, 384)])
def test_graph_replays(M, K):
    """Captured calls give the eager results, replay after replay, also on new inputs in the same places."""
    N, group = 200, 128
    g = ref.generator(6, M, K)
    wg, wu = ref.Weights(g, 1, N, K, group, True, "fp16"), ref.Weights(g, 1, N, K, group, True, "fp16")
    G, U = wg.operands(), wu.operands()
    A = rows(g, M, K)[1]
    C, D = out(M, N, N), out(M, N, N)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        wqd.i4a16_gemm(A, *G, C, M, N, K, group)
        wqd.i4a16_gated(A, *G, *U, D, M, N, K, group)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        wqd.i4a16_gemm(A, *G, C, M, N, K, group)
        wqd.i4a16_gated(A, *G, *U, D, M, N, K, group)
    for _ in range(4):
        A.copy_(rows(g, M, K)[1])
        C.fill_(CANARY), D.fill_(CANARY)
        graph.replay()
        torch.cuda.synchronize()
        got = C.clone(), D.clone()
        wqd.i4a16_gemm(A, *G, C, M, N, K, group)
        wqd.i4a16_gated(A, *G, *U, D, M, N, K, group)
        assert torch.equal(got[0], C) and torch.equal(got[1], D)
