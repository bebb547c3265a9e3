"""GPU tests of the router, the experts' lists and the experts' products against
their definitions in 64 bits (i4_reference)."""
import pytest
import torch

import i4_reference as ref
from parity import requires_gpu
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]

BF = torch.bfloat16
TYPES = {"fp32": torch.float32, "bf16": BF, "fp16": torch.float16}
CANARY = 768.0  # a BF16 value


# ------------------------------------------------------------ the router
def route(x, bias, top_k, ld=None, **how):
    T, E = x.shape
    wide = torch.full((T, ld or E), 1e4, dtype=x.dtype)
    wide[:, :E] = x
    ids = torch.full((T + 1, top_k), 77, dtype=torch.int32, device="cuda")
    weights = torch.full((T + 1, top_k), CANARY, device="cuda")
    wqd.moe_route(wide.cuda(), None if bias is None else bias.cuda(), ids, weights, T, E, top_k, row_stride=ld, **how)
    ids, weights = ids.cpu(), weights.cpu()
    assert bool((ids[T:] == 77).all() and (weights[T:] == CANARY).all())
    return ids[:T], weights[:T]


def check_route(x, bias, top_k, ld=None, **how):
    how = dict(scoring="softmax", groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0) | how
    ids, weights = route(x, bias, top_k, ld, **how)
    want, w = ref.route(x, bias, top_k, how["scoring"], how["groups"], how["top_groups"], how["group_top"], how["renormalize"], how["scale"])
    assert torch.equal(ids, want)
    # 64-bit arithmetic (2^-40 leaves room for exp and the sums), rounded to fp32 once
    assert bool(((weights.double() - w).abs() <= (2.0 ** -24 + 2.0 ** -40) * w.abs() + 2.0 ** -149).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("T,E,top_k,groups,top_groups", [
    (1, 1, 1, 1, 1), (3, 8, 2, 1, 1), (5, 64, 8, 1, 1), (6, 65, 7, 5, 2), (2, 128, 32, 4, 2), (7, 160, 6, 8, 3), (1, 256, 8, 8, 4), (9, 256, 8, 1, 1),
    (4, 384, 8, 1, 1), (3, 512, 10, 64, 9), (3, 1000, 5, 10, 10), (2, 1024, 32, 32, 1), (33, 60, 4, 1, 1)])
def test_route(T, E, top_k, groups, top_groups, t, scoring):
    g = ref.generator(T, E, top_k)
    x = (2.0 * torch.randn(T, E, generator=g)).to(TYPES[t])
    bias = 0.1 * torch.randn(E, generator=g)
    for b in (None, bias):
        for group_top in ((1, 2) if groups > 1 else (1,)):
            check_route(x, b, top_k, ld=E + T % 3, scoring=scoring, groups=groups, top_groups=top_groups, group_top=group_top,
                        renormalize=bool(T % 2), scale=1.0 if T % 2 else 2.5)


@pytest.mark.parametrize("bias", [False, True])
def test_route_ties(bias):
    """Few different values: the lowest index wins, of experts and of groups."""
    g = ref.generator(11)
    x = torch.randint(-1, 2, (40, 96), generator=g).to(BF)
    b = torch.randint(0, 2, (96,), generator=g).float() / 4 if bias else None
    for groups, top_groups, group_top in ((1, 1, 1), (6, 2, 1), (6, 3, 2), (12, 5, 2)):
        for scoring in ("softmax", "sigmoid"):
            check_route(x, b, 8, groups=groups, top_groups=top_groups, group_top=group_top, scoring=scoring)


def test_route_masked_experts():
    """Minus infinity and NaN take an expert out; rows may run out of experts; infinity is the largest value."""
    g = ref.generator(12)
    x = torch.randn(12, 40, generator=g)
    x[0] = -torch.inf
    x[1] = float("nan")
    x[2, 3:] = -torch.inf
    x[3, ::2] = float("nan")
    x[4, 7] = x[4, 30] = torch.inf
    x[5] = torch.inf
    x[6] = -3e38
    x[6, 4] = 3e38
    x[7] = torch.finfo(torch.float32).min
    x[8, :5], x[8, 5:] = -200.0, -torch.inf
    x[9] = -1000.0  # sigmoid: every score is 0
    bias = torch.zeros(40)
    bias[5], bias[6], bias[7] = -torch.inf, float("nan"), 1e30
    for b in (None, bias):
        for scoring in ("softmax", "sigmoid"):
            for groups in (1, 4):
                check_route(x, b, 6, scoring=scoring, groups=groups, top_groups=max(1, groups // 2), group_top=2, renormalize=True)
                check_route(x, b, 6, scoring=scoring, groups=groups, top_groups=max(1, groups // 2), group_top=1, renormalize=False)


# ------------------------------------------------------------ the lists
@pytest.mark.parametrize("T,top_k,E", [(0, 2, 5), (1, 1, 1), (1, 8, 64), (7, 3, 10), (100, 8, 64), (1000, 8, 256), (1025, 5, 33), (5000, 2, 1024)])
def test_lists(T, top_k, E):
    ids = torch.randint(-1, E + 1, (T, top_k), generator=ref.generator(T, E), dtype=torch.int32)  # -1 and E: none of these
    if T > 2:
        ids[1] = E // 2  # one expert in every slot
        ids[2] = -(1 << 31)
    order = torch.full((T * top_k + 1,), 77, dtype=torch.int32, device="cuda")
    offsets = torch.full((E + 2,), 77, dtype=torch.int32, device="cuda")
    wqd.moe_lists(ids.cuda(), order, offsets, T, top_k, E)
    want, at = ref.lists(ids, E)
    assert torch.equal(order.cpu()[:-1], want) and torch.equal(offsets.cpu()[:-1], at)
    assert int(order[-1]) == 77 and int(offsets[-1]) == 77


# ------------------------------------------------------------ the experts' products
def choice(g, T, E, top_k, absent=0.15):
    ids = torch.stack([torch.randperm(E, generator=g)[:top_k] for _ in range(T)]).to(torch.int32)
    ids[torch.rand(T, top_k, generator=g) < absent] = -1
    if T > 3:
        ids[2] = -1  # a padded token
        ids[3, 0] = E  # another GPU's expert
    return ids


def lists_of(ids, E):
    order, offsets = ref.lists(ids, E)
    return order.cuda(), offsets.cuda()


EXPERTS = [(1, 8, 2, 48, 256), (1, 64, 8, 100, 1024), (2, 4, 4, 17, 128), (5, 16, 3, 130, 1152), (33, 8, 2, 65, 640), (64, 4, 2, 257, 384),
           (100, 70, 5, 33, 256), (300, 3, 2, 300, 512), (700, 2, 1, 129, 256)]


def pair_products(rows, w, ids, E):
    """Sums of each pair's row with its expert's matrix and how far they may be off; zeros where there is none."""
    flat = ids.flatten().long()
    here = (flat >= 0) & (flat < E)
    values, size = w.values(), w.size()
    y, err = torch.zeros(len(flat), w.N, dtype=torch.float64), torch.zeros(len(flat), w.N, dtype=torch.float64)
    for e in range(E):
        at = here & (flat == e)
        y[at], err[at] = rows[at].double() @ values[e].T, ref.sum_error(rows[at].double().abs() @ size[e].T, w.K)
    return y, err, here


@pytest.mark.parametrize("group,zeros,scale", [(128, False, "fp16"), (64, True, "bf16"), (32, True, "fp16")])
@pytest.mark.parametrize("T,E,top_k,N,K", EXPERTS)
def test_experts_gated(T, E, top_k, N, K, group, zeros, scale):
    g = ref.generator(21, T, E, N, K)
    ids = choice(g, T, E, top_k)
    wg, wu = ref.Weights(g, E, N, K, group, zeros, scale), ref.Weights(g, E, N, K, group, zeros, scale)
    lda = K + 8 * (T % 2)
    a = torch.randn(T, K, generator=g).to(BF)
    A = torch.full((T, lda), float("nan"), dtype=BF)
    A[:, :K] = a
    rows = a.repeat_interleave(top_k, 0)
    gate, eg, here = pair_products(rows, wg, ids, E)
    up, eu, _ = pair_products(rows, wu, ids, E)
    want, err = ref.gated(gate, up, eg, eu)
    for order, offsets in ((None, None), lists_of(ids, E)):
        H = torch.full((T * top_k + 1, N), CANARY, dtype=BF, device="cuda")
        wqd.i4a16_experts_gated(A.cuda(), ids.cuda(), order, offsets, *wg.operands(), *wu.operands(), H, T, top_k, E, N, K, group, a_row_stride=lda)
        got = H.cpu().double()
        assert bool((got[-1] == CANARY).all() and (got[:-1][~here] == CANARY).all())
        assert bool(((got[:-1] - want).abs() <= ref.stored(want, err))[here].all())


@pytest.mark.parametrize("group,zeros,scale", [(128, False, "fp16"), (64, True, "bf16"), (32, True, "fp16")])
@pytest.mark.parametrize("T,E,top_k,N,K", EXPERTS)
def test_experts_down(T, E, top_k, N, K, group, zeros, scale):
    g = ref.generator(22, T, E, N, K)
    ids = choice(g, T, E, top_k)
    w = ref.Weights(g, E, N, K, group, zeros, scale)
    h = torch.randn(T * top_k, K, generator=g).to(BF)
    weights = torch.rand(T, top_k, generator=g)
    y, err, here = pair_products(h, w, ids, E)
    h[~here] = float("nan")  # rows of pairs without an expert are not read into anything
    s = (weights.double().flatten() * here).unsqueeze(1)
    want = (s * y).view(T, top_k, N).sum(1)
    # weighting a row and adding it: two roundings for each slot
    err = (s * err + (top_k + 2) * 2.0 ** -23 * s * (y.abs() + err)).view(T, top_k, N).sum(1)
    ldc = N + T % 3
    for order, offsets in ((None, None), lists_of(ids, E)):
        C = torch.full((T + 1, ldc), CANARY, dtype=BF, device="cuda")
        Y = None if order is None else torch.full((T * top_k, N), float("nan"), device="cuda")
        wqd.i4a16_experts_down(h.cuda(), ids.cuda(), weights.cuda(), order, offsets, *w.operands(), Y, C, T, top_k, E, N, K, group, c_row_stride=ldc)
        got = C.cpu().double()
        assert bool((got[T:] == CANARY).all() and (got[:T, N:] == CANARY).all())
        assert bool(((got[:T, :N] - want).abs() <= ref.stored(want, err)).all())
        if T > 3:
            assert bool((got[2, :N] == 0).all())


def test_the_same_expert_twice():
    """A token may name an expert in two slots."""
    T, E, top_k, N, K = 3, 4, 3, 40, 256
    g = ref.generator(23)
    w = ref.Weights(g, E, N, K, 64, False, "fp16", exact=True)
    ids = torch.tensor([[1, 1, 1], [0, 2, 0], [3, 3, 2]], dtype=torch.int32)
    h = torch.randint(-4, 5, (T * top_k, K), generator=g).to(BF)
    weights = torch.tensor([[0.5, 0.25, 0.25], [1.0, 0.5, 0.5], [0.25, 0.25, 0.5]])
    y = torch.stack([h[p].double() @ w.values()[ids.flatten()[p]].T for p in range(T * top_k)])
    want = (weights.double().flatten().unsqueeze(1) * y).view(T, top_k, N).sum(1).to(BF)
    for order, offsets in ((None, None), lists_of(ids, E)):
        C = torch.zeros(T, N, dtype=BF, device="cuda")
        Y = torch.empty(T * top_k, N, device="cuda")
        wqd.i4a16_experts_down(h.cuda(), ids.cuda(), weights.cuda(), order, offsets, *w.operands(), Y, C, T, top_k, E, N, K, 64)
        assert torch.equal(C.cpu(), want)


def test_lists_that_point_elsewhere_stay_inside():
    """Lists that are not moe_lists' of any ids are read and written within the operands all the same."""
    T, E, top_k, N, K = 6, 5, 2, 32, 128
    g = ref.generator(24)
    w = ref.Weights(g, E, N, K, 128, False, "fp16")
    ids = choice(g, T, E, top_k).cuda()
    A = torch.randn(T, K, generator=g).to(BF).cuda()
    for offsets in ([0, 100, 3, -5, 7, 1 << 30], [12, 12, 12, 12, 12, 12], [-1] * 6):
        for order in ([1 << 30] * 12, [-1] * 12, [11] * 12):
            H = torch.full((T * top_k + 64, N), CANARY, dtype=BF, device="cuda")
            wqd.i4a16_experts_gated(A, ids, torch.tensor(order, dtype=torch.int32).cuda(), torch.tensor(offsets, dtype=torch.int32).cuda(),
                                    *w.operands(), *w.operands(), H, T, top_k, E, N, K, 128)
            assert bool((H[T * top_k:] == CANARY).all())


# ------------------------------------------------------------ together, as they are used
@pytest.mark.parametrize("T", [1, 3, 40, 150])
def test_routed_block(T):
    """Router, lists, gated and last products: eagerly, and captured and replayed on new tokens; each step against its
    definition on what went into it."""
    E, top_k, D, F, group = 16, 4, 256, 384, 64
    g = ref.generator(31, T)
    wg, wu, wd = (ref.Weights(g, E, *n, group, z, "bf16") for n, z in (((F, D), True), ((F, D), True), ((D, F), False)))
    G, U, W = wg.operands(), wu.operands(), wd.operands()
    bias = (0.02 * torch.randn(E, generator=g)).cuda()
    x, logits = torch.empty(T, D, dtype=BF, device="cuda"), torch.empty(T, E, device="cuda")
    ids, weights = torch.empty(T, top_k, dtype=torch.int32, device="cuda"), torch.empty(T, top_k, device="cuda")
    order, offsets = torch.empty(T * top_k, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    H, Y, C = torch.empty(T * top_k, F, dtype=BF, device="cuda"), torch.empty(T * top_k, D, device="cuda"), torch.empty(T, D, dtype=BF, device="cuda")
    how = dict(scoring="sigmoid", groups=4, top_groups=2, group_top=2, renormalize=True, scale=1.5)

    def block(lists):
        wqd.moe_route(logits, bias, ids, weights, T, E, top_k, **how)
        o = (None, None)
        if lists:
            wqd.moe_lists(ids, order, offsets, T, top_k, E)
            o = (order, offsets)
        wqd.i4a16_experts_gated(x, ids, *o, *G, *U, H, T, top_k, E, F, D, group)
        wqd.i4a16_experts_down(H, ids, weights, *o, *W, Y if lists else None, C, T, top_k, E, D, F, group)

    def fresh():
        x.copy_(torch.randn(T, D, generator=g).to(BF))
        logits.copy_(torch.randn(T, E, generator=g))

    for lists in (False, True):
        fresh()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            block(lists)
        torch.cuda.synchronize()
        want, w = ref.route(logits.cpu(), bias.cpu(), top_k, *how.values())
        assert torch.equal(ids.cpu(), want)
        a = x.cpu().repeat_interleave(top_k, 0)
        sums = [pair_products(a, m, ids.cpu(), E)[:2] for m in (wg, wu)]
        y, err = ref.gated(sums[0][0], sums[1][0], sums[0][1], sums[1][1])
        assert bool(((H.cpu().double() - y).abs() <= ref.stored(y, err)).all())
        y, err, _ = pair_products(H.cpu(), wd, ids.cpu(), E)
        s = weights.cpu().double().flatten().unsqueeze(1)
        y, err = ((v.view(T, top_k, D).sum(1)) for v in (s * y, s * err + (top_k + 2) * 2.0 ** -23 * s * (y.abs() + err)))
        assert bool(((C.cpu().double() - y).abs() <= ref.stored(y, err)).all())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            block(lists)
        for _ in range(3):
            fresh()
            C.fill_(CANARY), H.fill_(CANARY), Y.fill_(CANARY)
            graph.replay()
            torch.cuda.synchronize()
            got = ids.clone(), weights.clone(), H.clone(), C.clone()
            block(lists)
            assert all(torch.equal(p, q) for p, q in zip(got, (ids, weights, H, C)))
