"""The 4-bit integer operators as they are measured: products with group-scaled weights, and a routed feed-forward block.

  product  i4a16_gemm: BF16 activations times 4-bit integer weights with a scale (and a zero point) per 32, 64 or 128 k
  gated    i4a16_gated: silu(A Wg^T) * (A Wu^T) over two such matrices
  route    moe_route and moe_lists: a router's scores to the experts and weights of each token, and to each expert's tokens
  experts  i4a16_experts_gated: the gated products of every token with its experts' matrices
  down     i4a16_experts_down: the experts' last products and their weighted sum for each token

Dense sizes are those of the benchmark (5120 x 5120 projections, 17408 x 5120 feed-forward matrices); experts are of
generic sizes. From one token (a decode step) to thousands (a prompt).
"""
import torch

own = False

DEVICE = "cuda"

SCALES = {"fp16": torch.float16, "bf16": torch.bfloat16}
LOGITS = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
MOST = 4096 * 5120 * 5120  # multiply-adds of a drawn case, at most


def listed():
    return [
        # one token through an attention projection
        {"name": "product 1x5120x5120", "kind": "product", "M": 1, "N": 5120, "K": 5120, "group": 128, "zeros": False, "scale": "fp16", "pad": 0},
        # sixteen sequences' tokens through the down projection, zero points
        {"name": "product 16x5120x17408", "kind": "product", "M": 16, "N": 5120, "K": 17408, "group": 64, "zeros": True, "scale": "bf16", "pad": 0},
        # a batch of odd size over an odd number of outputs, small groups, into a slice of a wider buffer
        {"name": "product 45x5119x5120", "kind": "product", "M": 45, "N": 5119, "K": 5120, "group": 32, "zeros": True, "scale": "fp16", "pad": 3},
        # a long prompt through an attention projection
        {"name": "product 4096x5120x5120", "kind": "product", "M": 4096, "N": 5120, "K": 5120, "group": 128, "zeros": False, "scale": "fp16", "pad": 0},
        # one token through the gate and up projections
        {"name": "gated 1x17408x5120", "kind": "gated", "M": 1, "N": 17408, "K": 5120, "group": 128, "zeros": False, "scale": "fp16", "pad": 0},
        # a prompt of five hundred tokens through the gate and up projections, zero points
        {"name": "gated 500x17408x5120", "kind": "gated", "M": 500, "N": 17408, "K": 5120, "group": 128, "zeros": True, "scale": "fp16", "pad": 0},
        # one token's router: sigmoid scores, a bias for balance, the best four of eight groups
        {"name": "route 1 of 256", "kind": "route", "T": 1, "E": 256, "top_k": 8, "logits": "fp32", "scoring": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renormalize": True},
        # a long prompt's router: softmax of 16-bit scores, which are often equal
        {"name": "route 4096 of 64", "kind": "route", "T": 4096, "E": 64, "top_k": 8, "logits": "bf16", "scoring": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renormalize": True},
        # one token through the gate and up matrices of its experts
        {"name": "experts 1 token", "kind": "experts", "T": 1, "E": 64, "top_k": 8, "N": 1024, "K": 2048, "group": 128, "zeros": False, "scale": "fp16", "lists": False, "absent": 0.0},
        # a long prompt through its experts
        {"name": "experts 4096 tokens", "kind": "experts", "T": 4096, "E": 64, "top_k": 8, "N": 1024, "K": 2048, "group": 128, "zeros": False, "scale": "fp16", "lists": True, "absent": 0.0},
        # a decode step of 33 sequences: the experts' last products, zero points, one slot in eight on another GPU
        {"name": "down 33 tokens", "kind": "down", "T": 33, "E": 64, "top_k": 8, "N": 2048, "K": 1024, "group": 64, "zeros": True, "scale": "bf16", "lists": True, "absent": 0.125},
        # a prompt of two thousand tokens
        {"name": "down 2048 tokens", "kind": "down", "T": 2048, "E": 64, "top_k": 8, "N": 2048, "K": 1024, "group": 128, "zeros": False, "scale": "fp16", "lists": True, "absent": 0.0},
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["product", "product", "gated", "route", "experts", "experts", "down", "down"])
    if kind == "route":
        g = rng.choice([1, 1, 2, 4, 8])
        e = g * _between(rng, 8, 512 // g)
        top_groups = rng.randint(1, g)
        return {"kind": kind, "T": _between(rng, 1, 8192), "E": e, "top_k": rng.randint(1, min(8, top_groups * (e // g))),
                "logits": rng.choice(list(LOGITS)), "scoring": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "groups": g, "top_groups": top_groups, "group_top": rng.choice([1, 2]), "renormalize": rng.random() < 0.7}
    weights = {"group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5, "scale": rng.choice(list(SCALES))}
    if kind in ("product", "gated"):
        c = {"kind": kind, "M": _between(rng, 1, 4096), "N": _between(rng, 16, 17408), "K": 128 * _between(rng, 1, 136),
             "pad": rng.choice([0, 0, 1, 8]), **weights}
        c["M"] = max(1, min(c["M"], MOST // (2 if kind == "gated" else 1) // (c["N"] * c["K"])))
        return c
    t, e = _between(rng, 1, 4096), _between(rng, 4, 128)
    c = {"kind": kind, "T": t, "E": e, "top_k": rng.randint(1, min(8, e)), "N": _between(rng, 16, 2048), "K": 128 * _between(rng, 1, 16),
         "lists": t > 4 or rng.random() < 0.3, "absent": rng.choice([0.0, 0.0, 0.3]), **weights}
    c["T"] = max(1, min(c["T"], MOST // (2 if kind == "experts" else 1) // (c["top_k"] * c["N"] * c["K"])))
    return c


# ------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _rows(g, m, k):
    """Activations: normal values, a few channels several times larger, as the residual stream of a model has them."""
    gain = torch.where(torch.rand(k, generator=g, device=DEVICE) < 0.01, 8.0, 1.0)
    return (_normal(g, m, k) * gain).to(torch.bfloat16)


def _laid_out(codes):
    """Codes as the library takes them: tiles of 16 rows x 128 k, 1024 bytes each, row tile by row tile. Byte 256 g +
    16 n + 4 j + b of a tile holds two codes of row n, k = 32 j + 8 g + (0, 2, 4, 6, 1, 3, 5, 7)[2 b] and [2 b + 1], the
    first in the low nibble. Rows past the last one hold zeros."""
    e, n, k = codes.shape
    q = torch.nn.functional.pad(codes, (0, 0, 0, -n % 16)).view(e, -1, 16, k // 128, 4, 4, 4, 2).permute(0, 1, 3, 5, 2, 4, 7, 6)
    q = q.reshape(e, -1, 4, 2)  # pairs (0, 2), (4, 6), (1, 3), (5, 7) of each 8
    return (q[..., 0] | q[..., 1] << 4).view(e, -1, k // 2)


def _weights(g, e, n, k, c):
    """Codes [e, n, k], scales and zero points [e, n, k / group] (None: 8 everywhere), and the same with the codes laid out."""
    z = torch.randint(5, 12, (e, n, k // c["group"]), generator=g, device=DEVICE, dtype=torch.uint8) if c["zeros"] else None
    q = (_normal(g, e, n, k // c["group"], c["group"]) * 2.5).round_()
    codes = q.add_(8.0 if z is None else z.unsqueeze(-1)).clamp_(0, 15).flatten(2).to(torch.uint8)
    s = ((0.5 + torch.rand(e, n, k // c["group"], generator=g, device=DEVICE)) * (0.4 * k ** -0.5)).to(SCALES[c["scale"]])
    return (codes, s, z), (_laid_out(codes), s, z)


def _lists(ids, e):
    """order: the pairs (token * top_k + slot) with an expert, expert by expert, ascending; offsets [e + 1]: where each
    expert's begin. Absent pairs follow the last one as -1."""
    flat = ids.flatten().to(torch.int64)
    key = torch.where((flat < 0) | (flat >= e), e, flat)
    order = torch.sort(key, stable=True).indices
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device=ids.device), torch.bincount(key, minlength=e + 1)[:e].cumsum(0)))
    order = torch.where(torch.arange(order.numel(), device=ids.device) < offsets[-1], order, -1)
    return order.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    kind, st = case["kind"], {"case": case}
    if kind == "route":
        t, e, k = case["T"], case["E"], case["top_k"]
        st.update(logits=(_normal(g, t, e) + 0.5 * _normal(g, e)).to(LOGITS[case["logits"]]),
                  bias=0.05 * _normal(g, e) if case["bias"] else None,
                  ids=torch.empty(t, k, dtype=torch.int32, device=DEVICE), weights=torch.empty(t, k, device=DEVICE),
                  order=torch.empty(t * k, dtype=torch.int32, device=DEVICE), offsets=torch.empty(e + 1, dtype=torch.int32, device=DEVICE))
        return st
    n, k = case["N"], case["K"]
    if kind in ("product", "gated"):
        st["A"] = _rows(g, case["M"], k)
        for name in ("W",) if kind == "product" else ("WG", "WU"):
            st[name], st[name + " laid"] = _weights(g, 1, n, k, case)
        st["C"] = torch.zeros(case["M"], n + case["pad"], dtype=torch.bfloat16, device=DEVICE)
        return st
    t, e, top = case["T"], case["E"], case["top_k"]
    score = _normal(g, t, e) + 0.5 * _normal(g, e)
    chosen = torch.topk(score, top)
    absent = torch.rand(t, top, generator=g, device=DEVICE) < case["absent"]
    st["ids"] = torch.where(absent, -1, chosen.indices).to(torch.int32)
    st["weights"] = torch.softmax(chosen.values, -1)
    st["order"], st["offsets"] = _lists(st["ids"], e)
    st["most"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())  # tokens of the busiest expert
    for name in ("WG", "WU") if kind == "experts" else ("W",):
        st[name], st[name + " laid"] = _weights(g, e, n, k, case)
    if kind == "experts":
        st["A"] = _rows(g, t, k)
        st["H"] = torch.zeros(t * top, n, dtype=torch.bfloat16, device=DEVICE)
    else:
        st["H"] = (0.3 * _rows(g, t * top, k).float()).to(torch.bfloat16)
        st["Y"] = torch.empty(t * top, n, device=DEVICE) if case["lists"] else None
        st["C"] = torch.zeros(t, n, dtype=torch.bfloat16, device=DEVICE)
    return st


# ------------------------------------------------------------------ the plain forms
def _dequantize(w, at=slice(None)):
    codes, s, z = w
    zero = 8.0 if z is None else z[at].unsqueeze(-1).float()
    q = codes[at].unflatten(-1, (s.shape[-1], -1)).float()
    return ((q - zero) * s[at].unsqueeze(-1).float()).flatten(-2)


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _grouped(rows, state, names):
    """Products of every pair's row with its expert's matrices, [pairs, N] each; zeros for absent pairs."""
    c, ids = state["case"], state["ids"].flatten().to(torch.int64)
    here = ids >= 0
    if ids.numel() <= c["E"]:  # few pairs: each with a copy of its expert's matrix
        return [(_dequantize(state[n], ids.clamp(min=0)) @ rows.unsqueeze(-1)).squeeze(-1) * here.unsqueeze(-1) for n in names]
    order, offsets = state["order"].to(torch.int64), state["offsets"].to(torch.int64)
    pairs = order.clamp(min=0)
    expert = torch.where(order >= 0, ids[pairs], c["E"])
    place = torch.where(order >= 0, torch.arange(order.numel(), device=ids.device) - offsets[expert.clamp(max=c["E"] - 1)], 0)
    wide = torch.zeros(c["E"] + 1, max(1, state["most"]), rows.shape[1], device=ids.device)
    wide[expert, place] = rows[pairs]
    full = [torch.bmm(wide[:-1], _dequantize(state[n]).transpose(1, 2))[expert.clamp(max=c["E"] - 1), place] for n in names]
    to = torch.where(order >= 0, order, ids.numel())
    return [torch.zeros(ids.numel() + 1, c["N"], device=ids.device).index_copy(0, to, y)[:-1] for y in full]


def _scores(x, scoring):
    """Scores of logits in 64 bits."""
    if scoring == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _route(state):
    c = state["case"]
    x = state["logits"].double()
    score = _scores(x, c["scoring"])
    key = score if state["bias"] is None else score + state["bias"].double()
    if c["groups"] > 1:
        best = torch.sort(key.unflatten(-1, (c["groups"], -1)), descending=True).values[..., : c["group_top"]].sum(-1)
        chosen = torch.sort(best, stable=True, descending=True).indices[:, : c["top_groups"]]
        inside = torch.zeros_like(best, dtype=torch.bool).scatter(1, chosen, True)
        key = torch.where(inside.repeat_interleave(c["E"] // c["groups"], 1), key, -torch.inf)
    ids = torch.sort(key, stable=True, descending=True).indices[:, : c["top_k"]]
    w = score.gather(1, ids)
    if c["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    ids = ids.to(torch.int32)
    order, offsets = _lists(ids, c["E"])
    return {"ids": ids, "weights": w.float(), "order": order, "offsets": offsets}


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    if c["kind"] == "route":
        return _route(state)
    if c["kind"] == "product":
        return (state["A"].float() @ _dequantize(state["W"])[0].T).to(torch.bfloat16)
    if c["kind"] == "gated":
        a = state["A"].float()
        return (_silu(a @ _dequantize(state["WG"])[0].T) * (a @ _dequantize(state["WU"])[0].T)).to(torch.bfloat16)
    if c["kind"] == "experts":
        gate, up = _grouped(state["A"].float().repeat_interleave(c["top_k"], 0), state, ("WG", "WU"))
        return (_silu(gate) * up).to(torch.bfloat16)
    y = _grouped(state["H"].float(), state, ("W",))[0]
    return (y.unflatten(0, (c["T"], -1)) * state["weights"].unsqueeze(-1)).sum(1).to(torch.bfloat16)


# ------------------------------------------------------------------ the library's calls
def _run_own(st, c):
    from weight_quantized_decode_block_amd import wqd
    if c["kind"] == "route":
        wqd.moe_route(st["logits"], st["bias"], st["ids"], st["weights"], c["T"], c["E"], c["top_k"], scoring=c["scoring"],
                      groups=c["groups"], top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renormalize"])
        wqd.moe_lists(st["ids"], st["order"], st["offsets"], c["T"], c["top_k"], c["E"])
        return {"ids": st["ids"], "weights": st["weights"], "order": st["order"], "offsets": st["offsets"]}
    n, k, group = c["N"], c["K"], c["group"]
    if c["kind"] == "product":
        wqd.i4a16_gemm(st["A"], *st["W laid"], st["C"], c["M"], n, k, group, c_row_stride=n + c["pad"])
        return st["C"][:, :n]
    if c["kind"] == "gated":
        wqd.i4a16_gated(st["A"], *st["WG laid"], *st["WU laid"], st["C"], c["M"], n, k, group, c_row_stride=n + c["pad"])
        return st["C"][:, :n]
    order, offsets = (st["order"], st["offsets"]) if c["lists"] else (None, None)
    if c["kind"] == "experts":
        wqd.i4a16_experts_gated(st["A"], st["ids"], order, offsets, *st["WG laid"], *st["WU laid"], st["H"], c["T"], c["top_k"],
                                c["E"], n, k, group)
        return st["H"]
    wqd.i4a16_experts_down(st["H"], st["ids"], st["weights"], order, offsets, *st["W laid"], st["Y"], st["C"], c["T"], c["top_k"],
                           c["E"], n, k, group)
    return st["C"]


# ------------------------------------------------------------------ what a pass cannot do without
def _here(case):
    """Experts with a token, at most, and pairs with an expert, about."""
    pairs = case["T"] * case["top_k"] * (1.0 - case["absent"])
    return min(case["E"], pairs), pairs


def work(case):
    kind = case["kind"]
    if kind == "route":
        t, e, k = case["T"], case["E"], case["top_k"]
        return {"bytes": t * e * LOGITS[case["logits"]].itemsize + (4 * e if case["bias"] else 0) + 12 * t * k + 4 * e + 4, "flops": 8 * t * e}
    n, k = case["N"], case["K"]
    matrix = n * k // 2 + n * k // case["group"] * (3 if case["zeros"] else 2)
    if kind in ("product", "gated"):
        m, count = case["M"], 1 if kind == "product" else 2
        return {"bytes": count * matrix + 2 * m * k + 2 * m * n, "flops": 2 * count * m * n * k}
    busy, pairs = _here(case)
    if kind == "experts":
        return {"bytes": int(2 * busy * matrix + 2 * case["T"] * k + 2 * pairs * n), "flops": int(4 * pairs * n * k)}
    return {"bytes": int(busy * matrix + 2 * pairs * k + 2 * case["T"] * n + 8 * pairs), "flops": int(2 * pairs * n * k)}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_matrix(w, e):
    codes, s, z = w
    group = codes.shape[2] // s.shape[2]
    q = codes[e].double()
    q -= 8.0 if z is None else torch.repeat_interleave(z[e].double(), group, dim=1)
    q *= torch.repeat_interleave(s[e].double(), group, dim=1)
    return q


def _exact_route(st, c):
    """Weights alone: expert by expert of a token, by comparing each score with all others."""
    x = st["logits"].double()
    score = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, 1)
    key = score + (0.0 if st["bias"] is None else st["bias"].double())
    t, e, g = c["T"], c["E"], c["groups"]
    if g > 1:
        best = torch.topk(key.reshape(t, g, e // g), c["group_top"], dim=2).values.sum(2)
        index = torch.arange(g, device=x.device)
        ahead = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & (index[None, None, :] < index[None, :, None]))
        out = ahead.sum(2) >= c["top_groups"]
        key = key.reshape(t, g, e // g).masked_fill(out.unsqueeze(2), -torch.inf).reshape(t, e)
    index = torch.arange(e, device=x.device)
    rank = torch.empty(t, e, dtype=torch.int64, device=x.device)
    for j in range(e):
        ahead = (key > key[:, j : j + 1]) | ((key == key[:, j : j + 1]) & (index < j))
        rank[:, j] = ahead.sum(1)
    place = torch.where(rank < c["top_k"], rank, c["top_k"])
    w = torch.zeros(t, c["top_k"] + 1, dtype=torch.float64, device=x.device).scatter_(1, place, score)[:, : c["top_k"]]
    return w / w.sum(1, keepdim=True) if c["renormalize"] else w


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "route":
        return {"ids": None, "weights": _exact_route(st, case), "order": None, "offsets": None}
    if kind == "product":
        return st["A"].double().matmul(_exact_matrix(st["W"], 0).t())
    if kind == "gated":
        a = st["A"].double()
        gate = a.matmul(_exact_matrix(st["WG"], 0).t())
        return gate * torch.sigmoid(gate) * a.matmul(_exact_matrix(st["WU"], 0).t())
    pairs = case["T"] * case["top_k"]
    flat = st["ids"].flatten()
    out = torch.zeros(pairs, case["N"], dtype=torch.float64, device=DEVICE)
    for e in range(case["E"]):
        at = torch.nonzero(flat == e).flatten()
        if not at.numel():
            continue
        if kind == "experts":
            a = st["A"][torch.div(at, case["top_k"], rounding_mode="floor")].double()
            gate = a.matmul(_exact_matrix(st["WG"], e).t())
            out[at] = gate * torch.sigmoid(gate) * a.matmul(_exact_matrix(st["WU"], e).t())
        else:
            out[at] = st["H"][at].double().matmul(_exact_matrix(st["W"], e).t()) * st["weights"].flatten()[at].double().unsqueeze(1)
    return out if kind == "experts" else out.reshape(case["T"], case["top_k"], case["N"]).sum(1)
