"""The microscaled operators as they are measured: the four kinds of call of the library's 4-bit path.

  round_trip  mx_quantize followed by mx_dequantize: rows to 4 or 8 bits with a scale per 32 values, and back
  norm        add_rmsnorm_mx8: residual addition, root-mean-square norm, rows out in 8 bits with scales
  product     w4a16_gemm, w4a8_gemm, w4a4_gemm: activations in BF16, MXFP8 or MXFP4 times weights in MXFP4
  gated       w4a16_gated, w4a8_gated, w4a4_gated: silu(A Wg^T) * (A Wu^T) over two such weight matrices

Sizes are those of the benchmark (projections of 5120 x 5120 and feed-forward matrices of 17408 x 5120), from one
row (a decode step) to thousands (a prompt).
"""
import torch

own = False

DEVICE = "cuda"

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6
MOST_PRODUCTS = 4096 * 17408 * 5120  # multiply-adds of the largest case


def listed():
    return [
        # a feed-forward matrix brought to 4 bits when a model is loaded, and unpacked again for a look at it
        {"name": "round trip 4 bit 17408x5120", "kind": "round_trip", "fmt": "mxfp4", "type": "bf16", "M": 17408, "K": 5120, "pad": 0},
        # the attention outputs of a few sequences brought to 8 bits before a projection
        {"name": "round trip 8 bit 33x17408", "kind": "round_trip", "fmt": "mxfp8", "type": "fp32", "M": 33, "K": 17408, "pad": 4},
        # one token's residual stream before a projection
        {"name": "norm 1x5120", "kind": "norm", "M": 1, "K": 5120, "residual": True, "plain_rows": False},
        # a prompt's rows before the feed-forward block
        {"name": "norm 4096x5120", "kind": "norm", "M": 4096, "K": 5120, "residual": True, "plain_rows": False},
        # one token through an attention projection
        {"name": "a16 1x5120x5120", "kind": "product", "fmt": "bf16", "M": 1, "N": 5120, "K": 5120, "pad": 0},
        # a prompt of a thousand tokens through the down projection, activations as they come
        {"name": "a16 1000x5120x17408", "kind": "product", "fmt": "bf16", "M": 1000, "N": 5120, "K": 17408, "pad": 0},
        # eight sequences' tokens through the down projection
        {"name": "a8 8x5120x17408", "kind": "product", "fmt": "mxfp8", "M": 8, "N": 5120, "K": 17408, "pad": 0},
        # a long prompt through an up projection
        {"name": "a8 4096x17408x5120", "kind": "product", "fmt": "mxfp8", "M": 4096, "N": 17408, "K": 5120, "pad": 0},
        # a batch of odd size over an odd number of outputs, 4-bit activations, a slice of a wider buffer
        {"name": "a4 77x5119x5120", "kind": "product", "fmt": "mxfp4", "M": 77, "N": 5119, "K": 5120, "pad": 3},
        # a long prompt through an attention projection, 4 bits on both sides
        {"name": "a4 4096x5120x5120", "kind": "product", "fmt": "mxfp4", "M": 4096, "N": 5120, "K": 5120, "pad": 0},
        # one token through the gate and up projections
        {"name": "gated a16 1x17408x5120", "kind": "gated", "fmt": "bf16", "M": 1, "N": 17408, "K": 5120, "pad": 0},
        # a prompt through the gate and up projections, from the norm's 8-bit rows
        {"name": "gated a8 2048x17408x5120", "kind": "gated", "fmt": "mxfp8", "M": 2048, "N": 17408, "K": 5120, "pad": 0},
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["round_trip", "norm", "product", "product", "product", "gated", "gated"])
    if kind == "round_trip":
        return {"kind": kind, "fmt": rng.choice(["mxfp4", "mxfp8"]), "type": rng.choice(["bf16", "fp16", "fp32"]),
                "M": _between(rng, 1, 8192), "K": 32 * _between(rng, 1, 544), "pad": rng.choice([0, 0, 8, 40])}
    if kind == "norm":
        return {"kind": kind, "M": _between(rng, 1, 8192), "K": 32 * _between(rng, 4, 544),
                "residual": rng.random() < 0.7, "plain_rows": rng.random() < 0.4}
    c = {"kind": kind, "fmt": rng.choice(["bf16", "mxfp8", "mxfp4"]), "M": _between(rng, 1, 4096),
         "N": _between(rng, 16, 17408), "K": 128 * _between(rng, 2, 136), "pad": rng.choice([0, 0, 1, 8])}
    most = MOST_PRODUCTS // (2 if kind == "gated" else 1)
    c["M"] = max(1, min(c["M"], most // (c["N"] * c["K"])))
    return c


# ------------------------------------------------------------------ the formats, in elementary operations
def _scale_values(s):
    """E8M0 bytes as fp32: 2^(s - 127); 255 stands for NaN, 0 for the subnormal 2^-127."""
    s = s.to(torch.int32)
    v = (s << 23).view(torch.float32)
    v = torch.where(s == 0, torch.full_like(v, 2.0 ** -127), v)
    return torch.where(s == 255, torch.full_like(v, float("nan")), v)


def _values4(q):
    """E2M1 codes, two a byte (the even element in the low nibble), as fp32."""
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    table = torch.cat((half, -half))
    pairs = torch.stack((table.repeat(16), table.repeat_interleave(16)), 1)
    return pairs[q.to(torch.int32)].flatten(-2)


def _dequantize(q, s, fmt):
    v = _values4(q) if fmt == "mxfp4" else q.view(E4M3).float()
    return (v.unflatten(-1, (-1, 32)) * _scale_values(s).unsqueeze(-1)).flatten(-2)


def _quantize(x, fmt):
    """fp32 rows to element codes and E8M0 scale bytes: the scale is the power of two of the block's largest magnitude
    over that of the format's largest value; elements round to nearest even and saturate; a block that holds an
    infinity or NaN has scale 255 and codes 0."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    good = torch.isfinite(amax)
    power = torch.frexp(torch.where(good, amax, torch.ones_like(amax))).exponent - 1  # floor(log2 amax)
    e = torch.where(amax == 0, torch.full_like(power, -127), power - (2 if fmt == "mxfp4" else 8)).clamp(min=-127)
    s = torch.where(good, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    y = b * ((127 - e).to(torch.int32) << 23).view(torch.float32).unsqueeze(-1)
    y = torch.where(good.unsqueeze(-1), y, torch.zeros_like(y)).flatten(-2)
    if fmt == "mxfp8":
        return y.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8), s
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
            + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    code = code + 8 * torch.signbit(y).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], s


# ------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _rows(g, m, k):
    """Activations: normal values, a few channels several times larger, as the residual stream of a model has them."""
    gain = torch.where(torch.rand(k, generator=g, device=DEVICE) < 0.01, 8.0, 1.0)
    return _normal(g, m, k) * gain


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    kind, m, k = case["kind"], case["M"], case["K"]
    st = {"case": case}
    if kind == "round_trip":
        t, fmt = TYPES[case["type"]], case["fmt"]
        wide = torch.zeros(m, k + case["pad"], dtype=t, device=DEVICE)
        wide[:, :k] = (_rows(g, m, k) * 0.02).to(t)
        st.update(X=wide, Q=torch.empty(m, k // 2 if fmt == "mxfp4" else k, dtype=torch.uint8, device=DEVICE),
                  S=torch.empty(m, k // 32, dtype=torch.uint8, device=DEVICE), Y=torch.empty(m, k, dtype=t, device=DEVICE))
        return st
    if kind == "norm":
        bf = torch.bfloat16
        st.update(X=_normal(g, m, k).to(bf), R=(4.0 * _rows(g, m, k)).to(bf) if case["residual"] else None,
                  G=(1.0 + 0.1 * _normal(g, k)).to(bf), H=torch.empty(m, k, dtype=bf, device=DEVICE) if case["residual"] else None,
                  Y=torch.empty(m, k, dtype=bf, device=DEVICE) if case["plain_rows"] else None,
                  Q=torch.empty(m, k, dtype=torch.uint8, device=DEVICE), S=torch.empty(m, k // 32, dtype=torch.uint8, device=DEVICE))
        return st
    a, fmt = _rows(g, m, k).to(torch.bfloat16), case["fmt"]
    st["A"], st["AS"] = (a, None) if fmt == "bf16" else _quantize(a.float(), fmt)
    for name in ("W",) if kind == "product" else ("WG", "WU"):
        st[name], st[name + "S"] = _quantize(_normal(g, case["N"], k) * k ** -0.5, "mxfp4")
    st["C"] = torch.zeros(m, case["N"] + case["pad"], dtype=torch.bfloat16, device=DEVICE)
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    if c["kind"] == "round_trip":
        q, s = _quantize(state["X"][:, : c["K"]].float(), c["fmt"])
        return _dequantize(q, s, c["fmt"]).to(TYPES[c["type"]])
    if c["kind"] == "norm":
        x, h = state["X"].float(), None
        if state["R"] is not None:
            h = (x + state["R"].float()).to(torch.bfloat16)
            x = h.float()
        y = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * state["G"].float()
        q, s = _quantize(y, "mxfp8")
        return {"h": h, "y": y.to(torch.bfloat16) if c["plain_rows"] else None, "codes": q.view(E4M3), "scales": s.view(E8M0)}
    a = state["A"].float() if c["fmt"] == "bf16" else _dequantize(state["A"], state["AS"], c["fmt"])
    if c["kind"] == "product":
        return (a @ _dequantize(state["W"], state["WS"], "mxfp4").T).to(torch.bfloat16)
    gate = a @ _dequantize(state["WG"], state["WGS"], "mxfp4").T
    up = a @ _dequantize(state["WU"], state["WUS"], "mxfp4").T
    return (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)


def _run_own(st, c):
    from weight_quantized_decode_block_amd import wqd
    m, k = c["M"], c["K"]
    if c["kind"] == "round_trip":
        wqd.mx_quantize(st["X"], st["Q"], st["S"], c["fmt"], m, k, x_row_stride=k + c["pad"])
        wqd.mx_dequantize(st["Q"], st["S"], st["Y"], c["fmt"], m, k)
        return st["Y"]
    if c["kind"] == "norm":
        wqd.add_rmsnorm_mx8(st["X"], st["R"], st["G"], st["H"], st["Y"], st["Q"], st["S"], m, k, EPS)
        return {"h": st["H"], "y": st["Y"], "codes": st["Q"].view(E4M3), "scales": st["S"].view(E8M0)}
    n, ldc = c["N"], c["N"] + c["pad"]
    if c["kind"] == "product":
        if c["fmt"] == "bf16":
            wqd.w4a16_gemm(st["A"], st["W"], st["WS"], st["C"], m, n, k, c_row_stride=ldc)
        else:
            call = wqd.w4a8_gemm if c["fmt"] == "mxfp8" else wqd.w4a4_gemm
            call(st["A"], st["AS"], st["W"], st["WS"], st["C"], m, n, k, c_row_stride=ldc)
    elif c["fmt"] == "bf16":
        wqd.w4a16_gated(st["A"], st["WG"], st["WGS"], st["WU"], st["WUS"], st["C"], m, n, k, c_row_stride=ldc)
    else:
        call = wqd.w4a8_gated if c["fmt"] == "mxfp8" else wqd.w4a4_gated
        call(st["A"], st["AS"], st["WG"], st["WGS"], st["WU"], st["WUS"], st["C"], m, n, k, c_row_stride=ldc)
    return st["C"][:, :n]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    kind, m, k = case["kind"], case["M"], case["K"]
    if kind == "round_trip":
        wide = TYPES[case["type"]].itemsize
        packed = m * k // 2 if case["fmt"] == "mxfp4" else m * k
        return {"bytes": 2 * (m * k * wide + packed + m * k // 32), "flops": 4 * m * k}
    if kind == "norm":
        rows = 2 + (4 if case["residual"] else 0) + (2 if case["plain_rows"] else 0)
        return {"bytes": m * k * rows + 2 * k + m * k + m * k // 32, "flops": 6 * m * k}
    n, weights = case["N"], 1 if kind == "product" else 2
    a = {"bf16": 2 * m * k, "mxfp8": m * k + m * k // 32, "mxfp4": m * k // 2 + m * k // 32}[case["fmt"]]
    return {"bytes": weights * (n * k // 2 + n * k // 32) + a + 2 * m * n, "flops": 2 * weights * m * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits
def _power_of_two(e):
    """2^e in 64 bits, from the bits: a library's exp2 or log2 may be off at the powers themselves."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exponent(a):
    """floor(log2 a) of positive normal 64-bit values."""
    return (a.contiguous().view(torch.int64) >> 52) - 1023


def _grid(a, lowest, bits, largest):
    """Magnitudes rounded to nearest even onto the values of a float with `bits` fraction bits and lowest exponent."""
    step = _power_of_two(_exponent(torch.clamp(a, min=2.0 ** lowest)) - bits)
    return torch.clamp(torch.round(a / step) * step, max=largest)


def _exact_blocks(x, fmt):
    """(element values, scales) of rows in 64 bits."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = b.abs().max(dim=-1, keepdim=True).values
    emax, lowest, bits, largest = (2, 0, 1, 6.0) if fmt == "mxfp4" else (8, -6, 3, 448.0)
    e = torch.where(top > 0, _exponent(top) - emax, torch.full_like(top, -127).to(torch.int64)).clamp(min=-127)
    scale = _power_of_two(e)
    v = b / scale
    return torch.sign(v) * _grid(v.abs(), lowest, bits, largest), scale


def _exact_values(q, s, fmt):
    if fmt == "mxfp4":
        code = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.int64, device=q.device)
        code[:, 0::2], code[:, 1::2] = q & 15, q >> 4
        mag = code & 7
        v = torch.where(mag < 2, 0.5 * mag.double(), (1.0 + 0.5 * (mag & 1).double()) * _power_of_two((mag >> 1) - 1))
        v = torch.where(code > 7, -v, v)
    else:
        v = q.view(E4M3).double()
    return v * torch.repeat_interleave(_power_of_two(s.to(torch.int64) - 127), 32, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    k = case["K"]
    if case["kind"] == "round_trip":
        v, scale = _exact_blocks(st["X"][:, :k].double(), case["fmt"])
        return (v * scale).reshape(case["M"], k)
    if case["kind"] == "norm":
        h = st["X"]
        if st["R"] is not None:
            h = (st["X"].double() + st["R"].double()).float().to(torch.bfloat16)
        d = h.double()
        y = d / torch.sqrt(d.square().sum(-1, keepdim=True) / k + EPS) * st["G"].double()
        v, scale = _exact_blocks(y, "mxfp8")
        return {"h": h.double() if st["R"] is not None else None, "y": y if case["plain_rows"] else None,
                "codes": v.reshape(y.shape), "scales": scale.squeeze(-1)}
    a = st["A"].double() if case["fmt"] == "bf16" else _exact_values(st["A"], st["AS"], case["fmt"])
    if case["kind"] == "product":
        return a.matmul(_exact_values(st["W"], st["WS"], "mxfp4").t())
    gate = a.matmul(_exact_values(st["WG"], st["WGS"], "mxfp4").t())
    up = a.matmul(_exact_values(st["WU"], st["WUS"], "mxfp4").t())
    return gate * torch.sigmoid(gate) * up
