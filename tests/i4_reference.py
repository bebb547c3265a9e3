"""The products with 4-bit integer weights and the routed block in 64 bits, from
their definitions, for the tests: torch on the CPU, no code shared with the library."""
from __future__ import annotations

import torch

SCALES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def generator(*seed):
    g = torch.Generator()
    g.manual_seed(sum((i + 1) * 1000003 ** i * int(s) for i, s in enumerate(seed)) % (1 << 62))
    return g


def laid_out(codes: torch.Tensor) -> torch.Tensor:
    """Codes [E, N, K] in the tiles that include/wqd.h describes, byte by byte."""
    E, N, K = codes.shape
    out = torch.zeros(E, (N + 15) // 16, K // 128, 1024, dtype=torch.uint8)
    first, second = (0, 4, 1, 5), (2, 6, 3, 7)  # of byte b
    row = torch.zeros(E, (N + 15) // 16 * 16, K, dtype=torch.uint8)
    row[:, :N] = codes
    row = row.view(E, -1, 16, K // 128, 4, 4, 8)  # k = 32 j + 8 g + i
    at = out.view(E, -1, K // 128, 4, 16, 4, 4)  # g, n, j, b
    for g in range(4):
        for j in range(4):
            for b in range(4):
                at[:, :, :, g, :, j, b] = (row[..., j, g, first[b]] | row[..., j, g, second[b]] << 4).transpose(2, 3)
    return out.view(E, -1)


def tiles(x: torch.Tensor, K: int) -> torch.Tensor:
    """Scales or zero points [E, N, K/group] in the order of the codes' tiles."""
    E, N, G = x.shape
    per = G * 128 // K
    out = torch.zeros(E, (N + 15) // 16, K // 128, 16, per, dtype=x.dtype)
    for n in range(N):
        out[:, n // 16, :, n % 16] = x[:, n].view(E, K // 128, per)
    return out.view(E, -1)


def rows_of_pairs(codes: torch.Tensor) -> torch.Tensor:
    """Codes two a byte, the even k in the low nibble."""
    return codes[..., 0::2] | codes[..., 1::2] << 4


class Weights:
    """E matrices [N, K]: codes, scales and zero points, and what the definition makes of them."""

    def __init__(self, g, E, N, K, group, zeros, scale, exact=False):
        self.E, self.N, self.K, self.group, self.scale = E, N, K, group, scale
        self.codes = torch.randint(0, 16, (E, N, K), generator=g, dtype=torch.uint8)
        if exact:  # powers of two
            s = torch.exp2(-torch.randint(4, 7, (E, N, K // group), generator=g).double())
        else:
            s = (torch.rand(E, N, K // group, generator=g).double() + 0.5) * K ** -0.5 * torch.where(
                torch.rand(E, N, K // group, generator=g) < 0.1, -1.0, 1.0)
        self.s = s.to(SCALES[scale])
        self.z = torch.randint(0, 16, (E, N, K // group), generator=g, dtype=torch.uint8) if zeros else None

    def zero(self):
        return torch.full(self.s.shape, 8.0, dtype=torch.float64) if self.z is None else self.z.double()

    def values(self):
        """w in 64 bits."""
        r = lambda x: x.repeat_interleave(self.group, -1)  # noqa: E731
        return (self.codes.double() - r(self.zero())) * r(self.s.double())

    def size(self):
        """What enters the sums, as it is rounded: |s| (16 + q + 16 + z)."""
        r = lambda x: x.repeat_interleave(self.group, -1)  # noqa: E731
        return (self.codes.double() + 32 + r(self.zero())) * r(self.s.double().abs())

    def operands(self, device="cuda"):
        return (laid_out(self.codes).to(device), tiles(self.s, self.K).to(device), None if self.z is None else tiles(self.z, self.K).to(device))


def silu(x):
    return x * torch.sigmoid(x)


def sum_error(size, K):
    """Of a sum of K products in any order, `size` the sum of their magnitudes: an addition is off by a unit in the
    last place of fp32 at most (2^-23: the matrix instruction may cut), and a group's scale, its zero point and the
    waves' joining add at most K / 32 + 16 more."""
    return (K + K // 32 + 16) * 2.0 ** -23 * size


def stored(value, error):
    """How far a BF16 output may be: the error before it, and half a step of what is stored."""
    return error + 2.0 ** -8 * (value.abs() + error) + 2.0 ** -134


def gated(gate, up, eg, eu):
    """silu(gate) * up, and how far it is off: |silu'| <= 1.1, silu itself within 2^-16 of the result."""
    y = silu(gate) * up
    err = 1.1 * eg * (up.abs() + eu) + silu(gate).abs() * eu
    return y, err + 2.0 ** -16 * (y.abs() + err)


def route(logits, bias, top_k, scoring, groups, top_groups, group_top, renormalize, scale):
    """(ids, weights) token by token, in 64 bits: the choice by comparing pairs."""
    T, E = logits.shape
    ids = torch.full((T, top_k), -1, dtype=torch.int32)
    weights = torch.zeros(T, top_k, dtype=torch.float64)
    big = torch.finfo(torch.float32).max
    for t in range(T):
        x = logits[t].double()
        ok = ~torch.isnan(x) & (x > -torch.inf)
        x = torch.where(ok, x.clamp(max=big), 0.0)
        if scoring == "sigmoid":
            p = 1.0 / (1.0 + torch.exp(-x))
        else:
            e = torch.where(ok, torch.exp(x - x[ok].max()), 0.0) if ok.any() else torch.zeros(E, dtype=torch.float64)
            p = e / e.sum() if ok.any() else e
        key = x.clone()
        if bias is not None:
            b = bias.double()
            ok = ok & ~torch.isnan(b) & (b > -torch.inf)
            key = p + torch.where(ok, b, 0.0)
        if groups > 1:
            size, best = E // groups, []
            value = key if bias is not None or group_top == 1 else p
            for i in range(groups):
                v = sorted((float(value[j]) for j in range(i * size, (i + 1) * size) if ok[j]), reverse=True)
                best.append(sum(v[:group_top]) if v else -torch.inf)
            order = sorted(range(groups), key=lambda i: (-best[i], i))[:top_groups]
            inside = torch.zeros(E, dtype=torch.bool)
            for i in order:
                inside[i * size:(i + 1) * size] = True
            ok = ok & inside
        chosen = sorted((j for j in range(E) if ok[j]), key=lambda j: (-float(key[j]), j))[:top_k]
        w = [float(p[j]) for j in chosen]
        total = sum(w)
        for s, j in enumerate(chosen):
            ids[t, s] = j
            weights[t, s] = (w[s] / total if total > 0 else 0.0) * scale if renormalize else w[s] * scale
    return ids, weights


def lists(ids, E):
    flat = ids.flatten().tolist()
    order, offsets = [], [0]
    for e in range(E):
        order += [p for p, i in enumerate(flat) if i == e]
        offsets.append(len(order))
    return torch.tensor(order + [-1] * (len(flat) - len(order)), dtype=torch.int32), torch.tensor(offsets, dtype=torch.int32)
