"""Gated products where the gate is far from zero: silu(g) * u for g from -350 to
350 and u up to 2^112, against 64 bits.

Gate and up sums are exact (a few products of one grid, different k for the two),
so what is left is the activation, which the library computes within 2^-19 of its
value (three roundings and an exponential of 3.5 steps of 2^-23 in each of two
factors, a reciprocal of 1 + e^2 within 6), and the store: half a BF16 step, 2^-8 of
the value, or half a subnormal one, 2^-134."""
import numpy as np
import pytest

import mx_reference as ref
from parity import requires_gpu
from test_gpu_mx import ACTS, product_gpu
from weight_quantized_decode_block_amd import inputs as gen

pytestmark = [pytest.mark.gpu, requires_gpu]


def operands(fmt, M, N, K):
    """Activations of 1 at k 0-7, 32-39 and 64, times 1, 1/2 or 1/4 by row; gate
    codes at the first sixteen, in steps of 8 and of 1/4, the up code at the last."""
    r = gen.rng(963, M, N)
    down = np.arange(M) % 3
    ones = np.r_[0:8, 32:40, 64]
    if fmt == "bf16":
        a = np.zeros((M, K))
        a[:, ones] = np.ldexp(1.0, -down)[:, None]
        a, s = gen.bf16_bits(a), None
    else:
        a = np.zeros((M, K), np.uint8)
        a[:, ones] = 0x38 if fmt == "mxfp8" else 2
        if fmt == "mxfp4":
            a = a[:, 0::2] | a[:, 1::2] << 4
        s = np.repeat((127 - down).astype(np.uint8)[:, None], K // 32, 1)
    g, u = np.zeros((N, K // 2), np.uint8), np.zeros((N, K // 2), np.uint8)
    gs, us = np.full((N, K // 32), 127, np.uint8), np.full((N, K // 32), 127, np.uint8)
    g[:, np.r_[0:4, 16:20]] = r.integers(0, 256, (N, 8), np.uint8)
    gs[:, 0], gs[:, 1] = 127 + 4, 127 - 1
    u[:, 32] = r.integers(1, 16, N)
    us[:, 2] = 127 + r.integers(-20, 110, N)
    return a, s, (g, gs, u, us)


@pytest.mark.parametrize("fmt", ACTS)
@pytest.mark.parametrize("M,N,K", [(3, 5000, 128), (24, 3000, 640), (64, 6000, 512), (300, 4096, 512), (300, 17000, 640)])
def test_far_gates(fmt, M, N, K):
    a, s, mats = operands(fmt, M, N, K)
    c = gen.bf16_values(product_gpu(fmt, a, s, mats, N, K)).astype(np.float64)
    av = ref.act_values(a, s, fmt)[:3]  # the rows repeat
    gate = av @ ref.values(mats[0], mats[1], "mxfp4").T
    up = av @ ref.values(mats[2], mats[3], "mxfp4").T
    want = ref.silu(gate) * up
    assert (gate < -150).any() and ((gate < -88.8) & (gate > -120) & (np.abs(want) > 1e-30)).any() and (gate > 150).any()
    e = 2.0 ** -19 * np.abs(want)
    want = np.resize(want, c.shape) if M > 3 else want
    e = np.resize(e, c.shape) if M > 3 else e
    assert (np.abs(c - want) <= 2.0 ** -8 * (np.abs(want) + e) + e + 2.0 ** -134).all()


@pytest.mark.parametrize("fmt", ACTS)
def test_gates_beyond_numbers(fmt):
    """Infinite sums: silu(inf) * u = inf * u, silu(-inf) is 0 / 0 by the formula,
    and an up sum of 0 makes 0 of every finite gate."""
    M, N, K = 1, 32, 128
    a, s, (g, gs, u, us) = operands(fmt, M, N, K)
    g[:], u[:], us[:] = 0, 0, 127
    g[:, 0] = np.where(np.arange(N) % 2, 0x0F, 0x07)  # -6 and 6
    gs[:, 0] = np.where(np.arange(N) < 16, 254, 131)
    u[:, 32] = np.where(np.arange(N) % 4 < 2, 2, 0)
    big = np.full((1, K // 32), 127 + 100, np.uint8)
    if fmt == "bf16":
        a = gen.bf16_bits(gen.bf16_values(a) * np.float32(2.0 ** 100))
    else:
        s = big
    c = gen.bf16_values(product_gpu(fmt, a, s, (g, gs, u, us), N, K))[0]
    n = np.arange(N)
    top = n < 16
    assert (c[top & (n % 4 == 0)] == np.inf).all()  # inf * 2^100
    assert np.isnan(c[top & (n % 2 == 1)]).all()
    assert np.isnan(c[top & (n % 4 == 2)]).all()  # inf * 0
    assert (c[~top & (n % 4 >= 2)] == 0).all() and (c[~top & (n % 4 == 1)] == 0).all()
    assert (c[~top & (n % 4 == 0)] == np.inf).all()  # 96 * 2^100 * 2^100 leaves fp32
