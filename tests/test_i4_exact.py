"""What test_gpu_i4_exact.py would notice, on the CPU: outputs without a group, without a wave's share of K, of a
neighbour's scales or of zeros are beyond its tolerances in every row, at every size."""
import pytest
import torch

import test_gpu_i4_exact as exact


def without(w, lo, hi):
    """w's matrix with no codes in k of lo .. hi - 1."""
    v = w.values()[0].clone()
    v[:, lo:hi] = 0
    return v


def mistakes(w):
    K, group = w.K, w.group
    steps = K // 128
    yield "the last group is lost", without(w, K - group, K)
    yield "the first group is lost", without(w, 0, group)
    yield "a step is lost", without(w, steps // 2 * 128, steps // 2 * 128 + 128)
    yield "a wave's share is lost", without(w, 128 * (steps * 7 // 8), K)
    yield "all is lost", torch.zeros_like(w.values()[0])
    if K > group:
        s, w.s = w.s, w.s.roll(1, -1)
        yield "a neighbour's scales", w.values()[0]
        w.s = s


@pytest.mark.parametrize("group,zeros,scale", exact.CONFIGS)
@pytest.mark.parametrize("M,N,K", exact.EXACT)
def test_a_mistake_shows(M, N, K, group, zeros, scale):
    (w,), a = exact.inputs(101, M, N, K, group, zeros, scale)
    want = exact.sums(a, w).to(exact.BF)
    (wg, wu), b = exact.inputs(102, M, N, K, group, zeros, scale, 2)
    gate, up = exact.sums(b, wg), exact.sums(b, wu)
    y, bound = exact.gated(gate, up)
    for (what, v), (_, vg) in zip(mistakes(w), mistakes(wg)):
        assert bool(((a.double() @ v.T).to(exact.BF) != want).any(1).all()), what
        wrong = exact.gated(b.double() @ vg.T, up)[0]
        assert bool(((wrong - y).abs() > 2.0 * bound).any(1).all()), what
