"""GPU tests of the products with 4-bit integer weights at the ends of what activations may be: the largest for which the
header promises finite outputs, and rows that are not finite, on every kernel that sizes choose."""
import pytest
import torch

import i4_reference as ref
from parity import requires_gpu
from test_gpu_i4 import BF, out, untouched
from weight_quantized_decode_block_amd import wqd

pytestmark = [pytest.mark.gpu, requires_gpu]

# the kernel for few rows of 4, 8 and 16, chunks of 32 rows, tiles of 64 and of 128 rows
SIZES = [(1, 40, 256), (6, 40, 256), (12, 40, 256), (97, 5120, 128), (300, 1000, 256), (5864, 385, 256), (5471, 898, 256)]


@pytest.mark.parametrize("top", [15, 255])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_the_largest_activations(M, N, K, group, top):
    """All of one sign, a step below 2^116 with zero points up to 15 and below 2^112 with any.  A group's sums have 8 bits of the
    activation, 7 of the count and 9 of 16 + z: exact in fp32, and so are the outputs before they are rounded."""
    w = ref.Weights(ref.generator(91, M, group), 1, N, K, group, True, "fp16")
    w.codes[:, ::3], w.codes[:, 1::3] = 0, 15
    w.z[:] = top
    w.z[:, N // 2:] = 0
    w.s[:] = 2.0 ** -14
    A = torch.full((M, K), (2.0 - 2.0 ** -7) * 2.0 ** (115 if top == 15 else 111), dtype=BF)
    A[1::2] *= -1.0
    C = out(M, N, N)
    wqd.i4a16_gemm(A.cuda(), *w.operands(), C, M, N, K, group)
    want = (A[:2].double() @ w.values()[0].T).to(BF)
    assert bool(torch.isfinite(want).all()) and torch.equal(C[:M].cpu(), want[torch.arange(M) % 2]) and untouched(C, M, N)
