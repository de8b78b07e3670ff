"""The bound on the bf16 token kernel's weights, and the inputs that pin it, on the CPU: weights held as the kernel holds
them stay inside, weights that lose their second part, or hold one rounded part, do not."""
import numpy as np
import pytest
import torch

from tests import attention64 as A


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def cut(x):
    """The number just below x in fp32, its lower 16 bits cut off."""
    bits = np.maximum(np.asarray(x, np.float32).view(np.uint32), 1) - 1
    return (bits & np.uint32(0xffff0000)).view(np.float32).astype(np.float64)


TWO_PARTS = lambda p: cut(p) + bf16(p - cut(p))  # noqa: E731
FIRST_PART = cut
ROUNDED = bf16


@pytest.mark.parametrize("n", [5, 40, 130, 300])
@pytest.mark.parametrize("hd,heads", [(64, 3), (128, 8), (64, 11), (128, 16)])
def test_the_bound_tells_two_parts_from_one(n, hd, heads):
    rng = np.random.default_rng(n + heads)
    q, k, v = A.cancelling(rng, n, hd, heads, bf16)
    worst = {}
    for hold in (TWO_PARTS, FIRST_PART, ROUNDED):
        ratio = 0.0
        for h in range(heads):
            o, tol = A.attend(q[h], k, v, np.ones(n, bool), 1.0, True, 2.0 ** -16)
            p = np.exp(k @ q[h])
            p = p.astype(np.float32).astype(np.float64)
            got = bf16((hold(p) @ v) / (hold(p).sum() if hold is ROUNDED else p.sum()))
            ratio = max(ratio, float((np.abs(got - o) / tol).max()))
        worst[hold] = ratio
    assert worst[TWO_PARTS] <= 1.0
    assert worst[FIRST_PART] > 1.5 and worst[ROUNDED] > 1.5, worst


def test_weights_in_two_parts():
    # 2^-16 of the weight at most, the rest more than 0 wherever the weight is, 0 and 0 for 0
    rng = np.random.default_rng(1)
    p = np.exp2(rng.uniform(-100, 8, 100000)).astype(np.float32).astype(np.float64)
    p[:20] = 2.0 ** np.arange(-11, 9)
    assert np.all(np.abs(TWO_PARTS(p) - p) <= 2.0 ** -16 * p)
    assert np.all(bf16(p - cut(p)) > 0) and np.all(cut(p) < p)
    assert TWO_PARTS(np.zeros(1)) == 0 and cut(np.zeros(1)) == 0
