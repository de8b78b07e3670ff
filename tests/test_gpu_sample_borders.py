"""Sampling at the borders of its definition."""
import numpy as np
import pytest
import torch

from tests import test_gpu_sample as T

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def D():
    from block_denoising_gb300 import build, dinfer
    build.build()
    return dinfer


@pytest.mark.parametrize("top", [0.0, 2.0 ** -11, 0.73, -1.0, 12.345, 3000.0])
@pytest.mark.parametrize("temperature", [1e-2, 1e-3, 1e-4, 1e-5, 1e-6])
def test_small_temperatures(D, top, temperature):
    """Logits that lie a few temperatures, some 10^-5 each, below the largest: their differences count as they are."""
    rng = np.random.default_rng(int(1e4 * abs(top)) + int(1e7 * temperature))
    for rows, vocab in ((8, 300), (4, 20000)):
        x = np.full((rows, vocab), top - 1.0) - rng.random((rows, vocab))
        for r in range(rows):
            at = rng.permutation(vocab)[:60]
            x[r, at] = top - temperature * rng.uniform(0.0, 12.0, 60)
            x[r, at[0]] = top
        x = torch.from_numpy(x.astype(np.float32)).to(dev)
        for _ in range(3):
            u = [float(np.float32(v)) for v in rng.random(rows) * 0.9999]
            for s in ({}, dict(top_p=[0.8] * rows), dict(top_k=[20] * rows, top_p=[0.9] * rows), dict(min_p=[0.01] * rows)):
                T.check(D, x, u, temperature=[temperature] * rows, unsure=2, **s)
