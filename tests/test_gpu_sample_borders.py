"""Sampling at the borders of its definition: small temperatures, weights that count as 0 between equal ones.

tests/sample64.py leaves a row out where a sum lies near a border and the weights are not all equal; the rows with weights
that count as 0 are made so that what is left is certain, and every one of them is compared.
"""
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


def tied(rows, vocab, dtype, tail, tops):
    """Logits 0 at tops, tail elsewhere."""
    x = torch.full((rows, vocab), tail, dtype=F32)
    x[:, tops] = 0.0
    return x.to(dtype).to(dev)


def draw(D, x, u, **settings):
    """Tokens of every row for every number of u, settings the same for all rows."""
    n = x.shape[0]
    full = {k: torch.full((n,), v, dtype=torch.int32 if k == "top_k" else F32, device=dev) for k, v in settings.items()}
    return [sorted(set(D.op_sample(x, torch.full((n,), v, dtype=F32, device=dev), **full)[0].tolist())) for v in u]


# e^(tail / T): 2^-44.7 and 2^-45.7, and far less: below 2^-44 each, which counts as 0
@pytest.mark.parametrize("dtype,tail,temperature", [(F32, -31.0, 1.0), (BF, -9.5, 0.3), (F32, -38.0, 1.0), (BF, -1000.0, 1.0), (F32, -0.031, 0.001)])
@pytest.mark.parametrize("rows,vocab", [(1, 64), (3, 5000), (1, 126464), (64, 40000), (400, 9001)])
def test_weights_that_count_as_zero(D, rows, vocab, dtype, tail, temperature):
    last = vocab - 1
    two = tied(rows, vocab, dtype, tail, [0, last])
    below = 1.0 - 2.0 ** -24
    t = dict(temperature=temperature)
    # two equal weights: the first sum above half of them is the second one's
    assert draw(D, two, [0.0, 0.5 - 2.0 ** -25, 0.5, 0.75, below, 1.0], **t) == [[0], [0], [last], [last], [last], [last]]
    # half of their weight is the first one's; more is both's
    assert draw(D, two, [0.0, 0.5, below, 1.0], top_p=0.5, **t) == [[0]] * 4
    assert draw(D, two, [0.25, 0.5, below], top_p=0.5 + 2.0 ** -24, **t) == [[0], [last], [last]]
    assert draw(D, two, [0.25, 0.5, below, 1.0], min_p=2.0 ** -43, **t) == [[0], [last], [last], [last]]
    # of the first `vocab - 1` of the order all that weighs is the two
    assert draw(D, two, [0.25, 0.5, below, 1.0], top_k=last, **t) == [[0], [last], [last], [last]]
    assert draw(D, two, [0.25, below, 1.0], top_k=last, top_p=0.5, **t) == [[0]] * 3
    one = tied(rows, vocab, dtype, tail, [0])
    assert draw(D, one, [0.0, 0.5, below, 1.0], **t) == [[0]] * 4
    assert draw(D, one, [0.0, 0.5, below, 1.0], top_p=below, **t) == [[0]] * 4
    four = tied(rows, vocab, dtype, tail, [1, 2, vocab // 2, last - 1])
    assert draw(D, four, [0.0, 0.25, 0.5, 0.75, 1.0], **t) == [[1], [2], [vocab // 2], [last - 1], [last - 1]]
    assert draw(D, four, [0.0, 0.34, 0.67, 1.0], top_p=0.75, **t) == [[1], [2], [vocab // 2], [vocab // 2]]


@pytest.mark.parametrize("vocab,dtype", [(3001, F32), (40000, BF), (126464, F32)])
def test_a_row_alone_and_in_batches(D, vocab, dtype):
    """A row's token does not hang on how many rows there are, and so on how many CTAs and threads share it: no sum lies
    within 2^-31 of its border here."""
    rng = np.random.default_rng(vocab)
    n = 320
    x = T.logits(rng, n, vocab, dtype)
    u = torch.from_numpy(rng.random(n).astype(np.float32)).to(dev).clamp(max=0.9999)
    pick = lambda v, t=F32: torch.tensor(v, dtype=t, device=dev)[torch.from_numpy(rng.integers(0, len(v), n)).to(dev)]  # noqa: E731
    s = dict(temperature=pick([0.0, 0.3, 1.0, 1.7]), top_k=pick([0, 0, 40, 2000], torch.int32), top_p=pick([1.0, 0.5, 0.9, 0.99]),
             min_p=pick([0.0, 0.0, 0.02]))
    for used in ({}, {"temperature": s["temperature"]}, {"top_p": s["top_p"]}, s):
        tok, conf = D.op_sample(x, u, **used)
        for size in (1, 3, 64, 160):
            for a in range(0, n, size) if size > 3 else (0, 100, n - size):
                got = D.op_sample(x[a:a + size], u[a:a + size], **{k: v[a:a + size] for k, v in used.items()})
                assert torch.equal(got[0], tok[a:a + size]), (size, a, list(used))
                assert torch.allclose(got[1], conf[a:a + size], rtol=2.0 ** -16, atol=0)  # each within 2^-17 of the definition


def test_rows_at_the_ends_every_one_compared(D):
    """Infinities, NaN and extreme temperatures, with numbers of which none lies near a border: no row is left out."""
    inf, nan = np.inf, np.nan
    rows = [[-inf] * 5, [nan] * 5, [nan, 1.0, -inf, 1.0, 0.0], [inf, 0.0, inf, nan, -inf], [3e38, -3e38, 3e38, 0.0, -inf], [1e-40, 0.0, -1e-40, -0.0, 2e-40],
            [-1e4, -1e4 - 1, -1e4 - 2, -inf, -1e4], [5000.5, 5000.25, 5000.0, 4999.0, 0.0], [0.0, -31.0, -30.4, -30.6, -29.0]]
    x = torch.tensor(rows, device=dev)
    n = len(rows)
    for u in (0.0, 0.27, 0.31, 0.62, 0.77, 0.9):
        for s in ({}, dict(temperature=1e-30), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=1e30), dict(top_k=2), dict(top_p=0.71),
                  dict(min_p=0.53), dict(top_k=3, top_p=0.91, min_p=0.13), dict(top_k=-1, top_p=1.5, min_p=-2.0)):
            T.check(D, x, [float(np.float32(u))] * n, unsure=0, **{k: [v] * n for k, v in s.items()})


@pytest.mark.parametrize("temperature", [1e37, 1e38, 3e38, float("inf")])
def test_logits_further_apart_than_the_largest_float(D, temperature):
    """Their differences overflow, what the temperature leaves of them does not."""
    rows = [[3e38, -3e38, 1e38, -1e38, 0.0], [-3.4e38, 3.4e38, 2e38, -2e38, 3.4e38], [3e38, -3e38, -3e38, -3e38, -3e38]] * 2
    x = torch.tensor(rows, device=dev)
    for u in (0.03, 0.27, 0.41, 0.62, 0.83, 0.97):
        for s in ({}, dict(top_k=3), dict(top_p=0.83), dict(min_p=0.013), dict(top_k=4, top_p=0.77, min_p=0.011)):
            if temperature < 1e39:
                T.check(D, x, [float(np.float32(u))] * 6, unsure=0, temperature=[temperature] * 6, **{k: [v] * 6 for k, v in s.items()})
        if temperature > 1e39:  # every weight is the largest
            tok, _ = D.op_sample(x, torch.full((6,), u, device=dev), temperature=torch.full((6,), temperature, device=dev))
            assert tok.tolist() == [int(u * 5)] * 6
