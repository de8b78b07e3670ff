"""Sampling on the GPU against its definition in 64 bits.

Tokens have to be equal wherever no sum of weights lies within 2^-28 of its border (tests/sample64.py); the kernel's
weights are off by some 2^-31.  The confidence is a quotient of two sums of up to 2^19 weights in fp32: each weight by
2^-21 at most (its argument, up to 2^4 where it counts, is rounded by 2^-20 at most; the power by 2^-22), the sum of a
thread's 64 numbers and of ten levels above it by 80 * 2^-24: 2^-17 in all.
"""
import numpy as np
import pytest
import torch

from tests import sample64 as S

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def D():
    from block_denoising_gb300 import build, dinfer
    build.build()
    return dinfer


def col(v, dtype=F32):
    return None if v is None else torch.tensor(v, dtype=dtype, device=dev)


def check(D, x, u, temperature=None, top_k=None, top_p=None, min_p=None, unsure=None):
    """x [rows, vocab] tensor on the GPU, settings lists or None; every row against the definition."""
    tok, conf = D.op_sample(x, col(u), temperature=col(temperature), top_k=col(top_k, torch.int32), top_p=col(top_p), min_p=col(min_p))
    tok, conf, h = tok.tolist(), conf.tolist(), x.double().cpu().numpy()
    f = lambda v, r: None if v is None else float(np.float32(v[r]))
    skipped = 0
    for r in range(x.shape[0]):
        t = 1.0 if temperature is None else f(temperature, r)
        want, c = S.draw(h[r], f(u, r), t, None if top_k is None else top_k[r], f(top_p, r), f(min_p, r))
        if want is None:
            skipped += 1
            continue
        assert tok[r] == want, (r, tok[r], want, t)
        assert abs(conf[r] - c) <= 2.0 ** -17 * c, (r, conf[r], c)
    assert skipped <= (len(u) // 50 + 1 if unsure is None else unsure)
    return tok


def logits(rng, rows, vocab, dtype, spread=2.0):
    x = rng.standard_normal((rows, vocab)) * spread
    for r in range(rows):
        at = rng.integers(0, vocab, 8)
        x[r, at] += rng.uniform(0, 10, 8)
    x[:, vocab - 1] = -np.inf if vocab > 1 else 0.0
    return torch.from_numpy(x.astype(np.float32)).to(dtype).to(dev)


SETTINGS = [
    {}, dict(temperature=[0.3, 0.7, 1.3, 3.0]), dict(top_k=[1, 2, 50, 1000]), dict(top_p=[0.1, 0.5, 0.9, 0.999]), dict(min_p=[0.01, 0.1, 0.5, 1.0]),
    dict(temperature=[0.7, 1.0, 1.5, 0.0], top_k=[20, 0, 400, 5], top_p=[0.9, 0.95, 0.5, 1.0], min_p=[0.0, 0.05, 0.001, 0.2]),
]


@pytest.mark.parametrize("settings", range(len(SETTINGS)))
@pytest.mark.parametrize("rows,vocab,dtype", [(3, 1, F32), (4, 2, BF), (8, 33, F32), (16, 1000, BF), (9, 2048, F32), (9, 2049, BF), (24, 4097, F32),
                                              (12, 30001, BF), (4, 126464, F32), (6, 157184, BF), (64, 157184, F32)])
def test_against_the_definition(D, rows, vocab, dtype, settings):
    rng = np.random.default_rng(rows * 1000 + vocab)
    x = logits(rng, rows, vocab, dtype)
    s = {n: [v[r % 4] for r in range(rows)] for n, v in SETTINGS[settings].items()}
    for _ in range(3):
        check(D, x, [float(np.float32(v)) for v in rng.uniform(0, 1, rows) * 0.999999], **s)


@pytest.mark.parametrize("vocab", [64, 5000, 126464])
def test_equal_logits(D, vocab):
    """Cuts and draws among ties go by the index, exactly."""
    rows = 6
    for value in (0.0, -3.25, 1e-30, 77.5):
        x = torch.full((rows, vocab), value, device=dev)
        u = [0.0, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -24, 0.125]
        assert check(D, x, u)[0] == 0
        check(D, x, u, top_k=[1, 3, vocab // 2, vocab - 1, vocab, 7])
        check(D, x, u, top_p=[0.5, 0.25, 0.75, 0.125, 0.0, 0.5])
        check(D, x, u, top_k=[8, 16, 32, 4, 2, 64], top_p=[0.5, 0.25, 0.75, 0.125, 0.0, 0.5], min_p=[1.0] * 6)
    x = torch.zeros((rows, vocab), device=dev)
    x[:, ::2] = -0.0
    check(D, x, u, top_k=[1, 3, vocab // 2, vocab - 1, vocab, 7])
    x[:, 1::3] = 1.0
    check(D, x, u, top_k=[vocab // 2] * rows, temperature=[1e30] * rows)


def test_rows_and_numbers_at_the_ends(D):
    inf, nan = np.inf, np.nan
    rows = [[-inf] * 5, [nan] * 5, [nan, 1.0, -inf, 1.0, 0.0], [inf, 0.0, inf, nan, -inf], [3e38, -3e38, 3e38, 0.0, -inf], [1e-40, 0.0, -1e-40, -0.0, 2e-40],
            [-1e4, -1e4 - 1, -1e4 - 2, -inf, -1e4], [5000.5, 5000.25, 5000.0, 4999.0, 0.0], [0.0, -31.0, -30.4, -30.6, -29.0]]
    x = torch.tensor(rows, device=dev)
    n = len(rows)
    for u in (0.0, 0.3, 0.6, 0.999):
        for s in ({}, dict(temperature=[1e-30] * n), dict(temperature=[0.0] * n), dict(temperature=[-1.0] * n), dict(temperature=[1e30] * n),
                  dict(top_k=[2] * n), dict(top_p=[0.7] * n), dict(min_p=[0.5] * n), dict(top_k=[3] * n, top_p=[0.9] * n, min_p=[0.1] * n),
                  dict(top_k=[-1] * n, top_p=[1.5] * n, min_p=[-2.0] * n)):
            check(D, x, [u] * n, unsure=n, **s)
    one = torch.tensor([[1.0, 2.0, 0.5]] * 6, device=dev)
    tok, _ = D.op_sample(one, torch.tensor([nan, -inf, -0.5, 1.0, inf, 7.0], device=dev))
    assert tok.tolist() == [0, 0, 0, 2, 2, 2]
    tok, _ = D.op_sample(one, torch.full((6,), 0.9, device=dev), temperature=torch.tensor([nan, inf, 1.0, 1.0, 1.0, 1.0], device=dev),
                         top_p=torch.tensor([1.0, 1.0, nan, -1.0, 1.0, 1.0], device=dev), min_p=torch.tensor([0, 0, 0, 0, nan, 9.0], device=dev))
    assert tok.tolist() == [1, 2, 2, 1, 2, 1]


def test_strides_alignment_and_outputs_of_ones_own(D):
    rng = np.random.default_rng(8)
    for dtype, off in ((F32, 1), (F32, 3), (BF, 1), (BF, 5), (BF, 7)):
        wide = logits(rng, 5, 9011, dtype)
        x = wide[:, off:off + 8999]
        tok, conf = torch.full((5,), -7, dtype=torch.int32, device=dev), torch.zeros(5, device=dev)
        u = torch.rand(5, device=dev)
        got = D.op_sample(x, u, tok=tok, conf=conf)
        assert got[0] is tok and got[1] is conf
        want = D.op_sample(x.contiguous(), u)
        assert torch.equal(tok, want[0]) and torch.allclose(conf, want[1], rtol=2.0 ** -17, atol=0)


def test_many_rows_and_the_same_tokens_again(D):
    rng = np.random.default_rng(4)
    x = logits(rng, 700, 3000, F32)
    u = [float(v) for v in rng.uniform(0, 0.9999, 700)]
    s = dict(temperature=[0.8] * 700, top_k=[100] * 700, top_p=[0.9] * 700)
    first = check(D, x, u, **s)
    assert check(D, x, u, **s) == first


def test_the_confidence_is_the_lm_heads(D):
    """Greedy over the logits that the fused LM head writes: its own token, and its confidence."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    X = torch.randn((64, 256), generator=g, device=dev).to(BF)
    W = (torch.randn((4096, 256), generator=g, device=dev) * 0.1).to(BF)
    want, conf, out = D.op_lmhead_bf16(X, W, 4095, 1.0, D.OpWorkspace(), want_logits=True)
    tok, c = D.op_sample(out, torch.zeros(64, device=dev), temperature=torch.zeros(64, device=dev))
    assert torch.equal(tok, want) and torch.allclose(c, conf, rtol=1e-5, atol=0)


def test_captured_and_on_another_stream(D):
    rng = np.random.default_rng(6)
    x, u = logits(rng, 3, 20000, F32), torch.rand(3, device=dev)
    tok, conf = torch.empty(3, dtype=torch.int32, device=dev), torch.empty(3, device=dev)
    D.op_sample(x, u, tok=tok, conf=conf)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        D.op_sample(x, u, tok=tok, conf=conf)
    for _ in range(3):
        u.copy_(torch.rand(3, device=dev))
        g.replay()
        want = D.op_sample(x, u)
        assert torch.equal(tok, want[0]) and torch.equal(conf, want[1])


def test_shares_follow_the_weights(D):
    """Evenly spread numbers draw every token as often as its weight says, to one draw at either end."""
    x = torch.tensor([[0.0, 1.0, -1.0, 2.0, 0.5]], device=dev).expand(1, 5)
    n = 4000
    u = (torch.arange(n, device=dev, dtype=F32) + 0.5) / n
    tok, _ = D.op_sample(x.expand(n, 5).contiguous(), u)
    share = torch.bincount(tok.long(), minlength=5).double().cpu().numpy()
    w = np.exp(x[0].double().cpu().numpy())
    assert np.abs(share - n * w / w.sum()).max() <= 2


@pytest.mark.parametrize("rows,vocab,dtype", [(512, 126464, BF), (300, 40000, F32), (64, 157184, F32)])
def test_many_full_rows_at_once(D, rows, vocab, dtype):
    """More rows than are at work together, of every kind side by side, several times: what a row's CTAs tell one another
    is told in the order in which it is read.  Some rows against the definition, all against the call before."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    pick = lambda values, dtype=F32: torch.tensor(values, dtype=dtype, device=dev)[torch.randint(0, len(values), (rows,), generator=g, device=dev)]
    rng = np.random.default_rng(rows)
    for turn in range(8):
        x = torch.randn((rows, vocab), generator=g, device=dev) * (0.5 + 2.5 * torch.rand((rows, 1), generator=g, device=dev))
        for _ in range(10):
            x.scatter_add_(1, torch.randint(0, vocab, (rows, 1), generator=g, device=dev), 12 * torch.rand((rows, 1), generator=g, device=dev))
        x = x.to(dtype)
        u = torch.rand(rows, generator=g, device=dev)
        s = dict(temperature=pick([0.0, 0.3, 0.7, 1.0, 1.3, 3.0]), top_k=pick([0, 0, 0, 20, 50, 1000], torch.int32), top_p=pick([1.0, 0.5, 0.9, 0.95]),
                 min_p=pick([0.0, 0.0, 0.05, 0.1]))
        tok, conf = D.op_sample(x, u, **s)
        for _ in range(3):
            again = D.op_sample(x, u, **s)
            assert torch.equal(again[0], tok) and torch.equal(again[1], conf)
        for r in rng.integers(0, rows, 6):
            f = {n: v[r].item() for n, v in s.items()}
            want, c = S.draw(x[r].double().cpu().numpy(), u[r].item(), f["temperature"], f["top_k"], f["top_p"], f["min_p"])
            assert want is None or (int(tok[r]) == want and abs(float(conf[r]) - c) <= 2.0 ** -17 * c)


@pytest.mark.parametrize("rows", [1, 64])
@pytest.mark.parametrize("vocab,period", [(131072, 512), (131072, 1024), (8192, 512), (16384, 1024)])
@pytest.mark.parametrize("inside", [True, False])
def test_rows_whose_eighth_misleads(D, rows, vocab, period, inside):
    """The part of a row that the first guess of top-p's cut looks at holds nothing, or nearly everything: the guess is
    found wrong, and made good."""
    rng = np.random.default_rng(rows + vocab + period)
    x = -5.0 * rng.random((rows, vocab))
    part = np.arange(vocab) % period < 128
    x[:, part if inside else ~part] -= 60.0 if inside else 4.0
    x = torch.from_numpy(x.astype(np.float32)).to(dev)
    for p in (0.2, 0.5, 0.9, 0.99):
        u = [float(np.float32(v)) for v in rng.random(rows) * 0.9999]
        if rows == 1:
            check(D, x, u, top_p=[p] * rows, unsure=1)
            check(D, x, u, top_p=[p] * rows, top_k=[vocab // 2] * rows, temperature=[0.5] * rows, unsure=1)
        else:
            tok, conf = D.op_sample(x, col(u), top_p=col([p] * rows))
            for r in (0, 31, 63):
                want, c = S.draw(x[r].double().cpu().numpy(), u[r], 1.0, None, float(np.float32(p)), None)
                assert want is None or int(tok[r]) == want
