"""Attention over shared prefixes on the GPU: against 64 bits, and against the attention that reads every sequence by itself.

The bound (tests/attention64.py) is derived from the kernels' arithmetic for every output element, with the weights of bf16
calls rounded to bf16; joining two sums adds a few roundings of 2^-23, which the bound's 64 spare ones hold.
"""
import numpy as np
import pytest
import torch

from tests import attention64 as A

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def D():
    from block_denoising_gb300 import build, dinfer
    build.build()
    return dinfer


@pytest.fixture(scope="module")
def ws(D):
    return D.OpWorkspace()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def values(rng, shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype).to(dev)


def make(D, rng, shared, own, page, kv_heads, hd, dtype=BF, order="token", layers=1, spare=0):
    """A cache of len(own) groups: group g's sequences fork one of shared[g] tokens and add own[g][i] (None: not in use).
    Returns the cache, the entries' sequences in a shuffled numbering, and the groups' bounds."""
    flat = [x for o in own for x in o]
    n, groups = len(flat), len(own)
    most = max(-(-(s + max([x or 0 for x in o] + [0])) // page) for s, o in zip(shared, own)) + 1
    pages = sum(-(-s // page) for s in shared) + sum(-(-(x or 0) // page) + 2 for x in flat) + spare + 2
    shape = (layers, pages, page, kv_heads, hd)
    kv = []
    for _ in range(2):
        t = values(rng, shape, dtype)
        kv.append(t if order == "token" else t.transpose(2, 3).contiguous().transpose(2, 3))
    c = D.PagedKV(kv[0], kv[1], torch.full((n + groups, most), -1, dtype=torch.int32, device=dev),
                  torch.zeros(n + groups, dtype=torch.int32, device=dev), torch.zeros(pages, dtype=torch.int32, device=dev))
    at = [int(x) for x in rng.permutation(n + groups)]
    seqs, firsts, bounds = at[:n], at[n:], [0]
    for g, o in enumerate(own):
        c.extend(ints([shared[g]]), ints([firsts[g]]))
        for i, x in enumerate(o):
            if x is not None:
                c.fork(ints([firsts[g]]), ints([seqs[bounds[-1] + i]]))
                c.extend(ints([x]), ints([seqs[bounds[-1] + i]]))
        c.free(ints([firsts[g]]))
        bounds.append(bounds[-1] + len(o))
    c.check()
    return c, seqs, bounds


def rows_of(c, seq, layer=0):
    """K and V of a sequence, float64 [len, kv_heads, hd]."""
    n, page = int(c.lens[seq]), c.k.shape[2]
    at = c.table[seq, :-(-n // page)].long()
    return tuple(t[layer, at].flatten(0, 1)[:n].double().cpu().numpy() for t in (c.k, c.v))


def check(c, seqs, q, o, layer=0, scale=None):
    hd, bf16 = q.shape[2], q.dtype == BF
    scale = hd ** -0.5 if scale is None else scale
    qh, oh = q.double().cpu().numpy(), o.double().cpu().numpy()
    worst = 0.0
    for i, s in enumerate(seqs):
        if s < 0 or s >= c.max_seqs or int(c.lens[s]) == 0:
            assert not oh[i].any()
            continue
        k, v = rows_of(c, s, layer)
        worst = max(worst, A.check(oh[i:i + 1], qh[i:i + 1], k, v, np.ones((1, len(k)), bool), scale, bf16, i))
    return worst


CASES = [
    # shared, own, heads, kv_heads, hd, page, dtype, order
    ([64], [[1, 9, 32, 5]], 4, 4, 64, 16, F32, "token"),
    ([64], [[1, 9, 32, 5]], 4, 4, 64, 16, BF, "token"),
    ([1], [[1, 2]], 1, 1, 128, 1, BF, "token"),
    ([500], [[1, 300]], 3, 1, 128, 24, BF, "head"),
    ([700], [[1, 80, 17, 3, 200, 64, 33, 128]], 32, 8, 128, 16, BF, "token"),
    ([129], [[7] * 33], 16, 2, 64, 8, BF, "head"),
    ([260, 31, 1000], [[1, 2, 3], [40], [5] * 20], 14, 2, 128, 32, BF, "token"),
    ([260, 31, 1000], [[1, 2, 3], [40], [5] * 20], 6, 3, 64, 7, F32, "head"),
    ([300], [[3] * 40], 8, 1, 64, 64, F32, "token"),
    ([2000, 0, 130], [[1, None, 30], [5, 70, 2], [None, None, 4]], 20, 4, 128, 16, BF, "token"),
    ([1100], [[11] * 70], 8, 2, 128, 128, BF, "head"),
    ([5000], [[1, 2, 3, 4]], 16, 16, 128, 64, BF, "token"),
    ([900], [[2, 1]], 17, 1, 128, 16, BF, "token"),
    ([900, 600], [[2, 1] * 40, [3] * 30], 8, 2, 64, 256, BF, "token"),
    ([1030] * 9, [[2, 1, 3]] * 9, 28, 4, 128, 40, BF, "head"),
    ([100] * 40, [[2, 1]] * 40, 12, 4, 128, 8, BF, "token"),
    ([64, 47], [[0, 3, 0], [0, 0]], 4, 2, 128, 16, BF, "token"),  # as many tokens as are shared, and no more
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_64_bits(D, ws, case):
    shared, own, heads, kv_heads, hd, page, dtype, order = CASES[case]
    rng = np.random.default_rng(case)
    c, seqs, bounds = make(D, rng, shared, own, page, kv_heads, hd, dtype, order, layers=2)
    n = len(seqs)
    q = values(rng, (n, heads + 3, hd), dtype)[:, 1:1 + heads]
    o = c.prefix_attention(1, q, ws, ints(shared), ints(bounds), seqs=ints(seqs))
    assert check(c, seqs, q, o, 1) > 0
    c.check()
    ws.check()
    # the same bits again, in place, and whatever less of the prefix is named
    assert torch.equal(o, c.prefix_attention(1, q, ws, ints(shared), ints(bounds), seqs=ints(seqs)))
    for part in (0.5, 0.0, -1.0):
        mine = q.contiguous()
        got = c.prefix_attention(1, mine, ws, ints([int(s * part) for s in shared]), ints(bounds), seqs=ints(seqs), out=mine)
        assert got is mine
        check(c, seqs, q, got, 1)
    c.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_groups_that_do_not_fit_the_entries(D, ws, dtype):
    """Entries outside every group, empty groups, a group of one, sequences named twice or not at all."""
    rng = np.random.default_rng(77)
    c, seqs, _ = make(D, rng, [200], [[3, 30, 1, 4, 15, 9]], 16, 2, 64, dtype)
    q = values(rng, (9, 4, 64), dtype)
    named = seqs + [seqs[0], -1, 99]
    for bounds in ([0, 9], [2, 4], [0, 1, 1, 5], [0, 0, 9], [9, 9], [4, 9]):
        o = c.prefix_attention(0, q, ws, ints([200] * (len(bounds) - 1)), ints(bounds), seqs=ints(named))
        check(c, named, q, o)
        with pytest.raises(D.DinferError, match="status 0x1:"):
            c.check()
    for bounds in ([0, 6, 3, 9], [-2, 4], [0, 10], [5, 3]):
        o = c.prefix_attention(0, q, ws, ints([200] * (len(bounds) - 1)), ints(bounds), seqs=ints(named))
        check(c, named, q, o)
        with pytest.raises(D.DinferError, match="status 0x11:"):
            c.check()
    # without seqs and groups: the first entries, all of one group
    o = c.prefix_attention(0, q[:c.max_seqs], ws, ints([200]))
    check(c, list(range(c.max_seqs)), q[:c.max_seqs], o)


def test_a_sequence_without_the_groups_pages_is_flagged(D, ws):
    rng = np.random.default_rng(5)
    c, seqs, bounds = make(D, rng, [64, 64], [[3, 5], [4, 8]], 16, 2, 128)
    q = values(rng, (4, 4, 128), BF)
    c.prefix_attention(0, q, ws, ints([64]), seqs=ints(seqs))
    with pytest.raises(D.DinferError, match="status 0x1:"):
        c.check()
    c.prefix_attention(0, q, ws, ints([64, 64]), ints(bounds), seqs=ints(seqs))
    c.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_that_are_not_there_or_not_finite(D, ws, dtype):
    """Slots behind the last tokens hold NaN; an infinite value makes its column infinite however small its weight, a NaN one
    NaN; sums of large values whose mean is finite stay finite."""
    rng = np.random.default_rng(9)
    c, seqs, bounds = make(D, rng, [160], [[3, 30, 1, 4]], 16, 2, 128, dtype)
    page = 16
    used = torch.zeros(c.k.shape[1:3], dtype=torch.bool, device=dev)
    for s in seqs:
        n = int(c.lens[s])
        j = torch.arange(n, device=dev)
        used[c.table[s, j // page].long(), j % page] = True
    for t in (c.k, c.v):
        t[0][~used] = float("nan")
    q = values(rng, (4, 6, 128), dtype)
    args = (ws, ints([160]), ints(bounds))
    o = c.prefix_attention(0, q, *args, seqs=ints(seqs))
    check(c, seqs, q, o)
    first = int(c.table[seqs[0], 0])
    own = int(c.table[seqs[1], 11])
    keep = c.v.clone()
    c.v[0, first, 3, 0, 5] = float("inf")
    c.v[0, first, 4, 1, 6] = float("nan")
    c.v[0, own, 2, 0, 7] = float("-inf")
    c.k[0, first, 3, 0] = -300.0 * q[0, 0].sign()  # the weight of the first one underflows for the first query
    o = c.prefix_attention(0, q, *args, seqs=ints(seqs)).float()
    assert bool(torch.isinf(o[:, :3, 5]).all()) and bool((o[:, :3, 5] > 0).all())
    assert bool(torch.isnan(o[:, 3:, 6]).all())
    assert bool((o[1, :3, 7] == float("-inf")).all()) and bool(torch.isfinite(o[[0, 2, 3], :3, 7]).all())
    rest = torch.ones(4, 6, 128, dtype=torch.bool, device=dev)
    rest[:, :3, 5] = rest[:, 3:, 6] = rest[1, :3, 7] = False
    assert bool(torch.isfinite(o[rest]).all())
    c.v.copy_(keep)
    c.v[0][used] = torch.sign(c.v[0][used]) * 3.0e38
    o = c.prefix_attention(0, q, *args, seqs=ints(seqs)).float()
    assert bool(torch.isfinite(o).all())
    c.k[0, first, 3, 0] = float("nan")  # a score that is NaN
    o = c.prefix_attention(0, q, *args, seqs=ints(seqs)).float()
    assert bool(torch.isnan(o[:, :3]).all()) and bool(torch.isfinite(o[:, 3:]).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_that_are_all_minus_infinity(D, ws, dtype):
    rng = np.random.default_rng(2)
    c, seqs, bounds = make(D, rng, [64], [[3, 5]], 16, 1, 64, dtype)
    c.k[..., 0] = float("-inf")
    q = values(rng, (2, 2, 64), dtype)
    q[..., 0] = 1.0
    o = c.prefix_attention(0, q, ws, ints([64]), seqs=ints(seqs))
    assert not bool(o.any())
    # only the shared ones, only the own ones
    c.k[0, c.table[seqs[0], 4].long(), 0] = 0.5
    o = c.prefix_attention(0, q, ws, ints([64]), seqs=ints(seqs))
    v = c.v[0, int(c.table[seqs[0], 4]), 0, 0]
    assert torch.equal(o[0], v.expand(2, 64)) and not bool(o[1].any())


def test_captured_while_the_sequences_grow(D, ws):
    rng = np.random.default_rng(3)
    c, seqs, bounds = make(D, rng, [300, 40], [[1, 2, 17, 4], [60, 3]], 16, 2, 128, spare=40)
    q = values(rng, (6, 8, 128), BF)
    out, prefix, b, sq = torch.empty_like(q), ints([300, 40]), ints(bounds), ints(seqs)
    k, v = values(rng, (6, 2, 128), BF), values(rng, (6, 2, 128), BF)
    rope = D.Rope(128)
    c.prefix_attention(0, q, ws, prefix, b, seqs=sq, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.extend(seqs=sq)
        c.append_rope(0, rope, k, v, seqs=sq)
        c.prefix_attention(0, q, ws, prefix, b, seqs=sq, out=out)
    for _ in range(5):
        q.copy_(values(rng, q.shape, BF))
        g.replay()
        torch.cuda.synchronize()
        check(c, seqs, q, out)
    c.check()


def test_beside_the_attention_that_shares_nothing(D, ws):
    """64 sequences of a long prompt: both attentions, within both bounds of one another."""
    rng = np.random.default_rng(4)
    own = [int(x) for x in rng.integers(1, 200, 64)]
    c, seqs, bounds = make(D, rng, [3000], [own], 16, 8, 128)
    q = values(rng, (64, 32, 128), BF)
    a = c.prefix_attention(0, q, ws, ints([3000]), seqs=ints(seqs)).float()
    b = c.attention(0, q, ws, seqs=ints(seqs)).float()
    assert float((a - b).abs().max()) < 2.0 ** -6 * float(b.abs().max())
    some = [0, 13, 40, 63]
    check(c, [seqs[i] for i in some], q[some], a[some])
