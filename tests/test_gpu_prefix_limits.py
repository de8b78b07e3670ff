"""Attention over shared prefixes at its limits: what it keeps of a weight, in every form that a call can take, and the
workspaces that it takes."""
import numpy as np
import pytest
import torch

from tests import attention64 as A
from tests import test_gpu_prefix_attention as PA

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
BF = torch.bfloat16
KEPT = 2.0 ** -16  # of a bf16 weight, held as two bf16 (tests/attention64.py)


@pytest.fixture(scope="module")
def D():
    from block_denoising_gb300 import build, dinfer
    build.build()
    return dinfer


@pytest.fixture(scope="module")
def ws(D):
    return D.OpWorkspace()


def rounded(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(BF).double().numpy()


def put(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(BF).to(dev)


# one piece of 16 rows; one tile of rows on every other key tile; two tiles; more than a unit
@pytest.mark.parametrize("members,group", [(2, 8), (5, 8), (16, 8), (19, 8), (40, 8), (3, 19)])
@pytest.mark.parametrize("hd,page", [(64, 16), (128, 16), (128, 24), (64, 128)])
def test_prefix_weights_in_two_bf16(D, ws, hd, page, members, group):
    # sums that nearly cancel: a weight that lost more shows (one bf16 alone is beyond this bound, tests/test_attention64.py)
    for n in (140, 430, 2200):
        rng = np.random.default_rng(hd + page + n)
        c, seqs, bounds = PA.make(D, rng, [n - 7], [[7] * members], page, 1, hd)
        q, k, v = A.cancelling(rng, n, hd, group, rounded)
        for s in seqs:
            j = torch.arange(n, device=dev)
            at = c.table[s, j // page].long(), j % page
            c.k[0][at[0], at[1], 0], c.v[0][at[0], at[1], 0] = put(k), put(v)
        x = put(np.broadcast_to(q, (members, group, hd)).copy())
        o = c.prefix_attention(0, x, ws, PA.ints([n - 7]), PA.ints(bounds), seqs=PA.ints(seqs), scale=1.0)
        some = [0, members // 2, members - 1]
        for i in some:
            A.check(o[i:i + 1].double().cpu().numpy(), q[None], k[:, None], v[:, None], np.ones((1, n), bool), 1.0, True, (n, i), KEPT)
        c.check()
        ws.check()


@pytest.mark.parametrize("case", [i for i, x in enumerate(PA.CASES) if x[6] is BF])
def test_plain_sums_within_what_is_kept(D, ws, case):
    shared, own, heads, kv_heads, hd, page, dtype, order = PA.CASES[case]
    rng = np.random.default_rng(case + 500)
    c, seqs, bounds = PA.make(D, rng, shared, own, page, kv_heads, hd, dtype, order)
    q = PA.values(rng, (len(seqs), heads, hd), dtype)
    o = c.prefix_attention(0, q, ws, PA.ints(shared), PA.ints(bounds), seqs=PA.ints(seqs))
    qh, oh = q.double().cpu().numpy(), o.double().cpu().numpy()
    for i in range(0, len(seqs), 1 + len(seqs) // 12):
        if int(c.lens[seqs[i]]) == 0:
            continue
        k, v = PA.rows_of(c, seqs[i])
        A.check(oh[i:i + 1], qh[i:i + 1], k, v, np.ones((1, len(k)), bool), hd ** -0.5, True, i, KEPT)


@pytest.mark.parametrize("hd,members", [(128, 40), (64, 40), (128, 5)])
def test_a_workspace_that_begins_at_16_bytes(D, ws, hd, members):
    rng = np.random.default_rng(hd + members)
    c, seqs, bounds = PA.make(D, rng, [1000], [[3] * members], 16, 2, hd)
    q = PA.values(rng, (members, 16, hd), BF)
    args = (PA.ints([1000]), PA.ints(bounds))
    want = c.prefix_attention(0, q, ws, *args, seqs=PA.ints(seqs))
    whole = torch.zeros(ws.nbytes + 32 + 64, dtype=torch.uint8, device=dev)
    off = -whole.data_ptr() % 32 + 16
    odd = D.OpWorkspace()
    odd.buf = whole[off:off + ws.nbytes]
    assert odd.buf.data_ptr() % 32 == 16
    whole[off + ws.nbytes:] = 77
    assert torch.equal(c.prefix_attention(0, q, odd, *args, seqs=PA.ints(seqs)), want)
    assert bool((whole[off + ws.nbytes:] == 77).all())
    c.check()
    odd.check()


@pytest.mark.parametrize("members,page,hd,dtype", [(2, 16, 128, BF), (12, 16, 128, BF), (12, 24, 64, BF), (40, 128, 128, BF), (40, 16, 64, BF), (5, 16, 64, torch.float32)])
def test_pages_that_are_none(D, ws, members, page, hd, dtype):
    """Table entries inside the shared and the own tokens that name no page: their keys are not there, for every member of
    the group, and the status says so."""
    rng = np.random.default_rng(members + page)
    shared, own = 6 * page, page + 5
    c, seqs, bounds = PA.make(D, rng, [shared], [[own] * members], page, 2, hd, dtype)
    q = PA.values(rng, (members, 8, hd), dtype)
    n, none = shared + own, {1: -1, 4: c.k.shape[1], 5: 1 << 30}
    keys = [PA.rows_of(c, s) for s in seqs]
    table = c.table.clone()
    for j, v in none.items():
        table[:, j] = v
    table[seqs[0], 6] = -7
    c.set_tables(table, c.lens.clone(), c.refs.clone())
    o = c.prefix_attention(0, q, ws, PA.ints([shared]), PA.ints(bounds), seqs=PA.ints(seqs))
    with pytest.raises(D.DinferError, match="status 0x4:"):
        c.check()
    for i in sorted({0, 1, members - 1}):
        seen = np.ones((1, n), bool)
        for j in list(none) + ([6] if i == 0 else []):
            seen[0, j * page:(j + 1) * page] = False
        A.check(o[i:i + 1].double().cpu().numpy(), q[i:i + 1].double().cpu().numpy(), *keys[i], seen, hd ** -0.5, dtype is BF, i,
                KEPT if dtype is BF else None)
    # no page at all: zeros
    table[:] = -1
    c.set_tables(table, c.lens.clone(), c.refs.clone())
    o = c.prefix_attention(0, q, ws, PA.ints([shared]), PA.ints(bounds), seqs=PA.ints(seqs))
    assert not bool(o.any())
    with pytest.raises(D.DinferError, match="status 0x4:"):
        c.check()
    ws.check()


# rows of a key head: one tile on every other key tile; two tiles; more than a unit
@pytest.mark.parametrize("members,hd,page", [(12, 128, 16), (12, 64, 24), (60, 128, 16), (60, 64, 16), (110, 128, 128)])
def test_values_that_are_not_finite_on_the_tensor_cores(D, ws, members, hd, page):
    """Infinite and NaN values touch their columns alone, however small their weight; a NaN key its rows; sums of large values
    whose mean is finite stay finite; slots behind the last tokens may hold anything."""
    rng = np.random.default_rng(members + hd)
    own = [int(x) for x in rng.integers(1, 60, members)]
    shared, heads, kv_heads = 560, 6, 2
    c, seqs, bounds = PA.make(D, rng, [shared], [own], page, kv_heads, hd)
    at = lambda s, t: (int(c.table[s, t // page]), t % page)  # noqa: E731
    used = torch.zeros(c.k.shape[1:3], dtype=torch.bool, device=dev)
    for s in seqs:
        j = torch.arange(int(c.lens[s]), device=dev)
        used[c.table[s, j // page].long(), j % page] = True
    for t in (c.k, c.v):
        t[0][~used] = float("nan")
    q = PA.values(rng, (members, heads, hd), BF)
    run = lambda: c.prefix_attention(0, q, ws, PA.ints([shared]), PA.ints(bounds), seqs=PA.ints(seqs)).float()  # noqa: E731
    some = [0, 1, members // 2, members - 1]
    clean = run()
    PA.check(c, [seqs[i] for i in some], q[some], clean[some].to(BF))
    keep_k, keep_v = c.k.clone(), c.v.clone()
    p0, t0 = at(seqs[0], 3)
    p1, t1 = at(seqs[0], 300)
    p2, t2 = at(seqs[1], shared + own[1] - 1)  # a token of its own of one member, or the last of the shared page it copied
    c.v[0, p0, t0, 0, 5] = float("inf")
    c.v[0, p1, t1, 1, 6] = float("nan")
    c.v[0, p2, t2, 0, 7] = float("-inf")
    c.k[0, p0, t0, 0] = -300.0 * q[0, 0].sign()  # its weight underflows for the first query
    o = run()
    g = heads // kv_heads
    want = torch.ones_like(o, dtype=torch.bool)
    want[:, :g, 5] = want[:, g:, 6] = want[1, :g, 7] = False
    assert torch.equal(torch.isfinite(o), want)
    assert bool((o[:, :g, 5] == float("inf")).all()) and bool((o[1, :g, 7] == float("-inf")).all())
    for i in some:  # rows with such a column are done again in another order: within the bound, not the same bits
        k, v = PA.rows_of(c, seqs[i])
        got = o[i:i + 1].double().cpu().numpy()
        v[~np.isfinite(v)] = 0.0
        got[:, :g, [5, 7]], got[:, g:, 6], v[:, 0, [5, 7]], v[:, 1, 6] = 0.0, 0.0, 0.0, 0.0
        A.check(got, q[i:i + 1].double().cpu().numpy(), k, v, np.ones((1, len(k)), bool), hd ** -0.5, True, i, KEPT)
    c.v.copy_(keep_v)
    c.k.copy_(keep_k)
    c.v[0][used] = torch.sign(c.v[0][used]) * 3.0e38
    o = run()
    assert bool(torch.isfinite(o).all()) and float(o.abs().max()) <= 3.4e38
    c.v.copy_(keep_v)
    c.k[0, p1, t1, 0] = float("nan")
    o = run()
    assert bool(torch.isnan(o[:, :g]).all()) and torch.equal(o[:, g:], clean[:, g:])
    # scores of -inf: of all shared keys, of all keys
    c.k.copy_(keep_k)
    first = q[..., 0].clone()
    q[..., 0] = 1.0
    j = torch.arange(shared // page * page, device=dev)
    c.k[0, c.table[seqs[0], j // page].long(), j % page, :, 0] = float("-inf")
    o = run()
    for i in some:
        k, v = PA.rows_of(c, seqs[i])
        seen = np.isfinite(k[:, 0, 0])[None]
        assert seen.sum() < shared
        k[~seen[0]] = 0.0
        A.check(o[i:i + 1].double().cpu().numpy(), q[i:i + 1].double().cpu().numpy(), k, v, seen, hd ** -0.5, True, i, KEPT)
    c.k[0, ..., 0] = float("-inf")
    assert not bool(run().any())
    q[..., 0] = first
    ws.check()
