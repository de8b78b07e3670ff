"""The paged KV cache and windowed attention at the ends of their ranges: sums beyond 2^31, very long pieces of work,
values near the type's largest, weights near its smallest,
and what is kept of a weight."""
import numpy as np
import pytest
import torch

from tests import attention64 as A

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")


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


def status(D, cache):
    try:
        cache.check()
    except D.DinferError as e:
        assert e.status == D.EDEVICE
        return int(str(e).split("status 0x")[1].split(":")[0], 16)
    return 0


@pytest.mark.parametrize("most,add", [(1 << 21, [5] + [1 << 21] * 1022 + [0]), (1 << 30, [5] + [1 << 30] * 4 + [3, 2])])
def test_wants_that_add_up_beyond_32_bits(D, most, add):
    # the first entry alone finds pages; the sums of the others pass 2^31, and 2^32 back to small numbers
    n = len(add)
    cache = D.PagedKV.empty(layers=1, pages=64, page_size=1, kv_heads=1, head_dim=64, max_seqs=n, max_pages=most)
    cache.extend(ints(add))
    assert status(D, cache) == D.KV_NO_PAGES
    assert cache.lens.tolist() == [5] + [0] * (n - 1)
    assert cache.refs.tolist() == [1] * 5 + [0] * 59
    assert cache.table[0, :6].tolist() == [0, 1, 2, 3, 4, -1]
    assert int((cache.table[0] >= 0).sum()) == 5 and not any(int(cache.table[s].max()) >= 0 for s in range(1, n))
    # forks of one long sequence likewise (its row names no pages behind the fifth; nobody is served, nothing is read)
    cache.lens[0] = most
    cache.state.zero_()
    cache.fork(ints([0] * (n - 1)), ints(range(1, n)), share=False)
    assert status(D, cache) == D.KV_NO_PAGES
    assert cache.lens.tolist() == [most] + [0] * (n - 1) and int(cache.refs.sum()) == 5


def far_keys(n, dtype, hd=64):
    """n keys of zeros of which the 40 last, 5 early and 5 middle ones hold values, and a query row that scores these
    at 80 and more where a key of zeros scores 0: the others' weights add up to n e^-80 < 1e-25.  Keys are values too."""
    rng = np.random.default_rng(n % 1000)
    at = np.r_[3:8, n // 2:n // 2 + 5, n - 40:n]
    x = rng.standard_normal((len(at), hd))
    x[:, 0] = 8.0
    q = np.zeros((1, hd))
    q[0, 0], q[0, 1:] = 12.0, rng.standard_normal(hd - 1) * 0.1
    x, q = (torch.from_numpy(t.astype(np.float32)).to(dtype) for t in (x, q))
    k = torch.zeros((n, 1, hd), dtype=dtype, device=dev)
    k[torch.from_numpy(at).to(dev), 0] = x.to(dev)
    x, xq = x.double().numpy(), q.double().numpy()
    assert (x @ xq[0]).min() > 80
    return q.to(dev)[:, None], k, xq[:, None], x[:, None]


def test_fp32_row_split_over_3e8_keys(D, ws):
    # 77 GB in 304 parts: part times key tiles passes 2^31
    q, k, xq, x = far_keys(300_000_000, torch.float32)
    o = D.op_window_attention(q, k, k, ws, scale=1.0)
    torch.cuda.synchronize()
    A.check(o.double().cpu().numpy(), xq, x, x, np.ones((1, len(x)), bool), 1.0, False)


# many rows of one tile; few rows over many keys, split; without a workspace nothing is split
SHAPES = [(torch.bfloat16, 128, 2, 200, 300), (torch.bfloat16, 64, 40, 130, 300), (torch.bfloat16, 128, 1, 5, 3000),
          (torch.float32, 64, 2, 200, 300), (torch.float32, 128, 40, 70, 200), (torch.float32, 64, 1, 5, 3000)]


@pytest.mark.parametrize("dtype,hd,heads,nq,nk", SHAPES)
def test_prompt_means_of_values_near_the_largest(D, ws, dtype, hd, heads, nq, nk):
    # sums of weights times values pass the type's range, the weighted means do not
    rng = np.random.default_rng(nk + heads)
    q, k = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dtype) for s in ((nq, heads, hd), (nk, 1, hd)))
    for low in (-3.3e38, 2.9e38):  # both signs; a mean near the largest value
        v = torch.from_numpy(rng.uniform(low, 3.3e38, (nk, 1, hd)).astype(np.float32)).to(dtype)
        o = D.op_window_attention(q.to(dev), k.to(dev), v.to(dev), ws, left=150, right=0, sinks=4)
        torch.cuda.synchronize()
        ws.check()
        pick = [0, 1, nq // 2, nq - 1]
        A.check(o[pick].double().cpu().numpy(), q[pick].double(), k.double(), v.double(), A.window_mask(nq, nk, 150, 0, 4)[pick],
                hd ** -0.5, dtype == torch.bfloat16)


@pytest.mark.parametrize("dtype,hd,heads,nq,nk", SHAPES)
def test_prompt_infinite_values_of_tiny_weight(D, ws, dtype, hd, heads, nq, nk):
    # a value that a row sees makes its column infinite though its weight is far below fp32's range, wherever the key
    # lies; the other columns are what the finite values give, and rows that do not see the key stay finite
    rng = np.random.default_rng(nk + hd)
    xq, xk = rng.standard_normal((nq, heads, hd)), rng.standard_normal((nk, 1, hd))
    xq[..., 0] = 8.0
    first, last = nk - nq, nk - nq + 3  # keys seen by every row, and by all but the first three
    xk[:, 0, 0] = 0.0
    xk[[first, last], 0, 0] = -400.0 / (hd ** -0.5)
    q, k, v = (torch.from_numpy(t.astype(np.float32)).to(dtype) for t in (xq, xk, rng.standard_normal((nk, 1, hd))))
    bad = v.clone()
    bad[first, 0, 3], bad[last, 0, 7] = float("inf"), float("-inf")
    o = D.op_window_attention(q.to(dev), k.to(dev), bad.to(dev), ws, left=-1, right=0).double().cpu().numpy()
    assert (o[:, :, 3] == np.inf).all()
    assert (o[3:, :, 7] == -np.inf).all() and np.isfinite(o[:3, :, 7]).all()
    rest = np.delete(np.arange(hd), [3, 7])
    assert np.isfinite(o[..., rest]).all()
    pick = [0, 2, 3, nq - 1]
    seen = A.window_mask(nq, nk, -1, 0, 0)[pick]
    for i, s in zip(pick, seen):
        for h in range(0, heads, 7):
            want, tol = A.attend(q[i, h].double().numpy(), k[:, 0].double().numpy(), v[:, 0].double().numpy(), s, hd ** -0.5,
                                 dtype == torch.bfloat16)
            assert (np.abs(o[i, h] - want) <= tol)[rest].all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_infinite_value_before_scores_that_rise(D, ws, dtype):
    # the infinite value comes first, with all the weight there is; the keys behind it take that away
    k = torch.zeros((64, 1, 64), dtype=dtype, device=dev)
    k[:, 0, 0] = torch.arange(64, device=dev) * 40.0
    v = torch.ones_like(k)
    v[0, 0, 5] = float("inf")
    q = torch.zeros((64, 2, 64), dtype=dtype, device=dev)
    q[..., 0] = 4.0
    o = D.op_window_attention(q, k, v, ws, right=0, scale=1.0)
    assert (o[:, :, 5] == float("inf")).all() and (o[:, :, :5] == 1).all() and (o[:, :, 6:] == 1).all()
    # scores of -inf alone give zeros, whatever the values
    k[:, 0, 0] = float("-inf")
    assert (D.op_window_attention(q, k, v, ws, right=0, scale=1.0) == 0).all()


def paged(D, keys, values, page=16, seed=0):
    """A cache of one layer that holds keys[s], values[s] [n, kv_heads, hd] on scattered pages; other slots hold NaN."""
    rng = np.random.default_rng(seed)
    held = [-(-len(k) // page) for k in keys]
    at = rng.permutation(sum(held) + 2)
    table, refs = torch.full((len(keys), max(held)), -1, dtype=torch.int32), torch.zeros(len(at), dtype=torch.int32)
    k, v = (torch.full((1, len(at), page, *keys[0].shape[1:]), float("nan"), dtype=keys[0].dtype) for _ in range(2))
    for s, h in enumerate(held):
        mine = torch.from_numpy(at[sum(held[:s]):sum(held[:s + 1])])
        table[s, :h], refs[mine] = mine.int(), 1
        p = torch.arange(len(keys[s]))
        k[0, mine[p // page], p % page], v[0, mine[p // page], p % page] = keys[s], values[s]
    return D.PagedKV(k.to(dev), v.to(dev), table.to(dev), ints([len(x) for x in keys]), refs.to(dev))


# one round of rows and several, whole pairs and ones joined over many CTAs
TOKENS = [(torch.bfloat16, 128, 3), (torch.bfloat16, 64, 8), (torch.bfloat16, 128, 17), (torch.bfloat16, 64, 11),
          (torch.float32, 64, 1), (torch.float32, 128, 2), (torch.float32, 64, 5), (torch.float32, 128, 12)]


@pytest.mark.parametrize("dtype,hd,group", TOKENS)
def test_token_means_of_values_near_the_largest(D, ws, dtype, hd, group):
    # as for prompts; in place, and with a page that is none among the keys
    rng = np.random.default_rng(hd + group)
    lens, kvh = [1, 40, 700, 6000], 2
    put = lambda x: torch.from_numpy(x.astype(np.float32)).to(dtype)  # noqa: E731
    q = put(rng.standard_normal((4, kvh * group, hd)))
    keys = [put(rng.standard_normal((n, kvh, hd))) for n in lens]
    for low in (-3.3e38, 2.9e38):
        vals = [put(rng.uniform(low, 3.3e38, (n, kvh, hd))) for n in lens]
        cache = paged(D, keys, vals)
        cache.table[1, 1] = 1 << 20
        for window, sinks in ((-1, 0), (300, 5)):
            seen = [A.window_mask(1, n, window, 0, sinks) for n in lens]
            seen[1][:, 16:32] = False
            o = cache.attention(0, q.to(dev), ws, window=window, sinks=sinks)
            assert status(D, cache) == D.KV_BAD_PAGE
            for s, n in enumerate(lens):
                A.check(o[s:s + 1].double().cpu().numpy(), q[s:s + 1].double(), keys[s].double(), vals[s].double(), seen[s],
                        hd ** -0.5, dtype == torch.bfloat16, (low, window, n))
            x = q.to(dev)
            assert torch.equal(cache.attention(0, x, ws, window=window, sinks=sinks, out=x), o)
            assert status(D, cache) == D.KV_BAD_PAGE


@pytest.mark.parametrize("dtype,hd,group", TOKENS)
def test_token_infinite_values_of_tiny_weight(D, ws, dtype, hd, group):
    rng = np.random.default_rng(hd + group)
    lens = [50, 5000]
    q = torch.from_numpy(rng.standard_normal((2, group, hd)).astype(np.float32)).to(dtype)
    q[..., 0] = 8.0
    keys = [torch.from_numpy(rng.standard_normal((n, 1, hd)).astype(np.float32)).to(dtype) for n in lens]
    clean = [torch.from_numpy(rng.standard_normal((n, 1, hd)).astype(np.float32)).to(dtype) for n in lens]
    vals = [v.clone() for v in clean]
    for k, v in zip(keys, vals):
        k[:, 0, 0] = 0.0
        k[[3, len(k) // 2], 0, 0] = -400.0 / (hd ** -0.5)
        v[3, 0, 3], v[len(k) // 2, 0, 7] = float("inf"), float("-inf")
    cache = paged(D, keys, vals)
    o = cache.attention(0, q.to(dev), ws).double().cpu().numpy()
    assert status(D, cache) == 0
    assert (o[:, :, 3] == np.inf).all() and (o[:, :, 7] == -np.inf).all()
    rest = np.delete(np.arange(hd), [3, 7])
    for s, n in enumerate(lens):
        for h in range(group):
            want, tol = A.attend(q[s, h].double().numpy(), keys[s][:, 0].double().numpy(), clean[s][:, 0].double().numpy(),
                                 np.ones(n, bool), hd ** -0.5, dtype == torch.bfloat16)
            assert (np.abs(o[s, h] - want) <= tol)[rest].all()
    # outside the window they touch nothing
    assert np.isfinite(cache.attention(0, q.to(dev), ws, window=20, sinks=3).double().cpu().numpy()).all()


@pytest.mark.parametrize("dtype,hd,group", TOKENS)
def test_token_large_value_without_weight(D, ws, dtype, hd, group):
    # keys whose weight is far below the smallest number add nothing, however large their (finite) values
    rng = np.random.default_rng(hd + group)
    lens = [50, 5000]
    put = lambda x: torch.from_numpy(x.astype(np.float32)).to(dtype)  # noqa: E731
    q = put(rng.standard_normal((2, group, hd)))
    q[..., 0] = 8.0
    keys = [put(rng.standard_normal((n, 1, hd))) for n in lens]
    vals = [put(rng.standard_normal((n, 1, hd))) for n in lens]
    for k, v in zip(keys, vals):
        k[:, 0, 0] = 0.0
        far = [1, 3, len(k) // 2, len(k) - 1]
        k[far, 0, 0] = -40.0 / (hd ** -0.5)
        v[far] = 3e38
    o = paged(D, keys, vals).attention(0, q.to(dev), ws).double().cpu().numpy()
    for s, n in enumerate(lens):
        A.check(o[s:s + 1], q[s:s + 1].double(), keys[s].double(), vals[s].double(), np.ones((1, n), bool), hd ** -0.5,
                dtype == torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_token_over_2147483647_keys(D, ws, dtype):
    # One page of one slot, held all the way along a table of 8.6 GB: every weight is the same, and the joins round weights
    # and outputs alike, each by 2^-24.  fp32 sums in a warp are exact (powers of two).  A tensor product of bf16 may cut
    # each of its terms off at the last place of the sum it is added to, 2^-23 of it: of N keys a warp (152 SMs, 8 warps:
    # 1.77e6) the j-th loses up to j 2^-23 of itself, N 2^-24 = 0.106 in the mean.  Then the output's own half step.
    n = 2 ** 31 - 1
    k = torch.ones((1, 1, 1, 1, 64), dtype=dtype, device=dev)
    v = (2.0 ** (torch.arange(64, device=dev) % 8) * (1 - 2 * (torch.arange(64, device=dev) % 2))).to(dtype).view(1, 1, 1, 1, 64)
    cache = D.PagedKV(k, v, torch.zeros((1, n), dtype=torch.int32, device=dev), ints([n]), ints([1]))
    q = torch.ones((1, 2, 64), dtype=dtype, device=dev)
    lost = 0.106 + 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -18
    for window, sinks in ((-1, 0), (n, 0), (2 ** 31 - 300, 100)):
        o = cache.attention(0, q, ws, window=window, sinks=sinks)
        assert status(D, cache) == 0
        assert (o.double() / v.double().view(64) - 1).abs().max() <= lost


def test_bf16_piece_that_lasts_seconds(D):
    # 3.6e8 keys of one row that no workspace lets split, some 3 s: the waits for its end outlast the limit of a wait
    # without progress (about a second)
    q, k, xq, x = far_keys(360_000_000, torch.bfloat16)
    o = torch.full_like(q, 7.0)
    st = D.lib().dinfer_op_window_attention(q.data_ptr(), k.data_ptr(), k.data_ptr(), o.data_ptr(), D.BF16, 1, None, None, 1, k.shape[0],
                                            1, 1, 64, 64, 64, 64, 64, -1, -1, 0, 1.0, None, 0,
                                            torch.cuda.current_stream().cuda_stream)
    assert st == D.OK
    torch.cuda.synchronize()
    A.check(o.double().cpu().numpy(), xq, x, x, np.ones((1, len(x)), bool), 1.0, True)


@pytest.mark.parametrize("hd,group", [(64, 3), (128, 8), (64, 11), (128, 16), (64, 1), (128, 19)])
def test_token_weights_in_two_bf16(D, ws, hd, group):
    # sums that nearly cancel, and plain ones: 2^-16 of a weight is lost, no more (tests/test_attention64.py: one part alone
    # is beyond this bound)
    rng = np.random.default_rng(hd + group)
    rounded = lambda x: torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()  # noqa: E731
    cases = [A.cancelling(rng, n, hd, group, rounded) for n in (5, 40, 130, 300)]
    cases += [tuple(rounded(rng.standard_normal(s)) for s in ((group, hd), (n, hd), (n, hd))) for n in (2, 33, 1500)]
    put = lambda x: torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    cache = paged(D, [put(k)[:, None] for _, k, _ in cases], [put(v)[:, None] for _, _, v in cases])
    q = put(np.stack([q for q, _, _ in cases]))
    o = cache.attention(0, q.to(dev), ws, scale=1.0)
    torch.cuda.synchronize()
    for s, (x, k, v) in enumerate(cases):
        A.check(o[s:s + 1].double().cpu().numpy(), x[None], k[:, None], v[:, None], np.ones((1, len(k)), bool), 1.0, True,
                (len(k),), 2.0 ** -16)


@pytest.mark.parametrize("rows,stored", [([0, 5, 7], [5, 2]), ([0, 5, 5], [5, 0]), ([2, 4, 7], [2, 3]), ([0, 5, 8], [5, 2]),
                                         ([0, 9, 9], None), ([0, 5, 3], None), ([-1, 2, 7], None), ([0, 5, 1 << 30], None)])
def test_row_bounds_of_append(D, rows, stored):
    # seven rows of k; bounds that name rows it does not have, or run backwards, set the status and touch no other sequence
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((7, 1, 64)).astype(np.float32)).to(dev)
    cache = D.PagedKV.empty(layers=1, pages=8, page_size=4, kv_heads=1, head_dim=64, max_seqs=3, max_pages=4, dtype=torch.float32)
    cache.k.zero_()
    cache.v.zero_()
    cache.extend(ints([9, 6, 5]))
    cache.append(0, x, x, rows=ints(rows), seqs=ints([0, 1]))
    bad = rows[0] < 0 or sorted(rows) != rows or rows[2] > 7
    assert status(D, cache) == (D.KV_FULL if bad else 0)
    assert not cache.k[0, cache.table[2, :2].long()].any()
    if not bad:
        for s, n in enumerate(stored):
            flat = cache.k[0, cache.table[s, :3 - s].long()].flatten(0, 1)[:9 - 3 * s]
            assert torch.equal(flat[len(flat) - n:], x[rows[s]:rows[s] + n]) and not flat[:len(flat) - n].any()


@pytest.mark.parametrize("share", [True, False])
def test_chained_forks_copy_what_was_there_before_the_call(D, share):
    cache = D.PagedKV.empty(layers=1, pages=12, page_size=4, kv_heads=1, head_dim=64, max_seqs=6, max_pages=4)
    cache.extend(ints([9, 3]))
    cache.fork(ints([0, 3, 1]), ints([3, 4, 5]), share=share)  # 3 is still empty: so is 4
    assert status(D, cache) == 0
    assert cache.lens.tolist() == [9, 3, 0, 9, 0, 3]
    assert (cache.table[4] == -1).all()
    cache.fork(ints([3]), ints([4]), share=share)  # a call each
    assert status(D, cache) == 0
    assert cache.lens.tolist() == [9, 3, 0, 9, 9, 3]
    held = [t[t >= 0].tolist() for t in cache.table]
    assert [len(h) for h in held] == [3, 1, 0, 3, 3, 1]
    assert cache.refs.tolist() == [sum(p in h for h in held) for p in range(12)]
    assert all((held[0][:2] == held[s][:2]) == share and held[0][2] != held[s][2] for s in (3, 4))


@pytest.mark.parametrize("dtype,hd,group", TOKENS)
def test_token_bad_values_touch_their_columns_alone(D, ws, dtype, hd, group):
    # NaN and infinities that a token sees, with and without a score; in place too.  The other columns are as before
    rng = np.random.default_rng(hd + group)
    lens = [1, 60, 3000, 17]
    put = lambda x: torch.from_numpy(x.astype(np.float32)).to(dtype)  # noqa: E731
    q = put(rng.standard_normal((4, group, hd)))
    keys, vals = ([put(rng.standard_normal((n, 1, hd))) for n in lens] for _ in range(2))
    clean = paged(D, keys, vals).attention(0, q.to(dev), ws)
    inf, nan = float("inf"), float("nan")
    for s, j, c, x in ((0, 0, 5, nan), (1, 7, 0, inf), (1, 50, 0, -inf), (1, 59, 9, -inf), (2, 0, hd - 1, nan), (2, 1500, 3, inf),
                       (2, 1501, 3, inf)):
        vals[s][j, 0, c] = x
    keys[3][:, 0, :] = 0.0
    keys[3][:, 0, 0] = -inf  # scores of -inf alone: zeros, whatever the values
    vals[3][4:9] = inf
    q[3, :, 0] = 1.0
    want = clean.clone()
    want[0, :, 5], want[1, :, 0], want[1, :, 9], want[2, :, hd - 1], want[2, :, 3], want[3] = nan, nan, -inf, nan, inf, 0.0
    cache = paged(D, keys, vals)
    for out in (None, q.to(dev)):
        o = cache.attention(0, q.to(dev) if out is None else out, ws, out=out)
        assert torch.equal(torch.isnan(o), torch.isnan(want)) and torch.equal(torch.isinf(o), torch.isinf(want))
        assert torch.equal(o[torch.isinf(o)], want[torch.isinf(want)])
        for s, n in enumerate(lens[:3]):
            bad = ~torch.isfinite(vals[s]).all(0)[0]
            v, got = vals[s].double(), o[s:s + 1].double().cpu()
            v[:, :, bad], got[..., bad] = 0.0, 0.0
            A.check(got.numpy(), q[s:s + 1].double(), keys[s].double(), v, np.ones((1, n), bool), hd ** -0.5,
                    dtype == torch.bfloat16)
        assert (o[3] == 0).all()
    # a NaN key makes the row NaN
    keys[1][3, 0, 2] = nan
    o = paged(D, keys, vals).attention(0, q.to(dev), ws)
    assert torch.isnan(o[1]).all() and torch.equal(torch.isnan(o[2]), torch.isnan(want[2])) and (o[3] == 0).all()
