"""The paged KV cache on the GPU: its pages against a plain-Python model, its attention against 64 bits.

Page contents are only moved, so they are compared bit for bit, as are the tables.  The attention's bound
(tests/attention64.py) is derived from the kernels' arithmetic for every output element.
"""
import numpy as np
import pytest
import torch

from tests import attention64 as A
from tests.paged_model import Model

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


def values(rng, shape, dtype):
    """Normal values that the type holds exactly: (float64 array, device tensor)."""
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)
    return t.double().numpy(), t.to(dev)


def make(D, rng, layers, pages, page, heads, hd, seqs, most, dtype=torch.bfloat16, order="token"):
    """A cache without sequences whose pages hold values already, and its model."""
    shape = (layers, pages, page, heads, hd)
    model = Model(np.zeros(shape), np.zeros(shape), seqs, most)
    kv = []
    for name in ("k", "v"):
        x, t = values(rng, shape, dtype)
        setattr(model, name, x.copy())
        kv.append(t if order == "token" else t.transpose(2, 3).contiguous().transpose(2, 3))
    cache = D.PagedKV(kv[0], kv[1], torch.full((seqs, most), -1, dtype=torch.int32, device=dev),
                      torch.zeros(seqs, dtype=torch.int32, device=dev), torch.zeros(pages, dtype=torch.int32, device=dev))
    return cache, model


def same(cache, model):
    torch.cuda.synchronize()
    assert np.array_equal(cache.lens.cpu().numpy(), model.lens)
    assert np.array_equal(cache.table.cpu().numpy(), model.table)
    assert np.array_equal(cache.refs.cpu().numpy(), model.refs)
    assert np.array_equal(cache.k.double().cpu().numpy(), model.k)
    assert np.array_equal(cache.v.double().cpu().numpy(), model.v)


def status(D, cache):
    try:
        cache.check()
    except D.DinferError as e:
        assert e.status == D.EDEVICE
        return int(str(e).split("status 0x")[1].split(":")[0], 16)
    return 0


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("page,heads,hd,dtype,order", [
    (16, 2, 64, torch.bfloat16, "token"),
    (16, 2, 64, torch.bfloat16, "head"),
    (1, 1, 128, torch.bfloat16, "token"),
    (24, 3, 128, torch.float32, "head"),
    (7, 5, 64, torch.float32, "token"),
    (128, 8, 128, torch.bfloat16, "token"),
])
def test_random_page_calls_follow_the_model(D, page, heads, hd, dtype, order):
    rng = np.random.default_rng(page * 131 + heads)
    cache, model = make(D, rng, 2, 40, page, heads, hd, 12, 9, dtype, order)
    for step in range(60):
        n = int(rng.integers(1, 5))
        seqs = [int(s) for s in rng.choice(12, n, replace=False)]
        op = rng.integers(0, 10)
        if op < 4:
            add = [int(x) for x in rng.integers(0, 3 * page + 2, n)]
            cache.extend(ints(add), ints(seqs))
            was = model.lens.copy()
            model.extend(seqs, add)
            grown = [int(model.lens[s] - was[s]) for s in seqs]
            counts = [min(g, 40) for g in grown]
            if sum(counts):
                xk, tk = values(rng, (sum(counts), heads, hd), dtype)
                xv, tv = values(rng, (sum(counts), heads, hd), dtype)
                rows = ints([0] + list(np.cumsum(counts)))
                for layer in range(2):
                    cache.append(layer, tk, tv, rows=rows, seqs=ints(seqs))
                    model.append(layer, seqs, counts, xk, xv)
        elif op < 7:
            dst = [int(s) for s in rng.choice(12, n, replace=False)]
            share = bool(rng.integers(0, 2))
            cache.fork(ints(seqs), ints(dst), share=share)
            model.fork(seqs, dst, share)
        elif op < 9:
            cache.free(ints(seqs))
            model.free(seqs)
        else:
            live = torch.zeros(1, dtype=torch.int32, device=dev)
            cache.compact(live)
            assert model.compact() == int(live)
        same(cache, model)
        assert status(D, cache) == model.status, step
        model.status = 0


def test_skipped_entries_are_flagged_and_left_alone(D):
    rng = np.random.default_rng(5)
    cache, model = make(D, rng, 1, 10, 8, 1, 64, 6, 4)
    for call, bit in (
        (lambda c: c.extend(ints([3, 4]), ints([1, 1])), 1),         # the same sequence twice: its first entry
        (lambda c: c.extend(ints([3, 4, 5]), ints([-1, 6, 2])), 1),  # out of range
        (lambda c: c.extend(ints([-1]), ints([2])), 1),
        (lambda c: c.extend(ints([33]), ints([3])), 16),             # more than max_pages
        (lambda c: c.fork(ints([2, 2]), ints([3, 3])), 1),           # one destination twice
        (lambda c: c.fork(ints([2]), ints([1])), 1),                 # a destination in use
        (lambda c: c.fork(ints([2, 9]), ints([-4, 4])), 1),
        (lambda c: c.free(ints([6, -1])), 1),
        (lambda c: c.extend(ints([30, 30, 20]), ints([4, 5, 0])), 2),  # the pages run out: 4 + 4 + 3 of 7
        (lambda c: c.append(0, *[torch.zeros(40, 1, 64, dtype=torch.bfloat16, device=dev)] * 2, rows=ints([0, 40]),
                            seqs=ints([1])), 16),                    # more rows than tokens: the last ones are stored
        (lambda c: c.append(0, *[torch.zeros(2, 1, 64, dtype=torch.bfloat16, device=dev)] * 2, seqs=ints([3, 3])), 1),
    ):
        call(cache)
        assert status(D, cache) == bit
    torch.cuda.synchronize()
    assert cache.lens.tolist() == [0, 3, 5, 5, 30, 0]
    assert int((cache.refs > 0).sum()) == 1 + 1 + 1 + 4
    # rows for a page that two sequences hold
    cache.free(ints([0, 1, 2, 3, 4]))
    cache.extend(ints([8]), ints([0]))
    cache.fork(ints([0]), ints([1]))
    before = cache.k.clone()
    ones = torch.ones(8, 1, 64, dtype=torch.bfloat16, device=dev)
    cache.append(0, ones, ones, rows=ints([0, 8]))
    assert status(D, cache) == 8
    assert torch.equal(before, cache.k)


def test_another_set_of_tables(D):
    rng = np.random.default_rng(27)
    cache, model = make(D, rng, 1, 4000, 4, 1, 64, 300, 50)
    add = [int(x) for x in rng.integers(0, 60, 200)]
    cache.extend(ints(add))
    model.extend(range(200), add)
    old = [t.clone() for t in (cache.table, cache.lens, cache.refs)]
    cache.extend(ints([7, 7]), ints([250, 250]))
    cache.free(ints([0, 3, 900]))
    for form in (lambda t: t, lambda t: t.cpu(), lambda t: t.long(), lambda t: torch.stack([t, t], -1)[..., 0]):
        cache.set_tables(*(form(t) for t in old))
        assert status(D, cache) == 0
        same(cache, model)
        cache.extend(ints([3, 70]), ints([250, 1]))
        cache.free(ints([2, -1]))
    cache.set_tables(*old)
    cache.extend(ints([5, 9]), ints([250, 299]))
    model.extend([250, 299], [5, 9])
    same(cache, model)
    with pytest.raises(ValueError):
        cache.set_tables(old[0][:5], old[1], old[2])


def test_append_one_row_each_and_strided_rows(D):
    rng = np.random.default_rng(6)
    for page, heads, hd, dtype in ((16, 4, 128, torch.bfloat16), (5, 3, 64, torch.float32)):
        cache, model = make(D, rng, 2, 64, page, heads, hd, 20, 12, dtype)
        add = [int(x) for x in rng.integers(1, 3 * page, 20)]
        cache.extend(ints(add))
        model.extend(range(20), add)
        x, t = values(rng, (20, (2 * heads + 4) * hd), dtype)  # slices of one projection's output
        cut = lambda y, a: y[:, a * hd:(a + heads) * hd].reshape(20, heads, hd)  # noqa: E731
        seqs = [int(s) for s in rng.permutation(20)]
        cache.append(1, t[:, 4 * hd:(4 + heads) * hd].unflatten(1, (heads, hd)),
                     t[:, (4 + heads) * hd:].unflatten(1, (heads, hd)), seqs=ints(seqs))
        model.append(1, seqs, [1] * 20, cut(x, 4), cut(x, 4 + heads))
        same(cache, model)
        assert status(D, cache) == 0


def test_append_leaves_rows_behind_the_last_sequence(D):
    rng = np.random.default_rng(7)
    cache, model = make(D, rng, 1, 8, 16, 2, 64, 3, 4)
    cache.extend(ints([20, 3, 1]))
    model.extend([0, 1, 2], [20, 3, 1])
    x, t = values(rng, (50, 2, 64), torch.bfloat16)
    cache.append(0, t, t, rows=ints([0, 19, 19, 20]))  # an empty entry, and 30 rows of nobody
    model.append(0, [0, 1, 2], [19, 0, 1], x, x)
    same(cache, model)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def filled(D, rng, lens, page, heads, hd, dtype, order="token", layers=1):
    """A cache whose sequences hold `lens` tokens on scattered pages; every other slot holds NaN."""
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 3
    at = rng.permutation(pages)
    table = np.full((len(lens), max(held + [1])), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    k = np.full((layers, pages, page, heads, hd), np.nan)
    v = k.copy()
    used, seqs = 0, []
    for s, n in enumerate(lens):
        table[s, :held[s]] = at[used:used + held[s]]
        refs[at[used:used + held[s]]] = 1
        used += held[s]
        xs = []
        for c in (k, v):
            x, _ = values(rng, (layers, n, heads, hd), dtype)
            p = np.arange(n)
            c[:, table[s, p // page], p % page] = x
            xs.append(x)
        seqs.append(xs)
    put = lambda c: torch.from_numpy(c.astype(np.float32)).to(dtype).to(dev)  # noqa: E731
    kt, vt = put(k), put(v)
    if order == "head":
        kt, vt = (t.transpose(2, 3).contiguous().transpose(2, 3) for t in (kt, vt))
    return D.PagedKV(kt, vt, ints(table), ints(lens), ints(refs)), seqs


def run(cache, ws, rng, seqs, group, layer=0, window=-1, sinks=0, scale=None, order=None, strided=False):
    dtype, hd, kvh = cache.k.dtype, cache.head_dim, cache.kv_heads
    n, heads = len(seqs), kvh * group
    x, t = values(rng, (n, heads + (3 if strided else 0), hd), dtype)
    order = list(range(n)) if order is None else order
    got = cache.attention(layer, t[:, :heads], ws, window=window, sinks=sinks, scale=scale,
                          seqs=None if order == list(range(n)) else ints(order))
    torch.cuda.synchronize()
    scale = hd ** -0.5 if scale is None else scale
    for i, s in enumerate(order):
        k, v = (c[layer] for c in seqs[s])
        seen = A.window_mask(1, len(k), window, 0, sinks) if len(k) else np.zeros((1, 0), bool)
        A.check(got[i:i + 1].double().cpu().numpy(), x[i:i + 1, :heads], k, v, seen, scale, dtype == torch.bfloat16,
                (i, len(k)))
    return t[:, :heads], got


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 200]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd,heads,group,page,order", [
    (128, 2, 1, 16, "token"),
    (128, 2, 4, 24, "head"),
    (64, 3, 7, 1, "token"),
    (64, 1, 17, 128, "head"),   # more query heads than one tile takes
    (128, 1, 9, 5, "token"),
])
def test_attention_lengths_layouts_groups(D, ws, dtype, hd, heads, group, page, order):
    rng = np.random.default_rng(hd + group)
    cache, seqs = filled(D, rng, LENS, page, heads, hd, dtype, order)
    run(cache, ws, rng, seqs, group)
    run(cache, ws, rng, seqs, group, order=[int(s) for s in rng.permutation(len(LENS))], strided=True, scale=0.3)
    assert status(D, cache) == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (1, 0), (16, 4), (63, 0), (64, 1), (100, 130), (5000, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_windows_and_sinks(D, ws, dtype, window, sinks):
    rng = np.random.default_rng(window + sinks)
    cache, seqs = filled(D, rng, LENS + [700], 16, 2, 64, dtype)
    run(cache, ws, rng, seqs, 3, window=window, sinks=sinks)


@pytest.mark.parametrize("lens", [[5000], [4000, 1, 900, 0, 2500], [64] * 40, [1] * 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_split_over_the_length_and_joined(D, ws, dtype, lens):
    rng = np.random.default_rng(len(lens))
    cache, seqs = filled(D, rng, lens, 32, 2, 128, dtype)
    q, a = run(cache, ws, rng, seqs, 2)
    for _ in range(3):  # the same bits every time, and the workspace's counters are left at zero
        assert torch.equal(cache.attention(0, q, ws), a)


def test_attention_of_peaked_and_infinite_scores(D, ws):
    # one key dominates by far; +-inf scores; scores of -inf alone
    rng = np.random.default_rng(3)
    for dtype in (torch.bfloat16, torch.float32):
        cache, seqs = filled(D, rng, [300, 300, 300], 16, 1, 64, dtype)
        k, v = seqs[0]
        k[0, 137] *= 40
        p = cache.table[0, 137 // 16]
        cache.k[0, p, 137 % 16] *= 40
        run(cache, ws, rng, seqs, 2)
        q = torch.ones(3, 2, 64, dtype=dtype, device=dev)
        cache.k[0, cache.table[1, 3], 5] = float("inf")   # a visible key of sequence 1
        cache.k[0, cache.table[2].long()] = float("-inf")  # all of sequence 2's
        o = cache.attention(0, q, ws)
        assert torch.isfinite(o[0]).all() and torch.isnan(o[1]).all() and (o[2] == 0).all()
        # the window leaves the infinite key of sequence 1 (position 53) out
        assert torch.isfinite(cache.attention(0, q, ws, window=100, sinks=53)[1]).all()


def test_attention_of_infinite_values(D, ws):
    # an infinite value that a token sees makes its column infinite, whatever its weight's bits; one behind the
    # sequence's end, or outside the window, does not touch it
    rng = np.random.default_rng(20)
    for dtype in (torch.bfloat16, torch.float32):
        cache, seqs = filled(D, rng, [200, 50], 16, 1, 128, dtype)
        for j, c, x in ((10, 3, float("inf")), (150, 7, float("-inf"))):
            cache.v[0, cache.table[0, j // 16], j % 16, 0, c] = x
        q = values(rng, (2, 16, 128), dtype)[1]
        o = cache.attention(0, q, ws)
        assert (o[0, :, 3] == float("inf")).all() and (o[0, :, 7] == float("-inf")).all()
        finite = torch.isfinite(o)
        assert int((~finite).sum()) == 32 and finite[1].all()
        o = cache.attention(0, q, ws, window=100, sinks=5)
        assert (o[0, :, 7] == float("-inf")).all() and int((~torch.isfinite(o)).sum()) == 16


def test_attention_bad_entries_are_flagged(D, ws):
    rng = np.random.default_rng(4)
    cache, seqs = filled(D, rng, [40, 40, 40], 16, 1, 64, torch.bfloat16)
    x, q = values(rng, (3, 2, 64), torch.bfloat16)
    out = cache.attention(0, q, ws, seqs=ints([0, 7, -1]))
    assert status(D, cache) == 1
    assert (out[1:] == 0).all() and torch.equal(out[:1], cache.attention(0, q[:1], ws))
    for bad in (-1, 1 << 20):  # the second page of sequence 1 is none: its keys are left out
        cache.table[1, 1] = bad
        out = cache.attention(0, q, ws)
        assert status(D, cache) == 4
        seen = np.r_[np.ones(16, bool), np.zeros(16, bool), np.ones(8, bool)][None]
        A.check(out[1:2].double().cpu().numpy(), x[1:2], *[c[0] for c in seqs[1]], seen, 64 ** -0.5, True)


def test_calls_on_another_stream_and_in_a_graph(D, ws):
    rng = np.random.default_rng(8)
    cache, model = make(D, rng, 1, 40, 16, 2, 64, 3, 10)
    cache.extend(ints([30, 1, 15]))
    model.extend([0, 1, 2], [30, 1, 15])
    xq, q = values(rng, (3, 4, 64), torch.bfloat16)
    xn, new = values(rng, (3, 2, 64), torch.bfloat16)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def step():
        cache.extend()
        cache.append(0, new, new)
        cache.attention(0, q, ws, window=20, sinks=2, out=out)

    def follow():
        model.extend([0, 1, 2], [1, 1, 1])
        model.append(0, [0, 1, 2], [1, 1, 1], xn, xn)
        same(cache, model)
        for s in range(3):
            k, v = model.sequence(0, s)
            A.check(out[s:s + 1].double().cpu().numpy(), xq[s:s + 1], k, v, A.window_mask(1, len(k), 20, 0, 2), 0.125, True)

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    follow()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(40):  # each replay is a token more; pages are handed out inside the graph
        graph.replay()
        follow()
    assert status(D, cache) == 0


def test_a_thousand_sequences(D, ws):
    rng = np.random.default_rng(21)
    cache, model = make(D, rng, 1, 4500, 4, 1, 64, 1024, 6)
    add = [int(x) for x in rng.integers(0, 21, 700)]
    model.extend(range(700), add)
    cache.extend(ints(add))
    xk, k = values(rng, (sum(add) + 3, 1, 64), torch.bfloat16)
    xv, v = values(rng, (sum(add) + 3, 1, 64), torch.bfloat16)
    rows = ints(np.cumsum([0] + add))
    cache.append(0, k, v, rows=rows)
    model.append(0, range(700), add, xk, xv)
    src, dst = [int(x) for x in rng.integers(0, 700, 324)], list(range(700, 1024))
    for share in (True, False):
        cache.fork(ints(src), ints(dst), share=share)
        model.fork(src, dst, share)
        same(cache, model)
        gone = dst if share else [int(x) for x in rng.permutation(1024)[:500]]
        cache.free(ints(gone))
        model.free(gone)
    cache.compact()
    model.compact()
    same(cache, model)
    xq, q = values(rng, (1024, 2, 64), torch.bfloat16)
    out = cache.attention(0, q, ws).double().cpu().numpy()
    assert status(D, cache) == 0
    for s in range(0, 1024, 9):
        mk, mv = model.sequence(0, s)
        A.check(out[s:s + 1], xq[s:s + 1], mk, mv, np.ones((1, len(mk)), bool), 0.125, True)


def test_a_sequence_twice_many_heads_and_in_place(D, ws):
    rng = np.random.default_rng(22)
    for dtype, hd in ((torch.bfloat16, 128), (torch.float32, 64)):
        cache, seqs = filled(D, rng, [700, 5, 3000, 0], 16, 1, hd, dtype)
        order = [2, 0, 2, 2, 3, 1, 2]
        x, q = values(rng, (len(order), 300, hd), dtype)  # 300 query heads on one key head
        out = cache.attention(0, q, ws, seqs=ints(order))
        for i in (0, 1, 3, 6):
            k, v = (c[0] for c in seqs[order[i]])
            A.check(out[i:i + 1].double().cpu().numpy(), x[i:i + 1], k, v, np.ones((1, len(k)), bool), hd ** -0.5,
                    dtype == torch.bfloat16)
        assert cache.attention(0, q, ws, seqs=ints(order), out=q) is q
        assert torch.equal(q, out)


def test_two_calls_at_once(D, ws):
    rng = np.random.default_rng(23)
    cache, _ = filled(D, rng, [5000, 1, 900, 40], 16, 2, 128, torch.bfloat16)
    _, q = values(rng, (4, 8, 128), torch.bfloat16)
    other, side = D.OpWorkspace(), torch.cuda.Stream()
    want = [cache.attention(0, q, ws), cache.attention(0, q, ws, window=700, sinks=3)]
    torch.cuda.synchronize()
    for _ in range(30):
        a = cache.attention(0, q, ws)
        with torch.cuda.stream(side):
            b = cache.attention(0, q, other, window=700, sinks=3)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_forks_and_compaction_captured_in_a_graph(D):
    rng = np.random.default_rng(9)
    cache, model = make(D, rng, 2, 30, 8, 2, 64, 6, 6)
    cache.extend(ints([40, 12]))
    model.extend([0, 1], [40, 12])
    src, dst, gone = ints([0, 1]), ints([3, 4]), ints([3, 4, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.fork(src, dst)
        cache.free(gone)
        cache.compact()
        cache.fork(src[1:], dst[:1], share=False)
        cache.free(dst)
    for _ in range(3):
        graph.replay()
        model.fork([0, 1], [3, 4], True)
        model.free([3, 4, 0])
        model.compact()
        model.fork([1], [3], False)
        model.free([3, 4])
        same(cache, model)


def test_offsets_beyond_32_bits(D, ws):
    # 2.2e9 elements a tensor: the last pages lie beyond 2^31 elements and 2^32 bytes
    pages, page, heads, hd = 17000, 128, 8, 128
    k = torch.empty((1, pages, page, heads, hd), dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    rng = np.random.default_rng(10)
    table = np.array([[16999, 3, 16990], [16998, 16997, -1]], np.int32)
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    refs[torch.from_numpy(table[table >= 0]).long().to(dev)] = 1
    cache = D.PagedKV(k, v, ints(table), ints([300, 256]), refs)
    xs = []
    for n in (300, 256):
        xs.append([values(rng, (n, heads, hd), torch.bfloat16) for _ in range(2)])
    cache.append(0, torch.cat([x[0][1] for x in xs]), torch.cat([x[1][1] for x in xs]), rows=ints([0, 300, 556]))
    run(cache, ws, rng, [[x[0][0][None], x[1][0][None]] for x in xs], 1)
    cache.compact()
    torch.cuda.synchronize()
    assert sorted(cache.table[0].tolist() + cache.table[1].tolist()[:2]) == [0, 1, 2, 3, 4]
    run(cache, ws, rng, [[x[0][0][None], x[1][0][None]] for x in xs], 1)
    assert status(D, cache) == 0
