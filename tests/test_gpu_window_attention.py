"""Prompt attention with a sliding window and sinks against 64 bits (bounds: tests/attention64.py)."""
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
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)
    return t.double().numpy(), t.to(dev)


def cum(v):
    return ints([0] + list(np.cumsum(v)))


def compare(got, xq, xk, xv, nq, nk, left, right, sinks, scale, bf16, rows=24):
    """Rows spread over each sequence (both ends, tile edges) against attend()."""
    a = b = 0
    for n, m in zip(nq, nk):
        if n:
            pick = sorted({0, n - 1, n // 2, *[i for i in (63, 64, 127, 128, 255, 256) if i < n],
                           *np.linspace(0, n - 1, rows).astype(int).tolist()})
            seen = A.window_mask(n, m, left, right, sinks)[pick]
            A.check(got[a:a + n][pick], xq[a:a + n][pick], xk[b:b + m], xv[b:b + m], seen, scale, bf16, (n, m))
        a, b = a + n, b + m


def run(D, ws, seed, nq, nk, heads, kv_heads, hd, dtype, left, right, sinks, scale=None, rows=24):
    rng = np.random.default_rng(seed)
    xq, q = values(rng, (sum(nq), heads, hd), dtype)
    xk, k = values(rng, (sum(nk), kv_heads, hd), dtype)
    xv, v = values(rng, (sum(nk), kv_heads, hd), dtype)
    one = len(nq) == 1
    o = D.op_window_attention(q, k, v, ws, cu_q=None if one else cum(nq), cu_k=None if one else cum(nk), left=left,
                              right=right, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    ws.check()
    compare(o.double().cpu().numpy(), xq, xk, xv, nq, nk, left, right, sinks, hd ** -0.5 if scale is None else scale,
            dtype == BF, rows)
    return q, k, v, o


MASKS = [(-1, 0, 0), (-1, -1, 0), (0, 0, 0), (5, 0, 2), (64, 64, 4), (127, 0, 130), (300, 20, 1), (-1, 7, 0), (40, -1, 3)]


@pytest.mark.parametrize("dtype,hd", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("left,right,sinks", MASKS)
def test_masks_over_ragged_sequences(D, ws, dtype, hd, left, right, sinks):
    nq = [1, 0, 17, 128, 300, 5, 129]
    nk = [1, 3, 17, 128, 300, 400, 100]  # more keys than rows, and fewer: rows before the first key
    run(D, ws, 7 + left + 2 * sinks, nq, nk, 2, 2, hd, dtype, left, right, sinks)


# enough heads for two tiles a CTA (of one head, of two), and for fp32 tiles of 16 rows from the last on, and of 64
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype,heads", [(BF, 14), (BF, 16), (F32, 14), (F32, 40)])
@pytest.mark.parametrize("left,right,sinks", MASKS)
def test_many_heads(D, ws, hd, dtype, heads, left, right, sinks):
    nq = [1, 0, 17, 128, 300, 5, 129]
    nk = [1, 3, 17, 128, 300, 400, 100]
    run(D, ws, 70 + left + 2 * sinks + heads, nq, nk, heads, 2, hd, dtype, left, right, sinks, rows=8)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads,kv_heads", [(6, 2), (4, 1), (7, 7), (5, 1)])
def test_grouped_heads(D, ws, dtype, heads, kv_heads):
    run(D, ws, heads, [70, 260], [70, 300], heads, kv_heads, 128, dtype, 90, 0, 4)
    run(D, ws, heads, [257], [257], heads, kv_heads, 64, dtype, -1, -1, 0)


@pytest.mark.parametrize("n", [1, 2, 31, 64, 65, 127, 128, 129, 255, 256, 257, 511, 700])
def test_lengths(D, ws, n):
    for dtype in (BF, F32):
        run(D, ws, n, [n], [n], 2, 1, 128, dtype, -1, 0, 0, rows=6)
        run(D, ws, n, [1], [n], 2, 1, 64, dtype, n // 2, 0, 1, rows=6)
    run(D, ws, n, [n], [n], 160, 2, 64, BF, -1, 0, 0, rows=2)
    run(D, ws, n, [n], [n], 153, 3, 128, BF, 100, 9, 1, rows=2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_sequence(D, ws, dtype):
    run(D, ws, 1, [3001], [3500], 2, 1, 128, dtype, 1000, 0, 4, rows=12)
    run(D, ws, 2, [2049], [2049], 1, 1, 64, dtype, -1, -1, 0, rows=12, scale=0.4)
    run(D, ws, 3, [3001], [3500], 8, 2, 128, dtype, 1000, 0, 4, rows=8)
    run(D, ws, 4, [3001], [3001], 7, 1, 64, dtype, -1, 0, 0, rows=8)


def test_strided_operands_and_rows_of_nobody(D, ws):
    rng = np.random.default_rng(11)
    for dtype in (BF, F32):
        H, KV, hd, T = 4, 2, 128, 333
        x, t = values(rng, (T, (H + 2 * KV) * hd), dtype)
        q, k, v = (t[:, a * hd:b * hd].unflatten(1, (b - a, hd)) for a, b in ((0, H), (H, H + KV), (H + KV, H + 2 * KV)))
        xq, xk, xv = (x[:, a * hd:b * hd].reshape(T, b - a, hd) for a, b in ((0, H), (H, H + KV), (H + KV, H + 2 * KV)))
        buf = torch.full((T, H + 1, hd), 7.0, dtype=dtype, device=dev)
        # sequences of 100 and 150 rows that begin at row 3; rows 0-2 and 253-332 belong to nobody
        cu = ints([3, 103, 253])
        D.op_window_attention(q, k, v, ws, cu_q=cu, cu_k=cu, left=60, right=60, sinks=3, out=buf[:, :H])
        torch.cuda.synchronize()
        got = buf.double().cpu().numpy()
        assert np.all(got[:3] == 7) and np.all(got[253:] == 7) and np.all(got[:, H] == 7)
        compare(got[3:253, :H], xq[3:253], xk[3:253], xv[3:253], [100, 150], [100, 150], 60, 60, 3, hd ** -0.5, dtype == BF)


@pytest.mark.parametrize("dtype,hd,heads", [(BF, 128, 2), (BF, 64, 2), (BF, 128, 40), (BF, 64, 39), (F32, 64, 2),
                                            (F32, 64, 40)])
def test_what_masked_keys_hold_does_not_matter(D, ws, dtype, hd, heads):
    # NaN and infinite keys and values touch the rows that see them and no other, tile neighbours included
    rng = np.random.default_rng(12)
    n, left, right, sinks = 500, 40, 10, 2
    xq, q = values(rng, (n, heads, hd), dtype)
    xk, k = values(rng, (n, 1, hd), dtype)
    xv, v = values(rng, (n, 1, hd), dtype)
    bad = {100: "k", 230: "v", 231: "v", 499: "k"}
    for j, what in bad.items():
        (k if what == "k" else v)[j] = float("nan") if j != 231 else float("inf")
    o = D.op_window_attention(q, k, v, ws, left=left, right=right, sinks=sinks).double().cpu().numpy()
    seen = A.window_mask(n, n, left, right, sinks)
    touched = seen[:, list(bad)].any(1)
    assert touched.any() and not touched.all()
    assert not np.isfinite(o[touched]).any()
    clean = ~touched
    A.check(o[clean][::5], xq[clean][::5], xk, xv, seen[clean][::5], hd ** -0.5, dtype == BF)
    # rows of another sequence in the same tile, and rows behind the last sequence
    k[:250], v[250:] = float("nan"), 1.0
    o = D.op_window_attention(q, k, v, ws, cu_q=ints([0, 250, 400]), cu_k=ints([0, 250, 400]), left=-1, right=0)
    assert torch.isnan(o[:250]).all() and torch.isfinite(o[250:350]).all()


def test_output_rows_that_begin_at_16_bytes(D, ws):
    rng = np.random.default_rng(28)
    for heads, hd in ((2, 64), (40, 128)):
        xq, q = values(rng, (500, heads, hd), BF)
        xk, k = values(rng, (500, 1, hd), BF)
        want = D.op_window_attention(q, k, k, ws, left=70, right=0, sinks=2)
        for pad, at in ((8, 0), (16, 8), (8, 8)):
            t = torch.full((500, heads * hd + pad), 7.0, dtype=BF, device=dev)
            o = t[:, at:at + heads * hd].unflatten(1, (heads, hd))
            D.op_window_attention(q, k, k, ws, left=70, right=0, sinks=2, out=o)
            assert torch.equal(o, want)
            assert (t[:, :at] == 7).all() and (t[:, at + heads * hd:] == 7).all()


def test_infinite_scores(D, ws):
    for dtype, heads in ((BF, 1), (BF, 160), (F32, 1)):
        q = torch.ones(200, heads, 64, dtype=dtype, device=dev)
        k = torch.ones(200, 1, 64, dtype=dtype, device=dev)
        v = torch.ones(200, 1, 64, dtype=dtype, device=dev)
        k[:] = float("-inf")  # every score is -inf: zeros
        assert (D.op_window_attention(q, k, v, ws) == 0).all()
        k[150:] = 1.0  # causal: rows before 150 see scores of -inf alone
        o = D.op_window_attention(q, k, v, ws, right=0)
        assert (o[:150] == 0).all()
        # n (1 / n) in fp32: half a step of 1 / n and half a step of the product
        assert ((o[150:].double() - 1).abs() <= 2.0 ** -23).all()


def test_growing_scores(D, ws):
    # key norms ramp up, so the running maximum grows tile after tile; every other row is damped
    rng = np.random.default_rng(14)
    for hd, heads in ((64, 2), (128, 2), (64, 21), (128, 20)):
        n = 900
        xq, _ = values(rng, (n, heads, hd), BF)
        xk, _ = values(rng, (n, 1, hd), BF)
        xq[1::2] *= 0.0625
        xk *= np.linspace(0.25, 6.0, n)[:, None, None]
        xv, v = values(rng, (n, 1, hd), BF)
        q, k = (torch.from_numpy(x.astype(np.float32)).to(BF) for x in (xq, xk))
        xq, xk = q.double().numpy(), k.double().numpy()
        o = D.op_window_attention(q.to(dev), k.to(dev), v, ws, right=0)
        torch.cuda.synchronize()
        compare(o.double().cpu().numpy(), xq, xk, xv, [n], [n], -1, 0, 0, hd ** -0.5, True)


def test_agrees_with_the_block_decoders_attention(D, ws):
    # unmasked with as many key heads as heads it is what the decoder's own attention computes
    rng = np.random.default_rng(15)
    xq, q = values(rng, (64, 4, 128), BF)
    xk, k = values(rng, (700, 4, 128), BF)
    xv, v = values(rng, (700, 4, 128), BF)
    a = D.op_window_attention(q, k, v, ws)
    b = D.op_attention_bf16(q.view(64, 512), k.view(1, 700, 512), v.view(1, 700, 512), 64, ws).view(64, 4, 128)
    torch.cuda.synchronize()
    seen = np.ones((64, 700), bool)
    for o in (a, b):
        A.check(o.double().cpu().numpy(), xq, xk, xv, seen, 128 ** -0.5, True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_beyond_32_bits(D, ws, dtype):
    # rows 2^17 elements apart: the last ones lie beyond 2^31 elements
    rng = np.random.default_rng(26)
    T, H, hd = 16500, 2, 128
    t = torch.empty((T, 1 << 17), dtype=dtype, device=dev)
    q, k, v, o = (t[:, a * hd:b * hd].unflatten(1, (b - a, hd)) for a, b in ((0, 2), (2, 3), (3, 4), (4, 6)))
    xs = []
    for x in (q, k, v):
        host, there = values(rng, x.shape, dtype)
        x.copy_(there)
        xs.append(host)
    D.op_window_attention(q, k, v, ws, left=50, right=0, sinks=2, out=o)
    torch.cuda.synchronize()
    ws.check()
    pick = [0, 1, 128, T // 2, T - 300, T - 2, T - 1]
    near = [sorted({0, 1, *range(max(0, i - 60), i + 1)}) for i in pick]  # keys 50 back, and some that are not seen
    for i, keys in zip(pick, near):
        seen = np.array([[j <= i and (j < 2 or j >= i - 50) for j in keys]])
        A.check(o[i:i + 1].double().cpu().numpy(), xs[0][i:i + 1], xs[1][keys], xs[2][keys], seen, hd ** -0.5, dtype == BF, i)


def test_bad_bounds_give_empty_sequences(D, ws):
    rng = np.random.default_rng(16)
    _, q = values(rng, (100, 1, 64), BF)
    out = torch.full_like(q, 7.0)
    for cu_q, cu_k in (([0, 200], [0, 100]), ([-5, 50], [0, 100]), ([60, 40], [0, 100])):
        D.op_window_attention(q, q, q, ws, cu_q=ints(cu_q), cu_k=ints(cu_k), out=out)
        assert (out == 7).all()
    for cu_k in ([0, 101], [-1, 50], [50, 50], [90, 10]):  # no keys: zeros
        o = D.op_window_attention(q, q, q, ws, cu_q=ints([0, 100]), cu_k=ints(cu_k))
        assert (o == 0).all()


def test_many_sequences(D, ws):
    rng = np.random.default_rng(17)
    nq = [int(x) for x in rng.integers(0, 40, 1000)]
    run(D, ws, 17, nq, nq, 1, 1, 64, BF, -1, 0, 0, rows=1)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hd,heads,kv_heads", [(128, 3, 1), (64, 4, 2), (128, 8, 1)])
@pytest.mark.parametrize("left,right,sinks", [(-1, 0, 0), (-1, -1, 0), (1500, 0, 130), (700, 20, 4)])
def test_few_rows_over_many_keys(D, ws, dtype, hd, heads, kv_heads, left, right, sinks):
    # the keys of a tile are dealt to several SMs: long and short sequences, one without keys, rows up to a whole tile
    nq = [1, 128, 3, 40, 7]
    nk = [6000, 2500, 130, 0, 900]
    q, k, v, o = run(D, ws, heads + left, nq, nk, heads, kv_heads, hd, dtype, left, right, sinks, rows=10)
    for _ in range(3):
        assert torch.equal(o, D.op_window_attention(q, k, v, ws, cu_q=cum(nq), cu_k=cum(nk), left=left, right=right,
                                                    sinks=sinks))
    # without a workspace the keys of a tile stay together: another order of the sums
    alone, cq, ck = torch.empty_like(o), cum(nq), cum(nk)
    st = D.lib().dinfer_op_window_attention(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), alone.data_ptr(), D.BF16 if dtype == BF else D.FP32, len(nq),
        cq.data_ptr(), ck.data_ptr(), sum(nq), sum(nk), heads, kv_heads, hd, heads * hd, kv_heads * hd, kv_heads * hd,
        heads * hd, left, right, sinks, hd ** -0.5, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == D.OK
    torch.cuda.synchronize()
    compare(alone.double().cpu().numpy(), *(t.double().cpu().numpy() for t in (q, k, v)), nq, nk, left, right, sinks,
            hd ** -0.5, dtype == BF, 10)


def test_masked_keys_and_infinite_scores_over_many_keys(D, ws):
    rng = np.random.default_rng(25)
    for dtype, hd in ((BF, 64), (BF, 128), (F32, 64), (F32, 128)):
        nq, nk = 50, 3000
        xq, q = values(rng, (nq, 2, hd), dtype)
        xk, k = values(rng, (nk, 1, hd), dtype)
        xv, v = values(rng, (nk, 1, hd), dtype)
        v[2990], k[2970] = float("nan"), float("nan")  # seen by rows 40 .., and 20 ..
        o = D.op_window_attention(q, k, v, ws, left=-1, right=0)
        seen = A.window_mask(nq, nk, -1, 0, 0)
        assert torch.isnan(o[20:]).all()
        A.check(o[:20].double().cpu().numpy(), xq[:20], xk, xv, seen[:20], hd ** -0.5, dtype == BF)
        k[:] = float("-inf")
        k[1000:1200], v[:] = 1.0, 1.0  # one part alone holds a score above -inf
        o = D.op_window_attention(q.abs(), k, v, ws, left=-1, right=0)
        assert ((o.double() - 1).abs() <= 2.0 ** -7).all()
        k[:] = float("-inf")
        assert (D.op_window_attention(q.abs(), k, v, ws, left=-1, right=0) == 0).all()


def test_two_calls_at_once(D, ws):
    rng = np.random.default_rng(24)
    other, side = D.OpWorkspace(), torch.cuda.Stream()
    for dtype, heads in ((BF, 4), (BF, 16), (F32, 4)):
        _, q = values(rng, (1500, heads, 64), dtype)
        _, k = values(rng, (1500, 2, 64), dtype)
        call = lambda w, left, right: D.op_window_attention(q, k, k, w, left=left, right=right, sinks=3)  # noqa: E731
        want = [call(ws, -1, 0), call(ws, 100, 7)]
        torch.cuda.synchronize()
        for _ in range(20):
            a = call(ws, -1, 0)
            with torch.cuda.stream(side):
                b = call(other, 100, 7)
            torch.cuda.synchronize()
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    ws.check()
    other.check()


def test_another_stream_and_a_graph(D, ws):
    rng = np.random.default_rng(18)
    xq, q = values(rng, (300, 2, 128), BF)
    xk, k = values(rng, (300, 1, 128), BF)
    out = torch.empty_like(q)
    want = D.op_window_attention(q, k, k, ws, left=50, right=0, sinks=4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = D.op_window_attention(q, k, k, ws, left=50, right=0, sinks=4)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.op_window_attention(q, k, k, ws, left=50, right=0, sinks=4, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # the graph reads its operands at replay
    q.copy_(q.flip(0))
    graph.replay()
    assert torch.equal(out, D.op_window_attention(q, k, k, ws, left=50, right=0, sinks=4))


# ---------------------------------------------------------------------------
# a serving run: prompts, tokens, forks, compaction, all four operators together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,hd,page", [(BF, 128, 16), (F32, 64, 24)])
def test_serving_run(D, ws, dtype, hd, page):
    from tests.paged_model import Model
    rng = np.random.default_rng(19)
    layers, pages, kv_heads, heads, left, sinks = 2, 64, 2, 6, 90, 4
    cache = D.PagedKV.empty(layers, pages, page, kv_heads, hd, 8, 16, dtype=dtype)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    model = Model(cache.k.double().cpu().numpy(), cache.v.double().cpu().numpy(), 8, 16)
    scale, bf = hd ** -0.5, dtype == BF

    def fused(n):
        x, t = values(rng, (n, (heads + 2 * kv_heads) * hd), dtype)
        cuts = ((0, heads), (heads, heads + kv_heads), (heads + kv_heads, heads + 2 * kv_heads))
        return ([x[:, a * hd:b * hd].reshape(n, b - a, hd) for a, b in cuts],
                [t[:, a * hd:b * hd].unflatten(1, (b - a, hd)) for a, b in cuts])

    lens = [150, 33, 1]
    cache.extend(ints(lens))
    model.extend([0, 1, 2], lens)
    for layer in range(layers):  # the prompts
        (xq, xk, xv), (q, k, v) = fused(sum(lens))
        o = D.op_window_attention(q, k, v, ws, cu_q=cum(lens), cu_k=cum(lens), left=left, right=0, sinks=sinks)
        cache.append(layer, k, v, rows=cum(lens))
        model.append(layer, [0, 1, 2], lens, xk, xv)
        compare(o.double().cpu().numpy(), xq, xk, xv, lens, lens, left, 0, sinks, scale, bf, rows=8)
    live = [0, 1, 2]
    for step in range(14):
        if step == 2:  # two continuations of sequence 0, one whole copy of sequence 1
            cache.fork(ints([0, 0]), ints([3, 4]))
            model.fork([0, 0], [3, 4], True)
            cache.fork(ints([1]), ints([5]), share=False)
            model.fork([1], [5], False)
            live = [0, 1, 2, 3, 4, 5]
        if step == 6:
            cache.free(ints([0, 4]))
            model.free([0, 4])
            live = [1, 2, 3, 5]
        if step == 8:
            cache.compact()
            model.compact()
        n = len(live)
        cache.extend(seqs=ints(live))
        model.extend(live, [1] * n)
        for layer in range(layers):
            (xq, xk, xv), (q, k, v) = fused(n)
            cache.append(layer, k, v, seqs=ints(live))
            model.append(layer, live, [1] * n, xk, xv)
            o = cache.attention(layer, q, ws, window=left, sinks=sinks, seqs=ints(live))
            torch.cuda.synchronize()
            for i, s in enumerate(live):
                kk, vv = model.sequence(layer, s)
                A.check(o[i:i + 1].double().cpu().numpy(), xq[i:i + 1], kk, vv, A.window_mask(1, len(kk), left, 0, sinks),
                        scale, bf, (step, layer, s))
        assert np.array_equal(cache.table.cpu().numpy(), model.table)
        assert np.array_equal(cache.refs.cpu().numpy(), model.refs)
    cache.check()
    assert np.array_equal(cache.k.double().cpu().numpy(), model.k, equal_nan=True)
