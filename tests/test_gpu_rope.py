"""Rotary positions on the GPU against 64 bits (80 where the machine has them), and rows rotated on their way to the pages.

The bound of a rotated element: the angle's quarter turn is rounded by at most pi / 4 * 2^-24, sincospif is off by two
units in the last place (2^-23 of a number up to 1), the magnitude's rounding and product by 2^-24 each, so a cosine
by 2^-22 of the magnitude; the two products and their sum add 2^-23; the frequency, a double, moves the angle by
|p| f 2^-50; the output is rounded by half a step of its type.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def D():
    from block_denoising_gb300 import build, dinfer
    build.build()
    return dinfer


def frequencies(rope, scaling):
    L = np.longdouble
    r, s = rope.rot_dim, L(rope.factor)
    i = np.arange(r // 2, dtype=L)
    f = L(rope.theta) ** (-2 * i / r)
    if scaling == "linear":
        f = f / s
    elif scaling == "base" and r > 2:
        f = f * s ** (-2 * i / (r - 2))
    elif scaling == "bands":
        two_pi = L("6.283185307179586476925286766559005768")
        g = np.clip((rope.trained * f / two_pi - L(rope.slow)) / (L(rope.fast) - L(rope.slow)), 0, 1)
        f = g * f + (1 - g) * f / s
    return f


def rotated(x, positions, rope, layout, scaling):
    """x [rows, heads, hd] float64 -> (y, bound without the output's rounding)."""
    f = frequencies(rope, scaling)
    p = np.asarray(positions, dtype=np.longdouble)[:, None]
    two_pi = np.longdouble("6.283185307179586476925286766559005768")
    angle = np.asarray(np.fmod(p * f, two_pi), dtype=np.float64)[:, None]
    slack = np.asarray(np.abs(p) * f, dtype=np.float64)[:, None] * 2.0 ** -50
    h, m = rope.rot_dim // 2, rope.magnitude
    a, b = (slice(0, h), slice(h, 2 * h)) if layout == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    y, bound = x.copy(), np.zeros_like(x)
    c, s = np.cos(angle) * m, np.sin(angle) * m
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    bound[..., a] = bound[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * m * (2.0 ** -22 + 2.0 ** -23 + slack)
    return y, bound


def check(got, y, bound, dtype, what=""):
    step = torch.finfo(dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - y)
    assert np.all(err <= bound + step * (np.abs(y) + bound)), (what, float((err - bound - step * np.abs(y)).max()))


def values(rng, shape, dtype):
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)
    return t.double().numpy(), t.to(dev)


@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
    ("bands", dict(factor=8.0, trained=8192, slow=1.0, fast=4.0, magnitude=1.25)),
])
@pytest.mark.parametrize("rows,heads,hd,rot,layout,dtype", [
    (1, 1, 64, 64, "half", BF), (1, 5, 128, 128, "pairs", F32), (7, 3, 128, 64, "half", BF), (33, 40, 128, 128, "half", BF),
    (96, 8, 64, 64, "half", F32), (5, 2, 96, 10, "half", BF), (5, 2, 80, 6, "pairs", F32), (3, 2, 256, 256, "pairs", BF),
    (3, 1, 8, 2, "half", BF), (4, 2, 4, 2, "pairs", F32), (2600, 2, 64, 32, "pairs", BF), (64, 64, 128, 20, "half", F32),
])
def test_rotation_against_64_bits(D, rows, heads, hd, rot, layout, dtype, scaling, kw):
    rng = np.random.default_rng(rows * 7 + hd + rot)
    rope = D.Rope(rot, layout=layout, scaling=scaling, theta=500000.0 if rows == 7 else 10000.0, **kw)
    x, t = values(rng, (rows, heads, hd), dtype)
    positions = rng.integers(-(1 << 20), 1 << 20, rows)
    got = D.op_rope(t, rope, positions=torch.tensor(positions, dtype=torch.int32, device=dev))
    y, bound = rotated(x, positions, rope, layout, scaling)
    check(got, y, bound, dtype)
    first = D.op_rope(t, rope, first=1000)
    y, bound = rotated(x, 1000 + np.arange(rows), rope, layout, scaling)
    check(first, y, bound, dtype)


def test_far_positions(D):
    rng = np.random.default_rng(3)
    positions = [0, 1, -1, (1 << 31) - 1, -(1 << 31), 123456789, 1 << 24, (1 << 24) + 1]
    rope = D.Rope(128)
    x, t = values(rng, (len(positions), 2, 128), F32)
    got = D.op_rope(t, rope, positions=torch.tensor(positions, dtype=torch.int32, device=dev))
    y, bound = rotated(x, positions, rope, "half", "none")
    check(got, y, bound, F32)
    assert torch.equal(got[0], t[0])


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("rot", [128, 64, 6])
def test_in_place_slices_and_the_way_back(D, layout, rot):
    """The query and key part of one projection's output in place; values and other rows stay; -p undoes p."""
    rng = np.random.default_rng(rot)
    _, x = values(rng, (50, 12, 128), BF)
    was = x.clone()
    rope = D.Rope(rot, layout=layout)
    want = D.op_rope(x[4:44, :8].contiguous(), rope, first=7)
    part = x[4:44, :8]
    assert D.op_rope(part, rope, first=7, out=part) is part
    assert torch.equal(part, want)
    assert torch.equal(x[:4], was[:4]) and torch.equal(x[44:], was[44:]) and torch.equal(x[:, 8:], was[:, 8:])
    xf = was.float()
    back = D.op_rope(D.op_rope(xf, rope, first=7), rope, positions=-torch.arange(7, 57, dtype=torch.int32, device=dev))
    assert float((back - xf).abs().max()) <= float(2 * xf.abs().max()) * 2 ** -20


def test_heads_of_the_block_decoders_layout(D):
    """Half layout, theta 10000: what the decoder's oracle computes."""
    from oracle import dinfer_oracle as O
    rng = np.random.default_rng(9)
    x, t = values(rng, (20, 3, 64), F32)
    got = D.op_rope(t, D.Rope(64)).double().cpu().numpy()
    want = O.rope(x, np.arange(20), 10000.0)
    assert np.abs(got - want).max() <= 2 * np.abs(x).max() * 2.0 ** -21


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def cache(D, rng, layers, pages, page, heads, hd, seqs, most, dtype, order):
    kv = []
    for _ in range(2):
        _, t = values(rng, (layers, pages, page, heads, hd), dtype)
        kv.append(t if order == "token" else t.transpose(2, 3).contiguous().transpose(2, 3))
    return D.PagedKV(kv[0], kv[1], torch.full((seqs, most), -1, dtype=torch.int32, device=dev), torch.zeros(seqs, dtype=torch.int32, device=dev),
                     torch.zeros(pages, dtype=torch.int32, device=dev))


def twin(D, c):
    t = D.PagedKV(c.k.clone(memory_format=torch.preserve_format), c.v.clone(memory_format=torch.preserve_format), c.table.clone(), c.lens.clone(),
                  c.refs.clone())
    assert t.k.stride() == c.k.stride()
    return t


def alike(a, b):
    torch.cuda.synchronize()
    return torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


@pytest.mark.parametrize("heads,kv_heads,hd,page,dtype,order,rot,layout", [
    (4, 2, 64, 16, BF, "token", 64, "half"), (3, 3, 128, 7, F32, "head", 64, "pairs"), (8, 1, 128, 24, BF, "head", 128, "half"),
    (10, 5, 64, 1, F32, "token", 6, "half"), (32, 8, 128, 16, BF, "token", 128, "pairs"),
])
def test_rotated_appends_are_rotations_and_appends(D, heads, kv_heads, hd, page, dtype, order, rot, layout):
    rng = np.random.default_rng(heads * 100 + page)
    c = cache(D, rng, 2, 120, page, kv_heads, hd, 6, 90, dtype, order)
    counts = [40, 0, 1, 17, 30]
    seqs = ints([5, 0, 3, 1, 2])
    c.extend(ints([n + 3 if n else 0 for n in counts]) if page > 1 else ints(counts), seqs)
    lens = c.lens.cpu().numpy()[[5, 0, 3, 1, 2]]
    t = twin(D, c)
    total = sum(counts)
    x = values(rng, (total, heads + 2 * kv_heads, hd), dtype)[1]
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    rows = ints([0] + list(np.cumsum(counts)))
    rope = D.Rope(rot, layout=layout, scaling="linear", factor=2.0)
    where = ints(np.concatenate([np.arange(n - r, n) for n, r in zip(lens, counts)]))
    out = c.append_rope(1, rope, k, v, q=q, rows=rows, seqs=seqs)
    t.append(1, D.op_rope(k, rope, positions=where), v, rows=rows, seqs=seqs)
    assert alike(c, t)
    assert torch.equal(out, D.op_rope(q, rope, positions=where))
    # positions of one's own, no queries, queries in place
    other = ints(rng.integers(0, 100000, total))
    assert c.append_rope(0, rope, k, v, rows=rows, seqs=seqs, positions=other) is None
    t.append(0, D.op_rope(k, rope, positions=other), v, rows=rows, seqs=seqs)
    want = D.op_rope(q, rope, positions=other)
    assert c.append_rope(0, rope, k, v, q=q, rows=rows, seqs=seqs, positions=other, out=q) is q
    assert torch.equal(q, want) and alike(c, t)
    c.check()


def test_one_row_each_in_a_graph_while_the_sequences_grow(D):
    rng = np.random.default_rng(1)
    c = cache(D, rng, 1, 60, 8, 2, 128, 5, 12, BF, "token")
    c.extend(ints([3, 9, 16, 1, 40]))
    t = twin(D, c)
    q, k, v = (values(rng, (5, n, 128), BF)[1] for n in (4, 2, 2))
    rope = D.Rope(128)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.append_rope(0, rope, k, v, q=q, out=out)  # set-up before the capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.extend()
            c.append_rope(0, rope, k, v, q=q, out=out)
        t.append(0, D.op_rope(k, rope, positions=t.lens - 1), v)
        for _ in range(6):
            k.copy_(values(rng, k.shape, BF)[1])
            g.replay()
            t.extend()
            t.append(0, D.op_rope(k, rope, positions=t.lens - 1), v)
            assert torch.equal(out, D.op_rope(q, rope, positions=t.lens - 1))
        assert alike(c, t)
    torch.cuda.current_stream().wait_stream(s)


def test_rows_that_are_not_stored_leave_their_queries(D):
    rng = np.random.default_rng(2)
    c = cache(D, rng, 1, 30, 8, 1, 64, 6, 4, F32, "token")
    c.extend(ints([5, 6, 8]), ints([0, 1, 2]))
    c.fork(ints([2]), ints([4]))          # 2 and 4 share their page
    rope = D.Rope(64)
    for seqs, skipped, bit in (([0, 1, 0], [2], 1), ([0, 9, 1], [1], 1), ([-1, 0, 1], [0], 1), ([0, 4, 1], [1], 8), ([3, 0, 1], [0], 16)):
        t = twin(D, c)
        q, k, v = (values(rng, (3, n, 64), F32)[1] for n in (2, 1, 1))
        out = torch.full_like(q, 7.0)
        c.append_rope(0, rope, k, v, q=q, seqs=ints(seqs), out=out)
        rest = [i for i in range(3) if i not in skipped]
        assert torch.equal(out[skipped], torch.full_like(out[skipped], 7.0))
        where = c.lens[[seqs[i] for i in rest]] - 1
        assert torch.equal(out[rest], D.op_rope(q[rest].contiguous(), rope, positions=where))
        t.append(0, D.op_rope(k[rest].contiguous(), rope, positions=where), v[rest].contiguous(), seqs=ints([seqs[i] for i in rest]))
        assert alike(c, t)
        with pytest.raises(D.DinferError, match="status 0x%x:" % bit):
            c.check()
    # bounds out of order, rows before the first and behind the last one
    q, k, v = (values(rng, (9, n, 64), F32)[1] for n in (2, 1, 1))
    t = twin(D, c)
    out = torch.full_like(q, 7.0)
    c.append_rope(0, rope, k, v, q=q, rows=ints([2, 5, 6]), seqs=ints([0, 1]), out=out)
    c.check()
    for i in (0, 1, 6, 7, 8):
        assert torch.equal(out[i], torch.full_like(out[i], 7.0))
    t.append(0, D.op_rope(k, rope, positions=ints([0, 0, 2, 3, 4, 5, 0, 0, 0])), v, rows=ints([2, 5, 6]), seqs=ints([0, 1]))
    assert alike(c, t)
    c.append_rope(0, rope, k, v, q=q, rows=ints([4, 2, 6]), seqs=ints([0, 1]), out=out)
    with pytest.raises(D.DinferError, match="too long"):
        c.check()
