"""A server's token step: the operators together, as a loop calls them, and each at the ends of its ranges."""
import ctypes

import numpy as np
import pytest
import torch

from tests import attention64 as A
from tests import sample64 as S
from tests import test_gpu_prefix_attention as PA
from tests import test_gpu_rope as R

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


def test_prompt_forks_and_tokens(D):
    """A prompt's rows rotated, attended and stored; six continuations forked from it; then tokens, one step of all of
    them at a time in a captured graph: projection, rotated append, attention over the shared prefix, logits, sampling.
    Every step's attention is checked in 64 bits from the cache, every token from the logits, every key from its row."""
    rng = np.random.default_rng(11)
    heads, kv_heads, hd, page, d, vocab, n, prompt = 8, 2, 128, 16, 256, 1024, 6, 150
    ws, rope = D.OpWorkspace(), D.Rope(hd, scaling="bands", factor=4.0, trained=64, slow=1.0, fast=4.0)
    w = lambda *shape: (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * shape[-1] ** -0.5).to(BF).to(dev)
    embed, w_qkv, w_o, w_lm = w(vocab, d), w((heads + 2 * kv_heads) * hd, d), w(d, heads * hd), w(vocab, d) * 4
    kv = D.PagedKV.empty(layers=1, pages=200, page_size=page, kv_heads=kv_heads, head_dim=hd, max_seqs=n + 1, max_pages=20)

    def project(x):
        return D.op_gemm_bf16(x, w_qkv, ws).to(BF).unflatten(1, (-1, hd))

    # the prompt, as sequence n
    ids = ints(rng.integers(0, vocab, prompt))
    qkv = project(embed[ids.long()])
    rotated = D.op_rope(qkv[:, :heads + kv_heads], rope)
    q, k, v = rotated[:, :heads], rotated[:, heads:], qkv[:, heads + kv_heads:]
    o = D.op_window_attention(q, k, v, ws, left=-1, right=0)
    some = [0, 1, 77, prompt - 1]
    mask = A.window_mask(prompt, prompt, -1, 0, 0)
    A.check(o[some].double().cpu().numpy(), q[some].double().cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(), mask[some], hd ** -0.5, True)
    kv.extend(ints([prompt]), ints([n]))
    kv.append(0, k, v, rows=ints([0, prompt]), seqs=ints([n]))
    twin = kv.k.clone()
    kv.append_rope(0, rope, qkv[:, heads:heads + kv_heads], v, rows=ints([0, prompt]), seqs=ints([n]))
    assert torch.equal(kv.k.view(torch.int16), twin.view(torch.int16))  # the two ways into the cache; what was never written may be NaN
    kv.fork(ints([n] * n), ints(range(n)))

    # six continuations
    tok, conf = ints([5] * n), torch.empty(n, device=dev)
    u, x = torch.empty(n, device=dev), torch.empty((n, d), dtype=BF, device=dev)
    q_rot, o = torch.empty((n, heads, hd), dtype=BF, device=dev), torch.empty((n, heads, hd), dtype=BF, device=dev)
    logits = torch.empty((n, vocab), device=dev)
    settings = dict(temperature=torch.tensor([0.0, 0.7, 1.0, 1.0, 1.0, 1.3], device=dev), top_k=ints([0, 0, 20, 0, 0, 50]),
                    top_p=torch.tensor([1.0, 1.0, 1.0, 0.9, 1.0, 0.8], device=dev), min_p=torch.tensor([0, 0, 0, 0, 0.1, 0.01], device=dev))
    prefix, seqs = ints([prompt]), ints(range(n))

    def step():
        kv.extend(seqs=seqs)
        torch.index_select(embed, 0, tok, out=x)
        qkv = project(x)
        kv.append_rope(0, rope, qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:], q=qkv[:, :heads], seqs=seqs, out=q_rot)
        kv.prefix_attention(0, q_rot, ws, prefix, seqs=seqs, out=o)
        y = D.op_gemm_bf16(o.flatten(1), w_o, ws) + x.float()
        D.op_gemm_bf16(y.to(BF), w_lm, ws, Y=logits)
        D.op_sample(logits, u, tok=tok, conf=conf, **settings)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        u.copy_(torch.rand(n, device=dev))
        step()  # set-up before the capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        for _ in range(20):
            before = tok.clone()
            u.copy_(torch.rand(n, device=dev))
            g.replay()
            torch.cuda.synchronize()
            PA.check(kv, list(range(n)), q_rot, o)
            at = kv.lens[:n].cpu().numpy() - 1
            qkv = project(embed[before.long()])
            assert torch.equal(q_rot, D.op_rope(qkv[:, :heads], rope, positions=ints(at)))
            keys = D.op_rope(qkv[:, heads:heads + kv_heads], rope, positions=ints(at))
            for i in range(n):
                slot = kv.k[0, int(kv.table[i, at[i] // page]), int(at[i] % page)]
                assert torch.equal(slot, keys[i])
                h = logits[i].double().cpu().numpy()
                f = {name: (v[i].item()) for name, v in settings.items()}
                want, c = S.draw(h, float(u[i]), f["temperature"], f["top_k"], f["top_p"], f["min_p"])
                assert want is None or (int(tok[i]) == want and abs(float(conf[i]) - c) <= 2.0 ** -17 * c)
    torch.cuda.current_stream().wait_stream(s)
    kv.check()
    ws.check()


def test_a_cache_beyond_2_31_elements(D, ws):
    """Pages whose places pass 2^31 and 2^32 elements: rotated rows go there and shared prefixes are read there."""
    pages, page, heads, hd = 34000, 128, 8, 128  # 4.5e9 elements: 9 GB each
    shape = (1, pages, page, heads, hd)
    k, v = (torch.empty(shape, dtype=BF, device=dev) for _ in range(2))
    far = [0, 16500, 33990, 33999, 20000, 33000]
    for t in (k, v):
        for p in far:
            t[0, p].normal_()
    seqs, per = 3, 3
    table = torch.full((seqs, 4), -1, dtype=torch.int32, device=dev)
    table[:, 0], table[:, 1] = 33990, 16500
    table[0, 2], table[1, 2], table[2, 2] = 33999, 20000, 33000
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    for p in far:
        refs[p] = 1
    refs[33990] = refs[16500] = 3
    kv = D.PagedKV(k, v, table, ints([256 + 5, 256 + 128, 256 + 77]), refs)
    q = torch.randn(3, 16, hd, device=dev).to(BF)
    new = torch.randn(3, heads, hd, device=dev).to(BF)
    rope = D.Rope(hd)
    rot = kv.append_rope(0, rope, new, new, q=q)
    want = D.op_rope(new, rope, positions=kv.lens - 1)
    for i, p in enumerate((33999, 20000, 33000)):
        assert torch.equal(k[0, p, (4, 127, 76)[i]], want[i]) and torch.equal(v[0, p, (4, 127, 76)[i]], new[i])
    o = kv.prefix_attention(0, rot, ws, ints([256]))
    PA.check(kv, [0, 1, 2], rot, o)
    kv.check()
    del k, v, kv


@pytest.mark.parametrize("order", ["token", "head"])
def test_two_captured_graphs_share_a_workspace(D, ws, order):
    rng = np.random.default_rng(21)
    c, seqs, bounds = PA.make(D, rng, [300, 90], [[1, 2, 17, 4], [60, 3]], 16, 2, 64, order=order)
    sq, pre, b = ints(seqs), ints([300, 90]), ints(bounds)
    qs = [PA.values(rng, (6, h, 64), BF) for h in (4, 12)]
    outs = [torch.empty_like(q) for q in qs]
    want = [c.prefix_attention(0, q, D.OpWorkspace(), pre, b, seqs=sq) for q in qs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for q, out in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.prefix_attention(0, q, ws, pre, b, seqs=sq, out=out)
            c.attention(0, q, ws, seqs=sq)  # an operator that wants the workspace's counters at zero
        graphs.append(g)
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    ws.check()


def test_two_calls_at_once(D):
    """Two streams, a workspace each, the same cache and the same logits."""
    rng = np.random.default_rng(22)
    c, seqs, bounds = PA.make(D, rng, [700], [[5] * 20], 16, 4, 128)
    q = PA.values(rng, (20, 16, 128), BF)
    x, u = torch.randn(20, 30000, device=dev), torch.rand(20, device=dev)
    pre, sq = ints([700]), ints(seqs)
    spaces = [D.OpWorkspace(), D.OpWorkspace()]
    want, tok = c.prefix_attention(0, q, spaces[0], pre, seqs=sq), D.op_sample(x, u, top_p=torch.full((20,), 0.8, device=dev))[0]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    p = torch.full((20,), 0.8, device=dev)
    torch.cuda.synchronize()
    for _ in range(10):
        for s, w, g in zip(streams, spaces, got):
            with torch.cuda.stream(s):
                g.append((c.prefix_attention(0, q, w, pre, seqs=sq), D.op_sample(x, u, top_p=p)[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(t, tok) for g in got for a, t in g)


def test_the_widest_vocabulary_and_rows_far_apart(D):
    """2^19 tokens (16 CTAs a row), rows whose places pass 2^31 elements, no confidence wanted."""
    rng = np.random.default_rng(23)
    x = torch.from_numpy(rng.standard_normal((3, 1 << 19)).astype(np.float32) * 2).to(dev)
    x[1] = 0.25
    u = [0.3, 0.5, 0.9]
    f = lambda v: torch.full((3,), v, device=dev)
    for kw, one in (({}, {}), (dict(top_p=f(0.75)), dict(top_p=0.75)), (dict(top_k=ints([1 << 18] * 3)), dict(top_k=1 << 18)),
                    (dict(min_p=f(0.25)), dict(min_p=0.25))):
        tok, _ = D.op_sample(x, torch.tensor(u, device=dev), **kw)
        for r in range(3):
            want, _ = S.draw(x[r].double().cpu().numpy(), float(np.float32(u[r])), **one)
            assert want is None or int(tok[r]) == want, (r, one)
    wide = torch.empty((70, (1 << 26) + 8), dtype=BF, device=dev)
    y = wide[:, :5001]
    y.normal_()
    v = torch.rand(70, device=dev)
    got = D.op_sample(y, v)
    want = D.op_sample(y.contiguous(), v)
    assert torch.equal(got[0], want[0])
    tok = torch.full((70,), -5, dtype=torch.int32, device=dev)
    L = D.lib()
    near = y.contiguous()
    torch.cuda.synchronize()
    st = L.dinfer_op_sample(near.data_ptr(), D.BF16, 70, 5001, 5001, None, None, None, None, v.data_ptr(), tok.data_ptr(), None,
                            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == D.OK
    assert torch.equal(tok, want[0])


def test_rope_rows_far_apart(D):
    wide = torch.empty((70, (1 << 26) + 8), dtype=BF, device=dev)
    x = wide[:, :512].unflatten(1, (4, 128))
    x.normal_()
    r = D.Rope(128)
    want = D.op_rope(x.contiguous(), r, first=9)
    assert torch.equal(D.op_rope(x, r, first=9), want)
    assert torch.equal(D.op_rope(x, r, first=9, out=x), want)
