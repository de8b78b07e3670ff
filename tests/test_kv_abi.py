"""Refusals of the paged cache's and window attention's entry points (no GPU): every call below must return
DINFER_EINVAL before it touches a device, and the binding must refuse what the C side cannot see."""
import ctypes
import re

import numpy as np
import pytest
import torch

from block_denoising_gb300 import build as B
from block_denoising_gb300 import dinfer
from tests import attention64, paged_model

P = 4096  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def L():
    B.build()
    return dinfer.lib()


def cache(**kw):
    hd, heads, page, pages, layers = 128, 8, 16, 100, 2
    f = dict(k=P, v=P, layer_stride=pages * page * heads * hd, page_stride=page * heads * hd, token_stride=heads * hd,
             head_stride=hd, table=P, lens=P, refs=P, state=P, n_layers=layers, num_pages=pages, page_size=page,
             kv_heads=heads, head_dim=hd, dtype=dinfer.BF16, max_seqs=4, max_pages=20)
    f.update(kw)
    return dinfer.KvCache(**f)


def calls(L, kc, p=P):
    """Every entry point with otherwise good arguments."""
    c = ctypes.byref(kc) if kc is not None else None
    yield "extend", lambda: L.dinfer_kv_extend(c, None, None, 4, None)
    yield "set", lambda: L.dinfer_kv_set(c, p, p, p, None)
    yield "append", lambda: L.dinfer_kv_append(c, 0, None, None, 4, p, p, 1024, 1024, 4, None)
    yield "fork", lambda: L.dinfer_kv_fork(c, p, p, 1, 1, None)
    yield "free", lambda: L.dinfer_kv_free(c, p, 1, None)
    yield "compact", lambda: L.dinfer_kv_compact(c, None, None)
    yield "attention", lambda: L.dinfer_kv_attention(c, 0, None, 4, p, p, 4096, 4096, 32, -1, 0, 0.1, p, 1 << 30, None)
    yield "status", lambda: L.dinfer_kv_status(c, None, None)


@pytest.mark.parametrize("bad,needle", [
    (dict(k=None), "NULL"), (dict(state=None), "NULL"), (dict(v=P + 8), "aligned"), (dict(lens=P + 2), "misaligned"),
    (dict(dtype=7), "dtype"), (dict(head_dim=96), "head_dim"), (dict(page_size=0), "size"), (dict(page_size=65537), "size"),
    (dict(num_pages=0), "size"), (dict(n_layers=0), "size"), (dict(kv_heads=0), "size"), (dict(max_seqs=0), "size"),
    (dict(max_pages=1 << 27), "2\\^31"), (dict(token_stride=1020), "16 bytes|overlap"), (dict(head_stride=64), "overlap"),
    (dict(page_stride=16 * 8 * 128 - 8), "overlap"), (dict(layer_stride=0), "overlap"), (dict(token_stride=-1024), "overlap"),
    (dict(page_stride=1 << 62), "overlap"),
])
def test_bad_caches_are_refused_by_every_call(L, bad, needle):
    for name, call in calls(L, cache(**bad)):
        assert call() == dinfer.EINVAL, name
        assert re.search(needle, L.dinfer_last_error(None).decode()), name


def test_null_cache_and_operands_are_refused(L):
    for name, call in calls(L, None):
        assert call() == dinfer.EINVAL, name
    for name, call in calls(L, cache(), None):
        if name in ("set", "append", "fork", "free", "attention"):
            assert call() == dinfer.EINVAL, name


def test_bad_call_arguments_are_refused(L):
    c = ctypes.byref(cache())
    ok = [c, 0, None, None, 4, P, P, 1024, 1024, 4, None]
    for i, v in ((1, -1), (1, 2), (4, 0), (4, 5), (5, P + 2), (7, 1000), (8, 1023), (9, 0), (7, 512)):
        a = list(ok)
        a[i] = v
        assert L.dinfer_kv_append(*a) == dinfer.EINVAL, (i, v)
    many = [c, 0, P, P, 1025, P, P, 1024, 1024, 4, None]  # more entries than a call may name
    assert L.dinfer_kv_append(*many) == dinfer.EINVAL
    many[2], many[4] = None, cache().max_seqs + 1
    assert L.dinfer_kv_append(*many) == dinfer.EINVAL
    ok = [c, 0, None, 4, P, P, 4096, 4096, 32, -1, 0, 0.1, P, 1 << 30, None]
    for i, v in ((1, 2), (3, 0), (3, 1025), (4, P + 4), (5, P + 4), (6, 4000), (7, 4095), (8, 0), (8, 31), (10, -1),
                 (11, float("nan")), (11, float("inf")), (11, 0.0), (11, -0.1), (12, None), (12, P + 8), (13, 1000)):
        a = list(ok)
        a[i] = v
        assert L.dinfer_kv_attention(*a) == dinfer.EINVAL, (i, v)
    for n in (0, -1, 1025):
        assert L.dinfer_kv_extend(c, None, None, n, None) == dinfer.EINVAL
        assert L.dinfer_kv_fork(c, P, P, n, 0, None) == dinfer.EINVAL
    assert L.dinfer_kv_free(c, P, 0, None) == dinfer.EINVAL
    for i in (1, 2, 3):
        for bad in (None, P + 2):
            a = [c, P, P, P, None]
            a[i] = bad
            assert L.dinfer_kv_set(*a) == dinfer.EINVAL
    # more units of keys than an int counts
    big = cache(max_pages=(1 << 27) - 1, max_seqs=1024)
    assert L.dinfer_kv_attention(ctypes.byref(big), 0, None, 1024, P, P, 4096, 4096, 32, -1, 0, 0.1, P, 1 << 30,
                                 None) == dinfer.EINVAL
    assert L.dinfer_kv_state_ints(0, 4) == 0 and L.dinfer_kv_state_ints(10, 4) >= 34


def test_window_attention_refuses_bad_arguments(L):
    ok = [P, P, P, P, dinfer.BF16, 2, P, P, 100, 100, 32, 8, 128, 4096, 1024, 1024, 4096, -1, 0, 0, 0.1, None, 0, None]
    for i, v in ((0, None), (3, None), (0, P + 8), (4, 3), (5, 0), (5, 1025), (6, None), (7, None), (8, 0), (9, 0),
                 (8, (1 << 30) + 1), (10, 0), (10, 30), (11, 0), (12, 80), (13, 4097), (14, 1020), (15, 512), (16, 0),
                 (19, -1), (20, float("nan")), (20, 0.0), (20, -1.0)):
        a = list(ok)
        a[i] = v
        assert L.dinfer_op_window_attention(*a) == dinfer.EINVAL, (i, v)
    a = list(ok)
    a[6] = a[7] = None  # two sequences need their bounds
    assert L.dinfer_op_window_attention(*a) == dinfer.EINVAL
    a = list(ok)
    a[21], a[22] = P, 100  # a workspace that is too small, one that is not aligned
    assert L.dinfer_op_window_attention(*a) == dinfer.EINVAL
    a[21], a[22] = P + 8, 1 << 30
    assert L.dinfer_op_window_attention(*a) == dinfer.EINVAL


def test_binding_refuses_what_the_library_cannot_see(L):
    k = torch.zeros(1, 4, 16, 2, 64)
    with pytest.raises(ValueError):  # not on a GPU
        dinfer.PagedKV(k, k, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                       torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        dinfer.PagedKV(k, k[:, :2], None, None, None)
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        dinfer.op_window_attention(q, q, q, None)
    cpu = torch.zeros(1).get_device()
    for t in (torch.zeros(4, 128), torch.zeros(4, 2, 32), torch.zeros(4, 3, 64), torch.zeros(4, 2, 64, dtype=torch.float64),
              torch.zeros(4, 64, 2).transpose(1, 2), torch.zeros(2, 4, 64).transpose(0, 1)):
        with pytest.raises(ValueError):
            dinfer._rows_of(t, "t", 2, 64, torch.float32, cpu)
    assert dinfer._rows_of(torch.zeros(4, 6, 64)[:, :2], "t", 2, 64, torch.float32, cpu) == (4, 2, 384)
    for t in (torch.zeros(3), torch.zeros(3, dtype=torch.int64), torch.zeros((2, 2), dtype=torch.int32),
              torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            dinfer._ints(t, "t", cpu)


def test_the_test_helpers_themselves():
    # window_mask against the sentence it implements, attend() against a hand case
    for nq, nk, left, right, sinks in ((3, 5, 1, 0, 1), (4, 2, -1, 0, 0), (2, 6, 0, 1, 2), (3, 3, -1, -1, 0)):
        m = attention64.window_mask(nq, nk, left, right, sinks)
        for i in range(nq):
            for j in range(nk):
                p = nk - nq + i
                assert m[i, j] == ((right < 0 or j <= p + right) and (left < 0 or j >= p - left or j < sinks))
    o, tol = attention64.attend(np.zeros(64), np.ones((4, 64)), np.arange(4.0)[:, None] * np.ones((1, 64)),
                                np.array([True, True, False, True]), 1.0, False)
    assert np.allclose(o, 4 / 3) and np.all(tol < 1e-4)
    # the page model: shared pages survive their first owner, compaction keeps contents
    rng = np.random.default_rng(0)
    k = rng.standard_normal((1, 8, 4, 1, 2))
    m = paged_model.Model(k, k, 3, 4)
    m.extend([0], [9])
    assert m.table[0].tolist() == [0, 1, 2, -1]
    m.fork([0], [1], True)
    assert m.table[1].tolist() == [0, 1, 3, -1] and m.refs[:4].tolist() == [2, 2, 1, 1]
    before = m.sequence(0, 1)[0].copy()
    m.free([0])
    assert m.compact() == 3 and m.table[1].tolist() == [0, 1, 2, -1]
    assert np.array_equal(m.sequence(0, 1)[0], before)
    m.extend([0, 2], [21, 16])
    assert m.status == 16 and m.lens.tolist() == [0, 9, 16] and m.table[2].tolist() == [3, 4, 5, 6]


def test_misaligned_index_operands_are_refused(L):
    c = ctypes.byref(cache())
    for bad in (P + 1, P + 2, P + 3):
        for call in (lambda: L.dinfer_kv_extend(c, bad, P, 4, None), lambda: L.dinfer_kv_extend(c, P, bad, 4, None),
                     lambda: L.dinfer_kv_append(c, 0, bad, None, 4, P, P, 1024, 1024, 4, None),
                     lambda: L.dinfer_kv_append(c, 0, None, bad, 4, P, P, 1024, 1024, 4, None),
                     lambda: L.dinfer_kv_fork(c, bad, P, 1, 1, None), lambda: L.dinfer_kv_fork(c, P, bad, 1, 1, None),
                     lambda: L.dinfer_kv_free(c, bad, 1, None), lambda: L.dinfer_kv_compact(c, bad, None),
                     lambda: L.dinfer_kv_attention(c, 0, bad, 4, P, P, 4096, 4096, 32, -1, 0, 0.1, P, 1 << 30, None),
                     lambda: L.dinfer_op_window_attention(P, P, P, P, dinfer.BF16, 2, bad, P, 100, 100, 32, 8, 128, 4096, 1024, 1024,
                                                          4096, -1, 0, 0, 0.1, None, 0, None),
                     lambda: L.dinfer_op_window_attention(P, P, P, P, dinfer.BF16, 2, P, bad, 100, 100, 32, 8, 128, 4096, 1024, 1024,
                                                          4096, -1, 0, 0, 0.1, None, 0, None)):
            assert call() == dinfer.EINVAL
            assert "misaligned" in L.dinfer_last_error(None).decode()


def test_binding_keeps_numbers_beyond_32_bits_at_their_end(L, monkeypatch):
    # a window or a side beyond int32 is an open one, not its lower 32 bits; a layer beyond it is refused
    assert [dinfer._i32(x) for x in (0, -1, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 10 ** 30, -2 ** 31, -2 ** 31 - 1, -2 ** 32)] == \
        [0, -1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, -2 ** 31, -2 ** 31, -2 ** 31]
    seen = {}
    monkeypatch.setattr(dinfer, "_run_on", lambda gpu, fn, *args: seen.update({fn.__name__: args}))
    monkeypatch.setattr(dinfer, "_require", lambda ok, what: None)
    far, t = 2 ** 32, torch.zeros(4, 2, 64)

    class Ws:
        buf, nbytes = torch.zeros(8), 32

    kv = object.__new__(dinfer.PagedKV)
    kv.gpu, kv.head_dim, kv.dtype, kv.kv_heads, kv.max_seqs, kv._desc = t.get_device(), 64, torch.float32, 2, 4, None
    kv.append(far, t, t)
    kv.attention(far, t, Ws, window=far, sinks=far)
    dinfer.op_window_attention(t, t, t, Ws, left=far, right=-far, sinks=far)
    end = 2 ** 31 - 1
    assert seen["dinfer_kv_append"][1] == end
    a = seen["dinfer_kv_attention"]
    assert (a[1], a[9], a[10]) == (end, end, end)
    assert seen["dinfer_op_window_attention"][17:20] == (end, -2 ** 31, end)


def test_limits_that_the_header_states(L):
    hd = 128
    c = ctypes.byref(cache(kv_heads=1025, token_stride=1025 * hd, page_stride=16 * 1025 * hd, layer_stride=100 * 16 * 1025 * hd))
    assert L.dinfer_kv_extend(c, None, None, 4, None) == dinfer.EINVAL
    wide = 1024 * hd  # 65536 slots of 1024 heads: a page of 2^33 elements
    c = ctypes.byref(cache(kv_heads=1024, page_size=65536, token_stride=wide, page_stride=65536 * wide, layer_stride=100 * 65536 * wide))
    assert L.dinfer_kv_extend(c, None, None, 4, None) == dinfer.EINVAL
    assert "page too large" in L.dinfer_last_error(None).decode()
    c = ctypes.byref(cache())
    assert L.dinfer_kv_attention(c, 0, P, 4, P, P, 65544 * hd, 65544 * hd, 65544, -1, 0, 0.1, P, 1 << 30, None) == dinfer.EINVAL


@pytest.mark.parametrize("dtype", [dinfer.BF16, dinfer.FP32])
def test_attention_refuses_what_could_take_too_many_steps(L, dtype):
    # by the cache's capacity or the window: below the stated bound nothing is refused for it, whatever the group
    big = ctypes.byref(cache(max_pages=(1 << 27) - 1, max_seqs=1024))

    def steps(size):  # the workspace has room for the counters: the steps are looked at
        L.dinfer_kv_attention(big, 0, None, 1024, P, P, 4096, 4096, 32, -1, 0, 0.1, P, size, None)
        return "steps" in L.dinfer_last_error(None).decode()

    # the smallest such workspace: its rest is too small on any GPU, so that no call below gets further than the checks
    lo, hi = 0, L.dinfer_op_workspace_bytes()
    while hi - lo > 1:
        lo, hi = (lo, (lo + hi) // 2) if steps((lo + hi) // 2) else ((lo + hi) // 2, hi)
    rng = np.random.default_rng(0)
    refused = 0
    for _ in range(400):
        n, kvh, group = int(2 ** rng.uniform(0, 10)), int(2 ** rng.uniform(0, 6)), int(2 ** rng.uniform(0, 6))
        pages, window, sinks = int(2 ** rng.uniform(4, 27)), int(rng.choice([-1, 0, 4095, 1 << 28])), int(rng.choice([0, 4]))
        kc = cache(kv_heads=kvh, token_stride=kvh * 128, page_stride=16 * kvh * 128, layer_stride=100 * 16 * kvh * 128, max_pages=pages,
                   max_seqs=1024, dtype=dtype)
        if pages * 16 >= 1 << 31:
            continue
        st = L.dinfer_kv_attention(ctypes.byref(kc), 0, None, n, P, P, kvh * group * 128, kvh * group * 128, kvh * group, window, sinks,
                                   0.1, P, hi, None)
        assert st != dinfer.OK
        why = L.dinfer_last_error(None).decode()
        keys = pages * 16 if window < 0 else min(pages * 16, window + 1 + sinks)
        if "steps" in why:
            refused += 1
            assert n * kvh * group * (keys / 16 + 11) >= 1 << 31
    assert refused > 10


def test_window_attention_refuses_to_write_over_its_operands(L):
    # rows that are done again still want their query
    at = [P, P + 4096, P + 8192, P + 12288]
    for i in range(3):
        for dtype in (dinfer.BF16, dinfer.FP32):
            assert L.dinfer_op_window_attention(*at[:3], at[i], dtype, 1, None, None, 1, 1, 32, 8, 128, 4096, 1024, 1024, 4096, -1, 0, 0,
                                                0.1, None, 0, None) == dinfer.EINVAL
            assert "overlap" in L.dinfer_last_error(None).decode()
