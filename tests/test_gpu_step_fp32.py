"""The token step's operators in fp32 over their sizes: rotated appends, shared prefixes."""
import numpy as np
import pytest
import torch

from tests import test_gpu_prefix_attention as PA
from tests import test_gpu_rope as R

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def D():
    from block_denoising_gb300 import build, dinfer
    build.build()
    return dinfer


@pytest.fixture(scope="module")
def ws(D):
    return D.OpWorkspace()


@pytest.mark.parametrize("heads,kv_heads,hd,page,order,rot,layout", [
    (4, 4, 64, 16, "token", 64, "half"), (32, 8, 128, 16, "head", 128, "pairs"), (7, 1, 128, 8, "token", 32, "half"),
    (16, 16, 64, 128, "head", 20, "half"), (12, 4, 128, 64, "token", 6, "pairs"), (40, 5, 64, 24, "head", 2, "pairs"),
])
def test_rotated_appends(D, heads, kv_heads, hd, page, order, rot, layout):
    R.test_rotated_appends_are_rotations_and_appends(D, heads, kv_heads, hd, page, F32, order, rot, layout)


@pytest.mark.parametrize("first", [0, 1000])
def test_a_long_prompt_of_rows(D, first):
    """More rows than blocks at a time, several a block."""
    rng = np.random.default_rng(first)
    n, heads, kv_heads, hd, page = 3001, 6, 2, 128, 32
    c = R.cache(D, rng, 1, 140, page, kv_heads, hd, 2, 130, F32, "token")
    c.extend(R.ints([first + n]), R.ints([1]))
    t = R.twin(D, c)
    x = R.values(rng, (n, heads + 2 * kv_heads, hd), F32)[1]
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    rope = D.Rope(hd, theta=500000.0, scaling="bands", factor=8.0, trained=2048, slow=1.0, fast=4.0)
    out = c.append_rope(0, rope, k, v, q=q, rows=R.ints([0, n]), seqs=R.ints([1]))
    t.append(0, D.op_rope(k, rope, first=first), v, rows=R.ints([0, n]), seqs=R.ints([1]))
    assert R.alike(c, t) and torch.equal(out, D.op_rope(q, rope, first=first))
    c.check()


@pytest.mark.parametrize("shared,own,heads,kv_heads,hd,page,order", [
    ([300], [[1, 2, 33]], 1, 1, 128, 16, "token"), ([1000, 77], [[5] * 9, [60, 1]], 8, 2, 128, 24, "head"), ([2500], [[17] * 30], 32, 8, 128, 16, "token"),
    ([130, 0, 64], [[1, None], [9, 3], [2] * 5], 16, 16, 128, 64, "head"), ([513], [[1] * 12], 14, 2, 128, 1, "token"), ([700], [[40, 4]], 64, 4, 64, 128, "head"),
    ([4000] * 3, [[1, 2]] * 3, 6, 2, 128, 32, "token"),
])
def test_shared_prefixes(D, ws, shared, own, heads, kv_heads, hd, page, order):
    rng = np.random.default_rng(sum(shared) + heads)
    c, seqs, bounds = PA.make(D, rng, shared, own, page, kv_heads, hd, F32, order)
    q = PA.values(rng, (len(seqs), heads, hd), F32)
    o = c.prefix_attention(0, q, ws, PA.ints(shared), PA.ints(bounds), seqs=PA.ints(seqs))
    assert PA.check(c, seqs, q, o) > 0
    assert torch.equal(o, c.prefix_attention(0, q, ws, PA.ints(shared), PA.ints(bounds), seqs=PA.ints(seqs)))
    c.check()
    ws.check()
