"""Refusals of a serving loop's other steps (no GPU): every call below must return DINFER_EINVAL before it touches a
device, and the binding must refuse what the C side cannot see."""
import ctypes

import pytest
import torch

from block_denoising_gb300 import build as B
from block_denoising_gb300 import dinfer
from tests.test_kv_abi import cache

P = 4096  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def L():
    B.build()
    return dinfer.lib()


def refused(L, fn, ok, changes):
    for i, v in changes:
        a = list(ok)
        a[i] = v
        assert fn(*a) == dinfer.EINVAL, (i, v)
        assert L.dinfer_last_error(None)


ROPES = [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(rot_dim=-2), dict(theta=0.0), dict(theta=float("nan")), dict(theta=float("inf")),
    dict(magnitude=0.0), dict(magnitude=float("inf")), dict(magnitude=1e300), dict(scaling="linear", factor=0.0), dict(scaling="base", factor=float("nan")),
    dict(scaling="bands", factor=2.0, trained=0), dict(scaling="bands", factor=2.0, trained=10, slow=4.0, fast=4.0),
    dict(scaling="bands", factor=2.0, trained=10, slow=-1.0, fast=4.0), dict(scaling="bands", factor=2.0, trained=10, fast=float("inf")),
    dict(theta=1e-300),
]


def test_rope_refuses_bad_arguments(L):
    rope = dinfer.Rope(128)
    ok = [P, 8 * P, dinfer.BF16, rope, None, 0, 4, 8, 128, 1024, 1024, None]
    refused(L, L.dinfer_op_rope, ok, (
        (0, None), (1, None), (2, 7), (3, None), (4, P + 2), (5, (1 << 31) - 2), (6, 0), (6, (1 << 30) + 1), (7, 0), (7, 65537), (8, 0), (8, 132),
        (8, 264), (8, 64), (9, 1000), (9, 1023), (10, 512), (0, P + 2), (1, P + 8)))
    refused(L, L.dinfer_op_rope, ok[:1] + [P] + ok[2:], ((10, 2048),))  # in place with another stride
    for name, v in (("layout", 9), ("scaling", -1), ("rot_dim", 130), ("ready", 0)):
        bad = dinfer.Rope(128)
        setattr(bad, name, v)
        refused(L, L.dinfer_op_rope, ok, ((3, ctypes.addressof(bad)),))


def test_bad_rotations_are_refused(L):
    assert L.dinfer_rope_init(None) == dinfer.EINVAL
    for kw in ROPES:
        with pytest.raises(dinfer.DinferError, match="rope"):
            dinfer.Rope(**{"rot_dim": 128, **kw})
    for name in ("layout", "scaling"):
        with pytest.raises(ValueError, match=name):
            dinfer.Rope(128, **{name: "other"})
        bad = dinfer.Rope(128)
        setattr(bad, name, 9)
        assert L.dinfer_rope_init(bad) == dinfer.EINVAL


def test_frequencies_are_fractions_of_a_turn(L):
    import math
    r = dinfer.Rope(8, theta=100.0, scaling="base", factor=3.0)
    for i in range(4):
        f = 100.0 ** (-i / 4) * 3.0 ** (-i / 3)
        assert abs(r.turns[i] / 2.0 ** 64 - f / (2 * math.pi)) < 1e-16
    assert list(r.turns[4:]) == [0] * 124
    two = dinfer.Rope(2, scaling="base", factor=3.0)  # a single pair is the fastest one
    assert abs(two.turns[0] / 2.0 ** 64 - 1 / (2 * math.pi)) < 1e-16


def test_rotated_append_refuses_bad_arguments(L):
    c = ctypes.byref(cache())
    rope = dinfer.Rope(128)
    ok = [c, 0, rope, None, None, None, 4, P, 8 * P, 32, 4096, 4096, P, P, 1024, 1024, 4, None]
    refused(L, L.dinfer_kv_append_rope, ok, (
        (0, None), (0, ctypes.byref(cache(head_dim=96))), (1, -1), (1, 2), (2, None), (2, dinfer.Rope(130)), (3, P + 1), (4, P + 2), (5, P + 3), (6, 0),
        (6, 5), (7, None), (8, None), (7, P + 8), (8, P + 8), (8, P), (9, 0), (9, 65537), (9, 33), (10, 4095), (11, 4000), (12, None), (13, None),
        (12, P + 2), (14, 1000), (15, 1023), (16, 0), (16, 3), (16, (1 << 30) + 1)))
    many = list(ok)
    many[4], many[5], many[6] = P, P, 1025
    assert L.dinfer_kv_append_rope(*many) == dinfer.EINVAL


def test_prefix_attention_refuses_bad_arguments(L):
    c = ctypes.byref(cache())
    big = 1 << 30
    ok = [c, 0, None, 4, None, P, 1, P, P, 4096, 4096, 32, 0.1, P, big, None]
    refused(L, L.dinfer_kv_prefix_attention, ok, (
        (0, None), (0, ctypes.byref(cache(page_size=0))), (1, -1), (1, 2), (2, P + 2), (3, 0), (3, 1025), (3, 1024), (4, P + 1), (5, None), (5, P + 2), (6, 0),
        (6, 2), (7, None), (8, None), (7, P + 8), (8, P + 4), (9, 4095), (10, 4000), (11, 0), (11, 31), (11, 65544), (12, 0.0), (12, float("nan")),
        (12, float("inf")), (13, None), (13, P + 8), (14, 1000)))
    many = list(ok)
    many[3], many[4], many[6] = 1000, P, 25  # together more than a call may name
    assert L.dinfer_kv_prefix_attention(*many) == dinfer.EINVAL
    wide = [ctypes.byref(cache(kv_heads=1024, token_stride=1024 * 128, page_stride=16 * 1024 * 128, layer_stride=100 * 16 * 1024 * 128)), 0, None, 1000, None, P,
            1, P, P, 1024 * 128, 1024 * 128, 1024, 0.1, P, dinfer.lib().dinfer_op_workspace_bytes(), None]
    assert L.dinfer_kv_prefix_attention(*wide) == dinfer.EINVAL  # the sums of a million rows
    assert "workspace" in L.dinfer_last_error(None).decode()
    long = [ctypes.byref(cache(max_pages=(1 << 27) - 1)), 0, None, 4, None, P, 1, P, P, 4096, 4096, 32, 0.1, P, big, None]
    assert L.dinfer_kv_prefix_attention(*long) == dinfer.EINVAL
    assert "2^31" in L.dinfer_last_error(None).decode()


def test_sample_refuses_bad_arguments(L):
    ok = [P, dinfer.FP32, 4, 1000, 1000, None, None, None, None, P, P, P, None]
    refused(L, L.dinfer_op_sample, ok, (
        (0, None), (0, P + 2), (1, 5), (2, 0), (2, (1 << 20) + 1), (3, 0), (3, (1 << 19) + 1), (4, 999), (4, -1000), (4, 1 << 41), (5, P + 2), (6, P + 1),
        (7, P + 2), (8, P + 3), (9, None), (9, P + 2), (10, None), (10, P + 1), (11, P + 2)))
    refused(L, L.dinfer_op_sample, [P + 1, dinfer.BF16] + ok[2:], ((2, 4),))


def test_the_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        dinfer.op_rope(x, dinfer.Rope(64))
    with pytest.raises(ValueError, match="GPU"):
        dinfer.op_sample(torch.zeros(2, 8), torch.zeros(2))
