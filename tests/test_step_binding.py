"""The binding of a serving loop's other steps (no GPU): what it hands to the library is what the caller holds."""
import copy
import ctypes
import gc
import pickle

import pytest
import torch

from block_denoising_gb300 import build as B
from block_denoising_gb300 import dinfer

P = 4096  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def L():
    B.build()
    return dinfer.lib()


def reason(L, rope):
    """Why a call with rows that overlap one another is refused: an unusable rotation is found first."""
    assert L.dinfer_op_rope(P, 8 * P, dinfer.BF16, rope, None, 0, 4, 8, 128, 1016, 1024, None) == dinfer.EINVAL
    return L.dinfer_last_error(None).decode()


COPIES = [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r)), lambda r: copy.deepcopy({"rope": [r]})["rope"][0]]


@pytest.mark.parametrize("how", range(len(COPIES)))
def test_a_copied_rotation_is_its_own(L, how):
    rope = dinfer.Rope(128, theta=10000.0, layout="pairs", scaling="linear", factor=2.0)
    turns = list(rope.turns)
    twin = COPIES[how](rope)
    assert "rows" in reason(L, rope) and "rows" in reason(L, twin)
    rope.ready = 0  # the copy does not hang on the original
    assert "filled" in reason(L, rope) and "rows" in reason(L, twin)
    rope.ready, ready = twin.ready, twin.ready
    twin.ready = 0  # nor the original on the copy
    assert "rows" in reason(L, rope) and "filled" in reason(L, twin)
    twin.ready = ready
    del rope
    gc.collect()
    others = [dinfer.Rope(128, theta=500000.0) for _ in range(64)]
    assert "rows" in reason(L, twin) and list(twin.turns) == turns and len(others) == 64
    assert [getattr(twin, n) for n in ("rot_dim", "layout", "scaling", "theta", "factor")] == [128, 1, 1, 10000.0, 2.0]
    assert twin._as_parameter_ == ctypes.addressof(twin)


CHANGES = dict(rot_dim=64, layout=0, scaling=0, trained=5, theta=500000.0, factor=3.0, slow=0.5, fast=8.0, magnitude=1.5)


@pytest.mark.parametrize("field", CHANGES)
def test_a_changed_rotation_is_refused_until_it_is_filled_again(L, field):
    rope = dinfer.Rope(128, layout="pairs", scaling="bands", factor=2.0, trained=4096, slow=1.0, fast=4.0)
    was = getattr(rope, field)
    setattr(rope, field, CHANGES[field])
    assert "filled" in reason(L, rope)  # its frequencies are those of the fields before
    setattr(rope, field, was)
    assert "rows" in reason(L, rope)
    setattr(rope, field, CHANGES[field])
    assert L.dinfer_rope_init(rope) == dinfer.OK
    assert "rows" in reason(L, rope)


@pytest.mark.parametrize("first", [1 << 31, 1 << 40, -(1 << 31) - 1, -(1 << 63), 1 << 32])
def test_positions_beyond_int32_are_refused(first):
    # not the end of the range in their place: a position there is another one
    with pytest.raises(ValueError, match="first"):
        dinfer.op_rope(torch.zeros(1, 2, 64), dinfer.Rope(64), first=first)
    with pytest.raises(ValueError, match="trained"):
        dinfer.Rope(64, scaling="bands", factor=2.0, trained=first)


def test_positions_at_the_ends_of_int32_are_not():
    for first in ((1 << 31) - 1, -(1 << 31)):
        with pytest.raises(ValueError, match="GPU"):  # what is refused next
            dinfer.op_rope(torch.zeros(1, 2, 64), dinfer.Rope(64), first=first)
    assert dinfer.Rope(64, scaling="bands", factor=2.0, trained=(1 << 31) - 1).trained == (1 << 31) - 1
