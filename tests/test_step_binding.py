"""The binding of a serving loop's other steps (no GPU): what it hands to the library is what the caller holds."""
import copy
import ctypes
import gc
import pickle

import pytest

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
