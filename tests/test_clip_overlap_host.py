"""Host tests (no GPU work) of the clipping's refusal of memory that two tensors would
share. Every call ends in an argument check: lists without overlap in that of the
workspace, which is too small."""
import ctypes
import os
import random

import pytest

pytest.importorskip("quantized_linear_layer_amd")
from quantized_linear_layer_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libfp4lin.so not built (run __graft_entry__.build())", allow_module_level=True)

L = _lib.load()
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced
A, B, C, D = 0x100000, 0x200000, 0x300000, 0x400000


def clip(entries):
    a = (_lib.Grad * len(entries))(*(_lib.Grad(*e) for e in entries))
    return L.fp4lin_clip_grads(a, len(entries), 1.0, FAKE, FAKE, 16, None)


def norm(entries):
    a = (_lib.Grad * len(entries))(*(_lib.Grad(*e) for e in entries))
    return L.fp4lin_grad_norm(a, len(entries), FAKE, FAKE, 16, None)


@pytest.mark.parametrize("entries", [
    [(A, A, 100, 0), (B, B, 100, 0), (A, A, 100, 0)],      # in place, listed twice
    [(A, C, 100, 0), (B, C, 100, 0)],                      # one output for two
    [(A, B, 100, 0), (B, C, 100, 0)],                      # an output on another's gradient
    [(A, B, 100, 0), (B, A, 100, 0)],
    [(A, A, 100, 0), (A, C, 100, 0)],
    [(A, A + 4, 100, 0)],                                  # on its own, but not in place
    [(A, A, 100, 0), (A + 396, A + 396, 1, 0)],            # the last element
    [(A, A, 100, 1), (A + 198, A + 198, 1, 1)],
    [(A, A, 1000, 0), (B, B, 8, 0), (A + 800, C, 8, 0)],   # inside a longer one
])
def test_shared_memory_is_refused(entries):
    assert clip(entries) == _lib.ERR_OVERLAP
    assert clip(entries[::-1]) == _lib.ERR_OVERLAP
    assert norm(entries) == _lib.ERR_WORKSPACE  # nothing is written but the norm


@pytest.mark.parametrize("entries", [
    [(A, A, 100, 0), (B, B, 100, 0)],
    [(A, B, 100, 0), (C, D, 100, 0)],
    [(A, B, 100, 0), (A, C, 100, 0)],                      # a gradient read twice
    [(A, A, 100, 0), (A + 400, A + 400, 1, 0)],            # neighbours
    [(A, A, 100, 1), (A + 200, A + 200, 1, 0)],
    [(A, A + 400, 100, 0)],
    [(A, A, 100, 0), (A, A, 0, 0), (None, None, 0, 0)],    # no elements
])
def test_separate_memory_is_not(entries):
    assert clip(entries) == _lib.ERR_WORKSPACE
    assert clip(entries[::-1]) == _lib.ERR_WORKSPACE


@pytest.mark.parametrize("count", [511, 512, 513, 1025, 2000])
def test_long_lists(count):
    """A shared output is found wherever its two entries are."""
    rng = random.Random(count)
    entries = [(A + 0x1000 * i, A + 0x1000 * i, 1024, 0) for i in range(count)]
    rng.shuffle(entries)
    assert clip(entries) == _lib.ERR_WORKSPACE
    for _ in range(5):
        i, j = rng.sample(range(count), 2)
        some = list(entries)
        some[i] = (D * 16, entries[j][1] + 4092, 1, 0)
        assert clip(some) == _lib.ERR_OVERLAP, (i, j)


def test_status_string():
    assert "overlap" in L.fp4lin_status_str(_lib.ERR_OVERLAP).decode()
