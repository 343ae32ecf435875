"""Ranges of columns of one buffer as logits and output: their rows lie between one another and are no overlap."""
import ctypes

import pytest

at = ctypes.c_void_p
BASE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from semi_autoregressive_drafting_gb300 import _build, _lib
    _build.build()
    return _lib.load()


# (bytes between the first rows, types, stride of both in bytes, whether rows share memory), V = 100 entries
CASES = [(400, 0, 0, 800, False), (400, 0, 0, 796, True), (396, 0, 0, 800, True), (404, 0, 0, 804, False),
         (404, 0, 0, 800, True), (-400, 0, 0, 800, False), (-396, 0, 0, 800, True), (800 + 400, 0, 0, 800, False),
         (800, 0, 0, 800, True), (200, 1, 0, 600, False), (400, 0, 1, 600, False), (400, 1, 0, 600, True),
         (-400, 1, 0, 600, False), (-200, 0, 1, 600, False), (200, 1, 1, 400, False), (-1600 - 200, 1, 1, 400, False),
         (198, 1, 1, 400, True)]


@pytest.mark.parametrize("shift,idt,odt,row,shared", CASES)
def test_columns(lib, shift, idt, odt, row, shared):
    # (a call whose arrays are let through is refused for another reason, so nothing is ever launched)
    size = (4, 2)
    z, out, ld, old = at(BASE), at(BASE + shift), row // size[idt], row // size[odt]
    assert lib.dspark_process_logits_grad(4, 2, 100, idt, z, ld, odt, None, 99, None, 0, 0, None, None, None, None, None, 0,
                                          0, None, out, old, None) == 1
    assert (b"overlaps" in lib.dspark_last_error()) == shared
    if idt == odt:
        for call in (lambda: lib.dspark_distill_loss(8, 100, 1.0, idt, z, ld, 5, z, z, None, 1.0, 0.0, 1, z, None, None,
                                                       out, old, None, 0, None),
                     lambda: lib.dspark_distill_grad(8, 100, 1.0, idt, z, ld, 5, z, z, z, z, 1.0, 0.0, 1, out, old,
                                                       None, 0, None)):
            assert call() == (1 if shared else 2)
