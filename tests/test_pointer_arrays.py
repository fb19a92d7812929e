"""Pointer lists of the step calls: every form of an address that ctypes takes."""
import ctypes

import numpy as np
import pytest


@pytest.mark.parametrize("given,want", [
    ([1, 2], [1, 2]), ((3,), [3]), ([None, 4], [None, 4]), ([], [None]), ([ctypes.c_void_p(8), 16], [8, 16]),
    ([ctypes.c_void_p(None), ctypes.c_void_p(24)], [None, 24]), ([-1], [2 ** 64 - 1]), ([np.uint64(32)], [32])])
def test_forms_of_addresses(given, want):
    from memory_lean_optimizer_gb300 import lmopt
    assert list(lmopt._ptr_array(given)) == want


def test_others_are_refused():
    from memory_lean_optimizer_gb300 import lmopt
    for bad in ([2.0], [b"x"], ["y"]):
        with pytest.raises(TypeError):
            lmopt._ptr_array(bad)
