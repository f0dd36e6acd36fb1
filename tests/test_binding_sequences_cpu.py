"""What the binding takes for arrays of pointers and sizes: any sequence of whole numbers, by value."""
import ctypes
from array import array

import numpy as np
import pytest

from cross_vendor_gradient_gb300 import binding as B

VALUES = [3, 0, 7, 120]


def as_list(c_array, n):
    return [int(c_array[i] or 0) for i in range(n)]


@pytest.mark.parametrize("typecode", list("bBhHiIlLqQfd"))
@pytest.mark.parametrize("convert", [B._ptrs, B._sizes], ids=["pointers", "sizes"])
def test_arrays_of_every_type_are_taken_by_value(convert, typecode):
    assert as_list(convert(array(typecode, VALUES)), 4) == VALUES
    assert len(convert(array(typecode))) == 1  # of nothing: one entry, not read


@pytest.mark.parametrize("convert", [B._ptrs, B._sizes], ids=["pointers", "sizes"])
def test_other_sequences(convert):
    big = [1 << 40, (1 << 63) + 5]
    for seq in (VALUES, tuple(VALUES), np.array(VALUES), np.array(VALUES, np.uint8), [np.int32(v) for v in VALUES],
                [float(v) for v in VALUES], np.array(VALUES, np.float32)):
        assert as_list(convert(seq), 4) == VALUES
    for seq in (big, array("Q", big), np.array(big, np.uint64)):
        assert as_list(convert(seq), 2) == big
    assert as_list(B._ptrs([None, 16, None]), 3) == [0, 16, 0]


def test_arrays_reach_the_library_by_value():
    st, c = B.gb_create([1])
    assert st == B.GB_OK
    n = 1 << 38  # the most elements that a call takes, twice: refused by their sum, before any device call
    out = 0x40000
    assert B.gb_grad_norm(c, array("Q", [0x10000, 0x20000]), array("d", [n, n]), B.GB_F32, 0.0, out) == B.GB_ERR_INVALID_ARG
    assert B.gb_adamw_step(c, array("I", [0]), array("I", [0]), array("I", [0]), array("I", [0]), None, array("H", [0]),
                           B.GB_F32, B.GB_CODEC_NONE, 256, B.Adamw(1e-3, 0.9, 0.99, 1e-8, 0.0, 1, 0)) == B.GB_OK
    B.gb_destroy(c)
    assert ctypes.sizeof(ctypes.c_size_t) == 8
