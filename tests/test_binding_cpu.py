"""CPU checks of the binding's argument marshalling: every way to give the ranks'
pointers yields the same array."""
import struct

import numpy as np
import pytest


@pytest.fixture(scope="module")
def fcc():
    import __graft_entry__
    __graft_entry__.build()
    import gemm_collective_gb300 as m
    return m


class Buffer:
    def __init__(self, at):
        self.at = at

    def data_ptr(self):
        return self.at


@pytest.mark.parametrize("n", [1, 3, 8, 64, 65, 200])
def test_pointer_arrays_hold_every_address(fcc, n):
    at = [16 * (i + 1) for i in range(n)]
    want = struct.pack(f"{n}P", *at)
    tensors = [Buffer(a) for a in at]
    mixed = [a if i % 2 else Buffer(a) for i, a in enumerate(at)]
    for seq in (at, tuple(at), map(int, at), (a for a in at), iter(at), np.array(at, np.uint64),
                tensors, map(Buffer, at), iter(tensors), mixed, iter(mixed), mixed[::-1][::-1],
                dict.fromkeys(at), dict(enumerate(tensors)).values()):
        assert bytes(fcc._ptrs(seq)) == want
    for seq in (at, map(int, at), iter(mixed), map(Buffer, at)):
        assert bytes(fcc.ptr_array(seq)) == want
    assert fcc._ptrs(None) is None
    built = fcc.ptr_array(at)
    assert fcc._ptrs(built) is built
    none = [None] + at[1:]
    assert bytes(fcc._ptrs(iter(none))) == struct.pack(f"{n}P", 0, *at[1:])
