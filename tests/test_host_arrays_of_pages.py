"""Page lists as the binding hands them to the library (no GPU): the same values whatever they come in."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def H():
    from sparse_mla_kv_indexer_gb300 import build
    build.build()
    from sparse_mla_kv_indexer_gb300 import hisparse
    return hisparse


def read(H, values, ctype):
    at, keep = H._host_array(values, ctype)
    address = at if isinstance(at, int) else at.value
    return list((ctype * len(values)).from_address(address)) if len(values) else []


@pytest.mark.parametrize("ctype,big", [(ctypes.c_int32, 2 ** 31 - 1), (ctypes.c_int64, 2 ** 63 - 1)])
def test_values_of_every_kind(H, ctype, big):
    want = [-1, 0, 5, big, -big - 1, 7]
    kinds = [want, tuple(want), np.array(want, np.int64), [np.int64(x) for x in want]]
    torch = pytest.importorskip("torch")
    kinds.append(torch.tensor(want, dtype=torch.int64))
    if ctype is ctypes.c_int32:
        kinds += [np.array(want, np.int32), torch.tensor(want, dtype=torch.int32)]
    for values in kinds:
        assert read(H, values, ctype) == want, type(values)
    # what int() takes and an index is not; bytes, element by element; more bits than there are: the low ones
    assert read(H, [3.0, np.float32(4.0), "5", True], ctype) == [3, 4, 5, 1]
    assert read(H, b"\x01\x02\x03\x04\x05\x06\x07\xff", ctype) == [1, 2, 3, 4, 5, 6, 7, 255]
    assert read(H, bytearray(b"\x09\x08"), ctype) == [9, 8]
    assert read(H, [2 ** 64 + 3, 1], ctype) == [3, 1]
    assert read(H, range(3), ctype) == [0, 1, 2]
    assert read(H, [], ctype) == [] and H._host_array(None, ctype) is None
    with pytest.raises((TypeError, ValueError)):
        H._host_array([None], ctype)


def test_the_values_are_taken_when_the_call_is_made(H):
    values = [1, 2, 3]
    at, keep = H._host_array(values, ctypes.c_int32)
    values[0] = 9
    assert list((ctypes.c_int32 * 3).from_address(at)) == [1, 2, 3] and len(keep) == 3
