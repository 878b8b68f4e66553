"""dspark_kv_compact refuses an output that shares memory with what its other blocks still read (runs without a GPU)."""
import ctypes

import pytest

from tests.test_abi_serving import FAKE, L, NULL  # noqa: F401  (L: the fixture)

B, N, PAGES = 4, 8, 10
BASE = 1 << 20
INPUTS = {4: B * PAGES * 4, 6: B * 4, 7: B * 4, 8: B * N * 4, 9: B * 4}       # by argument: block_table, kv_len, lengths, path, accepted


def _call(L, change):
    at = ctypes.c_void_p
    args = [FAKE, FAKE, 2, 100 * 4 * 16 * 64, at(BASE), PAGES, at(2 * BASE), at(3 * BASE), at(4 * BASE), at(5 * BASE), B, N, 4, 64, 100, 16,
            at(6 * BASE), FAKE, 256, NULL]
    for i, v in change.items():
        args[i] = v
    return L.dspark_kv_compact(*args)


@pytest.mark.parametrize("argument", sorted(INPUTS))
def test_outputs_that_overlap_an_input_are_refused(L, argument):
    size = INPUTS[argument]
    start = 7 * BASE
    for offset in (-B * 4 + 4, 0, 4, size - 4):
        assert _call(L, {argument: ctypes.c_void_p(start), 16: ctypes.c_void_p(start + offset)}) == 1, offset
    L.dspark_last_error.restype = ctypes.c_char_p
    assert b"overlap" in L.dspark_last_error()


def test_the_same_call_goes_on_to_the_device_without_an_overlap(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    assert _call(L, {}) == _call(L, {7: NULL}) == 2                           # no device here
    for argument, size in INPUTS.items():
        for offset in (-B * 4, size):                                         # next to it, on either side
            assert _call(L, {argument: ctypes.c_void_p(7 * BASE), 16: ctypes.c_void_p(7 * BASE + offset)}) == 2
