"""Host-side validation of the serving operators' C entry points (runs without a GPU)."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def L():
    from draft_sampling_verification_tcgen05_gb300 import _build
    _build.build()
    import draft_sampling_verification_tcgen05_gb300 as ds
    return ds.lib()


NULL, FAKE, ODD = ctypes.c_void_p(0), ctypes.c_void_p(4096), ctypes.c_void_p(4104)    # never dereferenced


def _refused(fn, good, changes):
    for i, v in changes:
        args = list(good)
        args[i] = v
        assert fn(*args) == 1, (i, v)


def test_workspace_sizes(L):
    assert L.dspark_workspace_size(8, 4, 4, 1000, 64) == 256
    assert L.dspark_workspace_size(12, 4, 1, 1000, 0) >= 256 + 4 * 4
    assert L.dspark_workspace_size(12, 0, 1, 1000, 0) == 0
    assert L.dspark_workspace_size(11, 4, 1000, 16, 0) >= 256 + 16 * (4 + 1000 // 64)
    assert L.dspark_workspace_size(11, 4, 0, 16, 0) == 0
    assert L.dspark_workspace_size(10, 4, 4, 32, 128) >= 256
    assert L.dspark_workspace_size(10, 0, 4, 32, 128) == 0


def test_kv_append(L):
    good = [FAKE, FAKE, FAKE, 1, 1024, 256, 256, FAKE, FAKE, FAKE, 100, 64, 0, NULL, NULL, 1e-6, 10, 16, 4, 64, FAKE, FAKE,
            FAKE, 8, 16, FAKE, 256, NULL]
    _refused(L.dspark_kv_append, good, [
        (0, NULL), (1, NULL), (2, NULL), (3, 0), (3, 7), (4, 1016), (4, 1028), (5, 8), (6, 260), (7, NULL), (8, NULL),
        (9, NULL), (10, 0), (11, 24), (11, 80), (16, 0), (17, -1), (18, 0), (19, 72), (19, 528), (20, NULL), (20, ODD),
        (21, NULL), (22, ODD), (23, 0), (24, 0), (23, 1 << 30), (25, NULL), (26, 128)])


def test_paged_attention(L):
    need = L.dspark_workspace_size(10, 4, 8, 16, 128)
    good = [FAKE, FAKE, FAKE, 1, FAKE, 10, FAKE, NULL, 0.1, 1, 4, 8, 16, 4, 128, 100, 16, FAKE, NULL, FAKE, need, NULL]
    _refused(L.dspark_paged_attention, good, [
        (0, NULL), (1, NULL), (2, NULL), (3, 0), (4, NULL), (5, 0), (6, NULL), (8, math.inf), (8, math.nan), (10, 0),
        (10, 65536), (11, 0), (12, 18), (13, 0), (14, 96), (15, 0), (16, 12), (16, 4), (16, 512), (17, NULL), (17, ODD),
        (19, NULL), (20, 64)])


def test_prompt_attention(L):
    need = L.dspark_workspace_size(11, 2, 50, 16, 0)
    good = [FAKE, FAKE, FAKE, 2, 1024, 256, 256, FAKE, 0.1, 1, 2, 50, 16, 4, 64, FAKE, NULL, FAKE, need, NULL]
    _refused(L.dspark_prompt_attention, good, [
        (0, NULL), (1, NULL), (2, ODD), (3, 0), (4, 1020), (5, 128), (6, 1 << 31), (7, NULL), (8, math.nan), (10, 0),
        (11, 0), (11, (1 << 24) + 1), (12, 15), (13, 0), (14, 80), (15, NULL), (18, 16)])


def test_sample(L):
    need = L.dspark_workspace_size(12, 4, 1, 1000, 0)
    good = [FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 1000, FAKE, NULL, FAKE, need, NULL]
    _refused(L.dspark_sample, good, [
        (0, NULL), (0, ODD), (1, 2), (2, NULL), (3, NULL), (4, NULL), (5, NULL), (6, NULL), (7, 0), (8, 0),
        (8, (1 << 21) + 1), (9, NULL), (10, ODD), (11, NULL), (12, 128)])
