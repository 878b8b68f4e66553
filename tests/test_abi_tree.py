"""Host-side validation of the tree operators' C entry points (runs without a GPU)."""
import ctypes
import math

import pytest

from tests.test_abi_serving import FAKE, L, NULL, ODD, _refused  # noqa: F401  (L: the fixture)

OTHER = ctypes.c_void_p(8192)


def test_workspace_sizes(L):
    paged = L.dspark_workspace_size(10, 4, 8, 16, 128)
    assert L.dspark_workspace_size(14, 4, 8, 16, 128) == paged
    assert L.dspark_workspace_size(13, 4, 8, 16, 128) >= paged + 4 * 8 * 8
    assert L.dspark_workspace_size(13, 4, 33, 16, 128) >= L.dspark_workspace_size(10, 4, 33, 16, 128) + 4 * 33 * 12
    for op in (13, 14):
        assert L.dspark_workspace_size(op, 0, 8, 16, 128) == 0 and L.dspark_workspace_size(op, 4, -1, 16, 128) == 0
    for op in (15, 16, 17):
        assert L.dspark_workspace_size(op, 4, 8, 0, 0) == 256
    assert L.dspark_workspace_size(18, 4, 8, 0, 0) == 0


def test_tree_attention(L):
    need = L.dspark_workspace_size(13, 4, 8, 16, 128)
    good = [FAKE, FAKE, FAKE, 1, FAKE, 10, FAKE, NULL, FAKE, 0, 0, 0.1, 4, 8, 16, 4, 128, 100, 16, FAKE, NULL, FAKE, need, NULL]
    _refused(L.dspark_tree_attention, good, [
        (0, NULL), (1, NULL), (2, NULL), (3, 0), (4, NULL), (5, 0), (6, NULL), (8, NULL), (9, 7), (9, -1), (10, -1),
        (11, math.inf), (11, math.nan), (12, 0), (12, 65536), (13, 0), (13, 257), (14, 18), (15, 0), (16, 96), (17, 0), (18, 12),
        (18, 512), (19, NULL), (19, ODD), (21, NULL), (22, need - 256)])


def test_window_attention(L):
    need = L.dspark_workspace_size(14, 4, 8, 16, 128)
    good = [FAKE, FAKE, FAKE, 1, FAKE, 10, FAKE, NULL, 64, 4, 0.1, 1, 4, 8, 16, 4, 128, 100, 16, FAKE, NULL, FAKE, need, NULL]
    _refused(L.dspark_window_attention, good, [
        (0, NULL), (1, ODD), (2, NULL), (3, 0), (4, NULL), (5, 0), (6, NULL), (8, 0), (8, -5), (9, -1), (10, math.nan), (12, 0),
        (13, 65536), (14, 18), (15, 0), (16, 32), (17, 0), (18, 4), (19, NULL), (21, ODD), (22, need - 256)])


def test_verify_tree(L):
    good = [FAKE, 0, FAKE, FAKE, FAKE, FAKE, NULL, 4, 8, 1000, FAKE, FAKE, FAKE, FAKE, 256, NULL]
    _refused(L.dspark_verify_tree, good, [
        (0, NULL), (0, ODD), (1, 2), (3, NULL), (4, NULL), (5, NULL), (7, 0), (7, 65536), (8, 0), (8, 257), (9, 0), (9, (1 << 21) + 1),
        (10, NULL), (11, NULL), (12, NULL), (13, NULL), (13, ODD), (14, 128)])
    good = [FAKE, FAKE, FAKE, NULL, 4, 8, FAKE, FAKE, FAKE, FAKE, 256, NULL]
    _refused(L.dspark_verify_tree_tokens, good, [
        (0, NULL), (1, NULL), (2, NULL), (4, 0), (4, 65536), (5, 0), (5, 257), (6, NULL), (7, NULL), (8, NULL), (9, NULL), (10, 64)])


def test_kv_compact(L):
    good = [FAKE, FAKE, 2, 100 * 4 * 16 * 64, FAKE, 10, FAKE, NULL, FAKE, FAKE, 4, 8, 4, 64, 100, 16, OTHER, FAKE, 256, NULL]
    _refused(L.dspark_kv_compact, good, [
        (0, NULL), (0, ODD), (1, ODD), (2, 0), (2, 1 << 17), (3, 100 * 4 * 16 * 64 - 8), (3, 100 * 4 * 16 * 64 + 4), (4, NULL), (5, 0),
        (5, 1 << 28), (6, NULL), (8, NULL), (9, NULL), (10, 0), (11, 0), (11, 257), (12, 0), (13, 4), (13, 60), (13, 520), (14, 0),
        (14, 1 << 30), (15, 0), (16, NULL), (16, FAKE), (17, NULL), (18, 128)])


def test_kv_copy_pages(L):
    good = [FAKE, FAKE, 2, 100 * 4 * 16 * 64, FAKE, FAKE, NULL, 3, 4, 64, 100, 16, FAKE, 256, NULL]
    _refused(L.dspark_kv_copy_pages, good, [
        (0, NULL), (1, ODD), (2, 0), (3, 8), (3, 100 * 4 * 16 * 64 + 1), (4, NULL), (5, NULL), (7, 0), (8, 0), (9, 12), (9, 1024),
        (10, 0), (11, 0), (11, 1 << 26), (12, NULL), (13, 255)])


def test_python_refuses_tensors_off_the_gpu(L):
    """The binding looks at its arguments before anything else: CPU tensors are refused by name."""
    import torch

    import draft_sampling_verification_tcgen05_gb300 as ds
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    q, cache = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: ds.dspark_tree_attention(q, cache, cache, i32(2, 2), i32(2), i32(2, 3), 0.1),
                 lambda: ds.dspark_window_attention(q, cache, cache, i32(2, 2), i32(2), 4, 0, 0.1),
                 lambda: ds.dspark_verify_tree(torch.zeros(2, 3, 10), i32(2, 3), i32(2, 3)),
                 lambda: ds.dspark_verify_tree_tokens(i32(2, 3), i32(2, 3), i32(2, 3)),
                 lambda: ds.dspark_kv_compact(cache, cache, i32(2, 2), i32(2), i32(2, 3), i32(2)),
                 lambda: ds.dspark_kv_copy_pages(cache, cache, i32(1), i32(1))):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
