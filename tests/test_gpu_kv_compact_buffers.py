"""GPU: dspark_kv_compact with its arrays side by side in one buffer, and with an output that overlaps an input."""
import numpy as np
import pytest

from tests.test_gpu_kv_move import CompactCase, _host, _ints

pytestmark = pytest.mark.gpu


def test_neighbours_in_one_buffer_and_overlaps(cuda_lib):
    import torch
    B = 5
    case = CompactCase(3, 2, 16, 64, [40, 33, 70, 64, 25], 9, lengths=[9, 4, 9, 0, 8])
    buf = torch.full((4 * B,), -7, dtype=torch.int32, device="cuda")
    parts = [buf[i * B:(i + 1) * B] for i in range(4)]
    for part, x in zip(parts, (case.kv_len, None, case.lengths, case.accepted)):
        if x is not None:
            part.copy_(_ints(x))
    table, path, before = _ints(case.table), _ints(case.path), _host(case.k)

    def call(out):
        return cuda_lib.dspark_kv_compact(case.k, case.v, table, parts[0], path, parts[3], lengths=parts[2], kv_len_out=out)

    for out in (parts[0], parts[2], parts[3], buf[1:B + 1], buf[2 * B - 1:3 * B - 1], path[0, :B], table.view(-1)[1:B + 1]):
        with pytest.raises(cuda_lib.DSparkError) as e:
            call(out)
        assert e.value.status == 1
    np.testing.assert_array_equal(_host(case.k), before)
    k, v, lens = case.expected()
    assert call(parts[1]).tolist() == lens
    np.testing.assert_array_equal(_host(case.k), k)
    np.testing.assert_array_equal(_host(case.v), v)
    assert torch.equal(parts[0], _ints(case.kv_len)) and torch.equal(parts[2], _ints(case.lengths))
