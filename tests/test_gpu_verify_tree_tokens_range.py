"""GPU: dspark_verify_tree_tokens takes every token from 0 to 2^31 - 1, and flags only what is below 0."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("token", [0, 1, 2 ** 31 - 2, 2 ** 31 - 1])
def test_the_largest_tokens(cuda_lib, token):
    import torch
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = cuda_lib.Workspace(cuda_lib.OP_VERIFY_TREE, 2, 3)
    parents, draft = i([[-1, 0, 1]] * 2), i([[5, token, 7], [5, 6, token]])
    out, accepted, path = cuda_lib.dspark_verify_tree_tokens(i([[token, 7, 9], [6, token, 8]]), parents, draft, workspace=ws)
    assert cuda_lib.dspark_read_status(ws) == (0, 0)
    assert out.tolist() == [[token, 7, 9], [6, token, 8]] and accepted.tolist() == [2, 2] and path.tolist() == [[0, 1, 2]] * 2


def test_tokens_below_zero(cuda_lib):
    import torch
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for token in (-1, -2 ** 31):
        ws = cuda_lib.Workspace(cuda_lib.OP_VERIFY_TREE, 1, 3)
        out, accepted, path = cuda_lib.dspark_verify_tree_tokens(i([[token, 3, 3]]), i([[-1, 0, 0]]), i([[0, token, 2]]), workspace=ws)
        assert cuda_lib.dspark_read_status(ws)[1] == cuda_lib.STATUS_INPUT_RANGE
        assert out.tolist() == [[token, -1, -1]] and accepted.tolist() == [0] and path.tolist() == [[0, -1, -1]]
