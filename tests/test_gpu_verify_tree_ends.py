"""GPU parity: draws of a tree's verification whose share of the mass lies behind all others, or where one warp's or
block's part of a row ends.

Which block and warp hold a share is found from fp32 sums, which do not add up alike everywhere; the token must be the
integer masses' all the same.  Uniforms next to 1 are the common case: one draw in 2^24 has the largest, and every
uniform that is too large is read as that.
"""
import math

import numpy as np
import pytest

from tests.test_gpu_sample import _weights

pytestmark = pytest.mark.gpu

# vocabulary and requests; with 152 SMs of four blocks: 1, 1, 1, 2, 4, 8 and 16 blocks to a request
SIZES = [(500, 400), (3000, 400), (20011, 700), (5003, 300), (9001, 150), (20011, 75), (151936, 30)]
LARGEST = 1.0 - 2.0 ** -24


def masses(x, T):
    """Inclusive sums of the rows' integer masses: x [R, V] fp32 or bf16, T [R]."""
    import torch
    return torch.floor(_weights(x.float(), T).double() * 2.0 ** 40).long().cumsum(dim=1)


def drawn(ends, u):
    """The definition's token of each row."""
    import torch
    total = ends[:, -1]
    U = torch.floor(u.double() * 2.0 ** 24).long()
    share = (total >> 24) * U + (((total & 0xFFFFFF) * U) >> 24)        # floor(total * U / 2^24), below 2^62
    return torch.searchsorted(ends, share[:, None], right=True)[:, 0].int()


def check(ds, V, B, u, read, seed, bf16, gain, status=0):
    """Three nodes in a row, each the token drawn before, all with the uniforms u [B, 3], which count as `read`."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, 3, V, generator=g, device="cuda") * gain
    x = x.to(torch.bfloat16) if bf16 else x
    T = torch.tensor([0.7, 1.0, 2.5], device="cuda").repeat(-(-B // 3))[:B].contiguous()
    u = u(x, T) if callable(u) else u
    read = u if read is None else read
    want = torch.stack([drawn(masses(x[:, i], T), read[:, i]) for i in range(3)], dim=1)
    tokens = torch.zeros(B, 3, dtype=torch.int32, device="cuda")
    tokens[:, 1:] = want[:, :2]
    chain = torch.tensor([-1, 0, 1], dtype=torch.int32, device="cuda").repeat(B, 1)
    ws = ds.Workspace(ds.OP_VERIFY_TREE, B, 3)
    out, accepted, path = ds.dspark_verify_tree(x, chain, tokens, T, u.contiguous(), workspace=ws)
    assert ds.dspark_read_status(ws)[1] == status
    assert torch.equal(out, want), f"{int((out != want).sum())} of {3 * B} tokens"
    assert bool((accepted == 2).all()) and torch.equal(path, torch.arange(3, dtype=torch.int32, device="cuda").repeat(B, 1))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V,B", SIZES)
def test_uniforms_next_to_one(cuda_lib, V, B, bf16):
    import torch
    for seed in range(-(-400 // B)):
        for gain in (1.0, 3.0):
            for u in (LARGEST, LARGEST - 2.0 ** -24):
                check(cuda_lib, V, B, torch.full((B, 3), u, device="cuda"), None, seed, bf16, gain)


@pytest.mark.parametrize("V,B", SIZES)
def test_uniforms_that_are_too_large(cuda_lib, V, B):
    import torch
    at_most = torch.full((B, 3), LARGEST, device="cuda")
    for seed, u in enumerate((1.0, 1.0000001, 3.0, math.inf)):
        check(cuda_lib, V, B, torch.full((B, 3), u, device="cuda"), at_most, seed, False, 1.0, cuda_lib.STATUS_INPUT_RANGE)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V,B", SIZES)
def test_shares_where_a_warp_s_or_block_s_part_ends(cuda_lib, V, B, bf16):
    """The least uniform past the end of the first k of 128 parts of a row (each count of warps divides 128), and the ones
    before it."""
    import torch

    def u(x, T):
        per, out = 8 if bf16 else 4, torch.empty(B, 3, device="cuda")
        for i in range(3):
            ends = masses(x[:, i], T)
            shift = ((torch.arange(B, device="cuda") * 3 + i) * V) % per      # entries of the first piece ahead of the row
            pieces = (shift + V + per - 1) // per
            k = (torch.arange(B, device="cuda") * 37 + i) % 127 + 1
            entry = (pieces * k // 128 * per - shift).clamp(1, V - 1)         # the first one behind the end
            before, total = ends.gather(1, entry[:, None] - 1)[:, 0], ends[:, -1]
            least = torch.tensor([-(-int(a) * 2 ** 24 // int(q)) for a, q in zip(before.tolist(), total.tolist())], device="cuda")
            out[:, i] = (least - torch.arange(B, device="cuda") % 3).clamp(0, 2 ** 24 - 1).double() * 2.0 ** -24
        return out

    for seed in range(-(-400 // B)):
        check(cuda_lib, V, B, u, None, seed, bf16, 1.0)


def test_the_expected_tokens_are_the_sampling_oracle_s(cuda_lib):
    import torch
    import oracle
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((6, 300)).astype(np.float32)).cuda()
    T = torch.tensor([0.7, 1.0, 2.5] * 2, device="cuda")
    u = torch.tensor([0.0, 0.3, 0.9, LARGEST, 2.0 ** -24, 0.5], device="cuda")
    w = _weights(x, T).cpu().numpy()
    want = [oracle.tree_token(x[r].cpu().numpy(), w[r], float(T[r]), float(u[r])) for r in range(6)]
    assert drawn(masses(x, T), u).tolist() == want
