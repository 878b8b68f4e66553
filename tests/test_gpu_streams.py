"""What a call on a given stream allocates belongs to that stream.

Memory of the current stream would be given to the current stream's next work as soon as the call returns (the
workspace) or the output is dropped, while the given stream may still use it.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _calls(ds):
    import torch
    f32 = lambda *size: torch.rand(*size, device="cuda")
    i32 = lambda *size, v=0: torch.full(size, v, dtype=torch.int32, device="cuda")
    bf = lambda *size: torch.randn(*size, device="cuda").to(torch.bfloat16)
    q, kv, cache = bf(4, 4, 64), bf(4, 2, 64), bf(2, 2, 16, 64)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    p = torch.softmax(f32(2, 3, 50), -1)
    return {
        "draft_logits": (ds.dspark_draft_logits, (bf(4, 64), bf(50, 64))),
        "markov_sample": (ds.dspark_markov_sample, (f32(2, 2, 50), i32(2), f32(50, 8), f32(50, 8), f32(2), 1, 0)),
        "verify": (ds.dspark_verify, (p, p[:, :2].contiguous(), i32(2, 2), None, 1, 0)),
        "verify_greedy": (ds.dspark_verify_greedy, (f32(2, 3, 50), i32(2, 2), None)),
        "schedule": (ds.dspark_schedule, (f32(2, 3), None, 3)),
        "kv_append": (ds.dspark_kv_append, (q, kv, kv, slots, slots, f32(8, 64), cache, cache.clone())),
        "paged_attention": (ds.dspark_paged_attention, (q.view(2, 2, 4, 64), cache, cache, i32(2, 1), i32(2, v=5), 0.1)),
        "prompt_attention": (ds.dspark_prompt_attention, (q, kv, kv, i32(1).new_tensor([0, 4]), 0.1)),
        "sample": (ds.dspark_sample, (f32(2, 50), f32(2), i32(2), f32(2), f32(2), f32(2))),
    }


@pytest.mark.parametrize("name", ["draft_logits", "markov_sample", "verify", "verify_greedy", "schedule", "kv_append",
                                  "paged_attention", "prompt_attention", "sample"])
def test_allocations_belong_to_the_given_stream(cuda_lib, name, monkeypatch):
    import torch
    call, args = _calls(cuda_lib)[name]
    flat = lambda r: list(r) if isinstance(r, tuple) else [r]
    want = [x.clone() for x in flat(call(*args))]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = []
    for maker in ("empty", "empty_like"):
        plain = getattr(torch, maker)

        def recorded(*a, plain=plain, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return plain(*a, **kw)

        monkeypatch.setattr(torch, maker, recorded)
    got = flat(call(*args, stream=other))
    current = torch.cuda.current_stream().cuda_stream
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert len(seen) >= 2 and set(seen) == {other.cuda_stream}             # an output and the workspace
    assert current != other.cuda_stream                                    # as it was before the call
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    seen.clear()


def test_a_stream_of_another_library(cuda_lib):
    """Anything with a cuda_stream attribute names a stream."""
    import torch
    call, args = _calls(cuda_lib)["sample"]

    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    other = torch.cuda.Stream()
    want = call(*args)
    torch.cuda.synchronize()
    got = call(*args, stream=Handle(other))
    other.synchronize()
    assert np.array_equal(want.cpu().numpy(), got.cpu().numpy())
