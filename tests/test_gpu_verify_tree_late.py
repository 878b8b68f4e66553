"""A block that comes late to its cluster: the waits of a tree's verification run out, and nothing else happens.

The test compiles verify_tree.cu with limits of 2 ms and one block of each cluster 20 ms late at one of its
exchanges, both chosen by the vocabulary's size, and calls it in a child process (DSPARK_LIBRARY names that
build).  Each call has to end with TIMEOUT in the status word, and the next call that needs no cluster to be
right.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
V0, EXCHANGES = 40000, 5                                   # V0 + 2 * exchange, + 1: the first block, else the last


def run_late():
    import torch
    import draft_sampling_verification_tcgen05_gb300 as ds
    B, N = 3, 6
    chain = (torch.arange(N, dtype=torch.int32, device="cuda") - 1).repeat(B, 1)
    full = lambda v: torch.full((B,), v, device="cuda")
    u = torch.full((B, N), 0.5, device="cuda")
    for V in range(V0, V0 + 2 * EXCHANGES):
        g = torch.Generator(device="cuda").manual_seed(V)
        x = torch.randn(B, N, V, generator=g, device="cuda")
        tokens = torch.randint(0, V, (B, N), generator=g, device="cuda", dtype=torch.int32)
        x[:, :-1].scatter_(2, tokens[:, 1:, None].long(), 60.0)          # the chain is accepted: two exchanges a row
        for T in (1.0, 0.0) if V < V0 + 4 else (1.0,):
            ws = ds.Workspace(ds.OP_VERIFY_TREE, B, N)
            ds.dspark_verify_tree(x, chain, tokens, full(T), u, workspace=ws)
            status, bits = ds.dspark_read_status(ws)
            assert status == 4 and bits == ds.STATUS_TIMEOUT, (V, T, status, bits)
        small = torch.randn(B, N, 1500, generator=g, device="cuda")      # a block to a request
        out, accepted, path = ds.dspark_verify_tree(small, chain, torch.full_like(tokens, 1500 - 1), workspace=ws)
        assert ds.dspark_read_status(ws) == (0, 0)
        assert torch.equal(out[:, 0].long(), small[:, 0].argmax(dim=1)) and bool((path[:, 0] == 0).all()), V
    print("late blocks: done")


def test_waits_that_run_out_leave_the_gpu_usable(cuda_lib, tmp_path):
    from draft_sampling_verification_tcgen05_gb300 import _build
    _build.build()
    obj, lib = str(tmp_path / "verify_tree.o"), str(tmp_path / "libdspark_late.so")
    late = [f"-DDSPARK_LATE_AT=((t.V-{V0})/2)", "-DDSPARK_LATE_RANK=((t.V&1)!=0?0:C-1)"]
    include = os.path.join(_build.PKG_DIR, "..", "include")
    for cmd in ([_build._nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, *late, "-I", include, "-c",
                 os.path.join(_build.CSRC, "verify_tree.cu"), "-o", obj],
                [_build._nvcc(), *_build.ARCH, "-shared", "-Xcompiler", "-fPIC", obj, "-o", lib,
                 *(os.path.join(_build.BUILD_DIR, f.replace(".cu", ".o")) for f in _build.SOURCES if f != "verify_tree.cu")]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=dict(os.environ, DSPARK_LIBRARY=lib, PYTHONPATH=ROOT),
                       cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "late blocks: done" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]


if __name__ == "__main__":
    run_late()
