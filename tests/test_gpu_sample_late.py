"""A block that comes late to its cluster: the sampler's waits run out, and nothing else happens.

The test compiles sample.cu with limits of 2 ms and one block of each cluster 20 ms late at one of its
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
V0, EXCHANGES = 40000, 4                                   # V0 + 2 * exchange, + 1: the first block, else the last


def run_late():
    import torch
    import draft_sampling_verification_tcgen05_gb300 as ds
    for V in range(V0, V0 + 2 * EXCHANGES):
        R = 3
        x = torch.randn(R, V, generator=torch.Generator(device="cuda").manual_seed(V), device="cuda")
        row = lambda v, t=torch.float32: torch.full((R,), v, dtype=t, device="cuda")
        ws = ds.Workspace(ds.OP_SAMPLE, R, 1, V)
        probs = torch.empty_like(x)
        ds.dspark_sample(x, row(1.0), row(0, torch.int32), row(0.9), row(0.0), row(0.5), probs=probs, workspace=ws)
        status, bits = ds.dspark_read_status(ws)
        assert status == 4 and bits == ds.STATUS_TIMEOUT, (V, status, bits)
        small = x[:, :5000].contiguous()                   # a block to a row
        tokens = ds.dspark_sample(small, row(0.0), row(0, torch.int32), row(1.0), row(0.0), row(0.5), workspace=ws)
        assert ds.dspark_read_status(ws) == (0, 0)
        assert torch.equal(tokens.long(), small.argmax(dim=1)), V
    print("late blocks: done")


def test_waits_that_run_out_leave_the_gpu_usable(cuda_lib, tmp_path):
    from draft_sampling_verification_tcgen05_gb300 import _build
    _build.build()
    obj, lib = str(tmp_path / "sample.o"), str(tmp_path / "libdspark_late.so")
    late = [f"-DDSPARK_LATE_AT=((p.V-{V0})/2)", f"-DDSPARK_LATE_RANK=((p.V&1)!=0?0:C-1)"]
    include = os.path.join(_build.PKG_DIR, "..", "include")
    for cmd in ([_build._nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, *late, "-I", include, "-c",
                 os.path.join(_build.CSRC, "sample.cu"), "-o", obj],
                [_build._nvcc(), *_build.ARCH, "-shared", "-Xcompiler", "-fPIC", obj, "-o", lib,
                 *(os.path.join(_build.BUILD_DIR, f.replace(".cu", ".o")) for f in _build.SOURCES if f != "sample.cu")]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=dict(os.environ, DSPARK_LIBRARY=lib, PYTHONPATH=ROOT),
                       cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "late blocks: done" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]


if __name__ == "__main__":
    run_late()
