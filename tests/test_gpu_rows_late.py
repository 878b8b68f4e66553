"""The two softmax threads of a row tell each other their maxima, and at the end their sums: neither may write before the
other has read.

The test compiles an attention kernel with one of the two 50 us late where it reads the other's maximum (which one
changes with the rows and the work items), runs it in a child process (DSPARK_LIBRARY names that build), and compares with
the 64-bit oracle there and bit for bit with the library as it is here.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LATE = "-DDSPARK_LATE_PART=static_cast<int>((quad+count)&1u)"


def windows(ds):
    """Rows of more than one tile over a single key tile, and over several whose scores grow to the last."""
    import torch
    from tests._trees import WindowCase
    got = []
    for dtype in ("bf16", "f16"):
        for D in (64, 128):
            for lens, grow in (([40, 77, 100, 128, 64, 41], False), ([128, 300, 257, 513], True)):
                case = WindowCase(len(lens), 40, 16, 4, D, 16, lens, dtype, seed=D, window=10 ** 6, sinks=0)
                for b, L in enumerate(lens if grow else []):
                    j = np.arange(L)
                    ramp = torch.linspace(0.01, 4.0, L, device="cuda")[:, None, None] * case.q[b, 0, ::4].float()
                    case.k[case.table[b, j // 16], :, j % 16] = ramp.to(case.k.dtype)
                for causal in (True, False):
                    got += case.check(ds, causal=causal, rows=60)
    return got


def prompts(ds):
    """Prompts of a single key tile, and longer ones whose scores grow to the last."""
    import torch
    from tests.test_gpu_prompt_attention import _check, _cu, _inputs
    got = []
    for dtype in ("bf16", "f16"):
        for D in (64, 128):
            for lens, grow in (([100, 1, 128, 77, 64, 65, 128, 33], False), ([300, 129, 513], True)):
                q, k, v = _inputs(sum(lens), 16, 4, D, dtype, D)
                if grow:
                    ramp = torch.cat([torch.linspace(0.01, 4.0, n, device="cuda") for n in lens])[:, None, None]
                    k = (ramp * torch.cat([q[a:a + 1, ::4].expand(n, -1, -1) for a, n in zip(_cu(lens), lens)]).float()).to(q.dtype)
                for causal in (True, False):
                    got += _check(ds, q, k, v, _cu(lens), dtype, causal, rows=60)
    return got


def _late_library(tmp_path, source):
    from draft_sampling_verification_tcgen05_gb300 import _build
    _build.build()
    obj, lib = str(tmp_path / "late.o"), str(tmp_path / "libdspark_late.so")
    include = os.path.join(_build.PKG_DIR, "..", "include")
    for cmd in ([_build._nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, LATE, "-I", include, "-c", os.path.join(_build.CSRC, source),
                 "-o", obj],
                [_build._nvcc(), *_build.ARCH, "-shared", "-Xcompiler", "-fPIC", obj, "-o", lib,
                 *(os.path.join(_build.BUILD_DIR, f.replace(".cu", ".o")) for f in _build.SOURCES if f != source)]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
    return lib


@pytest.mark.parametrize("source,cases", [("masked_attention.cu", "windows"), ("prompt_attention.cu", "prompts")])
def test_a_half_that_reads_late(cuda_lib, tmp_path, source, cases):
    import torch
    lib, out = _late_library(tmp_path, source), str(tmp_path / "late.pt")
    r = subprocess.run([sys.executable, os.path.abspath(__file__), cases, out], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, DSPARK_LIBRARY=lib, PYTHONPATH=ROOT))
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    late, here = torch.load(out), globals()[cases](cuda_lib)
    assert len(late) == len(here) and all(torch.equal(a, b.cpu()) for a, b in zip(late, here))


if __name__ == "__main__":
    import torch
    import draft_sampling_verification_tcgen05_gb300 as ds
    torch.save([t.cpu() for t in globals()[sys.argv[1]](ds)], sys.argv[2])
