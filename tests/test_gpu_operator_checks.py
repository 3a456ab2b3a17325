"""The 4-bit and embedding tests once more under the checks build (see
test_gpu_checks.py): every copy, shared-memory extent, list entry and output
index of their kernels is checked against its buffer before use, and the
conftest fixture fails a test in which a check fired."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_operators_under_the_checks_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_entropy_coded_canonical_b200.build import build
    build(checks=True)
    env = dict(os.environ, DFW_LIBRARY="checks")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_q4.py", "tests/test_gpu_embed.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=840)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-25:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
