"""The bounds-checked build (libsr_checked.so) on ragged calls of the elementwise recurrence, its gradients, the append to
the paged cache and the attention over it: no index outside its buffer, and the definitions' results."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_checked_build_runs_clean():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, SR_LIBRARY="libsr_checked.so")
    r = subprocess.run([sys.executable, os.path.join(HERE, "_checked_cases_cache.py")], env=env, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "every case clean" in r.stdout
