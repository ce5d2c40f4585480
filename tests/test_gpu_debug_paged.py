"""Bounded waits of the attention over pages and packed rows that run out (needs a B200): the call
ends, the status word says so, and the next call on the same workspace is right.

No GPU is faulted: the debug library, in a child process, makes the waits short and lets the kernels
expect more bytes than their copies bring (see test_gpu_debug.py)."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_waits_that_run_out_are_reported_and_recovered_from():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from decode_attention_kivi_b200 import build

    env = dict(os.environ, KIVI_LIBRARY=build.build(debug=True),
               PYTHONPATH=os.pathsep.join([ROOT, HERE]))
    r = subprocess.run([sys.executable, os.path.join(HERE, "gpu_debug_paged_child.py")], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "waits: ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
