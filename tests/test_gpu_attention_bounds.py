"""The attention, cache and norm cases again, on the bounds-checked build of the library
(-DCSA_DEBUG_BOUNDS): every output row that the attention kernels store is checked against the
outputs' extent and, instead of writing outside, the store is skipped and bit 8 of the handle's flag
raised, which the cases read back through csa_attention_status.  They run in a child process (the
library is loaded once per process) with CSA_LIBRARY_VARIANT=bounds, and with them the time-out path
(a test hook of this build only)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_attention_cases_on_the_bounds_checked_build():
    sys.path.insert(0, ROOT)
    from deepseek_v4_compressed_wkv_gb300 import build as b
    b.build(variant="bounds")
    env = dict(os.environ, CSA_LIBRARY_VARIANT="bounds")
    cases = [os.path.join(HERE, f) for f in ("test_gpu_attention.py", "test_gpu_layer_ops.py", "test_gpu_attention_calls.py",
                                             "test_gpu_attention_timeout.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *cases],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert "skipped" not in r.stdout.splitlines()[-1], r.stdout[-500:]
