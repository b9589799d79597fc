"""Cases of the attention layer's operators on the bounds-checked build of the library
(-DCSA_DEBUG_BOUNDS): every store with a computed index of the attention's kernels (outputs, pieces,
their statistics, records), of the cache write and of the norm is checked, left out where it is outside,
and reported.  Some cases need the build's test hooks.  They run in child processes with
CSA_LIBRARY_VARIANT=bounds (the library is loaded once per process)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def run_on_the_bounds_checked_build(*files):
    sys.path.insert(0, ROOT)
    from deepseek_v4_compressed_wkv_gb300 import build as b
    b.build(variant="bounds")
    env = dict(os.environ, CSA_LIBRARY_VARIANT="bounds")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        *(os.path.join(HERE, f) for f in files)],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert "skipped" not in r.stdout.splitlines()[-1], r.stdout[-500:]


def test_segments_published_late():
    run_on_the_bounds_checked_build("test_gpu_attention_late.py")


def test_the_checks_themselves():
    run_on_the_bounds_checked_build("test_gpu_layer_extents.py")


def test_values_and_streams():
    run_on_the_bounds_checked_build("test_gpu_attention_values.py", "test_gpu_layer_streams.py")
