"""The checked build runs the other suites of the operators around an FP8 projection too: a token an adapter, hidden rows,
rows that do not reach each other, the largest sizes and memory past 2^31 elements, the chain."""
import os
import subprocess
import sys

import pytest

from test_gpu_checks import ROOT, _checked_library

pytestmark = pytest.mark.gpu
SUITES = ["test_gpu_lora_few.py", "test_gpu_moe_hidden.py", "test_gpu_layer_rows.py", "test_gpu_layer_limits.py",
          "test_gpu_layer_mean.py", "test_gpu_layer_grid.py", "test_gpu_layer_chain.py"]


def test_the_other_layer_suites_on_the_checked_build():
    env = dict(os.environ, FP8Q_LIBRARY=_checked_library())
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu",
                        *(os.path.join("tests", s) for s in SUITES)], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
