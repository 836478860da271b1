"""The checked build (device-side bounds checks) runs the suites of the
operators around an FP8 projection with a clean status word: every computed
store index stays inside the extent its arguments give."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_layer_suites_on_the_checked_build():
    import importlib.util
    root = os.path.dirname(HERE)
    spec = importlib.util.spec_from_file_location("fp8q_build", os.path.join(root, "fine_grained_fp8_x128_b200", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    env = dict(os.environ, FP8Q_LIBRARY=b.build(checks=True))
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu",
                        os.path.join(HERE, "test_gpu_layer_norm.py"), os.path.join(HERE, "test_gpu_moe_few.py"),
                        os.path.join(HERE, "test_gpu_lora.py")], env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
