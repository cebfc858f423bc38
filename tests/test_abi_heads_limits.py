"""The C ABI of the rotation and of the decay attention at the limits of their sizes, without a GPU."""
import json
import os
import subprocess
import sys

import pytest

from gated_linear_sliding_gb300 import _build
from gated_linear_sliding_gb300 import lizard as lz

pytest.importorskip("torch")

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return lz.load()


def test_heads_wider_than_the_kernels_are_refused(lib):
    """Widths are looked at in 64 bits: 2^32 + 128 is not 128, and 2^31 is not negative."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, os.path.join(HERE, "_abi_heads_limits.py")], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    codes = json.loads(r.stdout.strip().splitlines()[-1])
    assert codes == {k: 0 if k.startswith("workspace") else lz.LIZARD_ERR_UNSUPPORTED for k in codes} and len(codes) == 30
