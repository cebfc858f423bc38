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


def test_workspaces_do_not_grow_with_the_sequences(lib):
    """A state for each segment of the time axis, and copies of the first states that another segment may
    overwrite: at most one for each cut."""
    state = 4 * 128 * 128
    for nseq in (2, 100, 8192, 1 << 20):
        dims = lz.lizard_decay_dims(B=1, L=65536, Hq=32, Hkv=8, dk=128, dv=128, nseq=nseq, scale=1.0, dtype=1)
        assert lz.lizard_decay_attn_fwd_workspace(dims) <= 256 + 2 * 152 * state
        assert lz.lizard_decay_attn_bwd_workspace(dims) <= 256 + 3 * 152 * state
        dims.dtype = 0  # fp32 arithmetic: segments for one CTA of 64 columns a SM
        assert lz.lizard_decay_attn_bwd_workspace(dims) <= 256 + 3 * 152 * state
    one = lz.lizard_decay_dims(B=1, L=65536, Hq=8, Hkv=8, dk=128, dv=128, nseq=1, scale=1.0, dtype=1)
    assert lz.lizard_decay_attn_fwd_workspace(one) == 256 + (19 + 1) * 8 * state  # 19 segments of 8 heads; one first state
