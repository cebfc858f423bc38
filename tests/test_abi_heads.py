"""The C ABI and binding of the rotation and of the decay attention without a GPU: struct layouts,
workspace queries and every refusal that happens on the host."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

from gated_linear_sliding_gb300 import _build
from gated_linear_sliding_gb300 import lizard as lz

torch = pytest.importorskip("torch")

HERE = os.path.dirname(os.path.abspath(__file__))
INCLUDE = os.path.join(os.path.dirname(HERE), "include")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return lz.load()


@pytest.mark.parametrize("name", ["lizard_rope_dims", "lizard_decay_dims"])
def test_dims_struct_layout(tmp_path, name):
    cls = getattr(lz, name)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "lizard.h"\n'
                   f'int main(void) {{ printf("%zu", sizeof({name}));\n' +
                   "".join(f'printf(" %zu", offsetof({name}, {n}));\n' for n, _ in cls._fields_) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", INCLUDE, "-o", str(exe), str(src)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, n).offset for n, _ in cls._fields_]


@pytest.fixture(scope="module")
def codes(lib):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, os.path.join(HERE, "_abi_heads.py")], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_good_calls_pass_every_check(codes):
    """With no device visible the device query is what stops them."""
    good = {k for k in codes if k.endswith("_ok")}
    assert {k: codes[k] for k in good} == {k: lz.LIZARD_ERR_CUDA for k in good} and len(good) == 11


def test_refusals(codes):
    bad = {k: v for k, v in codes.items() if not k.endswith("_ok")}
    for k, v in bad.items():
        want = (lz.LIZARD_ERR_WORKSPACE if k.endswith(("_small_ws", "_null_ws")) else
                lz.LIZARD_ERR_UNSUPPORTED if "_wide" in k else lz.LIZARD_ERR_INVALID_ARG)
        assert v == want, (k, v)
    assert len(bad) >= 90


def test_workspace_queries(lib):
    assert lz.lizard_qk_rope_bwd_workspace(lz.lizard_rope_dims(B=1, L=0, Hq=1, Hkv=1, d=1, axes=1)) == 256 + 8
    assert lz.lizard_qk_rope_bwd_workspace(lz.lizard_rope_dims(B=1, L=1, Hq=1, Hkv=1, d=1)) == 0  # no axis
    most = lz.lizard_qk_rope_bwd_workspace(lz.lizard_rope_dims(B=8, L=2048, Hq=32, Hkv=8, d=128, rot=128, axes=1, dtype=1))
    assert most == lz.lizard_qk_rope_bwd_workspace(lz.lizard_rope_dims(B=8, L=1 << 20, Hq=32, Hkv=8, d=128, rot=128, axes=1, dtype=1))
    many = lz.lizard_decay_dims(B=64, L=100, Hq=32, Hkv=32, dk=128, dv=128, scale=1.0, dtype=1)
    assert lz.lizard_decay_attn_fwd_workspace(many) == 256  # no segments
    few = lz.lizard_decay_dims(B=1, L=8192, Hq=4, Hkv=1, dk=128, dv=128, scale=1.0, dtype=1)
    f, b = lz.lizard_decay_attn_fwd_workspace(few), lz.lizard_decay_attn_bwd_workspace(few)
    assert f > 256 + 4 * 128 * 128 and b > f
    longer = lz.lizard_decay_dims(B=1, L=1 << 20, Hq=4, Hkv=1, dk=128, dv=128, scale=1.0, dtype=1)
    assert lz.lizard_decay_attn_fwd_workspace(longer) < 256 + 400 * 4 * 128 * 128  # does not grow with L
    assert lz.lizard_decay_attn_fwd_workspace(lz.lizard_decay_dims(B=1, L=5, Hq=3, Hkv=2, dk=8, dv=8, scale=1.0)) == 0
    assert lz.lizard_decay_attn_kernel(lz.lizard_decay_dims(B=1, L=5, Hq=3, Hkv=2, dk=8, dv=8, scale=1.0)) == -1
    assert lz.lizard_decay_attn_kernel(lz.lizard_decay_dims(B=1, L=5, Hq=2, Hkv=2, dk=33, dv=8, scale=1.0, dtype=1)) == 0


def test_binding_refuses_what_is_not_on_the_device():
    q = torch.zeros(1, 2, 2, 8)
    with pytest.raises(ValueError):
        lz.lizard_qk_rope_fwd(q, None, None)
    with pytest.raises(ValueError):
        lz.lizard_decay_attn_fwd(q, q, q, torch.zeros(2))
    with pytest.raises(ValueError):
        lz.lizard_decay_attn_step(q[:, 0], q[:, 0], q[:, 0], torch.zeros(2), torch.zeros(1, 2, 8, 8))
    with pytest.raises(ValueError):
        lz.lizard_decay_attn_fwd(q[0], q[0], q[0], torch.zeros(2))
