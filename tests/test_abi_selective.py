"""The selective block's C ABI and binding without a GPU: struct layouts, workspace queries and
every refusal that happens on the host."""
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


@pytest.mark.parametrize("name", ["lizard_conv_dims", "lizard_scan_dims", "lizard_norm_dims"])
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
    r = subprocess.run([sys.executable, os.path.join(HERE, "_abi_selective.py")], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_good_calls_pass_every_check(codes):
    """With no device visible the device query is what stops them."""
    good = ["conv_ok", "conv_no_ws", "conv_L0_null", "convb_ok", "convs_ok", "convs_K1_no_state", "scan_ok",
            "scan_optional_null", "scanb_ok", "scans_ok", "norm_ok", "normb_ok"]
    assert {k: codes[k] for k in good} == {k: lz.LIZARD_ERR_CUDA for k in good}


def test_refusals(codes):
    workspace = {k for k in codes if k.endswith(("_small_ws", "_null_ws"))}
    unsupported = {"scan_N65", "scans_N65", "norm_wide"}
    good = {k for k, v in codes.items() if v == lz.LIZARD_ERR_CUDA}
    for k, v in codes.items():
        if k in good:
            continue
        want = (lz.LIZARD_ERR_WORKSPACE if k in workspace else lz.LIZARD_ERR_UNSUPPORTED if k in unsupported
                else lz.LIZARD_ERR_INVALID_ARG)
        assert v == want, (k, v)
    assert len(codes) - len(good) >= 90 and len(good) == 12


def test_workspace_queries(lib):
    conv = lz.lizard_conv_dims(2, 100, 64, 4, 0, 0, 0, 0, 1, 1)
    assert lz.lizard_conv_bwd_workspace(conv) > 256
    conv.K = 9
    assert lz.lizard_conv_bwd_workspace(conv) == 0
    s = lz.lizard_scan_dims(B=1, L=100, C=64, N=16, G=1, dtype=1, softplus=1)
    assert lz.lizard_scan_states_bytes(s) == 7 * 64 * 16 * 4  # one state for every 16 tokens
    assert lz.lizard_scan_fwd_workspace(s) == 256               # a short prompt is one segment
    s.L = 1 << 16                                               # a long one with few channels is cut
    assert lz.lizard_scan_fwd_workspace(s) > 256
    s.L, s.C = 8192, 1 << 20                                    # and one with many is not
    assert lz.lizard_scan_fwd_workspace(s) == 256
    s.N = 65
    assert lz.lizard_scan_fwd_workspace(s) == lz.lizard_scan_states_bytes(s) == lz.lizard_scan_bwd_workspace(s) == 0
    n = lz.lizard_norm_dims(T=10 ** 6, D=4096, groups=1, dtype=1, res_dtype=1)
    w = lz.lizard_block_norm_bwd_workspace(n)
    n.T = 10 ** 7
    assert lz.lizard_block_norm_bwd_workspace(n) == w > 256  # the rows do not count once the GPU is full


def test_binding_refuses_before_the_library():
    """Shapes, types, devices and layouts are checked in Python; none of these tensors is on a GPU."""
    x = torch.zeros(2, 5, 8)
    w = torch.zeros(8, 4)
    for call in (lambda: lz.lizard_conv_fwd(x, w),
                 lambda: lz.lizard_conv_bwd(x, w, None, x),
                 lambda: lz.lizard_conv_step(x[:, 0], w, None, torch.zeros(2, 3, 8)),
                 lambda: lz.lizard_scan_fwd(x, x, torch.zeros(8, 4), torch.zeros(2, 5, 1, 4), torch.zeros(2, 5, 1, 4)),
                 lambda: lz.lizard_scan_step(x[:, 0], x[:, 0], torch.zeros(8, 4), torch.zeros(2, 1, 4),
                                             torch.zeros(2, 1, 4), torch.zeros(2, 8, 4)),
                 lambda: lz.lizard_block_norm_fwd(x[0]),
                 lambda: lz.lizard_block_norm_fwd(x),
                 lambda: lz.lizard_conv_fwd(x, w, cu_seqlens=[0, 10]),
                 lambda: lz.lizard_conv_fwd(x[:1], w, cu_seqlens=[0, 3, 2, 5]),
                 lambda: lz.lizard_conv_fwd(x[:1], w, cu_seqlens=[0, 4]),
                 lambda: lz.lizard_conv_fwd(x[:1], w, cu_seqlens=[1, 5])):
        with pytest.raises(ValueError):
            call()


def test_row_distance():
    """_ld on host tensors wrapped as CUDA ones: what counts as evenly spaced rows."""
    class Fake:
        is_cuda = True

        def __init__(self, t):
            self.t, self.shape, self.dtype = t, t.shape, t.dtype

        def is_contiguous(self):
            return self.t.is_contiguous()

        def stride(self):
            return self.t.stride()

    f = torch.float32
    wide = torch.zeros(2, 5, 40)
    assert lz._ld(Fake(torch.zeros(2, 5, 8)), "x", (2, 5, 8), f) == 0
    assert lz._ld(Fake(wide[..., 8:16]), "x", (2, 5, 8), f) == 40
    assert lz._ld(Fake(wide[..., 8:32].unflatten(-1, (3, 8))), "x", (2, 5, 3, 8), f) == 40
    assert lz._ld(Fake(wide[:, 2, 8:16]), "x", (2, 8), f, 1) == 200
    assert lz._ld(Fake(wide[:, :1, 8:16]), "x", (2, 1, 8), f) == 200
    for bad, shape, lead in ((wide[:, :3, :8], (2, 3, 8), 2), (wide[..., ::2], (2, 5, 20), 2),
                             (wide[..., :1].expand(2, 5, 8), (2, 5, 8), 2), (wide.transpose(1, 2), (2, 40, 5), 2),
                             (torch.zeros(1, 8).expand(4, 8), (4, 8), 1)):
        with pytest.raises(ValueError):
            lz._ld(Fake(bad), "x", shape, f, lead)
    with pytest.raises(ValueError):
        lz._ld(Fake(wide), "x", (2, 5, 41), f)
    with pytest.raises(ValueError):
        lz._ld(Fake(wide), "x", (2, 5, 40), torch.bfloat16)
