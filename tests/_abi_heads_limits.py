"""Sizes beyond what the rotation's kernels are compiled for, and far beyond 32 bits, in a child process with no
visible CUDA device so that no call can reach a launch.  The pointers are host buffers.  Prints one JSON object
of status codes; tests/test_abi_heads_limits.py runs it."""
import ctypes
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from gated_linear_sliding_gb300 import lizard as lz  # noqa: E402

WIDE = {"513": 513, "2^31": 1 << 31, "2^32": 1 << 32, "2^32+128": (1 << 32) + 128, "2^39": 1 << 39}


def rope(d, rot):
    return lz.lizard_rope_dims(B=1, L=2, Hq=2, Hkv=1, d=d, rot=rot, axes=1, eps=1e-6, dtype=1, norm=1)


def main():
    assert os.environ.get("CUDA_VISIBLE_DEVICES") == "", "must run without a visible device"
    lib = lz.load()
    buf = ctypes.create_string_buffer(1 << 16)
    ok = (ctypes.addressof(buf) + 63) & ~63
    out = {}
    for name, d in WIDE.items():
        for rot in (32, d - d % 2):
            dims = ctypes.byref(rope(d, rot))
            out[f"fwd {name} {rot}"] = lib.lizard_qk_rope_fwd(dims, *[ok] * 8, None)
            out[f"bwd {name} {rot}"] = lib.lizard_qk_rope_bwd(dims, *[ok] * 12, ok, 1 << 40, None)
            out[f"workspace {name} {rot}"] = lib.lizard_qk_rope_bwd_workspace(dims)
    print(json.dumps(out))


if __name__ == "__main__":
    main()
