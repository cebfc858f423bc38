"""Argument checks of the rotation's and the decay attention's entry points that need non-null pointers, run
in a child process with no visible CUDA device so that no call can reach a launch.  The pointers are host
buffers.  Prints one JSON object of status codes; tests/test_abi_heads.py runs it."""
import ctypes
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from gated_linear_sliding_gb300 import lizard as lz  # noqa: E402


def rope(section=None, **kw):
    d = dict(B=2, L=10, Hq=4, Hkv=2, d=32, rot=32, axes=1, eps=1e-6, dtype=1, norm=1)
    d.update(kw)
    r = lz.lizard_rope_dims(**d)
    for i, n in enumerate(section or []):
        r.section[i] = n
    return r


def decay(**kw):
    d = dict(B=2, L=10, Hq=4, Hkv=2, dk=32, dv=64, scale=0.5, dtype=1)
    d.update(kw)
    return lz.lizard_decay_dims(**d)


def main():
    assert os.environ.get("CUDA_VISIBLE_DEVICES") == "", "must run without a visible device"
    lib = lz.load()
    buf = ctypes.create_string_buffer(1 << 16)
    base = (ctypes.addressof(buf) + 63) & ~63
    ok, mis = base, base + 4
    big = 1 << 40
    out = {}

    def call(name, fn, dims, args, *tail):
        out[name] = fn(ctypes.byref(dims) if dims is not None else None, *args, *tail)

    def without(args, *at):
        return [None if i in at else p for i, p in enumerate(args)]

    rf = [ok] * 8  # q k w_q w_k freqs positions q_out k_out
    fwd = lib.lizard_qk_rope_fwd
    call("rope_ok", fwd, rope(), rf, None)
    call("rope_plain_ok", fwd, rope(norm=0, Hkv=0, rot=0), [ok, None, None, None, None, None, ok, None], None)
    call("rope_axes_ok", fwd, rope([4, 4, 8], axes=3), rf, None)
    call("rope_L0_ok", fwd, rope(L=0), [None] * 2 + [ok] * 3 + [None] * 3, None)
    call("rope_null_dims", fwd, None, rf, None)
    for i, n in ((0, "q"), (1, "k"), (4, "freqs"), (6, "q_out"), (7, "k_out")):
        call(f"rope_null_{n}", fwd, rope(), without(rf, i), None)
    for i in range(8):
        call(f"rope_mis_{i}", fwd, rope(), [mis + (1 if j == 5 else 0) if j == i else p for j, p in enumerate(rf)], None)
    for name, kw in dict(Hq=dict(Hq=0), Hkv=dict(Hkv=-1), d=dict(d=0), rot=dict(rot=34), odd=dict(rot=31), neg=dict(rot=-2),
                         axes0=dict(axes=0), axes5=dict(axes=5), sum=dict(axes=2, section=[8, 9]), minus=dict(axes=2, section=[17, -1]),
                         eps=dict(eps=-1.0), nan=dict(eps=float("nan")), dtype=dict(dtype=2), ldq=dict(ldq=127), ldko=dict(ldko=1),
                         B=dict(B=0), L=dict(L=1 << 31), over=dict(B=1 << 40, Hq=1 << 30)).items():
        call(f"rope_bad_{name}", fwd, rope(**kw), rf, None)
    call("rope_weight_no_norm", fwd, rope(norm=0), rf, None)
    call("rope_w_k_no_k", fwd, rope(Hkv=0), rf, None)
    call("rope_axes_no_positions", fwd, rope([8, 8], axes=2), without(rf, 5), None)
    call("rope_wide", fwd, rope(d=513, rot=512), rf, None)
    rb = [ok] * 12  # q k w_q w_k freqs positions dq_out dk_out dq dk dw_q dw_k
    bw = lib.lizard_qk_rope_bwd
    need = lz.lizard_qk_rope_bwd_workspace(rope())
    call("ropeb_ok", bw, rope(), rb, ok, need, None)
    call("ropeb_plain_ok", bw, rope(norm=0), without(rb, 0, 1, 2, 3, 10, 11), ok, need, None)
    call("ropeb_small_ws", bw, rope(), rb, ok, need - 1, None)
    call("ropeb_null_ws", bw, rope(), rb, None, big, None)
    for i, n in ((0, "q"), (1, "k"), (4, "freqs"), (6, "dq_out"), (7, "dk_out"), (8, "dq"), (9, "dk"), (10, "dw_q"), (3, "w_k")):
        call(f"ropeb_null_{n}", bw, rope(), without(rb, i), ok, need, None)

    df = [ok] * 8  # q k v log_decay s0 cu o s_out
    fwd = lib.lizard_decay_attn_fwd
    need = lz.lizard_decay_attn_fwd_workspace(decay())
    call("decay_ok", fwd, decay(), df, ok, need, None)
    call("decay_optional_ok", fwd, decay(), without(df, 4, 5, 7), ok, need, None)
    call("decay_L0_ok", fwd, decay(L=0), [None] * 3 + [ok, ok, None, None, ok], ok, need, None)
    call("decay_small_ws", fwd, decay(), df, ok, need - 1, None)
    call("decay_null_ws", fwd, decay(), df, None, big, None)
    for i, n in ((0, "q"), (1, "k"), (2, "v"), (3, "log_decay"), (6, "o")):
        call(f"decay_null_{n}", fwd, decay(), without(df, i), ok, need, None)
    call("decay_packed_no_cu", fwd, decay(B=1, nseq=2), without(df, 5), ok, big, None)
    for i in range(8):
        call(f"decay_mis_{i}", fwd, decay(B=1, nseq=2), [mis + (1 if j == 5 else 0) if j == i else p for j, p in enumerate(df)], ok, big, None)
    call("decay_mis_ws", fwd, decay(), df, mis, big, None)
    for name, kw in dict(heads=dict(Hq=3), Hkv=dict(Hkv=0), dk=dict(dk=0), dv=dict(dv=-1), B=dict(B=0), L=dict(L=-1), nseq=dict(nseq=2),
                         scale=dict(scale=float("inf")), dtype=dict(dtype=7), ldq=dict(ldq=127), ldo=dict(ldo=255), lddv=dict(lddv=1),
                         over=dict(Hq=1 << 40, Hkv=1 << 40)).items():
        call(f"decay_bad_{name}", fwd, decay(**kw), df, ok, big, None)
    call("decay_wide_k", fwd, decay(dk=193), df, ok, big, None)
    call("decay_wide_v", fwd, decay(dv=193), df, ok, big, None)
    db = [ok] * 12  # q k v log_decay s0 cu do ds_out dq dk dv ds0
    bw = lib.lizard_decay_attn_bwd
    need = lz.lizard_decay_attn_bwd_workspace(decay())
    call("decayb_ok", bw, decay(), db, ok, need, None)
    call("decayb_small_ws", bw, decay(), db, ok, need - 1, None)
    for i, n in ((0, "q"), (1, "k"), (2, "v"), (3, "log_decay"), (6, "do"), (8, "dq"), (9, "dk"), (10, "dv")):
        call(f"decayb_null_{n}", bw, decay(), without(db, i), ok, need, None)
    call("decayb_wide", bw, decay(dk=200), db, ok, big, None)
    ds = [ok] * 5  # q k v log_decay state
    st = lib.lizard_decay_attn_step
    call("decays_ok", st, decay(), ds, 2, None, ok, None, 0, None)
    call("decays_few_slots", st, decay(), ds, 1, None, ok, None, 0, None)
    call("decays_neg_slots", st, decay(), ds, -1, ok, ok, None, 0, None)
    for i, n in ((0, "q"), (1, "k"), (2, "v"), (3, "log_decay"), (4, "state")):
        call(f"decays_null_{n}", st, decay(), without(ds, i), 2, None, ok, None, 0, None)
    call("decays_null_o", st, decay(), ds, 2, None, None, None, 0, None)
    call("decays_mis_slots", st, decay(), ds, 2, mis, ok, None, 0, None)
    call("decays_small_ws", st, decay(), ds, 2, None, ok, ok, 255, None)
    call("decays_wide", st, decay(dv=193), ds, 2, None, ok, None, 0, None)
    print(json.dumps(out))


if __name__ == "__main__":
    main()
