"""Argument checks of the selective block's entry points that need non-null pointers, run in a
child process with no visible CUDA device so that no call can reach a launch.  The pointers are
host buffers.  Prints one JSON object of status codes; tests/test_abi_selective.py runs it."""
import ctypes
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from gated_linear_sliding_gb300 import lizard as lz  # noqa: E402


def conv(**kw):
    d = dict(B=2, L=10, C=16, K=4, nseq=0, ldx=0, ldy=0, lddx=0, dtype=1, act=1)
    d.update(kw)
    return lz.lizard_conv_dims(**d)


def scan(**kw):
    d = dict(B=2, L=10, C=16, N=16, G=2, dtype=1, softplus=1)
    d.update(kw)
    return lz.lizard_scan_dims(**d)


def norm(**kw):
    d = dict(T=4, D=32, groups=2, eps_post=1e-5, eps_pre=1e-5, dtype=1, res_dtype=1, act=1)
    d.update(kw)
    return lz.lizard_norm_dims(**d)


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

    # x, w, bias, state_in, cu, y, state_out
    cf = [ok, ok, ok, ok, ok, ok, ok]
    fwd = lib.lizard_conv_fwd
    call("conv_ok", fwd, conv(), cf, ok, 256, None)
    call("conv_no_ws", fwd, conv(), cf, None, 0, None)
    call("conv_small_ws", fwd, conv(), cf, ok, 255, None)
    call("conv_mis_ws", fwd, conv(), cf, mis, 256, None)
    call("conv_null_dims", fwd, None, cf, None, 0, None)
    for i, n in ((0, "x"), (1, "w"), (5, "y")):
        call(f"conv_null_{n}", fwd, conv(), [None if j == i else p for j, p in enumerate(cf)], None, 0, None)
    for i in range(7):
        call(f"conv_mis_{i}", fwd, conv(nseq=2, B=1), [mis + (1 if i == 4 else 0) if j == i else p for j, p in enumerate(cf)],
             None, 0, None)
    for name, kw in dict(K0=dict(K=0), K9=dict(K=9), B0=dict(B=0), Lneg=dict(L=-1), C0=dict(C=0), act=dict(act=2),
                         dtype=dict(dtype=2), ldx=dict(ldx=15), ldy=dict(ldy=-1), nseq=dict(nseq=2),
                         nseqneg=dict(nseq=-1, B=1), huge=dict(L=1 << 31), over=dict(B=1 << 40, C=1 << 40)).items():
        call(f"conv_bad_{name}", fwd, conv(**kw), cf, None, 0, None)
    call("conv_packed_no_cu", fwd, conv(B=1, nseq=2), cf[:4] + [None] + cf[5:], None, 0, None)
    call("conv_L0_null", fwd, conv(L=0), [None, ok, ok, ok, None, None, ok], None, 0, None)
    bw = lib.lizard_conv_bwd
    cb = [ok] * 11  # x w bias state_in cu dy dstate_out dx dw dbias dstate_in
    need = lz.lizard_conv_bwd_workspace(conv())
    call("convb_ok", bw, conv(), cb, ok, need, None)
    call("convb_small_ws", bw, conv(), cb, ok, need - 1, None)
    call("convb_null_ws", bw, conv(), cb, None, big, None)
    call("convb_bias_pair", bw, conv(), cb[:9] + [None, ok], ok, need, None)
    call("convb_null_dw", bw, conv(), cb[:8] + [None] + cb[9:], ok, need, None)
    st = lib.lizard_conv_step
    cs = [ok, ok, ok, ok]  # x w bias state
    call("convs_ok", st, conv(), cs, 3, ok, ok, None, 0, None)
    call("convs_few_slots", st, conv(), cs, 1, None, ok, None, 0, None)
    call("convs_neg_slots", st, conv(), cs, -1, ok, ok, None, 0, None)
    call("convs_null_state", st, conv(), [ok, ok, ok, None], 3, ok, ok, None, 0, None)
    call("convs_K1_no_state", st, conv(K=1), [ok, ok, ok, None], 3, ok, ok, None, 0, None)
    call("convs_mis_slots", st, conv(), cs, 3, mis, ok, None, 0, None)

    sf = [ok] * 13  # x dt A Bm Cm D z dt_bias h0 cu y h_out states
    fwd = lib.lizard_scan_fwd
    need = lz.lizard_scan_fwd_workspace(scan())
    call("scan_ok", fwd, scan(), sf, ok, need, None)
    call("scan_optional_null", fwd, scan(), [ok] * 5 + [None] * 5 + [ok, None, None], ok, need, None)
    call("scan_small_ws", fwd, scan(), sf, ok, need - 1, None)
    call("scan_null_ws", fwd, scan(), sf, None, big, None)
    for i, n in ((0, "x"), (1, "dt"), (2, "A"), (3, "Bm"), (4, "Cm"), (10, "y")):
        call(f"scan_null_{n}", fwd, scan(), [None if j == i else p for j, p in enumerate(sf)], ok, need, None)
    for i in range(13):
        call(f"scan_mis_{i}", fwd, scan(B=1, nseq=2), [mis + (1 if i == 9 else 0) if j == i else p for j, p in enumerate(sf)],
             ok, big, None)
    for name, kw in dict(N0=dict(N=0), G0=dict(G=0), G3=dict(G=3), G32=dict(G=32), ldb=dict(ldb=31), ldc=dict(ldc=1),
                         lddt=dict(lddt=8), B0=dict(B=0), dtype=dict(dtype=7), nseq=dict(nseq=3)).items():
        call(f"scan_bad_{name}", fwd, scan(**kw), sf, ok, big, None)
    call("scan_N65", fwd, scan(N=65), sf, ok, big, None)
    sb = [ok] * 22  # x dt A Bm Cm D z dt_bias h0 cu states dy dh_out dx ddt dz dBm dCm dA dD ddt_bias dh0
    bw = lib.lizard_scan_bwd
    need = lz.lizard_scan_bwd_workspace(scan())
    call("scanb_ok", bw, scan(), sb, ok, need, None)
    call("scanb_small_ws", bw, scan(), sb, ok, need - 1, None)
    for i, n in ((10, "states"), (11, "dy"), (13, "dx"), (14, "ddt"), (16, "dBm"), (17, "dCm"), (18, "dA")):
        call(f"scanb_null_{n}", bw, scan(), [None if j == i else p for j, p in enumerate(sb)], ok, need, None)
    for i, n in ((15, "dz"), (19, "dD"), (20, "ddt_bias")):
        call(f"scanb_pair_{n}", bw, scan(), [None if j == i else p for j, p in enumerate(sb)], ok, need, None)
    st = lib.lizard_scan_step
    ss = [ok] * 9
    call("scans_ok", st, scan(), ss, 2, None, ok, None, 0, None)
    call("scans_few_slots", st, scan(), ss, 1, None, ok, None, 0, None)
    call("scans_null_state", st, scan(), ss[:8] + [None], 2, None, ok, None, 0, None)
    call("scans_N65", st, scan(N=65), ss, 2, None, ok, None, 0, None)

    nf = [ok] * 8  # o gate r w_post scale w_pre r_out n_out
    fwd = lib.lizard_block_norm_fwd
    call("norm_ok", fwd, norm(), nf, None)
    call("norm_no_outputs", fwd, norm(), nf[:6] + [None, None], None)
    call("norm_n_without_w", fwd, norm(), nf[:5] + [None, ok, ok], None)
    call("norm_w_without_n", fwd, norm(), nf[:7] + [None], None)
    call("norm_null_o", fwd, norm(), [None] + nf[1:], None)
    call("norm_gate_no_act", fwd, norm(act=0), nf, None)
    for i in range(8):
        call(f"norm_mis_{i}", fwd, norm(), [mis if j == i else p for j, p in enumerate(nf)], None)
    for name, kw in dict(groups=dict(groups=3), groups0=dict(groups=0), D0=dict(D=0), T=dict(T=-1), eps=dict(eps_post=-1.0),
                         nan=dict(eps_pre=float("nan")), res=dict(dtype=0, res_dtype=1), ldo=dict(ldo=31), act=dict(act=3)).items():
        call(f"norm_bad_{name}", fwd, norm(**kw), nf, None)
    call("norm_wide", fwd, norm(D=16385, groups=1), nf, None)
    nb = [ok] * 14  # o gate r w_post scale w_pre dr_out dn_out do dgate dr dw_post dscale dw_pre
    bw = lib.lizard_block_norm_bwd
    need = lz.lizard_block_norm_bwd_workspace(norm())
    call("normb_ok", bw, norm(), nb, ok, need, None)
    call("normb_small_ws", bw, norm(), nb, ok, need - 1, None)
    for i, n in ((7, "dn_out"), (8, "do"), (9, "dgate"), (11, "dw_post"), (12, "dscale"), (13, "dw_pre")):
        call(f"normb_null_{n}", bw, norm(), [None if j == i else p for j, p in enumerate(nb)], ok, need, None)
    call("normb_no_upstream", bw, norm(), nb[:5] + [None, None, None] + nb[8:13] + [None], ok, need, None)
    print(json.dumps(out))


if __name__ == "__main__":
    main()
