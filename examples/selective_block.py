"""A selective state space block built from the library's calls: for prompts, for training and
for single tokens.

    u        the block's normalised input [B, L, dm]
    p        u W_in^T, whose columns are x, z [C each], dt [C], Bm, Cm [G N each]
    x        the short causal convolution with SiLU of p's x columns
    y        the selective scan of x with p's dt, Bm, Cm
    o        (the norm over heads of y silu(z)) W_out^T
    r, u     r + scale o, and the next block's normalised input

The three library calls (convolution, scan, block norm) read their inputs as column ranges of p and
write the columns of its gradient; the projections are plain matrix products.

    python examples/selective_block.py      # on a GB300, after the library is built
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from gated_linear_sliding_gb300 import lizard as lz  # noqa: E402


class SelectiveBlock:
    """Weights of one block (random), and its three ways of running."""

    def __init__(self, dm=512, C=1024, N=16, G=2, K=4, heads=8, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device).manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(shape, generator=g, device=device) * std

        self.C, self.N, self.G, self.K, self.heads, self.dtype = C, N, G, K, heads, dtype
        self.width = 3 * C + 2 * G * N
        self.W_in = normal(self.width, dm, std=dm ** -0.5).to(dtype)
        self.W_out = normal(dm, C, std=C ** -0.5).to(dtype)
        self.p = dict(w=normal(C, K, std=K ** -0.5), bias=torch.zeros(C, device=device),
                      A=-torch.arange(1, N + 1, device=device).float().repeat(C, 1), D=torch.ones(C, device=device),
                      dt_bias=normal(C, std=0.5) - 4.0, w_post=torch.ones(C, device=device),
                      scale=torch.full((dm,), 0.5, device=device), w_pre=torch.ones(dm, device=device))

    def columns(self, p):
        """x, z, dt, Bm, Cm as column ranges of p [..., width]."""
        C, GN = self.C, self.G * self.N
        x, z, dt, Bm, Cm = p.split([C, C, C, GN, GN], -1)
        return x, z, dt, Bm.unflatten(-1, (self.G, self.N)), Cm.unflatten(-1, (self.G, self.N))

    def _scan_args(self):
        return dict(D=self.p["D"], dt_bias=self.p["dt_bias"])

    def _out(self, y, z, r):
        """From the scan's output to the residual stream and the next block's input."""
        P, rows = self.p, y.numel() // self.C
        h, _ = lz.lizard_block_norm_fwd(y.reshape(rows, self.C), gate=z, w_post=P["w_post"], groups=self.heads,
                                        gate_first=True)
        o = h @ self.W_out.t()
        r, u = lz.lizard_block_norm_fwd(o, r=r, scale=P["scale"], w_pre=P["w_pre"])
        return h, o, r, u

    def prompt(self, u, r, cu_seqlens=None, conv_state=None, state=None):
        """u, r [B, L, dm] -> (r, u) [B, L, dm].  conv_state [sequences, K-1, C] and state
        [sequences, C, N] continue earlier calls and are moved on in place."""
        B, L, dm = u.shape
        x, z, dt, Bm, Cm = self.columns(u @ self.W_in.t())
        x = lz.lizard_conv_fwd(x, self.p["w"], self.p["bias"], act=lz.LIZARD_ACT_SILU, state_in=conv_state,
                               state_out=conv_state, cu_seqlens=cu_seqlens)
        y = lz.lizard_scan_fwd(x, dt, self.p["A"], Bm, Cm, h0=state, h_out=state, cu_seqlens=cu_seqlens,
                               **self._scan_args())
        _, _, r, u = self._out(y, z.flatten(0, 1), r.reshape(B * L, dm))
        return r.view(B, L, dm), u.view(B, L, dm)

    def step(self, u, r, conv_state, state, slots=None):
        """One token for each sequence: u, r [B, dm]; the states' slots are moved on in place."""
        x, z, dt, Bm, Cm = self.columns(u @ self.W_in.t())
        x = lz.lizard_conv_step(x, self.p["w"], self.p["bias"], conv_state, slots=slots, act=lz.LIZARD_ACT_SILU)
        y = lz.lizard_scan_step(x, dt, self.p["A"], Bm, Cm, state, slots=slots, **self._scan_args())
        _, _, r, u = self._out(y, z, r)
        return r, u

    def train(self, u, r, dr, du):
        """Forward and backward: outputs (r, u) and the gradients of u, r, the projections and every
        parameter against dr, du, the gradients of the outputs."""
        P, (B, L, dm) = self.p, u.shape
        rows = B * L
        p = u @ self.W_in.t()
        x0, z, dt, Bm, Cm = self.columns(p)
        x = lz.lizard_conv_fwd(x0, P["w"], P["bias"], act=lz.LIZARD_ACT_SILU)
        y, states = lz.lizard_scan_fwd(x, dt, P["A"], Bm, Cm, save_states=True, **self._scan_args())
        z2, y2, r2 = z.flatten(0, 1), y.view(rows, self.C), r.reshape(rows, dm)
        h, o, r_out, u_out = self._out(y, z2, r2)

        g2 = lz.lizard_block_norm_bwd(o, r=r2, scale=P["scale"], w_pre=P["w_pre"], dr_out=dr.reshape(rows, dm),
                                      dn_out=du.reshape(rows, dm))
        dh = g2["do"] @ self.W_out
        g1 = lz.lizard_block_norm_bwd(y2, gate=z2, w_post=P["w_post"], groups=self.heads, gate_first=True, dr_out=dh)
        dp = torch.empty_like(p)
        dx0, dz, ddt, dBm, dCm = self.columns(dp)
        gs = lz.lizard_scan_bwd(x, dt, P["A"], Bm, Cm, g1["do"].view(B, L, self.C), states, ddt=ddt, dBm=dBm, dCm=dCm,
                                **self._scan_args())
        gc = lz.lizard_conv_bwd(x0, P["w"], P["bias"], gs["dx"], act=lz.LIZARD_ACT_SILU, dx=dx0)
        dz.copy_(g1["dgate"].view(B, L, self.C))
        flat = dp.view(rows, self.width)
        grads = dict(u=(flat @ self.W_in).view(B, L, dm), r=g2["dr"].view(B, L, dm), W_in=flat.t() @ u.reshape(rows, dm),
                     W_out=g2["do"].t() @ h, w=gc["dw"], bias=gc["dbias"], A=gs["dA"], D=gs["dD"],
                     dt_bias=gs["ddt_bias"], w_post=g1["dw_post"], scale=g2["dscale"], w_pre=g2["dw_pre"])
        return r_out.view(B, L, dm), u_out.view(B, L, dm), grads


def main():
    blk = SelectiveBlock()
    g = torch.Generator("cuda").manual_seed(1)
    u, r = (torch.randn(2, 300, 512, generator=g, device="cuda").to(blk.dtype) for _ in range(2))
    # a prompt of 290 tokens, then ten single tokens, against the prompt of 300
    whole, _ = blk.prompt(u, r)
    conv = torch.zeros(2, blk.K - 1, blk.C, dtype=blk.dtype, device="cuda")
    state = torch.zeros(2, blk.C, blk.N, device="cuda")
    blk.prompt(u[:, :290].contiguous(), r[:, :290].contiguous(), conv_state=conv, state=state)
    steps = torch.stack([blk.step(u[:, t], r[:, t].contiguous(), conv, state)[0] for t in range(290, 300)], 1)
    diff = (steps.float() - whole[:, 290:].float()).abs().max().item()
    print(f"ten decoded tokens against the prompt: largest difference {diff:.3g} (bf16 step at 4: 0.031)")
    *_, grads = blk.train(u, r, torch.ones_like(r), torch.zeros_like(u))
    print("gradients:", ", ".join(f"{k} {v.float().norm().item():.3g}" for k, v in grads.items()))


if __name__ == "__main__":
    main()
