"""A stack of MoE blocks joined to their residual stream, as a program trains and serves it.

Each block normalises the residual r, runs the MoE layer on it, and adds the normalised, gated result back:
    u = rms(r) * w_pre;  y = moe(u);  r <- alpha r + beta gate * (rms(y) * w_post)
The norm that ends a block and the one that begins the next are one call (moe_block_norm_fwd), so between two MoE layers r
and y are read once and r and u written once.  Training keeps r, y and the layers' contexts and goes back the same way;
serving runs the few tokens of a decode step through moe_layer_decode.

    python examples/moe_block.py            # a forward, backward and decode step, with their times
"""
from __future__ import annotations

import os
import sys
import time

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from routing_grouped_expert_router_gb300 import binding as mb


class Stack:
    """`blocks` MoE blocks of one shape on the current device, random weights, fp32 residual stream."""

    def __init__(self, blocks, h, f, E, k, seed=0, eps=1e-5, alpha=1.0, beta=1.0):
        g = torch.Generator("cuda").manual_seed(seed)

        def normal(shape, std, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)

        self.h, self.f, self.E, self.k = h, f, E, k
        self.norm = dict(eps=eps, alpha=alpha, beta=beta)
        self.blocks = [dict(Wg=normal((h, E), h ** -0.5, torch.float32), W1=normal((E, h, f), h ** -0.5),
                            W3=normal((E, h, f), h ** -0.5), W2=normal((E, f, h), f ** -0.5),
                            w_pre=1 + normal((h,), 0.1, torch.float32), w_post=1 + normal((h,), 0.1, torch.float32),
                            gate=0.5 + normal((h,), 0.1, torch.float32)) for _ in range(blocks)]

    def _norm_dims(self, T):
        return mb.norm_dims(T, self.h, res_f32=True, gate=mb.GATE_CHANNEL, **self.norm)

    def _bytes(self, n):
        return torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")

    # ------------------------------------------------------------------ serving
    def decoder(self, T):
        """The buffers of a decode step for T sequences, kept from step to step."""
        d = mb.dims(T, self.h, self.f, self.E, self.k)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        return dict(d=d, nd=self._norm_dims(T), ws=self._bytes(mb.moe_workspace_bytes(d, mb.OP_LAYER_DECODE)),
                    u=torch.empty(T, self.h, **bf), y=torch.empty(T, self.h, **bf))

    def decode(self, buf, r):
        """One step: r [T, h] fp32 goes through every block, in place."""
        nd, u, y = buf["nd"], buf["u"], buf["y"]
        mb.moe_block_norm_fwd(nd, r, None, None, None, self.blocks[0]["w_pre"], None, u)
        for i, b in enumerate(self.blocks):
            mb.moe_layer_decode(buf["d"], u, b["Wg"], None, b["W1"], b["W3"], b["W2"], y, None, None, buf["ws"])
            last = i + 1 == len(self.blocks)
            mb.moe_block_norm_fwd(nd, r, y, b["w_post"], b["gate"], None if last else self.blocks[i + 1]["w_pre"], r,
                                  None if last else u)
        return r

    # ----------------------------------------------------------------- training
    def forward(self, r):
        """r [T, h] fp32 -> the residual after the last block, and what the backward needs."""
        T = r.shape[0]
        d, nd = mb.dims(T, self.h, self.f, self.E, self.k), self._norm_dims(T)
        ws = self._bytes(mb.moe_workspace_bytes(d, mb.OP_LAYER_FWD))
        u = torch.empty(T, self.h, dtype=torch.bfloat16, device="cuda")
        mb.moe_block_norm_fwd(nd, r, None, None, None, self.blocks[0]["w_pre"], None, u)
        kept = []
        for i, b in enumerate(self.blocks):
            saved, y = self._bytes(mb.moe_saved_bytes(d)), torch.empty_like(u)
            mb.moe_layer_fwd(d, u, b["Wg"], None, b["W1"], b["W3"], b["W2"], y, saved, ws)
            last = i + 1 == len(self.blocks)
            r_out, u_out = torch.empty_like(r), None if last else torch.empty_like(u)
            mb.moe_block_norm_fwd(nd, r, y, b["w_post"], b["gate"], None if last else self.blocks[i + 1]["w_pre"],
                                  r_out, u_out)
            kept.append(dict(r=r, u=u, y=y, saved=saved))
            r, u = r_out, u_out
        return r, (d, nd, kept, r)

    def backward(self, ctx, dr):
        """The gradient dr of the last residual -> (that of the first, one dict of weight gradients for each block)."""
        d, nd, kept, r_out = ctx
        ws, nws = self._bytes(mb.moe_workspace_bytes(d, mb.OP_LAYER_BWD)), self._bytes(mb.moe_norm_workspace_bytes(nd))
        grads = [{n: torch.empty(w.shape, dtype=torch.float32, device="cuda") for n, w in b.items()} for b in self.blocks]
        dr, du = dr.clone(), None
        for i in reversed(range(len(self.blocks))):
            b, g, c = self.blocks[i], grads[i], kept[i]
            last = i + 1 == len(self.blocks)
            dy, dx = torch.empty_like(c["y"]), torch.empty_like(c["u"])
            mb.moe_block_norm_bwd(nd, None if last else r_out, c["y"], b["w_post"], b["gate"],
                                  None if last else self.blocks[i + 1]["w_pre"], du, dr, dr, dy, g["w_post"], g["gate"],
                                  None if last else grads[i + 1]["w_pre"], nws)
            mb.moe_layer_bwd(d, c["u"], dy, b["Wg"], b["W1"], b["W3"], b["W2"], c["saved"], dx, g["Wg"], g["W1"], g["W3"],
                             g["W2"], ws)
            du, r_out = dx, c["r"]
        mb.moe_block_norm_bwd(nd, r_out, None, None, None, self.blocks[0]["w_pre"], du, dr, dr, None, None, None,
                              grads[0]["w_pre"], nws)
        return dr, grads


def _timed(name, fn, n=20):
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(n):
        fn()
    torch.cuda.synchronize()
    print(f"{name}: {(time.perf_counter() - t) / n * 1e6:.0f} us")


def main():
    s = Stack(blocks=2, h=2048, f=1408, E=64, k=6)
    for T in (1, 32):
        buf, r = s.decoder(T), torch.randn(T, s.h, device="cuda")
        _timed(f"decode step, 2 blocks, {T} tokens", lambda: s.decode(buf, r.clone()))
    r = torch.randn(8192, s.h, device="cuda")
    _, ctx = s.forward(r)
    _timed("forward, 2 blocks, 8192 tokens", lambda: s.forward(r))
    _timed("backward, 2 blocks, 8192 tokens", lambda: s.backward(ctx, r))


if __name__ == "__main__":
    main()
