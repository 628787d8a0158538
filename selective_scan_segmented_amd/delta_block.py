"""A token mixer of the gated delta rule and the group norm: forward, backward and token by token.

The block stands beside the mixer block around the scan (block.py), on the same
channel-last tokens X [B, L, C]:

    q, k, v = X W_qkv                         one projection, read in place as its slices
    g       = A softplus(X W_a + bias)        log decay per head, A < 0
    beta    = sigmoid(X W_b)                  gate per head
    o, S    = gated delta rule(q, k, v, g, beta)        sfm_gated_delta_fwd, unit queries and keys
    y       = silu(group norm(o))             sfm_group_norm_fwd, every token by itself, a group a head
    out     = y W_out

The projections and the gates' elementwise functions are PyTorch; weights are random (seeded).

    python -m selective_scan_segmented_amd.delta_block     # times one block on the GPU
"""
from __future__ import annotations

import dataclasses
import math


@dataclasses.dataclass(frozen=True)
class DeltaSizes:
    C: int            # model width
    H: int            # value heads
    Hk: int           # query and key heads; H is a multiple
    dk: int
    dv: int

    @property
    def qkv(self) -> int:
        return 2 * self.Hk * self.dk + self.H * self.dv


class DeltaBlock:
    """Random weights of the block on `device`, and its passes.  dtype: float32 or bfloat16 (io)."""

    def __init__(self, sizes: DeltaSizes, dtype=None, device="cuda", seed: int = 0):
        import torch
        self.z = z = sizes
        self.dtype = dtype = torch.bfloat16 if dtype is None else dtype
        gen = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen)
        w = lambda rows, cols: (rnd(rows, cols) / math.sqrt(rows)).to(device, dtype)
        self.W_qkv, self.W_a, self.W_b, self.W_out = w(z.C, z.qkv), w(z.C, z.H), w(z.C, z.H), w(z.H * z.dv, z.C)
        # decay rates 1 to 16, first steps 1e-3 to 1e-1 (inverse softplus)
        self.A = -torch.exp(torch.rand(z.H, generator=gen) * math.log(16.0)).to(device)
        dt = torch.exp(math.log(1e-3) + torch.rand(z.H, generator=gen) * math.log(100.0))
        self.bias = torch.log(torch.expm1(dt)).to(device)
        self.norm_w, self.norm_b = (1 + 0.1 * rnd(z.H * z.dv)).to(device), (0.1 * rnd(z.H * z.dv)).to(device)

    def _heads(self, X):
        """q, k, v as slices of one projection, and the raw gates."""
        import torch
        z = self.z
        p = torch.matmul(X, self.W_qkv)
        nk = z.Hk * z.dk
        q, k, v = p[..., :nk].unflatten(-1, (z.Hk, z.dk)), p[..., nk:2 * nk].unflatten(-1, (z.Hk, z.dk)), \
            p[..., 2 * nk:].unflatten(-1, (z.H, z.dv))
        # the gates in float32: a few columns, and what they are rounded to decides over whole states
        x = X.float()
        raw = torch.matmul(x, self.W_a.float()) + self.bias
        return q, k, v, (self.A * torch.nn.functional.softplus(raw)).to(self.dtype), \
            torch.sigmoid(torch.matmul(x, self.W_b.float())).to(self.dtype), raw

    def _norm(self, o):
        """Every token's heads normed by themselves: [tokens, 1, H dv] with a group a head."""
        import selective_scan_segmented_amd as sfm
        z = self.z
        return sfm.sfm_group_norm_fwd(o.reshape(-1, 1, z.H * z.dv), z.H, self.norm_w, self.norm_b, act="silu")

    def forward(self, X, state=None, return_state=False, keep=False):
        """X [B, L, C] -> out [B, L, C], and the heads' states if asked for.  keep: what backward() takes."""
        import torch

        import selective_scan_segmented_amd as sfm
        q, k, v, g, beta, raw = self._heads(X)
        r = sfm.sfm_gated_delta_fwd(q, k, v, g, beta, h0=state, l2norm=True, return_state=return_state)
        o, S = r if return_state else (r, None)
        y, mean, rstd = self._norm(o)
        y = y.view(X.shape[:2] + (-1,))
        out = torch.matmul(y, self.W_out)
        if keep:
            self.kept = (X, q, k, v, g, beta, raw, state, o, y, mean, rstd)
        return (out, S) if return_state else out

    def step(self, x, state, slots=None):
        """One token of each request: x [R, C]; state [pool, H, dk, dv] float32, updated in place."""
        import torch

        import selective_scan_segmented_amd as sfm
        q, k, v, g, beta, _ = self._heads(x)
        o = sfm.sfm_gated_delta_step(q, k, v, g, beta, state, slots=slots, l2norm=True)
        return torch.matmul(self._norm(o)[0].view(x.shape[0], -1), self.W_out)

    def backward(self, dout, dstate=None):
        """Gradients of the last forward(keep=True) for dout [B, L, C]: a dict of dX, dW_qkv, dW_a, dW_b, dW_out,
        dA, dbias, dnorm_w, dnorm_b (and dstate0 if it had a state)."""
        import torch

        import selective_scan_segmented_amd as sfm
        z = self.z
        X, q, k, v, g, beta, raw, state, o, y, mean, rstd = self.kept
        flat = lambda t: t.reshape(-1, t.shape[-1])
        grads = {"dW_out": flat(y).t() @ flat(dout)}
        dy = torch.matmul(dout, self.W_out.t())
        n = sfm.sfm_group_norm_bwd(dy.reshape(-1, 1, z.H * z.dv), o.reshape(-1, 1, z.H * z.dv), mean, rstd, self.norm_w,
                                   self.norm_b, act="silu")
        grads.update(dnorm_w=n["dw"], dnorm_b=n["db"])
        d = sfm.sfm_gated_delta_bwd(q, k, v, g, beta, n["dx"].view(o.shape), h0=state, dstate=dstate, l2norm=True)
        if state is not None:
            grads["dstate0"] = d["dh0"]
        dp = torch.cat([d["dq"].flatten(-2), d["dk"].flatten(-2), d["dv"].flatten(-2)], -1)
        dg, sig = d["dg"].float(), torch.sigmoid(raw)
        draw = dg * self.A * sig
        b, x = beta.float(), flat(X).float()
        db = d["dbeta"].float() * b * (1 - b)
        grads.update(dA=(dg * torch.nn.functional.softplus(raw)).sum((0, 1)), dbias=draw.sum((0, 1)),
                     dW_qkv=flat(X).t() @ flat(dp), dW_a=(x.t() @ flat(draw)).to(self.dtype),
                     dW_b=(x.t() @ flat(db)).to(self.dtype))
        dx = torch.matmul(dp, self.W_qkv.t()).float()
        dx += torch.matmul(draw, self.W_a.float().t())
        dx += torch.matmul(db, self.W_b.float().t())
        grads["dX"] = dx.to(self.dtype)
        return grads


def main() -> None:
    import torch
    B, L = 256, 198
    blk = DeltaBlock(DeltaSizes(C=320, H=5, Hk=5, dk=64, dv=64))
    X = torch.randn(B, L, 320, device="cuda").to(blk.dtype)
    dout = torch.randn_like(X)
    S = torch.zeros(B, 5, 64, 64, device="cuda")

    def timed(name, f, n=20):
        for _ in range(3):
            f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            f()
        b.record()
        torch.cuda.synchronize()
        print(f"{name}: {a.elapsed_time(b) / n * 1e3:.1f} us", flush=True)

    timed(f"forward  [{B}, {L}, 320] bf16", lambda: blk.forward(X))
    blk.forward(X, keep=True)
    timed("backward", lambda: blk.backward(dout))
    timed(f"step     {B} requests", lambda: blk.step(X[:, 0].contiguous(), S))


if __name__ == "__main__":
    main()
