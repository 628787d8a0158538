"""A token mixer of the gated linear recurrence: forward, backward and token by token.

The block stands beside the mixer blocks around the scan (block.py) and the gated
delta rule (delta_block.py), on the same channel-last tokens X [B, L, C]; hybrid
models alternate them:

    x, r, i, z = X W_in                       one projection, x, r and i read in place as its slices
    h          = gated recurrence(x, r, i)    sfm_gated_recurrence_fwd, one state a channel
    out        = (h silu(z)) W_out

The projections and the output gate are PyTorch; weights are random (seeded).

    python -m selective_scan_segmented_amd.recurrent_block     # times one block on the GPU
"""
from __future__ import annotations

import math


class RecurrentBlock:
    """Random weights of the block on `device`, and its passes.  C: model width, D: channels of the recurrence, c: its
    rate.  dtype: float32 or bfloat16 (io)."""

    def __init__(self, C: int, D: int, c: float = 8.0, dtype=None, device="cuda", seed: int = 0):
        import torch
        self.C, self.D, self.c = C, D, c
        self.dtype = dtype = torch.bfloat16 if dtype is None else dtype
        gen = torch.Generator().manual_seed(seed)
        w = lambda rows, cols: (torch.randn(rows, cols, generator=gen) / math.sqrt(rows)).to(device, dtype)
        self.W_in, self.W_out = w(C, 4 * D), w(D, C)
        # softplus(lam) = -log of decays between 0.9 and 0.999
        self.lam = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(D, generator=gen)))).to(device)

    def _project(self, X):
        import torch
        return torch.split(torch.matmul(X, self.W_in), self.D, dim=-1)

    def _gate(self, h, z):
        import torch
        return (h.float() * torch.nn.functional.silu(z.float())).to(self.dtype)

    def forward(self, X, state=None, return_state=False, keep=False):
        """X [B, L, C] -> out [B, L, C], and the channels' states [B, D] if asked for.  keep: what backward() takes."""
        import torch

        import selective_scan_segmented_amd as sfm
        x, r, i, z = self._project(X)
        got = sfm.sfm_gated_recurrence_fwd(x, r, i, self.lam, c=self.c, h0=state, return_state=return_state)
        h, S = got if return_state else (got, None)
        y = self._gate(h, z)
        out = torch.matmul(y, self.W_out)
        if keep:
            self.kept = (X, x, r, i, z, h, y, state)
        return (out, S) if return_state else out

    def step(self, x, state, slots=None):
        """One token of each request: x [R, C]; state [pool, D] float32, updated in place."""
        import torch

        import selective_scan_segmented_amd as sfm
        x, r, i, z = self._project(x)
        h = sfm.sfm_gated_recurrence_step(x, r, i, self.lam, state, slots=slots, c=self.c)
        return torch.matmul(self._gate(h, z), self.W_out)

    def backward(self, dout, dstate=None):
        """Gradients of the last forward(keep=True) for dout [B, L, C]: a dict of dX, dW_in, dW_out, dlam (and dstate0
        if it had a state)."""
        import torch

        import selective_scan_segmented_amd as sfm
        X, x, r, i, z, h, y, state = self.kept
        flat = lambda t: t.reshape(-1, t.shape[-1])
        dy = torch.matmul(dout, self.W_out.t()).float()
        zf = z.float()
        s = torch.sigmoid(zf)
        dz = (dy * h.float() * s * (1 + zf * (1 - s))).to(self.dtype)
        d = sfm.sfm_gated_recurrence_bwd(x, r, i, self.lam, h, (dy * zf * s).to(self.dtype), c=self.c, h0=state, dstate=dstate)
        dp = torch.cat([d["dx"], d["dr"], d["di"], dz], -1)
        grads = {"dW_out": flat(y).t() @ flat(dout), "dW_in": flat(X).t() @ flat(dp), "dlam": d["dlam"],
                 "dX": torch.matmul(dp, self.W_in.t())}
        if state is not None:
            grads["dstate0"] = d["dh0"]
        return grads


def main() -> None:
    import torch
    B, L, C = 256, 198, 320
    blk = RecurrentBlock(C, C)
    X = torch.randn(B, L, C, device="cuda").to(blk.dtype)
    dout = torch.randn_like(X)
    S = torch.zeros(B, C, device="cuda")

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

    timed(f"forward  [{B}, {L}, {C}] bf16", lambda: blk.forward(X))
    blk.forward(X, keep=True)
    timed("backward", lambda: blk.backward(dout))
    timed(f"step     {B} requests", lambda: blk.step(X[:, 0].contiguous(), S))


if __name__ == "__main__":
    main()
