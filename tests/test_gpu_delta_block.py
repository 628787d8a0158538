"""The mixer block of the gated delta rule and the group norm: its passes together against float64."""
import numpy as np
import pytest

import delta_reference as ref
from helpers import from_dev

pytestmark = pytest.mark.gpu


def reference(blk, X, state, dout, io):
    """The block in float64 from its own weights, forward and backward (the latter by chaining the references); what
    the block stores between its operators is rounded to the io type, as there."""
    z, io_of = blk.z, lambda a: ref.cast(a, io)
    W = {n: from_dev(getattr(blk, n)) for n in ("W_qkv", "W_a", "W_b", "W_out", "A", "bias", "norm_w", "norm_b")}
    B, L, _ = X.shape
    x = X.reshape(B * L, -1)
    p, nk = io_of(x @ W["W_qkv"]), z.Hk * z.dk
    q, k, v = p[:, :nk].reshape(-1, z.Hk, z.dk), p[:, nk:2 * nk].reshape(-1, z.Hk, z.dk), p[:, 2 * nk:].reshape(-1, z.H, z.dv)
    raw = x @ W["W_a"] + W["bias"]
    sp, sig = np.logaddexp(0, raw), 1 / (1 + np.exp(-raw))
    g, beta = io_of(W["A"] * sp), io_of(1 / (1 + np.exp(-(x @ W["W_b"]))))
    ends = np.arange(1, B + 1) * L
    o, S = ref.delta(q, k, v, g, beta, state, ends, z.dk ** -0.5, True)
    o = io_of(o)
    y, mean, rstd = ref.group_norm(o.reshape(B * L, 1, -1), z.H, W["norm_w"], W["norm_b"], 1e-5, True)
    y = io_of(y)
    out = y[:, 0] @ W["W_out"]
    d = dout.reshape(B * L, -1)
    do, dw, db = ref.group_norm_bwd(io_of(d @ W["W_out"].T)[:, None], o.reshape(B * L, 1, -1), mean, rstd, W["norm_w"], W["norm_b"], True)
    gr = ref.delta_bwd(q, k, v, g, beta, state, ends, z.dk ** -0.5, True, io_of(do).reshape(o.shape), np.zeros(S.shape))
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        gr[n] = io_of(gr[n])
    dp = np.concatenate([gr[n].reshape(B * L, -1) for n in ("dq", "dk", "dv")], -1)
    da, dbr = gr["dg"] * W["A"] * sig, gr["dbeta"] * beta * (1 - beta)
    grads = dict(dW_out=y[:, 0].T @ d, dnorm_w=dw, dnorm_b=db, dW_qkv=x.T @ dp, dW_a=x.T @ da, dW_b=x.T @ dbr,
                 dA=(gr["dg"] * sp).sum(0), dbias=da.sum(0), dstate0=gr["dh0"],
                 dX=(dp @ W["W_qkv"].T + da @ W["W_a"].T + dbr @ W["W_b"].T).reshape(X.shape))
    return out.reshape(B, L, -1), S, grads


# float32: a chain of products of up to 200 terms each way, 2e-4 of the rms.  bfloat16: every tensor between the
# operators is rounded (2^-9 each, some ten of them in a row): 5 % of the rms.
GRADE = {"f32": (2e-4, 2e-4), "bf16": (2.0 ** -6, 0.05)}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2)])
def test_forward_backward_and_steps(H, Hk, io):
    import torch
    from selective_scan_segmented_amd.delta_block import DeltaBlock, DeltaSizes
    B, L, C = 2, 70, 48
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    blk = DeltaBlock(DeltaSizes(C=C, H=H, Hk=Hk, dk=32, dv=48), dtype=dt, seed=H)
    rng = np.random.default_rng(7)
    X, dout = ref.cast(rng.standard_normal((B, L, C)), io), ref.cast(rng.standard_normal((B, L, C)), io)
    state = (rng.standard_normal((B, H, 32, 48)) / 6).astype(np.float32).astype(np.float64)
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    Xd, sd = dev(X, dt), dev(state, torch.float32)
    out, S = blk.forward(Xd, state=sd, return_state=True, keep=True)
    grads = blk.backward(dev(dout, dt))
    torch.cuda.synchronize()
    wo, wS, wg = reference(blk, X, state, dout, io)
    ref.close(from_dev(out), wo, io, "out", GRADE[io])
    ref.close(from_dev(S), wS, io, "state", GRADE[io])
    assert sorted(grads) == sorted(wg)
    for n in wg:
        ref.close(from_dev(grads[n]), wg[n], io, n, GRADE[io])
    # token by token from the same state
    pool = sd.clone()
    for t in range(3):
        o = blk.step(Xd[:, t].contiguous(), pool)
        ref.close(from_dev(o), wo[:, t], io, f"step {t}", GRADE[io])
