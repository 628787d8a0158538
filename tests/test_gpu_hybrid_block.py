"""A recurrence block and a delta block with normed and rotated queries and keys, one after the other as hybrid models
stack them: forward, backward, and token by token from the states, against float64."""
import numpy as np
import pytest

import delta_reference as dref
import recurrence_reference as ref
from delta_reference import cast, close
from helpers import from_dev

pytestmark = pytest.mark.gpu

# float32: chains of products of up to 200 terms each way, 2e-4 of the rms.  bfloat16: some ten tensors in a row are rounded
# on the way forward and again on the way back (2^-9 each in rms, not all in phase): 2^-6 and 5 % of the rms.
GRADE = {"f32": (2e-4, 2e-4), "bf16": (2.0 ** -6, 0.05)}
B, L, C, D = 2, 90, 48, 64
H, HK, DK, DV, ROT = 4, 2, 32, 24, 16


def recurrent(blk, X, state, io):
    """The recurrence block's forward in float64, what it stores between operators rounded to the io type."""
    io_of = lambda a: cast(a, io)
    W = {n: from_dev(getattr(blk, n)) for n in ("W_in", "W_out", "lam")}
    x = X.reshape(B * L, C)
    p = io_of(x @ W["W_in"])
    xs, r, i, z = (p[:, n * D:(n + 1) * D] for n in range(4))
    h, S = ref.recurrence(xs, r, i, W["lam"], state, np.arange(1, B + 1) * L, 8.0)
    h = io_of(h)
    y = io_of(h * z * ref.sigmoid(z))
    return dict(W=W, x=x, parts=(xs, r, i, z), h=h, y=y, S=S, out=(y @ W["W_out"]).reshape(B, L, C))


def recurrent_bwd(k, state, dout, io):
    io_of = lambda a: cast(a, io)
    xs, r, i, z = k["parts"]
    d = dout.reshape(B * L, C)
    dy = io_of(d @ k["W"]["W_out"].T)
    s = ref.sigmoid(z)
    g = ref.recurrence_bwd(xs, r, i, k["W"]["lam"], state, k["h"], np.arange(1, B + 1) * L, 8.0, io_of(dy * z * s), np.zeros(state.shape))
    dp = np.concatenate([io_of(g["dx"]), io_of(g["dr"]), io_of(g["di"]), io_of(dy * k["h"] * s * (1 + z * (1 - s)))], -1)
    return dict(dW_out=k["y"].T @ d, dW_in=k["x"].T @ dp, dlam=g["dlam"], dstate0=g["dh0"], dX=(dp @ k["W"]["W_in"].T).reshape(B, L, C))


def delta(blk, X, state, dout, io):
    """The delta block with rotation in float64: out, states, gradients."""
    io_of = lambda a: cast(a, io)
    W = {n: from_dev(getattr(blk, n)) for n in ("W_qkv", "W_a", "W_b", "W_out", "A", "bias", "norm_w", "norm_b", "wq", "wk", "freqs")}
    x = X.reshape(B * L, C)
    p, nk = io_of(x @ W["W_qkv"]), HK * DK
    q0, k0, v = p[:, :nk].reshape(-1, HK, DK), p[:, nk:2 * nk].reshape(-1, HK, DK), p[:, 2 * nk:].reshape(-1, H, DV)
    ang = np.tile(np.arange(L), B)[:, None] * W["freqs"]
    form = (ang, ROT, False, True, 1e-6)
    q, k = io_of(ref.rope(q0, W["wq"], *form)), io_of(ref.rope(k0, W["wk"], *form))
    raw = x @ W["W_a"] + W["bias"]
    sp, sig = np.logaddexp(0, raw), ref.sigmoid(raw)
    g, beta = io_of(W["A"] * sp), io_of(ref.sigmoid(x @ W["W_b"]))
    ends = np.arange(1, B + 1) * L
    o, S = dref.delta(q, k, v, g, beta, state, ends, DK ** -0.5, True)
    o = io_of(o)
    y, mean, rstd = dref.group_norm(o.reshape(B * L, 1, -1), H, W["norm_w"], W["norm_b"], 1e-5, True)
    y = io_of(y)
    d = dout.reshape(B * L, -1)
    do, dw, db = dref.group_norm_bwd(io_of(d @ W["W_out"].T)[:, None], o.reshape(B * L, 1, -1), mean, rstd, W["norm_w"], W["norm_b"], True)
    gr = dref.delta_bwd(q, k, v, g, beta, state, ends, DK ** -0.5, True, io_of(do).reshape(o.shape), np.zeros(S.shape))
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        gr[n] = io_of(gr[n])
    dq, dwq, _ = ref.rope_bwd(q0, W["wq"], *form, gr["dq"])
    dk, dwk, _ = ref.rope_bwd(k0, W["wk"], *form, gr["dk"])
    dp = np.concatenate([io_of(dq).reshape(B * L, -1), io_of(dk).reshape(B * L, -1), gr["dv"].reshape(B * L, -1)], -1)
    da, dbr = gr["dg"] * W["A"] * sig, gr["dbeta"] * beta * (1 - beta)
    grads = dict(dW_out=y[:, 0].T @ d, dnorm_w=dw, dnorm_b=db, dW_qkv=x.T @ dp, dW_a=x.T @ da, dW_b=x.T @ dbr, dwq=dwq, dwk=dwk,
                 dA=(gr["dg"] * sp).sum(0), dbias=da.sum(0), dstate0=gr["dh0"],
                 dX=(dp @ W["W_qkv"].T + da @ W["W_a"].T + dbr @ W["W_b"].T).reshape(X.shape))
    return (y[:, 0] @ W["W_out"]).reshape(B, L, -1), S, grads


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_stack_forward_backward_and_steps(io):
    import torch
    from selective_scan_segmented_amd.delta_block import DeltaBlock, DeltaSizes
    from selective_scan_segmented_amd.recurrent_block import RecurrentBlock
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    one = RecurrentBlock(C, D, dtype=dt, seed=1)
    two = DeltaBlock(DeltaSizes(C=C, H=H, Hk=HK, dk=DK, dv=DV, rot=ROT), dtype=dt, seed=2)
    rng = np.random.default_rng(7)
    X, dout = cast(rng.standard_normal((B, L, C)), io), cast(rng.standard_normal((B, L, C)), io)
    s1 = rng.standard_normal((B, D)).astype(np.float32).astype(np.float64)
    s2 = (rng.standard_normal((B, H, DK, DV)) / 6).astype(np.float32).astype(np.float64)
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    Xd, a1, a2 = dev(X, dt), dev(s1, torch.float32), dev(s2, torch.float32)

    m, S1 = one.forward(Xd, state=a1, return_state=True, keep=True)
    X1 = Xd + m
    out, S2 = two.forward(X1, state=a2, return_state=True, keep=True)
    g2 = two.backward(dev(dout, dt))
    g1 = one.backward(g2["dX"])
    torch.cuda.synchronize()

    k1 = recurrent(one, X, s1, io)
    x1 = cast(X + cast(k1["out"], io), io)
    wo, wS, wg2 = delta(two, x1, s2, dout, io)
    wg1 = recurrent_bwd(k1, s1, cast(wg2["dX"], io), io)
    for name, got, want in (("mixer", m, k1["out"]), ("state 1", S1, k1["S"]), ("out", out, wo), ("state 2", S2, wS)):
        close(from_dev(got), want, io, name, GRADE[io])
    assert sorted(g2) == sorted(wg2) and sorted(g1) == sorted(wg1)
    for got, want in ((g2, wg2), (g1, wg1)):
        for n in want:
            close(from_dev(got[n]), want[n], io, n, GRADE[io])

    # token by token on pools of states, whose slots are not in the requests' order
    slots = torch.tensor([2, 0], dtype=torch.int32).cuda()
    p1, p2 = torch.zeros(3, D, device="cuda"), torch.zeros(3, H, DK, DV, device="cuda")
    p1[slots.long()], p2[slots.long()] = a1, a2
    for t in range(3):
        x = Xd[:, t].contiguous()
        x1 = x + one.step(x, p1, slots=slots)
        o = two.step(x1, p2, slots=slots, positions=torch.full((B,), t, dtype=torch.int32, device="cuda"))
        close(from_dev(o), wo[:, t], io, f"step {t}", GRADE[io])
