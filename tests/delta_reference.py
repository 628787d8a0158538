"""The gated delta rule and the channel-last group norm by their definitions, in float64 numpy, token by token."""
import numpy as np

EPS = 1e-6


def unit(x, on):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + EPS) if on else x


def delta_row(q, k, v, g, beta, S, scale, l2norm):
    """One row: q, k [T, Hk, dk], v [T, H, dv], g, beta [T, H], S [H, dk, dv] -> o, S, and what the
    backward needs of every token."""
    share = v.shape[1] // q.shape[1]
    o = np.zeros(v.shape)
    S = S.copy()
    seen = []
    for t in range(len(q)):
        qt, kt = (np.repeat(unit(x[t], l2norm), share, 0) for x in (q, k))
        a = np.exp(g[t])[:, None, None]
        r = v[t] - np.einsum("hkv,hk->hv", a * S, kt)
        u = beta[t][:, None] * r
        new = a * S + kt[:, :, None] * u[:, None, :]
        seen.append((qt, kt, a, r, u, S, new))
        S = new
        o[t] = scale * np.einsum("hkv,hk->hv", S, qt)
    return o, S, seen


def delta_row_bwd(q, k, v, g, beta, S, scale, l2norm, do, dS):
    """Gradients of sum(o * do) + sum(S_end * dS) for one row."""
    share = v.shape[1] // q.shape[1]
    _, _, seen = delta_row(q, k, v, g, beta, S, scale, l2norm)
    dq, dk, dv, dg, db = (np.zeros(x.shape) for x in (q, k, v, g, beta))
    dS = dS.copy()

    def raw(d, x):
        d = d.reshape(x.shape[0], share, -1).sum(1)
        if l2norm:
            n = np.sqrt((x * x).sum(-1, keepdims=True) + EPS)
            d = d / n - x * (x * d).sum(-1, keepdims=True) / n ** 3
        return d

    for t in reversed(range(len(q))):
        qt, kt, a, r, u, S0, S1 = seen[t]
        at = dS + scale * qt[:, :, None] * do[t][:, None, :]
        du = np.einsum("hkv,hk->hv", at, kt)
        dr = beta[t][:, None] * du
        dq[t] = raw(scale * np.einsum("hkv,hv->hk", S1, do[t]), q[t])
        dk[t] = raw(np.einsum("hkv,hv->hk", at, u) - np.einsum("hkv,hv->hk", a * S0, dr), k[t])
        dv[t] = dr
        db[t] = (du * r).sum(-1)
        before = at - kt[:, :, None] * dr[:, None, :]
        dg[t] = (a * before * S0).sum((-1, -2))
        dS = a * before
    return dq, dk, dv, dg, db, dS


def delta(q, k, v, g, beta, h0, ends, scale, l2norm):
    """Packed rows [tokens, ...] with row ends; returns o and the states."""
    o, hT, lo = np.zeros(v.shape), np.zeros(h0.shape), 0
    for r, hi in enumerate(ends):
        o[lo:hi], hT[r], _ = delta_row(q[lo:hi], k[lo:hi], v[lo:hi], g[lo:hi], beta[lo:hi], h0[r], scale, l2norm)
        lo = hi
    return o, hT


def delta_bwd(q, k, v, g, beta, h0, ends, scale, l2norm, do, dhT):
    outs = [np.zeros(x.shape) for x in (q, k, v, g, beta)] + [np.zeros(h0.shape)]
    lo = 0
    for r, hi in enumerate(ends):
        got = delta_row_bwd(q[lo:hi], k[lo:hi], v[lo:hi], g[lo:hi], beta[lo:hi], h0[r], scale, l2norm, do[lo:hi], dhT[r])
        for out, x in zip(outs[:5], got[:5]):
            out[lo:hi] = x
        outs[5][r] = got[5]
        lo = hi
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), outs))


def group_norm(x, G, w, b, eps, act):
    N, L, C = x.shape
    xg = x.reshape(N, L, G, C // G)
    mean = xg.mean((1, 3))
    rstd = 1 / np.sqrt(((xg - mean[:, None, :, None]) ** 2).mean((1, 3)) + eps)
    xh = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(N, L, C)
    z = xh * w + b
    y = z / (1 + np.exp(-z)) if act else z
    return y, mean, rstd


def group_norm_bwd(dy, x, mean, rstd, w, b, act):
    N, L, C = x.shape
    G = mean.shape[1]
    xh = ((x.reshape(N, L, G, -1) - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(N, L, C)
    z = xh * w + b
    s = 1 / (1 + np.exp(-z))
    dz = dy * (s * (1 + z * (1 - s)) if act else 1.0)
    e = (dz * w).reshape(N, L, G, -1)
    xg = xh.reshape(N, L, G, -1)
    dx = rstd[:, None, :, None] * (e - e.mean((1, 3), keepdims=True) - xg * (e * xg).mean((1, 3), keepdims=True))
    return dx.reshape(N, L, C), (dz * xh).sum((0, 1)), dz.sum((0, 1))


def delta_inputs(seed, tokens, rows, Hk, H, dk, dv, l2norm, io):
    """float64 inputs that `io` holds exactly."""
    rng = np.random.default_rng(seed)
    q, k, v = rng.standard_normal((tokens, Hk, dk)), rng.standard_normal((tokens, Hk, dk)) + 0.5, rng.standard_normal((tokens, H, dv))
    if not l2norm:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True)) for x in (q, k))
    g = -np.exp(rng.uniform(np.log(1e-3), np.log(1.5), (tokens, H)))
    beta = 1 / (1 + np.exp(-rng.standard_normal((tokens, H))))
    h0 = (rng.standard_normal((rows, H, dk, dv)) / np.sqrt(dk)).astype(np.float32).astype(np.float64)
    do = rng.standard_normal((tokens, H, dv))
    return [cast(x, io) for x in (q, k, v, g, beta)] + [h0, cast(do, io)]


def cast(x, io):
    """float64 values rounded to the io type."""
    from selective_scan_segmented_amd import synth
    x = np.asarray(x, dtype=np.float32)
    return synth.bf16_bits_to_f64(synth.f32_to_bf16_bits(x)) if io == "bf16" else x.astype(np.float64)


def close(got, want, io, what, grade=None):
    """|got - want| <= rel |want| + part of its rms.  float32: sums of at most a few hundred products of unit
    size, 2^-24 each, so 2e-5 of both.  bfloat16: one rounding of the result, 2^-9 of it, doubled for results
    that sit at a rounding boundary, and 1e-4 of the rms for the arithmetic below it.  `grade`: another pair."""
    rel, part = grade or ((2e-5, 2e-5) if io == "f32" else (2.0 ** -8, 1e-4))
    want = np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if not want.size:
        return
    bound = rel * np.abs(want) + part * np.sqrt(np.mean(want * want)) + 1e-30
    err = np.abs(got - want)
    worst = np.max(np.where(np.isfinite(err), err / bound, np.inf))
    assert worst <= 1.0, f"{what}: worst error {worst:.3g} of its bound at {np.unravel_index(np.argmax(err / bound), err.shape)}"
