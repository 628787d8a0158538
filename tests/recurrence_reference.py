"""The gated linear recurrence and the norm with rotation of queries and keys by their definitions, in float64 numpy."""
import numpy as np

from delta_reference import cast


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-v))


def gates(r, i, lam, c):
    """a, log a, sqrt(1 - a^2), sigmoid(r), sigmoid(i)."""
    sr, si = sigmoid(r), sigmoid(i)
    la = -c * np.logaddexp(0, lam) * sr
    return np.exp(la), la, np.sqrt(-np.expm1(2 * la)), sr, si


def recurrence(x, r, i, lam, h0, ends, c):
    """Packed rows [tokens, D] with row ends; returns y and the states after the rows."""
    a, _, m, _, si = gates(r, i, lam, c)
    y, hT, lo = np.zeros(x.shape), h0.copy(), 0
    for row, hi in enumerate(ends):
        for t in range(lo, hi):
            hT[row] = y[t] = a[t] * hT[row] + m[t] * si[t] * x[t]
        lo = hi
    return y, hT


def recurrence_bwd(x, r, i, lam, h0, y, ends, c, dy, dhT):
    """Gradients of sum(y dy) + sum(hT dhT), the states that the decays see taken from y.  Beside dlam the sum of the
    magnitudes of the products that its terms are differences of (dlam_size).  A term p - q computed with products off by
    e |p| and e |q| is off by up to e (|p| + |q|), however small p - q is: that is what dlam's rounding goes by."""
    a, la, m, sr, si = gates(r, i, lam, c)
    G, before, back, lo = np.zeros(x.shape), np.zeros(x.shape), dhT.copy(), 0
    for row, hi in enumerate(ends):
        for t in reversed(range(lo, hi)):
            G[t] = dy[t] + back[row]
            back[row] = a[t] * G[t]
            before[t] = y[t - 1] if t > lo else h0[row]
        lo = hi
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(m > 0, a * a * la / m, 0.0)
    P = G * (a * la * before - q * si * x)
    ratio = sigmoid(lam) / np.logaddexp(0, lam)
    return dict(dx=G * m * si, dr=P * (1 - sr), di=G * m * x * si * (1 - si), dlam=ratio * P.sum(0), dh0=back,
                dlam_size=ratio * (np.abs(G) * (np.abs(a * la * before) + np.abs(q * si * x))).sum(0))


def recurrence_inputs(seed, tokens, rows, D, io):
    """x, r, i, lam, h0, dy, dhT: float64 values that `io` holds exactly (lam and states: float32)."""
    rng = np.random.default_rng(seed)
    f32 = lambda v: v.astype(np.float32).astype(np.float64)
    x, r, i, dy = (cast(rng.standard_normal((tokens, D)), io) for _ in range(4))
    lam = f32(np.log(np.expm1(-np.log(rng.uniform(0.9, 0.999, D)))))
    return x, r, i, lam, f32(rng.standard_normal((rows, D))), dy, f32(rng.standard_normal((rows, D)))


def places(d, rot, neighbours):
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if neighbours else (j, j + rot // 2)


def turn(z, angle, rot, neighbours):
    """The pairs of [tokens, heads, d] turned by angle [tokens, rot / 2]."""
    one, two = places(z.shape[-1], rot, neighbours)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    out = z.copy()
    out[..., one], out[..., two] = z[..., one] * c - z[..., two] * s, z[..., two] * c + z[..., one] * s
    return out


def angles(positions, freqs, sections):
    """[tokens, axes] positions -> [tokens, rot / 2]."""
    axis = np.repeat(np.arange(len(sections)), sections)
    return positions[:, axis].astype(np.float64) * freqs


def rope(x, w, angle, rot, neighbours, norm, eps):
    z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w if norm else x
    return turn(z, angle, rot, neighbours)


def rope_bwd(x, w, angle, rot, neighbours, norm, eps, dy):
    """dx, dw and the sum of dw's terms' magnitudes."""
    g = turn(dy, -angle, rot, neighbours)
    if not norm:
        return g, None, None
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh, gw = x * rstd, g * w
    return rstd * (gw - xh * (gw * xh).mean(-1, keepdims=True)), (g * xh).sum((0, 1)), np.abs(g * xh).sum((0, 1))
