"""Values behind the rotated part of a head: they are normed and weighted, and nothing that stands beside them reaches
them.  Infinities and NaN there stay in their place, by the definition in float64, value by value."""
import numpy as np
import pytest

import recurrence_reference as ref
from helpers import from_dev
from test_gpu_qk_rope import BACKWARD, EPS, FORWARD, dev, inputs

pytestmark = pytest.mark.gpu

PARTS = [(64, 0), (64, 32), (128, 96), (33, 16), (3, 2), (2, 0), (96, 48), (48, 46), (256, 64), (255, 100), (40, 8)]


def same(got, want, what, grade):
    """Non-finite where `want` is, with its sign, and NaN where it is NaN; else within rel |want| + part of the finite rms."""
    rel, part = grade
    fin = np.isfinite(want)
    assert (np.isfinite(got) == fin).all(), f"{what}: non-finite at {np.argwhere(np.isfinite(got) != fin)[:5].tolist()}"
    np.testing.assert_array_equal(got[~fin], want[~fin], err_msg=what)
    w = want[fin]
    bound = rel * np.abs(w) + part * np.sqrt(np.mean(w * w)) + 1e-30
    assert (np.abs(got[fin] - w) <= bound).all(), what


def place(t, rot, bad):
    """One value of every token's first head behind its rotated part; places move on from token to token."""
    t = t.copy()
    for n in range(len(t)):
        t[n, 0, rot + n % (t.shape[-1] - rot)] = bad
    return t


def form_of(rot, pos, freqs, neighbours, norm, weights=()):
    import torch
    form = dict(interleaved=neighbours, norm=norm, eps=EPS, **{n: dev(w, "f32") for n, w in weights})
    if rot:
        form.update(positions=torch.from_numpy(pos[:, 0].copy()).cuda(), freqs=dev(freqs, "f32"))
    return form


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,rot", PARTS)
def test_without_norm(d, rot, io, neighbours, bad):
    """Both directions copy the tail, to the bit."""
    import torch
    import selective_scan_segmented_amd as sfm
    tokens = max(40, d - rot)
    q, k, dq, dk, _, _, freqs, sec, pos = inputs(d, (tokens,), 2, 1, d, rot, io, weights=False)
    ang = ref.angles(pos, freqs, sec)
    form = form_of(rot, pos, freqs, neighbours, False)
    q, k, dq, dk = (place(t, rot, bad) for t in (q, k, dq, dk))
    tq, tk, uq, uk = (dev(t, io) for t in (q, k, dq, dk))
    qo, ko = sfm.sfm_qk_norm_rope_fwd(tq, tk, **form)
    g = sfm.sfm_qk_norm_rope_bwd(uq, uk, tq, tk, **form)
    bits = torch.int16 if io == "bf16" else torch.int32
    for got, by, x, sign, grade in ((qo, tq, q, 1, FORWARD), (ko, tk, k, 1, FORWARD), (g["dq"], uq, dq, -1, BACKWARD), (g["dk"], uk, dk, -1, BACKWARD)):
        a, b = got[..., rot:], by[..., rot:]
        number = ~torch.isnan(b)
        assert torch.equal(a.contiguous().view(bits)[number], b.contiguous().view(bits)[number]) and torch.isnan(a[~number]).all()
        if rot:
            z = x[..., :rot]
            same(from_dev(got)[..., :rot], ref.turn(z, sign * ang, rot, neighbours), "rotated", grade[io])


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,rot", PARTS)
def test_gradients_of_weights(d, rot, io, neighbours, bad):
    """A non-finite gradient behind the rotation reaches its own weight's gradient and no other's.  (Its head's dx goes
    by the mean of all its values, so that it is non-finite throughout.)"""
    import selective_scan_segmented_amd as sfm
    q, k, dq, dk, wq, wk, freqs, sec, pos = inputs(d + 1, (30,), 2, 1, d, rot, io)
    ang = ref.angles(pos, freqs, sec)
    j = rot + (d - rot) // 2
    dq[7, 1, j] = dk[11, 0, j] = bad
    form = form_of(rot, pos, freqs, neighbours, True, (("wq", wq), ("wk", wk)))
    g = sfm.sfm_qk_norm_rope_bwd(dev(dq, io), dev(dk, io), dev(q, io), dev(k, io), **form)
    for n, x, w, dy, head in (("q", q, wq, dq, (7, 1)), ("k", k, wk, dk, (11, 0))):
        with np.errstate(invalid="ignore"):
            dx, dw, size = ref.rope_bwd(x, w, ang, rot, neighbours, True, EPS, dy)
        got, other = from_dev(g["dw" + n]), np.arange(d) != j
        assert not np.isfinite(got[j]) and np.isnan(got[j]) == np.isnan(dw[j])
        assert (np.abs(got[other] - dw[other]) <= 1e-5 * size[other] + 1e-30).all(), "dw" + n
        rest = np.ones(x.shape[:2], bool)
        rest[head] = False
        same(from_dev(g["d" + n])[rest], dx[rest], "d" + n, BACKWARD[io])
        assert not np.isfinite(from_dev(g["d" + n])[head]).any()
