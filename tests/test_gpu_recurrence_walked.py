"""Rows that a workgroup walks block after block, forward and backward: every output against the definition in float64.

A row is walked where rows and their tiles of 32 lanes fill the card: equal rows backward from 640 of them on (forward
from 512), packed ones from 256 to 6144 on, by their lengths.  Blocks are of up to 128 tokens forward and 64 backward."""
import numpy as np
import pytest

from test_gpu_recurrence import BACKWARD, FORWARD

pytestmark = pytest.mark.gpu


def definition(x, r, i, lam, h0, dy, dhT, y=None):
    """float64 [rows, L, D], rows padded with r = -inf (a = 1) and zeros.  The states before tokens are taken from y."""
    import torch
    sp = torch.logaddexp(lam, torch.zeros_like(lam))
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    la = -8.0 * sp * sr
    a, m = la.exp(), (-torch.expm1(2 * la)).sqrt()
    h, states = h0, []
    for t in range(x.shape[1]):
        h = a[:, t] * h + m[:, t] * si[:, t] * x[:, t]
        states.append(h)
    out = {"y": torch.stack(states, 1), "state": h}
    if y is None:
        return out
    back, G = dhT, torch.zeros_like(x)
    for t in reversed(range(x.shape[1])):
        G[:, t] = dy[:, t] + back
        back = a[:, t] * G[:, t]
    before = torch.cat([h0.unsqueeze(1), y[:, :-1]], 1)
    q = torch.where(m > 0, a * a * la / m, torch.zeros_like(m))
    first, second = a * la * before, q * si * x
    P = G * (first - second)
    ratio = torch.sigmoid(lam) / sp
    out.update(dx=G * m * si, dr=P * (1 - sr), di=G * m * x * si * (1 - si), dh0=back, dlam=ratio * P.sum((0, 1)),
               dlam_size=ratio * (G.abs() * (first.abs() + second.abs())).sum((0, 1)))
    return out


def near(got, want, grade, what):
    import torch
    rel, part = grade
    bound = rel * want.abs() + part * want.square().mean().sqrt() + 1e-30
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), (what, float((err / bound).nan_to_num(nan=torch.inf).max()))


def check(lens, D, io, packed, seed):
    import torch
    import selective_scan_segmented_amd as sfm
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    rows, tokens, L = len(lens), int(sum(lens)), int(max(lens))
    lead = (1, tokens) if packed else (rows, L)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x, r, i, dy = (n(*lead, D).to(dt) for _ in range(4))
    lam = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda"))))
    h0, dhT = n(rows, D), n(rows, D)
    form = dict(h0=h0)
    if packed:
        form.update(offsets=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda"), max_len=L)
    y, state = sfm.sfm_gated_recurrence_fwd(x, r, i, lam, return_state=True, **form)
    g = sfm.sfm_gated_recurrence_bwd(x, r, i, lam, y, dy, dstate=dhT, **form)
    inside = torch.arange(L, device="cuda") < torch.tensor(lens, device="cuda").unsqueeze(1)

    def rows_of(t, none=0.0):
        full = torch.full((rows, L, D), none, dtype=torch.float64, device="cuda")
        full[inside] = t.reshape(-1, D).double()
        return full

    # (the state before a token is y of the one before it, so that what stands behind a row's end does not matter)
    w = definition(rows_of(x), rows_of(r, -float("inf")), rows_of(i), lam.double(), h0.double(), rows_of(dy), dhT.double(), rows_of(y))
    near(y.reshape(-1, D), w["y"][inside], FORWARD[io], "y")
    near(state, w["state"], FORWARD["f32"], "state")
    for k in ("dx", "dr", "di"):
        near(g[k].reshape(-1, D), w[k][inside], BACKWARD[io], k)
    near(g["dh0"], w["dh0"], BACKWARD["f32"], "dh0")
    assert bool(((g["dlam"].double() - w["dlam"]).abs() <= 1e-5 * w["dlam_size"]).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,L,D", [(256, 198, 320), (640, 150, 64), (40, 600, 1024), (330, 200, 63)])
def test_equal_rows(rows, L, D, io):
    check([L] * rows, D, io, False, L)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,most,D", [(900, 300, 256), (1300, 140, 129)])
def test_packed_rows(rows, most, D, io):
    """Some of them empty, one as long as they may be."""
    lens = np.random.default_rng(rows).integers(0, most, rows)
    lens[[0, 5, rows - 1]], lens[7] = 0, most
    check(lens, D, io, True, most)
