"""The gated recurrence beside gates that are shut and rates past any use: states that are kept, gradients of large
inputs that a shut gate keeps out, states beside a decay of zero.  Each gradient is a sum of products; float32 may be off
by its part of their magnitudes (1e-4: the tests' own for gradients), however small or large they are, and nothing turns
into NaN."""
import numpy as np
import pytest

import recurrence_reference as ref
from helpers import from_dev
from test_gpu_recurrence import dev

pytestmark = pytest.mark.gpu
L, D = 40, 16
PART, STEP = 1e-4, {"f32": 0.0, "bf16": 2.0 ** -8}


def magnitudes(x, r, i, lam, h0, y, dy, dhT):
    """What the gradients' products amount to, with the largest gradient of a channel's states in every token's place."""
    a, la, m, sr, si = ref.gates(r, i, lam, 8.0)
    G, back = np.zeros(x.shape), dhT[0].copy()
    for t in reversed(range(L)):
        G[t] = np.abs(dy[t]) + np.abs(back)
        back = a[t] * G[t]
    G = np.broadcast_to(G.max(0), G.shape)
    before = np.abs(np.concatenate([h0, y[:-1]]))
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(m > 0, a * a * np.abs(la) / m, 0.0)
    P = G * (a * np.abs(la) * before + q * si * np.abs(x))
    # Where sigmoid(r) or log a is below 2^-126 float32 has 0 in its place, and so 0 for the input's factor m.  log a is at
    # most c softplus(lam) <= 0.84 of sigmoid(r) there (rates from 0.9 on), so what is lost of m is below sqrt(2 2^-126) =
    # 2^-62.5; of a gradient at most that times G max(1, |x|) (dx: m si; di: m x si (1 - si); dr: m / 2 si x; dlam: their sum).
    lost = 2.0 ** -62 * G * np.maximum(1.0, np.abs(x))
    lost = dict(dx=lost, dr=lost, di=lost, dlam=lost.sum(0), dh0=0.0)
    return lost, dict(dx=G * m * si, dr=P * (1 - sr), di=G * m * np.abs(x) * si * (1 - si), dlam=ref.sigmoid(lam) / np.logaddexp(0, lam) * P.sum(0),
                dh0=(a[0] * G[0])[None])


def run(x, r, i, lam, s0, dy, dhT, io):
    import selective_scan_segmented_amd as sfm
    t = [dev(v, io).view(1, L, D) for v in (x, r, i)] + [dev(lam, "f32")]
    h0 = dev(s0, "f32")
    y = sfm.sfm_gated_recurrence_fwd(*t, h0=h0)
    got = sfm.sfm_gated_recurrence_bwd(*t, y, dev(dy, io).view(1, L, D), h0=h0, dstate=dev(dhT, "f32"))
    want = from_dev(y)[0]
    assert np.isfinite(want).all()
    w = ref.recurrence_bwd(x, r, i, lam, s0, want, [L], 8.0, dy, dhT)
    lost, size = magnitudes(x, r, i, lam, s0, want, dy, dhT)
    for n in ("dx", "dr", "di", "dlam", "dh0"):
        g = from_dev(got[n]).reshape(w[n].shape)
        assert np.isfinite(g).all(), f"{n}: not finite at {np.argwhere(~np.isfinite(g))[:4].tolist()}"
        step = 0.0 if n in ("dlam", "dh0") else STEP[io]
        bound = PART * size[n] + step * np.abs(w[n]) + lost[n] + 1e-30
        assert (np.abs(g - w[n]) <= bound).all(), (n, np.max(np.abs(g - w[n]) / bound))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shut", [-np.inf, -200.0, -84.0, -80.0])
@pytest.mark.parametrize("size", [1.0, 1e22, -1e30])
def test_large_inputs_of_shut_gates(size, shut, io):
    x, r, i, lam, s0, dy, dhT = ref.recurrence_inputs(11, L, 1, D, io)
    for n, tok in enumerate((0, 5, 7, 8, 16, 33, L - 1)):
        x[tok, n], r[tok, n] = ref.cast(np.array([size]), io)[0] if size != 1.0 else x[tok, n], shut
    # one input that is shut out for one channel's whole row
    x[:, 12], r[:, 12] = x[:, 12] * np.float64(2.0 ** 60), shut
    run(x, r, i, lam, s0, dy, dhT, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [20.0, 1e30, 1e37, 1e38, 3e38])
def test_states_beside_decays_of_zero(rate, io):
    """Rates that forget within a token: the decay's gradient is 0, whatever the states are."""
    x, r, i, lam, s0, dy, dhT = ref.recurrence_inputs(12, L, 1, D, io)
    lam[::3] = np.float32(rate)
    x[:, ::3] *= 1024.0
    run(x, r, i, lam, s0, dy, dhT, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_shut_gates_keep_states_to_the_bit_within_a_chunk(io):
    """Gates shut from token 4 to token 20; a lane walks tokens 0 to 15, another one 16 on."""
    import torch
    import selective_scan_segmented_amd as sfm
    x, r, i, lam, s0, _, _ = ref.recurrence_inputs(13, L, 1, D, io)
    r[4:21:2], r[5:21:2] = -np.inf, -200.0
    t = [dev(v, io).view(1, L, D) for v in (x, r, i)] + [dev(lam, "f32")]
    h0 = dev(s0, "f32")
    y = sfm.sfm_gated_recurrence_fwd(*t, h0=h0)[0]
    for tok in range(4, 16):
        assert torch.equal(y[tok], y[3]), tok
    for tok in range(17, 21):
        assert torch.equal(y[tok], y[16]), tok
    # Token 15 is 16 fused steps from h0.  Token 16 is A h0 + H: A of 16 products, H of 16 fused steps, each of these rounded
    # by 2^-24 of a state (H: of twice the largest, since H = h - A h0), and the last step: (16 + 16 + 2 16 + 2) 2^-24 apart.
    states = sfm.sfm_gated_recurrence_fwd(*[v[:, :16].float() for v in t[:3]], t[3], h0=h0)[0]
    largest = torch.cat([h0, states]).abs().max(0).values
    step = 66 * 2.0 ** -24 * largest + (2.0 ** -7 * y[3].float().abs() if io == "bf16" else 0)
    assert ((y[15].float() - y[16].float()).abs() <= step).all()
