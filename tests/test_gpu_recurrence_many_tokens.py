"""Packed and equal rows of more than 2^24 tokens, the packed ones without a bound, against the definition in float64.

Decays are at most 0.999^(8 sigmoid(r)), r from a normal distribution: over 6000 tokens a state keeps less than e^-20 of
itself, far below a rounding, so that the definition of a row's last tokens alone gives its end."""
import numpy as np
import pytest

import recurrence_reference as ref
from delta_reference import close
from helpers import from_dev
from test_gpu_recurrence import BACKWARD, FORWARD

pytestmark = pytest.mark.gpu
REACH, SEEN = 6000, 500


def tensors(seed, tokens, D, io):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    n = lambda: torch.randn(1, tokens, D, generator=gen, device="cuda").to(dt)
    lam = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda"))))
    return [n(), n(), n(), lam, n()]


def check(t, lens, io, **rows):
    """A few rows' ends forward (and beginnings backward) against the definition."""
    import selective_scan_segmented_amd as sfm
    x, r, i, lam, dy = t
    D = x.shape[-1]
    y, S = sfm.sfm_gated_recurrence_fwd(x, r, i, lam, return_state=True, **rows)
    g = sfm.sfm_gated_recurrence_bwd(x, r, i, lam, y, dy, **rows)
    flat = lambda v, a, b: from_dev(v.reshape(-1, D)[a:b])
    ends = np.cumsum(lens)
    for s in sorted({0, int(np.argmax(lens)), len(lens) // 2, len(lens) - 1}):
        lo, hi = int(ends[s] - lens[s]), int(ends[s])
        a = max(lo, hi - REACH)
        wy, wh = ref.recurrence(*(flat(v, a, hi) for v in (x, r, i)), from_dev(lam), np.zeros((1, D)), [hi - a], 8.0)
        seen = wy[-SEEN:] if a > lo else wy
        close(flat(y, hi - len(seen), hi), seen, io, "y", FORWARD[io])
        close(from_dev(S)[s:s + 1], wh, "f32", "state", FORWARD["f32"])
        b = min(hi, lo + REACH)  # the first tokens' gradients, from those that reach them
        w = ref.recurrence_bwd(*(flat(v, lo, b) for v in (x, r, i)), from_dev(lam), np.zeros((1, D)), flat(y, lo, b), [b - lo], 8.0,
                               flat(dy, lo, b), np.zeros((1, D)))
        n = SEEN if b < hi else b - lo
        for k in ("dx", "dr", "di"):
            close(flat(g[k], lo, lo + n), w[k][:n], io, k, BACKWARD[io])
    return y, S, g


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rest", [[], [5, 0, 700], [1] * 3000])
def test_one_long_row(io, rest):
    """A row that is longer than 2^24 tokens by itself, alone and before others."""
    import torch
    lens = [(1 << 24) + 3000] + rest
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    check(tensors(1, sum(lens), 2, io), np.array(lens), io, offsets=off)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_many_short_rows(io):
    import torch
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 400, 90000)
    assert lens.sum() > 1 << 24
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    t = tensors(2, int(lens.sum()), 2, io)
    y, S, g = check(t, lens, io, offsets=off)
    import selective_scan_segmented_amd as sfm
    y1, S1 = sfm.sfm_gated_recurrence_fwd(*t[:4], offsets=off, max_len=400, return_state=True)
    # (another plan: blocks fall elsewhere, 2^-14 of a state at most as chunks are joined in another order)
    assert torch.allclose(S, S1, rtol=1e-4, atol=1e-4)


def test_equal_rows():
    """One row, not packed: L itself is past 2^24."""
    n = (1 << 24) + 77
    check(tensors(3, n, 2, "bf16"), np.array([n]), "bf16")
