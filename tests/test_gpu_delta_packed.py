"""Packed rows of the gated delta rule: many of them, and calls that leave the longest row's bound out."""
import numpy as np
import pytest

import delta_reference as ref
from helpers import from_dev
from test_gpu_gated_delta import dev, f32
from test_gpu_gated_delta_bwd import GRADE, GRADE_H0

pytestmark = pytest.mark.gpu

# rows of every length next to one another: empty ones in runs, whole chunks, chunk ends, one long row
RAGGED = [0, 0, 1, 64, 63, 65, 0, 128, 127, 129, 300, 2, 0, 0, 0, 191, 5, 64, 64, 0]


def packed(lens, H, Hk, dk, dv, io, seed):
    import torch
    x = ref.delta_inputs(seed, sum(lens), len(lens), Hk, H, dk, dv, True, io)
    t = [dev(a[None], io) for a in x[:5] + [x[6]]]
    return x, t, torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Hk,H,dk,dv", [(2, 2, 64, 64), (1, 3, 128, 100)])
@pytest.mark.parametrize("rows", [20, 64, 65, 130])
def test_without_a_bound(rows, Hk, H, dk, dv, io):
    """max_len left out: forward and gradients of ragged rows, past 64 of them where they are found in two steps."""
    import torch
    import selective_scan_segmented_amd as sfm
    lens = (RAGGED * 7)[:rows]
    x, t, off = packed(lens, H, Hk, dk, dv, io, rows)
    h0 = f32(x[5])
    o, s = sfm.sfm_gated_delta_fwd(*t[:5], h0=h0, offsets=off, l2norm=True, return_state=True)
    got = sfm.sfm_gated_delta_bwd(*t, h0=h0, offsets=off, l2norm=True)
    torch.cuda.synchronize()
    ends = np.cumsum(lens)
    wo, ws = ref.delta(*x[:6], ends, dk ** -0.5, True)
    ref.close(from_dev(o)[0], wo, io, "o")
    ref.close(from_dev(s), ws, "f32", "state")
    want = ref.delta_bwd(*x[:6], ends, dk ** -0.5, True, x[6], np.zeros(x[5].shape))
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        ref.close(from_dev(got[n])[0], want[n], io, n, GRADE[io])
    ref.close(from_dev(got["dh0"]), want["dh0"], "f32", "dh0", GRADE_H0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_thousands_of_rows(io):
    """Rows found in three steps: more than 4096, most of them empty or of a token."""
    import torch
    import selective_scan_segmented_amd as sfm
    rng = np.random.default_rng(3)
    lens = [int(n) for n in np.where(rng.random(5000) < 0.5, 0, 1)]
    lens[0], lens[1700], lens[4099], lens[4999] = 70, 130, 65, 140
    x, t, off = packed(lens, 1, 1, 16, 16, io, 7)
    o, s = sfm.sfm_gated_delta_fwd(*t[:5], h0=f32(x[5]), offsets=off, l2norm=True, return_state=True)
    got = sfm.sfm_gated_delta_bwd(*t, h0=f32(x[5]), offsets=off, l2norm=True)
    torch.cuda.synchronize()
    ends = np.cumsum(lens)
    wo, ws = ref.delta(*x[:6], ends, 0.25, True)
    ref.close(from_dev(o)[0], wo, io, "o")
    ref.close(from_dev(s), ws, "f32", "state")
    want = ref.delta_bwd(*x[:6], ends, 0.25, True, x[6], np.zeros(x[5].shape))
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        ref.close(from_dev(got[n])[0], want[n], io, n, GRADE[io])


@pytest.mark.parametrize("Hk", [16, 32])
def test_a_loose_bound_launches(Hk, monkeypatch):
    """1024 rows of 65536 tokens: rows x the bound's chunks x heads is 2^24 workgroups, rows' own chunks are 2^15."""
    import torch
    import selective_scan_segmented_amd as sfm
    monkeypatch.setenv("SFM_DELTA_WALK", "prepared")  # (one way of walking, so that both bounds give the same bits)
    monkeypatch.setenv("SFM_DELTA_NARROW", "1")
    gen = torch.Generator(device="cuda").manual_seed(2)
    tokens, rows, H, d = 65536, 1024, 32, 16
    r = lambda h: torch.randn((1, tokens, h, d), generator=gen, device="cuda").bfloat16()
    q, k, v, do = r(Hk), r(Hk), r(H), r(H)
    g = -torch.rand((1, tokens, H), generator=gen, device="cuda").bfloat16()
    beta = torch.rand((1, tokens, H), generator=gen, device="cuda").bfloat16()
    off = torch.arange(0, tokens + 1, 64, dtype=torch.int32, device="cuda")
    off[1:-1] += torch.randint(-30, 30, (rows - 1,), generator=gen, device="cuda").int()
    most = int((off[1:] - off[:-1]).max())
    kw = dict(offsets=off, l2norm=True)
    o, s = sfm.sfm_gated_delta_fwd(q, k, v, g, beta, return_state=True, **kw)
    o2, s2 = sfm.sfm_gated_delta_fwd(q, k, v, g, beta, return_state=True, max_len=most, **kw)
    got = sfm.sfm_gated_delta_bwd(q, k, v, g, beta, do, **kw)
    want = sfm.sfm_gated_delta_bwd(q, k, v, g, beta, do, max_len=most, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, s2)
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("walk", ["whole", "prepared"])
def test_tokens_of_no_row_keep_what_was_there(walk, monkeypatch):
    """Tokens before the first row, behind the last and past a row's bound: outputs and gradients keep their old values."""
    import torch
    import selective_scan_segmented_amd as sfm
    monkeypatch.setenv("SFM_DELTA_WALK", walk)
    H, d, T = 2, 64, 400
    x = ref.delta_inputs(19, T, 3, 1, H, d, d, True, "f32")
    t = [f32(a[None]) for a in x[:5] + [x[6]]]
    off = torch.tensor([70, 170, 170, 330], dtype=torch.int32, device="cuda")  # 100, 0 and 160 tokens, at most 150 of them
    full = lambda a: torch.full_like(a, 7.0)
    o = full(t[2])
    g = {"dq": full(t[0]), "dk": full(t[1]), "dv": full(t[2]), "dg": full(t[3]), "dbeta": full(t[4])}
    sfm.sfm_gated_delta_fwd(*t[:5], offsets=off, max_len=150, l2norm=True, o=o)
    sfm.sfm_gated_delta_bwd(*t, offsets=off, max_len=150, l2norm=True, grads=g)
    torch.cuda.synchronize()
    mine = np.r_[70:170, 170:320]
    rest = np.setdiff1d(np.arange(T), mine)
    own = [a[mine] for a in x[:5]]
    zero = np.zeros(x[5].shape)
    wo, _ = ref.delta(*own, zero, [100, 100, 250], d ** -0.5, True)
    want = ref.delta_bwd(*own, zero, [100, 100, 250], d ** -0.5, True, x[6][mine], zero)
    ref.close(from_dev(o)[0][mine], wo, "f32", "o")
    assert (from_dev(o)[0][rest] == 7).all()
    for n in g:
        ref.close(from_dev(g[n])[0][mine], want[n], "f32", n, GRADE["f32"])
        assert (from_dev(g[n])[0][rest] == 7).all(), n
