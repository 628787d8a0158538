"""Where a NaN or an infinity of the gated delta rule's inputs may reach, by every way of walking the chunks: no other
row, and no earlier chunk of 64 tokens of its own.  Bit for bit against the clean call."""
import numpy as np
import pytest

import delta_reference as ref
from helpers import from_dev
from test_gpu_gated_delta import dev, f32

pytestmark = pytest.mark.gpu

LENS = [40, 210, 64, 130]  # the second row's second chunk is poisoned
BAD = 40 + 70


def inputs(io, H, dk, dv):
    import torch
    x = ref.delta_inputs(5, sum(LENS), len(LENS), 1, H, dk, dv, True, io)
    off = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int32).cuda()
    return x, off


def poisoned(x, which):
    y = [a.copy() for a in x]
    for i in which:
        y[i][BAD] = np.nan
        y[i][BAD + 1] = np.inf
    return y


def plan(monkeypatch, walk, narrow):
    monkeypatch.setenv("SFM_DELTA_WALK", walk)
    monkeypatch.setenv("SFM_DELTA_NARROW", narrow)


PLANS = [("whole", "0"), ("prepared", "0"), ("prepared", "1")]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("walk,narrow", PLANS)
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 40)])
@pytest.mark.parametrize("which", [[0], [1], [2], [3], [4], [0, 1, 2, 3, 4]])
@pytest.mark.parametrize("state", [True, False])
def test_forward(which, dk, dv, walk, narrow, io, state, monkeypatch):
    import torch
    import selective_scan_segmented_amd as sfm
    plan(monkeypatch, walk, narrow)
    x, off = inputs(io, 2, dk, dv)
    h0 = f32(x[5])

    def run(x):
        got = sfm.sfm_gated_delta_fwd(*[dev(a[None], io) for a in x[:5]], h0=h0, offsets=off, max_len=max(LENS), l2norm=True,
                                      return_state=state)
        torch.cuda.synchronize()
        return (from_dev(got[0])[0], from_dev(got[1])) if state else (from_dev(got)[0], None)

    (o, s), (o2, s2) = run(x), run(poisoned(x, which))
    assert not np.isfinite(o2[BAD:BAD + 2]).all()
    for lo, hi in ((0, 40), (40, 40 + 64), (250, 444)):
        assert np.array_equal(o[lo:hi], o2[lo:hi]), (lo, hi)
    if state:
        assert np.array_equal(s[[0, 2, 3]], s2[[0, 2, 3]])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("narrow", ["0", "1"])
@pytest.mark.parametrize("which", [[0], [1], [2], [3], [4], [6], [0, 1, 2, 3, 4, 6]])
def test_backward(which, narrow, io, monkeypatch):
    """The other rows' gradients, those of their initial states among them; of shared key heads too."""
    import torch
    import selective_scan_segmented_amd as sfm
    plan(monkeypatch, "prepared", narrow)
    x, off = inputs(io, 2, 64, 64)
    h0 = f32(x[5])

    def run(x):
        got = sfm.sfm_gated_delta_bwd(*[dev(a[None], io) for a in x[:5] + [x[6]]], h0=h0, dstate=h0, offsets=off,
                                      max_len=max(LENS), l2norm=True)
        torch.cuda.synchronize()
        return {n: from_dev(a) if n == "dh0" else from_dev(a)[0] for n, a in got.items()}

    clean, dirty = run(x), run(poisoned(x, which))
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        for lo, hi in ((0, 40), (250, 444)):
            assert np.array_equal(clean[n][lo:hi], dirty[n][lo:hi]), (n, lo, hi)
    assert np.array_equal(clean["dh0"][[0, 2, 3]], dirty["dh0"][[0, 2, 3]])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_poisoned_request_leaves_the_others(io):
    """The step: a request's NaN stays in its own state and output."""
    import torch
    import selective_scan_segmented_amd as sfm
    R, H, d = 5, 2, 64
    x = ref.delta_inputs(8, R, R, 1, H, d, d, True, io)
    S, S2 = f32(x[5]), f32(x[5])
    o = sfm.sfm_gated_delta_step(*[dev(a, io) for a in x[:5]], S, l2norm=True)
    y = [a.copy() for a in x]
    for a in y[:5]:
        a[2] = np.nan
    S2[2] = float("inf")
    o2 = sfm.sfm_gated_delta_step(*[dev(a, io) for a in y[:5]], S2, l2norm=True)
    torch.cuda.synchronize()
    rest = [0, 1, 3, 4]
    assert torch.equal(o[rest], o2[rest]) and torch.equal(S[rest], S2[rest])
    assert not torch.isfinite(o2[2].float()).any()
