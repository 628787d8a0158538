"""The gated delta rule's gradients on the GPU against the float64 formula and against differences."""
import numpy as np
import pytest

import delta_reference as ref
from helpers import from_dev
from test_gpu_gated_delta import dev, f32

pytestmark = pytest.mark.gpu

# float32: the forward's products and sums twice over and sums of differences, an order above its bar.  bfloat16:
# one rounding of the result, and 2^-10 of the rms for computed operands of 2^-17 whose products partly cancel.
GRADE = {"f32": (1e-4, 1e-4), "bf16": (2.0 ** -8, 2.0 ** -10)}
# the initial states' gradient is float32 in both (three parts to an operand)
GRADE_H0 = (2e-5, 1e-4)


def call_bwd(x, lens, packed, io, l2norm, h0, dhT, scale=None):
    import torch
    import selective_scan_segmented_amd as sfm
    lead = (1, len(x[0])) if packed else (len(lens), lens[0])
    t = [dev(a.reshape(lead + a.shape[1:]), io) for a in x[:5] + [x[6]]]
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda() if packed else None
    kw = dict(h0=None if h0 is None else f32(h0), dstate=None if dhT is None else f32(dhT), offsets=off,
              max_len=max(lens + [1]) if packed else None, scale=scale, l2norm=l2norm)
    got = sfm.sfm_gated_delta_bwd(*t, **kw)
    again = sfm.sfm_gated_delta_bwd(*t, **kw)
    torch.cuda.synchronize()
    for n in got:
        assert torch.equal(got[n], again[n]), f"{n}: not the same bits"
    return {n: from_dev(a) if n == "dh0" else from_dev(a).reshape((len(x[0]),) + a.shape[2:]) for n, a in got.items()}


def check(got, want, io, h0):
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        ref.close(got[n], want[n], io, n, GRADE[io])
    assert ("dh0" in got) == (h0 is not None)
    if h0 is not None:
        ref.close(got["dh0"], want["dh0"], "f32", "dh0", GRADE_H0)


CASES = [([1], 1, 1, 16, 16), ([1, 1, 1], 2, 4, 64, 64), ([51, 51], 2, 2, 64, 64), ([64, 64], 1, 1, 64, 32),
         ([65], 1, 3, 128, 128), ([198, 198], 1, 1, 64, 64), ([130], 2, 2, 40, 100), ([63, 63], 1, 2, 128, 256),
         ([300], 1, 1, 128, 16), ([129], 1, 1, 5, 7), ([17], 1, 2, 1, 1), ([100], 1, 1, 24, 192), ([257], 1, 4, 96, 80)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("l2norm", [True, False])
@pytest.mark.parametrize("lens,Hk,H,dk,dv", CASES)
def test_equal_rows(lens, Hk, H, dk, dv, io, l2norm):
    x = ref.delta_inputs(len(lens) * 1000 + lens[0], sum(lens), len(lens), Hk, H, dk, dv, l2norm, io)
    h0 = x[5] if lens[0] % 2 else None
    rng = np.random.default_rng(lens[0])
    dhT = rng.standard_normal(x[5].shape).astype(np.float32).astype(np.float64) if lens[0] % 4 == 1 else None
    got = call_bwd(x, lens, False, io, l2norm, h0, dhT)
    zero = np.zeros(x[5].shape)
    want = ref.delta_bwd(*x[:5], zero if h0 is None else h0, np.cumsum(lens), dk ** -0.5, l2norm, x[6], zero if dhT is None else dhT)
    check(got, want, io, h0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[3, 0, 70, 1, 64, 129, 0], [0, 0, 5], [200], [64, 64, 63, 65, 1, 1]])
def test_packed_rows(lens, io):
    x = ref.delta_inputs(7, sum(lens), len(lens), 1, 2, 64, 64, True, io)
    dhT = np.random.default_rng(1).standard_normal(x[5].shape).astype(np.float32).astype(np.float64)
    got = call_bwd(x, lens, True, io, True, x[5], dhT, scale=0.3)
    want = ref.delta_bwd(*x[:6], np.cumsum(lens), 0.3, True, x[6], dhT)
    check(got, want, io, x[5])
    for r, n in enumerate(lens):
        if n == 0:
            assert np.array_equal(got["dh0"][r], dhT[r])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decays(io):
    """Resets, decays below float32's range, none at all, gates of 0 and 1: finite gradients, dg zero at resets
    (to the rounding of the sums that cancel there)."""
    T, H, d = 150, 4, 32
    x = ref.delta_inputs(11, T, 1, 1, H, d, d, True, io)
    rng = np.random.default_rng(3)
    g, beta = x[3], x[4]
    g[rng.random((T, H)) < 0.1] = -np.inf
    g[rng.random((T, H)) < 0.1] = 0.0
    g[rng.random((T, H)) < 0.1] = -200.0
    beta[rng.random((T, H)) < 0.2] = 0.0
    beta[rng.random((T, H)) < 0.2] = 1.0
    got = call_bwd(x, [T], False, io, True, x[5], None)
    want = ref.delta_bwd(*x[:6], [T], d ** -0.5, True, x[6], np.zeros(x[5].shape))
    check(got, want, io, x[5])


def test_rows_are_separate():
    """NaN and infinity in one row leave the others' gradients alone, bit for bit."""
    lens = [40, 40, 90, 3]
    x = ref.delta_inputs(5, sum(lens), 4, 1, 2, 64, 64, True, "bf16")
    clean = call_bwd(x, lens, True, "bf16", True, x[5], None)
    import selective_scan_segmented_amd as sfm
    import torch
    for a in x[:5] + [x[6]]:
        a[45] = np.nan
        a[46] = np.inf
    t = [dev(a[None], "bf16") for a in x[:5] + [x[6]]]
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    dirty = sfm.sfm_gated_delta_bwd(*t, h0=f32(x[5]), offsets=off, max_len=90, l2norm=True)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        d = from_dev(dirty[n])[0]
        for lo, hi in ((0, 40), (80, 170), (170, 173)):
            assert np.array_equal(clean[n][lo:hi], d[lo:hi]), n


def test_against_differences():
    """Directional derivatives against central differences of the float32 forward (step 2^-6 of unit inputs:
    truncation and rounding both below 1e-3 of the derivative along the gradient itself)."""
    import selective_scan_segmented_amd as sfm
    import torch
    T, H, d = 90, 2, 32
    x = ref.delta_inputs(9, T, 1, 1, H, d, d, True, "f32")
    h0, do = x[5], x[6]
    dhT = np.random.default_rng(4).standard_normal(h0.shape).astype(np.float32).astype(np.float64)

    def loss(a):
        o, s = sfm.sfm_gated_delta_fwd(*[f32(b[None]) for b in a[:5]], h0=f32(a[5]), l2norm=True, return_state=True)
        torch.cuda.synchronize()
        return np.sum(from_dev(o)[0] * do) + np.sum(from_dev(s) * dhT)

    got = call_bwd(x, [T], False, "f32", True, h0, dhT)
    rng = np.random.default_rng(5)
    for i, n in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dh0")):
        step = got[n] / np.sqrt(np.mean(got[n] ** 2)) * rng.uniform(0.5, 1.5, got[n].shape)
        h = 2.0 ** -6 * np.sqrt(np.mean(x[i] ** 2)) / np.max(np.abs(step)) * 4
        up, down = ([a.copy() for a in x[:6]] for _ in range(2))
        up[i] += h * step
        down[i] -= h * step
        num, want = (loss(up) - loss(down)) / (2 * h), np.sum(got[n] * step)
        assert abs(num - want) <= 5e-3 * abs(want), (n, num, want)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strided_projection(io):
    """Gradients for q, k and v that are slices of one projection are those of contiguous copies."""
    import torch
    import selective_scan_segmented_amd as sfm
    B, L, H, d = 2, 70, 2, 24
    x = ref.delta_inputs(21, B * L, B, H, H, d, d, True, io)
    wide = dev(np.concatenate([a.reshape(B, L, -1) for a in x[:3]] + [np.zeros((B, L, 3))], -1), io)
    q, k, v = (wide[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
    g, beta, do = (dev(a.reshape((B, L) + a.shape[1:]), io) for a in (x[3], x[4], x[6]))
    a = sfm.sfm_gated_delta_bwd(q, k, v, g, beta, do, l2norm=True)
    b = sfm.sfm_gated_delta_bwd(q.contiguous(), k.contiguous(), v.contiguous(), g, beta, do, l2norm=True)
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("narrow", ["0", "1"])
@pytest.mark.parametrize("lens,Hk,H,dk,dv", [([200, 0, 64, 1, 130], 1, 2, 64, 64), ([300], 1, 1, 128, 130), ([129, 5], 2, 4, 33, 20)])
def test_by_every_plan(lens, Hk, H, dk, dv, narrow, io, monkeypatch):
    """Wide and narrow walks, whatever the sizes would choose."""
    monkeypatch.setenv("SFM_DELTA_NARROW", narrow)
    x = ref.delta_inputs(sum(lens), sum(lens), len(lens), Hk, H, dk, dv, True, io)
    dhT = np.random.default_rng(1).standard_normal(x[5].shape).astype(np.float32).astype(np.float64)
    check(call_bwd(x, lens, True, io, True, x[5], dhT), ref.delta_bwd(*x[:6], np.cumsum(lens), dk ** -0.5, True, x[6], dhT), io, x[5])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("narrow", ["0", "1"])
def test_many_chunks_of_shared_heads(io, narrow, monkeypatch):
    """Rows times chunks past the card's compute units: one workgroup prepares all value heads of a key head."""
    monkeypatch.setenv("SFM_DELTA_NARROW", narrow)
    lens, Hk, H, dk, dv = [130] * 44, 2, 6, 24, 16
    x = ref.delta_inputs(31, sum(lens), len(lens), Hk, H, dk, dv, True, io)
    got = call_bwd(x, lens, False, io, True, x[5], None)
    want = ref.delta_bwd(*x[:6], np.cumsum(lens), dk ** -0.5, True, x[6], np.zeros(x[5].shape))
    check(got, want, io, x[5])
