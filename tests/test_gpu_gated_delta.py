"""The gated delta rule on the GPU against the float64 token-by-token definition."""
import numpy as np
import pytest

import delta_reference as ref
from helpers import from_dev

pytestmark = pytest.mark.gpu


def dev(x, io):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16 if io == "bf16" else torch.float32).cuda()


def f32(x):
    return dev(x, "f32")


def call_fwd(x, lens, packed, io, l2norm, h0, scale=None, state=True):
    """x: the float64 inputs; packed or equal rows."""
    import torch
    import selective_scan_segmented_amd as sfm
    q, k, v, g, beta = x[:5]
    lead = (1, len(q)) if packed else (len(lens), lens[0])
    t = [dev(a.reshape(lead + a.shape[1:]), io) for a in (q, k, v, g, beta)]
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda() if packed else None
    got = sfm.sfm_gated_delta_fwd(*t, h0=None if h0 is None else f32(h0), offsets=off,
                                  max_len=max(lens + [1]) if packed else None, scale=scale, l2norm=l2norm,
                                  return_state=state)
    torch.cuda.synchronize()
    o = got[0] if state else got
    return from_dev(o).reshape(v.shape), from_dev(got[1]) if state else None


# rows' lengths (a packed list or equal rows), Hk, H, dk, dv
CASES = [
    ([1], 1, 1, 16, 16), ([1, 1, 1], 2, 4, 64, 64), ([7, 7], 1, 2, 32, 48), ([51, 51], 2, 2, 64, 64),
    ([64, 64], 1, 1, 64, 32), ([65], 1, 3, 128, 128), ([198, 198], 1, 1, 64, 64), ([130], 2, 2, 40, 100),
    ([63, 63], 1, 2, 128, 256), ([300], 1, 1, 128, 16), ([129], 1, 1, 5, 7), ([17], 1, 2, 1, 1),
    ([100], 1, 1, 24, 192), ([257], 1, 1, 96, 80), ([12, 12, 12], 1, 1, 128, 33),
]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("l2norm", [True, False])
@pytest.mark.parametrize("lens,Hk,H,dk,dv", CASES)
def test_forward_equal_rows(lens, Hk, H, dk, dv, io, l2norm):
    x = ref.delta_inputs(len(lens) * 1000 + lens[0], sum(lens), len(lens), Hk, H, dk, dv, l2norm, io)
    h0 = x[5] if lens[0] % 2 else None
    o, hT = call_fwd(x, lens, False, io, l2norm, h0)
    wo, wT = ref.delta(*x[:5], np.zeros(x[5].shape) if h0 is None else h0, np.cumsum(lens), dk ** -0.5, l2norm)
    ref.close(o, wo, io, "o")
    ref.close(hT, wT, "f32", "state")
    o2, _ = call_fwd(x, lens, False, io, l2norm, h0, state=False)
    ref.close(o2, wo, io, "o without the state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[3, 0, 70, 1, 64, 129, 0], [0, 0, 5], [200], [0], [64, 64, 63, 65, 1, 1]])
def test_forward_packed_rows(lens, io):
    Hk, H, dk, dv = 1, 2, 64, 64
    x = ref.delta_inputs(7, sum(lens), len(lens), Hk, H, dk, dv, True, io)
    o, hT = call_fwd(x, lens, True, io, True, x[5], scale=0.3)
    wo, wT = ref.delta(*x[:6], np.cumsum(lens), 0.3, True)
    ref.close(o, wo, io, "o")
    ref.close(hT, wT, "f32", "state")
    for r, n in enumerate(lens):
        if n == 0:
            assert np.array_equal(hT[r], x[5][r])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_forward_decays(io):
    """Resets (minus infinity), decays below float32's range, none at all (0) and gates of 0 and 1."""
    T, H, d = 150, 4, 32
    x = ref.delta_inputs(11, T, 1, 1, H, d, d, True, io)
    q, k, v, g, beta, h0, _ = x
    rng = np.random.default_rng(3)
    g[rng.random((T, H)) < 0.1] = -np.inf
    g[rng.random((T, H)) < 0.1] = 0.0
    g[rng.random((T, H)) < 0.1] = -200.0
    beta[rng.random((T, H)) < 0.2] = 0.0
    beta[rng.random((T, H)) < 0.2] = 1.0
    o, hT = call_fwd(x, [T], False, io, True, h0)
    wo, wT = ref.delta(q, k, v, g, beta, h0, [T], d ** -0.5, True)
    ref.close(o, wo, io, "o")
    ref.close(hT, wT, "f32", "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_forward_alike_keys(io):
    """All keys of a row the same and gates near 1: the chunk's triangular system at its least regular."""
    T, d = 128, 64
    x = ref.delta_inputs(12, T, 1, 1, 1, d, d, True, io)
    x[1][:] = x[1][:1]
    x[3][:] = ref.cast(-1e-3 * np.ones(x[3].shape), io)
    x[4][:] = ref.cast(0.99 * np.ones(x[4].shape), io)
    o, hT = call_fwd(x, [T], False, io, True, None)
    wo, wT = ref.delta(*x[:5], np.zeros(x[5].shape), [T], d ** -0.5, True)
    ref.close(o, wo, io, "o")
    ref.close(hT, wT, "f32", "state")


def test_forward_rows_are_separate():
    """NaN and infinity in one row leave the others' bits alone, also where rows share a chunk's tokens."""
    lens = [40, 40, 90, 3]
    x = ref.delta_inputs(5, sum(lens), 4, 1, 2, 64, 64, True, "bf16")
    clean, cs = call_fwd(x, lens, True, "bf16", True, x[5])
    for a in x[:5]:
        a[45] = np.nan
        a[46] = np.inf
    dirty, ds = call_fwd(x, lens, True, "bf16", True, x[5])
    for lo, hi, r in ((0, 40, 0), (80, 170, 2), (170, 173, 3)):
        assert np.array_equal(clean[lo:hi], dirty[lo:hi])
        assert np.array_equal(cs[r], ds[r])
    assert np.array_equal(clean[40:45], dirty[40:45]) or np.isnan(dirty[40:45]).any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv,pad", [(64, 64, 0), (64, 64, 3), (20, 12, 1), (64, 128, 8)])
def test_forward_strided_projection(io, dk, dv, pad):
    """q, k and v as slices of one projection, rows on odd and on even bounds."""
    import torch
    import selective_scan_segmented_amd as sfm
    B, L, H = 2, 70, 2
    x = ref.delta_inputs(21, B * L, B, H, H, dk, dv, True, io)
    q, k, v, g, beta = x[:5]
    wide = np.concatenate([q.reshape(B, L, -1), k.reshape(B, L, -1), v.reshape(B, L, -1), np.zeros((B, L, pad))], -1)
    w = dev(wide, io)
    n = H * dk
    qd, kd, vd = (s.unflatten(-1, (H, -1)) for s in (w[..., :n], w[..., n:2 * n], w[..., 2 * n:2 * n + H * dv]))
    gd, bd = (dev(a.reshape(B, L, H), io) for a in (g, beta))
    o = sfm.sfm_gated_delta_fwd(qd, kd, vd, gd, bd, l2norm=True)
    same = sfm.sfm_gated_delta_fwd(qd.contiguous(), kd.contiguous(), vd.contiguous(), gd, bd, l2norm=True)
    torch.cuda.synchronize()
    wo, _ = ref.delta(q, k, v, g, beta, np.zeros(x[5].shape), [L, 2 * L], dk ** -0.5, True)
    ref.close(from_dev(o).reshape(wo.shape), wo, io, "o")
    assert torch.equal(o, same)


@pytest.mark.parametrize("L", [3, 200])
def test_forward_state_in_place_and_streams(L):
    """The state may be handed on in its own buffer; another stream; the same bits each time."""
    import torch
    import selective_scan_segmented_amd as sfm
    x = ref.delta_inputs(31, 2 * L, 2, 1, 2, 64, 64, True, "bf16")
    t = [dev(a.reshape((2, L) + a.shape[1:]), "bf16") for a in x[:5]]
    h0 = f32(x[5])
    o, hT = sfm.sfm_gated_delta_fwd(*t, h0=h0, l2norm=True, return_state=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o2, h2 = sfm.sfm_gated_delta_fwd(*t, h0=h0, l2norm=True, return_state=True, state=h0)
    side.synchronize()
    assert h2.data_ptr() == h0.data_ptr()
    assert torch.equal(o, o2) and torch.equal(hT, h0)


def test_forward_two_halves_are_the_whole():
    """A row in two calls, the state handed on, agrees with the row in one."""
    T = 150
    x = ref.delta_inputs(41, T, 1, 2, 2, 64, 64, True, "f32")
    o, hT = call_fwd(x, [T], False, "f32", True, x[5])
    cut = 77
    o1, h1 = call_fwd([a[:cut] for a in x[:5]], [cut], False, "f32", True, x[5])
    o2, h2 = call_fwd([a[cut:] for a in x[:5]], [T - cut], False, "f32", True, h1)
    ref.close(np.concatenate([o1, o2]), o, "f32", "o")
    ref.close(h2, hT, "f32", "state")


def test_offsets_outside_the_tokens_are_cut():
    """Offsets past the tokens or falling are cut to them; nothing outside is read or written."""
    import torch
    import selective_scan_segmented_amd as sfm
    x = ref.delta_inputs(51, 100, 3, 1, 1, 64, 64, True, "f32")
    t = [f32(a[None]) for a in x[:5]]
    off = torch.tensor([0, 60, 20, 400], dtype=torch.int32).cuda()
    o, hT = sfm.sfm_gated_delta_fwd(*t, offsets=off, max_len=100, l2norm=True, return_state=True)
    torch.cuda.synchronize()
    wo, wT = ref.delta(*[a[:60] for a in x[:5]], np.zeros((1,) + x[5].shape[1:]), [60], 64 ** -0.5, True)
    ref.close(from_dev(hT)[:1], wT, "f32", "first row")
    assert torch.equal(hT[1], torch.zeros_like(hT[1]))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R,Hk,H,dk,dv", [(1, 1, 1, 64, 64), (5, 2, 4, 128, 128), (3, 1, 1, 16, 16), (7, 1, 2, 40, 100),
                                          (2, 1, 1, 5, 7), (2, 1, 1, 128, 256), (4, 1, 3, 96, 66)])
def test_step(R, Hk, H, dk, dv, io):
    import torch
    import selective_scan_segmented_amd as sfm
    x = ref.delta_inputs(R * 7 + dk, R, R, Hk, H, dk, dv, True, io)
    pool = R + 3
    rng = np.random.default_rng(2)
    slots = rng.permutation(pool)[:R].astype(np.int32)
    S = (rng.standard_normal((pool, H, dk, dv)) / 4).astype(np.float32)
    t = [dev(a, io) for a in x[:5]]
    Sd = f32(S)
    o = sfm.sfm_gated_delta_step(*t, Sd, slots=torch.from_numpy(slots).cuda(), l2norm=True)
    torch.cuda.synchronize()
    wo, wS = ref.delta(*x[:5], S[slots].astype(np.float64), np.arange(1, R + 1), dk ** -0.5, True)
    ref.close(from_dev(o), wo, io, "o")
    got = from_dev(Sd)
    ref.close(got[slots], wS, "f32", "states")
    rest = np.setdiff1d(np.arange(pool), slots)
    assert np.array_equal(got[rest], S[rest].astype(np.float64))


def test_step_padding_rows_and_no_slots():
    import torch
    import selective_scan_segmented_amd as sfm
    x = ref.delta_inputs(3, 4, 4, 1, 2, 64, 64, True, "bf16")
    t = [dev(a, "bf16") for a in x[:5]]
    S = f32(x[5])
    before = S.clone()
    o = sfm.sfm_gated_delta_step(*t, S, slots=torch.tensor([-1, 2, 4, -7], dtype=torch.int32).cuda(), l2norm=True)
    torch.cuda.synchronize()
    assert (o[0] == 0).all() and (o[2] == 0).all() and (o[3] == 0).all() and (o[1] != 0).any()
    assert torch.equal(S[[0, 1, 3]], before[[0, 1, 3]])
    S = before.clone()
    o = sfm.sfm_gated_delta_step(*t, S, l2norm=True)
    wo, wS = ref.delta(*x[:6], np.arange(1, 5), 64 ** -0.5, True)
    ref.close(from_dev(o), wo, "bf16", "o")
    ref.close(from_dev(S), wS, "f32", "states")


def test_step_continues_the_rows():
    """Whole rows, then token by token, agree with the longer rows."""
    import torch
    import selective_scan_segmented_amd as sfm
    B, T, n = 2, 70, 66
    x = ref.delta_inputs(61, B * T, B, 1, 2, 64, 64, True, "f32")
    t = [f32(a.reshape((B, T) + a.shape[1:])) for a in x[:5]]
    whole, wT = sfm.sfm_gated_delta_fwd(*t, l2norm=True, return_state=True)
    _, S = sfm.sfm_gated_delta_fwd(*[a[:, :n].contiguous() for a in t], l2norm=True, return_state=True)
    for i in range(n, T):
        o = sfm.sfm_gated_delta_step(*[a[:, i].contiguous() for a in t], S, l2norm=True)
        ref.close(from_dev(o), from_dev(whole[:, i]), "f32", f"token {i}")
    torch.cuda.synchronize()
    ref.close(from_dev(S), from_dev(wT), "f32", "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("walk,narrow", [("whole", "0"), ("prepared", "0"), ("prepared", "1")])
@pytest.mark.parametrize("lens,Hk,H,dk,dv", [([200, 0, 64, 1, 130], 1, 2, 64, 64), ([300], 1, 1, 128, 130), ([129, 5], 2, 2, 33, 20)])
def test_forward_by_every_plan(lens, Hk, H, dk, dv, walk, narrow, io, monkeypatch):
    """Each way of walking the chunks, whatever the sizes would choose."""
    monkeypatch.setenv("SFM_DELTA_WALK", walk)
    monkeypatch.setenv("SFM_DELTA_NARROW", narrow)
    x = ref.delta_inputs(sum(lens), sum(lens), len(lens), Hk, H, dk, dv, True, io)
    wo, wT = ref.delta(*x[:6], np.cumsum(lens), dk ** -0.5, True)
    for state in (True, False):
        o, hT = call_fwd(x, lens, True, io, True, x[5], state=state)
        ref.close(o, wo, io, "o")
        if state:
            ref.close(hT, wT, "f32", "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("narrow", ["0", "1"])
def test_forward_many_chunks_of_shared_heads(io, narrow, monkeypatch):
    """Rows times chunks past the card's compute units: one workgroup prepares all value heads of a key head."""
    monkeypatch.setenv("SFM_DELTA_WALK", "prepared")
    monkeypatch.setenv("SFM_DELTA_NARROW", narrow)
    lens, Hk, H, dk, dv = [130] * 44, 2, 6, 24, 16
    x = ref.delta_inputs(31, sum(lens), len(lens), Hk, H, dk, dv, True, io)
    o, hT = call_fwd(x, lens, False, io, True, x[5])
    wo, wT = ref.delta(*x[:6], np.cumsum(lens), dk ** -0.5, True)
    ref.close(o, wo, io, "o")
    ref.close(hT, wT, "f32", "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("walk", ["whole", "prepared"])
def test_forward_mild_and_steep_chunks(io, walk, monkeypatch):
    """Chunks whose decays are products of two exponentials next to one whose are not, and one that grows."""
    monkeypatch.setenv("SFM_DELTA_WALK", walk)
    T, H, d = 256, 2, 64
    x = ref.delta_inputs(13, T, 1, 1, H, d, d, True, io)
    x[3][:] = np.repeat([-0.01, -3.0, -0.7, 0.0625], 64)[:, None]
    x[3][:] = ref.cast(x[3], io)
    o, hT = call_fwd(x, [T], False, io, True, x[5])
    wo, wT = ref.delta(*x[:6], [T], d ** -0.5, True)
    ref.close(o, wo, io, "o")
    ref.close(hT, wT, "f32", "state")
