"""The gated delta rule's calls in the forms that a user's program gives them, against the float64 definition."""
import numpy as np
import pytest

import delta_reference as ref
from helpers import from_dev
from test_gpu_gated_delta import dev, f32
from test_gpu_gated_delta_bwd import GRADE_H0

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradient_of_states_that_were_zero(io):
    """dh0 into a tensor of the caller's without h0: that of states of zeros; one that does not fit is refused."""
    import torch
    import selective_scan_segmented_amd as sfm
    lens, H, dk, dv = [70, 70], 2, 64, 48
    x = ref.delta_inputs(17, sum(lens), 2, 1, H, dk, dv, True, io)
    t = [dev(a.reshape((2, 70) + a.shape[1:]), io) for a in x[:5] + [x[6]]]
    dh0 = torch.full((2, H, dk, dv), float("nan"), device="cuda")
    got = sfm.sfm_gated_delta_bwd(*t, l2norm=True, grads={"dh0": dh0})
    torch.cuda.synchronize()
    assert got["dh0"] is dh0
    zero = np.zeros(x[5].shape)
    want = ref.delta_bwd(*x[:5], zero, np.cumsum(lens), dk ** -0.5, True, x[6], zero)
    ref.close(from_dev(dh0), want["dh0"], "f32", "dh0", GRADE_H0)
    with pytest.raises(ValueError, match="dh0"):
        sfm.sfm_gated_delta_bwd(*t, l2norm=True, grads={"dh0": dh0[:1].contiguous()})
    with pytest.raises(TypeError, match="dh0"):
        sfm.sfm_gated_delta_bwd(*t, l2norm=True, grads={"dh0": dh0.bfloat16()})


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_one_token_of_each_row_of_a_projection(io):
    """q, k and v as one token of every row of a longer projection: the bits of contiguous copies."""
    import torch
    import selective_scan_segmented_amd as sfm
    R, T, H, d = 3, 5, 2, 64
    x = ref.delta_inputs(23, R * T, R, H, H, d, d, True, io)
    wide = dev(np.concatenate([a.reshape(R, T, -1) for a in x[:3]], -1), io)
    q, k, v = (wide[:, 2:3, i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
    g, beta, do = (dev(a.reshape((R, T) + a.shape[1:])[:, 2:3], io) for a in (x[3], x[4], x[6]))
    h0 = f32(x[5])
    o, s = sfm.sfm_gated_delta_fwd(q, k, v, g, beta, h0=h0, l2norm=True, return_state=True)
    got = sfm.sfm_gated_delta_bwd(q, k, v, g, beta, do, h0=h0, l2norm=True)
    own = [a.contiguous() for a in (q, k, v)]
    o2, s2 = sfm.sfm_gated_delta_fwd(*own, g, beta, h0=h0, l2norm=True, return_state=True)
    want = sfm.sfm_gated_delta_bwd(*own, g, beta, do, h0=h0, l2norm=True)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, s2)
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("max_len", [None, 0, 5])
def test_packed_rows_that_are_all_empty(io, max_len):
    """A batch without a token: the states pass through, forward and back."""
    import torch
    import selective_scan_segmented_amd as sfm
    R, H, dk, dv = 3, 2, 64, 48
    x = ref.delta_inputs(29, 1, R, 1, H, dk, dv, True, io)
    t = [dev(a[None, :0], io) for a in x[:5] + [x[6]]]
    h0, off = f32(x[5]), torch.zeros(R + 1, dtype=torch.int32, device="cuda")
    o, s = sfm.sfm_gated_delta_fwd(*t[:5], h0=h0, offsets=off, max_len=max_len, return_state=True)
    _, z = sfm.sfm_gated_delta_fwd(*t[:5], offsets=off, max_len=max_len, return_state=True)
    got = sfm.sfm_gated_delta_bwd(*t, h0=h0, dstate=h0 + 1, offsets=off, max_len=max_len)
    torch.cuda.synchronize()
    assert o.shape == t[2].shape and torch.equal(s, h0) and torch.equal(z, torch.zeros_like(h0))
    assert torch.equal(got["dh0"], h0 + 1) and got["dq"].numel() == 0


@pytest.mark.parametrize("L", [3, 40, 150])
def test_a_state_given_is_written(L):
    """The states go to the caller's tensor whether or not they are asked for as a result."""
    import torch
    import selective_scan_segmented_amd as sfm
    x = ref.delta_inputs(37, 2 * L, 2, 1, 2, 64, 64, True, "bf16")
    t = [dev(a.reshape((2, L) + a.shape[1:]), "bf16") for a in x[:5]]
    h0 = f32(x[5])
    o, want = sfm.sfm_gated_delta_fwd(*t, h0=h0, l2norm=True, return_state=True)
    o2 = sfm.sfm_gated_delta_fwd(*t, h0=h0, l2norm=True, state=h0)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(h0, want)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("walk,narrow", [("whole", "0"), ("prepared", "0"), ("prepared", "1")])
@pytest.mark.parametrize("L", [1, 3, 12, 51, 64])
def test_rows_of_one_chunk_by_every_plan(L, walk, narrow, io, monkeypatch):
    """The overrides, with rows that no plan prepares."""
    from test_gpu_gated_delta import call_fwd
    monkeypatch.setenv("SFM_DELTA_WALK", walk)
    monkeypatch.setenv("SFM_DELTA_NARROW", narrow)
    lens = [L, L]
    x = ref.delta_inputs(L, sum(lens), 2, 1, 2, 64, 48, True, io)
    wo, wT = ref.delta(*x[:6], np.cumsum(lens), 64 ** -0.5, True)
    for state in (True, False):
        o, hT = call_fwd(x, lens, False, io, True, x[5], state=state)
        ref.close(o, wo, io, "o")
        if state:
            ref.close(hT, wT, "f32", "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (8, 192), (128, 33)])
@pytest.mark.parametrize("dhT", [False, True])
def test_decay_of_rows_of_one_token(dhT, dk, dv, io):
    """A token that begins its row without a state has nothing to decay: its dg is zero, not the rounding of sums that
    cancel."""
    import torch
    import selective_scan_segmented_amd as sfm
    R, H = 40, 3
    x = ref.delta_inputs(dk + dv, R, R, 1, H, dk, dv, True, io)
    t = [dev(a[:, None], io) for a in x[:5] + [x[6]]]
    got = sfm.sfm_gated_delta_bwd(*t, dstate=f32(x[5]) if dhT else None, l2norm=True)
    torch.cuda.synchronize()
    assert (got["dg"] == 0).all()
    assert (got["dbeta"] != 0).any()
