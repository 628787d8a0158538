"""What the recurrence's and the rotation's binding checks before it calls the library (host only, stand-ins for GPU
tensors)."""
import types

import pytest
import torch

import selective_scan_segmented_amd as sfm
from test_delta_binding import Stub as Plain
from test_delta_binding import calls  # noqa: F401  (a fixture)

SIDE = types.SimpleNamespace(cuda_stream=0, device_index=0)
F32, I32 = torch.float32, torch.int32


class Stub(Plain):
    gpu = 0

    def get_device(self):
        return self.gpu


@pytest.fixture(autouse=True)
def here(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)


B, L, D = 2, 100, 64


def args(lead=(B, L)):
    return [Stub(*lead, D), Stub(*lead, D), Stub(*lead, D), Stub(D, dtype=F32)]


def fwd(t, **kw):
    lead = t[0].shape[:-1]
    return sfm.sfm_gated_recurrence_fwd(*t, **{"y": Stub(*lead, D), "workspace": Stub(1 << 20, dtype=torch.uint8), "stream": SIDE, **kw})


def bwd(t, **kw):
    lead = t[0].shape[:-1]
    g = {"dx": Stub(*lead, D), "dr": Stub(*lead, D), "di": Stub(*lead, D), "dlam": Stub(D, dtype=F32)}
    g.update(kw.pop("grads", {}))
    return sfm.sfm_gated_recurrence_bwd(*t, kw.pop("y", Stub(*lead, D)), kw.pop("dy", Stub(*lead, D)), grads=g,
                                        workspace=Stub(1 << 20, dtype=torch.uint8), stream=SIDE, **kw)


@pytest.mark.parametrize("lead", [(), (B,), (B, L, 3)])
def test_rows_take_three_dimensions(calls, lead):  # noqa: F811
    for f in (fwd, bwd):
        with pytest.raises(ValueError, match=r"\[B, L, D\]"):
            f(args(lead))
    assert not calls


@pytest.mark.parametrize("n,bad", [(0, Stub(B, L, D, dtype=torch.float16)), (1, Stub(B, L, D, dtype=F32)), (2, Stub(B, L, D + 1)),
                                   (3, Stub(D)), (3, Stub(D + 1, dtype=F32)), (1, Stub(B, L, D, stride=(L * D, D, 2))),
                                   (0, Stub(B, L, D, stride=(0, 0, 1))), (2, Stub(B, L, D, stride=(7 * D, D, 1)))])
def test_inputs_of_other_forms_are_refused(calls, n, bad):  # noqa: F811
    t = args()
    t[n] = bad
    for f in (fwd, bwd):
        with pytest.raises((TypeError, ValueError)):
            f(t)
    assert not any(name in ("sfm_gated_recurrence_fwd", "sfm_gated_recurrence_bwd") for name, _ in calls)


@pytest.mark.parametrize("kw", [dict(h0=Stub(B, D)), dict(h0=Stub(1, D, dtype=F32)), dict(dstate=Stub(B, D)), dict(y=Stub(B, L, D, dtype=F32)),
                                dict(dy=Stub(B, L, D, stride=(2 * L * D, 2 * D, 1))), dict(grads={"dlam": Stub(D)}),
                                dict(grads={"dh0": Stub(B, D)}), dict(grads={"dx": Stub(B, L, 2 * D)})])
def test_gradients_of_other_forms_are_refused(calls, kw):  # noqa: F811
    with pytest.raises((TypeError, ValueError)):
        bwd(args(), **kw)
    assert not any(name == "sfm_gated_recurrence_bwd" for name, _ in calls)


def test_packed_rows_are_one_batch_entry(calls):  # noqa: F811
    with pytest.raises(ValueError, match="one batch entry"):
        fwd(args(), offsets=Stub(3, dtype=I32))
    with pytest.raises(ValueError, match="offsets"):
        fwd(args((1, L)), offsets=Stub(1, dtype=I32))
    fwd(args((1, L)), offsets=Stub(4, dtype=I32), max_len=40, state=(s := Stub(3, D, dtype=F32)))
    name, a = calls[-1]
    assert name == "sfm_gated_recurrence_fwd" and a[6] == s.at and a[8:12] == (3, 40, L, D)


def test_slices_of_a_projection_are_taken_in_place(calls):  # noqa: F811
    t = args()
    t[:3] = [Stub(B, L, D, stride=(3 * L * D, 3 * D, 1)) for _ in range(3)]
    fwd(t)
    name, a = calls[-1]
    assert name == "sfm_gated_recurrence_fwd" and a[12:15] == (3 * D,) * 3
    t[:3] = [Stub(B, 1, D, stride=(5000, 7, 1)) for _ in range(3)]
    fwd(t)
    assert calls[-1][1][12:15] == (5000,) * 3
    t[:3] = [Stub(1, 1, D, stride=(1 << 40, 7, 1)) for _ in range(3)]  # one token in all: its strides say nothing
    fwd(t)
    assert calls[-1][1][12:15] == (D,) * 3


def test_a_step_takes_two_dimensions(calls):  # noqa: F811
    with pytest.raises(ValueError, match=r"\[R, D\]"):
        sfm.sfm_gated_recurrence_step(*args(), Stub(4, D, dtype=F32), y=Stub(B, L, D), stream=SIDE)
    for state in (Stub(4, D + 1, dtype=F32), Stub(4, 1, D, dtype=F32), Stub(4, D)):
        with pytest.raises((TypeError, ValueError)):
            sfm.sfm_gated_recurrence_step(*args((3,)), state, y=Stub(3, D), stream=SIDE)
    with pytest.raises((TypeError, ValueError)):
        sfm.sfm_gated_recurrence_step(*args((3,)), Stub(4, D, dtype=F32), slots=Stub(2, dtype=I32), y=Stub(3, D), stream=SIDE)
    assert not calls


def test_tensors_of_another_gpu_are_refused(calls):  # noqa: F811
    """The kernels are launched on the current one."""
    t = args()
    t[1] = Stub(B, L, D)
    t[1].gpu = 1
    for f in (fwd, bwd):
        with pytest.raises(ValueError, match="GPU 1"):
            f(t)
    with pytest.raises(ValueError, match="stream is of GPU 1"):
        fwd(args(), stream=types.SimpleNamespace(cuda_stream=0, device_index=1))
    q, k = heads()
    k.gpu = 1
    with pytest.raises(ValueError, match="GPU 1"):
        rope(q, k)
    assert not any(not name.endswith("_ws_size") for name, _ in calls)


H, HK, S = 4, 2, 32


def heads(lead=(B, L)):
    return Stub(*lead, H, S), Stub(*lead, HK, S)


def rope(q, k, **kw):
    return sfm.sfm_qk_norm_rope_fwd(q, k, **{"qo": Stub(*q.shape), "ko": Stub(*k.shape), "stream": SIDE, **kw})


ROT = dict(freqs=Stub(16, dtype=F32))


@pytest.mark.parametrize("kw", [dict(positions=Stub(B, L, dtype=I32)), dict(ROT), dict(ROT, positions=Stub(B, L + 1, dtype=I32)),
                                dict(ROT, positions=Stub(B, L, dtype=torch.int64)), dict(ROT, positions=Stub(B, L, 2, dtype=I32)),
                                dict(ROT, positions=Stub(B, L, dtype=I32), sections=(8, 8)), dict(sections=(8, 8)),
                                dict(freqs=Stub(4, 4, dtype=F32), positions=Stub(L, dtype=I32)), dict(wq=Stub(S)), dict(wk=Stub(S + 1, dtype=F32)),
                                dict(qo=Stub(B, L, H, S, stride=(9 * L * H * S, H * S, S, 1)))])
def test_rotations_of_other_forms_are_refused(calls, kw):  # noqa: F811
    with pytest.raises((TypeError, ValueError)):
        rope(*heads(), **kw)
    assert not calls


@pytest.mark.parametrize("lead,shape,sections,want", [
    ((B, L), (B, L), None, (B * L, B * L, 1)), ((B, L), (L,), None, (B * L, L, 1)), ((B, L), (L, 2), (6, 10), (B * L, L, 2)),
    ((B, L), (B, L, 2), (6, 10), (B * L, B * L, 2)), ((7,), (7,), None, (7, 7, 1)), ((7,), (7, 3), (4, 4, 8), (7, 7, 3)),
    ((B, L), (B, L, 1), (16,), (B * L, B * L, 1)), ((1, L), (L,), None, (L, L, 1))])
def test_positions(calls, lead, shape, sections, want):  # noqa: F811
    rope(*heads(lead), positions=Stub(*shape, dtype=I32), sections=sections, **ROT)
    name, a = calls[-1]
    assert name == "sfm_qk_norm_rope_fwd" and (a[8], a[9], a[14]) == want and a[13] == 32
    assert a[15] is None if want[2] == 1 else list(a[15]) == list(sections)


def test_norm_alone(calls):  # noqa: F811
    rope(*heads(), wq=Stub(S, dtype=F32))
    name, a = calls[-1]
    assert a[13] == 0 and a[20] == sfm.SFM_QK_NORM and a[4] is None
    rope(*heads(), norm=False, interleaved=True, positions=Stub(L, dtype=I32), **ROT)
    assert calls[-1][1][20] == sfm.SFM_QK_NEIGHBOURS
