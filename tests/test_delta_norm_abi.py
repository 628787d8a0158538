"""The gated delta rule's and the group norm's entry points refuse what they cannot run (host only)."""
import ctypes
import os

import numpy as np
import pytest

import delta_reference as ref
import selective_scan_segmented_amd as sfm

OK, NULL, SHAPE, DTYPE, UNSUP, HIP, ALIAS, ALIGN = range(8)
P = 0x1000000  # fake, never dereferenced: every call below fails its checks


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sfm.library_path()):
        from selective_scan_segmented_amd import build
        build.build(verbose=False)
    return sfm.load_library()


def fwd(lib, **kw):
    a = dict(q=P, k=2 * P, v=3 * P, g=4 * P, beta=5 * P, h0=None, o=6 * P, hT=None, off=None, rows=2, L=100, tokens=200,
             Hk=1, H=2, dk=64, dv=64, ldq=64, ldk=64, ldv=128, scale=0.125, io=1, flags=1, ws=100 * P, wsb=1 << 30)
    a.update(kw)
    return lib.sfm_gated_delta_fwd(*a.values(), None)


def step(lib, **kw):
    a = dict(q=P, k=2 * P, v=3 * P, g=4 * P, beta=5 * P, state=6 * P, slots=None, o=9 * P, rows=2, pool=4, Hk=1, H=2,
             dk=64, dv=64, ldq=64, ldk=64, ldv=128, scale=0.125, io=1, flags=1)
    a.update(kw)
    return lib.sfm_gated_delta_step(*a.values(), None)


SHARED = [(dict(q=None), NULL), (dict(beta=None), NULL), (dict(o=None), NULL), (dict(io=2), DTYPE), (dict(flags=2), SHAPE),
          (dict(Hk=0), SHAPE), (dict(Hk=3), SHAPE), (dict(dk=0), SHAPE), (dict(dk=129), SHAPE), (dict(dv=257), SHAPE),
          (dict(ldq=63), SHAPE), (dict(ldv=127), SHAPE), (dict(rows=0), SHAPE), (dict(q=P + 1), ALIGN),
          (dict(o=9 * P + 1), ALIGN), (dict(o=P), ALIAS), (dict(o=4 * P), ALIAS)]


@pytest.mark.parametrize("kw,want", SHARED + [(dict(tokens=199), SHAPE), (dict(L=0), SHAPE), (dict(tokens=-1, off=7 * P), SHAPE),
                                              (dict(hT=P), ALIAS), (dict(hT=8 * P, h0=8 * P + 64), ALIAS), (dict(hT=6 * P), ALIAS),
                                              (dict(h0=7 * P + 2), ALIGN), (dict(o=7 * P, h0=7 * P), ALIAS)])
def test_forward_refuses(lib, kw, want):
    assert fwd(lib, **kw) == want
    assert lib.sfm_last_error().startswith(b"sfm_gated_delta_fwd")


@pytest.mark.parametrize("kw,want", SHARED + [(dict(state=None), NULL), (dict(pool=0), SHAPE), (dict(pool=1), SHAPE),
                                              (dict(state=P), ALIAS), (dict(o=6 * P), ALIAS), (dict(slots=6 * P), ALIAS),
                                              (dict(state=6 * P + 2), ALIGN)])
def test_step_refuses(lib, kw, want):
    assert step(lib, **kw) == want


def bwd(lib, **kw):
    a = dict(q=P, k=2 * P, v=3 * P, g=4 * P, beta=5 * P, h0=None, dout=6 * P, dhT=None, dq=7 * P, dk_=8 * P, dv_=9 * P, dg=10 * P,
             dbeta=11 * P, dh0=None, off=None, rows=2, L=100, tokens=200, Hk=1, H=2, dk=64, dv=64, ldq=64, ldk=64, ldv=128, scale=0.125,
             io=1, flags=1, ws=100 * P, wsb=1 << 30)
    a.update(kw)
    return lib.sfm_gated_delta_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,want", [c for c in SHARED if "o" not in c[0]] + [
    (dict(dout=None), NULL), (dict(dg=None), NULL), (dict(ws=None), SHAPE), (dict(wsb=4096), SHAPE), (dict(ws=100 * P + 8), ALIGN),
    (dict(dq=P), ALIAS), (dict(dk_=7 * P + 64), ALIAS), (dict(dh0=6 * P), ALIAS), (dict(ws=10 * P), ALIAS), (dict(dg=10 * P + 1), ALIGN),
    (dict(tokens=100), SHAPE), (dict(dhT=12 * P + 2), ALIGN), (dict(rows=1 << 20, L=1 << 20, off=12 * P), SHAPE)])
def test_backward_refuses(lib, kw, want):
    assert bwd(lib, **kw) == want
    assert lib.sfm_last_error().startswith(b"sfm_gated_delta_bwd")


def test_workspace_sizes(lib):
    out = ctypes.c_int64(-1)
    f = lib.sfm_gated_delta_fwd_ws_size
    assert f(2, 100, 200, 2, 64, 64, 0, 1, ctypes.byref(out)) == OK and out.value >= 0
    assert f(2, 100, 200, 2, 64, 64, 0, 1, None) == NULL
    assert f(2, 100, 200, 2, 0, 64, 0, 1, ctypes.byref(out)) == SHAPE
    assert f(2, 100, 200, 2, 64, 64, 0, 9, ctypes.byref(out)) == DTYPE
    f = lib.sfm_gated_delta_bwd_ws_size
    assert f(2, 100, 200, 1, 2, 64, 64, 0, 1, None) == NULL
    assert f(2, 100, 200, 3, 2, 64, 64, 0, 1, ctypes.byref(out)) == SHAPE
    assert f(2, 100, 200, 1, 2, 64, 64, 0, 1, ctypes.byref(out)) == OK and out.value > 0
    f = lib.sfm_group_norm_fwd_ws_size
    assert f(2, 100, 64, 4, 1, None) == NULL
    assert f(2, 100, 64, 5, 1, ctypes.byref(out)) == SHAPE
    assert f(2, 100, 64, 4, 3, ctypes.byref(out)) == DTYPE
    assert f(2, 100, 64, 4, 1, ctypes.byref(out)) == OK and out.value == 0
    assert f(1, 100000, 64, 4, 1, ctypes.byref(out)) == OK and out.value > 0
    assert lib.sfm_group_norm_bwd_ws_size(2, 100, 64, 4, 0, 1, ctypes.byref(out)) == OK and out.value == 0
    assert lib.sfm_group_norm_bwd_ws_size(2, 100, 64, 4, 1, 1, ctypes.byref(out)) == OK and out.value > 0


def test_launch_plans(lib, monkeypatch):
    """Few long rows have their triangular inverses made beforehand (workspace); one chunk or many rows do not."""
    f = sfm.sfm_gated_delta_fwd_ws_size
    unit = lambda parts: 8 * 64 * 4 + 6 * 64 * 8 * 2 * (parts + 2)  # row scalars, two lower triangles of 6 fragments
    assert f(2, 8192, 16384, 16, 128, 128, True) == (16384 // 64 + 2) * 16 * unit(3)
    assert f(2, 8192, 16384, 16, 128, 128, False) == (16384 // 64 + 2) * 16 * unit(2)
    assert f(256, 51, 256 * 51, 10, 64, 64) == 0
    assert f(512, 198, 512 * 198, 8, 64, 64) == 0
    monkeypatch.setenv("SFM_DELTA_WALK", "whole")
    assert f(2, 8192, 16384, 16, 128, 128, True) == 0



@pytest.mark.parametrize("rows,L,H,dk,dv,beforehand", [
    (16, 1024, 16, 64, 64, True), (24, 1024, 16, 64, 64, False), (16, 1024, 16, 64, 128, True),
    (24, 1024, 16, 64, 128, False), (24, 1024, 16, 64, 32, True), (32, 1024, 16, 64, 32, False),
    (8, 128, 16, 64, 64, True), (16, 128, 16, 64, 64, False), (1, 64, 1, 64, 64, False)])
def test_inverses_beforehand_by_filled_workgroups(lib, rows, L, H, dk, dv, beforehand):
    """A workspace is asked for exactly where the chunks' triangular inverses are made beforehand."""
    assert (sfm.sfm_gated_delta_fwd_ws_size(rows, L, rows * L, H, dk, dv) > 0) == beforehand


def test_ragged_rows_count_by_their_tokens(lib):
    """Packed rows fill the card by their tokens, not by the longest row's."""
    assert sfm.sfm_gated_delta_fwd_ws_size(32, 2048, 32 * 2048, 16, 64, 64) == 0
    assert sfm.sfm_gated_delta_fwd_ws_size(32, 2048, 32 * 700, 16, 64, 64) > 0

def norm(lib, **kw):
    a = dict(x=P, w=2 * P, b=3 * P, y=4 * P, mean=5 * P, rstd=6 * P, N=2, L=100, C=64, G=4, eps=1e-5, act=1, io=1, ws=None, wsb=0)
    a.update(kw)
    return lib.sfm_group_norm_fwd(*a.values(), None)


def norm_bwd(lib, **kw):
    a = dict(dy=P, x=2 * P, mean=3 * P, rstd=4 * P, w=5 * P, b=6 * P, dx=7 * P, dw=8 * P, db=9 * P, N=2, L=100, C=64, G=4, act=1,
             io=1, ws=10 * P, wsb=1 << 20)
    a.update(kw)
    return lib.sfm_group_norm_bwd(*a.values(), None)


NORM = [(dict(x=None), NULL), (dict(mean=None), NULL), (dict(io=4), DTYPE), (dict(G=5), SHAPE), (dict(G=0), SHAPE),
        (dict(L=0), SHAPE), (dict(act=2), SHAPE), (dict(x=2 * P + 1), ALIGN)]


@pytest.mark.parametrize("kw,want", NORM + [(dict(y=None), NULL), (dict(y=P), ALIAS), (dict(mean=2 * P), ALIAS), (dict(eps=-1.0), SHAPE),
                                            (dict(L=100000), SHAPE), (dict(rstd=5 * P), ALIAS), (dict(w=2 * P + 2), ALIGN)])
def test_norm_refuses(lib, kw, want):
    assert norm(lib, **kw) == want


@pytest.mark.parametrize("kw,want", NORM + [(dict(dx=None), NULL), (dict(dx=P), ALIAS), (dict(dw=9 * P), ALIAS), (dict(ws=None), SHAPE),
                                            (dict(wsb=16), SHAPE), (dict(ws=10 * P + 4), ALIGN), (dict(ws=8 * P), ALIAS)])
def test_norm_backward_refuses(lib, kw, want):
    assert norm_bwd(lib, **kw) == want


@pytest.mark.parametrize("l2norm", [True, False])
def test_reference_gradient_against_differences(l2norm):
    """The float64 backward the GPU tests use, against central differences of the definition."""
    lens = [5, 0, 3]
    x = ref.delta_inputs(1, 8, 3, 1, 2, 3, 4, l2norm, "f32")
    q, k, v, g, beta, h0, do = x
    rng = np.random.default_rng(2)
    dhT = rng.standard_normal(h0.shape)
    ends = np.cumsum(lens)

    def loss(*a):
        o, hT = ref.delta(*a, ends, 0.7, l2norm)
        return np.sum(o * do) + np.sum(hT * dhT)

    got = ref.delta_bwd(q, k, v, g, beta, h0, ends, 0.7, l2norm, do, dhT)
    args = [q, k, v, g, beta, h0]
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dh0")):
        num = np.zeros(args[i].size)
        for j in range(args[i].size):
            up, down = ([a.copy() for a in args] for _ in range(2))
            up[i].reshape(-1)[j] += 1e-5
            down[i].reshape(-1)[j] -= 1e-5
            num[j] = (loss(*up) - loss(*down)) / 2e-5
        assert np.allclose(num.reshape(args[i].shape), got[name], rtol=1e-6, atol=1e-7), name


def test_reference_norm_gradient_against_differences():
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((2, 3, 6)), rng.standard_normal((2, 3, 6))
    w, b = rng.uniform(0.5, 1.5, 6), rng.standard_normal(6)
    _, mean, rstd = ref.group_norm(x, 2, w, b, 1e-5, True)
    got = ref.group_norm_bwd(dy, x, mean, rstd, w, b, True)
    args = [x, w, b]
    for i in range(3):
        num = np.zeros(args[i].size)
        for j in range(args[i].size):
            up, down = ([a.copy() for a in args] for _ in range(2))
            up[i].reshape(-1)[j] += 1e-5
            down[i].reshape(-1)[j] -= 1e-5
            f = lambda a: np.sum(dy * ref.group_norm(a[0], 2, a[1], a[2], 1e-5, True)[0])
            num[j] = (f(up) - f(down)) / 2e-5
        assert np.allclose(num.reshape(args[i].shape), got[i], rtol=1e-6, atol=1e-7)
