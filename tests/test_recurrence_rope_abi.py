"""The gated linear recurrence's and the norm and rotation's entry points refuse what they cannot run, and their
float64 references' gradients against differences (host only)."""
import ctypes
import os

import numpy as np
import pytest

import recurrence_reference as ref
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
    a = dict(x=P, r=2 * P, i=3 * P, lam=4 * P, h0=None, y=5 * P, hT=None, off=None, rows=2, L=1000, tokens=2000, D=64, ldx=64, ldr=64,
             ldi=64, c=8.0, io=1, ws=100 * P, wsb=1 << 30)
    a.update(kw)
    return lib.sfm_gated_recurrence_fwd(*a.values(), None)


def bwd(lib, **kw):
    a = dict(x=P, r=2 * P, i=3 * P, lam=4 * P, h0=None, y=5 * P, dy=6 * P, dhT=None, dx=7 * P, dr=8 * P, di=9 * P, dlam=10 * P,
             dh0=None, off=None, rows=2, L=1000, tokens=2000, D=64, ldx=64, ldr=64, ldi=64, c=8.0, io=1, ws=100 * P, wsb=1 << 30)
    a.update(kw)
    return lib.sfm_gated_recurrence_bwd(*a.values(), None)


def step(lib, **kw):
    a = dict(x=P, r=2 * P, i=3 * P, lam=4 * P, state=6 * P, slots=None, y=5 * P, rows=2, pool=4, D=64, ldx=64, ldr=64, ldi=64, c=8.0,
             io=1)
    a.update(kw)
    return lib.sfm_gated_recurrence_step(*a.values(), None)


SHARED = [(dict(x=None), NULL), (dict(i=None), NULL), (dict(lam=None), NULL), (dict(y=None), NULL), (dict(io=2), DTYPE),
          (dict(D=0), SHAPE), (dict(D=65537, ldx=65537, ldr=65537, ldi=65537), SHAPE), (dict(ldx=63), SHAPE), (dict(ldi=(1 << 36) + 1), SHAPE),
          (dict(rows=0), SHAPE), (dict(c=0.0), SHAPE), (dict(c=-8.0), SHAPE), (dict(c=float("nan")), SHAPE), (dict(c=float("inf")), SHAPE),
          (dict(x=P + 1), ALIGN), (dict(lam=4 * P + 2), ALIGN), (dict(y=5 * P + 1), ALIGN)]
ROWS = [(dict(tokens=1999), SHAPE), (dict(ldr=(1 << 31) // 2000 + 1), SHAPE), (dict(L=0), SHAPE), (dict(tokens=-1, off=7 * P), SHAPE), (dict(off=7 * P + 2), ALIGN),
        (dict(h0=11 * P + 2), ALIGN), (dict(rows=1 << 24, L=1, tokens=1 << 24), SHAPE)]


@pytest.mark.parametrize("kw,want", SHARED + ROWS + [
    (dict(y=P), ALIAS), (dict(y=4 * P), ALIAS), (dict(hT=P), ALIAS), (dict(hT=5 * P), ALIAS), (dict(hT=8 * P, h0=8 * P + 64), ALIAS),
    (dict(hT=8 * P + 2), ALIGN), (dict(y=7 * P, h0=7 * P), ALIAS), (dict(y=7 * P, off=7 * P), ALIAS)])
def test_forward_refuses(lib, kw, want):
    assert fwd(lib, **kw) == want
    assert lib.sfm_last_error().startswith(b"sfm_gated_recurrence_fwd")


@pytest.mark.parametrize("kw,want", SHARED + ROWS + [
    (dict(dy=None), NULL), (dict(dlam=None), NULL), (dict(dr=None), NULL), (dict(ws=None), SHAPE), (dict(wsb=16), SHAPE),
    (dict(ws=100 * P + 8), ALIGN), (dict(dx=P), ALIAS), (dict(dr=7 * P + 64), ALIAS), (dict(dx=5 * P), ALIAS), (dict(dlam=4 * P), ALIAS),
    (dict(dh0=6 * P), ALIAS), (dict(dh0=11 * P, dhT=11 * P), ALIAS), (dict(ws=10 * P), ALIAS), (dict(di=9 * P + 1), ALIGN),
    (dict(dhT=12 * P + 2), ALIGN)])
def test_backward_refuses(lib, kw, want):
    assert bwd(lib, **kw) == want
    assert lib.sfm_last_error().startswith(b"sfm_gated_recurrence_bwd")


@pytest.mark.parametrize("kw,want", SHARED + [(dict(state=None), NULL), (dict(pool=0), SHAPE), (dict(pool=1), SHAPE), (dict(state=P), ALIAS),
                                              (dict(y=6 * P), ALIAS), (dict(slots=6 * P), ALIAS), (dict(slots=7 * P + 2), ALIGN),
                                              (dict(state=6 * P + 2), ALIGN)])
def test_step_refuses(lib, kw, want):
    assert step(lib, **kw) == want
    assert lib.sfm_last_error().startswith(b"sfm_gated_recurrence_step")


def sections(*n):
    return (ctypes.c_int64 * len(n))(*n)


def rope(lib, **kw):
    a = dict(q=P, k=2 * P, wq=3 * P, wk=4 * P, pos=5 * P, freqs=6 * P, qo=7 * P, ko=8 * P, tokens=100, period=50, Hq=4, Hk=2, d=64, rot=64,
             axes=1, sections=None, ldq=256, ldk=128, eps=1e-6, io=1, flags=1)
    a.update(kw)
    return lib.sfm_qk_norm_rope_fwd(*a.values(), None)


def rope_bwd(lib, **kw):
    a = dict(dqo=9 * P, dko=10 * P, q=P, k=2 * P, wq=3 * P, wk=4 * P, pos=5 * P, freqs=6 * P, dq=7 * P, dk=8 * P, dwq=11 * P, dwk=12 * P,
             tokens=100, period=50, Hq=4, Hk=2, d=64, rot=64, axes=1, sections=None, ldq=256, ldk=128, eps=1e-6, io=1, flags=1,
             ws=100 * P, wsb=1 << 30)
    a.update(kw)
    return lib.sfm_qk_norm_rope_bwd(*a.values(), None)


ROPE = [(dict(q=None), NULL), (dict(k=None), NULL), (dict(pos=None), NULL), (dict(freqs=None), NULL), (dict(io=3), DTYPE),
        (dict(flags=4), SHAPE), (dict(flags=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(period=3), SHAPE), (dict(period=0), SHAPE),
        (dict(Hq=0), SHAPE), (dict(Hk=0), SHAPE), (dict(d=257, ldq=2000, ldk=2000), SHAPE), (dict(rot=63), SHAPE), (dict(rot=66), SHAPE),
        (dict(rot=-2), SHAPE), (dict(axes=0), SHAPE), (dict(axes=5), SHAPE), (dict(axes=2), SHAPE), (dict(axes=2, sections=sections(16, 15)), SHAPE),
        (dict(axes=2, sections=sections(33, -1)), SHAPE), (dict(ldq=255), SHAPE), (dict(ldk=(1 << 29) + 1), SHAPE), (dict(eps=0.0), SHAPE),
        (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(q=P + 1), ALIGN), (dict(wk=4 * P + 2), ALIGN),
        (dict(pos=5 * P + 2), ALIGN)]


@pytest.mark.parametrize("kw,want", ROPE + [(dict(qo=None), NULL), (dict(qo=P), ALIAS), (dict(ko=7 * P + 64), ALIAS), (dict(ko=5 * P), ALIAS),
                                            (dict(qo=7 * P + 1), ALIGN)])
def test_rope_refuses(lib, kw, want):
    assert rope(lib, **kw) == want
    assert lib.sfm_last_error().startswith(b"sfm_qk_norm_rope_fwd")


@pytest.mark.parametrize("kw,want", ROPE + [
    (dict(dqo=None), NULL), (dict(dk=None), NULL), (dict(dq=P), ALIAS), (dict(dq=9 * P), ALIAS), (dict(dwq=12 * P), ALIAS),
    (dict(ws=None), SHAPE), (dict(wsb=16), SHAPE), (dict(ws=100 * P + 8), ALIGN), (dict(ws=11 * P), ALIAS), (dict(dwk=12 * P + 2), ALIGN),
    (dict(dk=8 * P + 1), ALIGN), (dict(flags=0, wq=None, wk=None), SHAPE)])
def test_rope_backward_refuses(lib, kw, want):
    assert rope_bwd(lib, **kw) == want
    assert lib.sfm_last_error().startswith(b"sfm_qk_norm_rope_bwd")


def test_workspace_sizes(lib):
    out = ctypes.c_int64(-1)
    for f in (lib.sfm_gated_recurrence_fwd_ws_size, lib.sfm_gated_recurrence_bwd_ws_size):
        assert f(2, 100, 200, 64, 1, None) == NULL
        assert f(2, 100, 200, 0, 1, ctypes.byref(out)) == SHAPE
        assert f(2, 100, 200, 64, 2, ctypes.byref(out)) == DTYPE
        assert f(2, 100, 200, 64, 1, ctypes.byref(out)) == OK and out.value >= 0
        # workgroups of 512 lanes (rows nearly as long as the longest): a launch holds 2^32 lanes
        L, tokens = (256, (1 << 31) - 1) if f is lib.sfm_gated_recurrence_fwd_ws_size else (128, 1 << 30)
        assert f((1 << 23) - 8, L, tokens, 32, 0, ctypes.byref(out)) == OK
        assert f((1 << 23) + 8, L, tokens, 32, 0, ctypes.byref(out)) == SHAPE
    f = lib.sfm_qk_norm_rope_bwd_ws_size
    assert f(100, 4, 2, 64, 1, 1, None) == NULL
    assert f(100, 4, 2, 257, 1, 1, ctypes.byref(out)) == SHAPE
    assert f(100, 4, 2, 64, 1, 2, ctypes.byref(out)) == DTYPE
    assert f(100, 4, 2, 64, 0, 1, ctypes.byref(out)) == OK and out.value == 0
    assert f(100, 4, 2, 64, 1, 1, ctypes.byref(out)) == OK and out.value > 0


def differences(loss, args, i, step=1e-5):
    num = np.zeros(args[i].size)
    for j in range(args[i].size):
        up, down = ([a.copy() for a in args] for _ in range(2))
        up[i].reshape(-1)[j] += step
        down[i].reshape(-1)[j] -= step
        num[j] = (loss(*up) - loss(*down)) / (2 * step)
    return num.reshape(args[i].shape)


def test_reference_recurrence_gradient_against_differences():
    ends = np.cumsum([5, 0, 3])
    x, r, i, lam, h0, dy, dhT = ref.recurrence_inputs(1, 8, 3, 4, "f32")
    y, _ = ref.recurrence(x, r, i, lam, h0, ends, 8.0)
    got = ref.recurrence_bwd(x, r, i, lam, h0, y, ends, 8.0, dy, dhT)

    def loss(*a):
        y, hT = ref.recurrence(*a, ends, 8.0)
        return np.sum(y * dy) + np.sum(hT * dhT)

    for n, name in enumerate(("dx", "dr", "di", "dlam", "dh0")):
        assert np.allclose(differences(loss, [x, r, i, lam, h0], n), got[name], rtol=1e-6, atol=1e-8), name


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_reference_rope_gradient_against_differences(neighbours, norm):
    rng = np.random.default_rng(2)
    x, dy, w = rng.standard_normal((3, 2, 9)), rng.standard_normal((3, 2, 9)), rng.uniform(0.5, 1.5, 9)
    form = (ref.angles(rng.integers(0, 100, (3, 2)), rng.uniform(0, 1, 3), [1, 2]), 6, neighbours, norm, 1e-3)
    dx, dw, _ = ref.rope_bwd(x, w, *form, dy)
    loss = lambda x, w: np.sum(dy * ref.rope(x, w, *form))
    assert np.allclose(differences(loss, [x, w], 0), dx, rtol=1e-6, atol=1e-8)
    if norm:
        assert np.allclose(differences(loss, [x, w], 1), dw, rtol=1e-6, atol=1e-8)
