"""The channel-last group norm on the GPU against float64 numpy."""
import numpy as np
import pytest

import delta_reference as ref
from helpers import from_dev

pytestmark = pytest.mark.gpu


def dev(x, io):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16 if io == "bf16" else torch.float32).cuda()


def inputs(seed, N, L, C, io):
    rng = np.random.default_rng(seed)
    x = ref.cast(rng.standard_normal((N, L, C)) * rng.uniform(0.3, 2, C) + rng.standard_normal(C), io)
    dy = ref.cast(rng.standard_normal((N, L, C)), io)
    w, b = (a.astype(np.float32).astype(np.float64) for a in (rng.uniform(0.5, 1.5, C), 0.3 * rng.standard_normal(C)))
    return x, dy, w, b


# N, L, C, G: one token, odd widths, groups across units, whole slabs, two passes (long rows), many channels
CASES = [(1, 1, 8, 1), (3, 1, 64, 4), (2, 5, 6, 3), (2, 51, 640, 10), (3, 198, 320, 5), (1, 7, 135, 5), (2, 33, 160, 32),
         (1, 1000, 96, 1), (1, 3000, 160, 32), (2, 5000, 40, 8), (1, 2100, 27, 9), (1, 90, 2560, 32), (1, 40, 4100, 1),
         (5, 2, 12, 12), (1, 9001, 24, 3)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("N,L,C,G", CASES)
def test_forward_and_backward(N, L, C, G, act, io):
    import torch
    import selective_scan_segmented_amd as sfm
    x, dy, w, b = inputs(N + L + C, N, L, C, io)
    xd, dyd, wd, bd = dev(x, io), dev(dy, io), dev(w, "f32"), dev(b, "f32")
    y, mean, rstd = sfm.sfm_group_norm_fwd(xd, G, wd, bd, act=act)
    g = sfm.sfm_group_norm_bwd(dyd, xd, mean, rstd, wd, bd, act=act)
    again = sfm.sfm_group_norm_bwd(dyd, xd, mean, rstd, wd, bd, act=act)
    torch.cuda.synchronize()
    wy, wm, wr = ref.group_norm(x, G, w, b, 1e-5, act)
    # y: its group's values lie within a few standard deviations, so errors scale with the rms of z
    ref.close(from_dev(y), wy, io, "y")
    ref.close(from_dev(mean), wm, "f32", "mean")
    ref.close(from_dev(rstd), wr, "f32", "rstd")
    dx, dw, db = ref.group_norm_bwd(dy, x, from_dev(mean), from_dev(rstd), w, b, act)
    ref.close(from_dev(g["dx"]), dx, io, "dx")
    ref.close(from_dev(g["dw"]), dw, "f32", "dw", (2e-5, 1e-4))  # sums over N L values of either sign
    ref.close(from_dev(g["db"]), db, "f32", "db", (2e-5, 1e-4))
    for k in g:
        assert torch.equal(g[k], again[k]), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [20, 4000])
def test_without_weights_and_shapes(L, io):
    import torch
    import selective_scan_segmented_amd as sfm
    x, dy, _, _ = inputs(5, 2, L, 64, io)
    xd = dev(x, io).view(2, L // 10, 10, 64)
    y, mean, rstd = sfm.sfm_group_norm_fwd(xd, 4)
    g = sfm.sfm_group_norm_bwd(dev(dy, io).view(xd.shape), xd, mean, rstd)
    assert sorted(g) == ["dx"] and y.shape == xd.shape
    wy, _, _ = ref.group_norm(x, 4, 1.0, 0.0, 1e-5, None)
    dx, _, _ = ref.group_norm_bwd(dy, x, from_dev(mean), from_dev(rstd), np.ones(64), np.zeros(64), None)
    ref.close(from_dev(y).reshape(wy.shape), wy, io, "y")
    ref.close(from_dev(g["dx"]).reshape(dx.shape), dx, io, "dx")


@pytest.mark.parametrize("L", [60, 6000])
def test_mean_far_from_zero(L):
    """A mean 1000 standard deviations off: the input itself keeps 2^-24 x 1000 of a deviation, 6e-5, and the
    statistics must not lose more than a few times that."""
    import selective_scan_segmented_amd as sfm
    rng = np.random.default_rng(1)
    x = ref.cast(rng.standard_normal((2, L, 32)) + 1000.0, "f32")
    y, mean, rstd = sfm.sfm_group_norm_fwd(dev(x, "f32"), 4)
    wy, wm, wr = ref.group_norm(x, 4, 1.0, 0.0, 1e-5, None)
    ref.close(from_dev(rstd), wr, "f32", "rstd", (1e-4, 0))
    ref.close(from_dev(y), wy, "f32", "y", (0, 3e-4))


def test_constant_groups_and_large_values():
    """A constant group has variance 0 (y = bias); an infinity stays in its own group."""
    import selective_scan_segmented_amd as sfm
    rng = np.random.default_rng(4)
    x = ref.cast(rng.standard_normal((2, 30, 16)), "f32")
    x[0, :, :4] = 3.0
    x[1, 5, 9] = np.inf
    b = np.arange(16, dtype=np.float64)
    y, _, _ = sfm.sfm_group_norm_fwd(dev(x, "f32"), 4, None, dev(b, "f32"))
    y = from_dev(y)
    assert np.array_equal(y[0, :, :4], np.broadcast_to(b[:4], (30, 4)))
    assert np.isfinite(y[1][:, :8]).all() and np.isfinite(y[1][:, 12:]).all() and np.isnan(y[1][:, 8:12]).any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("off", [1, 3])
def test_unaligned_tensors(io, off):
    """Tensors that start off 16 bytes take the one-channel path and agree with the definition."""
    import torch
    import selective_scan_segmented_amd as sfm
    x, dy, w, b = inputs(8, 2, 50, 64, io)
    base = torch.zeros(x.size + off, dtype=dev(x, io).dtype, device="cuda")
    xd = base[off:].view(2, 50, 64)
    xd.copy_(dev(x, io))
    y, mean, rstd = sfm.sfm_group_norm_fwd(xd, 8, dev(w, "f32"), dev(b, "f32"), act="silu")
    wy, _, _ = ref.group_norm(x, 8, w, b, 1e-5, True)
    ref.close(from_dev(y), wy, io, "y")
    g = sfm.sfm_group_norm_bwd(dev(dy, io), xd, mean, rstd, dev(w, "f32"), dev(b, "f32"), act="silu")
    dx, _, _ = ref.group_norm_bwd(dy, x, from_dev(mean), from_dev(rstd), w, b, True)
    ref.close(from_dev(g["dx"]), dx, io, "dx")


def test_gradient_against_differences():
    """The gradient along random directions against central differences of the forward (float32, step 2^-7:
    truncation h^2 and rounding 2^-24 / h, both near 1e-4 of the directional derivative)."""
    import selective_scan_segmented_amd as sfm
    x, dy, w, b = inputs(9, 2, 40, 32, "f32")
    f = lambda x, w, b: np.sum(dy * from_dev(sfm.sfm_group_norm_fwd(dev(x, "f32"), 4, dev(w, "f32"), dev(b, "f32"), act="silu")[0]))
    _, mean, rstd = sfm.sfm_group_norm_fwd(dev(x, "f32"), 4, dev(w, "f32"), dev(b, "f32"), act="silu")
    g = sfm.sfm_group_norm_bwd(dev(dy, "f32"), dev(x, "f32"), mean, rstd, dev(w, "f32"), dev(b, "f32"), act="silu")
    rng, h = np.random.default_rng(6), 2.0 ** -7
    for name, i in (("dx", 0), ("dw", 1), ("db", 2)):
        a = [x, w, b]
        got = from_dev(g[name])
        d = np.sign(got) * rng.uniform(0.5, 1.0, got.shape)  # along the gradient: nothing cancels
        up, down = list(a), list(a)
        up[i], down[i] = a[i] + h * d, a[i] - h * d
        num = (f(*up) - f(*down)) / (2 * h)
        assert abs(num - np.sum(got * d)) <= 2e-3 * abs(num), name


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N,L,C,G", [(4, 3, 96, 32), (2, 40, 120, 40), (3, 6, 64, 64)])
def test_many_groups_to_a_slab(N, L, C, G, io):
    """More narrow groups to a workgroup than its rows need waves: they are joined by waves added for it."""
    import torch
    import selective_scan_segmented_amd as sfm
    x, dy, w, b = inputs(N + L + C, N, L, C, io)
    xd, dyd, wd, bd = dev(x, io), dev(dy, io), dev(w, "f32"), dev(b, "f32")
    y, mean, rstd = sfm.sfm_group_norm_fwd(xd, G, wd, bd, act="silu")
    g = sfm.sfm_group_norm_bwd(dyd, xd, mean, rstd, wd, bd, act="silu")
    torch.cuda.synchronize()
    wy, wm, wr = ref.group_norm(x, G, w, b, 1e-5, "silu")
    ref.close(from_dev(y), wy, io, "y")
    ref.close(from_dev(mean), wm, "f32", "mean")
    ref.close(from_dev(rstd), wr, "f32", "rstd")
    dx, dw, db = ref.group_norm_bwd(dy, x, from_dev(mean), from_dev(rstd), w, b, "silu")
    ref.close(from_dev(g["dx"]), dx, io, "dx")
    ref.close(from_dev(g["dw"]), dw, "f32", "dw", (2e-5, 1e-4))
    ref.close(from_dev(g["db"]), db, "f32", "db", (2e-5, 1e-4))
