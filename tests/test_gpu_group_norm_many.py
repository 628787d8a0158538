"""The group norm of more samples than one launch's workgroups hold: parts of the call agree with it bit for bit."""
import numpy as np
import pytest

import delta_reference as ref
from helpers import from_dev

pytestmark = pytest.mark.gpu


def inputs(N, C):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(N + C)
    x = torch.empty((N, 1, C), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = 0.5 + torch.rand(C, generator=gen, device="cuda")
    return x, w, torch.randn(C, generator=gen, device="cuda")


def parts(N):
    cut = [0, N // 3 | 1, N // 2 + 5, N]
    return zip(cut, cut[1:])


def some(N):
    return np.unique(np.r_[0, N // 2, N - 1, np.random.default_rng(1).integers(0, N, 20)])


# tokens normed by themselves.  Two passes: groups too wide for a slab, N x channels / 16 past 2^24; slabs: N workgroups
# of 512 threads at 2^32 work items.
WIDE = [(32768, 8200, 1), (1 << 23, 64, 32)]


@pytest.mark.parametrize("N,C,G", WIDE)
def test_forward(N, C, G):
    import torch
    import selective_scan_segmented_amd as sfm
    x, w, b = inputs(N, C)
    y, mean, rstd = sfm.sfm_group_norm_fwd(x, G, w, b, act="silu")
    for lo, hi in parts(N):
        for a, c in zip((y, mean, rstd), sfm.sfm_group_norm_fwd(x[lo:hi], G, w, b, act="silu")):
            assert torch.equal(a[lo:hi], c)
    at = some(N)
    wy, wm, wr = ref.group_norm(from_dev(x[at]), G, from_dev(w), from_dev(b), 1e-5, True)
    ref.close(from_dev(y[at]), wy, "bf16", "y")
    ref.close(from_dev(mean[at]), wm, "f32", "mean")
    ref.close(from_dev(rstd[at]), wr, "f32", "rstd")


@pytest.mark.parametrize("N,C,G,weights", [(32768, 8192, 1, True), (1 << 23, 64, 32, False)])
def test_backward(N, C, G, weights):
    import torch
    import selective_scan_segmented_amd as sfm
    x, w, b = inputs(N, C)
    dy = torch.flip(x, (0,))
    if not weights:
        w = b = None
    _, mean, rstd = sfm.sfm_group_norm_fwd(x, G, w, b, act="silu")
    got = sfm.sfm_group_norm_bwd(dy, x, mean, rstd, w, b, act="silu")
    dw, db = np.zeros(C), np.zeros(C)
    for lo, hi in parts(N):
        part = sfm.sfm_group_norm_bwd(dy[lo:hi], x[lo:hi], mean[lo:hi], rstd[lo:hi], w, b, act="silu")
        assert torch.equal(got["dx"][lo:hi], part["dx"])
        if weights:
            dw += from_dev(part["dw"])
            db += from_dev(part["db"])
    at = some(N)
    one = np.ones(C), np.zeros(C)
    wd, bd = (from_dev(w), from_dev(b)) if weights else one
    dx, _, _ = ref.group_norm_bwd(from_dev(dy[at]), from_dev(x[at]), from_dev(mean[at]), from_dev(rstd[at]), wd, bd, True)
    ref.close(from_dev(got["dx"][at]), dx, "bf16", "dx")
    if weights:  # sums over N values of either sign, joined in another order
        ref.close(from_dev(got["dw"]), dw, "f32", "dw", (2e-5, 1e-4))
        ref.close(from_dev(got["db"]), db, "f32", "db", (2e-5, 1e-4))
