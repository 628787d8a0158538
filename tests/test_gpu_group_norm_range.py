"""The group norm of values whose squares leave float32's range while their deviations' do not."""
import numpy as np
import pytest

import delta_reference as ref
from helpers import from_dev
from test_gpu_group_norm import dev

pytestmark = pytest.mark.gpu


# N, L, C, G: slabs with and without slots that hold no row, two passes in one range and in several
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N,L,C,G", [(2, 3, 64, 4), (2, 51, 640, 10), (1, 1, 48, 3), (3, 198, 320, 5), (300, 9, 4100, 1),
                                     (1, 3000, 160, 32), (2, 5000, 40, 8)])
def test_large_values(N, L, C, G, io):
    """x = 2^64 (1 or 1 + 2^-7), squares of 2^128 and of deviations 2^112: mean over deviation 256, so the statistics
    keep 2^-24 x 256 of a deviation, 2e-5, and may lose a few times that."""
    import selective_scan_segmented_amd as sfm
    rng = np.random.default_rng(N + L)
    x = 2.0 ** 64 * (1 + 2.0 ** -7 * rng.integers(0, 2, (N, L, C)))
    y, mean, rstd = sfm.sfm_group_norm_fwd(dev(x, io), G)
    wy, wm, wr = ref.group_norm(x, G, 1.0, 0.0, 1e-5, None)
    ref.close(from_dev(mean), wm, "f32", "mean")
    ref.close(from_dev(rstd), wr, "f32", "rstd", (1e-4, 0))
    ref.close(from_dev(y), wy, io, "y", (0, 3e-4) if io == "f32" else (2.0 ** -8, 3e-4))
    dy = ref.cast(rng.standard_normal((N, L, C)), io)
    g = sfm.sfm_group_norm_bwd(dev(dy, io), dev(x, io), mean, rstd)
    dx, _, _ = ref.group_norm_bwd(dy, x, from_dev(mean), from_dev(rstd), np.ones(C), np.zeros(C), None)
    assert np.isfinite(from_dev(g["dx"])).all()
    # dx is of the size of 1 / deviation, 2^-56; its terms' rounding as for y
    ref.close(from_dev(g["dx"]) * 2.0 ** 56, dx * 2.0 ** 56, io, "dx", (2e-5, 3e-4) if io == "f32" else (2.0 ** -8, 3e-4))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 5, 4000])
def test_large_constant_groups(L, io):
    """A constant group has variance 0 whatever its size: y is the bias."""
    import selective_scan_segmented_amd as sfm
    x = np.full((2, L, 32), 2.0 ** 100)
    b = np.arange(32, dtype=np.float64)
    y, mean, rstd = sfm.sfm_group_norm_fwd(dev(x, io), 4, None, dev(b, "f32"))
    assert (from_dev(mean) == 2.0 ** 100).all()
    ref.close(from_dev(rstd), np.full((2, 4), 1e-5 ** -0.5), "f32", "rstd")
    assert np.array_equal(from_dev(y), np.broadcast_to(b, x.shape))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("N,C", [(1, 1), (21, 64), (7, 135), (3, 2560)])
def test_groups_of_one_value(N, C, act, io):
    """y is the bias's, and nothing of dy reaches x or the weight: exact zeros, not their rounding by 1 / sqrt(eps)."""
    import selective_scan_segmented_amd as sfm
    rng = np.random.default_rng(C)
    x, dy = (ref.cast(rng.standard_normal((N, 1, C)), io) for _ in range(2))
    w, b = (rng.uniform(0.5, 1.5, C).astype(np.float32).astype(np.float64) for _ in range(2))
    y, mean, rstd = sfm.sfm_group_norm_fwd(dev(x, io), C, dev(w, "f32"), dev(b, "f32"), act=act)
    g = sfm.sfm_group_norm_bwd(dev(dy, io), dev(x, io), mean, rstd, dev(w, "f32"), dev(b, "f32"), act=act)
    assert np.array_equal(from_dev(mean)[:, None], x)
    wy, _, _ = ref.group_norm(x, C, w, b, 1e-5, act)
    _, _, db = ref.group_norm_bwd(dy, x, x[:, 0], from_dev(rstd), w, b, act)
    ref.close(from_dev(y), wy, io, "y")
    ref.close(from_dev(g["db"]), db, "f32", "db", (2e-5, 1e-4))
    assert (from_dev(g["dx"]) == 0).all() and (from_dev(g["dw"]) == 0).all()
