"""The norm and rotation of queries and keys on the GPU against their definition in float64."""
import numpy as np
import pytest

import recurrence_reference as ref
from delta_reference import cast, close
from helpers import from_dev

pytestmark = pytest.mark.gpu

# float32: the mean square, the root and the products 2^-24 each, sine and cosine some 3 2^-24 of one: 2e-6 of the value
# and its like.  bfloat16: the rounding's half step, and 2e-5 of the rms for what is below it.
FORWARD = {"f32": (2e-6, 2e-6), "bf16": (2.0 ** -8, 2e-5)}
# the gradient is a difference of two such, and sums over a head
BACKWARD = {"f32": (1e-5, 1e-5), "bf16": (2.0 ** -8, 1e-4)}
EPS = 1e-6


def dev(a, io):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(torch.bfloat16 if io == "bf16" else torch.float32)


def inputs(seed, lead, Hq, Hk, d, rot, io, sections=None, far=0, shared=False, weights=True):
    rng = np.random.default_rng(seed)
    tokens = int(np.prod(lead))
    q, k, dq, dk = (cast(rng.standard_normal((tokens, h, d)) * rng.uniform(0.3, 2.0, d) + 0.3, io) for h in (Hq, Hk, Hq, Hk))
    f32 = lambda v: np.asarray(v).astype(np.float32).astype(np.float64)
    wq, wk = (f32(rng.uniform(0.5, 1.5, d)) if weights else np.ones(d) for _ in range(2))
    freqs = f32(10000.0 ** (-np.arange(rot // 2) * 2 / max(2, rot)))
    sections = [rot // 2] if sections is None else sections
    n = lead[-1] if shared else tokens
    pos = rng.integers(-5 if not far else far - 1000, 300 if not far else far, (n, len(sections))).astype(np.int32)
    return q, k, dq, dk, wq, wk, freqs, sections, pos


def run(lead, Hq, Hk, d, rot, io, seed=0, sections=None, far=0, shared=False, weights=True, norm=True, neighbours=False, slices=False):
    import torch
    import selective_scan_segmented_amd as sfm
    weights = weights and norm
    q, k, dq, dk, wq, wk, freqs, sec, pos = inputs(seed, lead, Hq, Hk, d, rot, io, sections, far, shared, weights)
    tokens = len(q)
    tq, tk = dev(q, io).view(*lead, Hq, d), dev(k, io).view(*lead, Hk, d)
    if slices:
        p = torch.cat([tq.flatten(-2), tk.flatten(-2), tk.flatten(-2)], -1)
        tq, tk = p[..., :Hq * d].unflatten(-1, (Hq, d)), p[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    form = dict(interleaved=neighbours, norm=norm, eps=EPS)
    if weights:
        form.update(wq=dev(wq, "f32"), wk=dev(wk, "f32"))
    if rot:
        lead_p = (lead[-1],) if shared else lead
        at = torch.from_numpy(pos).cuda().view(*lead_p, len(sec))
        form.update(freqs=dev(freqs, "f32"), positions=at if sections else at.squeeze(-1), sections=sections)
    full = np.tile(pos, (tokens // len(pos), 1)) if len(pos) else np.zeros((0, len(sec)), int)
    ang = ref.angles(full, freqs, sec)
    qo, ko = sfm.sfm_qk_norm_rope_fwd(tq, tk, **form)
    for got, x, w, n in ((qo, q, wq, "qo"), (ko, k, wk, "ko")):
        assert got.is_contiguous() and got.shape == tuple(lead) + x.shape[1:]
        close(from_dev(got).reshape(x.shape), ref.rope(x, w, ang, rot, neighbours, norm, EPS), io, n, FORWARD[io])
    g = sfm.sfm_qk_norm_rope_bwd(dev(dq, io).view(*lead, Hq, d), dev(dk, io).view(*lead, Hk, d), tq, tk, **form)
    assert sorted(g) == sorted(["dq", "dk"] + ["dwq", "dwk"] * weights)
    for n, x, w, dy in (("q", q, wq, dq), ("k", k, wk, dk)):
        dx, dw, size = ref.rope_bwd(x, w, ang, rot, neighbours, norm, EPS, dy)
        close(from_dev(g["d" + n]).reshape(x.shape), dx, io, "d" + n, BACKWARD[io])
        if weights:  # float32 sums of terms each off by some 5e-7 of their like
            assert (np.abs(from_dev(g["dw" + n]) - dw) <= 1e-5 * size + 1e-30).all(), "dw" + n
    again = sfm.sfm_qk_norm_rope_bwd(dev(dq, io).view(*lead, Hq, d), dev(dk, io).view(*lead, Hk, d), tq, tk, **form)
    for n in g:
        assert torch.equal(g[n], again[n]), n


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [1, 2, 3, 5, 8, 16, 24, 32, 40, 64, 80, 96, 100, 128, 130, 160, 192, 255, 256])
def test_head_sizes(d, io, neighbours):
    run((2, 9), 3, 1, d, d // 2 * 2, io, seed=d, neighbours=neighbours)


@pytest.mark.parametrize("slices", [False, True])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,rot", [(64, 32), (64, 0), (64, 2), (128, 96), (96, 48), (33, 16), (256, 64), (48, 46), (40, 8), (128, 16), (256, 250)])
def test_part_of_a_head(d, rot, io, neighbours, slices):
    run((3, 5), 4, 2, d, rot, io, seed=rot, neighbours=neighbours, slices=slices)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 5), (8, 2), (7, 3), (32, 1), (16, 8), (64, 64)])
def test_heads(Hq, Hk, io):
    run((2, 11), Hq, Hk, 64, 64, io, seed=Hq)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lead", [(1,), (3,), (257,), (1, 1), (1, 300), (40, 1), (0,), (2, 0), (5, 198)])
def test_tokens(lead, io):
    run(lead, 4, 2, 64, 64, io, seed=len(lead))


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("sections", [(16, 16), (8, 12, 12), (0, 32), (32, 0), (1, 2, 3, 26)])
def test_position_axes(sections, neighbours, shared):
    run((3, 50), 5, 5, 64, 64, "f32", sections=sections, neighbours=neighbours, shared=shared)
    run((3, 50), 5, 5, 128, 64, "bf16", sections=sections, neighbours=neighbours, shared=shared)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("far", [1 << 14, 1 << 20, (1 << 31) - 1])
def test_far_positions(far, io):
    run((2, 20), 2, 1, 64, 64, io, far=far)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("norm,weights", [(False, False), (True, False)])
def test_without_norm_or_weights(norm, weights, io):
    run((2, 20), 4, 2, 80, 80, io, norm=norm, weights=weights, slices=True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_many_tokens(io):
    """More heads than a launch's waves: every workgroup takes several."""
    run((3, 3001), 6, 2, 32, 32, io, shared=True)


def test_gradient_against_differences():
    """The float32 backward against central differences of the float32 forward, along random directions."""
    import torch
    import selective_scan_segmented_amd as sfm
    q, k, dq, dk, wq, wk, freqs, sec, pos = inputs(3, (2, 30), 3, 2, 48, 40, "f32")
    t = [dev(v, "f32").view(2, 30, *v.shape[1:]) for v in (q, k)] + [dev(wq, "f32"), dev(wk, "f32")]
    up = [dev(v, "f32").view(2, 30, *v.shape[1:]) for v in (dq, dk)]
    form = dict(positions=torch.from_numpy(pos).cuda().view(2, 30), freqs=dev(freqs, "f32"))
    got = sfm.sfm_qk_norm_rope_bwd(*up, *t, **form)
    gen = torch.Generator(device="cuda").manual_seed(4)
    for n, name in enumerate(("dq", "dk", "dwq", "dwk")):
        way, step, ends = torch.randn(t[n].shape, generator=gen, device="cuda"), 2.0 ** -7, []
        for s in (1, -1):
            out = sfm.sfm_qk_norm_rope_fwd(*t[:n], t[n] + s * step * way, *t[n + 1:], **form)
            ends.append(sum((a.double() * b).sum().item() for a, b in zip(out, up)))
        num, ana = (ends[0] - ends[1]) / (2 * step), (got[name].double() * way).sum().item()
        # third derivatives of order one times step^2 / 6, float32's 1e-7 of the loss's terms over the step
        size = torch.linalg.vector_norm(got[name].double() * way).item()
        assert abs(num - ana) <= 1e-3 * size + 1e-3, (name, num, ana, size)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-30, 1e25, 1e38])
def test_values_far_from_one(size, io):
    """Squares that leave float32's range: eps decides, or the values' own scale does."""
    import torch
    import selective_scan_segmented_amd as sfm
    rng = np.random.default_rng(5)
    for d in (64, 24):
        x = cast(rng.uniform(-1, 1, (6, 2, d)) * size, io)
        x[2] = 0
        dy = cast(rng.standard_normal(x.shape), io)
        t, g = dev(x, io), dev(dy, io)
        qo, ko = sfm.sfm_qk_norm_rope_fwd(t, t.clone(), eps=EPS)
        want = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
        close(from_dev(qo), want, io, "qo", FORWARD[io])
        assert torch.equal(qo, ko)
        got = sfm.sfm_qk_norm_rope_bwd(g, g, t, t.clone(), eps=EPS)
        dx, _, _ = ref.rope_bwd(x, np.ones(d), np.zeros((6, 0)), 0, False, True, EPS, dy)
        # (a row's gradient goes by its own scale: gradients below float32's normal range may be zero)
        for row in range(6):
            bound = {"f32": 1e-5, "bf16": 2.0 ** -8}[io] * np.abs(dx[row]) + 1e-4 * np.sqrt(np.mean(dx[row] ** 2)) + 2.0 ** -126
            assert (np.abs(from_dev(got["dq"])[row] - dx[row]) <= bound).all(), row


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_nonfinite_values_stay_in_their_head(bad, io):
    import torch
    import selective_scan_segmented_amd as sfm
    q, k, dq, dk, wq, wk, freqs, sec, pos = inputs(3, (40,), 5, 3, 64, 64, io)
    t, up = [dev(q, io), dev(k, io)], [dev(dq, io), dev(dk, io)]
    form = dict(positions=torch.from_numpy(pos).cuda().view(40), freqs=dev(freqs, "f32"), wq=dev(wq, "f32"), wk=dev(wk, "f32"))
    q0, k0 = sfm.sfm_qk_norm_rope_fwd(*t, **form)
    g0 = sfm.sfm_qk_norm_rope_bwd(*up, *t, **form)
    t[0][17, 3, 5] = bad
    q1, k1 = sfm.sfm_qk_norm_rope_fwd(*t, **form)
    g1 = sfm.sfm_qk_norm_rope_bwd(*up, *t, **form)
    keep = torch.ones_like(q0, dtype=torch.bool)
    keep[17, 3] = False
    assert torch.equal(q0[keep], q1[keep]) and torch.equal(k0, k1)
    assert torch.equal(g0["dq"][keep], g1["dq"][keep]) and torch.equal(g0["dk"], g1["dk"]) and torch.equal(g0["dwk"], g1["dwk"])
