"""The gated linear recurrence on the GPU against its definition in float64: forward, backward, one token of many."""
import numpy as np
import pytest

import recurrence_reference as ref
from delta_reference import close
from helpers import from_dev

pytestmark = pytest.mark.gpu

# y: float32, a state is a sum over the last 1 / |log a| tokens (about 250 here at most) whose factors are each off by
# some 2^-23 in different directions: sqrt(250) 2^-22 = 4e-6 of it and of its like, 2e-5 with a margin for the largest of
# many.  bfloat16: the rounding's half step 2^-8 and 1e-4 of the rms for what is below it.
FORWARD = {"f32": (2e-5, 2e-5), "bf16": (2.0 ** -8, 1e-4)}
# Gradients: G as y, and the decay's is a difference of two products about as large as itself or some times larger.
BACKWARD = {"f32": (1e-4, 1e-4), "bf16": (2.0 ** -8, 4e-4)}

# rows' lengths: equal rows of one token to several blocks of any plan, and packed ones with empty rows
EQUAL = [[1], [2] * 3, [7] * 2, [15, 15], [16] * 2, [17] * 3, [31] * 2, [33], [51] * 4, [64] * 2, [65], [127] * 2, [129], [198] * 2,
         [255], [257] * 2, [511], [513] * 2, [1000], [1025] * 2, [2500]]
PACKED = [[1, 0, 5], [0, 0], [3, 64, 0, 65, 1, 200], [0, 700, 1, 0, 515], [16, 32, 48, 1, 15, 17], [1300, 1300]]


def dev(a, io):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(torch.bfloat16 if io == "bf16" else torch.float32)


def side_by_side(parts, io):
    """The tensors as slices of one projection."""
    import torch
    p = torch.cat([dev(a, io) for a in parts], -1)
    return torch.split(p, [a.shape[-1] for a in parts], -1)


def call(seed, lens, D, io, slices=False, h0=True, bound=True):
    """Inputs of a call: the float64 ones, the GPU's, and the row arguments."""
    import torch
    packed = lens in PACKED or len(set(lens)) > 1
    x, r, i, lam, s0, dy, dhT = ref.recurrence_inputs(seed, sum(lens), len(lens), D, io)
    if not h0:
        s0[:] = 0
    lead = (1, sum(lens)) if packed else (len(lens), lens[0])
    gates = side_by_side((x, r, i), io) if slices else [dev(t, io) for t in (x, r, i)]
    gates = [t.unflatten(0, lead) if t.numel() else t.view(*lead, D) for t in gates]
    rows = dict(h0=dev(s0, "f32") if h0 else None)
    if packed:
        rows.update(offsets=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda(), max_len=max(lens) if bound else None)
    return (x, r, i, lam, s0, dy, dhT), gates + [dev(lam, "f32")], rows, np.cumsum(lens), lead


def check_forward(seed, lens, D, io, c=8.0, **kw):
    import selective_scan_segmented_amd as sfm
    want, t, rows, ends, lead = call(seed, lens, D, io, **kw)
    y, state = sfm.sfm_gated_recurrence_fwd(*t, c=c, return_state=True, **rows)
    wy, wh = ref.recurrence(*want[:5], ends, c)
    assert y.shape == lead + (D,) and y.is_contiguous()
    close(from_dev(y).reshape(-1, D), wy, io, "y", FORWARD[io])
    close(from_dev(state), wh, "f32", "state", FORWARD["f32"])
    only = sfm.sfm_gated_recurrence_fwd(*t, c=c, **rows)
    assert (only == y).all() or not y.numel()


def check_backward(seed, lens, D, io, c=8.0, dstate=True, **kw):
    import selective_scan_segmented_amd as sfm
    want, t, rows, ends, lead = call(seed, lens, D, io, **kw)
    x, r, i, lam, s0, dy, dhT = want
    if not dstate:
        dhT[:] = 0
    y = sfm.sfm_gated_recurrence_fwd(*t, c=c, **rows)
    got = sfm.sfm_gated_recurrence_bwd(*t, y, dev(dy, io).view(*lead, D), c=c, dstate=dev(dhT, "f32") if dstate else None, **rows)
    w = ref.recurrence_bwd(x, r, i, lam, s0, from_dev(y).reshape(-1, D), ends, c, dy, dhT)
    assert sorted(got) == sorted(n for n in w if n != "dlam_size" and (n != "dh0" or rows["h0"] is not None))
    for n in ("dx", "dr", "di"):
        close(from_dev(got[n]).reshape(-1, D), w[n], io, n, BACKWARD[io])
    if "dh0" in got:
        close(from_dev(got["dh0"]), w["dh0"], "f32", "dh0", BACKWARD["f32"])
    # float32 sums of terms that are each off by some 1e-6 of themselves
    err = np.abs(from_dev(got["dlam"]) - w["dlam"])
    assert (err <= 1e-5 * w["dlam_size"] + 1e-30).all(), np.max(err / (w["dlam_size"] + 1e-30))
    again = sfm.sfm_gated_recurrence_bwd(*t, y, dev(dy, io).view(*lead, D), c=c, dstate=dev(dhT, "f32") if dstate else None, **rows)
    for n in got:
        assert (got[n] == again[n]).all() or not got[n].numel(), n


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", EQUAL + PACKED, ids=str)
def test_forward_by_length(lens, io):
    check_forward(len(lens), lens, 72, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", EQUAL + PACKED, ids=str)
def test_backward_by_length(lens, io):
    check_backward(len(lens), lens, 72, io)


WIDTHS = [1, 2, 3, 7, 8, 17, 31, 64, 66, 100, 129, 160, 256, 320, 640, 1000]


@pytest.mark.parametrize("slices", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_forward_by_width(D, io, slices):
    check_forward(D, [70] * 2, D, io, slices=slices)
    check_forward(D, [300, 0, 20], D, io, slices=slices, h0=False)


@pytest.mark.parametrize("slices", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_backward_by_width(D, io, slices):
    check_backward(D, [70] * 2, D, io, slices=slices)
    check_backward(D, [300, 0, 20], D, io, slices=slices, h0=False, dstate=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("c", [0.01, 1.0, 30.0])
def test_decays_of_other_rates(c, io):
    """A state that hardly decays, and one that forgets within a token (slow ones sum over the whole row)."""
    check_forward(3, [400] * 2, 40, io, c=c)
    check_backward(3, [400] * 2, 40, io, c=c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_many_rows(io):
    check_forward(5, [5] * 300, 24, io)
    check_backward(5, [5] * 300, 24, io)


def test_gradient_against_differences():
    """The float32 backward against central differences of the float32 forward, along random directions."""
    import torch
    import selective_scan_segmented_amd as sfm
    lens, D = [90, 0, 301], 48
    want, t, rows, ends, lead = call(9, lens, D, "f32")
    dy, dhT = dev(want[5], "f32").view(*lead, D), dev(want[6], "f32")
    y = sfm.sfm_gated_recurrence_fwd(*t, **rows)
    got = sfm.sfm_gated_recurrence_bwd(*t, y, dy, dstate=dhT, **rows)

    def loss(x, r, i, lam, h0):
        y, s = sfm.sfm_gated_recurrence_fwd(x, r, i, lam, h0=h0, offsets=rows["offsets"], max_len=rows["max_len"], return_state=True)
        return ((y.double() * dy).sum() + (s.double() * dhT).sum()).item()

    at = t + [rows["h0"]]
    gen = torch.Generator(device="cuda").manual_seed(4)
    for n, name in enumerate(("dx", "dr", "di", "dlam", "dh0")):
        way = torch.randn(at[n].shape, generator=gen, device="cuda")
        step = 2.0 ** -7
        ends_ = [loss(*at[:n], at[n] + s * step * way, *at[n + 1:]) for s in (1, -1)]
        num, ana = (ends_[0] - ends_[1]) / (2 * step), (got[name].double() * way).sum().item()
        # the differences' own error: third derivatives of order one times step^2 / 6 (1e-5 of the terms' size, which
        # random signs make sqrt(n) rms), and float32's 1e-7 of the loss's terms over the step
        size = torch.linalg.vector_norm(got[name].double() * way).item()
        assert abs(num - ana) <= 1e-3 * size + 1e-3, (name, num, ana, size)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R,D", [(1, 1), (1, 320), (3, 7), (5, 129), (40, 320), (256, 640), (7, 1000)])
def test_steps_are_the_rows_tokens(R, D, io):
    """Token by token on a pool of states: the definition, the other slots as they were, padding rows zero."""
    import torch
    import selective_scan_segmented_amd as sfm
    T, pool = 3, R + 3
    x, r, i, lam, s0, _, _ = ref.recurrence_inputs(R + D, R * T, pool, D, io)
    rng = np.random.default_rng(1)
    slots = rng.permutation(pool)[:R].astype(np.int32)
    state, want = dev(s0, "f32"), s0.copy()
    for t in range(T):
        at = [v[t * R:(t + 1) * R] for v in (x, r, i)]
        tensors = side_by_side(at, io) if t == 1 else [dev(v, io) for v in at]
        idx = slots.copy()
        if t == 2:
            idx[R // 2] = -1 if R % 2 else pool
        y = sfm.sfm_gated_recurrence_step(*tensors, dev(lam, "f32"), state, slots=torch.from_numpy(idx).cuda())
        a, _, m, _, si = ref.gates(at[1], at[2], lam, 8.0)
        wy = np.zeros((R, D))
        for row in range(R):
            if 0 <= idx[row] < pool:
                wy[row] = want[idx[row]] = a[row] * want[idx[row]] + m[row] * si[row] * at[0][row]
        close(from_dev(y), wy, io, "y", FORWARD[io])
        close(from_dev(state), want, "f32", "state", FORWARD["f32"])
    # without slots: state r
    y = sfm.sfm_gated_recurrence_step(*[dev(v[:R], io) for v in (x, r, i)], dev(lam, "f32"), dev(s0, "f32"))
    a, _, m, _, si = ref.gates(r[:R], i[:R], lam, 8.0)
    close(from_dev(y), a * s0[:R] + m * si * x[:R], io, "y", FORWARD[io])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_state_in_place_and_outputs_given(io):
    import torch
    import selective_scan_segmented_amd as sfm
    for lens in ([600] * 2, [0, 40, 900]):
        want, t, rows, ends, lead = call(2, lens, 96, io)
        y0, s0 = sfm.sfm_gated_recurrence_fwd(*t, return_state=True, **rows)
        y = torch.full_like(y0, 7)
        h = rows["h0"].clone()
        got = sfm.sfm_gated_recurrence_fwd(*t, y=y, state=h, **dict(rows, h0=h))
        assert got is y and torch.equal(y, y0) and torch.equal(h, s0)
        dy = dev(want[5], io).view(y.shape)
        g0 = sfm.sfm_gated_recurrence_bwd(*t, y, dy, **rows)
        into = {n: torch.full_like(v, 7) for n, v in g0.items()}
        g1 = sfm.sfm_gated_recurrence_bwd(*t, y, dy, grads=into, **rows)
        for n in g0:
            assert g1[n] is into[n] and torch.equal(g0[n], g1[n]), n


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_tokens_of_no_row_are_left_alone(io):
    """Offsets that start late, end early, leave gaps by max_len, or lie outside the tokens."""
    import torch
    import selective_scan_segmented_amd as sfm
    D, tokens = 40, 400
    x, r, i, lam, _, dy, _ = ref.recurrence_inputs(8, tokens, 1, D, io)
    t = [dev(v, io).view(1, tokens, D) for v in (x, r, i)] + [dev(lam, "f32")]
    for off, most in (([10, 100, 100, 380], 300), ([0, 350, 400], 120), ([-5, 90, 90, 1000], 310)):
        rows, idx = [], torch.tensor(off, dtype=torch.int32).cuda()
        for lo, hi in zip(off, off[1:]):
            lo = min(max(lo, 0), tokens)
            hi = lo if hi < lo else min(hi, tokens)
            rows.append((lo, min(hi, lo + most)))
        y = torch.full((1, tokens, D), 7.0, dtype=t[0].dtype, device="cuda")
        _, state = sfm.sfm_gated_recurrence_fwd(*t, offsets=idx, max_len=most, y=y, return_state=True)
        grads = {n: torch.full_like(y, 7) for n in ("dx", "dr", "di")}
        sfm.sfm_gated_recurrence_bwd(*t, y, dev(dy, io).view(y.shape), offsets=idx, max_len=most, grads=grads)
        inside = np.zeros(tokens, bool)
        for n, (lo, hi) in enumerate(rows):
            inside[lo:hi] = True
            wy, wh = ref.recurrence(x[lo:hi], r[lo:hi], i[lo:hi], lam, np.zeros((1, D)), [hi - lo], 8.0)
            close(from_dev(y)[0, lo:hi], wy, io, "y", FORWARD[io])
            close(from_dev(state)[n:n + 1], wh, "f32", "state", FORWARD["f32"])
        for g in (y, *grads.values()):
            g = from_dev(g)[0]
            assert (g[~inside] == 7).all() and (not inside.any() or (g[inside] != 7).any())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_nonfinite_values_stay_in_row_and_channel(bad, io):
    """x, r and i of one token: nothing before it, no other row, no other channel changes, in either direction."""
    import torch
    import selective_scan_segmented_amd as sfm
    lens, D, tok, ch = [700, 300, 700], 80, 700 + 130, 33
    want, t, rows, ends, lead = call(4, lens, D, io)
    dy = dev(want[5], io).view(1, -1, D)
    y0, s0 = sfm.sfm_gated_recurrence_fwd(*t, return_state=True, **rows)
    g0 = sfm.sfm_gated_recurrence_bwd(*t, y0, dy, **rows)
    for n in range(3):
        hurt = [v.clone() for v in t]
        hurt[n][0, tok, ch] = bad
        y, s = sfm.sfm_gated_recurrence_fwd(*hurt, return_state=True, **rows)
        same = torch.ones_like(y, dtype=torch.bool)
        same[0, tok:1000, ch] = False
        assert torch.equal(y[same], y0[same])
        rest = torch.ones_like(s, dtype=torch.bool)
        rest[1, ch] = False
        assert torch.equal(s[rest], s0[rest])
        g = sfm.sfm_gated_recurrence_bwd(*hurt, y, dy, **rows)
        same[0, 700:1000, ch] = False
        for name in ("dx", "dr", "di"):
            assert torch.equal(g[name][same], g0[name][same]), (n, name)
        assert torch.equal(g["dh0"][rest], g0["dh0"][rest])
        other = torch.arange(D, device="cuda") != ch
        assert torch.equal(g["dlam"][other], g0["dlam"][other])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gates_at_their_limits(io):
    """Gates of +-inf and far values are open or shut: a = 1 keeps the state, and its gradients are finite."""
    import torch
    import selective_scan_segmented_amd as sfm
    D = 16
    x, r, i, lam, s0, dy, dhT = ref.recurrence_inputs(6, 40, 1, D, io)
    r[5:9], r[9], i[12], i[13], r[20] = -np.inf, -200.0, -np.inf, np.inf, np.inf
    lam[3], lam[4] = -100.0, 20.0
    t = [dev(v, io).view(1, 40, D) for v in (x, r, i)] + [dev(lam, "f32")]
    h0 = dev(s0, "f32")
    y, s = sfm.sfm_gated_recurrence_fwd(*t, h0=h0, return_state=True)
    wy, wh = ref.recurrence(x, r, i, lam, s0, [40], 8.0)
    close(from_dev(y)[0], wy, io, "y", FORWARD[io])
    close(from_dev(s), wh, "f32", "state", FORWARD["f32"])
    # The state before a chunk of tokens is A h + H of the chunk before it, the tokens' own states are walked one by one:
    # 8 fused steps either way, each rounded by 2^-24 of a state of the chunk.  So kept states are the same bits within a
    # chunk (8 and 9) and within 16 2^-24 of the chunk's largest across it (4 and 8), of which bfloat16 may make a step.
    assert torch.equal(y[0, 8], y[0, 9]) and torch.equal(y[0, 4], y[0, 7])
    largest = torch.cat([h0, y[0, :9].float()]).abs().max(0).values
    step = 16 * 2.0 ** -24 * largest + (2.0 ** -7 * y[0, 4].float().abs() if io == "bf16" else 0)
    assert ((y[0, 4].float() - y[0, 8].float()).abs() <= step).all()
    assert torch.equal(s[0, 3], h0[0, 3])
    got = sfm.sfm_gated_recurrence_bwd(*t, y, dev(dy, io).view(1, 40, D), h0=h0, dstate=dev(dhT, "f32"))
    w = ref.recurrence_bwd(x, r, i, lam, s0, from_dev(y)[0], [40], 8.0, dy, dhT)
    for n in ("dx", "dr", "di"):
        close(from_dev(got[n])[0], w[n], io, n, BACKWARD[io])
    # softplus(-100) = 4e-44 is no normal float32 and taken as 0, so the input's factor m, its root's size, is 0 in place
    # of up to sqrt(2 c 2^-126) = 2^-61; the 40 terms of dlam are up to |G| |x| m / 2 each: below 2^-55 together
    assert (np.abs(from_dev(got["dlam"]) - w["dlam"]) <= 1e-5 * w["dlam_size"] + 2.0 ** -55).all()


def test_long_row_of_slow_decays():
    """One row of 70000 tokens: blocks by the hundred."""
    check_forward(1, [70000], 8, "f32", c=1.0)
    check_backward(1, [70000], 8, "bf16")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,L", [(3, 700), (4, 300), (5, 1100), (9, 530), (11, 260), (17, 400)])
def test_numbers_of_long_rows(rows, L, io):
    """Blocks handed on by rows that are no whole groups."""
    check_forward(rows, [L] * rows, 72, io)
    check_backward(rows, [L] * rows, 72, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D,low,high,most", [(33, 100, 300, 300), (34, 1, 60, 125), (66, 1, 20, 70)])
def test_many_packed_rows(D, low, high, most, io):
    """Packed rows that a workgroup walks each, some of them empty, some far longer than the others."""
    import torch
    import selective_scan_segmented_amd as sfm
    rng = np.random.default_rng(4)
    n = 4200
    lens = rng.integers(low, high, n)
    lens[[0, 7, 8, n - 1]] = 0
    lens[[1, 1000, 3000]] = most
    ends = np.cumsum(lens)
    x, r, i, lam, s0, dy, dhT = ref.recurrence_inputs(4, int(ends[-1]), n, D, io)
    t = [dev(v, io).view(1, -1, D) for v in (x, r, i)] + [dev(lam, "f32")]
    off = torch.tensor(np.concatenate([[0], ends]), dtype=torch.int32).cuda()
    rows = dict(h0=dev(s0, "f32"), offsets=off, max_len=most)
    y, state = sfm.sfm_gated_recurrence_fwd(*t, return_state=True, **rows)
    g = sfm.sfm_gated_recurrence_bwd(*t, y, dev(dy, io).view(y.shape), dstate=dev(dhT, "f32"), **rows)
    yh = from_dev(y)[0]
    for s in (0, 1, 7, 9, 1000, 2500, n - 2, n - 1):
        at, one = slice(ends[s] - lens[s], ends[s]), slice(s, s + 1)
        wy, wh = ref.recurrence(x[at], r[at], i[at], lam, s0[one], [lens[s]], 8.0)
        close(yh[at], wy, io, "y", FORWARD[io])
        close(from_dev(state)[one], wh, "f32", "state", FORWARD["f32"])
        w = ref.recurrence_bwd(x[at], r[at], i[at], lam, s0[one], yh[at], [lens[s]], 8.0, dy[at], dhT[one])
        for k in ("dx", "dr", "di"):
            close(from_dev(g[k])[0, at], w[k], io, k, BACKWARD[io])
        close(from_dev(g["dh0"])[one], w["dh0"], "f32", "dh0", BACKWARD["f32"])
    # dr is the terms of dlam times 1 - sigmoid(r), each rounded to its type once
    lam = t[3].double()
    terms = g["dr"][0].double() / torch.sigmoid(-t[1][0].double()) * (torch.sigmoid(lam) / torch.nn.functional.softplus(lam))
    step = 2.0 ** -8 if io == "bf16" else 2.0 ** -24
    assert ((g["dlam"].double() - terms.sum(0)).abs() <= (step + 1e-5) * terms.abs().sum(0)).all()


def test_replays_of_packed_rows_read_their_offsets():
    """A captured call of packed rows takes the offsets that its tensor holds at each replay."""
    import torch
    import selective_scan_segmented_amd as sfm
    D, tokens, most = 72, 2000, 900
    x, r, i, lam, s0, dy, _ = ref.recurrence_inputs(6, tokens, 5, D, "bf16")
    t = [dev(v, "bf16").view(1, tokens, D) for v in (x, r, i)] + [dev(lam, "f32")]
    dy, h0 = dev(dy, "bf16").view(1, tokens, D), dev(s0, "f32")
    off = torch.zeros(6, dtype=torch.int32, device="cuda")

    def both(y=None, grads=None):
        form = dict(h0=h0, offsets=off, max_len=most)
        y, state = sfm.sfm_gated_recurrence_fwd(*t, y=y, return_state=True, **form)
        return y, state, sfm.sfm_gated_recurrence_bwd(*t, y, dy, grads=grads, **form)

    outs = lambda: (torch.zeros_like(dy), {n: torch.zeros_like(dy) for n in ("dx", "dr", "di")})
    held = outs()
    both(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, state, g = both(*held)
    for ends in ([0, 900, 900, 1000, 1900, 2000], [0, 0, 0, 0, 0, 0], [5, 300, 600, 900, 1200, 1700], [0, 900, 900, 1000, 1900, 2000]):
        off.copy_(torch.tensor(ends, dtype=torch.int32))
        wy, ws, wg = both(*outs())
        for v in (held[0], *held[1].values()):
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(state, ws)
        for n in wg:
            assert torch.equal(g[n], wg[n]), n


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [8, 72, 200, 640])
@pytest.mark.parametrize("lens", [[3, 1, 0, 7, 2, 5, 0, 4] * 6, [3, 1, 0, 7, 2, 5, 0, 4, 700] * 4, [40, 90, 1, 60, 0, 77] * 5], ids=["short", "outliers", "middling"])
def test_packed_rows_without_a_bound(lens, D, io):
    check_forward(len(lens), lens, D, io, bound=False)
    check_backward(len(lens), lens, D, io, bound=False)
