"""Forms of the recurrence's and the rotation's calls: graphs, streams, workspaces, strided and sliced tensors."""
import numpy as np
import pytest

import recurrence_reference as ref

pytestmark = pytest.mark.gpu

# rows of one block, rows that a workgroup walks, rows handed on from block to block
SHAPES = [(3, 40, 96), (40, 600, 1024), (2, 1500, 96)]


def tensors(seed, B, L, D, io):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    lam = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda"))))
    return [r(B, L, D).to(io), r(B, L, D).to(io), r(B, L, D).to(io), lam, r(B, L, D).to(io), r(B, D), r(B, D)]


def rope_tensors(seed, B, L, H, Hk, d, io):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    return [r(B, L, H, d).to(io), r(B, L, Hk, d).to(io), r(B, L, H, d).to(io), r(B, L, Hk, d).to(io), r(d), r(d),
            torch.randint(0, 5000, (B, L), generator=gen, device="cuda", dtype=torch.int32), torch.rand(d // 2, generator=gen, device="cuda")]


def run_all(x, r, i, lam, dy, h0, dstate, pool, **more):
    import selective_scan_segmented_amd as sfm
    y, S = sfm.sfm_gated_recurrence_fwd(x, r, i, lam, h0=h0, return_state=True, **more)
    g = sfm.sfm_gated_recurrence_bwd(x, r, i, lam, y, dy, h0=h0, dstate=dstate, **more)
    pool.copy_(S)
    s = sfm.sfm_gated_recurrence_step(x[:, 0], r[:, 0], i[:, 0], lam, pool)
    return [y, S, *(g[n] for n in sorted(g)), s, pool]


def rope_all(q, k, dq, dk, wq, wk, positions, freqs):
    import selective_scan_segmented_amd as sfm
    form = dict(wq=wq, wk=wk, positions=positions, freqs=freqs)
    qo, ko = sfm.sfm_qk_norm_rope_fwd(q, k, **form)
    g = sfm.sfm_qk_norm_rope_bwd(dq, dk, q, k, **form)
    return [qo, ko, *(g[n] for n in sorted(g))]


@pytest.mark.parametrize("B,L,D", SHAPES)
def test_replays_are_the_eager_calls(B, L, D):
    import torch
    bf = torch.bfloat16
    every = lambda seed: tensors(seed, B, L, D, bf) + rope_tensors(seed, B, L, 4, 2, 24, bf)
    held, pool = every(0), torch.empty(B, D, device="cuda")
    both = lambda t, pool: run_all(*t[:7], pool) + rope_all(*t[7:])
    both(held, pool)  # (kernels are loaded before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(held, pool)
    for seed in (1, 2, 3, 1):
        t = every(seed)
        want = [v.clone() for v in both(t, torch.empty_like(pool))]
        torch.cuda.synchronize()
        for a, b in zip(held, t):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), (seed, n)


def test_two_graphs_that_share_a_workspace():
    """Both clear what they need of it: replayed in any order, each gives its own."""
    import torch
    import selective_scan_segmented_amd as sfm
    one, two = tensors(1, 2, 1500, 96, torch.bfloat16), tensors(2, 3, 2000, 160, torch.bfloat16)
    need = max(sfm.sfm_gated_recurrence_fwd_ws_size(t[0].shape[0], t[0].shape[1], t[0].shape[0] * t[0].shape[1], t[0].shape[2])
               for t in (one, two))
    ws = torch.full((need,), 0xa5, dtype=torch.uint8, device="cuda")
    call = lambda t: sfm.sfm_gated_recurrence_fwd(*t[:4], h0=t[5], workspace=ws)
    want = [call(t).clone() for t in (one, two)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(t))
        graphs.append(g)
    for n in (0, 1, 1, 0, 0, 1):
        outs[n].zero_()
        graphs[n].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[n], want[n])
        ws.fill_(n)


@pytest.mark.parametrize("B,L,D", SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_memory_comes_from_the_streams_pool(B, L, D, io):
    import torch
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    t = tensors(3, B, L, D, dt)
    import selective_scan_segmented_amd as sfm

    def call(stream):
        y, S = sfm.sfm_gated_recurrence_fwd(*t[:4], h0=t[5], return_state=True, stream=stream)
        return [y, S, *sfm.sfm_gated_recurrence_bwd(*t[:4], y, t[4], h0=t[5], dstate=t[6], stream=stream).values()]

    want = [v.clone() for v in call(None)]
    torch.cuda.synchronize()
    free = {v.data_ptr() for v in call(None)}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(side)
    side.synchronize()
    assert not free & {v.data_ptr() for v in got}
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,L,D", SHAPES)
def test_overlapping_calls_do_not_share_a_workspace(B, L, D):
    """Calls back to back on the current stream and on another, ten of each in flight: the serial bits."""
    import torch
    import selective_scan_segmented_amd as sfm
    t = tensors(4, B, L, D, torch.bfloat16)
    y0 = sfm.sfm_gated_recurrence_fwd(*t[:4], h0=t[5])
    call = lambda s: [sfm.sfm_gated_recurrence_fwd(*t[:4], h0=t[5], stream=s),
                      *sfm.sfm_gated_recurrence_bwd(*t[:4], y0, t[4], h0=t[5], dstate=t[6], stream=s).values()]
    want = [v.clone() for v in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [call(None if n % 2 == 0 else side) for n in range(20)]
    torch.cuda.synchronize()
    for outs in got:
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


def test_rotation_on_another_stream():
    import torch
    import selective_scan_segmented_amd as sfm
    q, k, dq, dk, wq, wk, pos, freqs = rope_tensors(1, 3, 700, 6, 2, 64, torch.bfloat16)
    form = dict(wq=wq, wk=wk, positions=pos, freqs=freqs)
    call = lambda s: [*sfm.sfm_qk_norm_rope_fwd(q, k, stream=s, **form), *sfm.sfm_qk_norm_rope_bwd(dq, dk, q, k, stream=s, **form).values()]
    want = [v.clone() for v in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [call(None if n % 2 == 0 else side) for n in range(12)]
    torch.cuda.synchronize()
    for outs in got:
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_any_alignment_gives_the_same_bits(io):
    """Tensors that start on a lone element, odd strides, outputs given: the aligned call's values."""
    import torch
    import selective_scan_segmented_amd as sfm
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    for B, L, D in ((2, 40, 64), (2, 700, 66)):
        x, r, i, lam, dy, h0, ds = tensors(5, B, L, D, dt)
        y0, S0 = sfm.sfm_gated_recurrence_fwd(x, r, i, lam, h0=h0, return_state=True)
        g0 = sfm.sfm_gated_recurrence_bwd(x, r, i, lam, y0, dy, h0=h0, dstate=ds)

        def moved(t, ld=None):
            ld = ld or D
            flat = torch.zeros(B * L * ld + 1, dtype=dt, device="cuda")
            v = flat[1:].view(B, L, ld)[..., :D]
            v.copy_(t)
            return v

        for lds in ((None, None, None), (D + 1, D + 7, 2 * D + 3)):
            a = [moved(t, ld) for t, ld in zip((x, r, i), lds)]
            y, S = sfm.sfm_gated_recurrence_fwd(*a, lam, h0=h0, return_state=True, y=moved(torch.zeros_like(x)))
            # (another width of the lanes: the same chunks, the same order of every sum)
            assert torch.equal(y, y0) and torch.equal(S, S0)
            g = sfm.sfm_gated_recurrence_bwd(*a, lam, y, moved(dy), h0=h0, dstate=ds)
            for n in ("dx", "dr", "di", "dh0"):
                assert torch.equal(g[n], g0[n]), n
        q, k, dq, dk, wq, wk, pos, freqs = rope_tensors(2, B, L, 3, 1, 64, dt)
        form = dict(wq=wq, wk=wk, positions=pos, freqs=freqs)
        shift = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)
        a0, b0 = sfm.sfm_qk_norm_rope_fwd(q, k, **form)
        a1, b1 = sfm.sfm_qk_norm_rope_fwd(shift(q), shift(k), **form)
        step = 2.0 ** -7 if io == "bf16" else 4e-7  # (squares are summed in another order: a bfloat16 step, float32's 2^-22)
        assert torch.allclose(a0.float(), a1.float(), rtol=step, atol=1e-6) and torch.allclose(b0.float(), b1.float(), rtol=step, atol=1e-6)


def test_one_token_of_each_row_in_place():
    """X[:, t:t + 1] of a projection: tokens are as far apart as the rows."""
    import torch
    import selective_scan_segmented_amd as sfm
    x, r, i, lam, dy, h0, _ = tensors(6, 5, 9, 48, torch.bfloat16)
    at = [t[:, 4:5] for t in (x, r, i)]
    y = sfm.sfm_gated_recurrence_fwd(*at, lam, h0=h0)
    assert torch.equal(y, sfm.sfm_gated_recurrence_fwd(*[t.contiguous() for t in at], lam, h0=h0))
    pool = h0.clone()
    assert torch.equal(y[:, 0], sfm.sfm_gated_recurrence_step(*[t[:, 0] for t in at], lam, pool))


def test_long_tensors_of_wide_strides():
    """Tokens whose offsets pass 2^31 elements, and blocks whose bytes are far apart."""
    import torch
    import selective_scan_segmented_amd as sfm
    # 300 tokens of 8 channels, 2^19 elements apart, 2 rows: 2 GB in bfloat16
    ld, L, D = 1 << 19, 1100, 8
    wide = torch.zeros(2, L, ld, dtype=torch.bfloat16, device="cuda")
    x, r, i, lam, dy, h0, ds = tensors(7, 2, L, D, torch.bfloat16)
    views = []
    for n, t in enumerate((x, r, i)):
        v = wide[..., n * D:(n + 1) * D]
        v.copy_(t)
        views.append(v)
    y0, S0 = sfm.sfm_gated_recurrence_fwd(x, r, i, lam, h0=h0, return_state=True)
    y, S = sfm.sfm_gated_recurrence_fwd(*views, lam, h0=h0, return_state=True)
    assert torch.equal(y, y0) and torch.equal(S, S0)
    g0 = sfm.sfm_gated_recurrence_bwd(x, r, i, lam, y0, dy, h0=h0, dstate=ds)
    g = sfm.sfm_gated_recurrence_bwd(*views, lam, y0, dy, h0=h0, dstate=ds)
    for n in g0:
        assert torch.equal(g[n], g0[n]), n
    # a step past 2^31 elements, and a rotation there
    pool = h0.clone()
    s = sfm.sfm_gated_recurrence_step(*[v[:, L - 1] for v in views], lam, pool)
    assert torch.equal(s, sfm.sfm_gated_recurrence_step(*[t[:, L - 1] for t in (x, r, i)], lam, h0.clone()))
    q, k = wide[..., 1000:1000 + 64].unflatten(-1, (2, 32)), wide[..., 2000:2032].unflatten(-1, (1, 32))
    q.normal_(), k.normal_()
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    freqs = torch.rand(16, device="cuda")
    a = sfm.sfm_qk_norm_rope_fwd(q, k, positions=pos, freqs=freqs)
    b = sfm.sfm_qk_norm_rope_fwd(q.contiguous(), k.contiguous(), positions=pos, freqs=freqs)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_duplicate_work_of_no_request():
    """All rows padding, and a pool of one state."""
    import torch
    import selective_scan_segmented_amd as sfm
    x, r, i, lam, _, h0, _ = tensors(8, 4, 1, 33, torch.float32)
    pool = h0[:1].clone()
    y = sfm.sfm_gated_recurrence_step(x[:, 0], r[:, 0], i[:, 0], lam, pool, slots=torch.full((4,), -1, dtype=torch.int32, device="cuda"))
    assert not y.any() and torch.equal(pool, h0[:1])
    slots = torch.tensor([-7, 0, 9, 1], dtype=torch.int32, device="cuda")
    y = sfm.sfm_gated_recurrence_step(x[:, 0], r[:, 0], i[:, 0], lam, pool, slots=slots)
    assert y[1].any() and not y[0].any() and not y[2:].any()


def test_tensors_past_32_bits():
    """2^32 elements and more: the last rows, tokens and heads are what they are by themselves."""
    import torch
    import selective_scan_segmented_amd as sfm
    B, L, D = 16387, 64, 4096
    gen = torch.Generator(device="cuda").manual_seed(1)
    lam = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda"))))
    x = torch.empty(B, L, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    assert x.numel() > 1 << 32
    S = torch.empty(B, D, device="cuda")
    y = sfm.sfm_gated_recurrence_fwd(x, x, x, lam, state=S)
    g = sfm.sfm_gated_recurrence_bwd(x, x, x, lam, y, x)
    last = x[-3:].clone()
    y1, S1 = sfm.sfm_gated_recurrence_fwd(last, last, last, lam, return_state=True)
    g1 = sfm.sfm_gated_recurrence_bwd(last, last, last, lam, y1, last)
    assert torch.equal(y[-3:], y1) and torch.equal(S[-3:], S1)
    for n in ("dx", "dr", "di"):
        assert torch.equal(g[n][-3:], g1[n]), n
    del g
    # one long row (handed on), and its end: decays are below 0.999^(8 sigmoid(r)), so 4000 tokens keep e^-16 of a state;
    # blocks fall elsewhere, where a block's decay is a product of up to 1024 factors: 2^-14 of states below 4
    x = x.view(1, B * L, D)
    y = sfm.sfm_gated_recurrence_fwd(x, x, x, lam, y=y.view(1, B * L, D))
    end = x[:, -4000:].contiguous()
    y1 = sfm.sfm_gated_recurrence_fwd(end, end, end, lam)
    assert torch.allclose(y[:, -64:].float(), y1[:, -64:].float(), rtol=2.0 ** -7, atol=2.0 ** -12)
    # heads
    H, d = 128, 128
    q, k = x.view(-1, H, d), x.view(-1, H, d)[:, :1]
    pos, freqs = torch.arange(q.shape[0], dtype=torch.int32, device="cuda"), torch.rand(d // 2, generator=gen, device="cuda")
    form = dict(wq=lam[:d].contiguous(), wk=lam[:d].contiguous(), freqs=freqs)
    qo, ko = sfm.sfm_qk_norm_rope_fwd(q, k, positions=pos, qo=y.view(q.shape), **form)
    g = sfm.sfm_qk_norm_rope_bwd(q, ko, q, k, positions=pos, **form)
    a, b, p = q[-100:].clone(), k[-100:].clone(), pos[-100:].clone()
    qo1, ko1 = sfm.sfm_qk_norm_rope_fwd(a, b, positions=p, **form)
    g1 = sfm.sfm_qk_norm_rope_bwd(a, ko1, a, b, positions=p, **form)
    assert torch.equal(qo[-100:], qo1) and torch.equal(ko[-100:], ko1)
    assert torch.equal(g["dq"][-100:], g1["dq"]) and torch.equal(g["dk"][-100:], g1["dk"])
