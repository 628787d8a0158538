"""The gated delta rule and the group norm recorded into a graph: every replay has the eager calls' bits."""
import numpy as np
import pytest

import delta_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,H,Hk", [(200, 4, 2), (40, 2, 2)])
def test_replays_are_the_eager_calls(L, H, Hk):
    import torch
    import selective_scan_segmented_amd as sfm
    B, d = 2, 64
    bf, f32 = torch.bfloat16, torch.float32

    def inputs(seed):
        x = ref.delta_inputs(seed, B * L, B, Hk, H, d, d, True, "bf16")
        t = [torch.from_numpy(np.ascontiguousarray(a)).to(bf).cuda().view(B, L, *a.shape[1:]) for a in x[:5] + [x[6]]]
        return t + [torch.from_numpy(np.ascontiguousarray(x[5])).to(f32).cuda()]

    held = [torch.empty_like(t) for t in inputs(0)]
    pool = torch.empty(B, H, d, d, dtype=f32, device="cuda")
    w = torch.linspace(0.5, 1.5, H * d, device="cuda")

    def run(q, k, v, g, beta, do, h0, pool):
        o, S = sfm.sfm_gated_delta_fwd(q, k, v, g, beta, h0=h0, l2norm=True, return_state=True)
        y, mean, rstd = sfm.sfm_group_norm_fwd(o.flatten(2), H, w, w, act="silu")
        n = sfm.sfm_group_norm_bwd(do.flatten(2), o.flatten(2), mean, rstd, w, w, act="silu")
        gr = sfm.sfm_gated_delta_bwd(q, k, v, g, beta, n["dx"].view(v.shape), h0=h0, l2norm=True)
        pool.copy_(S)
        s = sfm.sfm_gated_delta_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
                                     g[:, 0].contiguous(), beta[:, 0].contiguous(), pool, l2norm=True)
        return [o, S, y, mean, rstd, *n.values(), *gr.values(), s, pool]

    for a, b in zip(held, inputs(0)):
        a.copy_(b)
    run(*held, pool)  # (kernels are loaded before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*held, pool)
    for seed in (1, 2, 3, 1):
        x = inputs(seed)
        want = [t.clone() for t in run(*x, torch.empty_like(pool))]
        torch.cuda.synchronize()
        for a, b in zip(held, x):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), (seed, i)
