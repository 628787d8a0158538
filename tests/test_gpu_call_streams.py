"""Calls on a stream of the caller's: their memory comes from that stream's pool, and calls on two streams that
overlap in time do not share a workspace."""
import pytest

pytestmark = pytest.mark.gpu


def entries():
    """name -> (call(stream), every tensor it allocates)."""
    import torch
    import selective_scan_segmented_amd as sfm
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    u, dl, Bm, Cm = r(2, 64, 30), r(2, 64, 30), r(2, 8, 30), r(2, 8, 30)
    A, w = -torch.rand((64, 8), device="cuda"), r(64, 4)
    lu, ld, lB, lC = r(2, 64, 4000), r(2, 64, 4000), r(2, 8, 4000), r(2, 8, 4000)
    q, k, v = r(1, 300, 2, 64), r(1, 300, 2, 64), r(1, 300, 2, 64)
    g, beta = -torch.rand((1, 300, 2), device="cuda"), torch.rand((1, 300, 2), device="cuda")
    h0, do = r(1, 2, 64, 64), r(1, 300, 2, 64)
    x, dy = r(1, 6000, 64), r(1, 6000, 64)
    _, mean, rstd = sfm.sfm_group_norm_fwd(x, 4)
    delta = (q, k, v, g, beta)
    one = tuple(t[:, 0] for t in delta)

    def step(s):
        state = h0.clone()
        torch.cuda.synchronize()
        return [sfm.sfm_gated_delta_step(*one, state, l2norm=True, stream=s), state]

    return {
        "scan": lambda s: [sfm.sfm_selective_scan_fwd(u, dl, A, Bm, Cm, stream=s)],
        "scan_ws": lambda s: [sfm.sfm_selective_scan_fwd_ws(lu, ld, A, lB, lC, stream=s)],
        "scan_bwd": lambda s: list(sfm.sfm_selective_scan_bwd(u, dl, A, Bm, Cm, u, stream=s).values()),
        "pad_bwd": lambda s: [sfm.sfm_aux_pad_bwd(u, stream=s)],
        "conv": lambda s: [sfm.sfm_dwconv1d_fold(u, w, stream=s)],
        "pad": lambda s: [sfm.sfm_aux_pad_swap(u, mode="pad", stream=s)],
        "swap": lambda s: [sfm.sfm_aux_pad_swap(u, mode="swap", stream=s)],
        "delta": lambda s: list(sfm.sfm_gated_delta_fwd(*delta, h0=h0, return_state=True, l2norm=True, stream=s)),
        "delta_bwd": lambda s: list(sfm.sfm_gated_delta_bwd(*delta, do, h0=h0, l2norm=True, stream=s).values()),
        "step": step,
        "norm": lambda s: list(sfm.sfm_group_norm_fwd(x, 4, stream=s)),
        "norm_bwd": lambda s: list(sfm.sfm_group_norm_bwd(dy, x, mean, rstd, stream=s).values()),
    }


NAMES = ["scan", "scan_ws", "scan_bwd", "pad_bwd", "conv", "pad", "swap", "delta", "delta_bwd", "step", "norm", "norm_bwd"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_comes_from_the_streams_pool(name):
    """Blocks that the current stream has free are not handed to a call on another one."""
    import torch
    call = entries()[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    mine = 1 if name == "step" else None  # (the state is the caller's)
    free = {t.data_ptr() for t in call(None)[:mine]}  # outputs of a call, free again on the current stream
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(side)
    side.synchronize()
    assert not free & {t.data_ptr() for t in got[:mine]}
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # both streams' blocks are in hand again afterwards
    del got
    for a, b in zip(want, call(side)):
        side.synchronize()
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["scan_ws", "scan_bwd", "delta", "delta_bwd", "norm", "norm_bwd"])
def test_overlapping_calls_do_not_share_a_workspace(name):
    """Calls back to back on the current stream and on another, ten of each in flight: the serial bits."""
    import torch
    call = entries()[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [call(None if i % 2 == 0 else side) for i in range(20)]
    torch.cuda.synchronize()
    for outs in got:
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
