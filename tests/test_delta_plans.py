"""What the gated delta rule's size queries and checks answer (host only)."""
import pytest

import selective_scan_segmented_amd as sfm


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("walk", ["whole", "prepared"])
@pytest.mark.parametrize("L", [1, 3, 10, 51, 64])
def test_rows_of_one_chunk_need_no_workspace(L, walk, io, monkeypatch):
    """Whatever the override says: their inverses are made on the way, or they go token by token."""
    monkeypatch.setenv("SFM_DELTA_WALK", walk)
    for rows in (1, 4, 300):
        assert sfm.sfm_gated_delta_fwd_ws_size(rows, L, rows * L, 2, 64, 64, True, io) == 0


def bwd_size(rows, L, tokens, Hk, H, dk, dv):
    return sfm.sfm_gated_delta_bwd_ws_size(rows, L, tokens, Hk, H, dk, dv)


def fwd_size(rows, L, tokens, Hk, H, dk, dv):
    return sfm.sfm_gated_delta_fwd_ws_size(rows, L, tokens, H, dk, dv)


# sizes whose largest launch has 2^24 workgroups of 256 (2^32 work items), and one row fewer
@pytest.mark.parametrize("size,rows,L,Hk,H,dv", [
    (fwd_size, 1 << 20, 4, 1, 16, 64), (fwd_size, 1 << 19, 51, 1, 16, 128), (fwd_size, 1 << 18, 1, 1, 16, 256),
    (bwd_size, 1 << 19, 4, 16, 16, 64), (bwd_size, 1 << 19, 65, 4, 16, 16), (bwd_size, 1 << 18, 1, 16, 32, 16)])
def test_more_workgroups_than_a_launch_holds_are_refused(size, rows, L, Hk, H, dv):
    with pytest.raises(sfm.SFMError, match="more workgroups than a launch holds"):
        size(rows, L, rows * L, Hk, H, 16, dv)
    size(rows * 63 // 64, L, rows * 63 // 64 * min(L, 60), Hk, H, 16, dv)


def test_chunks_past_one_launch_are_not_prepared():
    """16 rows of 2^24 tokens and 16 heads: 2^26 chunks and heads, so their inverses are made on the way."""
    assert sfm.sfm_gated_delta_fwd_ws_size(16, 1 << 24, 1 << 28, 16, 64, 64) == 0
    assert sfm.sfm_gated_delta_fwd_ws_size(16, 1 << 20, 1 << 24, 16, 64, 64) > 0


P = 0x1000000  # an address that nothing reads: every call below fails its checks


def test_the_calls_refuse_what_the_queries_refuse():
    lib = sfm.load_library()
    tail = (0.125, 1, 1)
    rows = 1 << 20
    args = (P, 2 * P, 3 * P, 4 * P, 5 * P)
    assert lib.sfm_gated_delta_fwd(*args, None, 6 * P, None, None, rows, 4, 4 * rows, 1, 16, 64, 64, 64, 64, 1024, *tail, None, 0, None) == 2
    assert b"more workgroups than a launch holds" in lib.sfm_last_error()
    assert lib.sfm_gated_delta_bwd(*args, None, 6 * P, None, 7 * P, 8 * P, 9 * P, 10 * P, 11 * P, None, None, rows, 4, 4 * rows, 1, 16, 64,
                                   64, 64, 64, 1024, *tail, 100 * P, 1 << 40, None) == 2
    assert b"more workgroups than a launch holds" in lib.sfm_last_error()
    assert lib.sfm_gated_delta_step(*args, 6 * P, None, 9 * P, rows, rows, 1, 16, 64, 64, 64, 64, 1024, *tail, None) == 2
    assert b"more workgroups than a launch holds" in lib.sfm_last_error()


def test_rows_without_a_bound_are_planned_by_their_average():
    """L of all the tokens says nothing of the longest row: many short rows need no workspace then either."""
    f = sfm.sfm_gated_delta_fwd_ws_size
    assert f(1000, 400, 200000, 16, 128, 128) == 0
    assert f(1000, 200000, 200000, 16, 128, 128) == 0
    assert f(1000, 1 << 20, 200000, 16, 128, 128) == 0
    # few rows, or one among a few that may hold all the tokens: as by the bound
    for rows in (1, 2, 4, 8):
        assert f(rows, 20000, 20000, 16, 128, 128) > 0
    assert f(64, 64, 0, 16, 128, 128) == f(64, 1, 0, 16, 128, 128) == 0
