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
