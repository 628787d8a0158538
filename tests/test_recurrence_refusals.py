"""Calls of the gated linear recurrence that look like allowed ones and are refused (host only)."""
import ctypes

import pytest

from test_recurrence_rope_abi import ALIAS, OK, P, SHAPE, fwd, lib  # noqa: F401  (lib: a fixture)

ONE_ROW = dict(rows=1, L=1000, tokens=1000)


@pytest.mark.parametrize("kw,on", [
    (dict(ONE_ROW, hT=4 * P), b"lam"), (dict(ONE_ROW, hT=4 * P, h0=4 * P), b"lam"),
    (dict(ONE_ROW, D=2, ldx=2, ldr=2, ldi=2, off=20 * P, hT=20 * P), b"offsets"),
    (dict(rows=4, L=1, tokens=4, io=0, hT=P), b"x"), (dict(rows=4, L=1, tokens=4, io=0, hT=2 * P), b"r"),
    (dict(rows=4, L=1, tokens=4, io=0, hT=3 * P, h0=3 * P), b"i"), (dict(ONE_ROW, hT=20 * P, h0=20 * P + 4), b"h0")])
def test_states_go_in_place_of_no_input_but_h0(lib, kw, on):  # noqa: F811
    """Inputs as large as the states, in exactly their place: the call would leave states there."""
    assert fwd(lib, **kw) == ALIAS
    assert lib.sfm_last_error() == b"sfm_gated_recurrence_fwd: hT overlaps " + on


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("L,tokens", [((1 << 24) + 1, (1 << 24) + 1), (20_000_000, 20_000_000), ((1 << 31) - 1, (1 << 31) - 1), (1 << 30, 5000)])
def test_rows_without_a_bound_of_many_tokens(lib, L, tokens, back):  # noqa: F811
    """A bound that is all the tokens is no limit of them: up to 2^31 - 1."""
    out = ctypes.c_int64(-1)
    f = lib.sfm_gated_recurrence_bwd_ws_size if back else lib.sfm_gated_recurrence_fwd_ws_size
    for rows, D, io in ((1, 8, 1), (100, 8, 1), (100, 8, 0)):
        assert f(rows, L, tokens, D, io, ctypes.byref(out)) == OK, lib.sfm_last_error()
        assert out.value > 0
        assert f(rows, 1 << 31, tokens, D, io, ctypes.byref(out)) == SHAPE
        assert f(rows, L, 1 << 31, D, io, ctypes.byref(out)) == SHAPE
