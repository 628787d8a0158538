"""Calls of the gated linear recurrence that look like allowed ones and are refused (host only)."""
import pytest

from test_recurrence_rope_abi import ALIAS, P, fwd, lib  # noqa: F401  (lib: a fixture)

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
