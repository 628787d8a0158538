"""What the gated delta rule's binding checks before it calls the library (host only, stand-ins for GPU tensors)."""
import types

import pytest
import torch

import selective_scan_segmented_amd as sfm

SIDE = types.SimpleNamespace(cuda_stream=0)


class Stub:
    """A GPU tensor as the binding sees one: sizes, strides, type and an address that nothing reads."""
    is_cuda = True
    count = 0

    def __init__(self, *shape, dtype=torch.bfloat16, stride=None):
        self.shape, self.dtype = torch.Size(shape), dtype
        Stub.count += 1
        self.at = Stub.count << 32
        dense, n = [], 1
        for size in reversed(shape):
            dense.insert(0, n)
            n *= size
        self.dense, self.steps = tuple(dense), tuple(stride or dense)

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.steps

    def is_contiguous(self):
        return self.steps == self.dense

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize


@pytest.fixture
def calls(monkeypatch):
    """The library's calls in place of the calls: (name, arguments)."""
    seen = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_ws_size"):
                def size(*a):
                    seen.append((name, a))
                    return 0
                return size
            return lambda *a: seen.append((name, a)) or 0

    monkeypatch.setattr(sfm, "load_library", Library)
    monkeypatch.setattr(sfm, "_dev", check)
    return seen


def check(t, name, dtype=None, shape=None):
    """_dev for stand-ins."""
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {shape}")


B, L, HK, H, DK, DV = 2, 100, 1, 2, 64, 32


def args(lead=(B, L)):
    return [Stub(*lead, HK, DK), Stub(*lead, HK, DK), Stub(*lead, H, DV), Stub(*lead, H), Stub(*lead, H)]


def grads(lead=(B, L), **more):
    g = {"dq": Stub(*lead, HK, DK), "dk": Stub(*lead, HK, DK), "dv": Stub(*lead, H, DV), "dg": Stub(*lead, H), "dbeta": Stub(*lead, H)}
    return dict(g, **more)


def backward(g, **kw):
    return sfm.sfm_gated_delta_bwd(*args(), Stub(B, L, H, DV), grads=g, workspace=Stub(1 << 20, dtype=torch.uint8), stream=SIDE, **kw)


@pytest.mark.parametrize("dh0", [Stub(B, H, DK, 16, dtype=torch.float32), Stub(1, H, DK, DV, dtype=torch.float32),
                                 Stub(B, H, DK, DV), Stub(B, H, DK, DV, dtype=torch.float32, stride=(1, 1, 1, 1))])
@pytest.mark.parametrize("h0", [None, Stub(B, H, DK, DV, dtype=torch.float32)])
def test_a_wrong_dh0_is_refused_with_and_without_h0(calls, dh0, h0):
    with pytest.raises((TypeError, ValueError), match="dh0"):
        backward(grads(dh0=dh0), h0=h0)
    assert not any(n == "sfm_gated_delta_bwd" for n, _ in calls)


def test_dh0_without_h0_counts_in_the_workspace(calls):
    dh0 = Stub(B, H, DK, DV, dtype=torch.float32)
    assert backward(grads(dh0=dh0))["dh0"] is dh0
    size, call = calls
    assert size[0] == "sfm_gated_delta_bwd_ws_size" and size[1][7] == 1
    assert call[0] == "sfm_gated_delta_bwd" and call[1][13] == dh0.at


@pytest.mark.parametrize("lead", [(), (B,), (B, L, 3)])
@pytest.mark.parametrize("back", [False, True])
def test_rows_take_four_dimensions(calls, lead, back):
    """Tensors of another rank were read as far as two of their dimensions, and the rest of the output left as it was."""
    o = Stub(*lead, H, DV)
    with pytest.raises(ValueError, match=r"\[B, L, heads, size\]"):
        if back:
            sfm.sfm_gated_delta_bwd(*args(lead), o, grads=grads(lead), workspace=Stub(1 << 20, dtype=torch.uint8), stream=SIDE)
        else:
            sfm.sfm_gated_delta_fwd(*args(lead), o=o, workspace=Stub(1 << 20, dtype=torch.uint8), stream=SIDE)
    assert not calls


@pytest.mark.parametrize("lead", [(), (3, 2), (3, 1)])
def test_a_step_takes_three_dimensions(calls, lead):
    with pytest.raises(ValueError, match=r"\[R, heads, size\]"):
        sfm.sfm_gated_delta_step(*args(lead), Stub(4, H, DK, DV, dtype=torch.float32), o=Stub(3, H, DV), stream=SIDE)
    assert not calls


def test_values_of_another_rank_are_refused(calls):
    t = args()
    t[2] = Stub(B, L, 1, H, DV)
    with pytest.raises(ValueError, match=r"\[B, L, heads, size\]"):
        sfm.sfm_gated_delta_fwd(*t, o=Stub(B, L, H, DV), workspace=Stub(1 << 20, dtype=torch.uint8), stream=SIDE)


@pytest.mark.parametrize("rows,steps", [(3, (5000, 7, DK, 1)), (3, (5000, 5000, DK, 1)), (1, (7, 7, DK, 1))])
def test_one_token_of_each_row_of_a_projection(calls, rows, steps):
    """X[:, i:i + 1]: tokens are as far apart as the rows, whatever the stride of the dimension of one token says."""
    t = args((rows, 1))
    t[0] = Stub(rows, 1, HK, DK, stride=steps)
    t[2] = Stub(rows, 1, H, DV, stride=(9000, 11, DV, 1))
    sfm.sfm_gated_delta_fwd(*t, o=Stub(rows, 1, H, DV), stream=SIDE)
    (name, a), = calls
    assert name == "sfm_gated_delta_fwd"
    if rows > 1:
        assert a[16:19] == (5000, HK * DK, 9000)
    else:  # one token: any stride that holds its heads
        assert a[16] >= HK * DK and a[18] >= H * DV


@pytest.mark.parametrize("lead,steps", [((3, 1), (0, 7, DK, 1)), ((3, 1), (HK * DK - 1, 1, DK, 1)), ((2, 5), (7 * DK, DK, DK, 1)),
                                        ((2, 5), (0, DK, DK, 1)), ((2, 5), (5 * DK, DK, DK, 2))])
def test_tokens_on_top_of_one_another_or_unevenly_apart_are_refused(calls, lead, steps):
    t = args(lead)
    t[0] = Stub(*lead, HK, DK, stride=steps)
    with pytest.raises(ValueError, match="q: heads must be contiguous"):
        sfm.sfm_gated_delta_fwd(*t, o=Stub(*lead, H, DV), workspace=Stub(1 << 20, dtype=torch.uint8), stream=SIDE)


@pytest.mark.parametrize("max_len", [None, 0])
def test_packed_rows_that_are_all_empty(calls, max_len):
    off = Stub(4, dtype=torch.int32)
    h0 = Stub(3, H, DK, DV, dtype=torch.float32)
    state = Stub(3, H, DK, DV, dtype=torch.float32)
    sfm.sfm_gated_delta_fwd(*args((1, 0)), offsets=off, max_len=max_len, h0=h0, state=state, return_state=True,
                            o=Stub(1, 0, H, DV), stream=SIDE)
    (name, a), = calls
    assert name == "sfm_gated_delta_fwd" and a[9:12] == (3, 1, 0)


@pytest.mark.parametrize("given,asked", [(True, False), (True, True), (False, False)])
def test_a_state_given_is_written(calls, given, asked):
    """Also where it is not asked for as a result."""
    state = Stub(B, H, DK, DV, dtype=torch.float32) if given else None
    o = Stub(B, L, H, DV)
    got = sfm.sfm_gated_delta_fwd(*args(), o=o, state=state, return_state=asked, workspace=Stub(1 << 20, dtype=torch.uint8), stream=SIDE)
    size, call = calls
    assert size[1][6] == given and call[1][7] == (state.at if given else None)
    assert got == (o, state) if asked else got is o


def test_a_wrong_state_is_refused(calls):
    with pytest.raises(ValueError, match="state"):
        sfm.sfm_gated_delta_fwd(*args(), o=Stub(B, L, H, DV), state=Stub(1, H, DK, DV, dtype=torch.float32), stream=SIDE)


@pytest.mark.parametrize("tokens,max_len", [(0, -1), (0, -5), (7, 0), (7, -1)])
def test_a_bound_that_is_none_goes_to_the_library(calls, tokens, max_len):
    """Only rows without a token are taken as rows of one at most: other bounds below 1 are the library's to refuse."""
    sfm.sfm_gated_delta_fwd(*args((1, tokens)), offsets=Stub(4, dtype=torch.int32), max_len=max_len, o=Stub(1, tokens, H, DV), stream=SIDE)
    (name, a), = calls
    assert name == "sfm_gated_delta_fwd" and a[9:12] == (3, max_len, tokens)
