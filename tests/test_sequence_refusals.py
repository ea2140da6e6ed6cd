"""Refusals of the sequence operators' C entry points that need no GPU: invalid
calls return a status before anything is launched."""
import ctypes

import pytest

P = 0x1000          # an address that is never read


@pytest.fixture(scope="module")
def lib():
    from protein_structure_models_b200 import build, fipa
    build.build()
    return fipa.load_library()


def dims(rows=4, C=16, s=0, b=0, norm=0, eps=1e-5):
    from protein_structure_models_b200.fipa import FipaNormDims
    return FipaNormDims(rows, C, s, b, norm, eps)


def inputs(**kw):
    from protein_structure_models_b200.fipa import FipaNormInputs
    return FipaNormInputs(**({"s": P, "u": P} | kw))


@pytest.mark.parametrize("d,i,status", [
    (dict(rows=-1), {}, 1), (dict(C=0), {}, 1), (dict(C=8193), {}, 2), (dict(s=2), {}, 1), (dict(b=-1), {}, 1),
    (dict(norm=2), {}, 1), (dict(eps=0.0), {}, 1), (dict(eps=float("inf")), {}, 1), (dict(), dict(s=None), 1),
    (dict(), dict(u=None), 1), (dict(), dict(u=None, gate=P, pre_w=P), 1), (dict(), dict(post_b=P), 1),
    (dict(), dict(pre_b=P), 1), (dict(), dict(s=P + 2), 1), (dict(b=1), dict(u=P + 1), 1), (dict(), dict(res_scale=P + 1), 1)])
def test_norm_residual(lib, d, i, status):
    assert lib.fipa_norm_residual(dims(**d), inputs(**i), P, None, None, None) == status


def test_norm_residual_outputs_and_backward(lib):
    from protein_structure_models_b200.fipa import FipaNormGrads
    assert lib.fipa_norm_residual(None, inputs(), P, None, None, None) == 1
    assert lib.fipa_norm_residual(dims(), None, P, None, None, None) == 1
    assert lib.fipa_norm_residual(dims(), inputs(), None, None, None, None) == 1               # r missing
    assert lib.fipa_norm_residual(dims(), inputs(pre_w=P), P, None, None, None) == 1           # x missing
    assert lib.fipa_norm_residual(dims(), inputs(), P, P, None, None) == 1                     # x without pre_w
    assert lib.fipa_norm_residual(dims(), inputs(), P, None, P + 4, None) == 1                 # stats off 16 bytes
    n = ctypes.c_size_t()
    assert lib.fipa_norm_residual_backward_workspace_size(dims(), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.fipa_norm_residual_backward_workspace_size(dims(C=9000), ctypes.byref(n)) == 2
    bwd = lambda g, ws=P, size=1 << 30, stats=P, dx=None: lib.fipa_norm_residual_backward(  # noqa: E731
        dims(), inputs(), stats, P, dx, g, ws, size, None)
    assert bwd(None) == 1
    assert bwd(FipaNormGrads(), stats=None) == 1
    assert bwd(FipaNormGrads(), dx=P) == 1                       # d_x without pre_w
    assert bwd(FipaNormGrads(gate=P)) == 1
    assert bwd(FipaNormGrads(pre_w=P)) == 1
    assert bwd(FipaNormGrads(s=P + 2)) == 1
    assert bwd(FipaNormGrads(), ws=None) == 3
    assert bwd(FipaNormGrads(), size=8) == 3
    assert bwd(FipaNormGrads(), ws=P + 16) == 1


def test_embedding(lib):
    call = lambda dt=0, idx=P, tab=P, T=4, V=5, C=8, sc=1.0, out=P: lib.fipa_embedding(dt, idx, tab, T, V, C, sc, out, None)  # noqa: E731
    assert call(T=0) == 0
    for bad in (dict(dt=2), dict(idx=None), dict(tab=None), dict(out=None), dict(T=-1), dict(V=0), dict(C=0),
                dict(sc=float("nan")), dict(sc=1e300), dict(idx=P + 2), dict(tab=P + 2), dict(out=P + 1)):
        assert call(**bad) == 1, bad
    for big in (dict(T=2 ** 30 + 1), dict(C=65537), dict(V=2 ** 30 + 1)):
        assert call(**big) == 2, big
    n = ctypes.c_size_t()
    assert lib.fipa_embedding_backward_workspace_size(100, 5, 8, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.fipa_embedding_backward_workspace_size(100, 5, 8, None) == 1
    bwd = lambda d=P, g=P, ws=P, size=1 << 30: lib.fipa_embedding_backward(0, P, d, 4, 5, 8, 1.0, g, ws, size, None)  # noqa: E731
    assert bwd(d=None) == 1 and bwd(g=None) == 1 and bwd(g=P + 1) == 1 and bwd(ws=P + 128) == 1
    assert bwd(ws=None) == 3 and bwd(size=64) == 3


def test_window_attention_without_a_handle(lib):
    from protein_structure_models_b200.fipa import FipaHeads, FipaWindow
    w, t, n = FipaWindow(1, 1, 1, 1, 1, 8, 8, 1, 1, 0, 1.0), FipaHeads(P, 8, 8, 8), ctypes.c_size_t()
    assert lib.fipa_window_attention(None, t, t, t, None, None, w, P, None, None, 0, None) == 1
    assert lib.fipa_window_attention_backward(None, t, t, t, None, None, w, P, P, P, P, P, P, P, 1 << 20, None) == 1
    assert lib.fipa_window_attention_workspace_size(None, t, t, t, w, ctypes.byref(n)) == 1
    assert lib.fipa_window_attention_backward_workspace_size(None, t, t, t, w, ctypes.byref(n)) == 1


@pytest.mark.parametrize("eps", [1e-46, 1e-300, -1e-5, float("nan"), 1e39])
def test_norm_residual_eps_that_float32_does_not_hold(lib, eps):
    """An eps that float32 rounds to 0 would make a constant row 0 / 0."""
    assert lib.fipa_norm_residual(dims(eps=eps), inputs(), P, None, None, None) == 1
