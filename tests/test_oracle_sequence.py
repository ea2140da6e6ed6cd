"""The float64 definitions of the sequence operators: gradients against
differences and autograd, visibility against the rule read key by key."""
import pytest
import torch

from oracle import sequence as seq

D64 = torch.float64


def rnd(*shape, seed=0):
    return torch.randn(*shape, dtype=D64, generator=torch.Generator().manual_seed(seed))


def differences(f, x, d, h=1e-6):
    """<d, f(x + h e) - f(x - h e)> / 2h for every element e of x."""
    g = torch.zeros_like(x)
    for e in range(x.numel()):
        a, b = x.clone(), x.clone()
        a.view(-1)[e] += h
        b.view(-1)[e] -= h
        g.view(-1)[e] = ((f(a) - f(b)) * d).sum() / (2 * h)
    return g


@pytest.mark.parametrize("left,right,sinks", [(2, 0, 0), (1, 1, 2), (None, 0, 0), (0, 0, 3), (2, None, 1), (0, 3, 9)])
def test_visible_is_the_rule(left, right, sinks):
    B, Nq, Nk = 3, 4, 7
    mask = torch.rand(B, Nk, generator=torch.Generator().manual_seed(1)) < 0.7
    start = torch.tensor([-2, 3, 6], dtype=torch.int32)
    ok = seq.visible(B, Nq, Nk, left, right, sinks, mask, start)
    for b in range(B):
        for i in range(Nq):
            p = int(start[b]) + i
            for j in range(Nk):
                want = 0 <= p < Nk and bool(mask[b, p]) and bool(mask[b, j])
                want &= right is None or j <= p + right
                want &= left is None or j >= p - left or j < sinks
                assert bool(ok[b, i, j]) == want


def test_window_gradients_are_differences():
    q, k, v, d = rnd(2, 3, 4, 3), rnd(2, 5, 2, 3, seed=1), rnd(2, 5, 2, 2, seed=2), rnd(2, 3, 4, 2, seed=3)
    kw = dict(left=1, right=1, sinks=1, mask=torch.tensor([[1, 1, 0, 1, 1], [1, 0, 1, 1, 0]]).bool())
    g = seq.window_attention_backward(q, k, v, d, **kw)
    for name, x, f in (("q", q, lambda t: seq.window_attention(t, k, v, **kw)["out"]),
                       ("k", k, lambda t: seq.window_attention(q, t, v, **kw)["out"]),
                       ("v", v, lambda t: seq.window_attention(q, k, t, **kw)["out"])):
        torch.testing.assert_close(g[name], differences(f, x, d), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("kind,gate,post,masked", [("layer", True, True, True), ("rms", False, True, False),
                                                   ("layer", True, False, False), ("rms", True, True, True)])
def test_norm_gradients_are_differences(kind, gate, post, masked):
    n, C = 3, 5
    t = {"s": rnd(n, C), "u": rnd(n, C, seed=1), "res_scale": rnd(C, seed=3), "pre_w": rnd(C, seed=4), "pre_b": rnd(C, seed=5)}
    if gate:
        t["gate"] = rnd(n, C, seed=2)
    if post:
        t["post_w"], t["post_b"] = rnd(C, seed=6), rnd(C, seed=7)
    mask = torch.tensor([True, False, True]) if masked else None
    dr, dx = rnd(n, C, seed=8), rnd(n, C, seed=9)

    def args(t):
        return dict(gate=t.get("gate"), res_scale=t["res_scale"], post=(t["post_w"], t["post_b"]) if post else None,
                    pre=(t["pre_w"], t["pre_b"]), mask=mask, norm_kind=kind)

    g = seq.norm_residual_backward(t["s"], t["u"], dr, dx, **args(t))
    for name in t:
        def f(x):
            w = {**t, name: x}
            o = seq.norm_residual(w["s"], w["u"], **args(w))
            return torch.cat([o["r"], o["x"]])
        torch.testing.assert_close(g[name], differences(f, t[name], torch.cat([dr, dx])), rtol=1e-5, atol=1e-7)


def test_embedding_gradient_is_differences():
    idx = torch.tensor([2, -1, 0, 2, 4, 5], dtype=torch.int32)
    tab, d = rnd(5, 3), rnd(6, 3, seed=1)
    torch.testing.assert_close(seq.embedding_backward(idx, d, 5, 1.5),
                               differences(lambda x: seq.embedding(idx, x, 1.5), tab, d), rtol=1e-6, atol=1e-8)
    assert torch.equal(seq.embedding(idx, tab)[[1, 5]], torch.zeros(2, 3, dtype=D64))
