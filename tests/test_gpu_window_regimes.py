"""Window attention where one of its kernels works at full size: many more CTAs
than the GPU holds at once on tcgen05.  Bounds as in test_gpu_window.py; the
float64 definition is taken for sampled queries and keys, on the GPU."""
import math

import pytest
import torch

from test_gpu_window import TD, U, handles, rnd, within  # noqa: F401

pytestmark = pytest.mark.gpu


def spread(q, k, every, step):
    """Scores whose running maximum moves by more than 2^8 at every tile of 64 keys, for
    the queries at `every` only: a channel in which those queries are large and the keys
    climb a staircase of 64 keys a step, back to 0 every 1024."""
    N = q.shape[1]
    j = torch.arange(N, device="cuda")
    q[..., 0] = torch.where(every, step * math.sqrt(q.shape[3]), 0.0)[None, :, None].to(q.dtype)
    k[..., 0] = (j % 1024 // 64)[None, :, None].to(k.dtype)


def dense(q, k, v, d, rows, left, right, sinks):
    """Float64 quantities of the queries at positions `rows` of one sample (Nq = Nk): [H, rows, N]."""
    H, Hkv, D = q.shape[2], k.shape[2], q.shape[3]
    x = lambda t, r=slice(None): t[0, r].double().permute(1, 0, 2).repeat_interleave(H // t.shape[2], 0)  # noqa: E731
    Q, K, V, dO = x(q, rows), x(k), x(v), x(d, rows)
    p, j = rows[:, None], torch.arange(k.shape[1], device="cuda")[None]
    ok = (j <= p + right) & ((j >= p - left) | (j < sinks))
    sc = D ** -0.5
    S = (Q @ K.transpose(1, 2) * sc).masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(S, -1)
    P = torch.exp(S - lse[..., None])
    O = P @ V
    dS = P * (dO @ V.transpose(1, 2) - (dO * O).sum(-1, keepdim=True))
    u, Dv, n = U[q.dtype], v.shape[3], ok.sum(-1).double()[None, :, None]
    es = torch.where(ok, (D + 6) * 2.0 ** -23 * sc * (Q.abs() @ K.abs().transpose(1, 2)) + S.abs() * 2.0 ** -22 + 2.0 ** -20, 0.0)
    ep = 2 * es.amax(-1, keepdim=True)
    pv = P @ V.abs()
    edel = (2 * u + ep + n * 2.0 ** -23) * (dO.abs() * pv).sum(-1, keepdim=True)
    eds = dS.abs() * (ep + u) + P * (edel + (Dv + 6) * 2.0 ** -23 * (dO.abs() @ V.abs().transpose(1, 2)))
    return dict(Q=Q, K=K, V=V, dO=dO, P=P, O=O, lse=lse, dS=dS, ok=ok, sc=sc, u=u, n=n, ep=ep, pv=pv, eds=eds)


@pytest.mark.parametrize("N,H,Hkv,D,left,right,sinks", [(16384, 8, 2, 64, 511, 0, 4), (32768, 4, 4, 128, 255, 64, 0), (24576, 6, 6, 32, 300, 100, 9)])
def test_many_ctas_whose_warps_drift_apart(handles, N, H, Hkv, D, left, right, sinks):  # noqa: F811
    """Over a thousand CTAs of 128 rows; of their four finishing warps one rescales its sums at every tile, the
    others never do, so that they run tiles apart.  A hundred calls give the same bits, and sampled rows the definition's."""
    h, t = handles["bf16"], torch.bfloat16
    q, k, v, d = (rnd((1, N, x, D), t, 5 + i) for i, x in enumerate((H, Hkv, Hkv, H)))
    G = H // Hkv
    spread(q, k, torch.arange(N, device="cuda") * G // 32 % 4 == 2, 8.0)
    assert Hkv * (N * G // 128) >= 1000
    kw = dict(window=(left, right), sinks=sinks)
    first = h.window_attention(q, k, v, want_lse=True, **kw)
    for _ in range(100):
        again = h.window_attention(q, k, v, want_lse=True, **kw)
        assert torch.equal(again["out"], first["out"]) and torch.equal(again["lse"], first["lse"])
    g = h.window_attention_backward(q, k, v, first["out"], first["lse"], d, **kw)
    for _ in range(10):
        again = h.window_attention_backward(q, k, v, first["out"], first["lse"], d, **kw)
        assert all(torch.equal(again[x], g[x]) for x in g)
    h.sync_status()
    assert all(torch.isfinite(x).all() for x in (first["out"], first["lse"], *g.values()))
    rows = torch.unique(torch.cat([torch.tensor([0, 1, 63, left, N - 1]), torch.randint(0, N, (60,), generator=torch.Generator().manual_seed(3))])).cuda()
    x = dense(q, k, v, d, rows, left, right, sinks)
    u, row = x["u"], lambda t: t.permute(1, 0, 2).cpu()  # noqa: E731
    within(first["out"][0, rows], row(x["O"]), row(u * x["O"].abs() + (u + x["ep"] + x["n"] * 2.0 ** -23) * x["pv"]), "out")
    within(first["lse"][0, :, rows], x["lse"].cpu(), (x["ep"][..., 0] + x["lse"].abs() * 2.0 ** -22 + 2.0 ** -20).cpu(), "lse")
    dq = x["sc"] * x["dS"] @ x["K"]
    within(g["q"][0, rows], row(dq), row(u * dq.abs() + x["sc"] * (x["eds"] + x["n"] * 2.0 ** -23 * x["dS"].abs()) @ x["K"].abs() + 1e-30), "d_q")
    for j in (sinks, 700, 5000, N - left - 1, N - 1):                # keys that only their window's queries see
        rows = torch.arange(max(0, j - right), min(N, j + left + 1), device="cuda")
        x = dense(q, k, v, d, rows, left, right, sinks)
        fold = lambda t: t.view(Hkv, G, D).sum(1).cpu()  # noqa: E731
        P, dS, eds, n = x["P"][..., j], x["dS"][..., j], x["eds"][..., j], len(rows) * G
        dv, dk = torch.einsum("hr,hrd->hd", P, x["dO"]), torch.einsum("hr,hrd->hd", x["sc"] * dS, x["Q"])
        ev = torch.einsum("hr,hrd->hd", P * (u + x["ep"][..., 0] + n * 2.0 ** -23), x["dO"].abs())
        ek = torch.einsum("hr,hrd->hd", x["sc"] * (eds + n * 2.0 ** -23 * dS.abs()), x["Q"].abs())
        within(g["v"][0, j], fold(dv), u * fold(dv).abs() + fold(ev) + 1e-30, f"d_v of key {j}")
        within(g["k"][0, j], fold(dk), u * fold(dk).abs() + fold(ek) + 1e-30, f"d_k of key {j}")
