"""Window attention where one of its kernels works at full size: many more CTAs
than the GPU holds at once on tcgen05.  Bounds as in test_gpu_window.py; the
float64 definition is taken for sampled queries and keys, on the GPU."""
import math

import pytest
import torch

from test_gpu_window import TD, U, check, handles, rnd, within  # noqa: F401

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


class Sampled:
    """A handle whose calls run a whole batch; check() sees some of its samples."""

    def __init__(self, h, q, k, v, d, sel, shift=0):
        self.h, self.t, self.d, self.sel, self.shift = h, (q, k, v), d, sel, shift

    def buffer(self, shape, dtype):
        """Off 16-byte boundaries by `shift` elements, NaN all around."""
        b = torch.full((math.prod(shape) + 2 * 64,), math.nan, dtype=dtype, device="cuda")
        self.bufs.append(b)
        return b[64 + self.shift:][:math.prod(shape)].view(shape)

    def window_attention(self, q, k, v, window, want_lse, mask, q_start, **kw):
        self.bufs = []
        (B, Nq, H, _), Dv = self.t[0].shape, self.t[2].shape[3]
        self.o = {"out": self.buffer((B, Nq, H, Dv), q.dtype), "lse": self.buffer((B, H, Nq), torch.float32)}
        self.h.window_attention(*self.t, window, mask=self.mask, q_start=self.start, out=self.o, **kw)
        again = self.h.window_attention(*self.t, window, mask=self.mask, q_start=self.start, want_lse=True, **kw)
        if self.shift == 0:
            assert all(torch.equal(again[x], self.o[x]) for x in self.o)
        return {x: t[self.sel] for x, t in self.o.items()}

    def window_attention_backward(self, q, k, v, out, lse, d, window, mask, q_start, **kw):
        g = {n: self.buffer(t.shape, q.dtype) for n, t in zip("qkv", self.t)}
        args = (*self.t, self.o["out"], self.o["lse"], self.d, window)
        self.h.window_attention_backward(*args, mask=self.mask, q_start=self.start, grads=g, **kw)
        again = self.h.window_attention_backward(*args, mask=self.mask, q_start=self.start, **kw)
        if self.shift == 0:
            assert all(torch.equal(again[x], g[x]) for x in g)
        for b in self.bufs:
            assert b[:64 + self.shift].isnan().all() and b[self.shift - 64:].isnan().all()
        return {x: t[self.sel] for x, t in g.items()}

    def sync_status(self):
        self.h.sync_status()

    mask = start = None


# Calls that window_short.cu takes in both directions: 296 sequences or more (samples
# times key heads) of at most 512 rows and keys that fit half an SM's shared memory.
SHORT = [  # B, Nq, Nk, H, Hkv, D, Dv, left, right, sinks
    (300, 1, 1, 1, 1, 16, 16, 0, 0, 0),
    (40, 31, 31, 8, 8, 16, 16, 5, 0, 2),
    (40, 33, 33, 24, 8, 32, 32, None, None, 0),
    (37, 150, 150, 8, 8, 16, 16, 31, 31, 2),
    (38, 150, 150, 24, 8, 16, 16, 20, 3, 40),
    (40, 33, 33, 24, 8, 64, 64, 8, 8, 1),
    (40, 90, 90, 16, 8, 21, 21, 64, 0, 33),
    (75, 40, 200, 4, 4, 32, 24, 70, 9, 70),
    (300, 2, 100, 2, 1, 64, 40, 50, 0, 5),
    (296, 512, 512, 1, 1, 16, 8, 100, 0, 100),
    (60, 300, 300, 5, 5, 8, 13, 3, 3, 128),
]


def batch(case, seed=0):
    B, Nq, Nk, H, Hkv, D, Dv = case[:7]
    t = torch.bfloat16
    return rnd((B, Nq, H, D), t, seed), rnd((B, Nk, Hkv, D), t, seed + 1), rnd((B, Nk, Hkv, Dv), t, seed + 2), rnd((B, Nq, H, Dv), t, seed + 3)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("case", SHORT, ids=lambda c: "-".join(map(str, c)))
def test_many_short_sequences(handles, case, masked):  # noqa: F811
    """Whole and masked; a whole sample, the sinks, a tail and every other key masked, with NaN and infinities there."""
    B, Nq, Nk, left, right, sinks = case[0], case[1], case[2], *case[7:]
    q, k, v, d = batch(case)
    sel = torch.tensor([0, 1, 2, 3, B // 2, B - 1][:6 if Nk < 400 else 3], device="cuda")
    h = Sampled(handles["bf16"], q, k, v, d, sel)
    if masked:
        h.mask = torch.rand((B, Nk), generator=torch.Generator(device="cuda").manual_seed(8), device="cuda") < 0.6
        h.mask[0, Nk // 3:] = False
        h.mask[1] = False
        h.mask[2, :sinks] = False
        h.mask[3] = torch.arange(Nk, device="cuda") % 2 == 1
        gone = ~h.mask
        for t, rows, bad in ((q, gone[:, -Nq:], math.nan), (k, gone, math.inf), (v, gone, math.nan), (d, gone[:, -Nq:], -math.inf)):
            t[rows] = bad
    check(h, q[sel], k[sel], v[sel], left, right, sinks, mask=h.mask[sel] if masked else None, d_out=d[sel])


@pytest.mark.parametrize("case", [(75, 40, 200, 4, 4, 32, 24, 70, 9, 70), (100, 60, 128, 6, 3, 16, 16, 20, 0, 3), (43, 9, 33, 7, 7, 64, 64, 4, 2, 0)],
                         ids=lambda c: "-".join(map(str, c)))
def test_short_sequences_at_positions_of_their_own(handles, case):  # noqa: F811
    """Chunks of queries anywhere, partly and wholly outside the keys, the ends of int32 among them."""
    B, Nq, Nk, left, right, sinks = case[0], case[1], case[2], *case[7:]
    q, k, v, d = batch(case, 50)
    start = torch.randint(-Nq, Nk, (B,), generator=torch.Generator().manual_seed(9)).int()
    start[:9] = torch.tensor([0, Nk - Nq, Nk // 2, -1, Nk, -Nq, 1 - Nq, 2 ** 31 - 1, -2 ** 31])
    sel = torch.arange(12, device="cuda")
    h = Sampled(handles["bf16"], q, k, v, d, sel)
    h.start = start.cuda()
    check(h, q[sel], k[sel], v[sel], left, right, sinks, q_start=h.start[sel], d_out=d[sel])


@pytest.mark.parametrize("case", [SHORT[3], SHORT[6], SHORT[7]], ids=lambda c: "-".join(map(str, c)))
def test_short_sequences_into_buffers_off_16_bytes(handles, case):  # noqa: F811
    q, k, v, d = batch(case, 60)
    sel = torch.tensor([0, case[0] - 1], device="cuda")
    check(Sampled(handles["bf16"], q, k, v, d, sel, shift=1), q[sel], k[sel], v[sel], *case[7:], d_out=d[sel])


def test_short_sequences_in_a_graph(handles):  # noqa: F811
    h, (q, k, v, d) = handles["bf16"], batch(SHORT[4], 70)
    kw = dict(window=SHORT[4][7:9], sinks=SHORT[4][9])

    def step():
        o = h.window_attention(q, k, v, want_lse=True, **kw)
        return [o["out"], o["lse"], *h.window_attention_backward(q, k, v, o["out"], o["lse"], d, **kw).values()]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in (80, 81):
        for t in (q, k, v, d):
            t.copy_(rnd(t.shape, t.dtype, seed))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_at_the_ends_of_float32(handles, dtype):  # noqa: F811
    """A scale whose product with log2 e is not finite is refused (0 queries would give NaN); the largest that is not, with 0 queries, gives means."""
    from protein_structure_models_b200 import FipaError
    h = handles[dtype]
    q, k, v = (rnd((1, 40, 2, 16), TD[dtype], i) for i in range(3))
    q.zero_()
    for scale in (3e38, 2.4e38, math.nan, 1e-46, 0.0):
        with pytest.raises(FipaError) as e:
            h.window_attention(q, k, v, (5, 5), scale=scale)
        assert e.value.status == 1
    for scale in (2.3e38, 1e-30):
        check(h, q, k, v, 5, 5, 1, scale=scale, backward=False)
