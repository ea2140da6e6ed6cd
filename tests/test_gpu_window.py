"""Window attention with sinks (through the C ABI) against its float64
definition (oracle/sequence.py), forward and backward.

Tolerances are first-order error bounds, element by element.  With u the half
step of the tensors' type (bf16 2^-8, f32 2^-24) and n the number of terms:
  e_s   score: (D + 6) 2^-23 sum|q k| scale + |s| 2^-22 + 2^-20 (float32 sums, exp2 argument)
  e_p   relative error of a probability: e_s of the score plus that of lse <= 2 max e_s
  out   u |out| + (u + e_p + n 2^-23) sum p |v|   (p goes into the product in the tensors' type)
  delta (2 u + e_p + n 2^-23) sum |d_out| (sum p |v|)    (from the rounded out)
  ds    |ds| (e_p + u) + p (e_delta + (Dv + 6) 2^-23 sum |d_out v|)
  d_q   u |d_q| + scale sum (e_ds + n 2^-23 |ds|) |k|;  d_k, d_v likewise."""
import math

import pytest
import torch

from oracle import sequence as seq

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def handles():
    from protein_structure_models_b200 import Fipa, build
    build.build()
    h = {t: Fipa(t, 0) for t in TD}
    yield h
    for x in h.values():
        x.close()


def rnd(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def within(got, want, tol, name):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), name
    over = (got - want).abs() - tol
    assert (over <= 0).all(), f"{name}: off by {(got - want).abs().max():.3e}, {(over > 0).sum()} of {over.numel()} beyond " \
        f"the bound, worst {((got - want).abs() / tol.clamp(min=1e-300)).max():.2f} bounds"


def back(x):
    return x.permute(0, 2, 1, 3)


def check(h, q, k, v, left, right, sinks=0, mask=None, q_start=None, scale=None, d_out=None, seed=99, backward=True):
    """Runs both directions and holds every element to its bound; returns the results."""
    t, u = q.dtype, U[q.dtype]
    D, Dv = q.shape[3], v.shape[3]
    kw = dict(sinks=sinks, mask=mask, q_start=q_start, scale=scale)
    got = h.window_attention(q, k, v, (left, right), want_lse=True, **kw)
    d_out = rnd(got["out"].shape, t, seed) if d_out is None else d_out
    g = h.window_attention_backward(q, k, v, got["out"], got["lse"], d_out, (left, right), **kw) if backward else {}
    h.sync_status()
    lo, ri = (None if w is None or w < 0 else w for w in (left, right))
    b = seq.window_attention_backward(q, k, v, d_out, lo, ri, sinks, mask, q_start, scale)
    f, sc = b["f"], b["scale"]
    P, ok = f["P"], f["ok"]
    nk, nq = ok.sum(-1, keepdim=True).double(), ok.sum(-2).double()
    es = torch.where(ok, (D + 6) * 2.0 ** -23 * sc * (f["Q"].abs() @ f["K"].abs().transpose(-1, -2)) +
                     f["S"].abs() * 2.0 ** -22 + 2.0 ** -20, 0.0)
    ep = 2 * es.amax(-1, keepdim=True)
    pv = P @ f["V"].abs()
    within(got["out"], f["out"], u * f["out"].abs() + back((u + ep + nk * 2.0 ** -23) * pv) + 1e-30, "out")
    lse = got["lse"].cpu().double()
    empty = f["lse"] == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    within(lse.masked_fill(empty, 0), f["lse"].masked_fill(empty, 0), ep[..., 0] + f["lse"].masked_fill(empty, 0).abs() * 2.0 ** -22 +
           2.0 ** -20, "lse")
    if backward:
        dO = b["dO"]
        edel = (2 * u + ep + nk * 2.0 ** -23) * (dO.abs() * pv).sum(-1, keepdim=True)
        eds = b["dS"].abs() * (ep + u) + P * (edel + (Dv + 6) * 2.0 ** -23 * (dO.abs() @ f["V"].abs().transpose(-1, -2)))
        within(g["q"], b["q"], u * b["q"].abs() + back(sc * (eds + nk * 2.0 ** -23 * b["dS"].abs()) @ f["K"].abs()) + 1e-30, "d_q")
        n = nq[..., None, :] * (q.shape[2] // k.shape[2])
        kq = (sc * (eds + n * 2.0 ** -23 * b["dS"].abs())).transpose(-1, -2) @ f["Q"].abs()
        within(g["k"], b["k"], u * b["k"].abs() + b["fold"](kq) + 1e-30, "d_k")
        within(g["v"], b["v"], u * b["v"].abs() + b["fold"]((P * (u + ep + n * 2.0 ** -23)).transpose(-1, -2) @ dO.abs()) + 1e-30, "d_v")
    return got, g


def make(dtype, B, Nq, Nk, H, Hkv, D, Dv, seed=0):
    t = TD[dtype]
    return rnd((B, Nq, H, D), t, seed), rnd((B, Nk, Hkv, D), t, seed + 1), rnd((B, Nk, Hkv, Dv), t, seed + 2)


CASES = [  # B, Nq, Nk, H, Hkv, D, Dv, left, right, sinks
    (1, 1, 1, 1, 1, 1, 1, 0, 0, 0),
    (2, 5, 5, 2, 1, 3, 5, 1, 0, 0),
    (1, 64, 64, 2, 2, 16, 16, 15, 0, 2),
    (2, 65, 65, 4, 2, 32, 32, 20, 7, 1),
    (1, 127, 127, 3, 3, 24, 40, 200, 200, 5),
    (1, 129, 300, 6, 2, 64, 64, 31, 0, 4),
    (2, 150, 150, 8, 8, 16, 16, 31, 31, 2),
    (1, 333, 333, 4, 1, 64, 64, 100, 3, 65),
    (1, 700, 700, 4, 4, 32, 32, None, 0, 0),
    (1, 700, 700, 2, 2, 128, 128, None, None, 0),
    (1, 1000, 1000, 4, 1, 64, 48, 127, 0, 128),
    (1, 1030, 1030, 2, 2, 20, 128, 40, 90, 3),
    (3, 17, 800, 6, 2, 72, 8, 300, 5, 4),
    (1, 2100, 2100, 1, 1, 8, 8, 0, 0, 1),
    (1, 900, 900, 8, 1, 64, 64, 255, 0, 4),
    (1, 520, 520, 14, 2, 64, 64, 64, 64, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_definition(handles, dtype, case):
    B, Nq, Nk, H, Hkv, D, Dv, left, right, sinks = case
    q, k, v = make(dtype, B, Nq, Nk, H, Hkv, D, Dv)
    check(handles[dtype], q, k, v, left, right, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 21])
@pytest.mark.parametrize("N,left,right,sinks", [(150, 31, 31, 2), (300, 64, 0, 4), (260, None, None, 0), (600, 3, 3, 100)])
def test_masks_leave_rows_and_samples_empty(handles, dtype, D, N, left, right, sinks):
    """Padding, holes, masked sinks, a whole sample masked; NaN and infinities in the masked places are never used."""
    B, H, Hkv = 4, 4, 2
    q, k, v = make(dtype, B, N, N, H, Hkv, D, D, 7)
    mask = torch.rand((B, N), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda") < 0.6
    mask[0, N // 3:] = False
    mask[1, :sinks] = False
    mask[2] = False
    mask[3, 40:160] = False
    d = rnd((B, N, H, D), TD[dtype], 11)
    for t, bad in ((q, math.nan), (k, math.inf), (v, math.nan), (d, -math.inf)):
        t[~mask] = bad
    out, g = check(handles[dtype], q, k, v, left, right, sinks, mask=mask, d_out=d)
    assert (out["out"][~mask] == 0).all()
    for x in g.values():
        assert (x[~mask] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq,Nk", [(1, 1), (1, 70), (1, 2000), (3, 500), (5, 1100), (16, 400), (200, 333)])
@pytest.mark.parametrize("H,Hkv,D", [(8, 8, 32), (16, 4, 64), (6, 2, 20), (7, 1, 128)])
def test_tokens_against_a_cache(handles, dtype, Nq, Nk, H, Hkv, D):
    """Single tokens and chunks at positions of their own, some of them outside the cache."""
    B = 6
    q, k, v = make(dtype, B, Nq, Nk, H, Hkv, D, D, 3)
    start = torch.tensor([0, Nk - Nq, Nk // 2, -1, Nk, -Nq - 5], dtype=torch.int32, device="cuda")
    for left, sinks in ((63, 4), (700, 0), (None, 0), (0, 1)):
        check(handles[dtype], q, k, v, left, 0, sinks, q_start=start, backward=Nq in (3, 200))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq,Nk,H,Hkv,D", [(1, 300, 8, 8, 64), (3, 290, 6, 2, 20), (22, 203, 16, 8, 32), (100, 400, 2, 2, 16), (5, 70, 4, 4, 32)])
def test_tokens_of_a_padded_batch(handles, dtype, Nq, Nk, H, Hkv, D):
    """The last tokens of samples of several lengths: those behind a sample's end see nothing, though all their columns may be valid."""
    q, k, v = make(dtype, 5, Nq, Nk, H, Hkv, D, D, 21)
    ends = torch.tensor([Nk, Nk - Nq, Nk - Nq // 2, Nk - Nq - 16, 0], device="cuda")
    mask = torch.arange(Nk, device="cuda")[None] < ends[:, None]
    for left, sinks in ((Nk, 0), (180, 1), (20, 4)):
        got, _ = check(handles[dtype], q, k, v, left, 0, sinks, mask=mask)
        assert (got["out"][~mask[:, -Nq:]] == 0).all()


@pytest.mark.parametrize("big", [2 ** 31 - 1, -2 ** 31])
def test_start_positions_at_the_ends_of_int32(handles, big):
    q, k, v = make("bf16", 2, 4, 50, 2, 2, 16, 16)
    start = torch.tensor([big, 20], dtype=torch.int32, device="cuda")
    got, g = check(handles["bf16"], q, k, v, 10, 3, 2, q_start=start)
    assert (got["out"][0] == 0).all() and (g["q"][0] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,shift", [(32, 0), (32, 1), (33, 0), (64, 4)])
def test_strided_heads(handles, dtype, D, shift):
    """Slices of one fused projection, at aligned and odd offsets, and head-major storage."""
    B, N, H, Hkv = 2, 140, 4, 2
    buf = rnd((B, N, (H + 2 * Hkv) * D + shift + 3), TD[dtype], 21)
    x = buf[:, :, shift:shift + (H + 2 * Hkv) * D].unflatten(2, (H + 2 * Hkv, D))
    q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
    check(handles[dtype], q, k, v, 30, 10, 3)
    check(handles[dtype], *[t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (q, k, v)], 30, 10, 3)


def test_a_cache_beyond_32_bit_offsets(handles):
    """Keys and values whose element offsets pass 2^31, in the batch and in the position."""
    buf = torch.empty(2 ** 31 + 2 ** 25, dtype=torch.bfloat16, device="cuda")
    B, Nk, D = 2, 260, 32
    k = buf.as_strided((B, Nk, 1, D), (2 ** 31 + 64, D, D, 1))
    k.copy_(rnd(k.shape, torch.bfloat16, 1))
    q, v = rnd((B, 1, 4, D), torch.bfloat16, 2), rnd((B, Nk, 1, D), torch.bfloat16, 3)
    check(handles["bf16"], q, k, v, 100, 0, 4)
    del k
    k = buf.as_strided((1, Nk, 1, D), (0, 2 ** 23 + 64, D, 1))
    k.copy_(rnd(k.shape, torch.bfloat16, 4))
    check(handles["bf16"], rnd((1, Nk, 4, D), torch.bfloat16, 5), k, rnd((1, Nk, 1, D), torch.bfloat16, 6), 100, 20, 4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(handles, dtype):
    """Scores of several hundred: the running maximum moves and the first keys' weight vanishes."""
    q, k, v = make(dtype, 1, 400, 400, 2, 2, 64, 64, 31)
    k = (k * torch.linspace(0.1, 8, 400, device="cuda")[None, :, None, None]).to(k.dtype)
    check(handles[dtype], q * 4, k, v, 200, 0, 4)
    check(handles[dtype], q, k, v, 200, 100, 4, scale=3.0)


def test_repeats_are_identical_and_graphs_replay(handles):
    """Deterministic; one captured pass on another stream, replayed on new inputs, gives the eager result."""
    h = handles["bf16"]
    q, k, v = make("bf16", 2, 300, 300, 8, 2, 64, 64, 41)
    d = rnd((2, 300, 8, 64), torch.bfloat16, 44)
    kw = dict(window=(100, 10), sinks=3)

    def step():
        o = h.window_attention(q, k, v, want_lse=True, **kw)
        return o["out"], *h.window_attention_backward(q, k, v, o["out"], o["lse"], d, **kw).values()

    want = [x.clone() for x in step()]
    assert all(torch.equal(a, b) for a, b in zip(want, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    keep = [x.clone() for x in (q, k, v)]
    for x in (q, k, v):
        x.normal_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(res, step()))
    for x, y in zip((q, k, v), keep):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(res, want))


def test_only_the_outputs_are_written(handles):
    """Buffers behind the outputs and the workspace keep what they held."""
    h = handles["bf16"]
    q, k, v = make("bf16", 1, 77, 400, 4, 2, 24, 40, 51)
    kw = dict(window=(20, 0), sinks=5)

    def guarded(shape, dtype):
        n = math.prod(shape)
        b = torch.full((n + 512,), 7, dtype=dtype, device="cuda")
        return b, b[256:256 + n].view(shape)

    bo, out = guarded((1, 77, 4, 40), torch.bfloat16)
    bl, lse = guarded((1, 4, 77), torch.float32)
    h.window_attention(q, k, v, out={"out": out, "lse": lse}, **kw)
    bufs = [bo, bl]
    grads = {}
    for name, t in (("q", q), ("k", k), ("v", v)):
        b, grads[name] = guarded(t.shape, torch.bfloat16)
        bufs.append(b)
    need = h.window_attention_backward_workspace_size(q, k, v, **kw)
    ws = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    h.window_attention_backward(q, k, v, out, lse, rnd(out.shape, torch.bfloat16, 5), workspace=ws[256:256 + need], grads=grads, **kw)
    h.sync_status()
    for b in bufs + [ws]:
        assert (b[:256] == 7).all() and (b[-256:] == 7).all()


def test_refusals(handles):
    from protein_structure_models_b200 import FipaError
    h = handles["bf16"]
    q, k, v = make("bf16", 1, 4, 8, 2, 2, 16, 16)

    def refused(status, *a, **kw):
        with pytest.raises(FipaError) as e:
            h.window_attention(*a, **kw)
        assert e.value.status == status

    refused(1, q, k, v, (1, 1), sinks=-1)
    refused(1, q, k, v, (1, 1), scale=math.inf)
    refused(1, q, k, v, (1, 1), scale=-1.0)
    refused(2, q, k, v, (1, 1), sinks=129)
    refused(1, *make("bf16", 1, 4, 8, 3, 2, 16, 16), (1, 1))
    refused(1, *make("bf16", 1, 0, 8, 2, 2, 16, 16), (1, 1))
    refused(2, *make("bf16", 1, 4, 8, 2, 2, 129, 16), (1, 1))
    refused(2, *make("bf16", 1, 4, 8, 2, 2, 16, 136), (1, 1))
    with pytest.raises(ValueError):
        h.window_attention(q.float(), k, v, (1, 1))
    with pytest.raises(ValueError):
        h.window_attention(q, k[:, :7], v, (1, 1))
    with pytest.raises(ValueError):
        h.window_attention(q[..., ::2], k[..., ::2], v, (1, 1))
    with pytest.raises(ValueError):
        h.window_attention(q, k, v, (1, 1), mask=torch.ones(1, 7, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        h.window_attention(q, k, v, (1, 1), q_start=torch.zeros(1, dtype=torch.int64, device="cuda"))
    o = h.window_attention(q, k, v, (1, 1), want_lse=True)
    with pytest.raises(FipaError) as e:
        h.window_attention_backward(q, k, v, o["out"], o["lse"], o["out"], (1, 1),
                                    workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    odd = make("bf16", 1, 256, 256, 2, 2, 17, 16)
    assert h.window_attention_workspace_size(q, k, v, (1, 1)) == 0 < h.window_attention_workspace_size(*odd, (1, 1))
    with pytest.raises(FipaError) as e:
        h.window_attention(*odd, (1, 1), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(FipaError) as e:
        h.window_attention_backward(q, k, v, o["out"], o["lse"], rnd((129,), torch.bfloat16, 3)[1:].view(o["out"].shape), (1, 1))
    assert e.value.status == 1
    h.sync_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["width", "value width", "stride", "address"])
def test_off_16_byte_boundaries_as_on_them(handles, dtype, what):
    """Each way to be off 16-byte boundaries, with garbage beside and behind the
    tensors, a window far from most keys, and guarded buffers and workspaces."""
    h, td = handles[dtype], torch.bfloat16 if dtype == "bf16" else torch.float32
    B, Nq, Nk, H, Hkv = 2, 70, 301, 4, 2
    D, Dv = {"width": (21, 16), "value width": (16, 13)}.get(what, (16, 24))
    q, k, v = make(dtype, B, Nq, Nk, H, Hkv, D, Dv, 71)

    def moved(t):
        if what == "stride":
            w = torch.full((*t.shape[:3], t.shape[3] + 1), math.nan, dtype=td, device="cuda")[..., :t.shape[3]]
        else:
            w = torch.full((t.numel() + 2,), math.nan, dtype=td, device="cuda")[1 if what == "address" else 0:][:t.numel()].view(t.shape)
        return w.copy_(t)

    start = torch.tensor([231, 5], dtype=torch.int32, device="cuda")
    kw = dict(window=(9, 2), sinks=3, q_start=start)
    mq, mk, mv = moved(q), moved(k), moved(v)
    d = rnd((B, Nq, H, Dv), td, 72)
    o, g = check(h, mq, mk, mv, 9, 2, 3, q_start=start, d_out=d)
    room, bufs = [], []
    for size in (h.window_attention_workspace_size, h.window_attention_backward_workspace_size):
        n = size(mq, mk, mv, kw["window"], 3)
        bufs.append(torch.full((n + 512,), 0xff, dtype=torch.uint8, device="cuda"))       # NaN wherever nothing is written
        room.append(bufs[-1][256:256 + n])
    o2 = h.window_attention(mq, mk, mv, want_lse=True, workspace=room[0], **kw)
    g2 = h.window_attention_backward(mq, mk, mv, o["out"], o["lse"], d, workspace=room[1], **kw)
    assert all(torch.equal(a, b) for x, y in ((o, o2), (g, g2)) for a, b in zip(x.values(), y.values()))
    for w in bufs:
        assert (w[:256] == 0xff).all() and (w[-256:] == 0xff).all()
    h.sync_status()


def test_a_closed_handle():
    from protein_structure_models_b200 import Fipa, FipaError
    h = Fipa("bf16", 0)
    h.close()
    with pytest.raises(FipaError) as e:
        h.window_attention(*make("bf16", 1, 4, 8, 2, 2, 16, 16), (1, 1))
    assert e.value.status == 1


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 37), ("f32", 24), ("f32", 19)])
def test_captured_together_and_replayed(handles, dtype, D):
    """Two calls of different sizes in one graph, with temporaries of the graph's pool; replayed on new inputs."""
    h = handles[dtype]
    q, k, v = make(dtype, 1, 200, 300, 4, 2, D, D, 81)
    d = rnd(q.shape, TD[dtype], 82)
    kw = dict(window=(50, 0), sinks=4)

    def both():
        o = h.window_attention(q, k, v, want_lse=True, **kw)
        g = h.window_attention_backward(q, k, v, o["out"], o["lse"], d, **kw)
        p = h.window_attention(q[:, :1], k, v, **kw)
        return [o["out"], o["lse"], g["q"], g["k"], g["v"], p["out"]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for seed in (90, 91):
        for i, t in enumerate((q, k, v, d)):
            t.copy_(rnd(t.shape, t.dtype, seed + 10 * i))
        graph.replay()
        want = both()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_on_another_stream_with_its_own_allocations(handles):
    """A call on a side stream whose temporaries and results the allocator hands out on the current one."""
    h = handles["bf16"]
    q, k, v = make("bf16", 2, 512, 512, 8, 2, 64, 64, 61)
    d = rnd((2, 512, 8, 64), torch.bfloat16, 64)
    kw = dict(window=(200, 0), sinks=4)
    o = h.window_attention(q, k, v, want_lse=True, **kw)
    want = [x.clone() for x in h.window_attention_backward(q, k, v, o["out"], o["lse"], d, **kw).values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        s = h.window_attention(q, k, v, want_lse=True, stream=side, **kw)
        g = list(h.window_attention_backward(q, k, v, s["out"], s["lse"], d, stream=side, **kw).values())
        junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(8)]     # would land in freed temporaries
        del junk, s
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(g, want))
