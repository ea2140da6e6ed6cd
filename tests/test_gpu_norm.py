"""The norm / gate / residual junction (through the C ABI) against its float64
definition (oracle/sequence.py).

Tolerances: every value is the float32 result of at most 64 roundings along any
path (sums over C are trees of 8-term chains; 64 * 2^-24 = 2^-18), so it is off
by 2^-18 of the sum of the absolute values that it is made of, which is carried
along beside each formula; then one rounding to the output's type (half a step,
bf16 2^-8, f32 2^-24).  Parameter gradients add their rows in chains:
rows * 2^-24 of the absolute sum more."""
import pytest
import torch

from oracle import sequence as seq

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
E = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    from protein_structure_models_b200 import build
    build.build()


def rnd(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def within(got, want, tol, name):
    d = (got.detach().cpu().double() - want).abs()
    assert (d <= tol).all(), f"{name}: off by {d.max():.3e}, worst {(d / tol).max():.2f} bounds"


def mean(x):
    return x.mean(-1, keepdim=True)


def check(s, u=None, gate=None, res_scale=None, post=None, pre=None, mask=None, norm="layer", eps=1e-5, d_r=None, d_x=None):
    import protein_structure_models_b200 as fw
    kw = dict(gate=gate, res_scale=res_scale, post=post, pre=pre, mask=mask, norm=norm, eps=eps)
    got = fw.norm_residual(s, u, want_stats=True, **kw)
    g = fw.norm_residual_backward(s, u, got["stats"], d_r, d_x, **kw)
    torch.cuda.synchronize()
    kw["norm_kind"] = kw.pop("norm")
    b = seq.norm_residual_backward(s, u, d_r, d_x, **kw)
    o = b["o"]
    live, lay = o["live"], norm == "layer"
    ts, tb = U[s.dtype], U[u.dtype if u is not None else s.dtype]
    Ar = o["s"].abs()                                             # absolute sums behind r
    if u is not None:
        # uhat = (u - mean) rstd: |u| + mean|u| behind it; 1/deviation moves by as much of |uhat|
        Au = o["ru"] * (o["u"].abs() + mean(o["u"].abs())) + o["uhat"].abs() * (1 + mean(o["uhat"].abs() * o["ru"] * (
            o["u"].abs() + mean(o["u"].abs()))))
        Ay = Au * o["pw"].abs() + (o["pb"].abs() if o["pb"] is not None else 0.0) if post else o["u"].abs()
        Ar = Ar + torch.where(live, o["ga"].abs() * o["sg"] * Ay, 0.0)
        within(got["r"], o["r"], ts * o["r"].abs() + E * Ar, "r")
    if pre:
        c = Ar + mean(Ar)
        Az = torch.where(live, o["rr"] * c + o["rhat"].abs() * (1 + mean(o["rhat"].abs() * o["rr"] * c)), 0.0)
        Ax = Az * o["qw"].abs() + (o["qb"].abs() if o["qb"] is not None else 0.0)
        within(got["x"], o["x"], tb * o["x"].abs() + E * torch.where(live, Ax, 0.0) + 1e-30, "x")
    n = s.numel() // s.shape[-1]
    rows = lambda t: t.reshape(-1, t.shape[-1]).sum(0)  # noqa: E731

    def grad_abs(h, z, A, rstd):                                  # |terms| of Norm's gradient, z off by E A
        z = z.abs()
        return rstd * (h + A * mean(h * z) + z * mean(h * A) + z * mean(h * z) + (mean(h) if lay else 0.0)) + \
            rstd * mean(z * A) * (h + z * mean(h * z) + (mean(h) if lay else 0.0))   # 1/deviation itself

    Adt = d_r.cpu().double().abs() if d_r is not None else torch.zeros_like(o["s"])
    if pre:
        dx = b["dx"].abs()
        Adt = Adt + torch.where(live, grad_abs(dx * o["qw"].abs(), o["rhat"], Az, o["rr"]), 0.0)
        within(g["pre_w"], b["pre_w"], (E + n * 2.0 ** -24) * rows(dx * (Az + o["rhat"].abs())) + 1e-30, "pre_w")
        if g.get("pre_b") is not None:
            within(g["pre_b"], b["pre_b"], n * 2.0 ** -24 * rows(dx) + 1e-30, "pre_b")
    within(g["s"], b["s"], ts * b["s"].abs() + E * Adt + 1e-30, "d_s")
    if u is not None:
        Ada = torch.where(live, Adt, 0.0)
        Agy, ay = Ada * o["ga"].abs(), o["y"].abs()
        if gate is not None:
            k = o["sg"] * (1 - o["sg"])
            # sigmoid's own rounding, E of sg, also moves 1 - sg
            within(g["gate"], b["gate"], tb * b["gate"].abs() + E * Agy * (Ay + ay) * (k + o["sg"] ** 2) + 1e-30, "d_gate")
        if res_scale is not None:
            within(g["res_scale"], b["res_scale"], (E + n * 2.0 ** -24) * rows(Ada * o["sg"] * (Ay + ay)) + 1e-30, "d_res_scale")
        Ady = Agy * o["sg"]
        if post:
            within(g["post_w"], b["post_w"], (E + n * 2.0 ** -24) * rows(Ady * (Au + o["uhat"].abs())) + 1e-30, "post_w")
            if g.get("post_b") is not None:
                within(g["post_b"], b["post_b"], (E + n * 2.0 ** -24) * rows(Ady) + 1e-30, "post_b")
            Adu = grad_abs(Ady * o["pw"].abs(), o["uhat"], Au, o["ru"])
        else:
            Adu = Ady
        within(g["u"], b["u"], tb * b["u"].abs() + E * torch.where(live, Adu, 0.0) + 1e-30, "d_u")
    return got, g


def make(rows, C, ts, tb, gate=True, masked=False, seed=0, bias=True, smean=0.2):
    p = lambda i, m: rnd((C,), torch.float32, seed + 20 + i, 0.1, m)  # noqa: E731
    return dict(s=rnd((rows, C), TD[ts], seed, 1.5, smean), u=rnd((rows, C), TD[tb], seed + 1, 0.7, -0.1),
                gate=rnd((rows, C), TD[tb], seed + 2) if gate else None, res_scale=p(0, 0.5),
                post=(p(1, 1.0), p(2, 0.0) if bias else None), pre=(p(3, 1.0), p(4, 0.0) if bias else None),
                mask=(torch.rand(rows, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") < 0.6)
                if masked else None, d_r=rnd((rows, C), TD[ts], seed + 3), d_x=rnd((rows, C), TD[tb], seed + 4))


TYPES = [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("ts,tb", TYPES)
@pytest.mark.parametrize("rows,C", [(1, 1), (1, 8), (3, 7), (5, 64), (300, 256), (33, 255), (70, 257), (129, 1024), (40, 1537),
                                    (9, 2048), (7, 2056), (5, 4095), (4, 8192), (2, 8191), (2000, 16), (4097, 40)])
def test_against_the_definition(ts, tb, rows, C):
    check(**make(rows, C, ts, tb, masked=rows > 4), norm="layer" if rows % 2 else "rms")


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("drop", ["gate", "res_scale", "post", "pre", "mask", "bias", "d_r", "d_x"])
@pytest.mark.parametrize("C", [96, 101])
def test_without_a_part(norm, drop, C):
    a = make(50, C, "f32", "bf16", masked=True, bias=drop != "bias")
    if drop != "bias":
        a[drop] = None
    if drop == "pre":
        a["d_x"] = None
    check(**a, norm=norm)


@pytest.mark.parametrize("tb", ["f32", "bf16"])
def test_norm_alone(tb):
    """No branch: x = Norm(s), at any leading shape."""
    s = rnd((3, 5, 72), TD[tb], 1)
    pre = (rnd((72,), torch.float32, 2, 0.1, 1.0), rnd((72,), torch.float32, 3))
    got, g = check(s, pre=pre, d_x=rnd(s.shape, s.dtype, 4), mask=torch.rand(3, 5, device="cuda") < 0.7)
    assert "r" not in got and g["u"] is None


def test_padding_is_never_used():
    """NaN in the branch, the gate and the gradients of padded rows; a masked row's stream passes through."""
    a = make(64, 128, "f32", "bf16", masked=True)
    clean, gc = check(**a)
    m = a["mask"]
    for k in ("u", "gate", "d_x"):
        a[k] = a[k].clone()
        a[k][~m] = float("nan")
    import protein_structure_models_b200 as fw
    d_r, d_x = a.pop("d_r"), a.pop("d_x")
    got = fw.norm_residual(**a, want_stats=True)
    s, u = a.pop("s"), a.pop("u")
    g = fw.norm_residual_backward(s, u, got["stats"], d_r, d_x, **a)
    assert torch.equal(got["r"], clean["r"]) and torch.equal(got["x"], clean["x"]) and torch.equal(got["r"][~m], s[~m])
    for k in g:
        assert torch.equal(g[k], gc[k]), k
    assert torch.equal(g["s"][~m], d_r[~m])


GATES = [float("-inf"), -3e38, -1e30, -1e4, *(x / 2 for x in range(-260, 261)), 1e4, 1e30, 3e38, float("inf"), -0.0]


@pytest.mark.parametrize("ts,tb", TYPES)
@pytest.mark.parametrize("C", [256, 101])
def test_gates_of_any_size(ts, tb, C):
    """Closed and open gates: infinities, the largest finite values, every half from -130 to 130, the type's ends; as many rows as it takes."""
    t = TD[tb]
    v = torch.tensor([*GATES, torch.finfo(t).min, torch.finfo(t).max], device="cuda").to(t)
    rows = 2 * len(v) // C + 7
    a = make(rows, C, ts, tb, seed=30)
    a["gate"] = v.repeat(rows * C // len(v) + 1)[:rows * C].view(rows, C)
    for norm in ("layer", "rms"):
        got, g = check(**a, norm=norm)
        assert all(torch.isfinite(x).all() for x in (*got.values(), *g.values()))
    shut = torch.full_like(a["gate"], float("-inf"))                   # a row of closed gates: nothing of the branch is left
    a["gate"] = shut
    got, g = check(**a)
    assert torch.equal(got["r"], a["s"]) and (g["u"] == 0).all() and (g["gate"] == 0).all()


def test_a_gate_that_is_nan_spoils_its_row_only():
    a = make(9, 96, "f32", "bf16")
    clean, gc = check(**a)
    a["gate"][4, 7] = float("nan")
    import protein_structure_models_b200 as fw
    d_r, d_x = a.pop("d_r"), a.pop("d_x")
    got = fw.norm_residual(**a, want_stats=True)
    assert got["r"][4, 7].isnan() and got["x"][4].isnan().all()
    g = fw.norm_residual_backward(a.pop("s"), a.pop("u"), got["stats"], d_r, d_x, **a)
    other = torch.arange(9, device="cuda") != 4
    assert g["s"][4].isnan().all() and g["gate"][4, 7].isnan()
    assert all(torch.equal(x[other], y[other]) for x, y in ((got["r"], clean["r"]), (got["x"], clean["x"]), (g["s"], gc["s"]), (g["u"], gc["u"]), (g["gate"], gc["gate"])))


def test_large_mean_and_tiny_variance():
    """A mean a thousand times the deviation (absolute sums say what float32 can keep), a constant row, a zero row."""
    a = make(30, 200, "f32", "f32", smean=1000.0)
    a["u"][3] = 2.5
    a["u"][4] = 0.0
    check(**a)


def test_all_masked_and_no_rows():
    a = make(5, 40, "f32", "f32")
    a["mask"] = torch.zeros(5, dtype=torch.bool, device="cuda")
    got, g = check(**a)
    assert (got["x"] == 0).all() and all((g[k] == 0).all() for k in ("u", "gate", "post_w", "pre_w", "res_scale"))
    a = make(0, 40, "f32", "f32")
    _, g = check(**a)
    assert all((g[k] == 0).all() for k in ("post_w", "post_b", "pre_w", "pre_b", "res_scale"))


@pytest.mark.parametrize("C", [64, 1000])
def test_unaligned_buffers_in_place_and_repeats(C):
    """Tensors off the 16-byte grid give what aligned ones give to rounding order; r may be s; repeats are identical."""
    import protein_structure_models_b200 as fw
    a = make(37, C, "f32", "bf16", masked=True)

    def shifted(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:].copy_(t.reshape(-1))
        return b[1:].view(t.shape)

    got, g = check(**{k: shifted(v) if torch.is_tensor(v) and v.dim() == 2 else v for k, v in a.items()})
    got2, g2 = check(**{k: shifted(v) if torch.is_tensor(v) and v.dim() == 2 else v for k, v in a.items()})
    assert torch.equal(got["x"], got2["x"]) and all(torch.equal(g[k], g2[k]) for k in g)
    d_r, d_x = a.pop("d_r"), a.pop("d_x")
    want = fw.norm_residual(**a)
    s = a["s"].clone()
    x = torch.empty_like(want["x"])
    fw.norm_residual(**{**a, "s": s}, out={"r": s, "x": x})
    assert torch.equal(s, want["r"]) and torch.equal(x, want["x"])


def test_graph_and_stream():
    import protein_structure_models_b200 as fw
    a = make(500, 256, "f32", "bf16", masked=True)
    d_r, d_x = a.pop("d_r"), a.pop("d_x")
    s, u = a.pop("s"), a.pop("u")

    def step():
        o = fw.norm_residual(s, u, want_stats=True, **a)
        return [o["r"], o["x"], *fw.norm_residual_backward(s, u, o["stats"], d_r, d_x, **a).values()]

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = fw.norm_residual(s, u, stream=side, **a)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(res, want)) and torch.equal(o["x"], want[1])


def test_gradients_that_are_not_wanted_and_guards():
    import protein_structure_models_b200 as fw
    a = make(45, 72, "f32", "bf16", masked=True)
    _, full = check(**a)
    d_r, d_x = a.pop("d_r"), a.pop("d_x")
    s, u = a.pop("s"), a.pop("u")
    st = fw.norm_residual(s, u, want_stats=True, **a)["stats"]
    for only in ("s", "u", "gate", "post_w", "pre_b", "res_scale"):
        b = torch.full((full[only].numel() + 128,), 3.0, dtype=full[only].dtype, device="cuda")
        v = b[64:-64].view(full[only].shape)
        fw.norm_residual_backward(s, u, st, d_r, d_x, grads={only: v}, **a)
        assert torch.equal(v, full[only]) and (b[:64] == 3).all() and (b[-64:] == 3).all()


def test_refusals():
    import protein_structure_models_b200 as fw
    from protein_structure_models_b200 import FipaError
    a = make(4, 16, "f32", "bf16")
    d_r, d_x = a.pop("d_r"), a.pop("d_x")
    for bad in (dict(s=a["s"][:, :8]), dict(u=a["u"][:2]), dict(gate=a["gate"].float()), dict(norm="batch"),
                dict(res_scale=a["res_scale"].double()), dict(pre=(a["res_scale"][:3], None)),
                dict(mask=torch.ones(3, dtype=torch.bool, device="cuda")), dict(s=a["s"].cpu())):
        with pytest.raises(ValueError):
            fw.norm_residual(**{**a, **bad})
    for bad, status in ((dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(u=None, gate=None), 1), (dict(u=None, gate=None, res_scale=None, post=None, pre=None), 1),
                        (dict(pre=(None, a["res_scale"])), 1)):
        with pytest.raises(FipaError) as e:
            fw.norm_residual(**{**a, **bad})
        assert e.value.status == status
    big = torch.zeros(1, 8193, device="cuda")
    with pytest.raises(FipaError) as e:
        fw.norm_residual(big, big)
    assert e.value.status == 2
    st = fw.norm_residual(want_stats=True, **a)["stats"]
    s, u = a.pop("s"), a.pop("u")
    with pytest.raises(FipaError) as e:
        fw.norm_residual_backward(s, u, st, d_r, d_x, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"), **a)
    assert e.value.status == 3
    with pytest.raises(ValueError):
        fw.norm_residual_backward(s, u, st[:2], d_r, d_x, **a)
