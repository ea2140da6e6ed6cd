"""The sequence operators together, as a model uses them: residue types ->
embedding -> norm -> projection -> window attention with sinks -> projection ->
gate, residual and norm, forward and backward, over a padded batch.

Every operator's gradient call is fed by the next one's, so the last gradient
(that of the embedding table) has passed through all of them.  The reference is
the same chain in float64 with gradients by autograd.  Its tolerance is measured
on the reference itself: each stage's result and each gradient that a stage hands
back are disturbed by a relative 2^-18 (what the float32 operators' own tests
allow) with random signs; a result may be off by 8 times the change that this
makes (four disturbances with other signs, the largest, times two), relative to
the norm of each result."""
import pytest
import torch

from oracle import sequence as seq

pytestmark = pytest.mark.gpu
B, N, V, C, H, HKV, D = 3, 90, 21, 64, 4, 2, 16
LEFT, RIGHT, SINKS = 20, 5, 3
EPS = 1e-5


class Disturb(torch.autograd.Function):
    """x (1 + size e), e = -1 or 1, in both directions."""
    @staticmethod
    def forward(ctx, x, gen, size):
        ctx.gen, ctx.size = gen, size
        return x * (1 + size * (2 * torch.randint(0, 2, x.shape, generator=gen) - 1))

    @staticmethod
    def backward(ctx, g):
        return g * (1 + ctx.size * (2 * torch.randint(0, 2, g.shape, generator=ctx.gen) - 1)), None, None


def parameters():
    g = torch.Generator().manual_seed(2)
    r = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean)  # noqa: E731
    n_in = (H + 2 * HKV) * D
    p = {"table": r(V, C), "w_in": r(C, n_in, std=C ** -0.5), "w_out": r(H * D, C, std=(H * D) ** -0.5),
         "w_gate": r(C, C, std=C ** -0.5), "res_scale": r(C, std=0.1, mean=0.5)}
    for k in ("first", "post", "pre"):
        p[k + "_w"], p[k + "_b"] = r(C, std=0.1, mean=1.0), r(C, std=0.1)
    idx = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32)
    mask = torch.arange(N)[None, :] < torch.tensor([N, 57, 31])[:, None]
    idx[~mask] = -1
    return p, idx, mask, r(B, N, C), r(B, N, C)


def norm(x, w, b):
    return (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + EPS).sqrt() * w + b


def reference(p, idx, mask, d_r, d_x, size=0.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    dis = (lambda x: Disturb.apply(x, gen, size)) if size else (lambda x: x)
    p = {k: v.double().requires_grad_(True) for k, v in p.items()}
    on = mask[..., None].double()
    s = dis(p["table"][idx.long().clamp(min=0)] * 8.0 * on)
    x0 = dis(norm(s, p["first_w"], p["first_b"]) * on)
    h = dis(x0 @ p["w_in"]).view(B, N, H + 2 * HKV, D)
    q, k, v = h[:, :, :H], h[:, :, H:H + HKV], h[:, :, H + HKV:]
    ok = seq.visible(B, N, N, LEFT, RIGHT, SINKS, mask)[:, None]
    rep = lambda t: t.permute(0, 2, 1, 3).repeat_interleave(H // t.shape[2], dim=1)  # noqa: E731
    sc = (rep(q) @ rep(k).transpose(-1, -2) * D ** -0.5).masked_fill(~ok, -1e300)
    pr = torch.softmax(sc, -1) * ok.any(-1, keepdim=True)
    o = dis((pr @ rep(v)).permute(0, 2, 1, 3).reshape(B, N, H * D))
    u, gate = dis(o @ p["w_out"]), dis(x0 @ p["w_gate"])
    r = dis(s + on * p["res_scale"] * torch.sigmoid(gate) * norm(u, p["post_w"], p["post_b"]))
    x = dis(on * norm(r, p["pre_w"], p["pre_b"]))
    g = torch.autograd.grad((r * d_r.double()).sum() + (x * d_x.double()).sum(), list(p.values()))
    return {"r": r.detach(), "x": x.detach(), **{"d_" + k: t for k, t in zip(p, g)}}


def operators(h, p, idx, mask, d_r, d_x):
    import protein_structure_models_b200 as fw
    kw = dict(window=(LEFT, RIGHT), sinks=SINKS, mask=mask)
    s = fw.embedding(idx, p["table"], scale=8.0)["out"]
    first = dict(pre=(p["first_w"], p["first_b"]), mask=mask, eps=EPS)
    n0 = fw.norm_residual(s, want_stats=True, **first)
    x0 = n0["x"]
    z = (x0 @ p["w_in"]).view(B, N, H + 2 * HKV, D)
    q, k, v = z[:, :, :H], z[:, :, H:H + HKV], z[:, :, H + HKV:]
    o = h.window_attention(q, k, v, want_lse=True, **kw)
    u, gate = o["out"].view(B, N, H * D) @ p["w_out"], x0 @ p["w_gate"]
    join = dict(gate=gate, res_scale=p["res_scale"], post=(p["post_w"], p["post_b"]), pre=(p["pre_w"], p["pre_b"]), mask=mask, eps=EPS)
    j = fw.norm_residual(s, u, want_stats=True, **join)
    g = fw.norm_residual_backward(s, u, j["stats"], d_r, d_x, **join)
    do = (g["u"] @ p["w_out"].t()).view(B, N, H, D)
    ga = h.window_attention_backward(q, k, v, o["out"], o["lse"], do, **kw)
    dz = torch.cat([ga["q"], ga["k"], ga["v"]], 2).view(B, N, -1)
    dx0 = dz @ p["w_in"].t() + g["gate"] @ p["w_gate"].t()
    g0 = fw.norm_residual_backward(s, None, n0["stats"], None, dx0, **first)
    dt = fw.embedding_backward(idx, g["s"] + g0["s"], V, scale=8.0)["table"]
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    return {"r": j["r"], "x": j["x"], "d_table": dt, "d_w_in": flat(x0).t() @ flat(dz),
            "d_w_out": flat(o["out"].view(B, N, H * D)).t() @ flat(g["u"]), "d_w_gate": flat(x0).t() @ flat(g["gate"]),
            "d_res_scale": g["res_scale"], "d_first_w": g0["pre_w"], "d_first_b": g0["pre_b"], "d_post_w": g["post_w"],
            "d_post_b": g["post_b"], "d_pre_w": g["pre_w"], "d_pre_b": g["pre_b"]}


def test_a_block_of_a_sequence_model():
    from protein_structure_models_b200 import Fipa, build
    build.build()
    p, idx, mask, d_r, d_x = parameters()
    want = reference(p, idx, mask, d_r, d_x)
    tol = {k: 0.0 for k in want}
    for seed in range(1, 5):
        other = reference(p, idx, mask, d_r, d_x, size=2.0 ** -18, seed=seed)
        tol = {k: max(tol[k], 2 * float((other[k] - want[k]).norm())) for k in want}
    h = Fipa("f32", 0)
    try:
        before = torch.backends.cuda.matmul.allow_tf32
        torch.backends.cuda.matmul.allow_tf32 = False
        got = operators(h, {k: v.cuda() for k, v in p.items()}, idx.cuda(), mask.cuda(), d_r.cuda(), d_x.cuda())
        h.sync_status()
    finally:
        torch.backends.cuda.matmul.allow_tf32 = before
        h.close()
    assert set(got) == set(want)
    for k in want:
        off = float((got[k].cpu().double() - want[k]).norm())
        assert off <= 4 * tol[k], f"{k}: off by {off:.3e}, change of the disturbed reference {tol[k] / 2:.3e}"
