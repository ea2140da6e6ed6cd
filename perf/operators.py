"""Cases that measure the sequence operators of the framework: window attention
with sinks (forward, training step, single-token step), the norm / gate /
residual junction between two blocks, and the embedding with its gradient.

Every case is a dict of plain values; `prepare` makes its inputs from a seed,
`run` makes one pass (the plain form in elementary torch operations where `own`
is false, the framework's calls where it is true), `exact` the same outputs in
float64 from the definitions, `work` the bytes and operations of one pass."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one RNA-sized chain decoded against its cache: the smallest call, pure latency
        dict(name="attn-step-one", op="attn", mode="step", dtype="bf16", B=1, Nq=1, Nk=2048, H=8, Hkv=8, D=32, Dv=32,
             left=255, right=0, sinks=4, masked=False, ragged=False),
        # one token for each of many sequences of different lengths in one cache, shared key heads
        dict(name="attn-step-batch", op="attn", mode="step", dtype="bf16", B=64, Nq=1, Nk=4096, H=16, Hkv=4, D=64, Dv=64,
             left=1023, right=0, sinks=4, masked=False, ragged=True),
        # the RNA chain, attention along the chain in both directions (sampling: forward only)
        dict(name="attn-forward-chain", op="attn", mode="forward", dtype="bf16", B=1, Nq=2048, Nk=2048, H=8, Hkv=8, D=32, Dv=32,
             left=128, right=128, sinks=4, masked=False, ragged=False),
        # training step of the short-chain batch: padded chains of 40 to 150 residues
        dict(name="attn-train-short-chains", op="attn", mode="train", dtype="bf16", B=512, Nq=150, Nk=150, H=8, Hkv=8, D=16, Dv=16,
             left=31, right=31, sinks=2, masked=True, ragged=False),
        # training step of the longest chain of the length sweep, causal, shared key heads
        dict(name="attn-train-long", op="attn", mode="train", dtype="bf16", B=1, Nq=16384, Nk=16384, H=8, Hkv=2, D=64, Dv=64,
             left=511, right=0, sinks=4, masked=False, ragged=False),
        # float32 training step of the protein batch, padded proteins of 60 to 256 residues
        dict(name="attn-train-f32", op="attn", mode="train", dtype="f32", B=8, Nq=256, Nk=256, H=8, Hkv=8, D=16, Dv=16,
             left=64, right=64, sinks=1, masked=True, ragged=False),
        # junction between two blocks at the size of the protein batch (sampling: forward only)
        dict(name="norm-forward-protein", op="norm", mode="forward", stream="bf16", branch="bf16", rows=2048, C=256,
             norm="layer", gate=True, masked=False),
        # its training step at the size of the short-chain batch: float32 residual stream, bfloat16 branch, padding
        dict(name="norm-train-short-chains", op="norm", mode="train", stream="f32", branch="bf16", rows=76800, C=256,
             norm="layer", gate=True, masked=True),
        # an odd width that no vector load divides, root-mean-square norm, no gate
        dict(name="norm-train-odd", op="norm", mode="train", stream="f32", branch="f32", rows=4099, C=1537,
             norm="rms", gate=False, masked=False),
        # residue types of the protein batch to the single representation
        dict(name="embed-forward-residues", op="embed", mode="forward", dtype="f32", T=2048, V=21, C=256, spread="even"),
        # distogram bins of the 20 nearest neighbours of a long chain to pair features: few rows, very many tokens
        dict(name="embed-train-bins", op="embed", mode="train", dtype="bf16", T=327680, V=64, C=128, spread="bins"),
        # a large token vocabulary, frequencies as in text
        dict(name="embed-train-tokens", op="embed", mode="train", dtype="bf16", T=65536, V=32000, C=512, spread="zipf"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "norm", "embed"])
    if op == "attn":
        mode = rng.choice(["step", "forward", "train", "train"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        D = rng.choice([16, 32, 64, 128, rng.randint(5, 128)])
        Dv = D if rng.random() < 0.8 else rng.randint(3, 128)
        Hkv = rng.choice([1, 2, 3, 4, 8])
        H = Hkv * rng.choice([1, 1, 2, 3, 4])
        sinks = rng.choice([0, 1, 4, rng.randint(0, 64)])
        left = _log_int(rng, 1, 1024)
        right = 0 if mode == "step" or rng.random() < 0.4 else _log_int(rng, 1, 512)
        if mode == "step":
            B, Nq, Nk = _log_int(rng, 1, 96), rng.choice([1, 1, 1, 2, 5]), _log_int(rng, 16, 8192)
            return dict(op=op, mode=mode, dtype=dtype, B=B, Nq=Nq, Nk=Nk, H=H, Hkv=Hkv, D=D, Dv=Dv, left=left, right=0,
                        sinks=sinks, masked=False, ragged=rng.random() < 0.5)
        # rows x heads bounded by the longest listed case, float32 by a quarter of it
        rows = _log_int(rng, 64, (131072 if dtype == "bf16" else 32768) // H)
        Nk = min(rows, _log_int(rng, 16, 16384))
        Nq = Nk if rng.random() < 0.8 else rng.randint(1, Nk)
        case = dict(op=op, mode=mode, dtype=dtype, B=max(1, rows // Nk), Nq=Nq, Nk=Nk, H=H, Hkv=Hkv, D=D, Dv=Dv, left=left,
                    right=right, sinks=sinks, masked=rng.random() < 0.5, ragged=False)
        most = 5.5e10 if dtype == "bf16" else 1.4e10
        while work(case)["flops"] > most:
            case["left"], case["right"] = (case["left"] + 1) // 2, case["right"] // 2
        return case
    if op == "norm":
        stream, branch = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        C = rng.choice([64, 256, 384, 1024, _log_int(rng, 3, 4096)])
        rows = _log_int(rng, 1, min(131072, 20000000 // C))
        return dict(op=op, mode=rng.choice(["forward", "train"]), stream=stream, branch=branch, rows=rows, C=C,
                    norm=rng.choice(["layer", "rms"]), gate=rng.random() < 0.7, masked=rng.random() < 0.5)
    C = rng.choice([16, 128, 256, 512, _log_int(rng, 1, 1024)])
    T = _log_int(rng, 1, min(262144, 32000000 // C))
    V = _log_int(rng, 1, min(100000, 16000000 // C))
    return dict(op=op, mode=rng.choice(["forward", "train"]), dtype=rng.choice(["bf16", "f32"]), T=T, V=V, C=C,
                spread=rng.choice(["even", "bins", "zipf"]))


# ------------------------------------------------------------------ inputs
def _randn(g, shape, dtype, std=1.0, mean=0.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * std + mean).to(dtype)


def _arrays(case, seed):
    """The inputs of a case, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    a = {}
    if case["op"] == "attn":
        t = DTYPES[case["dtype"]]
        B, Nq, Nk, H, Hkv, D, Dv = (case[k] for k in ("B", "Nq", "Nk", "H", "Hkv", "D", "Dv"))
        a["q"] = _randn(g, (B, Nq, H, D), t)
        a["k"] = _randn(g, (B, Nk, Hkv, D), t)
        a["v"] = _randn(g, (B, Nk, Hkv, Dv), t)
        a["mask"] = a["q_start"] = None
        if case["masked"]:
            n = torch.randint(max(1, Nk // 4), Nk + 1, (B, 1), generator=g, device="cuda")
            a["mask"] = torch.arange(Nk, device="cuda")[None, :] < n
        if case["ragged"]:
            a["q_start"] = torch.randint(0, max(1, Nk - Nq + 1), (B,), generator=g, device="cuda", dtype=torch.int32)
        if case["mode"] == "train":
            a["d_out"] = _randn(g, (B, Nq, H, Dv), t)
    elif case["op"] == "norm":
        ts, tb = DTYPES[case["stream"]], DTYPES[case["branch"]]
        rows, C = case["rows"], case["C"]
        a["s"] = _randn(g, (rows, C), ts, 1.5, 0.2)
        a["u"] = _randn(g, (rows, C), tb, 0.7, -0.1)
        a["gate"] = _randn(g, (rows, C), tb) if case["gate"] else None
        a["mask"] = (torch.rand(rows, generator=g, device="cuda") < 0.7) if case["masked"] else None
        for k, mean in (("post_w", 1.0), ("post_b", 0.0), ("pre_w", 1.0), ("pre_b", 0.0), ("res_scale", 0.5)):
            a[k] = _randn(g, (C,), torch.float32, 0.1, mean)
        if case["mode"] == "train":
            a["d_r"] = _randn(g, (rows, C), ts)
            a["d_x"] = _randn(g, (rows, C), tb)
    else:
        t = DTYPES[case["dtype"]]
        T, V, C = case["T"], case["V"], case["C"]
        r = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        if case["spread"] == "even":
            idx = (r * V).long()
        elif case["spread"] == "bins":        # distances grow over the neighbours; one slot in twenty is empty
            idx = (V * r.sqrt() * 0.9).long()
            idx[torch.rand(T, generator=g, device="cuda") < 0.05] = -1
        else:                                 # probability falls as 1 / rank
            idx = (torch.exp(r * math.log(V + 1.0)) - 1.0).long()
        a["idx"] = idx.clamp(-1, V - 1).int()
        a["table"] = _randn(g, (V, C), t)
        a["scale"] = float(math.sqrt(C))
        if case["mode"] == "train":
            a["d_out"] = _randn(g, (T, C), t)
    return a


_handles = {}


def prepare(case, seed):
    a = _arrays(case, seed)
    if own:
        import protein_structure_models_b200 as fw
        a["fw"] = fw
        if case["op"] == "attn":
            if case["dtype"] not in _handles:
                _handles[case["dtype"]] = fw.Fipa(case["dtype"], 0)
            a["handle"] = _handles[case["dtype"]]
    return {"case": case, "a": a}


# ------------------------------------------------------------------ one pass
def run(state):
    case, a = state["case"], state["a"]
    if case["op"] == "attn":
        return _attn_own(case, a) if own else _attn_plain(case, a)
    if case["op"] == "norm":
        return _norm_own(case, a) if own else _norm_plain(case, a)
    return _embed_own(case, a) if own else _embed_plain(case, a)


def _attn_own(case, a):
    h, train = a["handle"], case["mode"] == "train"
    kw = dict(window=(case["left"], case["right"]), sinks=case["sinks"], mask=a["mask"], q_start=a["q_start"])
    o = h.window_attention(a["q"], a["k"], a["v"], want_lse=train, **kw)
    if not train:
        return {"out": o["out"]}
    g = h.window_attention_backward(a["q"], a["k"], a["v"], o["out"], o["lse"], a["d_out"], **kw)
    return {"out": o["out"], "d_q": g["q"], "d_k": g["k"], "d_v": g["v"]}


def _norm_own(case, a):
    fw, train = a["fw"], case["mode"] == "train"
    kw = dict(gate=a["gate"], res_scale=a["res_scale"], post=(a["post_w"], a["post_b"]), pre=(a["pre_w"], a["pre_b"]),
              mask=a["mask"], norm=case["norm"], eps=1e-5)
    o = fw.norm_residual(a["s"], a["u"], want_stats=train, **kw)
    if not train:
        return {"r": o["r"], "x": o["x"]}
    g = fw.norm_residual_backward(a["s"], a["u"], o["stats"], a["d_r"], a["d_x"], **kw)
    return {"r": o["r"], "x": o["x"], "grads": {k: v for k, v in g.items() if v is not None}}


def _embed_own(case, a):
    fw = a["fw"]
    out = fw.embedding(a["idx"], a["table"], scale=a["scale"])["out"]
    if case["mode"] == "forward":
        return {"out": out}
    g = fw.embedding_backward(a["idx"], a["d_out"], case["V"], scale=a["scale"])
    return {"out": out, "d_table": g["table"]}


# ------------------------------------------------------------------ plain forms
def _attn_plain(case, a):
    """Queries in blocks of `blk`; the keys that a block can see are gathered
    (the sinks, then its window), so that nothing N x N exists."""
    B, Nq, Nk, H, Hkv, D, Dv = (case[k] for k in ("B", "Nq", "Nk", "H", "Hkv", "D", "Dv"))
    left, right, sinks = case["left"], case["right"], min(case["sinks"], Nk)
    G = H // Hkv
    left, right = min(left, Nk), min(right, Nk)
    blk = max(1, min(Nq, max(64, (left + right) // 2)))
    nb = -(-Nq // blk)
    dev = a["q"].device
    start = a["q_start"].long() if a["q_start"] is not None else torch.full((B,), Nk - Nq, device=dev)
    i = torch.arange(nb * blk, device=dev)
    p = start[:, None] + i[None, :]                                                 # [B, nb*blk]
    live = (i[None, :] < Nq) & (p >= 0) & (p < Nk)
    mask = a["mask"] if a["mask"] is not None else torch.ones((B, Nk), dtype=torch.bool, device=dev)
    live = live & torch.gather(mask, 1, p.clamp(0, Nk - 1))
    first = start[:, None] + torch.arange(nb, device=dev)[None, :] * blk - left     # [B, nb]
    win = first[:, :, None] + torch.arange(blk + left + right, device=dev)          # [B, nb, w]
    sink = torch.arange(sinks, device=dev).expand(B, nb, sinks)
    j = torch.cat([sink, win], 2)                                                   # [B, nb, c]
    issink = torch.arange(j.shape[2], device=dev) < sinks
    pb = p.view(B, nb, blk, 1)
    jb = j[:, :, None, :]
    inwin = (jb >= pb - left) & (jb <= pb + right)
    see = torch.where(issink, (jb < pb - left) & (jb <= pb + right), inwin) & (jb >= 0) & (jb < Nk)
    jc = j.clamp(0, Nk - 1)
    see = see & torch.gather(mask, 1, jc.view(B, -1)).view(B, nb, 1, -1) & live.view(B, nb, blk, 1)
    bi = torch.arange(B, device=dev)[:, None]
    rows = i.clamp(max=Nq - 1)

    def qblocks(x):                                                                 # -> [B, nb, Hkv, G, blk, d] float32
        return x.float()[:, rows].view(B, nb, blk, Hkv, G, -1).permute(0, 1, 3, 4, 2, 5)

    def kblocks(x):                                                                 # -> [B, nb, Hkv, 1, c, d] float32
        return x.float()[bi, jc.view(B, -1)].view(B, nb, -1, Hkv, 1, x.shape[3]).permute(0, 1, 3, 4, 2, 5)

    q, k, v = qblocks(a["q"]), kblocks(a["k"]), kblocks(a["v"])
    scale = 1.0 / math.sqrt(D)
    see = see[:, :, None, None]
    s = (q @ k.transpose(-1, -2) * scale).masked_fill(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m.masked_fill(m == -math.inf, 0.0))
    l = e.sum(-1, keepdim=True)
    pr = e / l.masked_fill(l == 0, 1.0)
    o = pr @ v

    def rows_out(x):                                                                # back to [B, Nq, H, d]
        return x.permute(0, 1, 4, 2, 3, 5).reshape(B, nb * blk, H, -1)[:, :Nq]

    out = rows_out(o).to(a["q"].dtype).contiguous()
    if case["mode"] != "train":
        return {"out": out}
    do = qblocks(a["d_out"]) * live.view(B, nb, 1, 1, blk, 1)
    dp = do @ v.transpose(-1, -2)
    ds = pr * (dp - (do * o).sum(-1, keepdim=True)) * scale
    dq = rows_out(ds @ k)
    flat = (bi * Nk + jc.view(B, -1)).reshape(-1)

    def keys_out(x):                                                                # gathered keys back to their rows
        x = x.sum(3).permute(0, 1, 3, 2, 4).reshape(flat.numel(), -1)
        return torch.zeros((B * Nk, x.shape[1]), device=dev).index_add_(0, flat, x)

    dk = keys_out(ds.transpose(-1, -2) @ q).view(B, Nk, Hkv, D)
    dv = keys_out(pr.transpose(-1, -2) @ do).view(B, Nk, Hkv, Dv)
    t = a["q"].dtype
    return {"out": out, "d_q": dq.to(t).contiguous(), "d_k": dk.to(t), "d_v": dv.to(t)}


def _norm_fwd(x, kind, eps=1e-5):
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + eps)
    return c * rstd, rstd


def _norm_bwd(h, xhat, rstd, kind):
    out = h - xhat * (h * xhat).mean(-1, keepdim=True)
    if kind == "layer":
        out = out - h.mean(-1, keepdim=True)
    return out * rstd


def _norm_plain(case, a):
    kind = case["norm"]
    s, u = a["s"].float(), a["u"].float()
    live = a["mask"][:, None] if a["mask"] is not None else None
    uhat, ru = _norm_fwd(u, kind)
    y = uhat * a["post_w"] + a["post_b"]
    sg = torch.sigmoid(a["gate"].float()) if a["gate"] is not None else None
    gy = y * sg if sg is not None else y
    add = a["res_scale"] * gy
    r = s + (add if live is None else add.masked_fill(~live, 0.0))
    rhat, rr = _norm_fwd(r, kind)
    x = rhat * a["pre_w"] + a["pre_b"]
    x = x if live is None else x.masked_fill(~live, 0.0)
    out = {"r": r.to(a["s"].dtype), "x": x.to(a["u"].dtype)}
    if case["mode"] != "train":
        return out
    dr, dx = a["d_r"].float(), a["d_x"].float()
    dx = dx if live is None else dx.masked_fill(~live, 0.0)
    dtot = dr + _norm_bwd(dx * a["pre_w"], rhat, rr, kind)
    dadd = dtot if live is None else dtot.masked_fill(~live, 0.0)
    dgy = dadd * a["res_scale"]
    dy = dgy * sg if sg is not None else dgy
    g = {"s": dtot.to(a["s"].dtype), "u": _norm_bwd(dy * a["post_w"], uhat, ru, kind).to(a["u"].dtype)}
    if sg is not None:
        g["gate"] = (dgy * y * sg * (1 - sg)).to(a["u"].dtype)
    g["res_scale"] = (dadd * gy).sum(0)
    g["post_w"], g["post_b"] = (dy * uhat).sum(0), dy.sum(0)
    g["pre_w"], g["pre_b"] = (dx * rhat).sum(0), dx.sum(0)
    out["grads"] = g
    return out


def _embed_plain(case, a):
    ok = (a["idx"] >= 0)[:, None]
    at = a["idx"].clamp(min=0).long()
    out = (a["table"][at].float() * a["scale"]).masked_fill(~ok, 0.0).to(a["table"].dtype)
    if case["mode"] == "forward":
        return {"out": out}
    d = a["d_out"].float().masked_fill(~ok, 0.0)
    dt = torch.zeros((case["V"], case["C"]), device=d.device).index_add_(0, at, d) * a["scale"]
    return {"out": out, "d_table": dt}


# ------------------------------------------------------------------ float64
def exact(case, seed):
    a = _arrays(case, seed)
    return {"attn": _attn_exact, "norm": _norm_exact, "embed": _embed_exact}[case["op"]](case, a)


def _attn_exact(case, a):
    """Dense scores of one (sample, key head) group at a time, gradients by autograd."""
    B, Nq, Nk, H, Hkv, D, Dv = (case[k] for k in ("B", "Nq", "Nk", "H", "Hkv", "D", "Dv"))
    G, train = H // Hkv, case["mode"] == "train"
    dev = a["q"].device
    per = max(1, int(2.0e8 // max(1, Nq * Nk * G)))       # groups at a time
    if B * Hkv / per > 4000:
        return None
    t64 = lambda x, heads, d: x.double().view(B, -1, Hkv, heads, d).permute(0, 2, 3, 1, 4).reshape(B * Hkv, heads, -1, d)  # noqa: E731
    q, k, v = t64(a["q"], G, D), t64(a["k"], 1, D), t64(a["v"], 1, Dv)
    do = t64(a["d_out"], G, Dv) if train else None
    start = a["q_start"].long() if a["q_start"] is not None else torch.full((B,), Nk - Nq, device=dev)
    mask = a["mask"] if a["mask"] is not None else torch.ones((B, Nk), dtype=torch.bool, device=dev)
    got = {"out": [], "d_q": [], "d_k": [], "d_v": []}
    for g0 in range(0, B * Hkv, per):
        sl = slice(g0, min(B * Hkv, g0 + per))
        b = torch.arange(sl.start, sl.stop, device=dev) // Hkv
        pos = (start[b][:, None] + torch.arange(Nq, device=dev))[:, :, None]
        key = torch.arange(Nk, device=dev)[None, None, :]
        near = key >= pos - case["left"]
        ok = (key <= pos + case["right"]) & (near | (key < case["sinks"])) & mask[b][:, None, :]
        ok &= (pos >= 0) & (pos < Nk) & torch.gather(mask[b], 1, pos[:, :, 0].clamp(0, Nk - 1))[:, :, None]
        ok = ok[:, None]
        qq, kk, vv = (x[sl].clone().requires_grad_(train) for x in (q, k, v))
        s = torch.where(ok, qq @ kk.transpose(-1, -2) / math.sqrt(D), torch.full((), -1e300, dtype=torch.float64, device=dev))
        pr = torch.softmax(s, -1) * ok.any(-1, keepdim=True)
        o = pr @ vv
        got["out"].append(o.detach())
        if train:
            for name, x in zip(("d_q", "d_k", "d_v"), torch.autograd.grad((o * do[sl]).sum(), (qq, kk, vv))):
                got[name].append(x)
        del s, pr, o
    back = lambda xs, d: torch.cat(xs).view(B, Hkv, -1, xs[0].shape[2], d).permute(0, 3, 1, 2, 4).reshape(B, xs[0].shape[2], -1, d)  # noqa: E731
    res = {"out": back(got["out"], Dv)}
    if train:
        res |= {"d_q": back(got["d_q"], D), "d_k": back(got["d_k"], D), "d_v": back(got["d_v"], Dv)}
    return res


def _norm_exact(case, a):
    leaf = {k: a[k].double().requires_grad_(True) for k in ("s", "u", "gate", "res_scale", "post_w", "post_b", "pre_w", "pre_b")
            if a[k] is not None}
    on = a["mask"][:, None].double() if a["mask"] is not None else 1.0

    def norm(x, w, b):
        var, mean = (x.var(-1, unbiased=False, keepdim=True), x.mean(-1, keepdim=True)) if case["norm"] == "layer" \
            else (x.pow(2).mean(-1, keepdim=True), 0.0)
        return (x - mean) / (var + 1e-5).sqrt() * w + b

    y = norm(leaf["u"], leaf["post_w"], leaf["post_b"])
    if "gate" in leaf:
        y = y / (1.0 + torch.exp(-leaf["gate"]))
    r = leaf["s"] + on * leaf["res_scale"] * y
    x = on * norm(r, leaf["pre_w"], leaf["pre_b"])
    res = {"r": r.detach(), "x": x.detach()}
    if case["mode"] == "train":
        loss = (r * a["d_r"].double()).sum() + (x * a["d_x"].double()).sum()
        res["grads"] = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    return res


def _embed_exact(case, a):
    idx, V, scale = a["idx"].long(), case["V"], a["scale"]
    pad = torch.cat([a["table"].double() * scale, torch.zeros((1, case["C"]), dtype=torch.float64, device="cuda")])
    row = torch.where(idx < 0, torch.full_like(idx, V), idx)
    res = {"out": pad[row]}
    if case["mode"] == "train":
        d = torch.zeros((V + 1, case["C"]), dtype=torch.float64, device="cuda")
        d.index_add_(0, row, a["d_out"].double())
        res["d_table"] = d[:V] * scale
    return res


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "attn":
        B, Nq, Nk, H, Hkv, D, Dv = (case[k] for k in ("B", "Nq", "Nk", "H", "Hkv", "D", "Dv"))
        es = 2 if case["dtype"] == "bf16" else 4
        # visible keys of a query at each position, and how often each position is asked for
        p = np.arange(Nk, dtype=np.int64)
        hi = np.minimum(p + case["right"], Nk - 1)
        lo = np.maximum(p - case["left"], 0)
        seen = hi - lo + 1 + np.minimum(np.minimum(case["sinks"], lo), hi + 1)
        if case["masked"]:                     # lengths uniform between a quarter and all: 5/8 of the rows on average
            pairs, part = B * float(seen.mean()) * Nq * 0.625, 0.625
            used = Nk * part
        elif case["ragged"]:
            pairs, part = B * float(seen.mean()) * Nq, 1.0
            used = min(Nk, float(seen.mean()) + Nq - 1)
        else:
            pairs, part = B * float(seen[Nk - Nq:].sum()), 1.0
            used = min(Nk, Nq + case["left"] + case["sinks"])
        pairs *= H
        q, k, v, o = B * Nq * H * D * part, B * used * Hkv * D, B * used * Hkv * Dv, B * Nq * H * Dv
        fwd = {"bytes": es * (q + k + v + o), "flops": 2 * (D + Dv) * pairs}
        if case["mode"] != "train":
            return fwd
        # the gradients read q, k, v, out and d_out, write three tensors; five products a pair
        return {"bytes": fwd["bytes"] + es * (q + k + v + 2 * o * part + B * Nq * H * D + B * Nk * Hkv * (D + Dv)),
                "flops": fwd["flops"] + (6 * D + 4 * Dv) * pairs}
    if case["op"] == "norm":
        n, C = case["rows"] * case["C"], case["C"]
        es, eb = (2 if case[k] == "bf16" else 4 for k in ("stream", "branch"))
        gate = eb if case["gate"] else 0
        on = 0.7 if case["masked"] else 1.0    # a masked row's branch and gate need not be read
        nbytes = n * (2 * es + on * (eb + gate) + eb) + 20 * C
        flops = 20 * n
        if case["mode"] == "train":
            nbytes += n * (3 * es + on * (2 * eb + gate) + eb + gate) + 40 * C
            flops += 40 * n
        return {"bytes": nbytes, "flops": flops}
    T, V, C = case["T"], case["V"], case["C"]
    es = 2 if case["dtype"] == "bf16" else 4
    nbytes, flops = 4 * T + T * C * es + min(T, V) * C * es, T * C
    if case["mode"] == "train":
        nbytes += 4 * T + T * C * es + V * C * 4
        flops += 2 * T * C
    return {"bytes": nbytes, "flops": flops}
