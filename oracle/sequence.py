"""Float64 definitions of the sequence operators and their gradients, written
from the formulas in include/fipa.h: window attention with sinks, the norm /
gate / residual junction, the embedding.  Dense and slow; test infrastructure."""
from __future__ import annotations

import math
from typing import Optional

import torch

D64 = torch.float64


# ------------------------------------------------------------ window attention
def visible(B, Nq, Nk, left, right, sinks, mask=None, q_start=None):
    """[B, Nq, Nk] bool: which keys each query sees (left, right None: no bound)."""
    start = torch.full((B,), Nk - Nq) if q_start is None else q_start.cpu().long()
    p = (start[:, None] + torch.arange(Nq))[:, :, None]
    j = torch.arange(Nk)[None, None, :]
    ok = torch.ones((B, Nq, Nk), dtype=torch.bool)
    if right is not None:
        ok &= j <= p + right
    if left is not None:
        ok &= (j >= p - left) | (j < sinks)
    ok &= (p >= 0) & (p < Nk)
    if mask is not None:
        m = mask.cpu().bool()
        ok &= m[:, None, :] & torch.gather(m, 1, p[:, :, 0].clamp(0, Nk - 1))[:, :, None]
    return ok


def _heads(x, H):
    """[B, N, Hx, d] -> [B, H, N, d] float64, key heads repeated over their group."""
    x = x.detach().cpu().to(D64).permute(0, 2, 1, 3)
    return x.repeat_interleave(H // x.shape[1], dim=1)


def _clean(x, ok):
    """Zero where nothing may be read, whatever stands there."""
    return torch.where(ok, x, torch.zeros((), dtype=D64))


def window_attention(q, k, v, left, right, sinks=0, mask=None, q_start=None, scale: Optional[float] = None):
    """{"out" [B,Nq,H,Dv], "lse" [B,H,Nq], "P", "S", "ok" [B,H,Nq,Nk]} in float64."""
    B, Nq, H, D = q.shape
    Nk = k.shape[1]
    ok = visible(B, Nq, Nk, left, right, sinks, mask, q_start)
    row, key = ok.any(2)[:, None, :, None], ok.any(1)[:, None, :, None]
    Q, K, V = _clean(_heads(q, H), row), _clean(_heads(k, H), key), _clean(_heads(v, H), key)
    S = (Q @ K.transpose(-1, -2)) * (1.0 / math.sqrt(D) if scale is None else scale)
    okh = ok[:, None].expand_as(S)
    S = S.masked_fill(~okh, -math.inf)
    lse = torch.logsumexp(S, -1)
    P = torch.exp(S - lse.masked_fill(lse == -math.inf, 0.0)[..., None])
    return {"out": (P @ V).permute(0, 2, 1, 3).contiguous(), "lse": lse, "P": P, "S": S, "ok": okh, "Q": Q, "K": K, "V": V}


def window_attention_backward(q, k, v, d_out, left, right, sinks=0, mask=None, q_start=None, scale=None):
    """Gradients of <d_out, out> by the formulas; key heads sum over their group."""
    f = window_attention(q, k, v, left, right, sinks, mask, q_start, scale)
    B, Nq, H, D = q.shape
    Hkv = k.shape[2]
    sc = 1.0 / math.sqrt(D) if scale is None else scale
    dO = _clean(_heads(d_out, H), f["ok"].any(-1, keepdim=True))
    O = f["P"] @ f["V"]
    dS = f["P"] * (dO @ f["V"].transpose(-1, -2) - (dO * O).sum(-1, keepdim=True))
    fold = lambda x: x.view(B, Hkv, H // Hkv, *x.shape[2:]).sum(2).permute(0, 2, 1, 3).contiguous()  # noqa: E731
    return {"q": (sc * dS @ f["K"]).permute(0, 2, 1, 3).contiguous(),
            "k": fold(sc * dS.transpose(-1, -2) @ f["Q"]), "v": fold(f["P"].transpose(-1, -2) @ dO),
            "dS": dS, "dO": dO, "O": O, "f": f, "scale": sc, "fold": fold}


# --------------------------------------------------------- norm / gate / residual
def norm(z, kind, eps):
    """(zhat, mean, rstd) over the last axis."""
    mean = z.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(z[..., :1])
    c = z - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    return c * rstd, mean, rstd


def norm_residual(s, u=None, gate=None, res_scale=None, post=None, pre=None, mask=None, norm_kind="layer", eps=1e-5):
    """{"r", "x"} in float64; every intermediate beside them."""
    f = lambda t: None if t is None else t.detach().cpu().to(D64)  # noqa: E731
    s, u, gate = f(s), f(u), f(gate)
    live = torch.ones(s.shape[:-1], dtype=torch.bool) if mask is None else mask.cpu().bool()
    live = live[..., None]
    o = {"live": live, "s": s}
    r = s
    if u is not None:
        u = _clean(u, live)
        o["uhat"], o["mu"], o["ru"] = norm(u, norm_kind, eps)
        pw, pb = (f(t) for t in post) if post else (None, None)
        y = u if pw is None else o["uhat"] * pw + (0.0 if pb is None else pb)
        sg = 1.0 / (1.0 + torch.exp(-_clean(gate, live))) if gate is not None else torch.ones_like(y)
        ga = f(res_scale) if res_scale is not None else torch.ones(s.shape[-1], dtype=D64)
        o |= {"y": y, "sg": sg, "ga": ga, "pw": pw, "pb": pb, "u": u}
        r = s + _clean(ga * sg * y, live)
    o["r"] = r
    if pre:
        qw, qb = (f(t) for t in pre)
        o["rhat"], o["mr"], o["rr"] = norm(_clean(r, live), norm_kind, eps)
        o |= {"qw": qw, "qb": qb, "x": _clean(o["rhat"] * qw + (0.0 if qb is None else qb), live)}
    return o


def _norm_grad(h, zhat, rstd, kind):
    d = h - zhat * (h * zhat).mean(-1, keepdim=True)
    return rstd * (d - h.mean(-1, keepdim=True) if kind == "layer" else d)


def norm_residual_backward(s, u, d_r, d_x, gate=None, res_scale=None, post=None, pre=None, mask=None,
                           norm_kind="layer", eps=1e-5):
    """Gradients of <d_r, r> + <d_x, x> (either None: zero) by the formulas."""
    o = norm_residual(s, u, gate, res_scale, post, pre, mask, norm_kind, eps)
    live, f = o["live"], lambda t: t.detach().cpu().to(D64)
    rows = lambda t: t.reshape(-1, t.shape[-1]).sum(0)  # noqa: E731
    dt = f(d_r) if d_r is not None else torch.zeros_like(o["s"])
    g = {}
    if pre:
        dx = _clean(f(d_x), live) if d_x is not None else torch.zeros_like(o["s"])
        g |= {"pre_w": rows(dx * o["rhat"]), "pre_b": rows(dx), "dx": dx}
        dt = dt + _clean(_norm_grad(dx * o["qw"], o["rhat"], o["rr"], norm_kind), live)
    g["s"] = dt
    if u is not None:
        da = _clean(dt, live)
        dgy = da * o["ga"]
        dy = dgy * o["sg"]
        g |= {"res_scale": rows(da * o["sg"] * o["y"]), "gate": dgy * o["y"] * o["sg"] * (1 - o["sg"]),
              "post_w": rows(dy * o["uhat"]), "post_b": rows(dy), "da": da, "dy": dy,
              "u": _clean(_norm_grad(dy * o["pw"], o["uhat"], o["ru"], norm_kind) if post else dy, live)}
    return g | {"o": o}


# ---------------------------------------------------------------- embedding
def embedding(idx, table, scale=1.0):
    idx, table = idx.cpu().long(), table.detach().cpu().to(D64)
    ok = (idx >= 0) & (idx < table.shape[0])
    return _clean(scale * table[idx.clamp(0, table.shape[0] - 1)], ok[..., None])


def embedding_backward(idx, d_out, V, scale=1.0):
    idx, d = idx.cpu().long().reshape(-1), d_out.detach().cpu().to(D64).reshape(-1, d_out.shape[-1])
    ok = (idx >= 0) & (idx < V)
    return torch.zeros((V, d.shape[1]), dtype=D64).index_add_(0, idx[ok], d[ok]) * scale
