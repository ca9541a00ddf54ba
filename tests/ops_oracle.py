"""Plain 64-bit forms of the scan, norm and beam calls, written from their
formulas, with the bounds their tests hold the kernels to.

Bounds are running error bounds: E carries, beside each exact value, the sum of
the magnitudes whose roundings reach it, so that a kernel whose steps each
round a few times in fp32 stays within K * 2^-24 * E. K counts those roundings:
a gate to about 2 units (its exponential, its reciprocal with a Newton step),
the product beta x, the fused multiply-add, and the second rounding that the
tiled order adds to the products of decays: fewer than 12 half units of
2^-24 per step and magnitude. Storing in the tensors' type adds half a step of it.
"""
import math

import torch

U32 = 2.0 ** -24
K = 12.0


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gates64(a, b, logits):
    """alpha, 1 - alpha and beta in 64 bits."""
    a = a.double()
    if logits:
        alpha, keep = torch.sigmoid(-a), torch.sigmoid(a)
        beta = keep if b is None else torch.sigmoid(b.double())
    else:
        alpha, keep = a, 1.0 - a
        beta = keep if b is None else b.double()
    return alpha, keep, beta


def scan64(x, a, b, h0, logits):
    """One sequence [T, D]: all states h [T, D] and their running errors."""
    alpha, _, beta = gates64(a, b, logits)
    u = beta * x.double()
    T, D = u.shape
    h = torch.zeros(D, dtype=torch.float64) if h0 is None else h0.double()
    E = torch.zeros_like(h)
    hs, es = [], []
    for t in range(T):
        ah = alpha[t] * h
        h = ah + u[t]
        E = alpha[t].abs() * E + ah.abs() + u[t].abs()
        hs.append(h)
        es.append(E)
    if not hs:
        return torch.zeros(0, D, dtype=torch.float64), torch.zeros(0, D, dtype=torch.float64)
    return torch.stack(hs), torch.stack(es)


def scan_backward64(dy, x, a, b, h0, dhT, logits):
    """Gradients of one sequence and their running errors, as dicts."""
    alpha, keep, beta = gates64(a, b, logits)
    x, dy = x.double(), dy.double()
    T, D = x.shape
    h, eh = scan64(x, a, b, h0, logits)
    first = torch.zeros(1, D, dtype=torch.float64) if h0 is None else h0.double()[None]
    before = torch.cat([first, h[:-1]]) if T else first[:0]
    e_before = torch.cat([torch.zeros(1, D, dtype=torch.float64), eh[:-1]]) if T else first[:0]
    c = torch.zeros(D, dtype=torch.float64) if dhT is None else dhT.double()
    F = torch.zeros_like(c)
    g, eg = torch.zeros(T, D, dtype=torch.float64), torch.zeros(T, D, dtype=torch.float64)
    for t in range(T - 1, -1, -1):
        g[t] = dy[t] + c
        eg[t] = F + dy[t].abs() + c.abs()
        c = alpha[t] * g[t]
        F = alpha[t].abs() * eg[t] + c.abs()
    out = {"dx": g * beta, "dh0": c}
    err = {"dx": eg * beta.abs() + out["dx"].abs(), "dh0": F}
    inner = before - x if b is None else before
    e_inner = e_before + before.abs() + (x.abs() if b is None else 0.0)
    slope = -alpha * keep if logits else torch.ones_like(alpha)
    out["da"] = g * inner * slope
    err["da"] = slope.abs() * (eg * inner.abs() + g.abs() * e_inner) + out["da"].abs()
    if b is not None:
        sb = beta * torch.sigmoid(-b.double()) if logits else torch.ones_like(beta)
        out["db"] = g * x * sb
        err["db"] = sb.abs() * eg * x.abs() + out["db"].abs()
    return out, err


def assert_scan_close(got, want, err, dtype, what):
    got = got.detach().cpu().double()
    tol = K * U32 * err + (half_step(dtype) * want.abs() * (1 + 2.0 ** -8)
                           if dtype != torch.float32 else 0.0)
    bad = (got - want).abs() > tol + 1e-37
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs().max()),
                           float(((got - want).abs() / (tol + 1e-37)).max()))


def norm64(x, w, res, eps):
    r = x.double() + (0.0 if res is None else res.double())
    s = 1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    return r, s, r * s * w.double()


def norm_backward64(dy, r, w, dres, eps):
    """(dx, dw) and the magnitudes their roundings are relative to."""
    dy, r, w = dy.double(), r.double(), w.double()
    s = 1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    t = dy * w
    dx = s * t - r * s ** 3 * (t * r).mean(-1, keepdim=True)
    mag = (s * t).abs() + r.abs() * s ** 3 * (t * r).abs().mean(-1, keepdim=True)
    if dres is not None:
        dx = dx + dres.double()
        mag = mag + dres.double().abs()
    return dx, (dy * r * s).sum(0), mag, (dy * r * s).abs().sum(0)


def beam64(logits, scores, finished, eos):
    """Keys of all candidates [B, W * V] in 64 bits."""
    lg, sc = logits.double(), scores.double()
    B, W, V = lg.shape
    # a row with a NaN or +inf logit, or nothing but -inf, or a score that is not finite, is dead
    dead = (lg.isnan() | (lg == math.inf)).any(-1) | (lg == -math.inf).all(-1)
    done = torch.zeros(B, W, dtype=torch.bool) if finished is None else finished.bool()
    m = lg.nan_to_num(nan=0.0, posinf=0.0, neginf=-1e300).amax(-1, keepdim=True)
    key = sc[..., None] + ((lg - m) - torch.log(torch.exp(lg - m).sum(-1, keepdim=True)))
    key[dead] = -math.inf
    only = torch.full_like(key, -math.inf)
    if eos >= 0:
        only[..., eos] = sc
    key = torch.where(done[..., None], only, key)
    key[~sc.isfinite()] = -math.inf
    return key.reshape(B, W * V)


def beam_order(key, W):
    """The W best of each row: largest first, lowest place of equals."""
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :W]
