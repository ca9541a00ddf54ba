"""Cases of the operators beside the token mixer, and their plain forms.

Three families:
  scan   the gated linear recurrence h_t = alpha_t h_{t-1} + beta_t x_t per
         channel: prompt (dense, packed), training (forward and backward),
         single tokens against a pool of state slots;
  norm   root-mean-square norm with the residual's addition and an output in
         8 bits with scales, and its training form (forward and backward);
  beam   beam search's selection over beams and vocabulary, with the states
         reordered by it.

run(state) makes one pass: the library's calls where `own` is true, elementary
torch operations in 32 bits (64 where a comparison hangs on it) otherwise.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
EPS = 1e-6
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100  # smallest 8-bit scale: groups of zeros keep a finite one


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's rows of a 5,120-wide residual stream, 128-column scales
        {"name": "norm_token", "op": "norm", "rows": 8, "D": 5120, "group": 128, "res": True,
         "dtype": "bf16"},
        # a prompt's rows in front of the mixer's 8-bit projections
        {"name": "norm_prompt", "op": "norm", "rows": 16384, "D": 5120, "group": 128,
         "res": True, "dtype": "bf16"},
        # the mixer's output per value head (4,096 tokens x 48 heads of 128), one scale per row
        {"name": "norm_heads", "op": "norm", "rows": 196608, "D": 128, "group": 0, "res": False,
         "dtype": "bf16"},
        # training: norm and its gradients over a ragged number of rows
        {"name": "norm_train", "op": "norm_train", "rows": 8191, "D": 4096, "dtype": "bf16"},
        # one long prompt, 48 x 128 channels
        {"name": "scan_prompt", "op": "scan", "B": 1, "T": 65536, "D": 6144, "tied": False,
         "dtype": "bf16"},
        # a packed batch of prompts of very different lengths
        {"name": "scan_packed", "op": "scan_packed", "N": 33, "total": 20011, "D": 2048,
         "tied": False, "dtype": "f32"},
        # a training step: forward with prefix states, then backward
        {"name": "scan_train", "op": "scan_train", "B": 4, "T": 4097, "D": 2048, "tied": False,
         "dtype": "bf16"},
        # the same in fp32 with the tied gate and an odd width
        {"name": "scan_train_tied", "op": "scan_train", "B": 2, "T": 1000, "D": 1111,
         "tied": True, "dtype": "f32"},
        # one token per sequence of a serving batch, states in a pool of slots
        {"name": "scan_token", "op": "scan_token", "B": 64, "K": 1, "D": 6144, "dtype": "bf16"},
        # one sequence's four beams: latency
        {"name": "beam_token", "op": "beam", "B": 1, "W": 4, "V": 32000, "state": 0,
         "dtype": "f32"},
        # a batch of beams over a large vocabulary
        {"name": "beam_batch", "op": "beam", "B": 32, "W": 8, "V": 131072, "state": 0,
         "dtype": "bf16"},
        # selection, and the 48 x 128 x 128 fp32 states of one layer reordered by it
        {"name": "beam_states", "op": "beam", "B": 8, "W": 4, "V": 65537, "state": 48,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: half of them multiples of 64, the others as they fall (odd ones among them)."""
    d = _log(rng, lo, hi)
    return max(lo, d // 64 * 64) if rng.random() < 0.5 else d


def draw(rng):
    op = rng.choice(["norm", "norm_train", "scan", "scan_packed", "scan_train", "scan_token",
                     "beam", "beam"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        D = _width(rng, 64, 8192)
        return {"op": op, "rows": _log(rng, 1, min(262144, (1 << 26) // D)), "D": D,
                "group": rng.choice([0, 128]), "res": rng.random() < 0.7, "dtype": dtype}
    if op == "norm_train":
        D = _width(rng, 64, 8192)
        return {"op": op, "rows": _log(rng, 1, min(262144, (1 << 25) // D)), "D": D,
                "dtype": dtype}
    if op in ("scan", "scan_train"):
        D = _width(rng, 64, 8192)
        tokens = (1 << 27 if op == "scan" else 1 << 25) // D
        T = _log(rng, 1, min(32768, tokens))
        B = _log(rng, 1, max(1, min(64, tokens // T)))
        return {"op": op, "B": B, "T": T, "D": D, "tied": rng.random() < 0.3, "dtype": dtype}
    if op == "scan_packed":
        D = _width(rng, 64, 4096)
        N = _log(rng, 1, 128)
        return {"op": op, "N": N, "total": _log(rng, N, 24576), "D": D,
                "tied": rng.random() < 0.3, "dtype": dtype}
    if op == "scan_token":
        return {"op": op, "B": _log(rng, 1, 512), "K": _log(rng, 1, 8),
                "D": _width(rng, 64, 8192), "dtype": dtype}
    W = _log(rng, 1, 16)
    V = _log(rng, 500, 262144)
    state = rng.choice([0, 0, 16, 48])
    B = _log(rng, 1, max(1, min(64, (1 << 25) // (W * V), 64 // W if state else 64)))
    return {"op": "beam", "B": B, "W": W, "V": V, "state": state, "dtype": dtype}


# --------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _lengths(g, N, total):
    """N lengths that add up to total: one of them empty where there are enough sequences, the
    others spread over two powers of ten."""
    w = torch.exp(_randn(g, N).cpu().double() * 1.2)
    if N > 3:
        w[1] = 0.0
    cuts = torch.round(torch.cumsum(w, 0) / w.sum() * total).to(torch.int32)
    cuts[-1] = total
    return torch.cat([torch.zeros(1, dtype=torch.int32), cuts])


def _scan_inputs(g, lead, D, n, tied, dt):
    """x, gate logits (decays from a few tokens to thousands) and initial states of n sequences."""
    x = _randn(g, *lead, D, dtype=dt)
    a = (_randn(g, *lead, D) * 1.0 - torch.linspace(1.0, 7.0, D, device=DEV)).to(dt)
    b = None if tied else _randn(g, *lead, D, dtype=dt)
    return {"x": x, "a": a, "b": b, "h0": _randn(g, n, D)}


def prepare(case, seed):
    g = _gen(seed)
    c = case
    op, dt = c["op"], DT[c["dtype"]]
    s = {"case": c}
    if op in ("norm", "norm_train"):
        R, D = c["rows"], c["D"]
        s["x"] = _randn(g, R, D, dtype=dt)
        s["w"] = (1.0 + 0.2 * _randn(g, D)).to(dt)
        if c.get("res", True):
            s["res"] = (2.0 * _randn(g, R, D)).to(dt)
        if op == "norm_train":
            s["dy"] = _randn(g, R, D, dtype=dt)
            s["dres"] = _randn(g, R, D, dtype=dt)
    elif op in ("scan", "scan_train"):
        s.update(_scan_inputs(g, (c["B"], c["T"]), c["D"], c["B"], c["tied"], dt))
        if op == "scan_train":
            s["dy"] = _randn(g, c["B"], c["T"], c["D"], dtype=dt)
            s["dhT"] = _randn(g, c["B"], c["D"])
    elif op == "scan_packed":
        cu = _lengths(g, c["N"], c["total"])
        s.update(_scan_inputs(g, (c["total"],), c["D"], c["N"], c["tied"], dt))
        s["cu"] = cu.to(DEV)
    elif op == "scan_token":
        B, K, D = c["B"], c["K"], c["D"]
        s.update(_scan_inputs(g, (B, K), D, 2 * B, False, dt))
        perm = torch.randperm(2 * B, generator=g, device=DEV).to(torch.int32)
        s["src"], s["dst"] = perm[:B].contiguous(), perm[B:].contiguous()
        s["pool"] = s.pop("h0")
    else:
        B, W, V = c["B"], c["W"], c["V"]
        s["logits"] = (3.0 * _randn(g, B, W, V)).to(dt)
        s["scores"] = -20.0 + 2.0 * _randn(g, B, W)
        s["finished"] = (torch.rand(B, W, generator=g, device=DEV) < 0.15).to(torch.uint8)
        s["eos"] = 2
        s["slots"] = torch.randperm(B * W, generator=g, device=DEV).to(torch.int32).view(B, W)
        if c["state"]:
            s["states"] = _randn(g, B * W, c["state"], 128, 128)
    return s


# ------------------------------------------------------------ plain forms

def _gates(a, b):
    a = a.float()
    alpha = 1.0 / (1.0 + torch.exp(a))
    keep = 1.0 / (1.0 + torch.exp(-a))  # 1 - alpha without the cancellation
    beta = keep if b is None else 1.0 / (1.0 + torch.exp(-b.float()))
    return alpha, keep, beta


def _doubling(A, U):
    """h_t = A_t h_{t-1} + U_t over dim 1 from a zero state, by doubling the span."""
    T, s = U.shape[1], 1
    while s < T:
        U = torch.cat([U[:, :s], U[:, s:] + A[:, s:] * U[:, :-s]], 1)
        A = torch.cat([A[:, :s], A[:, s:] * A[:, :-s]], 1)
        s *= 2
    return U


def _plain_scan(s):
    x, h0 = s["x"].float(), s["h0"]
    alpha, _, beta = _gates(s["a"], s["b"])
    U = beta * x
    U[:, 0] += alpha[:, 0] * h0
    h = _doubling(alpha, U)
    return h.to(s["x"].dtype), h[:, -1].contiguous()


def _plain_packed(s):
    x, h0, cu = s["x"].float(), s["h0"], s["cu"].long()
    alpha, _, beta = _gates(s["a"], s["b"])
    U = beta * x
    some = cu[1:] > cu[:-1]
    starts = cu[:-1][some]
    U[starts] += alpha[starts] * h0[some]
    alpha[starts] = 0.0  # nothing crosses a sequence's start
    h = _doubling(alpha[None], U[None])[0]
    final = torch.where(some[:, None], h[(cu[1:] - 1).clamp(min=0)], h0)
    return h.to(s["x"].dtype), final


def _plain_scan_train(s):
    dt = s["x"].dtype
    x, h0, dy = s["x"].float(), s["h0"], s["dy"].float()
    alpha, keep, beta = _gates(s["a"], s["b"])
    U = beta * x
    U[:, 0] += alpha[:, 0] * h0
    h = _doubling(alpha, U)
    prev = torch.cat([h0[:, None], h[:, :-1]], 1)
    # g_t = dy_t + alpha_{t+1} g_{t+1}, run from the end
    G = dy.clone()
    G[:, -1] += s["dhT"]
    nxt = torch.cat([alpha[:, 1:], torch.zeros_like(alpha[:, :1])], 1)
    g = _doubling(nxt.flip(1), G.flip(1)).flip(1)
    dx = (g * beta).to(dt)
    if s["b"] is None:
        da = (-alpha * keep * g * (prev - x)).to(dt)
        db = None
    else:
        da = (-alpha * keep * g * prev).to(dt)
        db = (beta * (1.0 - beta) * g * x).to(dt)
    return [h.to(dt), h[:, -1].contiguous(), dx, da, db, alpha[:, 0] * g[:, 0]]


def _plain_scan_token(s):
    x = s["x"].float()
    alpha, _, beta = _gates(s["a"], s["b"])
    h = s["pool"][s["src"].long()]
    outs = []
    for k in range(x.shape[1]):
        h = alpha[:, k] * h + beta[:, k] * x[:, k]
        outs.append(h)
    s["pool"][s["dst"].long()] = h
    return torch.stack(outs, 1).to(s["x"].dtype), s["pool"]


def _plain_norm_y(s):
    r = s["x"].float()
    if "res" in s:
        r = r + s["res"].float()
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    return r, rstd, r * rstd * s["w"].float()


def _plain_norm(s):
    r, _, y = _plain_norm_y(s)
    R, D = y.shape
    group = s["case"]["group"] or D
    n = -(-D // group)
    z = torch.nn.functional.pad(y, (0, n * group - D)).view(R, n, group)
    scale = z.abs().amax(-1).clamp(min=E4M3_MAX * SCALE_FLOOR) / E4M3_MAX
    q = (z / scale[..., None]).view(R, n * group)[:, :D]
    out = [q.to(torch.float8_e4m3fn).contiguous(), scale]
    return out + ([r.to(s["x"].dtype)] if "res" in s else [])


def _plain_norm_train(s):
    dt = s["x"].dtype
    r, rstd, y = _plain_norm_y(s)
    res_out = r.to(dt)
    # the gradient is taken at the residual stream as it is kept
    r = res_out.float()
    D = r.shape[1]
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    dy, w = s["dy"].float(), s["w"].float()
    t = dy * w
    dr = rstd * t - r * (rstd * rstd * rstd / D) * (t * r).sum(-1, keepdim=True)
    dw = (dy * (r * rstd)).sum(0)
    return [y.to(dt), res_out, (dr + s["dres"].float()).to(dt), dw]


def _plain_beam(s):
    lg, W, V = s["logits"].double(), s["case"]["W"], s["case"]["V"]
    B = lg.shape[0]
    m = lg.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(lg - m).sum(-1, keepdim=True))
    score = s["scores"].double()[..., None]
    key = score + (lg - lse)
    done = s["finished"].bool()[..., None]
    tok = torch.arange(V, device=lg.device)
    key = torch.where(done, torch.where(tok == s["eos"], score, -math.inf), key).view(B, W * V)
    place = torch.arange(W * V, device=lg.device)
    scores, picks = [], []
    for _ in range(W):  # the largest, the lowest place of equal ones, W times
        best = key.amax(-1, keepdim=True)
        at = torch.where(key == best, place, W * V).amin(-1, keepdim=True)
        key = key.scatter(1, at, math.nan).nan_to_num(nan=-math.inf, neginf=-math.inf)
        scores.append(best)
        picks.append(at)
    scores, picks = torch.cat(scores, 1), torch.cat(picks, 1)
    parents, tokens = picks // V, picks % V
    fin = s["finished"].gather(1, parents).bool() | (tokens == s["eos"])
    slots = s["slots"].gather(1, parents)
    out = [scores.float(), tokens.int(), parents.int(), fin.to(torch.uint8), slots]
    return out + ([s["states"][slots.view(-1).long()]] if "states" in s else [])


# ------------------------------------------------------------------- run

def _own(s):
    import gated_deltanet_token_amd as gdn
    op = s["case"]["op"]
    if op == "norm":
        _, q, scale, r = gdn.gdn_rms_norm(s["x"], s["w"], s.get("res"), eps=EPS,
                                          group=s["case"]["group"], want_out=False,
                                          want_out8=True)
        return [q, scale] + ([r] if r is not None else [])
    if op == "norm_train":
        y, _, _, r = gdn.gdn_rms_norm(s["x"], s["w"], s["res"], eps=EPS)
        dx, dw = gdn.gdn_rms_norm_backward(s["dy"], r, s["w"], s["dres"], eps=EPS)
        return [y, r, dx, dw]
    if op == "scan":
        return gdn.gdn_scan_prefill(s["x"], s["a"], s["b"], s["h0"], flags=gdn.GDN_GATE_LOGITS)
    if op == "scan_packed":
        return gdn.gdn_scan_varlen_prefill(s["x"], s["a"], s["b"], s["cu"], s["h0"],
                                           flags=gdn.GDN_GATE_LOGITS)
    if op == "scan_train":
        x = s["x"]
        pre = torch.empty(gdn.prefix_state_rows(x.shape[0], x.shape[1], 2, False), x.shape[2],
                          device=x.device)
        y, hT = gdn.gdn_scan_prefill(x, s["a"], s["b"], s["h0"], prefix_states=pre,
                                     prefix_interval=2, flags=gdn.GDN_GATE_LOGITS)
        grads = gdn.gdn_scan_backward(s["dy"], x, s["a"], s["b"], s["h0"], prefix_states=pre,
                                      prefix_interval=2, dfinal=s["dhT"],
                                      flags=gdn.GDN_GATE_LOGITS)
        return [y, hT, *grads]
    if op == "scan_token":
        y = gdn.gdn_scan_decode(s["x"], s["a"], s["b"], s["pool"], s["src"], s["dst"],
                                flags=gdn.GDN_GATE_LOGITS)
        return y, s["pool"]
    out = gdn.gdn_beam_select(s["logits"], s["scores"], finished=s["finished"], eos=s["eos"],
                              beam_slots=s["slots"])
    if "states" not in s:
        return list(out)
    return [*out, gdn.gdn_gather_states(s["states"], out[4].view(-1))]


_PLAIN = {"norm": _plain_norm, "norm_train": _plain_norm_train, "scan": _plain_scan,
          "scan_packed": _plain_packed, "scan_train": _plain_scan_train,
          "scan_token": _plain_scan_token, "beam": _plain_beam}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    op, e = c["op"], ES[c["dtype"]]
    if op == "norm":
        n = c["rows"] * c["D"]
        groups = c["rows"] * (-(-c["D"] // c["group"]) if c["group"] else 1)
        return {"bytes": n * (e * (3 if c["res"] else 1) + 1) + c["D"] * e + groups * 4,
                "flops": n * 7}
    if op == "norm_train":  # forward x, res -> y, r; backward dy, r, dres -> dx
        n = c["rows"] * c["D"]
        return {"bytes": n * e * 8 + c["D"] * (2 * e + 4), "flops": n * 16}
    if op in ("scan", "scan_train"):
        n, rows = c["B"] * c["T"] * c["D"], c["B"] * c["D"] * 4
        io = 3 if c["tied"] else 4
        if op == "scan":
            return {"bytes": n * e * io + 2 * rows, "flops": n * 9}
        return {"bytes": n * e * (io + (5 if c["tied"] else 7)) + 5 * rows, "flops": n * 30}
    if op == "scan_packed":
        n = c["total"] * c["D"]
        return {"bytes": n * e * (3 if c["tied"] else 4) + 2 * c["N"] * c["D"] * 4,
                "flops": n * 9}
    if op == "scan_token":
        n = c["B"] * c["K"] * c["D"]
        return {"bytes": n * e * 4 + 2 * c["B"] * c["D"] * 4, "flops": n * 9}
    # every state row is written; at the least one row is read for each batch item
    state = (c["B"] * c["W"] + c["B"]) * c["state"] * 128 * 128 * 4
    n = c["B"] * c["W"] * c["V"]
    return {"bytes": n * e + c["B"] * c["W"] * 30 + state, "flops": n * 3}


# ----------------------------------------------------------------- exact

def _sig(z):
    return torch.sigmoid(z.double())


def _walk(alpha, u, h):
    """The recurrence token by token; alpha, u [B, T, D] in 64 bits. All h_t."""
    out = torch.empty_like(u)
    for t in range(u.shape[1]):
        h = torch.addcmul(u[:, t], alpha[:, t], h, out=out[:, t])
    return out


def _exact_scan(s):
    beta = _sig(s["a"]) if s["b"] is None else _sig(s["b"])
    h = _walk(_sig(-s["a"].double()), beta * s["x"].double(), s["h0"].double())
    return h


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "scan":
        h = _exact_scan(s)
        return h, h[:, -1]
    if op == "scan_packed":
        outs, finals = [], []
        cu = s["cu"].tolist()
        for n in range(case["N"]):
            lo, hi = cu[n], cu[n + 1]
            part = {"x": s["x"][None, lo:hi], "a": s["a"][None, lo:hi], "h0": s["h0"][n:n + 1],
                    "b": None if s["b"] is None else s["b"][None, lo:hi]}
            h = _exact_scan(part)[0]
            outs.append(h)
            finals.append(h[-1] if hi > lo else s["h0"][n].double())
        return torch.cat(outs), torch.stack(finals)
    if op == "scan_train":
        h = _exact_scan(s)
        x, h0 = s["x"].double(), s["h0"].double()
        alpha = _sig(-s["a"].double())
        g = torch.empty_like(h)
        back = s["dhT"].double()
        for t in range(h.shape[1] - 1, -1, -1):
            torch.add(s["dy"][:, t], back, out=g[:, t])
            back = alpha[:, t] * g[:, t]
        before = torch.cat([h0.unsqueeze(1), h[:, :-1]], 1)
        if s["b"] is None:
            beta, db = _sig(s["a"]), None
            dalpha = g * (before - x)
        else:
            beta = _sig(s["b"])
            db = g * x * beta * _sig(-s["b"].double())
            dalpha = g * before
        return [h, h[:, -1], g * beta, -dalpha * alpha * _sig(s["a"]), db, back]
    if op == "scan_token":
        h = _walk(_sig(-s["a"].double()), _sig(s["b"]) * s["x"].double(),
                  s["pool"].double()[s["src"].long()])
        pool = s["pool"].double()
        pool[s["dst"].long()] = h[:, -1]
        return h, pool
    if op in ("norm", "norm_train"):
        r = s["x"].double() + (s["res"].double() if "res" in s else 0.0)
        w = s["w"].double()
        rms = torch.sqrt(r.square().mean(1, keepdim=True) + EPS)
        y = r / rms * w
        if op == "norm_train":
            kept = r.to(s["x"].dtype).double()
            rms = torch.sqrt(kept.square().mean(1, keepdim=True) + EPS)
            unit = kept / rms
            t = s["dy"].double() * w
            dx = (t - unit * (t * unit).mean(1, keepdim=True)) / rms + s["dres"].double()
            return [y, r, dx, (s["dy"].double() * unit).sum(0)]
        cols = case["group"] or case["D"]
        parts = [p.abs().amax(1, keepdim=True) / E4M3_MAX for p in y.split(cols, 1)]
        q = [p / sc for p, sc in zip(y.split(cols, 1), parts)]
        return [torch.cat(q, 1), torch.cat(parts, 1)] + ([r] if "res" in s else [])
    # beam: the scores of the selected candidates, best first; what is chosen is whole numbers
    total = s["scores"].double()[..., None] + torch.log_softmax(s["logits"].double(), -1)
    done = s["finished"].bool()
    total[done] = -math.inf
    total[..., s["eos"]] = torch.where(done, s["scores"].double(), total[..., s["eos"]])
    best = total.flatten(1).topk(case["W"], 1).values
    return [best] + [None] * (5 if "states" in s else 4)
