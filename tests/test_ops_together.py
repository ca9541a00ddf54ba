"""The scan, norm and beam calls as a program uses them together: a beam-search
decode loop over state slots, a training step, graphs, streams and workspaces."""
import pytest

torch = pytest.importorskip("torch")
from tests.ops_oracle import U32, K, scan64  # noqa: E402

DEV = "cuda:0"
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_token_amd as g
    g.load_library()
    return g


# ------------------------------------------------------------- beam decoding

def weights(seed, V, D):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"emb": r(V, D), "norm": 1 + 0.1 * r(D), "wa": r(D, D) / D ** 0.5,
            "wb": r(D, D) / D ** 0.5, "wx": r(D, D) / D ** 0.5, "out": 2 * r(D, V) / D ** 0.5}


def search64(w, first, W, steps, eos):
    """Beam search in 64 bits on the CPU, states reordered by hand. Per step: tokens, parents,
    scores, and the least distance between neighbouring candidates around the selected ones."""
    w = {k: v.double() for k, v in w.items()}
    B, V, D = len(first), w["emb"].shape[0], w["emb"].shape[1]
    h = torch.zeros(B, W, D, dtype=torch.float64)
    score = torch.full((B, W), -float("inf"), dtype=torch.float64)
    score[:, 0] = 0.0
    tok = first[:, None].expand(B, W).clone()
    fin = torch.zeros(B, W, dtype=torch.bool)
    out, gap = [], float("inf")
    for _ in range(steps):
        r = w["emb"][tok] + h
        y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-6) * w["norm"]
        h = torch.sigmoid(-(y @ w["wa"])) * h + torch.sigmoid(y @ w["wb"]) * (y @ w["wx"])
        key = score[..., None] + torch.log_softmax(h @ w["out"], -1)
        only = torch.full_like(key, -float("inf"))
        only[..., eos] = score
        key = torch.where(fin[..., None], only, key).reshape(B, W * V)
        best = torch.sort(key, dim=1, descending=True, stable=True)
        gap = min(gap, float((best.values[:, :W] - best.values[:, 1:W + 1]).min()))
        place = best.indices[:, :W]
        par, tok, score = place // V, place % V, best.values[:, :W]
        h = h.gather(1, par[..., None].expand(B, W, D))
        fin = fin.gather(1, par) | (tok == eos)
        out.append((tok, par, score))
    return out, gap


@pytest.mark.parametrize("how", ["slots", "gather"])
def test_beam_decoding(gdn, how):
    """Norm, one recurrent token, logits, selection, states reordered: tokens of every step
    against the search in 64 bits."""
    V, D, B, W, steps, eos = 97, 64, 3, 4, 12, 5
    w = weights(11, V, D)
    first = torch.tensor([3, 50, 96])
    want, gap = search64(w, first, W, steps, eos)
    assert gap > 1e-4  # far above the fp32 path's error: the order is decided
    d = {k: v.to(DEV) for k, v in w.items()}
    n = B * W
    # two halves of slots in turn: no beam's destination is another's source
    pool = torch.zeros(2 * n, D, device=DEV)
    half = [torch.arange(n, dtype=torch.int32, device=DEV) + k * n for k in (0, 1)]
    src = half[0].clone()
    state = torch.zeros(n, D, device=DEV)
    score = torch.full((B, W), -float("inf"), device=DEV)
    score[:, 0] = 0.0
    fin = torch.zeros(B, W, dtype=torch.uint8, device=DEV)
    tok = first.to(DEV)[:, None].expand(B, W).to(torch.int32)
    for k in range(steps):
        h = state if how == "gather" else gdn.gdn_gather_states(pool, src)
        y, _, _, _ = gdn.gdn_rms_norm(d["emb"][tok.reshape(-1).long()], d["norm"], h)
        x, a, b = [(y @ d[m]).view(n, 1, D) for m in ("wx", "wa", "wb")]
        if how == "slots":
            dst = half[(k + 1) % 2]
            o = gdn.gdn_scan_decode(x, a, b, pool, src, dst, flags=gdn.GDN_GATE_LOGITS)
            now = dst
        else:
            now = half[0]
            o = gdn.gdn_scan_decode(x, a, b, state, now, now, flags=gdn.GDN_GATE_LOGITS)
        logits = (o[:, 0] @ d["out"]).view(B, W, V)
        score, tok, par, fin, nxt = gdn.gdn_beam_select(logits, score, finished=fin, eos=eos,
                                                        beam_slots=now.view(B, W))
        if how == "slots":
            src = nxt.reshape(-1)
        else:
            state = gdn.gdn_gather_states(state, nxt.reshape(-1))
        wt, wp, ws = want[k]
        assert torch.equal(tok.cpu().long(), wt) and torch.equal(par.cpu().long(), wp), k
        assert (score.cpu().double() - ws).abs().max() < 1e-3


def test_selection_drives_the_mixers_slots(gdn):
    """src_slots of the selection as the src_slot of the delta-rule decode: the same as gathering
    the states first and decoding in place."""
    B, W, H, D = 2, 3, 2, 64
    n = B * W
    g = torch.Generator().manual_seed(4)
    pool = torch.randn(2 * n, H, D, D, generator=g).to(DEV)
    logits = torch.randn(B, W, 50, generator=g).to(DEV)
    slots = torch.arange(n, dtype=torch.int32, device=DEV).view(B, W)
    _, _, par, _, src = gdn.gdn_beam_select(logits, torch.zeros(B, W, device=DEV), beam_slots=slots)
    q, k, v = [torch.randn(n, 1, H, D, generator=g).to(DEV) for _ in range(3)]
    al, be = [torch.rand(n, 1, H, generator=g).to(DEV) for _ in range(2)]
    gathered = gdn.gdn_gather_states(pool, src.reshape(-1))
    same = gathered.clone()
    ids = torch.arange(n, dtype=torch.int32, device=DEV)
    o2, _ = gdn.gdn_decode_multi(q, k, v, al, be, same, ids, ids)
    o1, _ = gdn.gdn_decode_multi(q, k, v, al, be, pool, src.reshape(-1), ids + n)
    assert torch.equal(o1, o2) and torch.equal(pool[n:], same)


# ------------------------------------------------------------- training step

def test_training_step(gdn):
    """Norm of x + residual, scan, a loss on the outputs and the last state: every gradient
    against automatic differentiation in 64 bits of the same formulas."""
    B, T, D = 2, 150, 72
    g = torch.Generator().manual_seed(21)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, res, a, b, w, h0 = r(B, T, D), r(B, T, D), 2 * r(B, T, D) - 2, r(B, T, D), 1 + 0.1 * r(D), \
        r(B, D)
    dy, dh, dres = r(B, T, D), r(B, D), r(B, T, D)
    leaves = [t.double().requires_grad_() for t in (x, res, a, b, w, h0)]
    X, R, A, Bt, Wt, H0 = leaves
    s = X + R
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-6) * Wt
    h, outs = H0, []
    for t in range(T):
        h = torch.sigmoid(-A[:, t]) * h + torch.sigmoid(Bt[:, t]) * y[:, t]
        outs.append(h)
    loss = (torch.stack(outs, 1) * dy.double()).sum() + (h * dh.double()).sum() \
        + (s * dres.double()).sum()
    want = torch.autograd.grad(loss, leaves)

    d = [t.to(DEV) for t in (x, res, a, b, w, h0, dy, dh, dres)]
    xd, rd, ad, bd, wd, hd, dyd, dhd, drd = d
    yd, _, _, sd = gdn.gdn_rms_norm(xd, wd, rd)
    pre = torch.empty(gdn.prefix_state_rows(B, T, 2, False), D, device=DEV)
    gdn.gdn_scan_prefill(yd, ad, bd, hd, prefix_states=pre, prefix_interval=2, flags=2)
    gy, ga, gb, gh = gdn.gdn_scan_backward(dyd, yd, ad, bd, hd, prefix_states=pre,
                                           prefix_interval=2, dfinal=dhd, flags=2)
    gx, gw = gdn.gdn_rms_norm_backward(gy, sd, wd, drd)
    # every value went through fewer than 2^7 roundings of 2^-24 relative to the largest value
    # beside it (decays below 0.9 here: memories of some ten tokens)
    for got, ref in zip((gx, gx, ga, gb, gw, gh), want):
        ref = ref.cpu()
        assert (got.cpu().double() - ref).abs().max() <= 2.0 ** -17 * ref.abs().max()


# ------------------------------------------- graphs, streams and workspaces

def everything(gdn, s, ws=None):
    """One pass through all calls, from and into the tensors of s."""
    kw = {} if ws is None else {"workspace": ws}
    y, q, sc, r = gdn.gdn_rms_norm(s["x"], s["w"], s["res"], group=128, want_out8=True)
    h, hT = gdn.gdn_scan_prefill(y, s["a"], s["b"], s["h0"], prefix_states=s["pre"],
                                 prefix_interval=2, flags=2, **kw)
    grads = gdn.gdn_scan_backward(s["dy"], y, s["a"], s["b"], s["h0"], prefix_states=s["pre"],
                                  prefix_interval=2, dfinal=hT, flags=2, **kw)
    gx, gw = gdn.gdn_rms_norm_backward(grads[0], r, s["w"], s["dy"])
    o = gdn.gdn_scan_decode(s["x"][:, :2].contiguous(), s["a"][:, :2].contiguous(),
                            s["b"][:, :2].contiguous(), s["pool"], s["src"], s["dst"], flags=2)
    beams = gdn.gdn_beam_select(s["logits"], s["score"], finished=s["fin"], eos=7,
                                beam_slots=s["slots"])
    moved = gdn.gdn_gather_states(s["pool"], beams[4].view(-1))
    return [y, q.view(torch.uint8), sc, r, h, hT, *grads, gx, gw, o, *beams, moved]


def make(seed, B=2, T=700, D=264):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = {k: r(B, T, D).bfloat16() for k in ("x", "res", "a", "b", "dy")}
    s.update(w=(1 + 0.1 * r(D)).bfloat16(), h0=r(B, D), pre=torch.empty(B * (T // 128), D),
             pool=r(4 * B, D), logits=3 * r(B, 2, 9001), score=r(B, 2),
             fin=(torch.rand(B, 2, generator=g) < 0.3).to(torch.uint8))
    ids = torch.randperm(4 * B, generator=g).to(torch.int32)
    s.update(src=ids[:B].clone(), dst=ids[B:2 * B].clone(), slots=ids[:2 * B].view(B, 2).clone())
    return {k: v.to(DEV) for k, v in s.items()}


def same(p, q):
    assert len(p) == len(q)
    for i, (a, b) in enumerate(zip(p, q)):
        assert torch.equal(a, b), i


def test_graph_replays(gdn):
    """All calls captured in one graph and replayed on new inputs, with eager work and
    synchronizations in between; a second graph shares the first one's workspace tensor."""
    static = make(1)
    n = gdn.gdn_scan_workspace_size(2, 700, 264, torch.bfloat16, False)
    assert n > 0  # the call is cut along time: counters and published words in the graph
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything(gdn, static)
        everything(gdn, static, ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for w in (None, ws, ws):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = everything(gdn, static, w)
        graphs.append((graph, outs))
    for seed in range(2, 7):
        fresh = make(seed)
        before = {k: v.clone() for k, v in fresh.items()}
        want = everything(gdn, fresh)
        torch.cuda.synchronize()
        for graph, outs in graphs:
            for k, v in before.items():
                static[k].copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            same(outs, want)
            assert torch.equal(static["pool"], fresh["pool"])
        ws.fill_(seed)  # what was left in the workspace does not matter


def test_other_streams(gdn):
    """On a stream that is not the current one, and on two at once with a workspace each."""
    s, t = make(30), make(31)
    keep = [{k: v.clone() for k, v in u.items()} for u in (s, t)]
    want = [everything(gdn, u) for u in keep]
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for u, stream in ((s, one), (t, two)):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            outs.append(everything(gdn, u))
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        same(got, ref)
    # named by argument, the current stream being another
    y, _, _, r = gdn.gdn_rms_norm(s["x"], s["w"], s["res"], stream=one)
    h, hT = gdn.gdn_scan_prefill(y, s["a"], s["b"], s["h0"], flags=2, stream=one)
    b = gdn.gdn_beam_select(s["logits"], s["score"], finished=s["fin"], eos=7, stream=two)
    one.synchronize()
    two.synchronize()
    same([y, r, h, hT, b[0], b[1]], [want[0][i] for i in (0, 3, 4, 5, 13, 14)])


@pytest.mark.parametrize("fill", [0x00, 0xFF, 0x5A])
def test_workspace_contents_do_not_matter(gdn, fill):
    s = make(40)
    keep = {k: v.clone() for k, v in s.items()}
    want = everything(gdn, keep)
    n = gdn.gdn_scan_workspace_size(2, 700, 264, torch.bfloat16, False)
    ws = torch.full((n + 64,), fill, dtype=torch.uint8, device=DEV)
    got = everything(gdn, s, ws[:n])
    same(got, want)
    assert (ws[n:] == fill).all()
    small = torch.full((n - 16,), fill, dtype=torch.uint8, device=DEV)
    s = make(40)
    same(everything(gdn, s, small), want)  # too small: the serial tiles, the same bits
    assert (small == fill).all()


def test_scan_after_other_work_on_its_rows(gdn):
    """Outputs given by the caller: rows behind the batch stay as they were."""
    T, D = 333, 40
    x, a, b = [torch.randn(1, T, D, device=DEV) for _ in range(3)]
    out = torch.full((1, T + 5, D), 9.0, device=DEV)
    h, hT = gdn.gdn_scan_prefill(x, a, b, out=out[:, :T], flags=2)
    assert h.data_ptr() == out.data_ptr() and (out[0, T:] == 9.0).all()
    want, err = scan64(x[0].cpu(), a[0].cpu(), b[0].cpu(), None, True)
    assert ((h[0].cpu().double() - want).abs() <= K * U32 * err + 1e-37).all()


def freed_after_the_call(call, *tensors):
    """call(stream, tensors...) on a busy side stream, its inputs freed at once and their memory
    written again on the current stream: the results are those of an undisturbed call."""
    want = [t.clone() for t in call(None, *[t.clone() for t in tensors]) if t is not None]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mine = [t.clone() for t in tensors]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # some 0.1 s
    got = [t for t in call(side, *mine) if t is not None]
    del mine
    other = [torch.empty_like(t) for t in tensors]
    for t in other:
        t.view(torch.uint8).fill_(0x3F)
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_inputs_freed_after_a_call_on_another_stream(gdn):
    s = make(50)
    freed_after_the_call(lambda st, x, w, r: gdn.gdn_rms_norm(x, w, residual=r, stream=st),
                         s["x"], s["w"], s["res"])
    freed_after_the_call(lambda st, dy, r, w: gdn.gdn_rms_norm_backward(dy, r, weight=w, stream=st),
                         s["dy"], s["x"], s["w"])
    freed_after_the_call(lambda st, x, a, b, h: gdn.gdn_scan_prefill(x, a, b, h, stream=st),
                         s["x"], s["a"], s["b"], s["h0"])
    freed_after_the_call(lambda st, lg, sc: gdn.gdn_beam_select(lg, scores=sc, stream=st),
                         s["logits"], s["score"])
    freed_after_the_call(lambda st, p, i: [gdn.gdn_gather_states(p, i, stream=st)],
                         s["pool"], s["src"])


def test_inputs_of_the_mixer_freed_after_a_call_on_another_stream(gdn):
    g = torch.Generator().manual_seed(51)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    B, T, Hk, Hv, D = 2, 200, 2, 4, 64
    q, k, v = 0.1 * r(B, T, Hk, D), 0.1 * r(B, T, Hk, D), r(B, T, Hv, D)
    al, be = torch.sigmoid(r(B, T, Hv)), torch.sigmoid(r(B, T, Hv))
    freed_after_the_call(lambda st, *t: gdn.gdn_prefill_chunked(*t, stream=st), q, k, v, al, be)
    cu = torch.tensor([0, 150, 400], dtype=torch.int32, device=DEV)
    flat = [t.flatten(0, 1) for t in (q, k, v, al, be)]
    freed_after_the_call(lambda st, *t: gdn.gdn_varlen_prefill(*t, stream=st), *flat, cu)
    freed_after_the_call(lambda st, *t: gdn.gdn_prefill_chunked_noalloc(*t, stream=st),
                         q, k, v, al, be)
    one = [t[:, 0].contiguous() for t in (q, k, v, al, be)]
    freed_after_the_call(lambda st, *t: [gdn.gdn_decode_step(*t, stream=st)], *one,
                         r(B, Hv, D, D))
    ids = torch.arange(B, dtype=torch.int32, device=DEV)
    freed_after_the_call(lambda st, *t: gdn.gdn_decode_multi(*t, stream=st),
                         *[t[:, :3].contiguous() for t in (q, k, v, al, be)], r(B, Hv, D, D), ids,
                         ids)


def test_autograd_through_a_function(gdn):
    """Results carry no history by themselves, as documented; the backward calls inside a
    torch.autograd.Function give every leaf the gradients that they give by hand."""
    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, res, w, a, b, h0):
            y, _, _, r = gdn.gdn_rms_norm(x, w, res)
            pre = torch.empty(gdn.prefix_state_rows(x.shape[0], x.shape[1], 2, False), x.shape[2],
                              device=x.device)
            h, hT = gdn.gdn_scan_prefill(y, a, b, h0, prefix_states=pre, prefix_interval=2,
                                         flags=gdn.GDN_GATE_LOGITS)
            ctx.save_for_backward(y, r, w, a, b, h0, pre)
            return h, r, hT

        @staticmethod
        def backward(ctx, dh, dr, dhT):
            y, r, w, a, b, h0, pre = ctx.saved_tensors
            dy, da, db, dh0 = gdn.gdn_scan_backward(
                dh.contiguous(), y, a, b, h0, prefix_states=pre, prefix_interval=2,
                dfinal=dhT.contiguous(), flags=gdn.GDN_GATE_LOGITS)
            dx, dw = gdn.gdn_rms_norm_backward(dy, r, w, dr.contiguous())
            return dx, dx, dw.to(w.dtype), da, db, dh0

    s = make(60)
    leaves = [s[k].requires_grad_() for k in ("x", "res", "w", "a", "b", "h0")]
    y, _, _, r = gdn.gdn_rms_norm(s["x"], s["w"], s["res"])
    assert not (y.requires_grad or r.requires_grad)
    h, r, hT = Layer.apply(*leaves)
    (h.float().sum() + (r * s["dy"]).float().sum() + 2 * hT.sum()).backward()
    with torch.no_grad():
        y, _, _, r = gdn.gdn_rms_norm(s["x"], s["w"], s["res"])
        gdn.gdn_scan_prefill(y, s["a"], s["b"], s["h0"], prefix_states=s["pre"], prefix_interval=2,
                             flags=2)
        dy, da, db, dh0 = gdn.gdn_scan_backward(
            torch.ones_like(y), y, s["a"], s["b"], s["h0"], prefix_states=s["pre"],
            prefix_interval=2, dfinal=torch.full_like(s["h0"], 2.0), flags=2)
        dx, dw = gdn.gdn_rms_norm_backward(dy, r, s["w"], s["dy"])
    for leaf, want in zip(leaves, (dx, dx, dw.bfloat16(), da, db, dh0)):
        assert torch.equal(leaf.grad, want)
