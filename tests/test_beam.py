"""Beam selection and the reordering of states against 64-bit sorting.

A key differs from the 64-bit one by the logsumexp's error: exponentials to a
few units of 2^-23 (their arguments are below 2^7 where they count), sums in
chains of at most 32 + 6 + 4 terms: below 2^-18 together. Where two candidates
are further apart than twice that, the order has to be the oracle's.
"""
import math

import pytest

torch = pytest.importorskip("torch")
from tests.ops_oracle import beam64, beam_order  # noqa: E402

DEV = "cuda:0"
gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = 2.0 ** -18


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_token_amd as g
    g.load_library()
    return g


def run(gdn, logits, scores, finished=None, eos=-1, slots=None):
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    out = gdn.gdn_beam_select(d(logits), d(scores), finished=d(finished), eos=eos,
                              beam_slots=d(slots))
    again = gdn.gdn_beam_select(d(logits), d(scores), finished=d(finished), eos=eos,
                                beam_slots=d(slots))
    for p, q in zip(out, again):
        assert p is None or torch.equal(p, q)
    return [None if t is None else t.cpu() for t in out]


def check(gdn, logits, scores, finished=None, eos=-1, slots=None, exact=False):
    B, W, V = logits.shape
    ns, tok, par, fin, src = run(gdn, logits, scores, finished, eos, slots)
    assert ((tok >= 0) & (tok < V) & (par >= 0) & (par < W)).all()
    key = beam64(logits, scores, finished, eos)
    order = beam_order(key, W)
    place = par.long() * V + tok.long()
    for b in range(B):
        assert len(set(place[b].tolist())) == W
        got, want = key[b, place[b]], key[b, order[b]]
        same = place[b] == order[b]
        if exact:
            assert same.all(), (place[b], order[b])
        # another candidate than the oracle's may stand only where the keys are that near, and
        # equal keys go by place
        near = (got - want).abs() <= 2 * TOL
        assert (same | (near & (got != want))).all(), (b, place[b], order[b], got, want)
        tol = TOL + got.abs().nan_to_num(posinf=0) * 2.0 ** -23
        live = got > -math.inf
        assert ((ns[b].double() - got).abs()[live] <= tol[live]).all()
        assert (ns[b][~live] == -math.inf).all()
        if fin is not None:
            f = torch.zeros(W, dtype=torch.bool) if finished is None else finished[b].bool()
            assert torch.equal(fin[b].bool(), f[par[b].long()] | (tok[b] == eos))
        if slots is not None:
            assert torch.equal(src[b], slots[b][par[b].long()])
    assert (fin is None) == (eos < 0) and (src is None) == (slots is None)
    return ns, tok, par


CASES = [(1, 1, 1, "f32"), (2, 4, 1, "bf16"), (1, 5, 3, "f32"), (3, 2, 7, "bf16"),
         (1, 4, 1000, "f32"), (2, 3, 8191, "bf16"), (2, 3, 8192, "f32"), (1, 2, 8193, "bf16"),
         (5, 8, 20011, "bf16"), (1, 32, 5000, "f32"), (1, 32, 40000, "bf16"),
         (2, 16, 65537, "f32"), (7, 1, 30000, "bf16"), (1, 6, 262147, "bf16")]


@gpu
@pytest.mark.parametrize("B,W,V,dt", CASES, ids=str)
@pytest.mark.parametrize("ended", [False, True])
def test_selection(gdn, B, W, V, dt, ended):
    g = torch.Generator().manual_seed(B * 100 + W * 10 + V)
    logits = (torch.randn(B, W, V, generator=g) * 3).to(DT[dt])
    scores = torch.randn(B, W, generator=g) * 2 - 20
    slots = torch.randperm(B * W, generator=g).to(torch.int32).view(B, W)
    if ended:
        fin = (torch.rand(B, W, generator=g) < 0.4).to(torch.uint8)
        check(gdn, logits, scores, fin, V // 2, slots)
    else:
        check(gdn, logits, scores, slots=slots)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 40, 9000, 30011])
def test_ties_go_to_the_lowest_place(gdn, dt, V):
    W = 4
    logits = torch.zeros(2, W, V).to(DT[dt])
    scores = torch.zeros(2, W)
    ns, tok, par = check(gdn, logits, scores, exact=True)
    assert tok[0].tolist() == [0, 1, 2, 3][:W] and par[0].tolist() == [0] * W
    # the same rows and scores on every beam; -0 and +0 are one value
    logits[:, :, 3] = 2.0
    logits[:, :, 1] = -0.0
    ns, tok, par = check(gdn, logits, scores, exact=True)
    assert tok[0].tolist() == [3] * W and par[0].tolist() == [0, 1, 2, 3]
    # many equal values in one thread's places and at the end of the row
    logits[:, 1, V - 2:] = 2.0
    check(gdn, logits, scores, exact=True)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_that_a_mask_leaves_nothing_of(gdn, dt):
    dtype, V, W = DT[dt], 700, 4
    low = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(1)
    base = torch.randn(1, W, V, generator=g).to(dtype)
    scores = torch.tensor([[-1.0, -2.0, -3.0, -4.0]])
    cases = []
    x = base.clone(); x[0, 1] = -math.inf; cases.append(x)              # noqa: E702 one dead beam
    x = base.clone(); x[0, :] = -math.inf; cases.append(x)              # noqa: E702 all dead
    x = base.clone(); x[0, 0] = low; cases.append(x)                    # noqa: E702 lowest finite
    x = base.clone(); x[0, 0, 1:] = low; cases.append(x)                # noqa: E702 one token left
    x = base.clone(); x[0, 0, 3:] = -math.inf; cases.append(x)          # noqa: E702 fewer than W
    x = base.clone(); x[0, 1:] = -math.inf; x[0, 0, 2:] = -math.inf; cases.append(x)  # noqa: E702
    x = base.clone(); x[0, 2, 5] = math.nan; cases.append(x)            # noqa: E702
    x = base.clone(); x[0, 0, 9] = math.inf; cases.append(x)            # noqa: E702
    x = base.clone(); x[0, 0, 9] = torch.finfo(dtype).max; cases.append(x)  # noqa: E702
    for x in cases:
        check(gdn, x, scores)
        check(gdn, x, scores, torch.tensor([[0, 1, 0, 0]], dtype=torch.uint8), 600)


@gpu
def test_dead_scores(gdn):
    """A first step: one live beam, the others at -inf; NaN and +inf scores are dead."""
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(1, 4, 5000, generator=g)
    inf = math.inf
    for s in ([0.0, -inf, -inf, -inf], [-inf, -inf, -inf, -3.0], [math.nan, -1.0, inf, -2.0],
              [-inf] * 4):
        ns, tok, par = check(gdn, logits, torch.tensor([s]))
    assert par[0].tolist() == [0] * 4 and tok[0].tolist() == [0, 1, 2, 3]
    fin = torch.tensor([[1, 1, 0, 0]], dtype=torch.uint8)
    check(gdn, logits, torch.tensor([[-inf, -0.5, -inf, math.nan]]), fin, 4999)
    check(gdn, logits, torch.tensor([[-inf] * 4]), fin, 4999)


@gpu
def test_an_ended_beam_keeps_its_score(gdn):
    logits = torch.zeros(1, 2, 100)
    logits[0, 1, 7] = 50.0
    fin = torch.tensor([[1, 0]], dtype=torch.uint8)
    ns, tok, par = check(gdn, logits, torch.tensor([[-3.25, -1.0]]), fin, 9, exact=True)
    assert tok[0].tolist() == [7, 9] and par[0].tolist() == [1, 0]
    assert ns[0, 1] == -3.25


@gpu
@pytest.mark.parametrize("rows,shape", [(1, (4,)), (7, (3, 8)), (5, (48, 16, 16)), (3, (4097, 4)),
                                        (0, (4,)), (4, (0, 4))], ids=str)
def test_gather(gdn, rows, shape):
    src = torch.randn(6, *shape, device=DEV)
    idx = torch.tensor([5, 0, 0, 3, 5, 2, 1][:rows], dtype=torch.int32, device=DEV)
    out = gdn.gdn_gather_states(src, idx)
    assert torch.equal(out, src[idx.long()])
    if rows >= 3 and src[0].numel():
        idx[0], idx[1], idx[2] = -1, 6, 2 ** 31 - 1
        out = gdn.gdn_gather_states(src, idx)
        assert (out[0] == 0).all() and out[1].isnan().all() and out[2].isnan().all()
        assert torch.equal(out[3:], src[idx[3:].long()])
    half = src.bfloat16().view(6, -1)
    if half.shape[1] and half.shape[1] % 8 == 0:
        assert torch.equal(gdn.gdn_gather_states(half, idx.clamp(0, 5)),
                           half[idx.clamp(0, 5).long()])


@gpu
def test_gather_refuses(gdn):
    src = torch.zeros(4, 3, device=DEV)
    idx = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_gather_states(src, idx)              # 12-byte rows
    src = torch.zeros(4, 4, device=DEV)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_gather_states(src, idx, out=src[:2])


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [20000, 8200])
def test_masks_over_several_pieces(gdn, dt, V):
    """Rows with fewer tokens left than beams, in one piece or spread; pieces of nothing but -inf;
    more equal values than the ranked list holds."""
    W = 6
    g = torch.Generator().manual_seed(V)
    scores = torch.randn(2, W, generator=g)
    x = torch.full((2, W, V), -math.inf)
    for b in range(2):
        for w in range(W):
            at = torch.randperm(V, generator=g)[:w + 1]
            x[b, w, at] = torch.randn(w + 1, generator=g)
    check(gdn, x.to(DT[dt]), scores)
    x[1, 2, V // 2:] = 1.0  # equal values, far more than fit
    x[0, :, 3000:] = -2.0
    check(gdn, x.to(DT[dt]), scores)
    check(gdn, x.to(DT[dt]), scores, torch.ones(2, W, dtype=torch.uint8), V - 1)


@gpu
@pytest.mark.parametrize("W,V", [(32, 70000), (16, 131072), (8, 300001), (3, 2100000)])
def test_many_candidates(gdn, W, V):
    """More pieces and beams than the joining threads hold."""
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (torch.randn(1, W, V, generator=g, device=DEV) * 3).bfloat16().cpu()
    check(gdn, x, torch.randn(1, W, generator=torch.Generator().manual_seed(W)))


@gpu
def test_offsets_past_32_bits(gdn):
    """Logits of over 2^31 elements and states of over 2^32 bytes: the last item is that of a call
    on it alone."""
    B, W, V = 66, 32, 1_050_000
    x = torch.randn(B, W, V, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV,
                    dtype=torch.bfloat16)
    s = torch.randn(B, W, generator=torch.Generator().manual_seed(9)).to(DEV)
    out = gdn.gdn_beam_select(x, s)
    one = gdn.gdn_beam_select(x[-1:].clone(), s[-1:].clone())
    for p, q in zip(out[:3], one):
        assert torch.equal(p[-1:], q)
    del x
    states = torch.arange(1500, dtype=torch.float32, device=DEV)[:, None].expand(
        1500, 786432).contiguous()
    idx = torch.randperm(1500, generator=torch.Generator().manual_seed(2)).to(torch.int32).to(DEV)
    moved = gdn.gdn_gather_states(states, idx)
    assert torch.equal(moved[:, 0], idx.float()) and torch.equal(moved[:, -1], idx.float())


FILLS = [1e5, 2.0 ** 20, 1.5e6, 1e9, 3e9, 1e10, 1e20, 1e30, 9e37, 2e38]


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,W,V", [(2, 4, 700), (1, 4, 2049), (1, 4, 6145), (8, 8, 32769)], ids=str)
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_large_finite_logits(gdn, dt, B, W, V, sign):
    """Masks and maxima of any finite size: over a whole row, a whole piece (of 2,048 logits, or of
    8,192 with many rows) or a last piece of one logit. A beam stays alive: only NaN, +inf or nothing
    but -inf end it."""
    piece = 2048 if B * W * -(-V // 8192) < 256 else 8192
    g = torch.Generator().manual_seed(V)
    base = torch.randn(B, W, V, generator=g) * 3
    scores = torch.randn(B, W, generator=g)
    for size in FILLS:
        fill = sign * size
        cases = []
        x = base.clone(); x[:, 1] = fill; cases.append(x)                  # noqa: E702 a whole row
        x = base.clone(); x[:] = fill; cases.append(x)                     # noqa: E702 all of them
        x = base.clone(); x[:, :, :min(piece, V - 1)] = fill; cases.append(x)  # noqa: E702 a piece
        x = base.clone(); x[..., -1] = fill; cases.append(x)               # noqa: E702 the last one
        if sign > 0:  # one best token of each beam: the W selected
            cases = [cases[0], cases[1], cases[3]]
        for x in cases:
            x = x.to(DT[dt])
            ns, tok, par = check(gdn, x, scores)
            assert ns.isfinite().all()


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_logits_beside_nan_and_inf(gdn, dt):
    """A NaN or +inf ends its beam also where the largest logit is extreme; -inf does not."""
    V = 3000
    g = torch.Generator().manual_seed(8)
    base = torch.randn(1, 4, V, generator=g)
    scores = torch.tensor([[-1.0, -2.0, -3.0, -4.0]])
    for fill in (-1e10, -1e30, 1e10, 1e30):
        for odd in (math.nan, math.inf, -math.inf):
            x = base.clone()
            x[0, 0] = fill
            x[0, 0, 7] = odd
            x = x.to(DT[dt])
            check(gdn, x, scores)
            # beside the others the live beam's best, -1 - log 2,999, may not be selected
            ns, _, _ = check(gdn, x[:, :1], scores[:, :1])
            assert ns.isfinite().all() == (odd == -math.inf)
