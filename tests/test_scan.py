"""The gated linear recurrence against its 64-bit form: prompt, packed batch,
backward, single tokens. Tolerances: tests/ops_oracle.py."""
import pytest

torch = pytest.importorskip("torch")
from tests.ops_oracle import (U32, K, assert_scan_close, half_step, scan64,  # noqa: E402
                              scan_backward64)

DEV = "cuda:0"
gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_token_amd as g
    g.load_library()
    return g


def inputs(seed, tokens, D, n, dtype, tied, logits, h0=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, D, generator=g).to(dtype)
    if logits:
        a = (torch.randn(tokens, D, generator=g) * 2 - torch.linspace(0, 7, D)).to(dtype)
        b = torch.randn(tokens, D, generator=g).to(dtype)
    else:
        a = (1 - torch.rand(tokens, D, generator=g) ** 3).to(dtype)
        b = torch.rand(tokens, D, generator=g).to(dtype)
    s = torch.randn(n, D, generator=g) if h0 else None
    return x, a, (None if tied else b), s


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


CASES = [  # B, T, D, dtype, tied, logits, initial state
    (1, 1, 1, "f32", False, True, True),
    (2, 1, 64, "bf16", False, True, False),
    (3, 2, 7, "bf16", True, True, True),
    (1, 127, 130, "f32", False, False, True),
    (2, 128, 128, "bf16", False, True, True),
    (1, 129, 136, "bf16", True, True, True),
    (2, 300, 72, "f32", True, False, False),
    (1, 515, 333, "bf16", False, False, True),
    (2, 640, 200, "f32", False, True, True),
    (1, 1000, 1111, "f32", True, True, True),
    (1, 1409, 264, "bf16", False, True, True),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_prompt(gdn, case):
    B, T, D, dt, tied, logits, h0 = case
    dtype, flags = DT[dt], gdn.GDN_GATE_LOGITS if logits else 0
    x, a, b, s = inputs(T * 7 + D, B * T, D, B, dtype, tied, logits, h0)
    xd, ad, bd, sd = dev(x, a, b, s)
    v = lambda t: None if t is None else t.view(B, T, D)  # noqa: E731
    out, fin = gdn.gdn_scan_prefill(v(xd), v(ad), v(bd), sd, flags=flags)
    again, fin2 = gdn.gdn_scan_prefill(v(xd), v(ad), v(bd), sd, flags=flags)
    one, fin3 = gdn.gdn_scan_prefill(v(xd), v(ad), v(bd), sd, flags=flags, workspace=None)
    assert torch.equal(out, again) and torch.equal(fin, fin2)
    assert torch.equal(out, one) and torch.equal(fin, fin3)
    for n in range(B):
        r = slice(n * T, (n + 1) * T)
        h, e = scan64(x[r], a[r], None if b is None else b[r], None if s is None else s[n], logits)
        assert_scan_close(out[n], h, e, dtype, "out")
        assert_scan_close(fin[n], h[-1], e[-1], torch.float32, "final")


@gpu
def test_no_tokens_hand_the_state_on(gdn):
    s = torch.randn(3, 20, device=DEV)
    e = torch.empty(3, 0, 20, device=DEV)
    out, fin = gdn.gdn_scan_prefill(e, e, e, s)
    assert out.shape == e.shape and torch.equal(fin, s)
    _, fin = gdn.gdn_scan_prefill(e, e, e)
    assert torch.equal(fin, torch.zeros_like(s))
    dx, da, db, dh0 = gdn.gdn_scan_backward(e, e, e, e, dfinal=s)
    assert dx.numel() == 0 and torch.equal(dh0, s)


@gpu
def test_state_in_place_and_resume(gdn):
    """A prompt cut at any token and resumed; final_state over initial_state."""
    B, T, D = 2, 400, 96
    x, a, b, s = inputs(5, B * T, D, B, torch.float32, False, True)
    xd, ad, bd, sd = dev(x, a, b, s)
    f = lambda t: t.view(B, T, D)  # noqa: E731
    out, fin = gdn.gdn_scan_prefill(f(xd), f(ad), f(bd), sd, flags=2)
    state = sd.clone()
    parts = []
    for lo, hi in ((0, 1), (1, 130), (130, 400)):
        cut = lambda t: f(t)[:, lo:hi].contiguous()  # noqa: E731
        o, r = gdn.gdn_scan_prefill(cut(xd), cut(ad), cut(bd), state, final_state=state, flags=2)
        assert r is state
        parts.append(o)
    for n in range(B):
        r = slice(n * T, (n + 1) * T)
        h, e = scan64(x[r], a[r], b[r], s[n], True)
        assert_scan_close(torch.cat(parts, 1)[n], h, e, torch.float32, "resumed")
        assert_scan_close(state[n], h[-1], e[-1], torch.float32, "state")


PACKED = [
    ([1], 8, "bf16"), ([0, 0, 5], 9, "f32"), ([128, 1, 0, 129, 64, 300], 64, "bf16"),
    ([700, 0, 1, 1, 1, 255, 256], 132, "f32"), ([3] * 70, 40, "bf16"), ([0, 0], 16, "f32"),
]


@gpu
@pytest.mark.parametrize("lengths,D,dt", PACKED, ids=str)
@pytest.mark.parametrize("tied", [False, True])
def test_packed_is_each_sequence_alone(gdn, lengths, D, dt, tied):
    dtype = DT[dt]
    total, N = sum(lengths), len(lengths)
    x, a, b, s = inputs(total + D, total, D, N, dtype, tied, True)
    cu = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32)
    xd, ad, bd, sd, cud = dev(x, a, b, s, cu)
    rows = gdn.prefix_state_rows(N, total, 2, True)
    pre = torch.full((rows, D), 77.0, device=DEV)
    # rows behind the batch stay as they were
    hold = torch.full((total + 3, D), 5.0, dtype=dtype, device=DEV)
    out, fin = gdn.gdn_scan_varlen_prefill(xd, ad, bd, cud, sd, out=hold[:total], flags=2,
                                           prefix_states=pre, prefix_interval=2)
    assert torch.equal(hold[total:], torch.full((3, D), 5.0, dtype=dtype, device=DEV))
    out2, fin2 = gdn.gdn_scan_varlen_prefill(xd, ad, bd, cud, sd, flags=2, workspace=None)
    assert torch.equal(out, out2) and torch.equal(fin, fin2)
    dy = torch.randn(total, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    dhT = torch.randn(N, D, generator=torch.Generator().manual_seed(2))
    grads = gdn.gdn_scan_varlen_backward(dy.to(DEV), xd, ad, bd, cud, sd, prefix_states=pre,
                                         prefix_interval=2, dfinal=dhT.to(DEV), flags=2)
    used = torch.zeros(rows, dtype=torch.bool)
    for n in range(N):
        lo, hi = int(cu[n]), int(cu[n + 1])
        bn = None if b is None else b[lo:hi]
        h, e = scan64(x[lo:hi], a[lo:hi], bn, s[n], True)
        assert_scan_close(out[lo:hi], h, e, dtype, "out")
        assert_scan_close(fin[n], h[-1] if hi > lo else s[n].double(),
                          e[-1] if hi > lo else s[n].double() * 0, torch.float32, "final")
        for i in range((hi - lo) // 128):
            row = lo // 128 + n + i
            used[row] = True
            assert_scan_close(pre[row], h[128 * i + 127], e[128 * i + 127], torch.float32, "prefix")
        cut = lambda t: None if t is None else t[lo:hi][None].contiguous()  # noqa: E731
        if hi > lo:
            o1, f1 = gdn.gdn_scan_prefill(cut(xd), cut(ad), cut(bd), sd[n:n + 1].clone(), flags=2)
            assert torch.equal(o1[0], out[lo:hi]) and torch.equal(f1[0], fin[n])
        want, err = scan_backward64(dy[lo:hi], x[lo:hi], a[lo:hi], bn, s[n], dhT[n], True)
        for name, got in zip(("dx", "da", "db"), grads):
            if got is not None:
                assert_scan_close(got[lo:hi], want[name], err[name], dtype, name)
        assert_scan_close(grads[3][n], want["dh0"], err["dh0"], torch.float32, "dh0")
    assert (pre[~used.to(DEV)] == 77.0).all()  # rows that no block maps to


@gpu
@pytest.mark.parametrize("interval", [1, 2, 3, 5])
@pytest.mark.parametrize("T", [63, 64, 200, 640])
def test_prefix_states(gdn, interval, T):
    B, D = 2, 48
    x, a, b, s = inputs(T, B * T, D, B, torch.bfloat16, False, True)
    xd, ad, bd, sd = dev(x, a, b, s)
    L = 64 * interval
    pre = torch.full((B * (T // L), D), -9.0, device=DEV)
    f = lambda t: t.view(B, T, D)  # noqa: E731
    gdn.gdn_scan_prefill(f(xd), f(ad), f(bd), sd, flags=2, prefix_states=pre,
                         prefix_interval=interval)
    for n in range(B):
        r = slice(n * T, (n + 1) * T)
        h, e = scan64(x[r], a[r], b[r], s[n], True)
        for i in range(T // L):
            assert_scan_close(pre[n * (T // L) + i], h[L * (i + 1) - 1], e[L * (i + 1) - 1],
                              torch.float32, i)


@gpu
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("interval", [1, 2])
def test_backward(gdn, case, interval):
    B, T, D, dt, tied, logits, h0 = case
    dtype, flags = DT[dt], gdn.GDN_GATE_LOGITS if logits else 0
    x, a, b, s = inputs(T * 3 + D, B * T, D, B, dtype, tied, logits, h0)
    g = torch.Generator().manual_seed(9)
    dy = torch.randn(B * T, D, generator=g).to(dtype)
    dhT = torch.randn(B, D, generator=g) if h0 else None
    xd, ad, bd, sd, dyd, dhd = dev(x, a, b, s, dy, dhT)
    v = lambda t: None if t is None else t.view(B, T, D)  # noqa: E731
    pre = torch.empty(gdn.prefix_state_rows(B, T, interval, False), D, device=DEV)
    gdn.gdn_scan_prefill(v(xd), v(ad), v(bd), sd, flags=flags, prefix_states=pre,
                         prefix_interval=interval)
    run = lambda **k: gdn.gdn_scan_backward(  # noqa: E731
        v(dyd), v(xd), v(ad), v(bd), sd, prefix_states=pre, prefix_interval=interval, dfinal=dhd,
        flags=flags, **k)
    grads, again, one = run(), run(), run(workspace=None)
    for p, q, r in zip(grads, again, one):
        assert p is None or (torch.equal(p, q) and torch.equal(p, r))
    assert (grads[2] is None) == tied
    for n in range(B):
        r = slice(n * T, (n + 1) * T)
        want, err = scan_backward64(dy[r], x[r], a[r], None if b is None else b[r],
                                    None if s is None else s[n], None if dhT is None else dhT[n],
                                    logits)
        for name, got in zip(("dx", "da", "db"), grads):
            if got is not None:
                assert_scan_close(got[n], want[name], err[name], dtype, name)
        assert_scan_close(grads[3][n], want["dh0"], err["dh0"], torch.float32, "dh0")


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("logits", [False, True])
def test_the_formula_is_the_derivative(tied, logits):
    """The backward oracle against central differences of the forward one."""
    T, D = 9, 3
    x, a, b, s = inputs(4, T, D, 1, torch.float64, tied, logits)
    s = s.double()
    g = torch.Generator().manual_seed(3)
    dy, dhT = torch.randn(T, D, generator=g).double(), torch.randn(D, generator=g).double()

    def loss(x, a, b, s):
        h, _ = scan64(x, a, b, s[0], logits)
        return float((h * dy).sum() + (h[-1] * dhT).sum())

    got, _ = scan_backward64(dy, x, a, b, s[0], dhT, logits)
    step = 1e-5
    for name, t, grad in (("x", x, got["dx"]), ("a", a, got["da"]), ("b", b, got.get("db")),
                          ("s", s, got["dh0"][None])):
        if t is None:
            continue
        for i in range(t.numel()):
            keep = t.view(-1)[i].item()
            t.view(-1)[i] = keep + step
            up = loss(x, a, b, s)
            t.view(-1)[i] = keep - step
            down = loss(x, a, b, s)
            t.view(-1)[i] = keep
            # third derivatives of a few units times step^2, and rounding / step
            assert abs((up - down) / (2 * step) - float(grad.reshape(-1)[i])) < 1e-7, (name, i)


@gpu
def test_backward_against_differences(gdn):
    """The kernels' own loss along a direction, fp32, against their gradients."""
    B, T, D, step = 1, 150, 64, 2.0 ** -8
    x, a, b, s = inputs(8, T, D, 1, torch.float32, False, True)
    g = torch.Generator().manual_seed(6)
    dy = torch.randn(T, D, generator=g)
    along = [torch.randn(t.shape, generator=g) for t in (x, a, b, s)]

    def out(sign):
        xs, as_, bs, ss = [t + sign * step * d for t, d in zip((x, a, b, s), along)]
        o, _ = gdn.gdn_scan_prefill(*[t.view(B, T, D).to(DEV) for t in (xs, as_, bs)],
                                    ss.to(DEV), flags=2)
        return o.cpu().double()[0]

    xd, ad, bd = [t.view(B, T, D).to(DEV) for t in (x, a, b)]
    pre = torch.empty(1, D, device=DEV)
    gdn.gdn_scan_prefill(xd, ad, bd, s.to(DEV), flags=2, prefix_states=pre, prefix_interval=2)
    grads = gdn.gdn_scan_backward(dy.view(B, T, D).to(DEV), xd, ad, bd, s.to(DEV),
                                  prefix_states=pre, prefix_interval=2, flags=2)
    diff = ((out(1) - out(-1)) * dy.double()).sum() / (2 * step)
    lin = sum((p.cpu().double().reshape(d.shape) * d.double()).sum()
              for p, d in zip(grads, along))
    # the central difference's own error in 64 bits (third derivatives), and the
    # outputs' rounding over the step: K units of E each, summed against |dy|
    def exact(sign):
        xs, as_, bs, ss = [t.double() + sign * step * d.double()
                           for t, d in zip((x, a, b, s), along)]
        return scan64(xs, as_, bs, ss[0], True)
    (up, e), (down, _) = exact(1), exact(-1)
    curve = abs(((up - down) * dy.double()).sum() / (2 * step) - lin)
    noise = 2 * K * U32 * (e * dy.double().abs()).sum() / (2 * step)
    assert abs(diff - lin) <= curve + noise
    assert curve <= 0.05 * abs(lin) + 1.0  # the check says something


@gpu
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f32", 33), ("bf16", 1000), ("f32", 260)])
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("Kt", [0, 1, 5])
def test_decode_slots(gdn, dt, D, tied, Kt):
    dtype, B, slots = DT[dt], 6, 9
    x, a, b, _ = inputs(D + Kt, B * Kt, D, 1, dtype, tied, True)
    g = torch.Generator().manual_seed(5)
    pool = torch.randn(slots, D, generator=g)
    src = torch.tensor([3, -1, 0, 5, 9, 2], dtype=torch.int32)     # zero state; past the pool
    dst = torch.tensor([3, 1, -4, 8, 4, 12], dtype=torch.int32)    # in place; not written; past
    xd, ad, bd, pd, sd, dd = dev(x, a, b, pool, src, dst)
    v = lambda t: None if t is None else t.view(B, Kt, D)  # noqa: E731
    out = gdn.gdn_scan_decode(v(xd), v(ad), v(bd), pd, sd, dd, flags=2)
    want_pool = pool.double().clone()
    err_pool = torch.zeros_like(want_pool)
    for n in range(B):
        if src[n] >= slots or dst[n] >= slots:
            assert out[n].isnan().all()
            continue
        r = slice(n * Kt, (n + 1) * Kt)
        s = pool[src[n]] if src[n] >= 0 else None
        h, e = scan64(x[r], a[r], None if b is None else b[r], s, True)
        assert_scan_close(out[n], h, e, dtype, "out")
        if dst[n] >= 0:
            want_pool[dst[n]] = h[-1] if Kt else (0 if s is None else s.double())
            err_pool[dst[n]] = e[-1] if Kt else 0
    assert_scan_close(pd, want_pool, err_pool, torch.float32, "pool")


@gpu
def test_masked_places_and_infinities(gdn):
    """NaN in one sequence or channel reaches no other; alpha 0 forgets, alpha 1 and beta 0 keep."""
    B, T, D = 2, 260, 72
    x, a, b, s = inputs(3, B * T, D, B, torch.float32, False, False)
    a[100] = 0.0
    a[130:140], b[130:140] = 1.0, 0.0
    xd, ad, bd, sd = dev(x, a, b, s)
    f = lambda t: t.view(B, T, D)  # noqa: E731
    clean, _ = gdn.gdn_scan_prefill(f(xd), f(ad), f(bd), sd)
    # A kept state is formed anew wherever a group of tokens begins (A h + H in place of the
    # walk through the group in front), so its values are equal up to their roundings: each is
    # within K 2^-24 E of the exact one, two of them within twice that.
    h, e = scan64(x[:T], a[:T], b[:T], s[0], False)
    moved = (clean[0, 130:140] - clean[0, 129]).cpu().double().abs()
    assert (moved <= 2 * K * U32 * e[139]).all()
    assert (h[130:140] == h[129]).all()
    xd.view(B, T, D)[1, 17, 5] = float("nan")
    out, fin = gdn.gdn_scan_prefill(f(xd), f(ad), f(bd), sd)
    assert out[1, 17:, 5].isnan().all() and fin[1, 5].isnan()
    keep = torch.ones(B, T, D, dtype=torch.bool)
    keep[1, 17:, 5] = False
    assert torch.equal(out.cpu()[keep], clean.cpu()[keep])


@gpu
def test_extreme_logits(gdn):
    """Gate logits far out on either side: alpha and beta saturate without NaN."""
    vals = torch.tensor([-3e38, -200.0, -90.0, -20.0, 0.0, 20.0, 79.0, 90.0, 200.0, 3e38])
    T, D = 4, 10
    x = torch.full((1, T, D), 2.0)
    a = vals.expand(1, T, D).contiguous()
    b = vals.flip(0).expand(1, T, D).contiguous()
    s = torch.full((1, D), 3.0)
    for bb in (b, None):
        out, fin = gdn.gdn_scan_prefill(*dev(x, a, bb, s), flags=2)
        h, e = scan64(x[0], a[0], None if bb is None else bb[0], s[0], True)
        # e^z is held at e^80: gates below e^-80 < 2e-35 move by less than that, a state by
        # 4 tokens x 2e-35 x (|h| + |x|) <= 4 x 2e-35 x 13 < 1.1e-33, a gradient by that times
        # |g| <= 5, twice: < 1.1e-32
        off = 1.1e-32 / (K * U32)
        assert_scan_close(out[0], h, e + off, torch.float32, "out")
        g = gdn.gdn_scan_backward(*dev(torch.ones_like(x), x, a, bb, s), flags=2)
        want, err = scan_backward64(torch.ones(T, D), x[0], a[0], None if bb is None else bb[0],
                                    s[0], None, True)
        for name, got in zip(("dx", "da", "db"), g):
            if got is not None:
                assert got.isfinite().all()
                assert_scan_close(got[0], want[name], err[name] + off, torch.float32, name)


@gpu
def test_offsets_past_32_bits(gdn):
    """A prompt whose tensors are over 2^32 bytes: its tail against the same tokens run from the
    last prefix state."""
    T, D = 400_000, 6144
    x = torch.empty(1, T, D, dtype=torch.bfloat16, device=DEV)
    a, b = torch.empty_like(x), torch.empty_like(x)
    for lo in range(0, T, 50_000):
        g = torch.Generator(device=DEV).manual_seed(lo)
        for t, shift in ((x, 0.0), (a, -3.0), (b, 0.0)):
            t[0, lo:lo + 50_000] = torch.randn(50_000, D, generator=g, device=DEV,
                                               dtype=torch.bfloat16) + shift
    L = 64 * 100
    pre = torch.empty(T // L, D, device=DEV)
    out, fin = gdn.gdn_scan_prefill(x, a, b, flags=2, prefix_states=pre, prefix_interval=100)
    lo = T // L * L  # 396,800: a multiple of the tile
    tail = [t[:, lo:].contiguous() for t in (x, a, b)]
    o2, f2 = gdn.gdn_scan_prefill(*tail, pre[-1:].clone(), flags=2)
    h, e = scan64(*[t[0, :, :64].cpu() for t in tail], pre[-1, :64].cpu(), True)
    assert_scan_close(out[0, lo:, :64], h, e, torch.bfloat16, "tail")
    assert_scan_close(o2[0, :, :64], h, e, torch.bfloat16, "rerun")
    # the carry of the tile in front differs by the order of its roundings only
    scale = e.max() * K * U32 * 2 + half_step(torch.bfloat16) * h.abs().max() * 2
    assert (out[0, lo:].double() - o2[0].double()).abs().max() <= scale
    assert (fin - f2).abs().max() <= scale


MANY = [  # B, T, D, dtype, tied: chains of one published word; enough sequences for none
    (4, 400, 2048, "bf16", False), (3, 385, 1600, "f32", True), (2, 300, 1999, "bf16", True),
    (2, 260, 2001, "f32", False), (2100, 130, 8, "bf16", False), (130, 257, 1024, "f32", False),
]


@gpu
@pytest.mark.parametrize("case", MANY, ids=str)
def test_many_chains(gdn, case):
    """Forward and backward where the call has many (sequence, column block) pairs: the same bits
    with and without a workspace, and the oracle on some sequences and columns."""
    B, T, D, dt, tied = case
    dtype = DT[dt]
    g = torch.Generator(device=DEV).manual_seed(T + D)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, dy = r(B, T, D).to(dtype), r(B, T, D).to(dtype)
    a, b = (r(B, T, D) * 2 - 3).to(dtype), None if tied else r(B, T, D).to(dtype)
    s, dh = r(B, D), r(B, D)
    pre = torch.empty(gdn.prefix_state_rows(B, T, 1, False), D, device=DEV)
    kw = dict(flags=2, prefix_states=pre, prefix_interval=1)
    out, fin = gdn.gdn_scan_prefill(x, a, b, s, **kw)
    kept = pre.clone()
    grads = gdn.gdn_scan_backward(dy, x, a, b, s, dfinal=dh, **kw)
    out2, fin2 = gdn.gdn_scan_prefill(x, a, b, s, workspace=None, **kw)
    assert torch.equal(out, out2) and torch.equal(fin, fin2) and torch.equal(pre, kept)
    for p, q in zip(grads, gdn.gdn_scan_backward(dy, x, a, b, s, dfinal=dh, workspace=None, **kw)):
        assert p is None or torch.equal(p, q)
    cols = torch.tensor(sorted({0, 1, D // 2, D - 2, D - 1, min(D - 1, 127), min(D - 1, 128)}))
    for n in sorted({0, B // 2, B - 1}):
        cut = lambda t: None if t is None else t[n].cpu()[..., cols]  # noqa: E731
        h, e = scan64(cut(x), cut(a), cut(b), cut(s), True)
        assert_scan_close(cut(out), h, e, dtype, "out")
        assert_scan_close(cut(fin), h[-1], e[-1], torch.float32, "final")
        want, err = scan_backward64(cut(dy), cut(x), cut(a), cut(b), cut(s), cut(dh), True)
        for name, got in zip(("dx", "da", "db"), grads):
            if got is not None:
                assert_scan_close(cut(got), want[name], err[name], dtype, name)
        assert_scan_close(cut(grads[3]), want["dh0"], err["dh0"], torch.float32, "dh0")


@gpu
def test_debug_checks_offsets(gdn, monkeypatch):
    """GDN_DEBUG=1: malformed offsets are refused before any launch."""
    x = torch.zeros(300, 8, device=DEV)
    monkeypatch.setenv("GDN_DEBUG", "1")
    for cu in ([0, 200, 100], [1, 100, 300], [0, 100, 299], [0, 301, 300]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        with pytest.raises(gdn.GDNError):
            gdn.gdn_scan_varlen_prefill(x, x, x, c)
        with pytest.raises(gdn.GDNError):
            gdn.gdn_scan_varlen_backward(x, x, x, x, c, prefix_states=torch.zeros(4, 8, device=DEV),
                                         prefix_interval=2)
    c = torch.tensor([0, 100, 300], dtype=torch.int32, device=DEV)
    gdn.gdn_scan_varlen_prefill(x, x, x, c)


@gpu
@pytest.mark.parametrize("N,most,D", [(700, 3, 8), (5000, 40, 8), (1100, 400, 16)])
def test_many_packed_sequences(gdn, N, most, D):
    """More sequences than a workgroup has threads: the same bits with and without a workspace, and
    each final state from the oracle on its own tokens."""
    g = torch.Generator().manual_seed(N)
    lengths = torch.randint(0, most, (N,), generator=g)
    lengths[N // 2] = 1000
    cu = torch.cat([torch.zeros(1), lengths.cumsum(0)]).to(torch.int32)
    total = int(cu[-1])
    x, a, b, s = inputs(N, total, D, N, torch.float32, False, True)
    xd, ad, bd, sd, cud = dev(x, a, b, s, cu)
    out, fin = gdn.gdn_scan_varlen_prefill(xd, ad, bd, cud, sd, flags=2)
    out2, fin2 = gdn.gdn_scan_varlen_prefill(xd, ad, bd, cud, sd, flags=2, workspace=None)
    assert torch.equal(out, out2) and torch.equal(fin, fin2)
    for n in [0, 1, N // 3, N // 2 - 1, N // 2, N // 2 + 1, N - 2, N - 1]:
        lo, hi = int(cu[n]), int(cu[n + 1])
        h, e = scan64(x[lo:hi], a[lo:hi], b[lo:hi], s[n], True)
        assert_scan_close(out[lo:hi], h, e, torch.float32, n)
        assert_scan_close(fin[n], h[-1] if hi > lo else s[n].double(),
                          e[-1] if hi > lo else torch.zeros(D).double(), torch.float32, n)


@gpu
def test_backward_past_32_bits(gdn):
    """Gradients of tensors over 2^32 bytes: the last tokens' are those of a call on them alone
    from the prefix state in front of them, bit by bit."""
    T, D = 360_065, 6144
    make = lambda seed, shift=0.0: torch.randn(  # noqa: E731
        1, T, D, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV,
        dtype=torch.bfloat16) + shift
    x, a, b, dy = make(1), make(2, -3.0), make(3), make(4)
    pre = torch.empty(T // 128, D, device=DEV)
    kw = dict(flags=2, prefix_interval=2)
    out, _ = gdn.gdn_scan_prefill(x, a, b, prefix_states=pre, **kw)
    del out
    grads = gdn.gdn_scan_backward(dy, x, a, b, prefix_states=pre, **kw)
    lo = (T // 128 - 3) * 128
    cut = lambda t: t[:, lo:].contiguous()  # noqa: E731
    tail = gdn.gdn_scan_backward(cut(dy), cut(x), cut(a), cut(b), pre[lo // 128 - 1][None].clone(),
                                 prefix_states=pre[lo // 128:].clone(), **kw)
    for p, q in zip(grads[:3], tail):
        assert torch.equal(p[:, lo:], q)
    # the tokens in front of them: what reaches them is the tail's gradient of its first state
    mid = lo - 256
    part = lambda t: t[:, mid:lo].contiguous()  # noqa: E731
    front = gdn.gdn_scan_backward(part(dy), part(x), part(a), part(b),
                                  pre[mid // 128 - 1][None].clone(), dfinal=tail[3],
                                  prefix_states=pre[mid // 128:lo // 128].clone(), **kw)
    for p, q in zip(grads[:3], front):
        assert torch.equal(p[:, mid:lo], q)


EVEN = [  # B, T, D, dtype, tied, logits, initial state: bf16 rows of pairs, not of 8 or 16 bytes
    (1, 1, 2, "bf16", False, True, True), (2, 129, 126, "bf16", True, True, True),
    (1, 260, 130, "bf16", False, False, False), (3, 385, 66, "bf16", True, False, True),
    (2, 1000, 258, "bf16", False, True, True), (1, 300, 1102, "bf16", False, True, False),
    (2, 257, 132, "bf16", False, True, True), (2, 300, 160, "bf16", False, True, True),
]


@gpu
@pytest.mark.parametrize("case", EVEN, ids=str)
def test_even_widths(gdn, case):
    test_prompt(gdn, case)
    test_backward(gdn, case, 1)
    test_backward(gdn, case, 2)


@gpu
@pytest.mark.parametrize("tied", [False, True])
def test_even_widths_elsewhere(gdn, tied):
    """Packed, decoded and in many chains, as the other widths."""
    # sequences that start on 16 bytes, which a call on one of them alone asks for
    test_packed_is_each_sequence_alone(gdn, (0, 136, 8, 304, 0, 129), 134, "bf16", tied)
    test_decode_slots(gdn, "bf16", 102, tied, 3)
    test_many_chains(gdn, (3, 385, 2046, "bf16", tied))
    test_many_chains(gdn, (2100, 130, 6, "bf16", tied))


@gpu
@pytest.mark.parametrize("T,D,dt", [(300, 72, "f32"), (300, 72, "bf16"), (700, 33, "f32")])
@pytest.mark.parametrize("ws", ["auto", None])
def test_infinities_stay_in_their_channel(gdn, T, D, dt, ws):
    """An infinite state or input: what lies before it and beside it keeps its bits, what lies
    behind it in its channel is not finite. Decays of 2^-10 (products of 0 over a tile)."""
    B, dtype = 3, DT[dt]
    x, a, b, s = inputs(T + D, B * T, D, B, dtype, False, False)
    a[:, ::2] = 2.0 ** -10
    a[a == 0] = 0.5  # 0 times infinity would be NaN token by token too
    b[b == 0] = 0.5
    dy = torch.randn(B * T, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    dh = torch.randn(B, D, generator=torch.Generator().manual_seed(2))
    xd, ad, bd, sd, dyd, dhd = dev(x, a, b, s, dy, dh)
    v = lambda t: t.view(B, T, D)  # noqa: E731
    pre = torch.empty(B * (T // 128), D, device=DEV)
    kw = dict(prefix_states=pre, prefix_interval=2, workspace=ws)
    fwd = lambda: gdn.gdn_scan_prefill(v(xd), v(ad), v(bd), sd, **kw)  # noqa: E731
    back = lambda: gdn.gdn_scan_backward(v(dyd), v(xd), v(ad), v(bd), sd, dfinal=dhd,  # noqa: E731
                                         **kw)
    out, fin = fwd()
    grads = back()
    inf = float("inf")
    hit = torch.zeros(B, T, D, dtype=torch.bool)
    sd[0, 4], sd[1, 5] = inf, -inf
    v(xd)[2, 140, 6], v(xd)[2, T - 1, 7] = inf, -inf
    hit[0, :, 4] = hit[1, :, 5] = True
    hit[2, 140:, 6] = hit[2, T - 1:, 7] = True
    o, f = fwd()
    assert torch.equal(o.cpu()[~hit], out.cpu()[~hit]) and not o.cpu()[hit].isfinite().any()
    last = hit[:, -1]
    assert torch.equal(f.cpu()[~last], fin.cpu()[~last]) and not f.cpu()[last].isfinite().any()
    # the gradients of clean inputs under an infinite gradient: from its token towards the first
    sd.copy_(s)
    xd.copy_(x)
    fwd()
    hit[:] = False
    dhd[0, 4] = inf
    v(dyd)[1, 140, 6] = -inf
    hit[0, :, 4] = hit[1, :141, 6] = True
    got = back()
    for p, q in zip(got[:3], grads):
        p, q = p.cpu(), q.cpu()
        assert torch.equal(p[~hit], q[~hit]) and not p[hit].isfinite().any()
    first = hit[:, 0]
    p, q = got[3].cpu(), grads[3].cpu()
    assert torch.equal(p[~first], q[~first]) and not p[first].isfinite().any()
