"""The RMS norm with residual and 8-bit output, and its gradients, against
64-bit forms.

Roundings counted for the tolerances: the sum of squares is a tree over
per-thread chains of at most 16 terms plus 10 levels, each addition half a unit
of 2^-24 relative to a sum of positive terms, halved by the square root, then
the division, the square root's own and two products: y stays within
32 * 2^-24 = 2^-19 relative, and so do the scales (one more division).
"""
import pytest

torch = pytest.importorskip("torch")
from tests.ops_oracle import U32, half_step, norm64, norm_backward64  # noqa: E402

DEV = "cuda:0"
gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
REL = 32 * U32


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_token_amd as g
    g.load_library()
    return g


def inputs(seed, rows, D, dtype, res=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, D, generator=g).to(dtype)
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(dtype)
    r = (torch.randn(rows, D, generator=g) * 3).to(dtype) if res else None
    return x, w, r


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def check_y(got, y, dtype):
    tol = REL * y.abs() + (half_step(dtype) * y.abs() * (1 + REL) if dtype != torch.float32 else 0)
    assert ((got.cpu().double() - y).abs() <= tol + 1e-37).all()


def check_8bit(q, scale, y, group):
    """q * scale stands for y: scales to REL, values to half a step of e4m3 (2^-4 relative,
    2^-10 below the smallest normal)."""
    D = y.shape[-1]
    cols = group or D
    scale = scale.cpu().double()
    for i, part in enumerate(y.split(cols, -1)):
        want = (part.abs().amax(-1) / 448).clamp(min=2.0 ** -100)
        assert ((scale[..., i] - want).abs() <= REL * want).all()
        got = q[..., i * cols:i * cols + part.shape[-1]].cpu().float().double()
        s = scale[..., i:i + 1]
        tol = part.abs() * (2.0 ** -4 * (1 + 2.0 ** -10) + 4 * REL) + s * 2.0 ** -10
        assert ((got * s - part).abs() <= tol).all()
        # the largest value of a group is the largest e4m3 value (or the group is zero)
        top = got.abs().amax(-1)
        assert ((top == 448) | (part.abs().amax(-1) < 448 * 2.0 ** -100)).all()


SHAPES = [(1, 1), (3, 7), (5, 8), (17, 64), (33, 100), (16, 128), (70, 129), (9, 200), (4, 512),
          (3, 520), (2, 1027), (7, 2048), (3, 5120), (2, 8192), (2, 8200), (1, 9001), (2, 16384),
          (1000, 128), (1, 16383)]


@gpu
@pytest.mark.parametrize("rows,D", SHAPES, ids=str)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
def test_norm(gdn, rows, D, dt, res):
    dtype = DT[dt]
    x, w, r = inputs(rows * 31 + D, rows, D, dtype, res)
    xd, wd, rd = dev(x, w, r)
    total, s, y = norm64(x, w, r, 1e-6)
    for group in (0, 128):
        out, q, scale, ro = gdn.gdn_rms_norm(xd, wd, rd, group=group, want_out8=True)
        check_y(out, y, dtype)
        check_8bit(q, scale, y, group)
        assert (ro is None) == (not res)
        if res:  # the sum is rounded to fp32, then to the type
            tol = total.abs() * (half_step(dtype) * (1 + U32) + U32)
            assert ((ro.cpu().double() - total).abs() <= tol).all()
    # each output alone gives the same bits
    o1, none, none2, _ = gdn.gdn_rms_norm(xd, wd, rd)
    assert none is None and none2 is None and torch.equal(o1, out)
    none, q1, s1, ro1 = gdn.gdn_rms_norm(xd, wd, rd, group=128, want_out=False, want_out8=True,
                                         want_residual=False)
    assert none is None and ro1 is None
    assert torch.equal(q1.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s1, scale)


@gpu
def test_residual_in_place_and_leading_dims(gdn):
    x, w, r = inputs(1, 30, 256, torch.bfloat16)
    xd, wd, rd = dev(x, w, r)
    want = gdn.gdn_rms_norm(xd, wd, rd)
    mine = rd.clone()
    out, _, _, ro = gdn.gdn_rms_norm(xd.view(2, 3, 5, 256), wd, mine.view(2, 3, 5, 256),
                                     residual_out=mine.view(2, 3, 5, 256))
    assert torch.equal(out.view(30, 256), want[0]) and torch.equal(mine, want[3])
    mine = xd.clone()
    gdn.gdn_rms_norm(mine, wd, rd, residual_out=mine)
    assert torch.equal(mine, want[3])


@gpu
def test_zero_rows_and_zero_values(gdn):
    w = torch.ones(128, device=DEV)
    out, q, s, _ = gdn.gdn_rms_norm(torch.empty(0, 128, device=DEV), w, want_out8=True)
    assert out.shape == (0, 128) and q.shape == (0, 128) and s.shape == (0, 1)
    x = torch.zeros(2, 128, device=DEV)
    x[1, 3] = 5.0
    for group in (0, 128):
        out, q, s, _ = gdn.gdn_rms_norm(x, w, want_out8=True, group=group)
        assert (out[0] == 0).all() and (q.float()[0] == 0).all() and s[0, 0] == 2.0 ** -100
        assert q.float()[1, 3] == 448 and (q.float()[1] != 0).sum() == 1
    dx, dw = gdn.gdn_rms_norm_backward(torch.empty(0, 128, device=DEV),
                                       torch.empty(0, 128, device=DEV), w)
    assert dx.shape == (0, 128) and (dw == 0).all()


@gpu
@pytest.mark.parametrize("D", [128, 300, 2048, 1001])
def test_nan_and_inf_stay_in_their_row(gdn, D):
    x, w, r = inputs(4, 9, D, torch.float32)
    xd, wd, rd = dev(x, w, r)
    clean = gdn.gdn_rms_norm(xd, wd, rd, want_out8=True)
    xd[2, D // 2] = float("nan")
    xd[5, 1] = float("inf")
    out, q, s, _ = gdn.gdn_rms_norm(xd, wd, rd, want_out8=True)
    assert out[2].isnan().all() and q.float()[2].isnan().all()
    assert out[5].isnan().any() and q.float()[5].isnan().any()
    keep = [i for i in range(9) if i not in (2, 5)]
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(s[keep], clean[2][keep])
    assert torch.equal(q[keep].view(torch.uint8), clean[1][keep].view(torch.uint8))


@gpu
@pytest.mark.parametrize("rows,D", SHAPES + [(600, 264), (1300, 4096), (5000, 40)], ids=str)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
def test_backward(gdn, rows, D, dt, res):
    dtype = DT[dt]
    r, w, dres = inputs(rows * 13 + D, rows, D, dtype, res)
    dy = torch.randn(rows, D, generator=torch.Generator().manual_seed(7)).to(dtype)
    rd, wd, dyd, drd = dev(r, w, dy, dres)
    dx, dw = gdn.gdn_rms_norm_backward(dyd, rd, wd, drd, eps=1e-5)
    dx2, dw2 = gdn.gdn_rms_norm_backward(dyd, rd, wd, drd, eps=1e-5)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    want, want_w, mag, mag_w = norm_backward64(dy, r, w, dres, 1e-5)
    tol = 2 * REL * mag + (half_step(dtype) * want.abs() * (1 + REL) if dt == "bf16" else 0)
    assert ((dx.cpu().double() - want).abs() <= tol + 1e-37).all()
    # rows are summed in chains of at most rows / 16 per thread and 40 joins behind them
    tol = (REL + U32 * (min(rows, rows / 16 + 80) + 40)) * mag_w
    assert ((dw.cpu().double() - want_w).abs() <= tol + 1e-37).all()
    # without the weight's gradient, and into dresidual itself
    dx3, none = gdn.gdn_rms_norm_backward(dyd, rd, wd, drd, eps=1e-5, want_dweight=False)
    assert none is None and torch.equal(dx3, dx)
    if res:
        mine = drd.clone()
        gdn.gdn_rms_norm_backward(dyd, rd, wd, mine, eps=1e-5, dx=mine)
        assert torch.equal(mine, dx)


def test_the_formula_is_the_derivative():
    g = torch.Generator().manual_seed(2)
    r, w, dy, dres = [torch.randn(*s, generator=g).double() for s in ((3, 6), (6,), (3, 6), (3, 6))]
    dx, dw, _, _ = norm_backward64(dy, r, w, dres, 1e-3)
    loss = lambda: float((norm64(r, w, None, 1e-3)[2] * dy).sum() + (r * dres).sum())  # noqa: E731
    for t, grad in ((r, dx), (w, dw)):
        for i in range(t.numel()):
            keep = t.view(-1)[i].item()
            t.view(-1)[i] = keep + 1e-5
            up = loss()
            t.view(-1)[i] = keep - 1e-5
            down = loss()
            t.view(-1)[i] = keep
            assert abs((up - down) / 2e-5 - float(grad.view(-1)[i])) < 1e-6


@gpu
def test_backward_against_differences(gdn):
    """The kernels' own loss along a direction, fp32, against their gradients."""
    step = 2.0 ** -7
    r, w, _ = inputs(11, 20, 200, torch.float32, False)
    g = torch.Generator().manual_seed(12)
    dy = torch.randn(20, 200, generator=g)
    dr, dw = torch.randn(20, 200, generator=g), torch.randn(200, generator=g)
    gx, gw = gdn.gdn_rms_norm_backward(*dev(dy, r, w))
    lin = (gx.cpu().double() * dr.double()).sum() + (gw.cpu().double() * dw.double()).sum()
    y = lambda s: gdn.gdn_rms_norm(*dev(r + s * step * dr, w + s * step * dw))[0]  # noqa: E731
    diff = ((y(1) - y(-1)).cpu().double() * dy.double()).sum() / (2 * step)
    exact = lambda s: norm64(r.double() + s * step * dr.double(),  # noqa: E731
                             w.double() + s * step * dw.double(), None, 1e-6)[2]
    curve = abs(((exact(1) - exact(-1)) * dy.double()).sum() / (2 * step) - lin)
    noise = 4 * REL * (exact(1).abs() * dy.double().abs()).sum() / (2 * step)
    assert abs(diff - lin) <= curve + noise
    assert curve <= 0.05 * abs(lin) + 1.0


@gpu
def test_offsets_past_32_bits(gdn):
    """Over 2^32 bytes and 2^31 elements: the last rows are those of a call on them alone."""
    rows, D = 550_001, 4096
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(rows, D, generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.randn(D, generator=g, device=DEV, dtype=torch.bfloat16)
    out, q, s, r = gdn.gdn_rms_norm(x, w, x, group=128, want_out8=True)
    n = 7
    o1, q1, s1, r1 = gdn.gdn_rms_norm(x[-n:].clone(), w, x[-n:].clone(), group=128, want_out8=True)
    assert torch.equal(out[-n:], o1) and torch.equal(r[-n:], r1) and torch.equal(s[-n:], s1)
    assert torch.equal(q[-n:].view(torch.uint8), q1.view(torch.uint8))
    dx, dw = gdn.gdn_rms_norm_backward(out, x, w)
    d1, _ = gdn.gdn_rms_norm_backward(out[-n:].clone(), x[-n:].clone(), w)
    assert torch.equal(dx[-n:], d1) and dw.isfinite().all()


@gpu
@pytest.mark.parametrize("rows,D", [(9000, 531), (4100, 1024), (5003, 2048), (17000, 72),
                                    (2100, 1016), (2049, 520)], ids=str)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward_of_many_rows(gdn, rows, D, dt):
    """Workgroups that take several rows each, and more than 512 of them."""
    test_backward(gdn, rows, D, dt, True)


def e4m3_ties():
    """448 and the 126 values halfway between neighbouring e4m3 values of 0 to 448."""
    v = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    return torch.cat([torch.tensor([448.0]), (v[1:] + v[:-1]) / 2, torch.tensor([-1.0])])


@gpu
@pytest.mark.parametrize("D", [128, 129, 512, 516, 1024, 4100, 16384])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("group", [0, 128])
def test_quotients_at_ties(gdn, D, dt, group):
    """out8 is y / scale, ties to even: rows of +-1 have s = 1 and y = +-w, and with a
    largest value of 448 c the scale is c and every quotient is a tie. Exact in every step: D / D,
    eps below half a unit of 1, and c times a tie (5 bits) in 8 bits."""
    assert torch.tensor(1.0 / D).mul(D) == 1  # the kernel's mean: the sum D times 1 / D in fp32
    g = torch.Generator().manual_seed(D)
    r = (torch.randint(0, 2, (3, D), generator=g) * 2 - 1).to(DT[dt])
    ties = e4m3_ties()
    for c in (1.0, 3.0, 5.0, 7.0, 1.5 * 2.0 ** 40, 1.75 * 2.0 ** -60):
        w = (ties * c).repeat(-(-D // 128))[:D].to(DT[dt])
        assert torch.equal(w.float(), (ties * c).repeat(-(-D // 128))[:D])
        out, q, scale, _ = gdn.gdn_rms_norm(*dev(r, w), eps=2.0 ** -126, group=group,
                                            want_out8=True)
        assert torch.equal(out.cpu(), r * w)
        assert (scale == c).all()
        want = (r.float() * ties.repeat(-(-D // 128))[:D]).to(torch.float8_e4m3fn)
        assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8)), c


def e4m3_of(q):
    """64-bit values of at most 448 rounded to e4m3 once, ties to even; and each value's distance,
    relative, from the next tie."""
    _, e = torch.frexp(q.abs().clamp(min=2.0 ** -9))
    step = torch.ldexp(torch.ones_like(q), (e - 1).clamp(min=-6) - 3)
    units = q / step
    return torch.round(units) * step, (units.abs().frac() - 0.5).abs() / units.abs().clamp(min=1)


@gpu
@pytest.mark.parametrize("rows,D", [(8192, 128), (5000, 200), (1000, 1024), (300, 5120), (99, 10001)],
                         ids=str)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("how", ["bf16", "bf16+residual", "f32"])
def test_8bit_is_the_64bit_forms(gdn, rows, D, group, how):
    """out8 against y / scale in 64 bits, s cancelled: 448 r w / max |r w|. Without a residual the
    products of two bf16 are exact, a quotient that is no tie is at least 2^-21 from one (integers
    of 16 and 21 bits), and every value has to be the definition's. Else r w, max |r w| and the
    quotient are rounded by 2^-24 each: a value within 2^-22 of a tie may go either way."""
    dtype = torch.float32 if how == "f32" else torch.bfloat16
    x, w, r = inputs(rows + D, rows, D, dtype, how != "bf16")
    _, q, scale, _ = gdn.gdn_rms_norm(*dev(x, w, r), group=group, want_out=False, want_out8=True)
    t = (x.float() if r is None else x.float() + r.float()).double() * w.double()
    q, scale = q.cpu().float().double(), scale.cpu().double()
    _, s, _ = norm64(x, w, r, 1e-6)
    cols, ties = group or D, 0
    for i, part in enumerate(t.split(cols, -1)):
        top = part.abs().amax(-1, keepdim=True)
        assert ((scale[:, i:i + 1] - s * top / 448).abs() <= REL * s * top / 448).all()
        want, off = e4m3_of(part * 448 / top)
        same = q[:, i * cols:i * cols + part.shape[-1]] == want
        ties += int((off == 0).sum())
        assert same.all() if how == "bf16" else (same | (off < 2.0 ** -22)).all()
    assert ties > 0 or how != "bf16" or t.numel() < 10 ** 6  # the check says something


@gpu
def test_8bit_of_values_past_the_range(gdn):
    """y past fp32's range (a large weight): an infinite scale, 0 for the finite values, NaN for the
    infinite one; the other groups are as they were."""
    for D, group in ((128, 0), (256, 128), (2048, 128), (2048, 0)):
        x, w = torch.ones(2, D), torch.ones(D)
        x[:, 5], w[5] = 3.0, 3e38
        out, q, scale, _ = gdn.gdn_rms_norm(*dev(x, w), group=group, want_out8=True)
        q, scale = q.cpu().float(), scale.cpu()
        assert out[:, 5].isinf().all() and scale[:, 0].isinf().all()
        n = group or D
        assert q[:, 5].isnan().all() and (q[:, :5] == 0).all() and (q[:, 6:n] == 0).all()
        if n < D:
            assert (q[:, n:] == 448).all() and scale[:, 1:].isfinite().all()


@gpu
@pytest.mark.parametrize("D", [128, 300, 1024, 2048, 9001])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size,eps", [(0.0, 1e-30), (0.0, 2.0 ** -126), (1e-14, 1e-30),
                                      (1e-17, 2.0 ** -126), (1.0, 2.0 ** -126), (1e14, 1e-6),
                                      (1e16, 1e-6)], ids=str)
def test_backward_of_small_and_large_rows(gdn, D, dt, size, eps):
    """Every eps that is a normal number, and rows whose squares fp32 holds: s^3 alone would leave
    its range. The largest |dx| here is s |w dy| < 2^63 * 20."""
    dtype = DT[dt]
    r, w, _ = inputs(D, 5, D, dtype, False)
    r = (r.float() * size).to(dtype)
    dy = torch.randn(5, D, generator=torch.Generator().manual_seed(3)).to(dtype)
    dx, dw = gdn.gdn_rms_norm_backward(*dev(dy, r, w), eps=eps)
    want, want_w, mag, mag_w = norm_backward64(dy, r, w, None, float(torch.tensor(eps)))
    tol = 2 * REL * mag + (half_step(dtype) * want.abs() * (1 + REL) if dt == "bf16" else 0)
    assert ((dx.cpu().double() - want).abs() <= tol + 1e-37).all()
    assert ((dw.cpu().double() - want_w).abs() <= (REL + U32 * 45) * mag_w + 1e-37).all()
