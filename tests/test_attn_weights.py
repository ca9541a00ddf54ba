"""Weights at the ends of their range in attention and its gradients: scores so large that fp32
holds them in steps of a quarter, weights so small that 16 bits lose them, weights that are a part
of a row's, weights of 0. Scores are sums of integers below 2^24 and exact in fp32 in any order, so
the bounds of the tests of large ones hold no error of theirs."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests.attn_oracle import U32, backward64, causal, half_step, within  # noqa: E402

DEV = "cuda:0"
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_token_amd as g
    g.load_library()
    return g


def dev(*ts):
    return [t.to(DEV) for t in ts]


def gradients(gdn, q, k, v, do, scale):
    qd, kd, vd, dd = dev(q, k, v, do)
    out, lse = gdn.gdn_attn_prefill(qd, kd, vd, scale=scale, want_lse=True)
    return (out, lse, *gdn.gdn_attn_backward(dd, qd, kd, vd, out, lse, scale=scale))


# ------------------------------------------------------------ weights far below 1


@pytest.mark.parametrize("drop", [16, 28, 44, 68])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_gradients_of_keys_with_small_weights(gdn, dt, D, drop):
    """Two keys whose scores lie `drop` nats below the others (weights of 2^-23 to 2^-98): their
    gradients are as exact, relative to their size, as any other key's."""
    T, Hq, Hk = 150, 4, 2
    g = torch.Generator().manual_seed(D + drop)
    q, do = (torch.randn(1, T, Hq, D, generator=g).to(DT[dt]) for _ in range(2))
    k, v = (torch.randn(1, T, Hk, D, generator=g).to(DT[dt]) for _ in range(2))
    scale = D ** -0.5
    q[..., 0] = 1 / scale      # a power of two, or 11.3: the score falls by about `drop`
    k[..., 0] = 0.0
    low = [37, 101]
    k[:, low, :, 0] = -float(drop)
    got = gradients(gdn, q, k, v, do, scale)[2:]
    want, tol = backward64(do[0], q[0], k[0], v[0], DT[dt], scale)
    weight = math.exp(-drop)
    assert 0 < want[1][low].abs().max() < 1e3 * weight  # that small, and not nothing
    for x, w, t, name in zip(got, want, tol, ("dq", "dk", "dv")):
        within(x[0], w, t, name)


# ---------------------------------------------------------------- large scores


def integers(seed, T, Hq, Hk, D, level, dtype):
    """q, k whose scores (scale 1) are level + 0 to 24 in whole numbers, exact in bf16 and in
    fp32; level a power of two from 2^10 to 2^23, either sign."""
    g = torch.Generator().manual_seed(seed)
    q = torch.zeros(1, T, Hq, D)
    k = torch.zeros(1, T, Hk, D)
    a = 2.0 ** min(10, int(math.log2(abs(level))))
    q[..., 0], k[..., 0] = math.copysign(a, level), abs(level) / a
    q[..., 1:5] = torch.randint(0, 3, (1, T, Hq, 4), generator=g).float()
    k[..., 1:5] = torch.randint(0, 4, (1, T, Hk, 4), generator=g).float()
    v, do = (torch.randn(1, T, h, D, generator=g).to(dtype) for h in (Hk, Hq))
    return q.to(dtype), k.to(dtype), v, do


def whole64(q, k, v, do, dtype, spread):
    """The oracle's values with bounds for exact scores that differ by up to `spread` in a row.
    A weight is 2^x with x a difference of at most spread log2(e) + 8 formed by one fused
    multiply-add from the scale in log2 units, both rounded to U, and exp2, good to 2 U; it is
    divided by a sum of n such: p off by (2 spread + 6) U from x (8 ln 2 < 6), as much from the
    sum, and by (n + 16) U. Rounded to the type as operands: u each."""
    T, Hq, D = q.shape
    Hk = k.shape[1]
    g, u = Hq // Hk, half_step(dtype)
    out, to = (torch.zeros(T, Hq, D).double() for _ in range(2))
    dq, tq = (torch.zeros(T, Hq, D).double() for _ in range(2))
    dk, dv, tk, tv = (torch.zeros(T, Hk, D).double() for _ in range(4))
    pe = (2 * (2 * spread + 6) + T + 32) * U32
    for h in range(Hq):
        j = h // g
        a, b, c, d = q[:, h].double(), k[:, j].double(), v[:, j].double(), do[:, h].double()
        s = (a @ b.T).masked_fill(~causal(T), -math.inf)
        p = torch.softmax(s, 1)
        out[:, h] = p @ c
        to[:, h] = (u + pe) * (p @ c.abs()) + u * out[:, h].abs()
        dp = d @ c.T
        delta = (d * out[:, h]).sum(1, keepdim=True)
        edp = (D + 4) * U32 * (d.abs() @ c.abs().T)
        edelta = ((d.abs() * to[:, h]).sum(1, keepdim=True) +
                  (D + 4) * U32 * (d * out[:, h]).abs().sum(1, keepdim=True))
        ds = p * (dp - delta)
        eds = p * ((3 * u + pe) * (dp - delta).abs() + edp + edelta)
        more = g * (T + 16) * U32
        dq[:, h] = ds @ b
        tq[:, h] = (eds + more * ds.abs()) @ b.abs()
        dk[:, j] += ds.T @ a
        tk[:, j] += (eds + more * ds.abs()).T @ a.abs()
        dv[:, j] += p.T @ d
        tv[:, j] += (p * (u + pe + more)).T @ d.abs()
    for x, t in ((dq, tq), (dk, tk), (dv, tv)):
        t += u * x.abs() + 1e-37
    return (out, dq, dk, dv), (to, tq, tk, tv)


@pytest.mark.parametrize("level", [2.0 ** 10, -2.0 ** 16, 2.0 ** 20, -2.0 ** 22, 1.5 * 2 ** 22])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64),
                                  ("f32", 128), ("f32", 256)])
def test_large_scores(gdn, dt, D, level):
    """Out and the gradients depend on the differences of a row's scores alone: with the 64-bit
    values at the bounds of small scores, whatever their level."""
    T, Hq, Hk = 140, 4, 2
    q, k, v, do = integers(D, T, Hq, Hk, D, level, DT[dt])
    out, lse, dq, dk, dv = gradients(gdn, q, k, v, do, 1.0)
    want, tol = whole64(q[0], k[0], v[0], do[0], DT[dt], 24.0)
    for x, w, t, name in zip((out, dq, dk, dv), want, tol, ("out", "dq", "dk", "dv")):
        within(x[0], w, t, name)


@pytest.mark.parametrize("level", [2.0 ** 15, 2.0 ** 18, 1.25 * 2 ** 20, -1.5 * 2 ** 20,
                                   1.75 * 2 ** 22])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_equal_scores_have_equal_weights(gdn, dt, level):
    """Every key of a row has the same score: dv_j = sum over t >= j of dout_t / (t + 1)."""
    T, D = 100, 64
    q, k = torch.zeros(1, T, 1, D), torch.zeros(1, T, 1, D)
    q[..., 0], k[..., 0] = math.copysign(1024.0, level), abs(level) / 1024
    g = torch.Generator().manual_seed(1)
    v, do = (torch.randn(1, T, 1, D, generator=g).to(DT[dt]) for _ in range(2))
    dv = gradients(gdn, q.to(DT[dt]), k.to(DT[dt]), v, do, 1.0)[4]
    p = causal(T).double() / torch.arange(1, T + 1).double()[:, None]
    want = p.T @ do[0, :, 0].double()
    u = half_step(DT[dt])
    tol = (u + (2 * T + 32) * U32) * (p.T @ do[0, :, 0].double().abs()) + u * want.abs()
    within(dv[0, :, 0], want, tol)


# ---------------------------------------------- how far off the results are as a whole

# The error of n rounded values relative to their norm: half a step is u = 2^-8 (bf16) at a
# mantissa of 1, evenly spread errors have u / sqrt(3) m^-1 of the value at mantissa m. Over
# values whose logarithms are spread evenly, with E m^2 = 3 / (2 ln 2), that is
# u / sqrt(3) / sqrt(2.164) = 1.53e-3; for values of a normal distribution 1.66e-3 (most of the
# norm lies where mantissas are a little below the average). Independent roundings add in squares.
ROUNDED = 1.66e-3


def off(x, want):
    x, want = x.detach().cpu().double(), want.double()
    return float((x - want).norm() / want.norm())


def test_key_gradients_as_a_whole(gdn):
    """bf16 dk: ds rounded as an operand, the sum rounded, and the weights in ds held to 2^-10
    (a quarter of bf16's error): sqrt(1 + 1 + 1/16) 1.66e-3 = 2.4e-3, and delta's part from out as
    stored. With the weights in ds rounded to bf16 as well it would be sqrt(3) 1.66e-3 = 2.9e-3."""
    T, Hq, Hk, D = 600, 4, 1, 128
    g = torch.Generator().manual_seed(11)
    q = (1.5 * torch.randn(1, T, Hq, D, generator=g)).bfloat16()
    k, v = (torch.randn(1, T, Hk, D, generator=g).bfloat16() for _ in range(2))
    do = torch.randn(1, T, Hq, D, generator=g).bfloat16()
    dk = gradients(gdn, q, k, v, do, D ** -0.5)[3]
    want, _ = backward64(do[0], q[0], k[0], v[0], torch.bfloat16)
    assert off(dk[0], want[1]) < 2.65e-3


@pytest.mark.parametrize("D", [64, 128, 256])
def test_gradients_of_short_sequences_as_a_whole(gdn, D):
    """bf16, sequences of two tokens: dout . v - delta is a small difference of large terms. ds and
    the sum rounded: 2.3e-3; dk sums two of them per head. From out as stored it came out 2e-2 off;
    the limit lies between."""
    N, Hq, Hk = 400, 2, 1
    g = torch.Generator().manual_seed(D)
    q = (1.5 * torch.randn(N, 2, Hq, D, generator=g)).bfloat16()
    k, v = (torch.randn(N, 2, Hk, D, generator=g).bfloat16() for _ in range(2))
    do = torch.randn(N, 2, Hq, D, generator=g).bfloat16()
    got = gradients(gdn, q, k, v, do, D ** -0.5)[2:]
    want = [torch.stack(x) for x in
            zip(*[backward64(do[i], q[i], k[i], v[i], torch.bfloat16)[0] for i in range(N)])]
    for x, w, name in zip(got, want, ("dq", "dk", "dv")):
        assert off(x, w) < 4e-3, name


@pytest.mark.parametrize("level", [2.0 ** 12, -2.0 ** 20, 1.5 * 2 ** 22])
@pytest.mark.parametrize("K", [1, 5, 40])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 256), ("f32", 128)])
def test_large_scores_against_the_cache(gdn, dt, D, K, level):
    """The same against a cache, its parts joined: without a prefix, and with the first 96 tokens
    as a prefix. Each of at most 32 parts is multiplied by 2^(m_i - m), one rounding and 2 U."""
    n, Hq, Hk, page = 500, 4, 2, 16
    q, k, v, _ = integers(D + K, n, Hq, Hk, D, level, DT[dt])
    q = q[:, -K:].contiguous()
    u, g = half_step(DT[dt]), Hq // Hk
    pe = (2 * (2 * 24.0 + 6) + n + 32 + 3 * 32) * U32
    seen = torch.arange(n) <= (n - K + torch.arange(K))[:, None]
    pools = [t[0].contiguous() for t in (k, v)]
    pools = [torch.cat([t, t.new_full((-n % page, Hk, D), math.nan)]).view(-1, page, Hk, D).to(DEV)
             for t in pools]
    table = torch.arange(pools[0].shape[0], dtype=torch.int32, device=DEV)[None]

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)
    first = 96
    calls = [(table, i32(n), {}),
             (table[:, first // page:].contiguous(), i32(n - first),
              {"prefix_table": table[:, :first // page].contiguous(), "prefix_lengths": i32(first),
               "prefix_groups": i32(0, 1)})]
    for pages, lengths, shared in calls:
        out, _ = gdn.gdn_attn_decode(q.to(DEV), *pools, pages, lengths, scale=1.0, **shared)
        for h in range(Hq):
            a, b, c = q[0, :, h].double(), k[0, :, h // g].double(), v[0, :, h // g].double()
            p = torch.softmax((a @ b.T).masked_fill(~seen, -math.inf), 1)
            want = p @ c
            within(out[0, :, h], want, (u + pe) * (p @ c.abs()) + u * want.abs(), (h, len(shared)))


# ------------------------------------------------- weights that are a part of a row's


@pytest.mark.parametrize("P", [1, 40, 300])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64),
                                  ("f32", 128), ("f32", 256)])
def test_gradients_of_the_keys_behind_others(gdn, dt, D, P):
    """The formulas hold with the out and lse of queries that see P keys more than are given: p and
    delta are the whole row's. Against all P + T keys in 64 bits: dk and dv of the keys given, and
    dq's part over them; the oracle's bounds of the whole sequence."""
    T, Hq, Hk = 90, 4, 2
    g = torch.Generator().manual_seed(D + P)
    n, dtype = P + T, DT[dt]
    q, do = (torch.randn(1, n, Hq, D, generator=g).to(dtype) for _ in range(2))
    k, v = (torch.randn(1, n, Hk, D, generator=g).to(dtype) for _ in range(2))
    qd, kd, vd, dd = dev(q, k, v, do)
    out, lse = gdn.gdn_attn_prefill(qd, kd, vd, want_lse=True)
    part = [t[:, P:].contiguous() for t in (dd, qd, kd, vd, out, lse)]
    dq, dk, dv = gdn.gdn_attn_backward(*part)
    want, tol = backward64(do[0], q[0], k[0], v[0], dtype)
    within(dk[0], want[1][P:], tol[1][P:], "dk")
    within(dv[0], want[2][P:], tol[2][P:], "dv")
    for h in range(Hq):
        a, b, c, d = (x[0, :, i].double() for x, i in ((q, h), (k, h // 2), (v, h // 2), (do, h)))
        p = torch.softmax((a @ b.T * D ** -0.5).masked_fill(~causal(n), -math.inf), 1)
        ds = p * (d @ c.T - (d * (p @ c)).sum(1, keepdim=True))
        exact = (D ** -0.5 * ds[:, P:] @ b[P:])[P:]
        within(dq[0, :, h], exact, tol[0][P:, h] + half_step(dtype) * exact.abs(), "dq")


# ---------------------------------------------------------------- weights of 0


def test_a_value_that_is_not_finite_behind_infinite_keys(gdn):
    """A tile of keys whose scores are all -infinity (keys of infinity against a negative query)
    beside a tile of ordinary ones, dealt to another wave or the same: a NaN among the tile's
    values is seen and reaches its column of out, as it does over whole prompts."""
    D, page, n = 64, 32, 96
    for tile in (0, 1, 2):
        q = torch.full((1, 1, 1, D), -1.0)
        k = torch.randn(n, 1, D, generator=torch.Generator().manual_seed(tile))
        v = torch.randn(n, 1, D, generator=torch.Generator().manual_seed(tile + 9))
        k[32 * tile:32 * tile + 32, 0, 3] = float("inf")
        v[32 * tile + 5, 0, 7] = float("nan")
        for dtype in (torch.bfloat16, torch.float32):
            kc, vc = (x.view(n // page, page, 1, D).to(dtype).to(DEV) for x in (k, v))
            table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None]
            out, _ = gdn.gdn_attn_decode(q.to(dtype).to(DEV), kc, vc, table,
                                         torch.tensor([n], dtype=torch.int32, device=DEV))
            lost = torch.zeros(D, dtype=torch.bool)
            lost[7] = True
            out = out[0, 0, 0].cpu()
            assert torch.isnan(out[lost]).all() and torch.isfinite(out[~lost]).all(), (tile, dtype)
