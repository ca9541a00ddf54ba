"""How far bf16 results are off as a whole, relative to their norm. The bounds of single values
(tests/attn_oracle.py) add up the largest error of every rounding; these count roundings.

Half a step is u = 2^-8 at a mantissa of 1, and errors are spread evenly: a rounded value x of
mantissa m is off by u / (sqrt(3) m) |x|. Over values whose logarithms are spread evenly (E m^2 =
3 / (2 ln 2)) that is 1.53e-3 of the norm; for a normal distribution, whose large values lie below
the average mantissa, 1.66e-3 (4 million values). Independent roundings add in squares."""
import pytest

torch = pytest.importorskip("torch")
from tests.attn_oracle import attend64, backward64  # noqa: E402
from tests.test_attn_cache import cache  # noqa: E402

DEV = "cuda:0"
pytestmark = pytest.mark.gpu
ONE = 1.66e-3  # of one rounding


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_token_amd as g
    g.load_library()
    return g


def off(got, want):
    got, want = got.detach().cpu().double(), want.double()
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("K", [1, 4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tokens_against_the_cache(gdn, D, K):
    """Up to 32 rows per key head: out is rounded and nothing else. With weights rounded to bf16
    it would be sqrt(2) as far off, 2.3e-3."""
    lengths, Hq, Hk, page = [700, 90, 333, 1200], 12, 2, 16
    kc, vc, table, _, own, _ = cache(D, lengths, [], page, Hk, D, torch.bfloat16)
    q = (1.5 * torch.randn(len(lengths), K, Hq, D,
                           generator=torch.Generator().manual_seed(K))).bfloat16()
    out, _ = gdn.gdn_attn_decode(*[t.to(DEV) for t in (
        q, kc, vc, table, torch.tensor(lengths, dtype=torch.int32))])
    want = torch.empty(q.shape, dtype=torch.float64)
    for b, n in enumerate(lengths):
        seen = torch.arange(n) <= (n - K + torch.arange(K))[:, None]
        for h in range(Hq):
            k, v = (x[:, h // (Hq // Hk)] for x in own[b])
            want[b, :, h] = attend64(q[b, :, h], k, v, seen, torch.bfloat16)[0]
    far = off(out, want)
    assert far < 1.1 * ONE


def gradients(gdn, q, k, v, do):
    q, k, v, do = (t.to(DEV) for t in (q, k, v, do))
    out, lse = gdn.gdn_attn_prefill(q, k, v, want_lse=True)
    return gdn.gdn_attn_backward(do, q, k, v, out, lse)


def test_key_gradients_as_a_whole(gdn):
    """bf16 dk: ds rounded as an operand, the sum rounded, and the weights in ds held to 2^-10
    (a quarter of bf16's error): sqrt(1 + 1 + 1/16) 1.66e-3 = 2.4e-3, and delta's part from out as
    stored. With the weights in ds rounded to bf16 as well it would be sqrt(3) 1.66e-3 = 2.9e-3."""
    T, Hq, Hk, D = 600, 4, 1, 128
    g = torch.Generator().manual_seed(11)
    q = (1.5 * torch.randn(1, T, Hq, D, generator=g)).bfloat16()
    k, v = (torch.randn(1, T, Hk, D, generator=g).bfloat16() for _ in range(2))
    do = torch.randn(1, T, Hq, D, generator=g).bfloat16()
    dk = gradients(gdn, q, k, v, do)[1]
    want, _ = backward64(do[0], q[0], k[0], v[0], torch.bfloat16)
    far = off(dk[0], want[1])
    assert far < 2.65e-3


@pytest.mark.parametrize("D", [64, 128, 256])
def test_gradients_of_short_sequences_as_a_whole(gdn, D):
    """bf16, sequences of two tokens: dout . v - delta is a small difference of large terms. ds and
    the sum rounded: sqrt(2) 1.66e-3 = 2.3e-3. From out as stored these come out 5e-3 off (in 64 bits
    with those roundings alone), single sequences more; the limit lies between."""
    N, Hq, Hk = 400, 2, 1
    g = torch.Generator().manual_seed(D)
    q = (1.5 * torch.randn(N, 2, Hq, D, generator=g)).bfloat16()
    k, v = (torch.randn(N, 2, Hk, D, generator=g).bfloat16() for _ in range(2))
    do = torch.randn(N, 2, Hq, D, generator=g).bfloat16()
    got = gradients(gdn, q, k, v, do)
    want = [torch.stack(x) for x in
            zip(*[backward64(do[i], q[i], k[i], v[i], torch.bfloat16)[0] for i in range(N)])]
    for x, w, name in zip(got, want, ("dq", "dk", "dv")):
        far = off(x, w)
        assert far < 4e-3, name
