"""How far bf16 results are off as a whole, relative to their norm. The bounds of single values
(tests/attn_oracle.py) add up the largest error of every rounding; these count roundings.

Half a step is u = 2^-8 at a mantissa of 1, and errors are spread evenly: a rounded value x of
mantissa m is off by u / (sqrt(3) m) |x|. Over values whose logarithms are spread evenly (E m^2 =
3 / (2 ln 2)) that is 1.53e-3 of the norm; for a normal distribution, whose large values lie below
the average mantissa, 1.66e-3 (4 million values). Independent roundings add in squares."""
import pytest

torch = pytest.importorskip("torch")
from tests.attn_oracle import attend64  # noqa: E402
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
