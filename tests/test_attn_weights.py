"""Weights at the ends of their range in the gradients of causal attention: so small that 16 bits
could lose them."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests.attn_oracle import backward64, within  # noqa: E402

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
