"""Attention at the sizes where its kernels take another path than in the small tests: key tiles
whose query heads one workgroup walks (all of them, or some), workgroups of eight waves, units of
more rows than a tile, rows joined from more parts than a row has lanes, pieces of prompts and
longer sequences. Against the 64-bit forms of tests/attn_oracle.py; the path is asserted by the
workspace's size where that shows it."""
import pytest

torch = pytest.importorskip("torch")
from tests.attn_oracle import backward64, prompt64, within  # noqa: E402
from tests.test_attn import inputs  # noqa: E402
from tests.test_attn_cache import check_decode  # noqa: E402

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


def fits(rows, cus=256):
    """The paths below are chosen by the number of compute units."""
    if torch.cuda.get_device_properties(0).multi_processor_count != cus:
        pytest.skip(f"sizes chosen for {cus} compute units")
    return rows


def split_of(gdn, n, tokens, total, Hq, Hk, D, dtype, packed):
    """Workgroups that share the query heads of a key head, from the workspace: statistics of
    (query head, token), and the parts of dk and dv where there is more than one."""
    size = gdn.gdn_attn_backward_workspace_size(n, tokens, Hq, Hk, D, dtype, packed)
    part = 2 * total * Hk * D * 4
    return max(1, size // part) if size >= 2 * part else 1


def check_backward(gdn, got, out, q, k, v, do, lo, hi, dt):
    o, _, to, _ = prompt64(q[lo:hi], k[lo:hi], v[lo:hi], DT[dt])
    within(out[lo:hi], o, to, "out")
    want, tol = backward64(do[lo:hi], q[lo:hi], k[lo:hi], v[lo:hi], DT[dt])
    for x, w, t, name in zip(got, want, tol, ("dq", "dk", "dv")):
        within(x[lo:hi], w, t, name)


# sequences of 60 tokens: one key tile each; 8 key heads of 4 query heads
@pytest.mark.parametrize("N,split", [(64, 1), (33, 2), (20, 4)])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64),
                                  ("f32", 128), ("f32", 256)])
@pytest.mark.parametrize("packed", [False, True])
def test_query_heads_walked_by_a_workgroup(gdn, N, split, dt, D, packed):
    fits(N)
    T, Hq, Hk = 60, 32, 8  # within a key tile of every type and width (64 rows at the least)
    total = N * T
    q, k, v, do = inputs(N + D, (total,), Hq, Hk, D, DT[dt], 4)
    qd, kd, vd, dd = dev(q, k, v, do)
    if packed:
        cu = torch.arange(0, total + 1, T, dtype=torch.int32, device=DEV)
        out, lse = gdn.gdn_attn_varlen_prefill(qd, kd, vd, cu, want_lse=True)
        got = gdn.gdn_attn_varlen_backward(dd, qd, kd, vd, out, lse, cu)
        # a packed batch counts total / rows tiles more: at the most as many parts
        assert split_of(gdn, N, total, total, Hq, Hk, D, DT[dt], True) <= split
    else:
        dense = [t.view(N, T, *t.shape[1:]) for t in (qd, kd, vd, dd)]
        out, lse = gdn.gdn_attn_prefill(*dense[:3], want_lse=True)
        got = [t.flatten(0, 1) for t in
               gdn.gdn_attn_backward(dense[3], *dense[:3], out, lse)]
        out = out.flatten(0, 1)
        assert split_of(gdn, N, T, total, Hq, Hk, D, DT[dt], False) == split
    for n in (0, N // 2, N - 1):
        check_backward(gdn, got, out, q, k, v, do, n * T, (n + 1) * T, dt)


@pytest.mark.parametrize("N,Hq", [(33, 24), (20, 32)])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64),
                                  ("f32", 128), ("f32", 256)])
def test_query_heads_walked_over_several_tiles(gdn, N, Hq, dt, D):
    """Two key tiles and more per sequence, and query tiles that start in the middle of the head:
    a workgroup restarts at its own first tile for every head (all three, or two of four)."""
    T, Hk = 300, 8
    fits(N)
    q, k, v, do = inputs(D, (N, T), Hq, Hk, D, DT[dt], 4)
    qd, kd, vd, dd = dev(q, k, v, do)
    out, lse = gdn.gdn_attn_prefill(qd, kd, vd, want_lse=True)
    got = gdn.gdn_attn_backward(dd, qd, kd, vd, out, lse)
    assert split_of(gdn, N, T, N * T, Hq, Hk, D, DT[dt], False) < Hq // Hk
    for n in (0, N - 1):
        check_backward(gdn, [x[n] for x in got], out[n], q[n], k[n], v[n], do[n], 0, T, dt)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("packed", [False, True])
def test_fp32_workgroups_of_eight_waves(gdn, D, packed):
    """At least one tile of 128 queries (the gradients of 256-wide heads: 64) and head per
    compute unit."""
    N, T, Hq, Hk = fits(27), 150, 8, 4
    q, k, v, do = inputs(D + 7, (N * T,), Hq, Hk, D, torch.float32, 4)
    qd, kd, vd, dd = dev(q, k, v, do)
    if packed:
        cuts = [0] + [i * T + (i % 5) * 3 for i in range(1, N)] + [N * T]
        cu = torch.tensor(cuts, dtype=torch.int32, device=DEV)
        out, lse = gdn.gdn_attn_varlen_prefill(qd, kd, vd, cu, want_lse=True)
        got = gdn.gdn_attn_varlen_backward(dd, qd, kd, vd, out, lse, cu)
    else:
        cuts = list(range(0, N * T + 1, T))
        dense = [t.view(N, T, *t.shape[1:]) for t in (qd, kd, vd, dd)]
        out, lse = gdn.gdn_attn_prefill(*dense[:3], want_lse=True)
        got = [t.flatten(0, 1) for t in
               gdn.gdn_attn_backward(dense[3], *dense[:3], out, lse)]
        out = out.flatten(0, 1)
    for n in (0, 7, N - 1):
        check_backward(gdn, got, out, q, k, v, do, cuts[n], cuts[n + 1], "f32")


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64),
                                  ("f32", 128), ("f32", 256)])
@pytest.mark.parametrize("packed", [False, True])
def test_longer_sequences(gdn, dt, D, packed):
    lengths = [701, 0, 1, 390] if packed else [701]
    Hq, Hk = 2, 1
    q, k, v, do = inputs(D + 3, (sum(lengths),), Hq, Hk, D, DT[dt], 4)
    qd, kd, vd, dd = dev(q, k, v, do)
    cuts = torch.tensor([0] + lengths).cumsum(0).tolist()
    if packed:
        cu = torch.tensor(cuts, dtype=torch.int32, device=DEV)
        out, lse = gdn.gdn_attn_varlen_prefill(qd, kd, vd, cu, want_lse=True)
        got = gdn.gdn_attn_varlen_backward(dd, qd, kd, vd, out, lse, cu)
    else:
        out, lse = gdn.gdn_attn_prefill(qd[None], kd[None], vd[None], want_lse=True)
        got = [x[0] for x in
               gdn.gdn_attn_backward(dd[None], qd[None], kd[None], vd[None], out, lse)]
        out = out[0]
    for lo, hi in zip(cuts, cuts[1:]):
        if hi > lo:
            check_backward(gdn, got, out, q, k, v, do, lo, hi, dt)


# ------------------------------------------------------------------- decode


@pytest.mark.parametrize("dt,D,length", [("bf16", 64, 9000), ("bf16", 128, 13000),
                                         ("bf16", 256, 26000), ("f32", 64, 9000)])
def test_rows_of_more_parts_than_lanes(gdn, dt, D, length):
    """One sequence of one key head is dealt out ten tiles of 32 keys to a workgroup, some of them
    taken by the unit's start: more parts than the D / 4 lanes that join a row."""
    assert length / 320 > D / 4
    check_decode(gdn, D, 1, [length], [], None, 64, 2, 1, D, dt)


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f32", 128)])
def test_prefixes_of_more_parts_than_lanes(gdn, dt, D):
    check_decode(gdn, D + 1, 1, [5, 40], [20000], [0, 2], 64, 2, 1, D, dt)


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64),
                                  ("f32", 128), ("f32", 256)])
@pytest.mark.parametrize("B,cuts", [(64, [0, 64]), (70, [0, 3, 70]), (87, [0, 43, 87])])
def test_groups_of_more_rows_than_a_tile(gdn, dt, D, B, cuts):
    """Six rows per sequence: a full tile of 256 and a half one (384), two full ones (402, of
    which a small group of 18 is in front), groups of 258 and 264; from tile to head and from
    head to group."""
    g = torch.Generator().manual_seed(B)
    lengths = torch.randint(1, 40, (B,), generator=g).tolist()
    prefixes = [700, 333][:len(cuts) - 1]
    check_decode(gdn, B + D, 1, lengths, prefixes, cuts, 16, 12, 2, D, dt)


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64),
                                  ("f32", 256)])
@pytest.mark.parametrize("lengths,prefix", [([300, 300], 0), ([300, 1100], 0), ([320, 300], 200)])
def test_pieces_of_prompts(gdn, dt, D, lengths, prefix):
    """300 new tokens at once: the first of a prompt, behind cached ones, behind a prefix."""
    check_decode(gdn, D + 5, 300, lengths, [prefix] if prefix else [], [0, 2] if prefix else None,
                 32, 4, 2, D, dt)
