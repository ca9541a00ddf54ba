"""Malformed offsets of the attention and cache calls: their results mean nothing, but nothing
outside the tensors is written. Every output lies inside a larger buffer whose surroundings are
looked at afterwards; inputs lie inside buffers of NaN. All offsets are clamped by the kernels, so
every access of these calls is in bounds."""
import pytest

torch = pytest.importorskip("torch")

DEV = "cuda:0"
pytestmark = pytest.mark.gpu
PAD = 8192  # elements on both sides


class Guarded:
    """A contiguous tensor inside a buffer of a value that no kernel writes."""

    def __init__(self, *shape, dtype=torch.bfloat16, like=None):
        n = 1
        for s in shape:
            n *= s
        self.buffer = torch.full((n + 2 * PAD,), -77.0, dtype=dtype, device=DEV)
        self.t = self.buffer[PAD:PAD + n].view(*shape)
        if like is not None:
            self.t.copy_(like)

    def untouched(self):
        torch.cuda.synchronize()
        return bool((self.buffer[:PAD] == -77).all() and (self.buffer[-PAD:] == -77).all())


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_token_amd as g
    g.load_library()
    return g


def randn(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


BAD = [[0, 500, 100], [-5, 30, 100], [90, 10, 100], [0, 50, 20], [0, 40, 1 << 30],
       [-(1 << 31), -7, -1], [200, 300, 400]]


@pytest.mark.parametrize("cu", BAD)
@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 64), (torch.bfloat16, 256),
                                     (torch.float32, 128)])
def test_prompts_and_gradients(gdn, cu, dtype, D):
    T, Hq, Hk = 100, 4, 2
    q, k, v, do = (randn(i, T, h, D, dtype=dtype) for i, h in enumerate((Hq, Hk, Hk, Hq)))
    out, lse = Guarded(T, Hq, D, dtype=dtype), Guarded(T, Hq, dtype=torch.float32)
    gdn.gdn_attn_varlen_prefill(q, k, v, i32(cu), out=out.t, lse=lse.t)
    assert out.untouched() and lse.untouched()
    # the gradients take any out and lse: those of one whole sequence
    o, l = gdn.gdn_attn_varlen_prefill(q, k, v, i32([0, 0, T]), want_lse=True)
    grads = [Guarded(*t.shape, dtype=dtype) for t in (q, k, v)]
    size = gdn.gdn_attn_backward_workspace_size(2, T, Hq, Hk, D, dtype, True)
    ws = Guarded(size // 4, dtype=torch.float32)
    gdn.gdn_attn_varlen_backward(do, q, k, v, o, l, i32(cu), dq=grads[0].t, dk=grads[1].t,
                                 dv=grads[2].t, workspace=ws.t)
    assert all(x.untouched() for x in (*grads, ws))


@pytest.mark.parametrize("cu", BAD)
@pytest.mark.parametrize("lengths", [[3, 20], [-(1 << 31), (1 << 31) - 1], [31, -40]])
def test_append(gdn, cu, lengths):
    T, Hq, Hk, D, page = 100, 3, 2, 64, 16
    q, k, v = (randn(i, T, h, D) for i, h in enumerate((Hq, Hk, Hk)))
    pools = [Guarded(20, page, Hk, D, like=randn(7 + i, 20, page, Hk, D)) for i in range(2)]
    q_out, k_out = Guarded(T, Hq, D), Guarded(T, Hk, D)
    # a page on either side of the pool, and some of no sequence's: those are left as they were
    table = i32([[0, 1, 2, -1, 4, 20, 6, 7], [8, 9, 10, 11, 1 << 30, 13, 14, -(1 << 31)]])
    free = [3, 5, 12, 15, 16, 17, 18, 19]
    before = [p.t[free].clone() for p in pools]
    freq = torch.ones(8, device=DEV)
    gdn.gdn_kv_append(k, v, pools[0].t, pools[1].t, table, i32(lengths), cu_seqlens=i32(cu), q=q,
                      inv_freq=freq, q_out=q_out.t, k_out=k_out.t)
    assert all(x.untouched() for x in (*pools, q_out, k_out))
    assert all(torch.equal(p.t[free], b) for p, b in zip(pools, before))


@pytest.mark.parametrize("K", [1, 40])
@pytest.mark.parametrize("groups", [[0, 500, 5], [-5, 2, 5], [4, 1, 5], [0, 3, 2], [1, 2, 3],
                                    [-(1 << 31), -3, 1 << 30], [9, 9, 9]])
@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 256), (torch.float32, 64)])
def test_groups_of_prefixes(gdn, groups, K, dtype, D):
    """Sequences that no group holds stand behind no prefix: they have the results of a call
    without prefixes, up to its rounding."""
    B, Hq, Hk, page, cols = 5, 6, 2, 16, 5
    pool = 40
    kc, vc = (randn(i, pool, page, Hk, D, dtype=dtype) for i in range(2))
    q = randn(3, B, K, Hq, D, dtype=dtype)
    table = torch.randperm(pool, generator=torch.Generator().manual_seed(1))[:B * cols]
    table = table.view(B, cols).int().to(DEV)
    lengths = i32([80, 41, 40, 57, 63])
    ptable, plengths = table[:2].contiguous(), i32([70, 33])
    out, lse = Guarded(B, K, Hq, D, dtype=dtype), Guarded(B, K, Hq, dtype=torch.float32)
    size = gdn.gdn_attn_decode_workspace_size(B, K, Hq, Hk, D, page, cols, 2, cols, dtype)
    ws = Guarded((size + 3) // 4, dtype=torch.float32)
    gdn.gdn_attn_decode(q, kc, vc, table, lengths, prefix_table=ptable, prefix_lengths=plengths,
                        prefix_groups=i32(groups), out=out.t, lse=lse.t, workspace=ws.t)
    assert all(x.untouched() for x in (out, lse, ws))
    assert torch.isfinite(out.t.float()).all()
    alone, _ = gdn.gdn_attn_decode(q, kc, vc, table, lengths)
    inside = [max(0, min(B, x)) for x in groups]
    for b in range(B):
        if not any(lo <= b < hi for lo, hi in zip(inside, inside[1:])):
            assert torch.allclose(out.t[b].float(), alone[b].float(), rtol=2e-2, atol=2e-2)
