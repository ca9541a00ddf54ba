"""C-ABI checks of the scan, norm and beam calls that need no GPU: exports,
argument validation before any HIP call, and the binding's refusals."""
import os
import re

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLP, SHAPE, UNSUP, MISAL, ALIAS, HIPERR = range(7)
F32, BF16 = 0, 1
A, MB = 1 << 40, 1 << 20


def P(i):
    return A + i * (1 << 36)  # disjoint, aligned regions; never dereferenced


@pytest.fixture(scope="module")
def lib():
    import gated_deltanet_token_amd as g
    return g.load_library()


def test_exports(lib):
    text = open(os.path.join(ROOT, "include", "gdn.h")).read()
    names = re.findall(r"^\s*(?:gdn_status_t|size_t)\s*(gdn_\w+)\s*\(", text, flags=re.M)
    import gated_deltanet_token_amd as g
    for want in ("gdn_scan_prefill", "gdn_scan_varlen_prefill", "gdn_scan_backward",
                 "gdn_scan_varlen_backward", "gdn_scan_decode", "gdn_scan_workspace_size",
                 "gdn_rms_norm", "gdn_rms_norm_backward", "gdn_rms_norm_workspace_size",
                 "gdn_beam_select", "gdn_beam_workspace_size", "gdn_gather_states"):
        assert want in names and want in g.EXPORTS and hasattr(lib, want), want


def scan(lib, x=P(0), a=P(1), b=P(2), h0=P(3), out=P(4), hT=P(5), pre=None, every=0, B=2, T=300,
         D=64, dtype=BF16, flags=0, ws=None, wsb=0):
    return lib.gdn_scan_prefill(x, a, b, h0, out, hT, pre, every, B, T, D, dtype, flags, ws, wsb,
                                None)


def packed(lib, x=P(0), a=P(1), b=P(2), cu=P(6), N=3, total=300, h0=P(3), out=P(4), hT=P(5),
           pre=None, every=0, D=64, dtype=BF16, flags=0, ws=None, wsb=0):
    return lib.gdn_scan_varlen_prefill(x, a, b, cu, N, total, h0, out, hT, pre, every, D, dtype,
                                       flags, ws, wsb, None)


def back(lib, dy=P(7), x=P(0), a=P(1), b=P(2), h0=P(3), pre=P(8), every=2, dhT=P(9), dx=P(10),
         da=P(11), db=P(12), dh0=P(13), B=2, T=300, D=64, dtype=BF16, flags=0, ws=None, wsb=0):
    return lib.gdn_scan_backward(dy, x, a, b, h0, pre, every, dhT, dx, da, db, dh0, B, T, D, dtype,
                                 flags, ws, wsb, None)


def test_scan_validation(lib):
    assert scan(lib, x=None) == NULLP
    assert scan(lib, out=None) == NULLP
    assert scan(lib, B=0) == SHAPE
    assert scan(lib, T=-1) == SHAPE
    assert scan(lib, D=0) == SHAPE
    assert scan(lib, D=(1 << 22) + 1) == UNSUP
    assert scan(lib, dtype=3) == UNSUP
    for f in (1, 3, 4, 1 << 31):  # only the gate logits apply here
        assert scan(lib, flags=f) == UNSUP
        assert back(lib, flags=f) == UNSUP
    assert scan(lib, a=P(1) + 8) == MISAL
    assert scan(lib, out=P(0)) == ALIAS
    assert scan(lib, hT=P(3) + 16) == ALIAS        # neither the initial state nor apart from it
    assert scan(lib, hT=P(4) + 4096) == ALIAS
    assert scan(lib, pre=P(14), every=0) == SHAPE
    assert scan(lib, pre=P(4), every=1) == ALIAS
    assert scan(lib, ws=P(4), wsb=4096) == ALIAS
    assert scan(lib, ws=P(14) + 4, wsb=4096) == MISAL
    assert scan(lib, B=1 << 30, T=1 << 40) == SHAPE
    assert scan(lib, x=None, a=None, b=None, out=None, hT=None, T=0) == OK
    assert packed(lib, cu=None) == NULLP
    assert packed(lib, N=0) == SHAPE
    assert packed(lib, total=1 << 31) == SHAPE
    assert packed(lib, cu=P(6) + 4) == MISAL
    assert packed(lib, out=P(6)) == ALIAS


def test_scan_backward_validation(lib):
    assert back(lib, dy=None) == NULLP
    assert back(lib, dx=None) == NULLP
    assert back(lib, db=None) == NULLP
    assert back(lib, b=None) == SHAPE                      # tied gates take no dbeta
    assert back(lib, pre=None) == NULLP                    # 300 tokens need prefix states
    assert back(lib, every=3) == UNSUP                     # 192 does not divide the tile
    assert back(lib, every=4) == UNSUP
    assert back(lib, every=0) == SHAPE
    assert back(lib, dx=P(0)) == ALIAS
    assert back(lib, da=P(10) + 64) == ALIAS
    assert back(lib, dh0=P(3)) == ALIAS
    assert back(lib, dh0=P(9)) == ALIAS
    assert back(lib, dy=P(7) + 2) == MISAL


def test_scan_decode_validation(lib):
    def call(x=P(0), a=P(1), b=P(2), pool=P(3), ns=8, src=P(4), dst=P(5), out=P(6), B=4, K=2,
             D=64, dtype=BF16, flags=0):
        return lib.gdn_scan_decode(x, a, b, pool, ns, src, dst, out, B, K, D, dtype, flags, None)
    assert call(pool=None) == NULLP
    assert call(src=None) == NULLP
    assert call(out=None) == NULLP
    assert call(B=0) == SHAPE
    assert call(K=-1) == SHAPE
    assert call(ns=0) == SHAPE
    assert call(D=0) == SHAPE
    assert call(flags=1) == UNSUP
    assert call(dtype=2) == UNSUP
    assert call(src=P(4) + 2) == MISAL
    assert call(pool=P(0)) == ALIAS
    assert call(src=P(3) + 64) == ALIAS


def test_norm_validation(lib):
    def call(x=P(0), res=P(1), w=P(2), ro=P(3), out=P(4), o8=P(5), sc=P(6), group=0, rows=10,
             D=100, dtype=BF16, eps=1e-6):
        return lib.gdn_rms_norm(x, res, w, ro, out, o8, sc, group, rows, D, dtype, eps, None)
    assert call(x=None) == NULLP
    assert call(w=None) == NULLP
    assert call(out=None, o8=None, sc=None) == NULLP
    assert call(sc=None) == NULLP
    assert call(o8=None) == NULLP
    assert call(res=None) == NULLP                 # residual_out without a residual
    assert call(rows=-1) == SHAPE
    assert call(D=0) == SHAPE
    assert call(D=16385) == UNSUP
    assert call(group=64) == UNSUP
    assert call(dtype=2) == UNSUP
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(eps=eps) == SHAPE
    assert call(w=P(2) + 2) == MISAL
    assert call(out=P(0)) == ALIAS
    assert call(ro=P(0) + 64) == ALIAS             # neither x nor the residual, nor apart
    assert call(ro=P(4)) == ALIAS
    assert call(sc=P(5)) == ALIAS
    assert call(rows=0) == OK

    def back(dy=P(0), r=P(1), w=P(2), dres=P(3), dx=P(4), dw=P(5), rows=10, D=100, dtype=BF16,
             eps=1e-6, ws=P(6), wsb=1 << 20):
        return lib.gdn_rms_norm_backward(dy, r, w, dres, dx, dw, rows, D, dtype, eps, ws, wsb,
                                         None)
    assert back(dx=None) == NULLP
    assert back(ws=None, wsb=0) == NULLP
    assert back(wsb=16) == SHAPE
    assert back(dx=P(0)) == ALIAS
    assert back(dw=P(4)) == ALIAS
    assert back(ws=P(5)) == ALIAS
    assert back(rows=0, dw=None) == OK
    assert lib.gdn_rms_norm_workspace_size(10, 100) >= 400
    assert lib.gdn_rms_norm_workspace_size(0, 100) == 0
    assert lib.gdn_rms_norm_workspace_size(10, 0) == 0


def test_beam_validation(lib):
    def call(lg=P(0), s=P(1), fin=P(2), sl=P(3), ns=P(4), tok=P(5), par=P(6), nf=P(7), src=P(8),
             B=2, W=4, V=1000, eos=2, dtype=BF16, ws=P(9), wsb=1 << 24):
        return lib.gdn_beam_select(lg, s, fin, sl, ns, tok, par, nf, src, B, W, V, eos, dtype, ws,
                                   wsb, None)
    assert call(lg=None) == NULLP
    assert call(par=None) == NULLP
    assert call(sl=None) == NULLP                  # src_slots without beam_slots
    assert call(src=None) == NULLP
    assert call(ws=None, wsb=0) == SHAPE or call(ws=None, wsb=0) == NULLP
    assert call(wsb=64) == SHAPE
    assert call(B=0) == SHAPE
    assert call(W=0) == SHAPE
    assert call(W=33) == UNSUP
    assert call(V=0) == SHAPE
    assert call(V=1 << 31) == SHAPE
    assert call(eos=1000) == SHAPE
    assert call(eos=-2) == SHAPE
    assert call(eos=-1) == SHAPE                   # finished needs an end token
    assert call(dtype=9) == UNSUP
    assert call(lg=P(0) + 8) == MISAL
    assert call(tok=P(5) + 2) == MISAL
    assert call(ns=P(1)) == ALIAS
    assert call(tok=P(6)) == ALIAS
    assert call(ws=P(0)) == ALIAS
    assert lib.gdn_beam_workspace_size(2, 4, 1000, BF16) > 0
    assert lib.gdn_beam_workspace_size(2, 33, 1000, BF16) == 0
    assert lib.gdn_beam_workspace_size(0, 4, 1000, BF16) == 0


def test_gather_validation(lib):
    def call(src=P(0), n=8, idx=P(1), dst=P(2), rows=4, rb=4096):
        return lib.gdn_gather_states(src, n, idx, dst, rows, rb, None)
    assert call(src=None) == NULLP
    assert call(idx=None) == NULLP
    assert call(dst=None) == NULLP
    assert call(n=-1) == SHAPE
    assert call(rows=-1) == SHAPE
    assert call(rb=24) == UNSUP
    assert call(src=P(0) + 8) == MISAL
    assert call(idx=P(1) + 1) == MISAL
    assert call(dst=P(0) + 16) == ALIAS
    assert call(idx=P(2) + 64) == ALIAS
    assert call(rows=1 << 40, rb=1 << 40) == SHAPE


def test_valid_calls_without_a_device(lib):
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is present; this checks the no-device path only")
    assert scan(lib) == HIPERR
    assert packed(lib) == HIPERR
    assert back(lib) == HIPERR
    assert lib.gdn_scan_workspace_size(1, 4096, 64, BF16, 0) == 0


def test_binding_refuses_bad_tensors():
    import gated_deltanet_token_amd as g
    x = torch.zeros(2, 5, 8)
    with pytest.raises(ValueError):                # host tensors
        g.gdn_scan_prefill(x, x, x)
    with pytest.raises(TypeError):
        g.gdn_scan_prefill(x.half(), x, x)
    with pytest.raises(ValueError):
        g.gdn_scan_prefill(x[0], x, x)
    with pytest.raises(ValueError):                # strided
        g.gdn_scan_prefill(x.transpose(0, 1), x, x)
    with pytest.raises(ValueError):
        g.gdn_scan_prefill(x, x[:1], x)
    with pytest.raises(TypeError):
        g.gdn_scan_prefill(x, x.bfloat16(), x)
    with pytest.raises(ValueError):
        g.gdn_scan_prefill(x, x, x, torch.zeros(3, 8))
    with pytest.raises(ValueError):
        g.gdn_scan_prefill(x, x, x, prefix_states=torch.zeros(0, 8))
    with pytest.raises(ValueError):                # tied gates take no dbeta
        g.gdn_scan_backward(x, x, x, None, dbeta=x)
    long = torch.zeros(1, 200, 8)
    with pytest.raises(ValueError):                # prefix states needed
        g.gdn_scan_backward(long, long, long, long)
    with pytest.raises(ValueError):
        g.gdn_rms_norm(x, torch.zeros(7))
    with pytest.raises(ValueError):
        g.gdn_rms_norm(x, torch.zeros(8), group=32)
    with pytest.raises(ValueError):
        g.gdn_rms_norm(x, torch.zeros(8), residual_out=x)
    with pytest.raises(ValueError):
        g.gdn_beam_select(x, torch.zeros(2, 4))
    with pytest.raises(ValueError):
        g.gdn_beam_select(x, torch.zeros(2, 5), finished=torch.zeros(2, 5, dtype=torch.uint8))
    with pytest.raises(TypeError):
        g.gdn_gather_states(x, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        g.gdn_gather_states(x, torch.zeros(2, dtype=torch.int32))


def test_binding_refuses_what_32_bits_do_not_hold():
    """ctypes drops the upper bits of an integer: a prefix interval of 2^32 + 1 would ask for no
    rows here and write every 64 tokens in the library."""
    import gated_deltanet_token_amd as g
    wrap = 2 ** 32
    x = torch.zeros(1, 200, 8)
    none = torch.zeros(0, 8)
    for kw in ({"prefix_states": none, "prefix_interval": wrap + 1}, {"flags": wrap},
               {"flags": -1}):
        with pytest.raises(ValueError, match="out of range"):
            g.gdn_scan_prefill(x, x, x, **kw)
        with pytest.raises(ValueError, match="out of range"):
            g.gdn_scan_backward(x, x, x, x, **kw)
    cu = torch.tensor([0, 200], dtype=torch.int32)
    with pytest.raises(ValueError, match="out of range"):
        g.gdn_scan_varlen_prefill(x[0], x[0], x[0], cu, prefix_states=torch.zeros(1, 8),
                                  prefix_interval=wrap + 1)
    e = torch.zeros(1, 0, wrap + 8)
    with pytest.raises(ValueError, match="out of range"):
        g.gdn_scan_prefill(e, e, e)
    with pytest.raises(ValueError, match="out of range"):
        g.gdn_rms_norm(e, torch.zeros(8))
    slots = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="out of range"):
        g.gdn_scan_decode(x, x, x, torch.zeros(2, 8), slots, slots, flags=wrap)
    with pytest.raises(ValueError, match="out of range"):
        g.gdn_scan_decode(e, e, e, torch.zeros(0, wrap + 8), slots, slots)
    with pytest.raises(ValueError, match="out of range"):
        g.gdn_beam_select(x, torch.zeros(1, 200), eos=wrap + 3)
    assert g.gdn_scan_workspace_size(wrap + 1, 4096, 64, torch.float32, False) == 0
    assert g.gdn_scan_workspace_size(1, 4096, wrap + 64, torch.float32, False) == 0
    q, ab = torch.zeros(1, 200, 1, 64), torch.zeros(1, 200, 1)
    pre = torch.zeros(0, 1, 64, 64)
    with pytest.raises(ValueError, match="out of range"):
        g.gdn_prefill_chunked(q, q, q, ab, ab, prefix_states=pre, prefix_interval=wrap + 1)
    with pytest.raises(ValueError, match="out of range"):
        g.gdn_varlen_prefill(q[0], q[0], q[0], ab[0], ab[0], cu, prefix_states=pre[:0].new_zeros(
            1, 1, 64, 64), prefix_interval=wrap + 1)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64])
def test_refused_types_are_named(dtype):
    """By what they are, not by the mixer's arguments."""
    import gated_deltanet_token_amd as g
    x = torch.zeros(1, 4, 8, dtype=dtype)
    for call in (lambda: g.gdn_scan_prefill(x, x, x), lambda: g.gdn_rms_norm(x, x[0, 0]),
                 lambda: g.gdn_beam_select(x, torch.zeros(1, 4))):
        with pytest.raises(TypeError, match=str(dtype)) as e:
            call()
        assert "q, k, v" not in str(e.value)
