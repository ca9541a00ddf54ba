"""Calls of more threads than one dimension of a launch holds (2^32): the launch shapes on the host,
and each kernel against calls on parts of the same data."""
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")
HERE = os.path.dirname(os.path.abspath(__file__))
DEV = "cuda:0"
gpu = pytest.mark.gpu


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_launch_shapes(tmp_path):
    exe = str(tmp_path / "check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", exe, os.path.join(HERE, "grid_check.cpp")],
                   check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and "grids ok" in res.stdout, res.stdout


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_token_amd as g
    g.load_library()
    return g


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def parts_of(n, part):
    return [slice(lo, min(n, lo + part)) for lo in range(0, n, part)]


@gpu
def test_gather_of_many_short_rows(gdn):
    rows = 2 ** 24 + 5  # a workgroup of 256 threads each
    src = torch.randn(1000, 4, generator=gen(1), device=DEV)
    idx = torch.randint(0, 1000, (rows,), generator=gen(2), device=DEV, dtype=torch.int32)
    out = torch.full((rows + 1, 4), 9.0, device=DEV)
    gdn.gdn_gather_states(src, idx, out=out[:rows])
    assert torch.equal(out[:rows], src[idx.long()]) and (out[rows] == 9.0).all()


@gpu
def test_norm_of_many_narrow_rows(gdn):
    rows = 2 ** 29 + 5  # 8 threads each
    x = torch.randn(rows, 1, generator=gen(3), device=DEV, dtype=torch.bfloat16)
    w = torch.full((1,), 1.5, device=DEV, dtype=torch.bfloat16)
    out, _, _, _ = gdn.gdn_rms_norm(x, w)
    for r in parts_of(rows, 2 ** 27):
        assert torch.equal(out[r], gdn.gdn_rms_norm(x[r], w)[0])


@gpu
def test_norm_of_many_wide_rows(gdn):
    rows, D, part = 2 ** 25 + 3, 520, 2 ** 17  # 128 threads each; 35 GB in and out
    base = torch.randn(part, D, generator=gen(4), device=DEV, dtype=torch.bfloat16)
    w = torch.randn(D, generator=gen(5), device=DEV, dtype=torch.bfloat16)
    want = gdn.gdn_rms_norm(base, w)[0]
    x = torch.empty(rows, D, device=DEV, dtype=torch.bfloat16)
    for r in parts_of(rows, part):
        x[r] = base[:r.stop - r.start]
    out, _, _, _ = gdn.gdn_rms_norm(x, w)
    del x
    for r in parts_of(rows, part):
        assert torch.equal(out[r], want[:r.stop - r.start])


@gpu
def test_scan_of_many_short_sequences(gdn):
    B = 2 ** 22 + 9  # a workgroup of 1,024 threads each
    x, a, b, dy = [torch.randn(B, 1, 1, generator=gen(s), device=DEV, dtype=torch.bfloat16)
                   for s in range(6, 10)]
    h0 = torch.randn(B, 1, generator=gen(10), device=DEV)
    dh = torch.randn(B, 1, generator=gen(11), device=DEV)
    run = lambda r: [  # noqa: E731
        *gdn.gdn_scan_prefill(x[r], a[r], b[r], h0[r], flags=2),
        *gdn.gdn_scan_backward(dy[r], x[r], a[r], b[r], h0[r], dfinal=dh[r], flags=2)]
    got = run(slice(0, B))
    for r in parts_of(B, 2 ** 20):
        for p, q in zip(got, run(r)):
            assert torch.equal(p[r], q)


@gpu
def test_decode_of_many_channels(gdn):
    B, D = 2 ** 22 + 1, 1025  # a thread per channel; 8.6 GB a tensor
    x = torch.randn(B, 1, D, generator=gen(12), device=DEV, dtype=torch.bfloat16)
    a = torch.randn(B, 1, D, generator=gen(13), device=DEV, dtype=torch.bfloat16)
    pool = torch.randn(4, D, generator=gen(14), device=DEV)
    src = torch.randint(-1, 4, (B,), generator=gen(15), device=DEV, dtype=torch.int32)
    dst = torch.full_like(src, -1)
    out = gdn.gdn_scan_decode(x, a, None, pool, src, dst, flags=2)
    for r in parts_of(B, 2 ** 19):
        o = gdn.gdn_scan_decode(x[r], a[r], None, pool, src[r].clone(), dst[r].clone(), flags=2)
        assert torch.equal(out[r], o)


@gpu
def test_selection_of_many_items(gdn):
    B, W, V = 2 ** 24 + 3, 1, 2  # a workgroup of 256 threads each, in both kernels
    x = torch.randn(B, W, V, generator=gen(16), device=DEV, dtype=torch.bfloat16)
    s = torch.randn(B, W, generator=gen(17), device=DEV)
    out = gdn.gdn_beam_select(x, s)
    for r in parts_of(B, 2 ** 22):
        for p, q in zip(out[:3], gdn.gdn_beam_select(x[r].clone(), s[r].clone())):
            assert torch.equal(p[r], q)
