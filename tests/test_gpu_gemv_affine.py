"""Matrix-vector products with affine 4-bit weights against 64 bits.

Tolerance of one sum y = sum_g S sum x (128 + u) + (B - 128 S) sum x: the inner sums run over g elements (any order: g + 4 roundings of 2^-24 of the
sum of magnitudes, scales' products included), the outer one over K / g groups in each of eight runs, two terms a group, of which each is at most
its group's sum of magnitudes: another 2^-24 of that for each group's own two additions, and the running sum's own size, below the sum of
|y|'s parts, K / g times.  The result is rounded to bf16 once, 2^-8.  With a residual that is one addition more; silu(gate) up carries its factors'
errors: |d silu| <= 1.1 |d gate|, and 2^-20 for the exponential and the division.
"""
import numpy as np
import pytest
import torch

import binary_bit_gemm_amd as lb

pytestmark = pytest.mark.gpu


def make(M, rows, K, g, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=gen).bfloat16().cuda()
    levels = torch.randint(0, 16, (rows, K), generator=gen, dtype=torch.uint8).cuda()
    words, bad = lb.pack_u4(levels)
    assert bad == 0
    s = ((torch.rand(rows, K // g, generator=gen) + 0.5) * 0.02).half().cuda()
    b = (torch.randn(rows, K // g, generator=gen) * 0.1).half().cuda()
    return x, levels, words, s, b


def products(x, levels, s, b, g):
    """(X W^T, a bound of its error) in 64 bits."""
    xd, u = x.double().cpu().numpy(), levels.cpu().numpy().astype(np.float64)
    sd, bd = (np.repeat(t.double().cpu().numpy(), g, 1) for t in (s, b))
    y = xd @ (sd * u + bd).T
    size = np.abs(xd) @ (np.abs(sd) * (u + 256) + np.abs(bd)).T
    parts = np.zeros_like(y)
    for j in range(0, u.shape[1], g):
        parts += np.abs(xd[:, j:j + g] @ (sd * u + bd)[:, j:j + g].T)
    return y, 2.0 ** -24 * ((g + 8) * size + u.shape[1] / g * parts)


def check(got, want, bound):
    got = got.double().cpu().numpy()
    off = np.abs(got - want) - (bound + 2.0 ** -8 * (np.abs(want) + bound))
    assert np.isfinite(got).all() and off.max(initial=-1) <= 0, f"over its bound by {off.max()}"


SHAPES = [(1, 16, 64, 64), (1, 48, 128, 64), (2, 16, 192, 64), (3, 256, 640, 128), (16, 64, 1088, 64), (5, 160, 2560, 64), (1, 320, 4096, 128),
          (11, 32, 9728, 64), (16, 16, 128, 128), (7, 2560, 320, 64), (1, 16, 16384, 64)]


@pytest.mark.parametrize("M,N,K,g", SHAPES)
def test_plain_and_residual(M, N, K, g):
    x, levels, w, s, b = make(M, N, K, g)
    y, bound = products(x, levels, s, b, g)
    check(lb.gemv_affine(x, w, s, b, g), y, bound)
    r = torch.randn(M, N, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    want = y + r.double().cpu().numpy()
    out = r.clone()
    check(lb.gemv_affine(x, w, s, b, g, residual=r), want, bound + 2.0 ** -24 * np.abs(want))
    assert lb.gemv_affine(x, w, s, b, g, residual=out, out=out) is out  # in place
    check(out, want, bound + 2.0 ** -24 * np.abs(want))


@pytest.mark.parametrize("M,N,K,g", SHAPES)
def test_swiglu(M, N, K, g):
    x, levels, w, s, b = make(M, 2 * N, K, g, seed=1)
    y, bound = products(x, levels, s, b, g)
    gate, up, eg, eu = y[:, :N], y[:, N:], bound[:, :N], bound[:, N:]
    silu = gate / (1 + np.exp(-gate))
    want = silu * up
    off = np.abs(up) * 1.1 * eg + np.abs(silu) * eu + 1.1 * eg * eu + 2.0 ** -20 * np.abs(want)
    check(lb.gemv_affine(x, w, s, b, g, swiglu=True), want, off)


def test_matches_gemm_affine_on_exact_values():
    """Small whole numbers: every sum is exact, so the results are the same to the bit."""
    gen = torch.Generator().manual_seed(4)
    for M, N, K, g in ((1, 64, 512, 64), (16, 128, 256, 128)):
        x = torch.randint(-3, 4, (M, K), generator=gen).bfloat16().cuda()
        levels = torch.randint(0, 16, (N, K), generator=gen, dtype=torch.uint8).cuda()
        w, _ = lb.pack_u4(levels)
        s = torch.randint(1, 3, (N, K // g), generator=gen).half().cuda()
        b = torch.randint(-9, 10, (N, K // g), generator=gen).half().cuda()
        assert torch.equal(lb.gemv_affine(x, w, s, b, g), lb.gemm_affine(x, w, s, b, g))


def test_no_rows_and_no_elements():
    x, _, w, s, b = make(1, 32, 128, 64)
    assert lb.gemv_affine(x[:0], w, s, b, 64).shape == (0, 32)
    none = torch.empty(2, 0, dtype=torch.bfloat16, device="cuda")
    e = torch.empty(32, 0, dtype=torch.float16, device="cuda")
    r = torch.randn(2, 32).bfloat16().cuda()
    assert (lb.gemv_affine(none, w[:, :0].contiguous(), e, e, 64) == 0).all()
    assert torch.equal(lb.gemv_affine(none, w[:, :0].contiguous(), e, e, 64, residual=r), r)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,N,K,g", [(3, 48, 192, 64), (16, 32, 64, 64), (5, 32, 1088, 64), (9, 64, 256, 128), (1, 32, 320, 64)])
def test_infinities_and_nan_stay_in_their_row_and_column(M, N, K, g, swiglu):
    """A NaN in a row of X reaches that row of Y, one in a weight row's last scale that column: a K that ends inside a step, whose
    reads go past the row, included."""
    x, levels, w, s, b = make(M, 2 * N if swiglu else N, K, g, seed=2)
    clean = lb.gemv_affine(x, w, s, b, g, swiglu=swiglu)
    x[M - 1, K - 1] = float("nan")
    s[N - 2, -1] = float("inf")
    b[5, 0] = float("nan")
    s[7, 0] = float("nan")
    got = lb.gemv_affine(x, w, s, b, g, swiglu=swiglu)
    rows, cols = torch.ones(M, dtype=torch.bool), torch.ones(N, dtype=torch.bool)
    rows[M - 1] = False
    cols[[5, 7, N - 2]] = False
    assert torch.equal(got[rows.cuda()][:, cols.cuda()], clean[rows.cuda()][:, cols.cuda()])
    assert got[M - 1].isnan().all() and got[:, [5, 7]].isnan().all() and not got[:, N - 2].isfinite().any()


def test_captured_and_on_another_stream():
    """A graph of gate, up and down products replayed with new inputs and eager work between, and the same on a stream of one's own."""
    M, K, N, g = 3, 256, 320, 64
    x, _, w1, s1, b1 = make(M, 2 * N, K, g, seed=3)
    _, _, w2, s2, b2 = make(1, K, N, g, seed=4)
    step = lambda x: lb.gemv_affine(lb.gemv_affine(x, w1, s1, b1, g, swiglu=True), w2, s2, b2, g, residual=x)  # noqa: E731
    step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x)
    stream = torch.cuda.Stream()
    for i in range(4):
        x.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(20 + i)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step(x))
        with torch.cuda.stream(stream):
            stream.wait_stream(torch.cuda.default_stream())
            other = step(x)
        torch.cuda.synchronize()
        assert torch.equal(other, out)


@pytest.mark.parametrize("M,swiglu,residual", [(1, False, False), (7, True, False), (16, False, True)])
def test_launch_log(M, swiglu, residual, capfd, monkeypatch):
    x, _, w, s, b = make(M, 96 if swiglu else 48, 256, 64)
    r = torch.zeros(M, 48, dtype=torch.bfloat16, device="cuda") if residual else None
    monkeypatch.setenv("LOWBIT_TRACE", "1")
    capfd.readouterr()
    lb.gemv_affine(x, w, s, b, 64, swiglu=swiglu, residual=r)
    torch.cuda.synchronize()
    lines = [t for t in capfd.readouterr().err.splitlines() if t.startswith("lowbit: gemv_affine ")]
    assert len(lines) == 1 and f"problem={M}x48x256" in lines[0] and lines[0].endswith("swiglu" if swiglu else "residual" if residual else "x256")


def test_launch_log_names_both_forms(capfd, monkeypatch):
    x, _, w, s, b = make(2, 96, 256, 64)
    r = torch.zeros(2, 48, dtype=torch.bfloat16, device="cuda")
    monkeypatch.setenv("LOWBIT_TRACE", "1")
    capfd.readouterr()
    lb.gemv_affine(x, w, s, b, 64, swiglu=True, residual=r)
    torch.cuda.synchronize()
    lines = [t for t in capfd.readouterr().err.splitlines() if t.startswith("lowbit: gemv_affine ")]
    assert len(lines) == 1 and lines[0].endswith("problem=2x48x256 swiglu residual")


@pytest.mark.parametrize("M,N,K,g", SHAPES)
def test_swiglu_and_a_residual_together(M, N, K, g):
    x, levels, w, s, b = make(M, 2 * N, K, g, seed=5)
    y, bound = products(x, levels, s, b, g)
    gate, up, eg, eu = y[:, :N], y[:, N:], bound[:, :N], bound[:, N:]
    silu = gate / (1 + np.exp(-gate))
    r = (torch.randn(M, N, generator=torch.Generator().manual_seed(10)) * 3).bfloat16().cuda()
    want = silu * up + r.double().cpu().numpy()
    off = np.abs(up) * 1.1 * eg + np.abs(silu) * eu + 1.1 * eg * eu + 2.0 ** -20 * np.abs(silu * up) + 2.0 ** -24 * np.abs(want)
    got = lb.gemv_affine(x, w, s, b, g, residual=r, swiglu=True)
    check(got, want, off)
    out = r.clone()
    assert lb.gemv_affine(x, w, s, b, g, residual=out, swiglu=True, out=out) is out  # in place
    assert torch.equal(out, got)


@pytest.mark.parametrize("M,N,K,g", [(1, 32, 320, 64), (3, 48, 256, 128), (11, 16, 2560, 64), (16, 32, 192, 64)])
def test_large_and_infinite_activations(M, N, K, g):
    """Elements up to 2^110 (143 times a group of 128 of them is below 2^125): sums stay finite and right.  An infinite one leaves its row of Y without a
    number, and the other rows as they were to the bit."""
    x, levels, w, s, b = make(M, N, K, g, seed=6)
    clean = lb.gemv_affine(x, w, s, b, g)
    big = (x.float() * 2.0 ** 107).bfloat16()  # exact: a power of two; randn stays below 2^3
    assert float(big.abs().max()) < 2.0 ** 110
    y, bound = products(big, levels, s, b, g)
    check(lb.gemv_affine(big, w, s, b, g), y, bound)
    for value in (float("inf"), -float("inf")):
        odd = x.clone()
        odd[M - 1, K // 2] = value
        got = lb.gemv_affine(odd, w, s, b, g)
        assert torch.equal(got[:M - 1], clean[:M - 1]) and not got[M - 1].isfinite().any()
