"""Low-rank adapters beside a packed GEMM, against the formula in 64 bits (the oracle's dequantised weights).

Tolerance, per element: one rounding to bf16 (8 significant bits: 2^-8 of the result); the packed product's
fp32 sums, groups of g products and then K / g group sums and a few more additions, (g + K / g + 32) * 2^-24 of the sum of magnitudes;
the adapter's term, whose first sum of K products is kept to 16 bits: (K * 2^-24 + 2^-16) of alpha * sum_r
(sum_k |x| |a|) |b|, plus its sum over the rank, 2 rank * 2^-24 of the same.
"""
import numpy as np
import pytest
import torch

import binary_bit_gemm_amd as lb
import oracle
import workloads as W

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, M, N, K, bits, g, rank, adapters, rows, seed=0):
        rng = np.random.default_rng([seed, M, N, K, bits, g, rank, adapters])
        self.bits, self.g, self.K, self.rank = bits, g, K, rank
        inp = W.make_inputs(W.Problem("lora", M, N, K, bits, g, 0, 0), seed=seed)
        self.x = torch.from_numpy(inp.x.view(np.int16)).view(torch.bfloat16).cuda()
        self.words, bad = lb.pack(torch.from_numpy(inp.codes).cuda(), bits)
        assert bad == 0
        self.scales = torch.from_numpy(inp.scales).cuda()
        self.w = oracle.dequant_f64(inp.codes, inp.scales, g)
        self.a = torch.from_numpy(rng.standard_normal((adapters, rank, K)) / np.sqrt(K)).bfloat16().cuda()
        self.b = torch.from_numpy(rng.standard_normal((adapters, N, rank)) * 0.2).bfloat16().cuda()
        self.alpha = torch.from_numpy(rng.uniform(-2, 2, adapters)).float().cuda()
        if rows == "one":
            r = np.full(M, adapters - 1)
        elif rows == "segments":
            r = np.sort(rng.integers(0, adapters, M))
        elif rows == "none":
            r = np.full(M, -1)
        else:  # scattered, some without an adapter, some out of range
            r = rng.integers(-1, adapters + 1, M)
        self.rows = torch.from_numpy(r.astype(np.int32)).cuda()

    def run(self, **kw):
        return lb.gemm_lora(self.x, self.words, self.scales, self.g, self.bits, self.a, self.b, self.alpha, self.rows, **kw)

    def reference(self):
        x = self.x.double().cpu().numpy()
        y, mag = x @ self.w.T, np.abs(x) @ np.abs(self.w).T
        lora = np.zeros_like(y)
        for e in range(self.a.shape[0]):
            m = self.rows.cpu().numpy() == e
            if m.any():
                a, b = self.a[e].double().cpu().numpy(), self.b[e].double().cpu().numpy()
                al = float(self.alpha[e])
                y[m] += al * (x[m] @ a.T) @ b.T
                lora[m] = abs(al) * (np.abs(x[m]) @ np.abs(a).T) @ np.abs(b).T
        bound = (self.g + self.K / self.g + 32) * 2.0 ** -24 * mag + ((self.K + 2 * self.rank) * 2.0 ** -24 + 2.0 ** -16) * lora
        return y, bound

    def check(self, got):
        want, bound = self.reference()
        got = got.double().cpu().numpy()
        assert np.isfinite(got).all()
        off = np.abs(got - want) - (2.0 ** -8 * (np.abs(want) + bound) + bound)
        assert off.max(initial=-1) <= 0, f"worst element over its bound by {off.max()}"


@pytest.mark.parametrize("bits,g", [(2, 64), (2, 128), (1, 64), (1, 128), (4, 64), (4, 128)])
@pytest.mark.parametrize("M,N,K,rank,adapters,rows", [
    (1, 16, 128, 8, 1, "one"), (1, 272, 512, 16, 3, "one"), (16, 256, 256, 16, 16, "scattered"), (15, 1040, 640, 24, 5, "segments"),
    (33, 320, 768, 64, 4, "scattered"), (64, 128, 1024, 128, 2, "segments"), (300, 528, 384, 32, 3, "segments"),
    (97, 192, 192, 40, 7, "scattered"), (130, 512, 1280, 16, 1, "none"), (289, 208, 256, 8, 20, "scattered"),
])
def test_parity(M, N, K, rank, adapters, rows, bits, g):
    if K % g:
        K = K // g * g + g
    c = Case(M, N, K, bits, g, rank, adapters, rows)
    c.check(c.run())


@pytest.mark.parametrize("variant_m", [1025, 1536, 4608])
@pytest.mark.parametrize("rows", ["one", "segments", "scattered"])
def test_large_tiles(variant_m, rows):
    c = Case(variant_m, 2304, 576, 2, 64, 32, 4, rows, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("bits", [1, 2])
@pytest.mark.parametrize("M,N,K", [(1, 9216, 3072), (16, 3072, 9216), (16, 3072, 3072), (9, 512, 12288), (32, 9216, 3072), (20, 1024, 4096)])
def test_skinny(M, N, K, bits):
    """The shapes on which lowbit_gemm runs its skinny kernels."""
    for rows in ("one", "scattered"):
        c = Case(M, N, K, bits, 64, 16, 6, rows, seed=2)
        c.check(c.run())


def test_rows_without_an_adapter_are_the_plain_product():
    c = Case(300, 512, 512, 2, 64, 16, 4, "none", seed=3)
    plain = c.x.double().cpu().numpy() @ c.w.T
    got = c.run().double().cpu().numpy()
    assert (np.abs(got - plain) <= 2.0 ** -8 * np.abs(plain) + 2.0 ** -8).all()
    c.rows[:] = 99
    assert torch.equal(c.run(), c.run()) and np.array_equal(c.run().double().cpu().numpy(), got)


@pytest.mark.parametrize("M", [7, 16, 32, 200, 1100])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_requests_do_not_touch_each_other(M, bad):
    """An adapter and a row that hold no numbers reach their own rows only."""
    c = Case(M, 400, 512, 2, 64, 16, 3, "scattered", seed=4)
    c.rows[0], c.rows[1], c.rows[2] = 1, 0, 2
    want = c.run()
    c.a[1, :, 5] = bad
    c.b[1, 7] = bad
    got = c.run()
    own = c.rows == 1
    assert torch.equal(got[~own], want[~own])
    assert not bool(torch.isfinite(got[own][:, 7]).any())
    c = Case(M, 400, 512, 2, 64, 16, 3, "one", seed=5)
    want = c.run()
    c.x[M // 2, 3] = bad
    got = c.run()
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(got[keep], want[keep]) and not bool(torch.isfinite(got[M // 2]).any())


def test_workspace_content_and_repeats():
    c = Case(70, 512, 1024, 2, 64, 24, 5, "scattered", seed=6)
    want = c.run()
    ws = torch.full((lb.lora_workspace_size(70, 24),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns
    ws[:4096] = 0  # the arrival counters
    for _ in range(3):
        assert torch.equal(c.run(workspace=ws), want) and not bool(ws[:4096].any())
    long = Case(50, 256, 16384, 2, 64, 64, 3, "scattered", seed=6)  # K split across workgroups
    ws = torch.zeros(lb.lora_workspace_size(50, 64), dtype=torch.uint8, device="cuda")
    want = long.run(workspace=ws)
    long.check(want)
    for _ in range(3):
        assert torch.equal(long.run(workspace=ws), want) and not bool(ws[:4096].any())


@pytest.mark.parametrize("M", [12, 30, 150, 700])
def test_many_adapters(M):
    """More adapters than a scalar word has bits, far apart in the table, every row with its own."""
    c = Case(M, 208, 256, 2, 64, 8, 3000, "one", seed=10)
    g = torch.Generator().manual_seed(M)
    c.rows.copy_(torch.randint(-1, 3000, (M,), generator=g, dtype=torch.int32))
    c.check(c.run())


@pytest.mark.parametrize("bits,g", [(2, 64), (1, 128), (4, 64), (4, 128)])
@pytest.mark.parametrize("M,N,K,rows", [(509, 1024, 2048, "segments"), (100, 320, 4096, "scattered"), (64, 128, 1536, "one"), (190, 2048, 1664, "scattered")])
def test_k_split_across_workgroups(M, N, K, rows, bits, g):
    c = Case(M, N, K, bits, g, 16, 5, rows, seed=11)
    n = lb.lora_workspace_size(M, 16, N, K, g, bits)
    assert n > lb.lora_workspace_size(M, 16)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0
    got = c.run(workspace=ws)
    c.check(got)
    for _ in range(2):
        assert torch.equal(c.run(workspace=ws), got) and not bool(ws[:4096].any())
    c.check(c.run())


@pytest.mark.parametrize("bits,g", [(2, 64), (1, 128), (4, 64)])
@pytest.mark.parametrize("rows", ["segments", "scattered"])
def test_many_small_tiles(rows, bits, g):  # 640 tiles of 64 x 128, not split
    c = Case(260, 16384, 512, bits, g, 16, 5, rows, seed=12)
    c.check(c.run())


def test_no_adapters_and_empty_calls():
    c = Case(5, 256, 256, 2, 64, 8, 1, "one", seed=7)
    plain = lb.gemm(c.x, c.words, c.scales, 64, 2)
    none = lb.gemm_lora(c.x, c.words, c.scales, 64, 2, c.a[:0], c.b[:0], c.alpha[:0], c.rows)
    assert torch.equal(none, plain)
    assert lb.gemm_lora(c.x[:0], c.words, c.scales, 64, 2, c.a, c.b, c.alpha, c.rows[:0]).shape == (0, 256)


def test_adapters_past_32_bits():
    """A table of adapters longer than 2^32 bytes, of which the last is used."""
    c = Case(40, 256, 4096, 2, 64, 128, 1, "one", seed=8)
    want = c.run()
    n = (1 << 32) // (128 * 4096 * 2) + 2
    a = torch.empty(n, 128, 4096, dtype=torch.bfloat16, device="cuda")
    b = torch.empty(n, 256, 128, dtype=torch.bfloat16, device="cuda")
    a[-1], b[-1] = c.a[0], c.b[0]
    c.a, c.b, c.alpha = a, b, c.alpha.expand(n).contiguous()
    c.rows[:] = n - 1
    assert torch.equal(c.run(), want)


def test_on_another_stream_and_in_a_graph():
    c = Case(64, 1024, 1024, 2, 64, 16, 4, "scattered", seed=9)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.run()
    s.synchronize()
    assert torch.equal(got, want)
    ws = torch.zeros(lb.lora_workspace_size(64, 16), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    c.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out, workspace=ws)
    for k in range(3):
        c.x.copy_(torch.randn(c.x.shape, generator=torch.Generator().manual_seed(k)).bfloat16())
        want = c.run()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("bits,N,K", [(2, 9216, 3072), (2, 1040, 1024), (1, 3072, 1024)])
@pytest.mark.parametrize("M", [1, 7, 13, 15])
def test_one_request_of_any_length_has_the_same_bits(M, bits, N, K):
    """Fewer rows of one request than a block of 16 go the same way as a whole block: the sums over the rank are taken in the same
    order (an adapter's term far above the packed product shows another order's last bits)."""
    c = Case(16, N, K, bits, 64, 128, 2, "one", seed=13)
    c.b.mul_(64)
    whole = c.run()
    c.check(whole)
    c.x, c.rows = c.x[:M].contiguous(), c.rows[:M].contiguous()
    assert torch.equal(c.run(), whole[:M])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("M,N,K", [(5, 9216, 512), (30, 512, 512), (509, 1024, 1024), (1100, 2304, 512)])
def test_one_request_with_an_adapter_that_holds_no_numbers(M, N, K, bad):
    """Rows past the last of a call whose rows all have such an adapter: the other columns stay as they were."""
    c = Case(M, N, K, 2, 64, 16, 3, "one", seed=14)
    want = c.run()
    c.b[2, 7] = bad
    got = c.run()
    other = torch.arange(N, device="cuda") != 7
    assert torch.equal(got[:, other], want[:, other]) and not bool(torch.isfinite(got[:, 7]).any())


# Several adapters of 16 rows share a workgroup of the first product from about 200 workgroups on.
SHARED = [(1021, 256, 512, 8, 12), (1100, 208, 1280, 8, 40), (520, 256, 320, 8, 16), (3100, 256, 256, 8, 2), (1533, 256, 256, 8, 5),
          (500, 256, 512, 16, 12), (1021, 256, 384, 16, 30)]


@pytest.mark.parametrize("bits,g", [(2, 64), (1, 128), (4, 64)])
@pytest.mark.parametrize("M,N,K,rank,adapters", SHARED)
def test_adapters_that_share_a_workgroup(M, N, K, rank, adapters, bits, g):
    c = Case(M, N, K // g * g, bits, g, rank, adapters, "scattered", seed=15)
    got = c.run()
    c.check(got)
    order = torch.randperm(M, generator=torch.Generator().manual_seed(15)).cuda()  # other neighbours, the same sums
    c.x, c.rows = c.x[order].contiguous(), c.rows[order].contiguous()
    c.check(c.run())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("M,N,K,rank,adapters", SHARED)
def test_adapters_that_share_a_workgroup_do_not_touch_each_other(M, N, K, rank, adapters, bad):
    for e in (0, adapters // 2, adapters - 1):
        c = Case(M, N, K, 2, 64, rank, adapters, "scattered", seed=16)
        c.x[:, 5] = 1  # the bad element takes part in every row's sum
        want = c.run()
        c.a[e, rank // 2, 5] = bad
        c.b[e, :, rank // 2] = 1
        got = c.run()
        own = c.rows == e
        assert bool(own.any()) and torch.equal(got[~own], want[~own])
        assert not bool(torch.isfinite(got[own]).any())


@pytest.mark.parametrize("M", [1, 16, 130])
@pytest.mark.parametrize("N,bits,g", [(18432, 2, 64), (27648, 2, 64), (27648, 1, 128), (18432, 4, 64)])
@pytest.mark.parametrize("rows", ["one", "scattered"])
def test_the_widest_linears(rows, N, bits, g, M):
    c = Case(M, N, 384, bits, g, 16, 5, rows, seed=17)
    c.check(c.run())


def test_a_workspace_that_is_too_small():
    c = Case(70, 512, 1024, 2, 64, 24, 5, "scattered", seed=18)
    for n in (lb.lora_workspace_size(70, 24) - 1, 4096, 0):
        with pytest.raises(lb.LowbitError):
            c.run(workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    # too small to split the product along K: unsplit, as with the least
    c = Case(509, 1024, 2048, 2, 64, 16, 5, "segments", seed=18)
    most, least = lb.lora_workspace_size(509, 16, 1024, 2048, 64, 2), lb.lora_workspace_size(509, 16)
    assert most > least
    want = c.run(workspace=torch.zeros(least, dtype=torch.uint8, device="cuda"))
    ws = torch.zeros(most - 16, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.run(workspace=ws), want)


def test_split_adapters_and_split_attention_take_turns_on_a_workspace():
    c = Case(509, 1024, 2048, 2, 64, 16, 5, "segments", seed=19)      # the product split along K
    few = Case(50, 256, 16384, 2, 64, 64, 3, "scattered", seed=19)    # the first product split along K
    g = torch.Generator().manual_seed(19)
    q = torch.randn(2, 40, 2, 128, generator=g).bfloat16().cuda()
    k, v = (torch.randn(2, 4000, 2, 128, generator=g).bfloat16().cuda() for _ in range(2))
    sizes = [lb.lora_workspace_size(509, 16, 1024, 2048, 64, 2), lb.lora_workspace_size(50, 64, 256, 16384, 64, 2),
             lb.attention_workspace_size(q, k, v), lb.attention_workspace_size(q[:, :1], k, v)]
    assert sizes[0] > lb.lora_workspace_size(509, 16) and min(sizes) > 4096
    calls = [lambda ws: c.run(workspace=ws), lambda ws: lb.attention(q, k, v, workspace=ws), lambda ws: few.run(workspace=ws),
             lambda ws: lb.attention(q[:, :1], k, v, workspace=ws)]
    alone = [f(torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")) for f in calls]
    c.check(alone[0])
    few.check(alone[2])
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    for turn in ((0, 1, 2, 3), (3, 2, 1, 0), (1, 0, 3, 2), (2, 0, 1, 1)):
        for i in turn:
            assert torch.equal(calls[i](ws), alone[i]) and not bool(ws[:4096].any())
