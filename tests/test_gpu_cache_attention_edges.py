"""Attention over the paged cache where it can go wrong: what is in slots that a row does not take, lengths and tables out of
range, rows left alone, strides, caches past 4 GiB, ranges of values, and calls that share a device, a workspace or a graph.

Tolerances are those of the formula's test (test_gpu_cache_attention.py)."""
import math

import numpy as np
import pytest
import torch

import binary_bit_gemm_amd as lb
from tests import cache_reference as R
from tests.test_gpu_cache_attention import Problem, kernel, random_tree  # noqa: F401 (kernel: a fixture)

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
def test_nan_in_a_drafted_token_reaches_its_descendants_alone(dim, bits, kernel):
    """Tokens 3 (NaN in its key) and 7 (in its value) of a tree: rows that take one are NaN (values: where the format has it), all others are as if
    the two held zeros."""
    nodes, n = 20, 73
    tree = random_tree(nodes, 5)
    tree[9] = tree[3] | 1 << 9
    tree[11] = tree[7] | 1 << 11
    p = Problem([n], [nodes], 4, 2, dim, bits, 16, tree=[tree], seed=11)
    base = n - nodes
    p.k[0][base + 3, :, 5] = NAN
    p.v[0][base + 7, :, dim - 3] = NAN
    p.write()
    got = p.call()
    p.k[0][base + 3], p.v[0][base + 7] = 0, 0
    has = np.array([[(t >> j) & 1 for j in (3, 7)] for t in tree], bool)
    assert has.any(0).all() and not has.any(1).all()
    p.check(got, rows=lambda b: ~has.any(1))
    key = torch.from_numpy(has[:, 0]).cuda()
    value = torch.from_numpy(~has[:, 0] & has[:, 1]).cuda()
    assert got[0, key].isnan().all()
    hit = {16: slice(dim - 3, dim - 2), 8: slice(0, dim), 4: slice(dim - 64, dim)}[bits]
    assert got[0, value][..., hit].isnan().all()
    rest = torch.ones(dim, dtype=torch.bool)
    rest[hit] = False
    assert got[0, value][..., rest.cuda()].isfinite().all()


@pytest.mark.parametrize("dim", [64, 128])
def test_infinities_in_values_of_16_bits(dim, kernel):
    """An infinite value reaches its column in the rows that take it, with its sign; both signs make a NaN."""
    n, new = 50, 6
    p = Problem([n], [new], 2, 1, dim, 16, 16, seed=12)
    p.v[0][n - 4, 0, 9] = INF       # tokens 2 .. 5 take it
    p.v[0][n - 2, 0, 9] = -INF      # tokens 4 and 5
    p.v[0][n - 1, 0, 1] = -INF      # token 5
    p.write()
    got = p.call().float()
    assert got[0, :2].isfinite().all()
    assert (got[0, 2:4, :, 9] == INF).all() and got[0, 4:, :, 9].isnan().all() and (got[0, 5, :, 1] == -INF).all()
    others = [c for c in range(dim) if c not in (1, 9)]
    assert got[..., others].isfinite().all()


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_lengths_out_of_range(bits, kernel):
    """More keys than kv_len count as kv_len, fewer than none as none; more new tokens than q_len as q_len."""
    p = Problem([40, 64, 64], [3, 3, 3], 4, 2, 64, bits, 16, seed=13)
    out = torch.full_like(p.q, 5.0)
    got = lb.cache_attention(p.q, p.cache, p.table, ints([-7, 1000, 2 ** 31 - 1]), q_lens=ints([2, 100, -3]), out=out)
    p.lens, p.q_lens = [0, 64, 0], [2, 3, 0]
    p.k[0], p.v[0], p.k[2], p.v[2] = (x[:0] for x in (p.k[0], p.v[0], p.k[2], p.v[2]))
    p.check(got)
    assert (got[0, :2] == 0).all() and (got[0, 2] == 5).all() and (got[2] == 5).all()


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
def test_entries_outside_the_cache(dim, bits, tree, kernel):
    """Keys of a page that the table puts outside the cache are left out, whole pages or all of them (zeros), and where a page ends inside a tile."""
    page, new = 16, 4
    lens = [150, 150, 40]
    p = Problem(lens, [new] * 3, 4, 2, dim, bits, page, seed=14, tree=[[1, 3, 5, 9]] * 3 if tree else None)
    bad = {0: [0, 3, 8], 1: [9], 2: [0, 1, 2]}
    for b, pages in bad.items():
        for i, at in enumerate(pages):
            p.table[b, at] = (-1, p.cache.k.shape[0], 2 ** 31 - 1)[i % 3]
    got = R.bf16(p.call())
    none = R.bf16(p.call(workspace=None))
    for b in range(3):
        takes = R.taken(lens[b], new, new, p.tree[b] if tree else None)
        for at in bad[b]:
            takes[:, at * page:(at + 1) * page] = False
        for h in range(4):
            k, v = (R.stands_for(R.bf16(x[b][:, h // 2]), bits) for x in (p.k, p.v))
            q = R.bf16(p.q[b, :, h])
            want, mag, _ = R.attend(q, k, v, takes, 1 / math.sqrt(dim))
            for g in (got, none):
                # 2^-7 of the magnitudes covers the roundings of p (2^-8) and of O (2^-8); codes' offsets add 2^-9 of the range (8 bits)
                assert (np.abs(g[b, :, h] - want) <= 2.0 ** -7 * mag + (2.0 ** -9 * np.abs(v).max(initial=0) * takes.any(1)[:, None])).all()
            if b == 2:
                assert (got[b] == 0).all()


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
def test_strides_and_rows_left_alone(dim, bits, kernel):
    """q out of a fused projection, o in another order with room around it: only the rows asked for are written."""
    p = Problem([90, 7], [5, 2], 6, 2, dim, bits, 32, seed=15)
    qkv = torch.full((2, 5, 10, dim), NAN, dtype=torch.bfloat16, device="cuda")
    qkv[:, :, 1:7] = p.q
    plain = p.call()
    p.q = qkv[:, :, 1:7]
    room = torch.full((8, 2, 7, dim + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    out = room[1:7, :, 1:6, :dim].permute(1, 2, 0, 3)
    assert out.shape == p.q.shape and out.stride(-1) == 1
    p.call(out=out)
    assert torch.equal(out[0], plain[0]) and torch.equal(out[1, :2], plain[1, :2])
    p.check(plain)
    assert (out[1, 2:] == 3).all()
    assert (room[0] == 3).all() and (room[7] == 3).all() and (room[:, :, 0] == 3).all() and (room[:, :, 6] == 3).all() and (room[..., dim:] == 3).all()


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_pages_past_4_gib(bits, kernel):
    """A cache whose codes take more than 4 GiB, a request in its last pages and one in its first."""
    page, dim, heads = 256, 128, 4
    pages = (1 << 32) // (page * dim * heads * bits // 8) + 40
    p = Problem([700, 700], [3, 3], 8, heads, dim, bits, page, seed=16)
    small = p.cache
    p.cache = lb.kv_cache(pages, heads, dim, bits, page)
    p.table = torch.stack([torch.arange(pages - 1, pages - 4, -1), torch.arange(3)]).to(torch.int32).cuda()
    p.write()
    got = p.call()
    p.check(got)
    at = torch.arange(700)
    slots = (p.table[0].cpu()[at // page].long() * page + at % page).to(torch.int32).cuda()
    back = lb.cache_read(p.cache, slots)
    lb.cache_write(small, p.k[0].cuda(), p.v[0].cuda(), torch.arange(700, dtype=torch.int32, device="cuda"))
    same = lb.cache_read(small, torch.arange(700, dtype=torch.int32, device="cuda"))
    assert torch.equal(back[0], same[0]) and torch.equal(back[1], same[1])


@pytest.mark.parametrize("scale_k,scale_v,q_scale", [(30.0, 1.0, 1.0), (1.0, 2.0 ** -40, 1.0), (1.0, 2.0 ** 25, 1.0), (2.0 ** 60, 1.0, 2.0 ** -60),
                                                     (2.0 ** -70, 1.0, 2.0 ** 68)])
@pytest.mark.parametrize("bits", [4, 8, 16])
def test_ranges_of_values(scale_k, scale_v, q_scale, bits, kernel):
    p = Problem([400], [5], 4, 2, 128, bits, 64, seed=17, scale_k=scale_k, scale_v=scale_v)
    p.q = (p.q.float() * q_scale).bfloat16()
    p.check(p.call())


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_scores_that_rise_and_fall(bits, kernel):
    """Key by key larger scores, values by 2^20 apart from token to token and zeros among them: the row's exponent moves often, up from nothing and by
    steps of any size."""
    n, dim = 900, 128
    for seed, slope in ((18, 80.0), (19, -80.0)):
        p = Problem([n], [2], 2, 1, dim, bits, 64, seed=seed)
        u = torch.nn.functional.normalize(p.q[0, 0, 0].float().cpu(), dim=0)
        ramp = torch.linspace(-slope, slope, n)
        p.k[0] = (ramp[:, None, None] * u + 0.1 * p.k[0].float()).bfloat16()
        step = 2.0 ** (-20.0 * (torch.arange(n) % 2)) * (torch.arange(n) % 5 != 3)
        p.v[0] = (p.v[0].float() * step[:, None, None]).bfloat16()
        p.write()
        p.check(p.call())


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_values_all_zero_or_constant(bits, kernel):
    """Scales of zero everywhere: zeros stay zeros, and constant rows (4 bits: b alone) come back."""
    p = Problem([333], [3], 4, 2, 64, bits, 16, seed=20, scale_v=0.0)
    assert (p.call() == 0).all()
    p.v[0][:] = 0.75
    p.write()
    got = p.call().float()
    # 8 bits: scale up(0.75 / 127), code 127 or so: half a code; O's own rounding
    assert (got - 0.75).abs().max() <= 0.75 * (2.0 ** -8 + (0.5 / 127 if bits == 8 else 0)) + 2.0 ** -11


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_many_requests_of_all_lengths(bits, kernel):
    lens = [1, 0, 4000, 17, 2, 350, 16, 31, 33, 1000, 64, 5]
    p = Problem(lens, [1] * len(lens), 4, 1, 64, bits, 32, seed=21)
    got = p.call()
    p.check(got)
    assert (got[1] == 0).all()


def test_pages_shared_between_and_within_requests(kernel):
    """Two requests with a common prefix in the same pages, and a table that names a page twice."""
    p = Problem([128, 128], [4, 4], 4, 2, 128, 8, 32, seed=22)
    p.table[1, :2] = p.table[0, :2]
    for x in (p.k, p.v):
        x[1][:64] = x[0][:64]
    p.check(p.call())
    p.answers.clear()
    p.table[0, 1] = p.table[0, 0]
    for x in (p.k, p.v):
        x[0][32:64] = x[0][:32]
        x[1][32:64] = x[1][32:64]
    p.check(p.call(), rows=lambda b: np.full(4, b == 0))


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_the_same_every_time(bits, kernel):
    p = Problem([3000, 1700], [7, 7], 8, 2, 128, bits, 64, seed=23)
    first = p.call()
    for _ in range(5):
        assert torch.equal(p.call(), first)


def test_two_streams_with_a_workspace_each(kernel):
    a = Problem([5000], [1], 8, 2, 128, 4, 64, seed=24)
    b = Problem([5000], [1], 8, 2, 128, 8, 64, seed=25)
    want = a.call(), b.call()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.zeros(lb.cache_attention_workspace_size(p.q, p.cache, 5000) + 16, dtype=torch.uint8, device="cuda") for p in (a, b)]
    lens = ints([5000])
    outs = [torch.empty_like(p.q) for p in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s, w, o in zip((a, b), streams, ws, outs):
            with torch.cuda.stream(s):
                lb.cache_attention(p.q, p.cache, p.table, lens, out=o, workspace=w)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_captured_and_replayed_with_new_lengths(kernel):
    """A graph of write and attention, replayed with eager work between, sees the tensors' contents of each replay; a second graph shares the
    workspace."""
    page, dim, heads = 64, 128, 2
    p = Problem([2100, 900], [1, 1], 8, heads, dim, 4, page, seed=26, kv_len=2200)
    ws = torch.zeros(lb.cache_attention_workspace_size(p.q, p.cache, 2200) + 16, dtype=torch.uint8, device="cuda")
    lens, slots = ints([2101, 901]), ints([0, 0])
    k, v = (torch.zeros(2, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    outs = [torch.zeros_like(p.q) for _ in range(2)]

    def step(out):
        lb.cache_write(p.cache, k, v, slots)
        lb.cache_attention(p.q, p.cache, p.table, lens, kv_len=2200, out=out, workspace=ws)

    graphs = []
    slots.fill_(-1)
    step(outs[0])
    torch.cuda.synchronize()
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(o)
        graphs.append(g)
    gen = torch.Generator().manual_seed(27)
    for i in range(6):
        new = [torch.randn(2, heads, dim, generator=gen).bfloat16() for _ in range(2)]
        for b in range(2):
            at = p.lens[b] + i
            slots[b] = int(p.table[b, at // page]) * page + at % page
            lens[b] = at + 1
        k.copy_(new[0])
        v.copy_(new[1])
        p.q.copy_(torch.randn(p.q.shape, generator=gen).bfloat16())
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for b in range(2):
            p.k[b], p.v[b] = torch.cat([p.k[b], new[0][b:b + 1]]), torch.cat([p.v[b], new[1][b:b + 1]])
        p.answers.clear()
        lens_then, p.lens = p.lens, [n + i + 1 for n in p.lens]
        p.check(outs[i % 2])
        eager = torch.empty_like(p.q)
        lb.cache_attention(p.q, p.cache, p.table, lens, kv_len=2200, out=eager, workspace=ws)
        assert torch.equal(eager, outs[i % 2])
        p.lens = lens_then
    assert (ws[:4096] == 0).all()


def test_a_workspace_too_small_is_not_used(kernel):
    p = Problem([3000], [1], 8, 2, 64, 8, 64, seed=28)
    n = lb.cache_attention_workspace_size(p.q, p.cache, 3000)
    lens = ints([3000])
    want = p.call(workspace=None)
    for size in (16, 4096, max(n - 16, 32)):
        ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
        if size < n:
            got = lb.cache_attention(p.q, p.cache, p.table, lens, workspace=ws)
            assert torch.equal(got, want) and (ws == 0x5A).all()


@pytest.mark.parametrize("rows,keys,force,line", [
    (1, 300, None, "few rows=16 splits=1 "), (1, 5000, None, "few rows=16 splits="), (5, 100, None, "few rows=16 splits=1 "),
    (16, 500, None, "few rows=16 splits="), (5, 2000, None, "many rows=32 splits="), (16, 2000, None, "many rows=64 splits="), (64, 4000, None, "many rows="), (2, 100, "many128", "many rows=128 splits="), (40, 100, "few", "few rows=16 "),
])
def test_launch_log(rows, keys, force, line, capfd, monkeypatch):
    if force:
        monkeypatch.setenv("LOWBIT_CACHE_ATTENTION", force)
    p = Problem([keys], [rows], 8, 2, 64, 8, 64, seed=29)
    monkeypatch.setenv("LOWBIT_TRACE", "1")
    capfd.readouterr()
    p.call()
    torch.cuda.synchronize()
    lines = [x for x in capfd.readouterr().err.splitlines() if x.startswith("lowbit: cache_attention ")]
    assert len(lines) == 1 and line in lines[0], lines
    assert f"problem=1x{rows}x{keys}x8 kv_heads=2 dim=64 bits=8" in lines[0]


def test_refusals_of_the_binding():
    p = Problem([100], [2], 4, 2, 64, 8, 16, seed=30)
    lens = ints([100])
    call = lambda q=p.q, cache=p.cache, table=p.table, n=lens, **kw: lb.cache_attention(q, cache, table, n, **kw)  # noqa: E731
    call()
    for bad in (dict(q=p.q.float()), dict(q=p.q[0]), dict(q=p.q[..., :32]), dict(q=p.q[:, :, :3]), dict(table=p.table.long()), dict(table=p.table[:0]),
                dict(n=lens.long()), dict(n=ints([1, 2])), dict(q_lens=ints([1, 1])), dict(kv_len=1000), dict(kv_len=-1), dict(out=torch.empty_like(p.q).float()),
                dict(out=torch.empty(1, 2, 4, 32, dtype=torch.bfloat16, device="cuda")), dict(tree=ints([[1, 3]])), dict(out=p.q.cpu()), dict(table=p.table.cpu()),
                dict(q=p.q.transpose(2, 3).contiguous().transpose(2, 3)), dict(tree=torch.ones(1, 3, dtype=torch.int64, device="cuda"))):
        with pytest.raises((TypeError, ValueError, lb.LowbitError)):
            call(**bad)
    long = torch.zeros(1, 65, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lb.LowbitError):
        lb.cache_attention(long, p.cache, p.table, lens, tree=torch.ones(1, 65, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
def test_nan_and_infinities_in_queries_stay_in_their_row(dim, bits, kernel):
    p = Problem([150], [6], 4, 2, dim, bits, 16, seed=31)
    whole = p.q.clone()
    p.q[0, 1, 2, 3] = NAN
    p.q[0, 4, 0, 0] = INF
    got = p.call()
    assert got[0, 1, 2].isnan().all() and not got[0, 4, 0].isfinite().any()
    got[0, 1, 2], got[0, 4, 0] = 0, 0
    p.q = whole
    clean = p.call()
    p.check(clean)
    clean[0, 1, 2], clean[0, 4, 0] = 0, 0
    for b, h in [(0, h) for h in range(4)]:
        bound = torch.from_numpy(p.wanted(1 / math.sqrt(dim))[b, h][1]).cuda()
        assert ((got[b, :, h].double() - clean[b, :, h].double()).abs() <= 2 * bound).all()  # both lie within their bounds of the formula


@pytest.mark.parametrize("dim", [64, 128])
def test_one_key_gives_its_value_back_at_16_bits(dim, kernel):
    """Probabilities are divided by the sum of what they were rounded to: a row with one key, or with one whose score is past the others' by more than
    fp32's range, has p v / p, two fp32 roundings away from the bf16 v, and so v itself."""
    p = Problem([1, 1, 33, 2500], [1, 1, 1, 1], 8, 2, dim, 16, 16, seed=32)
    at = {0: 0, 1: 0, 2: 20, 3: 1777}
    for b, j in at.items():
        p.k[b][:] = 0
        for h in range(2):  # its head's queries all lie about along it, others score 0
            p.q[b, 0, 4 * h:4 * h + 4] = (p.q[b, 0, 4 * h] * torch.tensor([1.0, 1.01, 1.3, 2.7], device="cuda")[:, None]).bfloat16()
            p.k[b][j, h] = (p.q[b, 0, 4 * h].float().cpu() * 40).bfloat16()
    p.write()
    for ws in ("enough", None):
        got = p.call(ws)
        for b, j in at.items():
            assert torch.equal(got[b, 0].cpu(), p.v[b][j].repeat_interleave(4, 0)), f"request {b}"


@pytest.mark.parametrize("low", [INF, -INF, NAN])
@pytest.mark.parametrize("dim", [64, 128])
def test_smallest_values_that_are_not_finite_stay_with_the_rows_that_take_them(dim, low, kernel):
    """4 bits: a drafted token that no row takes, whose slot holds anything (a scale that is a number, a smallest value that is none), and one that
    some rows take: all others as if the two held zeros."""
    nodes, n = 20, 73
    tree = [t & ~(1 << 19) for t in random_tree(nodes, 6)]  # nobody takes token 19, not even itself
    tree[9] |= 1 << 4
    p = Problem([n], [nodes], 4, 2, dim, 4, 16, tree=[tree], seed=33)
    base = n - nodes
    for token in (4, 19):
        key = base + token
        slot = int(p.table[0, key // p.page]), key % p.page
        p.cache.v_scales[slot[0], :, slot[1], :, 1] = low
        if token == 19:
            p.cache.k_scales[slot[0], :, slot[1], :, 1] = low
    got = p.call()
    none = p.call(workspace=None)
    takes = np.array([(t >> 4) & 1 for t in tree], bool)
    assert takes.any() and not takes.all()
    for o in (got, none):
        p.check(o, rows=lambda b: ~takes)
        assert not o[0, torch.from_numpy(takes).cuda()].isfinite().any()


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("q_scale,k_scale", [(2.0 ** 118, 2.0 ** -116), (2.0 ** 118, 2.0 ** -8), (2.0 ** -120, 2.0 ** 119)])
def test_queries_near_the_ends_of_the_range(q_scale, k_scale, bits, kernel):
    """Scale times the largest |q| (4.5 standard deviations and less) up to 2^117, with keys that make scores of ordinary size, or so large that one key
    takes all; the largest |q| below 2^-117 (elements are kept out of bf16's subnormal range); then with a token of ordinary queries beside the large
    ones, whose scores are tiny."""
    p = Problem([400], [4], 4, 2, 128, bits, 64, seed=34)
    away = lambda x, s: (x.float().sign() * x.float().abs().clamp(min=2.0 ** -5) * s).bfloat16()  # noqa: E731
    p.q, p.k[0] = away(p.q, q_scale), away(p.k[0], k_scale)
    p.write()
    p.check(p.call())
    p.answers.clear()
    if q_scale > 1:
        p.q[0, 2] = (p.q[0, 2].float() / q_scale).bfloat16()  # scores of 2^-119: every key the same
        p.check(p.call())


def test_arguments_that_are_no_tensors_are_type_errors():
    p = Problem([100], [2], 4, 2, 64, 8, 16, seed=39)
    lens, c = ints([100]), p.cache
    slots = ints([0, 1])
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: lb.cache_attention(p.q, c, [[1]], lens), lambda: lb.cache_attention(p.q, c, p.table, [100]),
                 lambda: lb.cache_attention(p.q, c, p.table, 100), lambda: lb.cache_attention(p.q, None, p.table, lens),
                 lambda: lb.cache_attention(p.q, c.k, p.table, lens), lambda: lb.cache_attention(p.q, c, p.table, lens, workspace=4096),
                 lambda: lb.cache_attention(p.q, c, p.table, lens, q_lens=[2]), lambda: lb.cache_attention(p.q, c, p.table, lens, tree=[[1, 3]]),
                 lambda: lb.cache_attention(p.q, c, p.table, lens, out="q"), lambda: lb.cache_attention("q", c, p.table, lens),
                 lambda: lb.cache_attention_workspace_size(p.q, c.k, 100), lambda: lb.KVCache(c.k, None, c.k_scales, c.v_scales),
                 lambda: lb.KVCache(c.k, 5, c.k_scales, c.v_scales), lambda: lb.KVCache(c.k, c.v, [1.0], c.v_scales), lambda: lb.KVCache(c.k, c.v),
                 lambda: lb.cache_write(c.k, x, x, slots), lambda: lb.cache_write(c, x, None, slots), lambda: lb.cache_write(c, x, x, [0, 1]),
                 lambda: lb.cache_read(None, slots), lambda: lb.cache_read(c, [0, 1]), lambda: lb.cache_read(c, slots, k_out=3)):
        with pytest.raises(TypeError):
            call()


def test_part_of_a_wider_table(kernel):
    """The first pages of every request's row of a table, and rows of a transposed one, which lie apart."""
    p = Problem([200, 150], [2, 2], 4, 2, 64, 8, 16, seed=38)
    want = p.call(workspace=None)
    pages = p.table.shape[1]
    wide = torch.full((2, pages + 9), -1, dtype=torch.int32, device="cuda")
    wide[:, :pages] = p.table
    lens = ints(p.lens)
    assert torch.equal(lb.cache_attention(p.q, p.cache, wide[:, :pages], lens, kv_len=200), want)
    assert torch.equal(lb.cache_attention(p.q[1:], p.cache, wide[1:, :pages], lens[1:], kv_len=200), want[1:])
    every = torch.full((4, pages), -1, dtype=torch.int32, device="cuda")
    every[::2] = p.table
    assert torch.equal(lb.cache_attention(p.q, p.cache, every[::2], lens, kv_len=200), want)
    both = p.q[:1].expand(2, -1, -1, -1)
    one = lb.cache_attention(both, p.cache, p.table[:1].expand(2, -1), lens[:1].expand(2).contiguous(), kv_len=200)
    assert torch.equal(one[0], one[1]) and torch.equal(one[:1], want[:1])
    with pytest.raises(ValueError, match="page_table"):
        lb.cache_attention(p.q, p.cache, p.table.t().contiguous().t(), lens, kv_len=200)


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("scale", [0.02, 0.5, 1.0])
def test_scales_other_than_the_default(scale, bits, kernel):
    for dim, lens, new in ((64, [90, 7], [3, 2]), (128, [700], [5]), (128, [1, 60], [1, 1])):
        p = Problem(lens, new, 4, 2, dim, bits, 32, seed=35)
        for ws in ("enough", None):
            p.check(p.call(ws, scale=scale), scale=scale)


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
def test_trees_of_unequal_sizes(dim, bits, kernel):
    """Requests with fewer drafted tokens than the tree has rows, bits set past a request's last token (which say nothing), no drafted token at all,
    more of them than keys; rows past the last are left as they were."""
    nodes, q_lens, lens = 40, [40, 7, 0, 23, 33], [300, 77, 50, 23, 12]
    tree = [random_tree(nodes, s) for s in range(5)]
    p = Problem(lens, q_lens, 4, 2, dim, bits, 16, tree=tree, seed=36)
    clean = p.call(out=torch.full_like(p.q, 3.0))
    p.check(clean)
    p.tree = [[t | (0xFFFFFFFFFFFFFFFF << n & 0xFFFFFFFFFFFFFFFF) for t in row] for row, n in zip(tree, q_lens)]
    for ws in ("enough", None):
        got = p.call(ws, out=torch.full_like(p.q, 3.0))
        p.check(got)
        for b, n in enumerate(q_lens):
            assert (got[b, n:] == 3).all()


def test_pages_named_twice_change_their_request_alone(kernel):
    """A table that names a page of the common prefix twice for request 0; request 1 keeps the shared prefix."""
    p = Problem([128, 128], [4, 4], 4, 2, 128, 8, 32, seed=37)
    p.table[1, :2] = p.table[0, :2]
    for x in (p.k, p.v):
        x[1][:64] = x[0][:64]
    p.check(p.call())
    p.answers.clear()
    p.table[0, 1] = p.table[0, 0]
    for x in (p.k, p.v):
        x[0] = torch.cat([x[0][:32], x[0][:32], x[0][64:]])
    p.check(p.call())
