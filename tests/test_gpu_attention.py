"""Attention against the formula in 64 bits.

Tolerance, per element of O = sum_j p_j v_j: the probabilities are rounded to bf16 (8 significant bits: 2^-8
of each, so 2^-8 of A = sum_j p_j |v_j|), the result is rounded once (2^-8 of it), and the fp32 work before the
rounding (scores as sums of up to 128 products, exponentials, sums) stays below 2^-12 of A for the inputs
here, whose scores are sums of |q k| / sqrt(D) below 32: 128 * 2^-24 * 32 = 2^-12 is the bound of a
sum in any order.
"""
import math

import numpy as np
import pytest
import torch

import binary_bit_gemm_amd as lb

pytestmark = pytest.mark.gpu


def allowed(B, Lq, Lk, mask, lens, causal, start):
    ok = np.ones((B, Lq, Lk), dtype=bool)
    if mask is not None:
        ok &= mask.cpu().numpy().astype(bool)[:, None]
    if lens is not None:
        ok &= np.arange(Lk)[None, None] < lens.cpu().numpy()[:, None, None]
    if causal:
        s = start.cpu().numpy() if start is not None else np.zeros(B, dtype=np.int64)
        ok &= np.arange(Lk)[None, None] <= (s[:, None] + np.arange(Lq))[:, :, None]
    return ok


def reference(q, k, v, mask=None, lens=None, causal=False, start=None, scale=None):
    """(O, sum p |v|) in 64 bits on the CPU; rows without keys are zeros, and what no row takes is left out."""
    B, Lq, Hq, D = q.shape
    Lk, Hk = k.shape[1], k.shape[2]
    ok = allowed(B, Lq, Lk, mask, lens, causal, start)
    qd, kd, vd = (x.double().cpu().numpy() for x in (q, k, v))
    out, mag = np.zeros((B, Lq, Hq, D)), np.zeros((B, Lq, Hq, D))
    scale = scale if scale is not None else 1 / math.sqrt(D)
    for b in range(B):
        for h in range(Hq):
            kh, vh = kd[b, :, h * Hk // Hq], vd[b, :, h * Hk // Hq]
            for rows in np.array_split(np.arange(Lq), max(1, Lq // 256)):
                with np.errstate(invalid="ignore", over="ignore"):
                    s = np.where(ok[b, rows], (qd[b, rows, h] @ np.where(ok[b, rows].any(0)[:, None], kh, 0).T) * scale, -np.inf)
                top = s.max(-1, keepdims=True, initial=-np.inf)
                p = np.exp(s - np.where(np.isfinite(top), top, 0))
                tot = p.sum(-1, keepdims=True)
                p = p / np.where(tot == 0, 1, tot)
                used = ok[b, rows].any(0)
                out[b, rows, h] = p[:, used] @ vh[used]
                mag[b, rows, h] = p[:, used] @ np.abs(vh[used])
    return out, mag


def check(got, want, mag):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - want) - ((2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * np.abs(want))
    assert off.max(initial=-1) <= 0, f"worst element over its bound by {off.max()}"


def make(B, Lq, Lk, Hq, Hk, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, Lq, Hq, D, generator=g).bfloat16().cuda()
    k, v = (torch.randn(B, Lk, Hk, D, generator=g).bfloat16().cuda() for _ in range(2))
    return q, k, v


@pytest.fixture(params=["few", "many", "many64", "many128", "auto"])
def kernel(request, monkeypatch):
    """Each of the kernels in turn (many rows: 64 and 128 per workgroup), and the one that the library takes."""
    if request.param != "auto":
        monkeypatch.setenv("LOWBIT_ATTENTION", request.param)
    return request.param


def scratch(q, k, v):
    n = lb.attention_workspace_size(q, k, v)
    ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0  # the arrival counters; the rest may hold anything
    return ws if n else None


SHAPES = [  # B, Lq, Lk, Hq, Hk, D
    (1, 1, 1, 1, 1, 128), (1, 1, 63, 2, 1, 64), (2, 1, 257, 32, 8, 128), (1, 1, 5000, 8, 2, 64), (3, 2, 130, 6, 6, 128),
    (1, 5, 4097, 8, 1, 128), (2, 33, 65, 4, 2, 64), (1, 128, 128, 3, 3, 128), (1, 129, 191, 2, 2, 64), (1, 300, 300, 4, 4, 128),
    (2, 511, 511, 2, 1, 128), (1, 64, 2049, 4, 4, 64), (1, 31, 1000, 7, 7, 128), (1, 700, 33, 2, 2, 128),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal", [False, True])
def test_shapes(shape, causal, kernel):
    B, Lq, Lk = shape[:3]
    q, k, v = make(*shape)
    start = torch.full((B,), Lk - Lq, dtype=torch.int32, device="cuda") if causal else None
    want = reference(q, k, v, causal=causal, start=start)
    check(lb.attention(q, k, v, causal=causal, q_start=start), *want)
    check(lb.attention(q, k, v, causal=causal, q_start=start, workspace=scratch(q, k, v)), *want)


@pytest.mark.parametrize("shape", [(2, 1, 777, 8, 2, 128), (3, 70, 70, 4, 4, 64), (2, 200, 333, 2, 2, 128), (4, 1, 64, 4, 4, 64)])
@pytest.mark.parametrize("causal", [False, True])
def test_masks_lengths_and_empty_rows(shape, causal, kernel):
    B, Lq, Lk, Hq, Hk, D = shape
    q, k, v = make(*shape, seed=1)
    g = torch.Generator().manual_seed(2)
    mask = (torch.rand(B, Lk, generator=g) < 0.6)
    mask[0] = False  # nothing left for a whole batch entry
    mask[-1, : Lk // 2] = False
    mask = mask.cuda()
    lens = torch.randint(0, Lk + 1, (B,), generator=g, dtype=torch.int32)
    lens[-1] = Lk
    lens = lens.cuda()
    start = torch.arange(B, dtype=torch.int32).cuda() * 17 - 9 if causal else None  # rows before the first key too
    ws = scratch(q, k, v)
    for m, n in ((mask, None), (None, lens), (mask, lens), (mask.to(torch.uint8) * 3, None)):
        want = reference(q, k, v, m, n, causal, start)
        check(lb.attention(q, k, v, key_mask=m, key_lens=n, causal=causal, q_start=start), *want)
        check(lb.attention(q, k, v, key_mask=m, key_lens=n, causal=causal, q_start=start, workspace=ws), *want)
    got = lb.attention(q, k, v, key_mask=mask, causal=causal, q_start=start)
    assert not bool(got[0].any())


@pytest.mark.parametrize("lens", [[0, 0], [-3, 1], [1, 500], [64, 65]])
def test_lengths_out_of_range_and_short(lens, kernel):
    q, k, v = make(2, 3, 100, 4, 2, 128, seed=3)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    check(lb.attention(q, k, v, key_lens=n), *reference(q, k, v, lens=n))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min])
def test_anything_in_places_that_are_left_out(bad, D, kernel):
    """Padding in the middle and past the length holds infinities, NaN or the type's lowest value."""
    q, k, v = make(2, 90, 200, 4, 2, D, seed=4)
    mask = torch.ones(2, 200, dtype=torch.bool)
    mask[0, 30:77] = False
    mask[1, 0] = mask[1, 199] = False
    mask = mask.cuda()
    lens = torch.tensor([200, 150], dtype=torch.int32).cuda()
    want = lb.attention(q, k, v, key_mask=mask, key_lens=lens)
    check(want, *reference(q, k, v, mask, lens))
    out = ~mask | (torch.arange(200, device="cuda") >= lens[:, None])
    k[out] = bad
    v[out] = bad
    assert torch.equal(lb.attention(q, k, v, key_mask=mask, key_lens=lens), want)
    ws = scratch(q, k, v)
    if ws is not None:
        check(lb.attention(q, k, v, key_mask=mask, key_lens=lens, workspace=ws), *reference(q, k, v, mask, lens))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_later_keys_do_not_reach_earlier_queries(bad, D, kernel):
    """Causal: a value that is no number at key j leaves queries before j alone and reaches the others."""
    q, k, v = make(1, 150, 150, 2, 2, D, seed=5)
    want = lb.attention(q, k, v, causal=True)
    v2 = v.clone()
    v2[0, 70, 0, 5] = bad
    got = lb.attention(q, k, v2, causal=True)
    assert torch.equal(got[0, :70], want[0, :70]) and torch.equal(got[0, :, 1], want[0, :, 1])
    seen = got[0, 70:, 0, 5]
    assert bool(torch.isnan(seen).all()) if math.isnan(bad) else bool((seen == bad).all())
    k2 = k.clone()
    k2[0, 70, 0] = float("nan")
    got = lb.attention(q, k2, v, causal=True)
    assert torch.equal(got[0, :70], want[0, :70]) and bool(torch.isnan(got[0, 70:, 0]).all())


def test_large_scores_and_growing_maxima(kernel):
    """Scores that grow along the keys (the running maximum moves at every tile) and reach thousands."""
    q, k, v = make(1, 40, 1000, 2, 2, 128, seed=6)
    k = (k.float() * torch.linspace(0.1, 4, 1000, device="cuda")[None, :, None, None]).bfloat16()
    want, mag = reference(q, k, v)
    got = lb.attention(q, k, v)
    check(got, want, mag)
    q = (q.float() * 64).bfloat16()  # scores up to some thousands: fp32 sums of them are off by more, so only the shape of the result
    want, mag = reference(q, k, v)
    off = np.abs(lb.attention(q, k, v).double().cpu().numpy() - want)
    assert (off <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -5) * mag + 1e-6).all()


def test_views_of_a_fused_projection_and_other_layouts(kernel):
    g = torch.Generator().manual_seed(7)
    B, L, Hq, Hk, D = 2, 77, 6, 2, 128
    qkv = torch.randn(B, L, Hq + 2 * Hk, D, generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
    want = lb.attention(q.contiguous(), k.contiguous(), v.contiguous(), causal=True)
    check(want, *reference(q, k, v, causal=True))
    assert torch.equal(lb.attention(q, k, v, causal=True), want)
    kh, vh = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))  # head-major cache
    out = torch.empty(B, Hq, L, D, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    assert torch.equal(lb.attention(q, kh, vh, causal=True, out=out), want)
    one = lb.attention(q, k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1))  # one cache for the batch
    assert torch.equal(one[1], lb.attention(q[1:], k[:1], v[:1])[0])
    mask = torch.rand(L, generator=g) < 0.7
    mask = mask.cuda()[None].expand(B, -1)
    check(lb.attention(q, k, v, key_mask=mask), *reference(q, k, v, mask))


def test_scale_and_empty_calls(kernel):
    q, k, v = make(1, 20, 50, 2, 2, 64, seed=8)
    check(lb.attention(q, k, v, scale=0.01), *reference(q, k, v, scale=0.01))
    assert not bool(lb.attention(q, k[:, :0], v[:, :0]).any())
    assert lb.attention(q[:, :0], k, v).shape == (1, 0, 2, 64)
    assert lb.attention(q[:0], k[:0], v[:0]).shape == (0, 20, 2, 64)


def test_offsets_past_32_bits(kernel):
    """A cache whose tokens lie 2^25 bytes apart: the last ones start past 2^32 bytes."""
    n, step = 200, 1 << 24
    g = torch.Generator().manual_seed(9)
    buf = torch.empty(n * step, dtype=torch.bfloat16, device="cuda")
    small = torch.randn(1, n, 2, 128, generator=g).bfloat16().cuda()
    k = buf.as_strided((1, n, 2, 128), (n * step, step, 128, 1))
    v = buf.as_strided((1, n, 2, 128), (n * step, step, 128, 1), 1024)
    k.copy_(small)
    v.copy_(small.flip(1))
    q = torch.randn(1, 3, 4, 128, generator=g).bfloat16().cuda()
    assert torch.equal(lb.attention(q, k, v), lb.attention(q, k.contiguous(), v.contiguous()))


def test_runs_repeat_bitwise_and_on_another_stream(kernel):
    q, k, v = make(1, 3, 6000, 16, 4, 128, seed=10)
    ws = scratch(q, k, v)
    want = lb.attention(q, k, v, workspace=ws)
    for _ in range(3):
        assert torch.equal(lb.attention(q, k, v, workspace=ws), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = lb.attention(q, k, v, workspace=ws)
    s.synchronize()
    assert torch.equal(got, want)


def test_counters_are_left_at_zero_and_shapes_take_turns(kernel):
    calls = [make(*shape, seed=20 + i) for i, shape in enumerate([(1, 1, 9000, 8, 2, 128), (4, 2, 1500, 16, 4, 64), (2, 40, 4000, 2, 2, 128)])]
    ws = torch.zeros(max(lb.attention_workspace_size(*c) for c in calls), dtype=torch.uint8, device="cuda")
    first = [lb.attention(*c, workspace=ws) for c in calls]
    for _ in range(2):
        for c, f in zip(calls, first):
            got = lb.attention(*c, workspace=ws)
            assert torch.equal(got, f) and not bool(ws[:4096].any())
            check(got, *reference(*c))


def test_in_a_graph(kernel):
    q, k, v = make(1, 2, 3000, 8, 8, 64, seed=11)
    ws = scratch(q, k, v)
    out = torch.empty_like(q)
    lb.attention(q, k, v, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lb.attention(q, k, v, out=out, workspace=ws)
    for seed in (12, 13, 14):
        for t, n in zip((q, k, v), make(1, 2, 3000, 8, 8, 64, seed=seed)):
            t.copy_(n)
        want = lb.attention(q, k, v, workspace=ws)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("power", [16, 24, 27, 28, 29, 31, 34, 40, 60, 90])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("shape", [(1, 40, 1000, 2, 2, 128), (2, 90, 300, 4, 2, 64), (1, 1, 5000, 8, 2, 64), (1, 40, 4000, 2, 2, 128)])
def test_scores_of_any_size(shape, sign, power, kernel):
    """Queries times a power of two: a row's largest score then takes all of the softmax, and every key is there twice, so its
    result is the mean of two values.  Rows whose largest scores lie closer than an fp32 sum of 128 products is off (2^-12 of
    the power, see above) or closer than 2^-4 of the power (an exponent of 2^12 at the least) are left out."""
    B, Lq, Lk, Hq, Hk, D = shape
    q, k, v = make(B, Lq, Lk, Hq, Hk, D, seed=30)
    if sign < 0:  # every score below zero
        q, k = q.abs(), -k.abs()
    k[:, Lk // 2:] = k[:, :Lk // 2]
    s = torch.einsum("bthd,bjhd->bhtj", q.double().cpu(), k.double().cpu()[:, :Lk // 2].repeat_interleave(Hq // Hk, 2))
    top, at = s.topk(2, -1)
    clear = (top[..., 0] - top[..., 1] > 2.0 ** -4 * math.sqrt(D)).transpose(1, 2)  # [B, Lq, Hq]
    assert clear.float().mean() > 0.5
    vd = v.double().cpu().repeat_interleave(Hq // Hk, 2).transpose(1, 2)  # [B, Hq, Lk, D]
    first = at[..., :1].expand(-1, -1, -1, D)
    a, b = vd.gather(2, first), vd.gather(2, first + Lk // 2)
    want, mag = ((a + b) / 2).transpose(1, 2), ((a.abs() + b.abs()) / 2).transpose(1, 2)
    q = (q.float() * 2.0 ** power).bfloat16()
    for ws in (None, scratch(q, k, v)):
        got = lb.attention(q, k, v, workspace=ws)
        check(got[clear], want[clear].numpy(), mag[clear].numpy())


@pytest.mark.parametrize("heads,D,queries,keys,start,rows", [
    (24, 128, 2560, 2560, "end", 64), (24, 128, 2560, 3840, "end", 64), (24, 128, 2560, 7680, "end", 128),
    (24, 128, 2560, 20480, "end", 128), (16, 128, 4096, 16384, "end", 128), (24, 128, 2560, 20480, None, 64),
    (24, 64, 2560, 7680, "end", 64), (24, 64, 2560, 20480, "end", 128),
    (24, 128, 1100, 8800, "end", 64), (16, 128, 2048, 16384, "end", 64),  # 64 rows fill the compute units better
])
def test_rows_of_a_workgroup_for_a_chunk_after_a_long_cache(heads, D, queries, keys, start, rows, capfd, monkeypatch):
    """A causal prompt takes 64 rows at a time; a chunk of queries after many keys, of which every row tile has about as many, what
    a call without the causal rule takes.  (Last queries only: their results against the formula.)"""
    q, k, v = make(1, queries, keys, heads, 1, D, seed=40)
    k, v = (x.expand(-1, -1, heads, -1) for x in (k, v))
    first = keys - queries if start else 0
    s = torch.tensor([first], dtype=torch.int32, device="cuda") if start else None
    monkeypatch.setenv("LOWBIT_TRACE", "1")
    capfd.readouterr()
    got = lb.attention(q, k, v, causal=True, q_start=s)
    torch.cuda.synchronize()
    lines = [l for l in capfd.readouterr().err.splitlines() if l.startswith("lowbit: attention ")]
    assert len(lines) == 1 and f"many rows={rows} splits=1 " in lines[0], lines
    assert f"problem=1x{queries}x{keys}x{heads} kv_heads={heads} dim={D} causal" in lines[0]
    last = torch.tensor([first + queries - 3], dtype=torch.int32, device="cuda")
    check(got[:, -3:, :2], *reference(q[:, -3:, :2], k[:, :, :2], v[:, :, :2], causal=True, start=last))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_splits_share_the_keys_there_are(causal, D, monkeypatch):
    """Many rows, keys split, lengths and positions far below the cache's: the partial results (behind the counters: O, then the
    maximum and the sum of each row) show that the splits took even shares of the keys that a row has."""
    monkeypatch.setenv("LOWBIT_ATTENTION", "many")
    B, Lq, Lk, H = 2, 40, 4000, 2
    q, k, v = make(B, Lq, Lk, H, H, D, seed=41)
    ws = scratch(q, k, v)
    rows = (ws.numel() - 4096) // ((D + 2) * 4)
    splits = rows // (B * H * Lq)
    assert rows == B * H * Lq * splits and splits >= 8
    keys = torch.tensor([1000, 3000], dtype=torch.int32).cuda()
    mask = dict(causal=True, q_start=keys - Lq) if causal else dict(key_lens=keys)
    got = lb.attention(q, k, v, workspace=ws, **mask)
    check(got, *reference(q, k, v, lens=mask.get("key_lens"), causal=causal, start=mask.get("q_start")))
    sums = ws[4096 + rows * D * 4:].view(torch.float32).view(B, H, splits, Lq, 2)[..., 1]
    for b in range(B):
        tiles = -(-int(keys[b]) // 64)
        taken = -(-tiles // -(-tiles // splits))  # splits that an even share reaches
        assert bool((sums[b, :, :taken - 1] > 0).all()) and not bool(sums[b, :, taken:].any())


# Keys split across workgroups in both kernels, with a workspace: 2 x 40 queries over 4000 keys.
SPLIT = [(2, 40, 4000, 2, 2, 128), (2, 40, 4000, 4, 2, 64), (3, 33, 5000, 2, 1, 128)]


def split_scratch(q, k, v, kernel):
    ws = scratch(q, k, v)
    if kernel != "many64":  # 64 rows are taken unsplit
        assert ws is not None
    return ws


@pytest.mark.parametrize("shape", SPLIT)
@pytest.mark.parametrize("causal", [False, True])
def test_masks_lengths_and_empty_rows_of_split_keys(shape, causal, kernel):
    """Empty partial results: rows without a key in some splits and in all of them."""
    B, Lq, Lk, Hq, Hk, D = shape
    q, k, v = make(*shape, seed=50)
    g = torch.Generator().manual_seed(51)
    ws = split_scratch(q, k, v, kernel)
    sparse = torch.rand(B, Lk, generator=g) < 0.02
    sparse[0] = False  # nothing left for a whole batch entry
    middle = torch.zeros(B, Lk, dtype=torch.bool)
    middle[:, 1500:1600] = True  # one split's keys, or two's
    middle[1, Lk - 1] = True
    end = torch.full((B,), Lk, dtype=torch.int32)
    end[0] = 3
    short = torch.tensor([0, 70, -1][:B], dtype=torch.int32)
    starts = [None, torch.tensor([-20, 0, 5][:B], dtype=torch.int32), torch.tensor([Lk - Lq, 100, 2000][:B], dtype=torch.int32)]
    for start in starts if causal else [None]:
        start = None if start is None else start.cuda()
        for m, n in ((sparse, None), (middle, None), (None, short), (None, end), (middle, end), (sparse, short), (None, None)):
            m, n = (None if x is None else x.cuda() for x in (m, n))
            got = lb.attention(q, k, v, key_mask=m, key_lens=n, causal=causal, q_start=start, workspace=ws)
            check(got, *reference(q, k, v, m, n, causal, start))
            ok = torch.from_numpy(allowed(B, Lq, Lk, m, n, causal, start).any(-1)).cuda()
            assert not bool(got[~ok].any())
            if ws is not None:
                assert not bool(ws[:4096].any())


@pytest.mark.parametrize("shape", SPLIT[:2])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min])
def test_anything_in_places_that_split_keys_leave_out(bad, shape, kernel):
    B, Lq, Lk = shape[:3]
    q, k, v = make(*shape, seed=52)
    ws = split_scratch(q, k, v, kernel)
    mask = torch.ones(B, Lk, dtype=torch.bool)
    mask[0, 300:2777] = False  # whole splits
    mask[1, 0] = mask[1, 640:650] = mask[1, Lk - 1] = False
    mask = mask.cuda()
    lens = torch.tensor([Lk, 1850], dtype=torch.int32).cuda()
    want = lb.attention(q, k, v, key_mask=mask, key_lens=lens, workspace=ws)
    check(want, *reference(q, k, v, mask, lens))
    out = ~mask | (torch.arange(Lk, device="cuda") >= lens[:, None])
    k[out] = bad
    v[out] = bad
    assert torch.equal(lb.attention(q, k, v, key_mask=mask, key_lens=lens, workspace=ws), want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_later_keys_do_not_reach_earlier_queries_of_split_keys(bad, D, kernel):
    q, k, v = make(1, 40, 4000, 2, 2, D, seed=53)
    ws = split_scratch(q, k, v, kernel)
    start = torch.tensor([3000], dtype=torch.int32, device="cuda")
    call = lambda k, v: lb.attention(q, k, v, causal=True, q_start=start, workspace=ws)  # noqa: E731
    want = call(k, v)
    check(want, *reference(q, k, v, causal=True, start=start))
    v2 = v.clone()
    v2[0, 3017, 0, 5] = bad  # the 17th query on
    got = call(k, v2)
    assert torch.equal(got[0, :17], want[0, :17]) and torch.equal(got[0, :, 1], want[0, :, 1])
    seen = got[0, 17:, 0, 5]
    assert bool(torch.isnan(seen).all()) if math.isnan(bad) else bool((seen == bad).all())
    k2 = k.clone()
    k2[0, 3017, 0] = float("nan")
    got = call(k2, v)
    assert torch.equal(got[0, :17], want[0, :17]) and bool(torch.isnan(got[0, 17:, 0]).all())


def test_a_workspace_that_is_too_small_is_not_used(kernel):
    """The call runs unsplit, as without one, and leaves the buffer alone."""
    for shape in SPLIT[:2]:
        q, k, v = make(*shape, seed=54)
        n = lb.attention_workspace_size(q, k, v)
        want = lb.attention(q, k, v)
        for size in (n - 1, 4096, 16):
            if size > 0:
                ws = torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")
                assert torch.equal(lb.attention(q, k, v, workspace=ws), want) and bool((ws == 0xAB).all())


@pytest.mark.parametrize("power", [-70, 90])
@pytest.mark.parametrize("shape", [(1, 40, 1000, 2, 2, 128), (1, 1, 5000, 8, 2, 64), (2, 200, 333, 2, 2, 128)])
def test_values_of_any_size(shape, power, kernel):
    """O is kept undivided, the largest probability anywhere from 2^-32 to 2: at the ends of the range that is promised for values,
    with scores that grow along the keys, what fp32 loses is below 2^-126 of a sum of at least 2^-102."""
    q, k, v = make(*shape, seed=60)
    Lk = shape[2]
    k = (k.float() * torch.linspace(0.1, 4, Lk, device="cuda")[None, :, None, None]).bfloat16()
    v = (v.float().abs().clamp(0.5, 2) * v.float().sign() * 2.0 ** power).bfloat16()
    for ws in (None, scratch(q, k, v)):
        check(lb.attention(q, k, v, workspace=ws), *reference(q, k, v))
