"""Norms of queries and keys with the position rotation, against the formula in 64 bits.

Tolerance, per element: one rounding to bf16 (8 significant bits: 2^-8 of the result) and the fp32 work before it.  The
fraction of a turn is rounded to fp32 (2^-25 of a turn, 2^-22.3 rad), sine and cosine and the norm to a
few units of 2^-24 each, and the turned element is a difference of two products: 2^-19 of |u| + |v|
covers them, (u, v) the pair before the turn.
"""
import numpy as np
import pytest
import torch

import binary_bit_gemm_amd as lb

pytestmark = pytest.mark.gpu


def reference(x, w, positions, freqs, dims, eps, interleaved):
    """(result, |u| + |v|) in 64 bits on the CPU."""
    x = x.double().cpu().numpy()
    D = x.shape[-1]
    if w is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w.double().cpu().numpy()
    y, mag = x.copy(), np.abs(x)
    half = sum(dims) // 2
    if half:
        axis = np.repeat(np.arange(len(dims)), [d // 2 for d in dims])
        angle = positions.cpu().numpy().astype(np.float64)[:, axis] * freqs.double().cpu().numpy()
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        one = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
        two = one + 1 if interleaved else one + half
        u, v = x[..., one], x[..., two]
        y[..., one], y[..., two] = u * c - v * s, u * s + v * c
        mag[..., one] = mag[..., two] = np.abs(u) + np.abs(v)
    return y, mag


def check(got, want, mag):
    got = got.double().cpu().numpy()
    off = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + 2.0 ** -19 * mag + 1e-38)
    assert off.max(initial=-1) <= 0, f"worst element over its bound by {off.max()}"


def make(T, Hq, Hk, D, dims, seed=0, weights=True, big=4096):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g).bfloat16().cuda()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2)] if weights else [None, None]
    pos = torch.randint(-big, big + 1, (T, len(dims)), generator=g, dtype=torch.int32).cuda()
    freqs = lb.rope_freqs(dims, 2000.0)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hk], w, pos, freqs


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,Hq,Hk,D,dims", [
    (1, 1, 1, 128, (128,)), (1, 32, 8, 128, (128,)), (3, 5, 1, 64, (16, 24, 24)), (17, 24, 24, 128, (32, 32, 32, 32)),
    (130, 16, 4, 64, (32, 16)), (7, 3, 3, 32, (16,)), (5, 4, 2, 256, (64, 96, 96)), (9, 0, 3, 128, (48, 16)),
    (9, 3, 0, 64, (64,)), (33, 7, 7, 256, (256,)), (1000, 9, 2, 128, (16, 56, 56)),
])
def test_norm_and_rotation(T, Hq, Hk, D, dims, interleaved):
    q, k, w, pos, freqs = make(T, Hq, Hk, D, dims)
    qo, ko = lb.qk_norm_rope(q, k, pos, freqs, dims, *w, eps=1e-6, interleaved=interleaved)
    check(qo, *reference(q, w[0], pos, freqs, dims, 1e-6, interleaved))
    check(ko, *reference(k, w[1], pos, freqs, dims, 1e-6, interleaved))


@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_rotation_alone_and_norm_alone(D):
    q, k, w, pos, freqs = make(21, 6, 2, D, (D,), seed=1)
    qo, ko = lb.qk_norm_rope(q, k, pos, freqs, (D,), interleaved=False)
    check(qo, *reference(q, None, pos, freqs, (D,), 0, False))
    check(ko, *reference(k, None, pos, freqs, (D,), 0, False))
    qo, ko = lb.qk_norm_rope(q, k, None, None, (), *w, eps=1e-5)
    check(qo, *reference(q, w[0], None, None, (), 1e-5, True))
    check(ko, *reference(k, w[1], None, None, (), 1e-5, True))
    qo, ko = lb.qk_norm_rope(q, k, pos, freqs, (D,), None, w[1])  # one of the two normed
    check(qo, *reference(q, None, pos, freqs, (D,), 0, True))
    check(ko, *reference(k, w[1], pos, freqs, (D,), 1e-6, True))
    qo, ko = lb.qk_norm_rope(q, k, None, None, ())  # neither: a copy
    assert torch.equal(qo, q) and torch.equal(ko, k)


def test_positions_of_a_million():
    """The angle keeps its accuracy where fp32 would not: position 10^6 on a frequency of 1."""
    q, k, w, pos, freqs = make(64, 4, 4, 128, (128,), seed=2, big=1 << 20)
    qo, _ = lb.qk_norm_rope(q, k, pos, freqs, (128,), *w)
    check(qo, *reference(q, w[0], pos, freqs, (128,), 1e-6, True))
    pos[:] = 2 ** 31 - 1
    qo, _ = lb.qk_norm_rope(q, k, pos, freqs, (128,), *w)
    check(qo, *reference(q, w[0], pos, freqs, (128,), 1e-6, True))


@pytest.mark.parametrize("interleaved", [True, False])
def test_in_place_equals_out_of_place(interleaved):
    q, k, w, pos, freqs = make(77, 12, 4, 128, (32, 48, 48), seed=3)
    qo, ko = lb.qk_norm_rope(q, k, pos, freqs, (32, 48, 48), *w, interleaved=interleaved)
    a, b = lb.qk_norm_rope(q, k, pos, freqs, (32, 48, 48), *w, interleaved=interleaved, q_out=q, k_out=k)
    assert a.data_ptr() == q.data_ptr() and torch.equal(a, qo) and torch.equal(b, ko)


def test_head_major_layouts_and_untouched_neighbours():
    q, k, w, pos, freqs = make(19, 5, 3, 64, (64,), seed=4)
    want = lb.qk_norm_rope(q, k, pos, freqs, (64,), *w)
    qh = q.transpose(0, 1).contiguous().transpose(0, 1)  # [heads, tokens, D] in memory
    guard = torch.full((5, 21, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guard[:, 1:20, 8:72].transpose(0, 1)
    got = lb.qk_norm_rope(qh, k, pos, freqs, (64,), *w, q_out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    guard[:, 1:20, 8:72] = 7.0
    assert bool((guard == 7.0).all())


def test_infinities_stay_in_their_heads_and_partial_rotation_passes_through():
    q, k, w, pos, freqs = make(6, 4, 2, 128, (32,), seed=5)
    want, _ = lb.qk_norm_rope(q, k, pos, freqs, (32,))
    assert torch.equal(want[..., 32:], q[..., 32:])
    q = q.clone()
    q[2, 1, 100] = float("inf")
    q[3, 0, 90] = float("nan")
    got, _ = lb.qk_norm_rope(q, k, pos, freqs, (32,))
    keep = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    assert torch.equal(got[2, 1, :100], want[2, 1, :100]) and torch.isinf(got[2, 1, 100]) and torch.isnan(got[3, 0, 90])
    keep[2, 1] = keep[3, 0] = False
    assert torch.equal(got[keep], want[keep])


def test_zero_rows_and_empty_calls():
    q, k, w, pos, freqs = make(4, 2, 2, 64, (64,), seed=6)
    z = torch.zeros_like(q)
    qo, _ = lb.qk_norm_rope(z, k, pos, freqs, (64,), *w)
    assert not bool(qo.any())
    qo, ko = lb.qk_norm_rope(q[:0], k[:0], pos[:0], freqs, (64,), *w)
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 2, 64)


def test_offsets_past_32_bits():
    """Tokens more than 2^32 bytes apart."""
    buf = torch.empty(5 << 29, dtype=torch.bfloat16, device="cuda")  # 5 GiB
    q = buf.as_strided((5, 2, 64), (1 << 29, 64, 1))
    g = torch.Generator().manual_seed(7)
    q.copy_(torch.randn(5, 2, 64, generator=g).bfloat16())
    pos = torch.arange(5, dtype=torch.int32, device="cuda")[:, None]
    freqs = lb.rope_freqs((64,))
    small = q.contiguous()
    want, _ = lb.qk_norm_rope(small, small, pos, freqs, (64,))
    got, _ = lb.qk_norm_rope(q, small, pos, freqs, (64,))
    assert torch.equal(got, want)
    lb.qk_norm_rope(q, small, pos, freqs, (64,), q_out=q)
    assert torch.equal(q, want)


def test_more_tokens_than_a_launch_has_waves():
    """2^26 + 77 tokens, one head of 32 each (the input is one row, read again for every token)."""
    T = (1 << 26) + 77
    g = torch.Generator().manual_seed(9)
    row = torch.randn(1, 1, 32, generator=g).bfloat16().cuda()
    none = row.new_empty(T, 0, 32)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[:, None] % 4099
    freqs = lb.rope_freqs((32,))
    got, _ = lb.qk_norm_rope(row.expand(T, 1, 32), none, pos, freqs, (32,))
    first = torch.arange(300, device="cuda")
    for at in (first, first + (1 << 25), first + (1 << 26) - 270, first + T - 300):
        q = row.expand(300, 1, 32)
        want, _ = lb.qk_norm_rope(q, none[:300], pos[at], freqs, (32,))
        assert torch.equal(got[at], want)


def test_on_another_stream():
    q, k, w, pos, freqs = make(300, 8, 8, 128, (128,), seed=8)
    want = lb.qk_norm_rope(q, k, pos, freqs, (128,), *w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = lb.qk_norm_rope(q, k, pos, freqs, (128,), *w)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
