"""Writing rows into the paged cache and reading them back, against the definition.

Codes, scales and smallest values are exact: fp32 products and divisions are correctly rounded on both sides and rint goes to even.  A row
reads back as its value rounded to bf16 (8 bits: the product of a bf16 and a code is exact in fp32, so one rounding; 4 bits: s u
is exact, s u + b is rounded to fp32 and then to bf16), which numpy repeats to the bit.
"""
import numpy as np
import pytest
import torch

import binary_bit_gemm_amd as lb
from tests import cache_reference as R

pytestmark = pytest.mark.gpu


def rows(tokens, heads, dim, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(tokens, heads, dim, generator=g) * scale).bfloat16().cuda()


def slots_of(n, pages, page, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages * page, generator=g)[:n].to(torch.int32).cuda()


def read_back(x, bits):
    """bf16 tensor -> what its rows read back as, as bf16."""
    return torch.from_numpy(R.stands_for(R.bf16(x), bits).astype(np.float32)).bfloat16()


def same(got, want):
    got, want = got.cpu(), want.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(got.float(), nan=0.0), torch.nan_to_num(want.float(), nan=0.0))


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens,heads,page,pages", [(1, 1, 16, 1), (3, 2, 32, 2), (67, 8, 16, 9), (255, 3, 64, 5), (1000, 5, 256, 4)])
def test_round_trip(bits, dim, tokens, heads, page, pages):
    cache = lb.kv_cache(pages, heads, dim, bits, page)
    k, v = rows(tokens, heads, dim, 1), rows(tokens, heads, dim, 2, 30.0)
    slots = slots_of(tokens, pages, page)
    lb.cache_write(cache, k, v, slots)
    ko, vo = lb.cache_read(cache, slots)
    same(ko, read_back(k, bits))
    same(vo, read_back(v, bits))


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
def test_layout(bits, dim):
    """Every byte of the cache: written rows where the layout puts them, all else untouched."""
    heads, page, pages, tokens = 3, 32, 4, 50
    cache = lb.kv_cache(pages, heads, dim, bits, page)
    for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
        if t is not None:
            t.view(torch.uint8).fill_(0xA5)
    k, v = rows(tokens, heads, dim, 3), rows(tokens, heads, dim, 4)
    slots = slots_of(tokens, pages, page, 5)
    lb.cache_write(cache, k, v, slots)
    T = R.v_block(dim, bits)
    want = {}
    for name, x in (("k", k), ("v", v)):
        row = dim * bits // 8
        codes = np.full((pages, heads, page, row), 0xA5, np.uint8)
        blocks = codes.reshape(pages, heads, page // T, 16, T, row // 16)
        scales = np.full((pages, heads, page, {16: 0, 8: 2, 4: dim // 16}[bits]), 0xA5, np.uint8)
        for i, slot in enumerate(slots.tolist()):
            at, w = slot // page, slot % page
            for h in range(heads):
                if bits == 16:
                    units = x[i, h].cpu().view(torch.uint8).numpy()
                    codes[at, h, w] = units if name == "k" else codes[at, h, w]
                    pieces = units.reshape(16, -1)
                else:
                    q, s, low = R.quantise(R.bf16(x[i, h]), bits)
                    pieces = R.v_pieces(q, bits)
                    if name == "k":
                        codes[at, h, w] = R.k_units(q, bits)
                    both = s if bits == 8 else np.stack([s, low], -1).reshape(-1)
                    scales[at, h, w] = (both.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16).view(np.uint8)
                if name == "v":
                    blocks[at, h, w // T, :, w % T] = pieces
        want[name], want[name + "_scales"] = codes, scales
    for name in ("k", "v"):
        assert np.array_equal(getattr(cache, name).view(torch.uint8).cpu().numpy().reshape(-1), want[name].reshape(-1)), name
        if bits != 16:
            got = getattr(cache, name + "_scales").view(torch.uint8).cpu().numpy()
            assert np.array_equal(got.reshape(-1), want[name + "_scales"].reshape(-1)), name


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_strides_padding_and_rows_left_alone(bits):
    """Views of a fused projection, rows without a slot, outputs with strides: nothing else is written."""
    tokens, heads, dim, page, pages = 41, 4, 128, 16, 6
    qkv = rows(tokens, 3 * heads, dim, 6)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    slots = slots_of(tokens, pages, page, 7)
    slots[3] = -1
    slots[17] = pages * page        # one past the last
    slots[40] = -2 ** 31
    cache = lb.kv_cache(pages, heads, dim, bits, page)
    before = [t.clone() for t in (cache.k, cache.v)]
    lb.cache_write(cache, k, v, slots)
    wide = torch.full((tokens, 2 * heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    ko, vo = wide[:, :heads], torch.full((heads, tokens, dim), 9.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    lb.cache_read(cache, slots, k_out=ko, v_out=vo)
    live = torch.ones(tokens, dtype=torch.bool)
    live[[3, 17, 40]] = False
    same(ko[live.cuda()], read_back(k, bits)[live])
    same(vo[live.cuda()], read_back(v, bits)[live])
    assert (ko[~live.cuda()] == 7).all() and (vo[~live.cuda()] == 9).all() and (wide[:, heads:] == 7).all()
    other = torch.ones(pages * page, dtype=torch.bool)
    other[slots[live.cuda()].cpu().long()] = False
    ks = cache.k.transpose(1, 2).reshape(pages * page, -1).cpu()
    assert torch.equal(ks[other], before[0].transpose(1, 2).reshape(pages * page, -1).cpu()[other])


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
def test_awkward_values(bits, dim):
    """Zeros, constants, subnormals, the largest values, ties, infinities and NaN, which stay in their row (4 bits: their group)."""
    big = torch.finfo(torch.bfloat16).max
    x = torch.zeros(14, 1, dim)
    x[1] = 3.25
    x[2] = -3.25
    x[3] = torch.linspace(-1e-40, 1e-40, dim)
    x[4, 0, ::2] = big
    x[4, 0, 1::2] = -big
    x[5, 0, 7] = float("inf")
    x[6, 0, dim - 1] = float("nan")
    x[7, 0, 0] = -float("inf")
    x[8] = torch.arange(dim) - 0.5        # quotients halfway between codes
    x[9] = torch.arange(dim) * 0.5 - 31.75
    x[10, 0, 5] = 1e-38
    x[11] = torch.where(torch.arange(dim) % 3 == 0, 127.0, 0.5)
    x[12] = torch.where(torch.arange(dim) % 2 == 0, big, 1.0)
    x[13] = torch.randn(dim, generator=torch.Generator().manual_seed(1)) * 1e30
    x = x.bfloat16().cuda()
    cache = lb.kv_cache(1, 1, dim, bits, 16)
    slots = torch.arange(14, dtype=torch.int32, device="cuda")
    lb.cache_write(cache, x, x.flip(0).contiguous(), slots)
    ko, vo = lb.cache_read(cache, slots)
    with np.errstate(invalid="ignore", over="ignore"):
        want = read_back(x, bits)
    same(ko, want)
    same(vo, want.flip(0))


def test_nothing_to_do():
    cache = lb.kv_cache(2, 2, 64, 8, 16)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int32, device="cuda")
    lb.cache_write(cache, none, none, slots)
    assert lb.cache_read(cache, slots)[0].shape == (0, 2, 64)
    empty = lb.kv_cache(0, 2, 64, 8, 16)
    x = rows(3, 2, 64)
    lb.cache_write(empty, x, x, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert (lb.cache_read(empty, torch.zeros(3, dtype=torch.int32, device="cuda"))[0] == 0).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_more_rows_than_one_grid(bits):
    """A head per 4099 and more blocks of tokens than workgroups are launched for: each takes several turns."""
    tokens, heads, dim, page = 8300, 4099, 64, 16
    pages = -(-tokens // page)
    assert -(-tokens // 32) * heads > 1 << 20
    one = rows(tokens, 1, dim, 12)
    slots = torch.arange(tokens, dtype=torch.int32, device="cuda")
    cache = lb.kv_cache(pages, heads, dim, bits, page)
    lb.cache_write(cache, one.expand(-1, heads, -1), one.flip(0).contiguous().expand(-1, heads, -1), slots)
    want = [read_back(x, bits) for x in (one, one.flip(0))]
    for at in (torch.arange(40), torch.arange(tokens - 40, tokens), torch.randint(0, tokens, (40,), generator=torch.Generator().manual_seed(1))):
        for got, w in zip(lb.cache_read(cache, at.to(torch.int32).cuda()), want):
            assert (got == got[:, :1]).all()
            same(got[:, :1], w[at])
    out = torch.zeros(tokens, heads, dim, dtype=torch.bfloat16, device="cuda")
    k, _ = lb.cache_read(cache, slots, k_out=out, v_out=torch.zeros_like(out))
    assert (k == k[:, :1]).all()
    same(k[:, :1], want[0])
