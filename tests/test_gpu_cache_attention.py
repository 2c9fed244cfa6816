"""Attention over the paged cache against the formula in 64 bits, on the values that the written rows stand for.

Tolerance, per element of O = sum_j p_j v_j, with A = sum_j p_j M_j and M_j what stands behind v_j in the second product (16 bits: |v|; 8
bits: s |code|; 4 bits: s u + |b|, of which u is multiplied and b added in fp32):
  * p s is rounded to fp16, 2^-11 of it (16 bits: p to bf16, 2^-8); below fp16's normal range by 2^-25 of the row's largest p s instead, which is
    kept within 2^8 of 1: 2^-17 of the largest p s for each code unit (8 bits: the sum that is taken off again carries the same rounding);
  * scores are fp32 sums of D products and what is added to them: (D + 8) 2^-24 of sum_d |q_d| (|k's code| + offset) s at most, which moves p by that
    factor of itself (and the normalising sum as much);
  * the sums over keys, the exponentials and the divisions: 2^-12 of A (8 bits: of A + 128 sum p s, since codes are summed with their offset) covers
    the chains here, fewer than 2000 additions for any lane;
  * the result is rounded once: 2^-8 of it.
"""
import functools
import math

import numpy as np
import pytest
import torch

import binary_bit_gemm_amd as lb
from tests import cache_reference as R

pytestmark = pytest.mark.gpu


class Problem:
    """Requests with their keys and values written through the cache, in pages that lie anywhere."""

    def __init__(self, lens, q_lens, q_heads, kv_heads, dim, bits, page, tree=None, seed=0, kv_len=None, scale_k=1.0, scale_v=1.0, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.q_lens, self.hq, self.hk, self.dim, self.bits, self.page = lens, q_lens, q_heads, kv_heads, dim, bits, page
        self.B, self.q_len = len(lens), max(q_lens)
        self.kv_len = kv_len if kv_len is not None else max(max(lens), 1)
        each = -(-self.kv_len // page)
        pages = self.B * each + spare
        order = torch.randperm(pages, generator=g)
        self.table = order[:self.B * each].view(self.B, each).to(torch.int32).cuda()
        self.cache = lb.kv_cache(pages, kv_heads, dim, bits, page)
        for t in (self.cache.k, self.cache.v, self.cache.k_scales, self.cache.v_scales):
            if t is not None:
                t.view(torch.uint8).fill_(0xFF)  # what nobody wrote: NaN scales, NaN elements
        self.q = torch.randn(self.B, self.q_len, q_heads, dim, generator=g).bfloat16().cuda()
        self.k = [(torch.randn(n, kv_heads, dim, generator=g) * scale_k).bfloat16() for n in lens]
        self.v = [(torch.randn(n, kv_heads, dim, generator=g) * scale_v).bfloat16() for n in lens]
        self.tree, self.answers = tree, {}
        self.write()

    def write(self):
        for b in range(self.B):
            n = self.lens[b]
            if n == 0:
                continue
            at = torch.arange(n)
            slots = (self.table[b].cpu()[at // self.page] * self.page + at % self.page).to(torch.int32).cuda()
            lb.cache_write(self.cache, self.k[b].cuda(), self.v[b].cuda(), slots)

    def call(self, workspace="enough", out=None, scale=None, kv_len=None):
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        tree = None
        if self.tree is not None:
            tree = torch.from_numpy(np.array(self.tree, dtype=np.uint64).view(np.int64).copy()).cuda()
        ws = None
        if workspace == "enough":
            n = lb.cache_attention_workspace_size(self.q, self.cache, kv_len or self.kv_len)
            ws = torch.full((max(n, 16),), 0xAB, dtype=torch.uint8, device="cuda")
            ws[:4096] = 0
        ragged = any(x != self.q_len for x in self.q_lens)
        got = lb.cache_attention(self.q, self.cache, self.table, dev(self.lens), q_lens=dev(self.q_lens) if ragged else None, tree=tree,
                                 kv_len=kv_len or self.kv_len, scale=scale, out=out, workspace=ws)
        if ws is not None:
            assert (ws[:4096] == 0).all(), "the arrival counters are zero again"
        return got

    def wanted(self, scale):
        """(request, head) -> what the formula gives and how far from it a result may lie; once per problem and scale."""
        if scale in self.answers:
            return self.answers[scale]
        answers = {}
        for b in range(self.B):
            n = self.lens[b]
            takes = R.taken(n, self.q_lens[b], self.q_len, None if self.tree is None else self.tree[b])
            for hk in range(self.hk):
                k, v = (R.stands_for(R.bf16(x[b][:, hk]), self.bits).reshape(n, self.dim) for x in (self.k, self.v))
                kmag, vmag, unit = np.abs(k), np.abs(v), np.zeros((n, self.dim))
                if self.bits == 8 and n:
                    ks, vs = (R.quantise(R.bf16(x[b][:, hk]), 8)[1] for x in (self.k, self.v))
                    kmag, unit = kmag + 256 * ks, np.broadcast_to(vs, (n, self.dim))
                if self.bits == 4 and n:
                    (kq, ks, kl), (vq, vs, vl) = (R.quantise(R.bf16(x[b][:, hk]), 4) for x in (self.k, self.v))
                    rep = lambda x: np.repeat(x, R.GROUP, -1)  # noqa: E731
                    kmag, vmag, unit = kq * rep(ks) + np.abs(rep(kl)), vq * rep(vs) + np.abs(rep(vl)), rep(vs)
                for h in range(hk * self.hq // self.hk, (hk + 1) * self.hq // self.hk):
                    q = R.bf16(self.q[b, :, h])
                    want, _, p = R.attend(q, k, v, takes, scale)
                    shift = (self.dim + 8) * 2.0 ** -24 * scale * (np.abs(q) @ kmag.T).max(initial=0)
                    A = p @ vmag
                    most = {16: 0, 8: 255, 4: 15}[self.bits]
                    floor = 2.0 ** -17 * most * (p @ unit if n else 0)
                    rounding = 2.0 ** -8 if self.bits == 16 else 2.0 ** -11
                    sums = 2.0 ** -12 * (A + (128 * (p @ unit) if self.bits == 8 else 0))
                    bound = (rounding + 2 * shift) * (A + (128 * (p @ unit) if self.bits == 8 else 0)) + floor + sums + 2.0 ** -8 * np.abs(want)
                    answers[b, h] = want, bound
        self.answers[scale] = answers
        return answers

    def check(self, got, scale=None, rows=None):
        """rows: (request) -> the new tokens to look at (bool [q_len])."""
        got = R.bf16(got)
        for (b, h), (want, bound) in self.wanted(scale if scale is not None else 1 / math.sqrt(self.dim)).items():
            live = np.arange(self.q_len) < self.q_lens[b]
            live = live if rows is None else live & rows(b)
            off = np.abs(got[b, live, h] - want[live]) - bound[live]
            assert np.isfinite(got[b, live, h]).all()
            assert off.max(initial=-1) <= 0, f"request {b}, head {h}: over its bound by {off.max()}"


@functools.lru_cache(maxsize=None)
def problem_of(lens, q_lens, hq, hk, dim, bits, page, tree=None, seed=0):
    return Problem(lens, q_lens, hq, hk, dim, bits, page, tree=tree, seed=seed)


@pytest.fixture(params=["few", "many32", "many64", "many128", "auto"])
def kernel(request, monkeypatch):
    """Each of the kernels in turn (many rows: 32, 64 and 128 per workgroup), and the one that the library takes."""
    if request.param != "auto":
        monkeypatch.setenv("LOWBIT_CACHE_ATTENTION", request.param)
    return request.param


SHAPES = [  # lens, q_lens, q heads, kv heads, page
    ([1], [1], 1, 1, 16), ([17], [1], 8, 2, 16), ([33, 1, 64], [1, 1, 1], 4, 4, 32), ([500, 3, 0, 129], [1, 1, 1, 1], 8, 1, 64),
    ([2000], [1], 16, 2, 16), ([40, 31], [5, 2], 6, 3, 16), ([300], [9], 4, 2, 128), ([257, 90], [40, 33], 5, 1, 256), ([3000], [1], 2, 2, 64),
    ([70], [70], 2, 1, 32), ([20, 5], [3, 7], 4, 2, 16),
]


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, dim, bits, kernel):
    lens, q_lens, hq, hk, page = shape
    p = problem_of(tuple(lens), tuple(q_lens), hq, hk, dim, bits, page)
    for ws in ("enough", None):
        p.check(p.call(ws))


def random_tree(n, seed):
    rng = np.random.default_rng(seed)
    bits = [1]
    for i in range(1, n):
        bits.append(bits[int(rng.integers(0, i))] | 1 << i)
    return bits


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,nodes,hq,hk,page", [([100], 64, 4, 1, 16), ([77, 1000, 30], 27, 8, 4, 32), ([64], 64, 2, 2, 64), ([45, 6], 6, 1, 1, 16),
                                                   ([2500], 33, 8, 2, 128)])
def test_trees(lens, nodes, hq, hk, page, dim, bits, kernel):
    trees = tuple(tuple(random_tree(nodes, s)) for s in range(len(lens)))
    p = problem_of(tuple(lens), (nodes,) * len(lens), hq, hk, dim, bits, page, trees, 3)
    for ws in ("enough", None):
        p.check(p.call(ws))
