"""A causal layer on affine 4-bit weights and a paged, quantised cache (examples/affine_decode_layer.py): prompts in chunks, decoded tokens of several
requests, a drafted tree and what is kept of it, against the same computation in 64 bits.

The reference takes keys and values as the cache holds them, and checks the rows that were written against its own.  Tolerances, as relative norms:
  * a row of the stream: rounded to bf16 on the way are the normed stream (twice), QKV, the turned q, the mixed values, the stream after the output
    linear, the MLP's inner values and the result, 2^-9 of the norm each if roundings spread evenly, 2^-8 at most; q off by 3 * 2^-8 (norm, QKV, turned)
    moves the scores by a few units of that and the probabilities by a few per cent at most: 8 * 2^-8 for the roundings and as much for the scores;
  * k: three roundings to bf16 before the cache (normed stream, QKV, turned), v: two; then the cache's step.  A step is at most
    4.5 sigma / 127 * (1 + 2^-7) of 128 elements' largest (8 bits), or 9 sigma / 15 (4 bits); evenly spread, its rounding has a norm of step / sqrt(12):
    below 2^-6 of sigma, below 2^-2.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "affine_decode_layer.py")
STREAM = 16 * 2.0 ** -8
STEP = {16: 0.0, 8: 2.0 ** -6, 4: 2.0 ** -2}


def load():
    spec = importlib.util.spec_from_file_location("affine_decode_layer", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def apart(got, want):
    assert bool(torch.isfinite(got).all())
    return float((got.double() - want).norm() / want.norm())


def check_rows(m, layer, requests, r, x, positions, takes, got, bits, new):
    """`got` of the tokens x of request r, whose keys are the last `new` of takes.shape[1]."""
    tokens = takes.shape[1]
    keys, values = m.stored(requests, r, tokens)
    want, k, v = m.reference(layer, x, positions, keys, values, takes)
    assert apart(got, want) <= STREAM
    assert apart(keys[tokens - new:], k) <= 3 * 2.0 ** -8 + STEP[bits] and apart(values[tokens - new:], v) <= 3 * 2.0 ** -8 + STEP[bits]


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dim,heads,kv,inner,page", [(256, 4, 2, 512, 16), (512, 8, 1, 832, 64), (192, 3, 3, 320, 256)])
def test_prompts_tokens_and_drafts(dim, heads, kv, inner, page, bits):
    m = load()
    layer = m.Layer(dim, heads, kv, inner, seed=5)
    requests = m.Requests(layer, 3, 700, bits, page)
    gen = torch.Generator(device="cuda").manual_seed(6)
    rows = lambda n: torch.randn(n, dim, generator=gen, device="cuda").bfloat16()  # noqa: E731
    ws = m.scratch(layer, requests, 13)
    lower = lambda rows, tokens: torch.ones(rows, tokens, dtype=torch.bool, device="cuda").tril(tokens - rows)  # noqa: E731
    for r, chunks in enumerate([(37,), (1,), (500, 70)]):
        done = 0
        for n in chunks:
            x = rows(n)
            got = m.prompt(layer, requests, r, x)
            done += n
            check_rows(m, layer, requests, r, x, torch.arange(done - n, done, device="cuda"), lower(n, done), got, bits, n)
    for _ in range(3):
        x = rows(3)
        before = requests.filled.clone()
        got = m.decode(layer, requests, x, ws)
        for r in range(3):
            n = int(before[r]) + 1
            check_rows(m, layer, requests, r, x[r:r + 1], before[r:r + 1], lower(1, n), got[r:r + 1], bits, 1)
    for r in range(3):
        tree, depth, path = m.draft(13, seed=r)
        x, n = rows(13), int(requests.filled[r])
        got = m.verify(layer, requests, r, x, tree, depth, ws)
        takes = lower(13, n + 13)
        takes[:, n:] = (tree[:, None] >> torch.arange(13, device="cuda")) & 1 == 1
        check_rows(m, layer, requests, r, x, n + depth, takes, got, bits, 13)
        drafted = m.stored(requests, r, n + 13)
        m.keep(requests, r, path)
        assert int(requests.filled[r]) == n + len(path)
        for was, now in zip(drafted, m.stored(requests, r, n + len(path))):
            assert torch.equal(now[:n], was[:n])
            # read back and stored again: once more to bf16 and half a step; at 16 bits the same
            again = apart(now[n:], was[n:][path].double())
            assert again <= (0 if bits == 16 else 2.0 ** -8 + STEP[bits])
    assert (ws[:4096] == 0).all()


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_decoding_as_a_graph(bits):
    """Captured once and replayed for every token: the device's own lengths lead, with eager work between."""
    m = load()
    layer = m.Layer(256, 4, 2, 512, seed=7)
    gen = torch.Generator(device="cuda").manual_seed(8)
    rows = lambda n: torch.randn(n, 256, generator=gen, device="cuda").bfloat16()  # noqa: E731
    prompts, tokens = [rows(n) for n in (90, 600)], [rows(2) for _ in range(6)]
    eager, graphed = (m.Requests(layer, 2, 700, bits) for _ in range(2))
    ws = m.scratch(layer, eager, 2)
    for r in range(2):
        for requests in (eager, graphed):
            m.prompt(layer, requests, r, prompts[r])
    want = [m.decode(layer, eager, x, ws) for x in tokens]
    x = tokens[0].clone()
    start = graphed.filled.clone()
    m.decode(layer, graphed, x, ws)  # (its slots are written again)
    graphed.filled.copy_(start)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.decode(layer, graphed, x, ws)
    for i, token in enumerate(tokens):
        x.copy_(token)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        m.stored(graphed, 1, 600)
    assert torch.equal(graphed.filled, eager.filled)


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_kept_drafts_hold_what_was_verified(bits):
    """Rows of accepted drafted tokens, once moved to their places, are the rows that verify() attended, to the bit: quantised once, from the same keys
    and values."""
    m = load()
    layer = m.Layer(256, 4, 2, 512, seed=9)
    requests = m.Requests(layer, 2, 300, bits)
    gen = torch.Generator(device="cuda").manual_seed(10)
    rows = lambda n: torch.randn(n, 256, generator=gen, device="cuda").bfloat16()  # noqa: E731
    ws = m.scratch(layer, requests, 13)
    for r, n in enumerate((40, 129)):
        m.prompt(layer, requests, r, rows(n))
    for turn in range(2):
        for r in range(2):
            tree, depth, path = m.draft(13, seed=11 + 2 * r + turn)
            n = int(requests.filled[r])
            m.verify(layer, requests, r, rows(13), tree, depth, ws)
            drafted = m.stored(requests, r, n + 13)
            m.keep(requests, r, path)
            for was, now in zip(drafted, m.stored(requests, r, n + len(path))):
                assert torch.equal(now[:n], was[:n]) and torch.equal(now[n:], was[n:][path])


def test_scratch_serves_fewer_requests():
    """The layer's workspace is enough for every number of requests and drafted tokens up to its rows: what a call can use grows as a batch shrinks."""
    m = load()
    layer = m.Layer(128, 8, 8, 128)
    requests = m.Requests(layer, 1, 4200, 8)
    size = m.scratch(layer, requests, 7).numel()
    assert size <= m.lb.CACHE_ATTENTION_WORKSPACE_BYTES
    for rows in range(1, 8):
        q = torch.empty(rows, 1, 8, 128, dtype=torch.bfloat16, device="cuda")
        for x in (q, q.transpose(0, 1)):
            assert m.lb.cache_attention_workspace_size(x, requests.cache, 4200) <= size
