"""A causal layer on affine 4-bit weights that answers requests from a paged, quantised cache: prompts, one token of many requests, and a
tree of drafted tokens.

    python examples/affine_decode_layer.py [--bits 8] [--requests 8] [--cached-tokens 4096] [--drafted 12] [--check]

A decoded token of each request (or the drafted tokens of one), at most 16 rows together:

    QKV      lowbit_gemv_affine        every weight read once for all rows
    norm     lowbit_qk_norm_rope       q and k by their tokens' positions (a drafted token's: its depth in the tree)
    store    lowbit_cache_write        the rows' keys and values, quantised, into their requests' pages
    mixing   lowbit_cache_attention    each request's pages, to its own length; drafted tokens see their ancestors
    output   lowbit_gemv_affine        added to the residual stream
    MLP      lowbit_gemv_affine        gate and up with SwiGLU, then down, added to the stream

A prompt (or the next chunk of one) takes lowbit_gemm_affine for its linears, and lowbit_attention over what lowbit_cache_read gives back: the
same values that the decoded tokens will see.

Weights and activations are random (there are no checkpoints here).
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import binary_bit_gemm_amd as lb  # noqa: E402

G = 64


class Linear:
    """[n, k] weights scale * level + bias per 64 of them, and their levels for checks."""

    def __init__(self, n, k, gen):
        self.levels = torch.randint(0, 16, (n, k), generator=gen, device="cuda").to(torch.uint8)
        self.scales = ((torch.rand(n, k // G, generator=gen, device="cuda") * 0.2 + 0.1) / math.sqrt(k)).half()
        self.biases = (-7.5 * self.scales.float()).half()
        self.words, _ = lb.pack_u4(self.levels, count_invalid=False)

    def __call__(self, x, **kw):
        return lb.gemv_affine(x, self.words, self.scales, self.biases, G, **kw)

    def many(self, x):
        return lb.gemm_affine(x, self.words, self.scales, self.biases, G)

    def dense(self):
        wide = lambda t: t.double().repeat_interleave(G, 1)  # noqa: E731
        return self.levels.double() * wide(self.scales) + wide(self.biases)


class Layer:
    def __init__(self, dim, heads, kv_heads, inner, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dim, self.heads, self.kv_heads, self.inner = dim, heads, kv_heads, inner
        self.qkv, self.out = Linear(128 * (heads + 2 * kv_heads), dim, gen), Linear(dim, 128 * heads, gen)
        self.gate_up, self.down = Linear(2 * inner, dim, gen), Linear(dim, inner, gen)
        weight = lambda n: (1 + 0.1 * torch.randn(n, generator=gen, device="cuda")).bfloat16()  # noqa: E731
        self.norm, self.qk_norm = (weight(dim), weight(dim)), (weight(128), weight(128))
        self.freqs = lb.rope_freqs((128,))


class Requests:
    """The cache's pages, which of them each request has, and how many tokens it holds."""

    def __init__(self, layer, count, capacity, bits, page=64, seed=0):
        each = -(-capacity // page)
        self.cache = lb.kv_cache(count * each, layer.kv_heads, 128, bits, page)
        order = torch.randperm(count * each, generator=torch.Generator().manual_seed(seed))
        self.table = order.view(count, each).to(torch.int32).cuda()
        self.filled = torch.zeros(count, dtype=torch.int32, device="cuda")
        self.drafted = {}  # request -> keys and values of the tokens that verify() last took

    def slots(self, request, index):
        """Slots of tokens `index` (int64 tensor) of requests `request` (the same shape, or one)."""
        page = self.cache.shape[2]
        return self.table[request, index // page] * page + (index % page).int()


def project(layer, x, positions, linear):
    """The rows' q, k and v [rows, heads, 128] after their norms and rotation."""
    heads, kv = layer.heads, layer.kv_heads
    h = torch.nn.functional.rms_norm(x, (layer.dim,), layer.norm[0], 1e-6)
    qkv = linear(h).view(-1, heads + 2 * kv, 128)
    q, k, v = qkv.split([heads, kv, kv], 1)
    lb.qk_norm_rope(q, k, positions[:, None], layer.freqs, (128,), *layer.qk_norm, interleaved=False, q_out=q, k_out=k)
    return q, k, v


def prompt(layer, requests, r, x):
    """x: bf16 [tokens, dim], the next tokens of request r.  Stores their keys and values and returns their rows of the stream."""
    tokens, done = x.shape[0], int(requests.filled[r])
    index = torch.arange(done + tokens, device="cuda")
    q, k, v = project(layer, x, index[done:].int(), layer.qkv.many)
    lb.cache_write(requests.cache, k, v, requests.slots(r, index[done:]))
    keys, values = lb.cache_read(requests.cache, requests.slots(r, index))
    start = torch.tensor([done], dtype=torch.int32, device="cuda")
    mixed = lb.attention(q[None], keys[None], values[None], causal=True, q_start=start)
    x = x + layer.out.many(mixed.view(tokens, -1))
    h = torch.nn.functional.rms_norm(x, (layer.dim,), layer.norm[1], 1e-6)
    gate, up = layer.gate_up.many(h).chunk(2, 1)
    requests.filled[r] += tokens
    return x + layer.down.many(torch.nn.functional.silu(gate.float()).mul(up.float()).bfloat16())


def finish(layer, x, mixed):
    x = layer.out(mixed.view(x.shape[0], -1), residual=x)
    h = torch.nn.functional.rms_norm(x, (layer.dim,), layer.norm[1], 1e-6)
    return layer.down(layer.gate_up(h, swiglu=True), residual=x)


def decode(layer, requests, x, workspace, out=None):
    """x: bf16 [requests, dim], one new token of each.  All on the device, so it can be captured."""
    q, k, v = project(layer, x, requests.filled, layer.qkv)
    each = torch.arange(x.shape[0], device="cuda")
    lb.cache_write(requests.cache, k, v, requests.slots(each, requests.filled.long()))
    mixed = lb.cache_attention(q[:, None], requests.cache, requests.table, requests.filled + 1, workspace=workspace)
    requests.filled += 1
    return finish(layer, x, mixed)


def verify(layer, requests, r, x, tree, depth, workspace):
    """x: bf16 [drafted, dim], drafted tokens of request r; tree: int64 [drafted], bit i for ancestor i and the token itself; depth: int32 [drafted].
    Their rows of the stream; the request's length stays (the caller keeps the accepted ones, with keep())."""
    n = x.shape[0]
    q, k, v = project(layer, x, requests.filled[r] + depth, layer.qkv)
    slots = requests.slots(r, requests.filled[r].long() + torch.arange(n, device="cuda"))
    lb.cache_write(requests.cache, k, v, slots)
    requests.drafted[r] = k, v
    mixed = lb.cache_attention(q[None], requests.cache, requests.table[r:r + 1], requests.filled[r:r + 1] + n, tree=tree[None], workspace=workspace)
    return finish(layer, x, mixed)


def keep(requests, r, path):
    """The accepted ones of the tokens that verify() last took (a path of the tree, int64 indices) to where the request's next tokens belong: their keys
    and values are written there once more.  Codes depend on these alone, so the rows are those that verify() attended, to the bit; rows
    read back and written again would be quantised a second time."""
    keys, values = (x[path] for x in requests.drafted[r])
    slots = requests.slots(r, requests.filled[r].long() + torch.arange(len(path), device="cuda"))
    lb.cache_write(requests.cache, keys, values, slots)
    requests.filled[r] += len(path)


def reference(layer, x, positions, keys, values, takes):
    """Rows of the stream in 64 bits from what the cache holds: keys, values [tokens, kv_heads, 128], takes bool [rows, tokens].
    Returns (rows, the rows' own k and v)."""
    rows, heads, kv = x.shape[0], layer.heads, layer.kv_heads
    normed = lambda y, w: y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()  # noqa: E731
    x = x.double()
    qkv = (normed(x, layer.norm[0]) @ layer.qkv.dense().T).view(rows, -1, 128)
    q, k, v = qkv.split([heads, kv, kv], 1)
    angle = positions.double()[:, None, None] * layer.freqs.double()
    turned = []
    for y, w in zip((q, k), layer.qk_norm):
        y = normed(y, w)
        turned.append(torch.cat([y[..., :64] * angle.cos() - y[..., 64:] * angle.sin(), y[..., :64] * angle.sin() + y[..., 64:] * angle.cos()], -1))
    keys, values = (t.double().repeat_interleave(heads // kv, 1).transpose(0, 1).contiguous() for t in (keys, values))
    s = (turned[0].transpose(0, 1) @ keys.transpose(1, 2).contiguous() / math.sqrt(128)).masked_fill(~takes, -math.inf)
    x = x + (torch.softmax(s, -1) @ values).transpose(0, 1).reshape(rows, -1) @ layer.out.dense().T
    gate, up = (normed(x, layer.norm[1]) @ layer.gate_up.dense().T).chunk(2, 1)
    return x + (torch.nn.functional.silu(gate) * up) @ layer.down.dense().T, turned[1], v


def stored(requests, r, tokens):
    return lb.cache_read(requests.cache, requests.slots(r, torch.arange(tokens, device="cuda")))


def draft(tokens, seed=0):
    """A random tree: (bits of ancestors and itself int64, depth int32, a deepest path int64)."""
    gen = torch.Generator().manual_seed(seed)
    parent = [-1] + [int(torch.randint(0, i, (1,), generator=gen)) for i in range(1, tokens)]
    bits, depth, paths = [], [], []
    for i, p in enumerate(parent):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
        paths.append((paths[p] if p >= 0 else []) + [i])
    cuda = lambda x, t: torch.tensor(x, dtype=t, device="cuda")  # noqa: E731
    return cuda(bits, torch.int64), cuda(depth, torch.int32), cuda(max(paths, key=len), torch.int64)


def scratch(layer, requests, rows):
    """A workspace for one token of any number of requests, or any number of drafted tokens of one, up to `rows`."""
    q = torch.empty(rows, 1, layer.heads, 128, dtype=torch.bfloat16, device="cuda")
    capacity = requests.table.shape[1] * requests.cache.shape[2]
    need = max(lb.cache_attention_workspace_size(x, requests.cache, capacity) for n in range(1, rows + 1) for x in (q[:n], q[:n].transpose(0, 1)))
    return torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--bits", type=int, default=8, choices=(4, 8, 16), help="of the cache")
    ap.add_argument("--requests", type=int, default=8, help="up to 16")
    ap.add_argument("--cached-tokens", type=int, default=4096)
    ap.add_argument("--drafted", type=int, default=12, help="tokens of a drafted tree, up to 16")
    ap.add_argument("--dim", type=int, default=2560)
    ap.add_argument("--inner", type=int, default=9728)
    ap.add_argument("--check", action="store_true", help="compare with the same computation in 64 bits")
    a = ap.parse_args()
    layer = Layer(a.dim, 32, 8, a.inner)
    requests = Requests(layer, a.requests, a.cached_tokens + 80, a.bits)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = lambda n: torch.randn(n, a.dim, generator=gen, device="cuda").bfloat16()  # noqa: E731
    for r in range(a.requests):
        prompt(layer, requests, r, rows(a.cached_tokens))
    workspace = scratch(layer, requests, max(a.requests, a.drafted))
    tree, depth, _ = draft(a.drafted)
    x, drafted = rows(a.requests), rows(a.drafted)
    steps = {f"one token of {a.requests} requests": lambda: decode(layer, requests, x, workspace),
             f"{a.drafted} drafted tokens of one": lambda: verify(layer, requests, 0, drafted, tree, depth, workspace)}
    for name, step in steps.items():
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graph.replay()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(20):
            graph.replay()
        torch.cuda.synchronize()
        print(f"{name}, {a.cached_tokens} cached tokens in {a.bits} bits, hidden size {a.dim}: {(time.perf_counter() - t) * 5e4:.0f} us")
    if a.check:
        n = int(requests.filled[0])
        got = verify(layer, requests, 0, drafted, tree, depth, workspace)
        takes = torch.ones(a.drafted, n + a.drafted, dtype=torch.bool, device="cuda")
        takes[:, n:] = (tree[:, None] >> torch.arange(a.drafted, device="cuda")) & 1 == 1
        want = reference(layer, drafted, n + depth, *stored(requests, 0, n + a.drafted), takes)[0]
        print(f"relative error against 64 bits {float((got.double() - want).norm() / want.norm()):.2e}")


if __name__ == "__main__":
    main()
