"""The attention half of a double-stream block, and one decoded token of a causal layer, with low-rank adapters of several
requests on packed weights.

    python examples/adapted_attention_block.py [--image-tokens 4096] [--text-tokens 512] [--heads 24] [--check]
    python examples/adapted_attention_block.py --decode [--requests 16] [--cached-tokens 4096] [--check]

In the block every request brings an image stream and a text stream (padded prompt) of one length each and its own adapter:

    QKV      lowbit_gemm_lora       packed ternary QKV linear of the stream + the request's adapter, written
                                    into the request's rows of one joint [text | image] buffer
    norm     lowbit_qk_norm_rope    norms of q and k for each head and the rotation by (frame, row, column, index)
                                    positions, in place in that buffer
    mixing   lowbit_attention       text and image tokens together, padding masked out
    output   lowbit_gemm_residual   packed output linear, gated and added to the residual stream

A decoded token (--decode) is a row of all requests together: one lowbit_gemm_lora per linear takes every row with its own
request's adapter, lowbit_qk_norm_rope turns it by its request's position, and lowbit_attention reads each request's cache to its
own length.

Weights, adapters and activations are random (there are no checkpoints here); the shapes are those of the
FLUX.2 Klein 4B transformer's double-stream blocks by default: hidden size 3072, 24 heads of 128.
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import binary_bit_gemm_amd as lb  # noqa: E402

AXES = (32, 32, 32, 32)  # dimensions of a head that turn with the frame, the row, the column and the index
G, BITS = 64, 2


class Linear:
    """A packed ternary linear [n, k] with a scale per 64 weights, and its codes and scales for checks."""

    def __init__(self, n, k, gen):
        self.codes = (torch.randint(0, 4, (n, k), generator=gen, device="cuda") % 3 - 1).to(torch.int8)
        self.scales = ((torch.rand(n, k // G, generator=gen, device="cuda") * 0.04 + 0.01) * (48 / math.sqrt(k))).half()
        self.words, _ = lb.pack(self.codes, BITS, count_invalid=False)

    def dense(self):
        return self.codes.double() * self.scales.double().repeat_interleave(G, 1)


class Block:
    def __init__(self, heads, adapters, rank, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.dim = heads, 128 * heads
        self.qkv = {s: Linear(3 * self.dim, self.dim, gen) for s in ("text", "image")}
        self.out = {s: Linear(self.dim, self.dim, gen) for s in ("text", "image")}
        rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
        self.a = {s: (rand(adapters, rank, self.dim) / math.sqrt(self.dim)).bfloat16() for s in ("text", "image")}
        self.b = {s: (rand(adapters, 3 * self.dim, rank) * 0.1).bfloat16() for s in ("text", "image")}
        self.alpha = torch.ones(adapters, device="cuda")
        self.norm = {s: tuple((1 + 0.1 * rand(128)).bfloat16() for _ in range(2)) for s in ("text", "image")}
        self.gate = {s: (0.5 * rand(self.dim)).bfloat16() for s in ("text", "image")}
        self.freqs = lb.rope_freqs(AXES, theta=2000.0)


def positions(text, image):
    """int32 [text + image, 4]: the prompt's index; an image's rows and columns (as square as it goes)."""
    p = torch.zeros(text + image, 4, dtype=torch.int32)
    width = max(1, int(math.sqrt(image)))
    i = torch.arange(image, dtype=torch.int32)
    p[:text, 3] = torch.arange(text, dtype=torch.int32)
    p[text:, 1], p[text:, 2] = i // width, i % width
    return p.cuda()


def attention_half(block, x, adapter, mask, pos, workspace):
    """x: {"text": bf16 [requests, text, dim], "image": bf16 [requests, image, dim]}; adapter: int32 [requests] on the host;
    mask: bool [requests, text + image].  Returns the updated streams."""
    requests, text, dim = x["text"].shape
    image, heads = x["image"].shape[1], block.heads
    total = text + image
    qkv = torch.empty(requests, total, 3 * heads, 128, dtype=torch.bfloat16, device="cuda")
    for r in range(requests):
        for s, rows in (("text", slice(0, text)), ("image", slice(text, total))):
            n = rows.stop - rows.start
            lin = block.qkv[s]
            lb.gemm_lora(x[s][r], lin.words, lin.scales, G, BITS, block.a[s], block.b[s], block.alpha,
                         torch.full((n,), int(adapter[r]), dtype=torch.int32, device="cuda"),
                         out=qkv[r, rows].view(n, 3 * dim), workspace=workspace)
            q, k = qkv[r, rows, :heads], qkv[r, rows, heads:2 * heads]
            lb.qk_norm_rope(q, k, pos[rows], block.freqs, AXES, *block.norm[s], q_out=q, k_out=k)
    q, k, v = (qkv[:, :, i * heads:(i + 1) * heads] for i in range(3))
    mixed = lb.attention(q, k, v, key_mask=mask, workspace=workspace).view(requests, total, dim)
    result = {}
    for s, rows in (("text", slice(0, text)), ("image", slice(text, total))):
        lin = block.out[s]
        flat = mixed[:, rows].reshape(-1, dim)
        result[s] = lb.gemm_residual(flat, lin.words, lin.scales, G, BITS, x[s].reshape(-1, dim), block.gate[s]).view(x[s].shape)
    return result


class Layer:
    """The attention half of a causal layer with grouped heads: QKV and output linear, both with adapters, and the caches."""

    def __init__(self, requests, capacity, heads, kv_heads, adapters, rank, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, 128 * heads
        width = 128 * (heads + 2 * kv_heads)
        self.qkv, self.out = Linear(width, self.dim, gen), Linear(self.dim, self.dim, gen)
        rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
        self.a = [(rand(adapters, rank, self.dim) / math.sqrt(self.dim)).bfloat16() for _ in range(2)]
        self.b = [(rand(adapters, n, rank) * 0.1).bfloat16() for n in (width, self.dim)]
        self.alpha = torch.ones(adapters, device="cuda")
        self.norm = tuple((1 + 0.1 * rand(128)).bfloat16() for _ in range(2))
        self.freqs = lb.rope_freqs((128,))
        self.keys, self.values = (rand(requests, capacity, kv_heads, 128).bfloat16() for _ in range(2))


def decode_step(layer, x, adapter, filled, workspace):
    """x: bf16 [requests, dim], one new token of each; adapter: int32 [requests] (-1: none); filled: int32 [requests], the tokens that
    each cache holds already.  Stores the new keys and values and returns x plus the layer's attention."""
    requests, heads, kv = x.shape[0], layer.heads, layer.kv_heads
    lora = lambda x, lin, i: lb.gemm_lora(x, lin.words, lin.scales, G, BITS, layer.a[i], layer.b[i], layer.alpha, adapter,  # noqa: E731
                                          workspace=workspace)
    qkv = lora(x, layer.qkv, 0).view(requests, heads + 2 * kv, 128)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    lb.qk_norm_rope(q, k, filled[:, None], layer.freqs, (128,), *layer.norm, interleaved=False, q_out=q, k_out=k)
    at = torch.arange(requests, device="cuda"), filled.long()
    layer.keys[at], layer.values[at] = k, v
    mixed = lb.attention(q[:, None], layer.keys, layer.values, key_lens=filled + 1, workspace=workspace)
    return x + lora(mixed.view(requests, -1), layer.out, 1)


def decode_reference(layer, x, adapter, filled):
    """The same in 64 bits from the caches before the step, without the roundings to bf16 in between."""
    group = layer.heads // layer.kv_heads
    dense = layer.qkv.dense(), layer.out.dense()
    result = []
    for r in range(x.shape[0]):
        e, n = int(adapter[r]), int(filled[r])

        def linear(y, i):
            z = dense[i] @ y
            return z if e < 0 else z + float(layer.alpha[e]) * (layer.b[i][e].double() @ (layer.a[i][e].double() @ y))
        qkv = linear(x[r].double(), 0).view(-1, 128)
        q, k, v = qkv.split([layer.heads, layer.kv_heads, layer.kv_heads])
        c, s = (n * layer.freqs.double()).cos(), (n * layer.freqs.double()).sin()
        turned = []
        for y, w in zip((q, k), layer.norm):
            y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
            turned.append(torch.cat([y[:, :64] * c - y[:, 64:] * s, y[:, :64] * s + y[:, 64:] * c], -1))
        keys = torch.cat([layer.keys[r, :n].double(), turned[1][None]]).repeat_interleave(group, 1)
        values = torch.cat([layer.values[r, :n].double(), v[None]]).repeat_interleave(group, 1)
        p = torch.softmax((turned[0] * keys).sum(-1) / math.sqrt(128), 0)  # [tokens, heads]
        result.append(x[r].double() + linear((p[..., None] * values).sum(0).flatten(), 1))
    return torch.stack(result)


def decode_example(requests, capacity, heads, kv_heads, rank=16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer = Layer(requests, capacity, heads, kv_heads, adapters=max(1, requests // 2), rank=rank, seed=seed + 1)
    x = torch.randn(requests, layer.dim, generator=gen, device="cuda").bfloat16()
    adapter = torch.arange(requests, dtype=torch.int32, device="cuda") % (layer.alpha.shape[0] + 1) - 1  # some have none
    filled = torch.randint(0, capacity, (requests,), generator=gen, device="cuda", dtype=torch.int32)
    filled[0] = 0
    return layer, x, adapter, filled


def decode_workspace(layer, requests, rank=16):
    q = torch.empty(requests, 1, layer.heads, 128, dtype=torch.bfloat16, device="cuda")
    need = max(lb.attention_workspace_size(q, layer.keys, layer.values), lb.lora_workspace_size(requests, rank))
    return torch.zeros(need, dtype=torch.uint8, device="cuda")


def reference(block, x, adapter, mask, pos):
    """The same in 64 bits, without the roundings to bf16 in between."""
    requests, text, dim = x["text"].shape
    heads = block.heads
    out = {"text": [], "image": []}
    axis = torch.repeat_interleave(torch.arange(4), torch.tensor([d // 2 for d in AXES])).cuda()
    angle = (pos.double()[:, axis] * block.freqs.double())[:, None]
    for r in range(requests):
        parts = []
        for s in ("text", "image"):
            e = int(adapter[r])
            xs = x[s][r].double()
            y = xs @ block.qkv[s].dense().T
            if e >= 0:
                y += float(block.alpha[e]) * (xs @ block.a[s][e].double().T) @ block.b[s][e].double().T
            y = y.view(-1, 3, heads, 128)
            for i in range(2):
                y[:, i] = y[:, i] / (y[:, i].square().mean(-1, keepdim=True) + 1e-6).sqrt() * block.norm[s][i].double()
            parts.append(y)
        qkv = torch.cat(parts)
        for i in range(2):
            u, v = qkv[:, i, :, 0::2].clone(), qkv[:, i, :, 1::2].clone()
            qkv[:, i, :, 0::2], qkv[:, i, :, 1::2] = u * angle.cos() - v * angle.sin(), u * angle.sin() + v * angle.cos()
        q, k, v = (qkv[:, i].transpose(0, 1) for i in range(3))
        p = torch.softmax((q @ k.transpose(1, 2) / math.sqrt(128)).masked_fill(~mask[r], -math.inf), -1)
        mixed = (p @ v).transpose(0, 1).reshape(-1, dim)
        for s, rows in (("text", mixed[:text]), ("image", mixed[text:])):
            out[s].append(x[s][r].double() + block.gate[s].double() * (rows @ block.out[s].dense().T))
    return {s: torch.stack(v) for s, v in out.items()}


def example(requests, text, image, heads, rank=16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    block = Block(heads, adapters=3, rank=rank, seed=seed + 1)
    x = {s: torch.randn(requests, n, block.dim, generator=gen, device="cuda").bfloat16() for s, n in (("text", text), ("image", image))}
    adapter = [r % 4 - 1 for r in range(requests)]  # the first request has none
    filled = torch.randint(1, text + 1, (requests, 1), generator=gen, device="cuda")
    i = torch.arange(text + image, device="cuda")
    mask = (i < filled) | (i >= text)
    return block, x, adapter, mask, positions(text, image)


def decode_main(a):
    requests = a.requests or 16
    kv_heads = max(1, a.heads // 3) if a.heads % 3 == 0 else a.heads
    layer, x, adapter, filled = args = decode_example(requests, a.cached_tokens + 1, a.heads, kv_heads)
    workspace = decode_workspace(layer, requests)
    want = decode_reference(*args) if a.check else None
    got = decode_step(*args, workspace)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(50):
        decode_step(*args, workspace)
    torch.cuda.synchronize()
    print(f"one token of {requests} requests, caches of up to {a.cached_tokens} tokens, {a.heads} / {kv_heads} heads, hidden size "
          f"{layer.dim}: {(time.perf_counter() - t) * 2e4:.0f} us")
    if a.check:
        print(f"relative error against 64 bits {float((got.double() - want).norm() / want.norm()):.2e}")


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, help="default 2, or 16 with --decode")
    ap.add_argument("--text-tokens", type=int, default=512)
    ap.add_argument("--image-tokens", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=24)
    ap.add_argument("--check", action="store_true", help="compare with the same computation in 64 bits")
    ap.add_argument("--decode", action="store_true", help="one token of each request through a causal layer")
    ap.add_argument("--cached-tokens", type=int, default=4096)
    a = ap.parse_args()
    if a.decode:
        return decode_main(a)
    a.requests = a.requests or 2
    args = example(a.requests, a.text_tokens, a.image_tokens, a.heads)
    tokens = a.text_tokens + a.image_tokens
    block = args[0]
    q = torch.empty(a.requests, tokens, a.heads, 128, dtype=torch.bfloat16, device="cuda")
    need = max(lb.attention_workspace_size(q, q, q), lb.lora_workspace_size(max(a.text_tokens, a.image_tokens), 16))
    workspace = torch.zeros(need, dtype=torch.uint8, device="cuda")
    got = attention_half(*args, workspace)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(10):
        attention_half(*args, workspace)
    torch.cuda.synchronize()
    print(f"{a.requests} requests of {a.text_tokens} + {a.image_tokens} tokens, {a.heads} heads, hidden size {block.dim}: "
          f"{(time.perf_counter() - t) * 100:.2f} ms")
    if a.check:
        want = reference(*args)
        for s in ("text", "image"):
            err = (got[s].double() - want[s]).norm() / want[s].norm()
            print(f"{s} stream: relative error against 64 bits {float(err):.2e}")


if __name__ == "__main__":
    main()
