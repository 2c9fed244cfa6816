"""The operators around a block's packed linears, as cases that can be timed: low-rank adapters beside
a packed projection, the norms of queries and keys with their position rotation, and attention.

`own` chooses what run() calls: False, the operators written in elementary torch operations in 32 bits;
True, the package's kernels.  exact() gives the same results in 64 bits, from the definitions.
"""
import math

import torch

own = False

# One scratch buffer that a program keeps for its calls (split sums, adapter products).
SCRATCH_BYTES = 64 << 20
STEP = 64  # scale groups and packed words line up with multiples of this along K


# ---------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------

def _lora(name, m, n, k, bits, g, rank, adapters, rows):
    return {"name": name, "op": "lora", "m": m, "n": n, "k": k, "bits": bits, "g": g, "rank": rank,
            "adapters": adapters, "rows": rows}


def _rope(name, tokens, q_heads, kv_heads, head_dim, axes, paired, norm):
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "axes": axes, "paired": paired, "norm": norm}


def _attn(name, batch, q_heads, kv_heads, head_dim, q_len, kv_len, causal, keys, fused):
    return {"name": name, "op": "attention", "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "q_len": q_len, "kv_len": kv_len, "causal": causal, "keys": keys, "fused": fused}


def listed():
    return [
        # sixteen requests of one token each through the packed QKV linear, every one with its own adapter
        _lora("lora_16_requests", 16, 9216, 3072, 2, 64, 16, 16, "scattered"),
        # the text stream of a double-stream block, two requests of unequal prompts, binary weights in groups of 128
        _lora("lora_text_binary", 509, 3072, 9216, 1, 128, 32, 2, "segments"),
        # three 512 x 512 images denoised together, each with its own style adapter, through the QKV linear
        _lora("lora_three_images", 4608, 9216, 3072, 2, 64, 32, 3, "segments"),
        # 4-bit text encoder width, odd token count, rows of many requests interleaved, some without an adapter
        _lora("lora_interleaved_4bit", 1021, 2560, 4096, 4, 64, 8, 12, "scattered"),
        # one decoded token, grouped heads, norm and rotation of halves
        _rope("rope_one_token", 1, 32, 8, 128, "128", False, True),
        # a 1024 x 1024 image with 512 text tokens, four position axes on interleaved pairs, norm of every head
        _rope("rope_image_4_axes", 4608, 24, 24, 128, "32,32,32,32", True, True),
        # a video's latent frames, three axes, heads of 64, rotation alone, odd token count
        _rope("rope_video_3_axes", 16383, 16, 16, 64, "16,24,24", True, False),
        # four requests decode one token each from caches of unequal length, grouped heads
        _attn("attn_decode_4", 4, 32, 8, 128, 1, 4099, False, "lengths", False),
        # one request decodes from a long cache
        _attn("attn_decode_long", 1, 32, 8, 128, 1, 40007, False, "all", False),
        # a text encoder's prompt padded to 512, causal, grouped heads
        _attn("attn_text_causal", 1, 32, 8, 128, 512, 512, True, "padded", True),
        # joint attention of a 1024 x 1024 image's 4096 tokens and 512 text tokens
        _attn("attn_joint_4608", 1, 24, 24, 128, 4608, 4608, False, "all", True),
        # two 512 x 512 images with padded prompts in front, heads of 64, odd length
        _attn("attn_joint_padded_64", 2, 16, 16, 64, 1533, 1533, False, "padded", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "rope", "attention"])
    if op == "lora":
        m = _log(rng, 1, 4608)
        bits = rng.choice([1, 2, 4])
        g = rng.choice([64, 128])
        n = 16 * _log(rng, 16, 576)
        k = 128 * _log(rng, 2, 72)
        k = max(128, min(k, int(4608 * 9216 * 3072 / m / n) // 128 * 128))
        return {key: v for key, v in _lora("", m, n, k, bits, g, rng.choice([8, 16, 24, 32, 64]), rng.randint(1, 16),
                                           rng.choice(["segments", "scattered"])).items() if key != "name"}
    if op == "rope":
        head_dim = rng.choice([64, 128])
        axes = rng.choice(["64", "16,24,24", "32,32"] if head_dim == 64 else ["128", "64", "32,32,32,32", "16,56,56"])
        kv_heads = rng.choice([2, 4, 8, 16, 24])
        q_heads = min(32, kv_heads * rng.choice([1, 1, 2, 4]) if kv_heads <= 16 else kv_heads)
        return {key: v for key, v in _rope("", _log(rng, 1, 8192), q_heads, kv_heads, head_dim, axes,
                                           rng.random() < 0.5, rng.random() < 0.7).items() if key != "name"}
    head_dim = rng.choice([64, 128])
    kv_heads = rng.choice([2, 4, 8, 16, 24])
    group = rng.choice([1, 2, 4]) if kv_heads <= 8 else 1
    batch = rng.randint(1, 4)
    if rng.random() < 0.4:  # a few tokens against a cache
        q_len = _log(rng, 1, 64)
        kv_len = max(q_len, _log(rng, 64, 32768 // batch))
        return {key: v for key, v in _attn("", batch, kv_heads * group, kv_heads, head_dim, q_len, kv_len,
                                           rng.random() < 0.5, "lengths", False).items() if key != "name"}
    length = _log(rng, 1, 4608 // batch)
    return {key: v for key, v in _attn("", batch, kv_heads * group, kv_heads, head_dim, length, length,
                                       rng.random() < 0.5, rng.choice(["all", "padded"]), True).items() if key != "name"}


# ---------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _packed_codes(gen, n, k, bits):
    """Packed words [n, k * bits / 32] of uniform codes (ternary: half of them zero, the field 11 never written)."""
    if bits != 2:
        return torch.randint(-2 ** 31, 2 ** 31, (n, k * bits // 32), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    fields = torch.tensor([0, 0, 1, 2], device="cuda")[torch.randint(0, 4, (n, k // 16, 16), generator=gen, device="cuda")]
    words = (fields << (2 * torch.arange(16, device="cuda"))).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def _adapter_rows(gen, case):
    """The adapter of every row: requests one after the other, or row by row; -1 for a row without one."""
    m, adapters = case["m"], case["adapters"]
    if case["rows"] == "scattered":
        return torch.randint(-1 if m > adapters else 0, adapters, (m,), generator=gen, device="cuda", dtype=torch.int32)
    cuts = torch.sort(torch.randint(0, m + 1, (adapters - 1,), generator=gen, device="cuda")).values
    return torch.searchsorted(cuts, torch.arange(m, device="cuda"), right=True).to(torch.int32)


def _positions(case):
    """Whole-number positions [tokens, axes]: a running index on one axis; a prompt followed by an image's rows and columns, or a video's
    frames, rows and columns, on several."""
    t, axes = case["tokens"], len(case["axes"].split(","))
    i = torch.arange(t, device="cuda", dtype=torch.int32)
    if axes == 1:
        return (i + 257)[:, None].contiguous()
    if axes == 2:
        return torch.stack([i // 64, i % 64], 1).contiguous()
    if axes == 3:
        return torch.stack([i // 1024, i // 32 % 32, i % 32], 1).contiguous()
    text = i < t // 9
    p = i - t // 9
    zero = torch.zeros_like(i)
    return torch.stack([zero, torch.where(text, zero, p // 64), torch.where(text, zero, p % 64), torch.where(text, i, zero)], 1).contiguous()


def _frequencies(case):
    """Radians per unit position of every pair, and the axis that the pair turns with."""
    dims = [int(d) for d in case["axes"].split(",")]
    f = torch.cat([10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) for d in dims])
    axis = torch.cat([torch.full((d // 2,), i) for i, d in enumerate(dims)])
    return f.to(torch.float32).cuda(), axis.cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "scratch": torch.zeros(SCRATCH_BYTES, dtype=torch.uint8, device="cuda")}
    if case["op"] == "lora":
        m, n, k, g, r, e = case["m"], case["n"], case["k"], case["g"], case["rank"], case["adapters"]
        s["x"] = _normal(gen, m, k).bfloat16()
        s["words"] = _packed_codes(gen, n, k, case["bits"])
        s["scales"] = (torch.rand(n, k // g, generator=gen, device="cuda") * 0.045 + 0.005).half()
        s["a"] = (_normal(gen, e, r, k) / math.sqrt(k)).bfloat16()
        s["b"] = (_normal(gen, e, n, r) * 0.1).bfloat16()
        s["alpha"] = torch.rand(e, generator=gen, device="cuda") + 0.5
        s["rows"] = _adapter_rows(gen, case)
        s["out"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "rope":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
        qkv = _normal(gen, t, hq + 2 * hk, d).bfloat16()  # one fused projection's output
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["q_weight"] = (1 + 0.1 * _normal(gen, d)).bfloat16() if case["norm"] else None
        s["k_weight"] = (1 + 0.1 * _normal(gen, d)).bfloat16() if case["norm"] else None
        s["positions"] = _positions(case)
        s["freqs"], s["axis"] = _frequencies(case)
        s["q_out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(t, hk, d, dtype=torch.bfloat16, device="cuda")
    else:
        b, hq, hk, d, lq, lk = (case[x] for x in ("batch", "q_heads", "kv_heads", "head_dim", "q_len", "kv_len"))
        if case["fused"]:  # columns of one fused projection's output
            qkv = _normal(gen, b, lq, hq + 2 * hk, d).bfloat16()
            s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:]
        else:  # new tokens against a cache
            s["q"] = _normal(gen, b, lq, hq, d).bfloat16()
            s["k"], s["v"] = _normal(gen, b, lk, hk, d).bfloat16(), _normal(gen, b, lk, hk, d).bfloat16()
        s["mask"] = s["lengths"] = s["start"] = None
        if case["keys"] == "padded":  # a prompt in front whose end is padding, then tokens that are all there
            prompt = max(1, lk // 3)
            filled = torch.randint(1, prompt + 1, (b, 1), generator=gen, device="cuda")
            i = torch.arange(lk, device="cuda")
            s["mask"] = ((i < filled) | (i >= prompt)).contiguous()
        if case["keys"] == "lengths":  # every request has filled its own part of the cache
            low = max(lq, lk - lk // 2)
            s["lengths"] = torch.randint(low, lk + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
            s["start"] = s["lengths"] - lq  # the new tokens are the last ones
        s["out"] = torch.empty(b, lq, hq, d, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------

def run(s):
    return _kernels(s) if own else _PLAIN[s["case"]["op"]](s)


def _kernels(s):
    import binary_bit_gemm_amd as lb
    c = s["case"]
    if c["op"] == "lora":
        return lb.gemm_lora(s["x"], s["words"], s["scales"], c["g"], c["bits"], s["a"], s["b"], s["alpha"], s["rows"],
                            out=s["out"], workspace=s["scratch"])
    if c["op"] == "rope":
        return lb.qk_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], tuple(map(int, c["axes"].split(","))),
                               q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6, interleaved=c["paired"],
                               q_out=s["q_out"], k_out=s["k_out"])
    return lb.attention(s["q"], s["k"], s["v"], key_mask=s["mask"], key_lens=s["lengths"], causal=c["causal"],
                        q_start=s["start"], out=s["out"], workspace=s["scratch"])


def _codes(words, bits):
    """Packed words -> codes [n, k] in 32-bit floats."""
    per = 32 // bits
    fields = (words[:, :, None] >> (bits * torch.arange(per, device=words.device, dtype=torch.int32))) & ((1 << bits) - 1)
    if bits == 2:
        codes = (fields == 1).float() - (fields == 2).float()
    elif bits == 1:
        codes = fields.float() * 2 - 1
    else:
        codes = fields.float() - 16 * (fields > 7).float()
    return codes.flatten(1)


def _plain_lora(s):
    c = s["case"]
    x = s["x"].float()
    w = _codes(s["words"], c["bits"]) * s["scales"].float().repeat_interleave(c["g"], 1)
    y = x @ w.t()
    # every row through every adapter's first factor, then only its own one kept
    u = (x @ s["a"].float().flatten(0, 1).t()).view(c["m"], c["adapters"], c["rank"])
    mine = s["rows"][:, None] == torch.arange(c["adapters"], device=x.device, dtype=torch.int32)
    u = torch.where(mine[:, :, None], u * s["alpha"][None, :, None], 0.0)
    y = y + u.flatten(1) @ s["b"].float().transpose(1, 2).flatten(0, 1)
    s["out"].copy_(y)
    return s["out"]


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].float()[:, s["axis"]] * s["freqs"]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    rot = 2 * angle.shape[1]

    def one(x, weight, out):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        if c["paired"]:
            p, q = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack([p * cos - q * sin, p * sin + q * cos], -1).flatten(-2)
        else:
            p, q = x[..., :rot // 2], x[..., rot // 2:rot]
            turned = torch.cat([p * cos - q * sin, p * sin + q * cos], -1)
        out.copy_(torch.cat([turned, x[..., rot:]], -1))
        return out

    return one(s["q"], s["q_weight"], s["q_out"]), one(s["k"], s["k_weight"], s["k_out"])


def _allowed(s, dev):
    """Which keys each query sees, [batch, 1, q_len, kv_len], or None for all."""
    c = s["case"]
    key = torch.arange(c["kv_len"], device=dev)
    seen = torch.ones(c["batch"], 1, c["q_len"], c["kv_len"], dtype=torch.bool, device=dev)
    if s["mask"] is not None:
        seen = seen & s["mask"][:, None, None, :]
    if s["lengths"] is not None:
        seen = seen & (key < s["lengths"][:, None, None, None])
    if c["causal"]:
        at = torch.arange(c["q_len"], device=dev)[None, :] + (s["start"][:, None] if s["start"] is not None else 0)
        seen = seen & (key <= at[:, None, :, None])
    return seen


def _plain_attention(s):
    c = s["case"]
    group = c["q_heads"] // c["kv_heads"]
    q, k, v = (s[x].float().transpose(1, 2) for x in ("q", "k", "v"))
    b, hk, lk, d = k.shape
    q = q.reshape(b, hk, group * c["q_len"], d)
    scores = (q @ k.transpose(2, 3)).view(b, hk, group, c["q_len"], lk) / math.sqrt(d)
    if c["causal"] or s["mask"] is not None or s["lengths"] is not None:
        scores = torch.where(_allowed(s, q.device)[:, :, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    o = (p.view(b, hk, group * c["q_len"], lk) @ v).view(b, c["q_heads"], c["q_len"], d)
    s["out"].copy_(o.transpose(1, 2))
    return s["out"]


_PLAIN = {"lora": _plain_lora, "rope": _plain_rope, "attention": _plain_attention}


# ---------------------------------------------------------------------------------------------------
# What a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "lora":
        m, n, k, r, e = case["m"], case["n"], case["k"], case["rank"], min(case["adapters"], case["m"])
        return {"bytes": 2 * m * k + n * k * case["bits"] // 8 + 2 * n * (k // case["g"]) + 2 * e * r * (n + k) + 4 * m + 2 * m * n,
                "flops": 2 * m * n * k + 2 * m * r * (n + k)}
    if case["op"] == "rope":
        rows = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        axes = len(case["axes"].split(","))
        return {"bytes": 4 * rows * case["head_dim"] + 4 * axes * case["tokens"], "flops": 8 * rows * case["head_dim"]}
    b, hq, hk, d, lq, lk = (case[x] for x in ("batch", "q_heads", "kv_heads", "head_dim", "q_len", "kv_len"))
    keys = lk if case["keys"] != "lengths" else (max(lq, lk - lk // 2) + lk) / 2
    seen = keys - (lq - 1) / 2 if case["causal"] else keys
    return {"bytes": int(2 * b * d * (2 * hq * lq + 2 * hk * keys)), "flops": int(4 * b * hq * d * lq * seen)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"lora": _exact_lora, "rope": _exact_rope, "attention": _exact_attention}[case["op"]](case, s)


def _exact_lora(case, s):
    bits, g, k = case["bits"], case["g"], case["k"]
    per = 32 // bits
    w = torch.empty(case["n"], k, dtype=torch.float64, device="cuda")
    unsigned = s["words"].long() & 0xFFFFFFFF
    value = {1: [-1, 1], 2: [0, 1, -1, 0], 4: [0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1]}[bits]
    value = torch.tensor(value, dtype=torch.float64, device="cuda")
    for j in range(per):  # code j of every word
        w[:, j::per] = value[(unsigned // 2 ** (bits * j)) % 2 ** bits]
    for j in range(k // g):
        w[:, j * g:(j + 1) * g] *= s["scales"][:, j:j + 1].double()
    x = s["x"].double()
    y = x @ w.T
    for e in range(case["adapters"]):
        mine = torch.nonzero(s["rows"] == e).flatten()
        y[mine] += float(s["alpha"][e]) * ((x[mine] @ s["a"][e].double().T) @ s["b"][e].double().T)
    return y


def _exact_rope(case, s):
    results = []
    dims = [int(d) for d in case["axes"].split(",")]
    pair_of = [(a, i) for a, d in enumerate(dims) for i in range(d // 2)]
    half = len(pair_of)
    for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double().clone()
        if weight is not None:
            y /= torch.sqrt(torch.sum(y ** 2, -1, keepdim=True) / case["head_dim"] + 1e-6)
            y *= weight.double()
        turned = y.clone()
        for j, (a, _) in enumerate(pair_of):
            first, second = (2 * j, 2 * j + 1) if case["paired"] else (j, j + half)
            angle = (s["positions"][:, a].double() * s["freqs"][j].double())[:, None]
            turned[..., first] = y[..., first] * torch.cos(angle) - y[..., second] * torch.sin(angle)
            turned[..., second] = y[..., first] * torch.sin(angle) + y[..., second] * torch.cos(angle)
        results.append(turned)
    return tuple(results)


def _exact_attention(case, s):
    group = case["q_heads"] // case["kv_heads"]
    out = torch.zeros(case["batch"], case["q_len"], case["q_heads"], case["head_dim"], dtype=torch.float64, device="cuda")
    index = torch.arange(case["kv_len"], device="cuda")
    for b in range(case["batch"]):
        live = torch.ones(case["kv_len"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"][b]
        if s["lengths"] is not None:
            live = live & (index < s["lengths"][b])
        keep = live[None, :].expand(case["q_len"], -1)
        if case["causal"]:
            first = int(s["start"][b]) if s["start"] is not None else 0
            keep = keep & (index[None, :] <= first + torch.arange(case["q_len"], device="cuda")[:, None])
        some = keep.any(1)
        for h in range(case["q_heads"]):
            logits = s["q"][b, :, h].double() @ s["k"][b, :, h // group].double().T * case["head_dim"] ** -0.5
            p = torch.softmax(logits.masked_fill(~keep, -math.inf)[some], -1)
            out[b, some, h] = p @ s["v"][b, :, h // group].double()
    return out
