"""The operators of a decoding step around 4-bit linears, as cases that can be timed: a paged cache of keys and values
that is quantised as it is written and read back, attention of new or drafted tokens over such a cache, and matrix-vector products with 4-bit
weights in affine groups.

`own` chooses what run() calls: False, the operators written in elementary torch operations in 32 bits;
True, the package's kernels.  exact() gives the same results in 64 bits, from the definitions.
"""
import math

import torch

own = False

# One scratch buffer that a program keeps for its calls (results of ranges of keys).
SCRATCH_BYTES = 64 << 20
GROUP = 64  # elements that share a scale and a smallest value in a 4-bit cache


# ---------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------

def _store(name, requests, past, new, reads, kv_heads, head_dim, bits, page):
    return {"name": name, "op": "store", "requests": requests, "past": past, "new": new, "reads": reads, "kv_heads": kv_heads,
            "head_dim": head_dim, "bits": bits, "page": page}


def _attn(name, batch, q_len, kv_len, q_heads, kv_heads, head_dim, bits, page, tree, lengths):
    return {"name": name, "op": "attention", "batch": batch, "q_len": q_len, "kv_len": kv_len, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "bits": bits, "page": page, "tree": tree, "lengths": lengths}


def _gemv(name, m, n, k, g, form):
    return {"name": name, "op": "gemv", "m": m, "n": n, "k": k, "g": g, "form": form}


def listed():
    return [
        # sixty-one requests decode: one token of each goes into the cache, and comes back as attention will see it
        _store("store_one_token_each", 61, 700, 1, "new", 8, 128, 8, 32),
        # a padded prompt's last 509 tokens join 16,000 that are there, and the whole goes back to bf16 for the prompt's attention
        _store("store_chunk_4bit", 1, 16001, 509, "all", 8, 128, 4, 64),
        # four prompts of 1021 tokens, heads of 64, written and read back
        _store("store_prompts_64", 4, 0, 1021, "all", 16, 64, 8, 16),
        # one token of one short request: latency alone
        _attn("attn_short", 1, 1, 77, 32, 8, 128, 8, 16, False, "full"),
        # four requests decode one token each from caches of unequal length
        _attn("attn_decode_4", 4, 1, 4099, 32, 8, 128, 8, 64, False, "spread"),
        # one request decodes from a long cache of 4-bit codes
        _attn("attn_decode_long_4bit", 1, 1, 40007, 32, 8, 128, 4, 64, False, "full"),
        # sixty-one requests decode together
        _attn("attn_decode_61", 61, 1, 2050, 32, 8, 128, 8, 32, False, "spread"),
        # trees of 27 drafted tokens for three requests, 4-bit codes, heads of 64
        _attn("attn_tree_27_4bit", 3, 27, 8191, 16, 4, 64, 4, 16, True, "spread"),
        # a tree of 64 drafted tokens for each of four requests, keys and values kept in 16 bits
        _attn("attn_tree_64_16bit", 4, 64, 4099, 32, 8, 128, 16, 64, True, "spread"),
        # the text encoder's gate and up projections with their activation, one token
        _gemv("gemv_gate_up", 1, 9728, 2560, 64, "swiglu"),
        # its down projection, added to the residual stream
        _gemv("gemv_down", 1, 2560, 9728, 64, "residual"),
        # eleven drafted tokens through an output projection in groups of 128
        _gemv("gemv_11_rows", 11, 2560, 4096, 128, "plain"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "attention", "attention", "gemv"])
    if op == "gemv":
        g = rng.choice([64, 128])
        k = g * _log(rng, 1, 9728 // g)
        n = 16 * _log(rng, 4, max(4, min(1216, 19456 * 2560 // k // 16)))
        form = rng.choice(["plain", "residual", "swiglu"])
        case = _gemv("", rng.choice([1, 1, 1, 2, 3, 4, 5, 7, 8, 11, 16]), 16 * max(1, n // 32) if form == "swiglu" else n, k, g, form)
    else:
        kv_heads, head_dim, bits, page = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128]), rng.choice([4, 8, 8, 16]), rng.choice([16, 32, 64, 128])
        if op == "store":
            requests = _log(rng, 1, 64)
            most = max(2, 16384 * 8 // kv_heads // requests)
            new = _log(rng, 1, max(1, min(4608, most // 2)))
            case = _store("", requests, _log(rng, 1, max(1, most - new)) - 1, new, rng.choice(["new", "all"]), kv_heads, head_dim, bits, page)
        else:
            batch, tree = _log(rng, 1, 64), rng.random() < 0.4
            q_len = _log(rng, 2, 64) if tree else rng.choice([1, 1, 1, 2, 5])
            group = rng.choice([1, 2, 4, 5, 8])
            most = min(40007, 60 * 2050 * 8 // kv_heads // batch, 4 * 4099 * 8 * 64 * 4 // (kv_heads * batch * q_len * group))
            case = _attn("", batch, q_len, max(q_len, _log(rng, 16, max(17, most))), kv_heads * group, kv_heads, head_dim, bits, page, tree,
                         rng.choice(["full", "spread"]))
    return {key: v for key, v in case.items() if key != "name"}


# ---------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _fill_cache(s, gen, pages):
    """A cache of `pages` pages in the package's layout, full of what earlier tokens left: random codes, each with a scale (4 bits: and the
    group's smallest value)."""
    c = s["case"]
    h, d, bits, page = c["kv_heads"], c["head_dim"], c["bits"], c["page"]
    for x in ("k", "v"):
        if bits == 16:
            s[x + "_cache"], s[x + "_scales"] = _normal(gen, pages, h, page, d).bfloat16(), None
            continue
        codes = torch.randint(0, 2 ** 31, (pages, h, page, d * bits // 32), generator=gen, device="cuda", dtype=torch.int32)
        codes = codes ^ (torch.randint(0, 2, codes.shape, generator=gen, device="cuda", dtype=torch.int32) << 31)
        codes = codes.view(torch.uint8).view(pages, h, page, d * bits // 8)
        scale = torch.rand(pages, h, page, *(() if bits == 8 else (d // GROUP, 1)), generator=gen, device="cuda") + 0.5
        if bits == 8:
            s[x + "_cache"] = codes.clamp_(min=1)  # code -128 is never written
            s[x + "_scales"] = (scale * (1.7 / 127)).bfloat16()  # uniform codes of unit variance
        else:
            s[x + "_cache"] = codes
            step = scale * (3.4 / 15)
            s[x + "_scales"] = torch.cat([step, -7.5 * step + 0.1 * _normal(gen, *step.shape)], -1).bfloat16().contiguous()


def _scatter_pages(gen, case, sequences, tokens):
    """(page table [sequences, pages of each], pages in all): the sequences' pages lie anywhere among a few more."""
    each = -(-tokens // case["page"])
    pages = sequences * each + 3
    return torch.randperm(pages, generator=gen, device="cuda")[:sequences * each].view(sequences, each).to(torch.int32), pages


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "store":
        r, past, new, h, d, page = (case[x] for x in ("requests", "past", "new", "kv_heads", "head_dim", "page"))
        table, pages = _scatter_pages(gen, case, r, past + new)
        _fill_cache(s, gen, pages)
        at = torch.arange(past + new, device="cuda")
        slots = (table[:, at // page] * page + at % page).to(torch.int32)
        s["write_slots"] = slots[:, past:].reshape(-1).contiguous()
        s["read_slots"] = s["write_slots"] if case["reads"] == "new" else slots.reshape(-1).contiguous()
        qkv = _normal(gen, r * new, 4 * h, d).bfloat16()  # one fused projection's output: two query heads for each key head
        s["k"], s["v"] = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
        rows = s["read_slots"].numel()
        s["k_out"] = torch.empty(rows, h, d, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty(rows, h, d, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "attention":
        b, lq, lk, hq, d = (case[x] for x in ("batch", "q_len", "kv_len", "q_heads", "head_dim"))
        s["table"], pages = _scatter_pages(gen, case, b, lk)
        _fill_cache(s, gen, pages)
        s["q"] = _normal(gen, b, lq, hq, d).bfloat16()
        low = max(lq, lk // 2)
        s["lengths"] = (torch.full((b,), lk, dtype=torch.int32, device="cuda") if case["lengths"] == "full" else
                        torch.randint(low, lk + 1, (b,), generator=gen, device="cuda", dtype=torch.int32))
        s["tree"] = _trees(gen, b, lq) if case["tree"] else None
        s["scratch"] = torch.zeros(SCRATCH_BYTES, dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty(b, lq, hq, d, dtype=torch.bfloat16, device="cuda")
    else:
        m, n, k, g = (case[x] for x in ("m", "n", "k", "g"))
        rows = 2 * n if case["form"] == "swiglu" else n  # gate rows, then up rows
        s["x"] = _normal(gen, m, k).bfloat16()
        s["words"] = torch.randint(-2 ** 31, 2 ** 31, (rows, k // 8), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
        scale = (torch.rand(rows, k // g, generator=gen, device="cuda") + 0.5) * (0.2 / math.sqrt(k))
        s["scales"] = scale.half()
        s["biases"] = (scale * (-7.5 + 0.5 * _normal(gen, rows, k // g))).half()
        s["residual"] = _normal(gen, m, n).bfloat16() if case["form"] == "residual" else None
        s["out"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    return s


def _trees(gen, batch, nodes):
    """Ancestors of every drafted token, itself among them, as bits of an int64 [batch, nodes]: every token's parent is one of those before it."""
    parents = (torch.rand(batch, nodes, generator=gen, device="cuda") * torch.arange(nodes, device="cuda")).long().tolist()
    trees = []
    for row in parents:
        bits = [1]
        for i in range(1, nodes):
            bits.append(bits[row[i]] | 1 << i)
        trees.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in bits])
    return torch.tensor(trees, dtype=torch.int64, device="cuda")


# ---------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------

def run(s):
    return _kernels(s) if own else _PLAIN[s["case"]["op"]](s)


def _kernels(s):
    import binary_bit_gemm_amd as lb
    c = s["case"]
    if c["op"] == "gemv":
        return lb.gemv_affine(s["x"], s["words"], s["scales"], s["biases"], c["g"], residual=s["residual"], swiglu=c["form"] == "swiglu",
                              out=s["out"])
    cache = lb.KVCache(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], bits=c["bits"])
    if c["op"] == "store":
        lb.cache_write(cache, s["k"], s["v"], s["write_slots"])
        return lb.cache_read(cache, s["read_slots"], k_out=s["k_out"], v_out=s["v_out"])
    return lb.cache_attention(s["q"], cache, s["table"], s["lengths"], tree=s["tree"], kv_len=c["kv_len"], out=s["out"],
                              workspace=s["scratch"])


# Where the codes lie.  A row of K at 8 bits is its codes + 128; at 4 bits it is four parts of 8 bytes for each group of 64, part p with elements
# 16 p .. 16 p + 15 of every group, two words of 8 codes, element e of a word at nibble e / 2 + 4 (e % 2).  V goes in blocks of T tokens,
# [16 pieces][T][piece]: piece l holds elements l D / 16 .. of a row, at 4 bits 4 l .. 4 l + 3 of every group, the first in the low nibble.

def _block(c):
    """(tokens of a block of V, units of a piece: bytes, or elements at 16 bits)."""
    size = c["head_dim"] * c["bits"] // 128
    return min(4, 16 // size), c["head_dim"] // 16 if c["bits"] == 16 else size


def _v_view(c, cache):
    t, p = _block(c)
    pages, h, page, _ = cache.shape
    return cache.view(pages, h, page // t, 16, t, p)


def _plain_quantise(x, bits):
    """fp32 [..., D] -> (codes as floats, scales bf16): [...] at 8 bits, [..., groups, 2] at 4."""
    def up(t):  # the smallest bf16 that is not below
        return ((t.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)
    if bits == 8:
        scale = up(x.abs().amax(-1) / 127)
        safe = torch.where(scale > 0, scale, 1.0)
        return torch.round(x / safe[..., None]).clamp(-127, 127), scale.bfloat16()
    x = x.unflatten(-1, (-1, GROUP))
    low = x.amin(-1)
    scale = up((x.amax(-1) - low) / 15)
    safe = torch.where(scale > 0, scale, 1.0)
    codes = torch.round((x - low[..., None]) / safe[..., None]).clamp(0, 15)
    return codes.flatten(-2), torch.stack([scale, low], -1).bfloat16()


def _plain_store(s):
    c = s["case"]
    h, d, bits, page = c["kv_heads"], c["head_dim"], c["bits"], c["page"]
    slot = s["write_slots"].long()
    at, within = slot // page, slot % page
    t, p = _block(c)
    if bits == 16:
        s["k_cache"][at, :, within] = s["k"]
        _v_view(c, s["v_cache"])[at, :, within // t, :, within % t] = s["v"].reshape(-1, h, 16, p)
    else:
        k, s["k_scales"][at, :, within] = _plain_quantise(s["k"].float(), bits)
        v, s["v_scales"][at, :, within] = _plain_quantise(s["v"].float(), bits)
        if bits == 8:
            k, v = (k + 128).to(torch.uint8), (v + 128).to(torch.uint8).view(-1, h, 16, p)
        else:
            k = k.to(torch.uint8).view(-1, h, d // GROUP, 4, 2, 4, 2).permute(0, 1, 3, 2, 4, 6, 5)  # part, group, word, half of the word, nibble
            k = k.reshape(-1, h, d // 2, 2)
            v = v.to(torch.uint8).view(-1, h, d // GROUP, 16, 2, 2).transpose(2, 3).reshape(-1, h, 16, p, 2)
            k, v = k[..., 0] | k[..., 1] << 4, v[..., 0] | v[..., 1] << 4
        s["k_cache"][at, :, within] = k
        _v_view(c, s["v_cache"])[at, :, within // t, :, within % t] = v
    slot = s["read_slots"].long()
    k, v = _plain_gather(s, slot // page, slot % page)
    s["k_out"].copy_(k)
    s["v_out"].copy_(v)
    return s["k_out"], s["v_out"]


def _plain_gather(s, at, within):
    """The keys and values of these places, fp32 [..., heads, D]."""
    c = s["case"]
    h, d, bits = c["kv_heads"], c["head_dim"], c["bits"]
    t, _ = _block(c)
    k = s["k_cache"][at, :, within]
    v = _v_view(c, s["v_cache"])[at, :, within // t, :, within % t].flatten(-2)
    if bits == 16:
        return k.float(), v.float()
    if bits == 8:
        return tuple((x.float() - 128) * scales[at, :, within].float()[..., None] for x, scales in ((k, s["k_scales"]), (v, s["v_scales"])))
    k, v = (torch.stack([x & 15, x >> 4], -1).float() for x in (k, v))
    k = k.reshape(*at.shape, h, 4, d // GROUP, 2, 2, 4).movedim(-4, -5).transpose(-1, -2).reshape(*at.shape, h, d // GROUP, GROUP)
    v = v.reshape(*at.shape, h, 16, d // GROUP, 4).transpose(-2, -3).reshape(*at.shape, h, d // GROUP, GROUP)
    sk, sv = s["k_scales"][at, :, within].float(), s["v_scales"][at, :, within].float()
    return (k * sk[..., :1] + sk[..., 1:]).flatten(-2), (v * sv[..., :1] + sv[..., 1:]).flatten(-2)


def _plain_attention(s):
    c = s["case"]
    b, lq, lk, hq, hk, d = (c[x] for x in ("batch", "q_len", "kv_len", "q_heads", "kv_heads", "head_dim"))
    key = torch.arange(lk, device="cuda")
    k, v = _plain_gather(s, s["table"].long()[:, key // c["page"]], (key % c["page"]).expand(b, lk))
    group = hq // hk
    q = s["q"].float().view(b, lq, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * lq, d)
    scores = (q @ k.permute(0, 2, 3, 1).contiguous()).view(b, hk, group, lq, lk) / math.sqrt(d)
    base = s["lengths"].long() - lq
    drafted = key - base[:, None]  # [batch, keys]: which drafted token a key is
    if s["tree"] is None:
        seen = drafted[:, None] <= torch.arange(lq, device="cuda")[:, None]
    else:
        seen = (drafted < 0)[:, None] | ((s["tree"][:, :, None] >> drafted.clamp(0, 63)[:, None]) & 1).bool()
    seen = seen & (drafted < lq)[:, None]
    scores = torch.where(seen[:, None, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    o = p.view(b, hk, group * lq, lk) @ v.transpose(1, 2).contiguous()
    s["out"].copy_(o.view(b, hk, group, lq, d).permute(0, 3, 1, 2, 4).reshape(b, lq, hq, d))
    return s["out"]


def _plain_gemv(s):
    c = s["case"]
    levels = ((s["words"][:, :, None] >> (4 * torch.arange(8, device="cuda", dtype=torch.int32))) & 15).float().flatten(1)
    w = levels * s["scales"].float().repeat_interleave(c["g"], 1) + s["biases"].float().repeat_interleave(c["g"], 1)
    y = s["x"].float() @ w.t()
    if c["form"] == "swiglu":
        gate, up = y[:, :c["n"]], y[:, c["n"]:]
        y = gate / (1 + torch.exp(-gate)) * up
    if c["form"] == "residual":
        y = y + s["residual"].float()
    s["out"].copy_(y)
    return s["out"]


_PLAIN = {"store": _plain_store, "attention": _plain_attention, "gemv": _plain_gemv}


# ---------------------------------------------------------------------------------------------------
# What a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------------------------------

def _row_bytes(case):
    """A token's key or value of one head in the cache."""
    d, bits = case["head_dim"], case["bits"]
    return d * bits // 8 + {16: 0, 8: 2, 4: 4 * d // GROUP}[bits]


def work(case):
    if case["op"] == "gemv":
        m, n, k, g = (case[x] for x in ("m", "n", "k", "g"))
        rows = 2 * n if case["form"] == "swiglu" else n
        return {"bytes": rows * k // 2 + 4 * rows * (k // g) + 2 * m * k + (4 if case["form"] == "residual" else 2) * m * n,
                "flops": 2 * m * rows * k}
    h, d = case["kv_heads"], case["head_dim"]
    if case["op"] == "store":
        written = case["requests"] * case["new"]
        read = written if case["reads"] == "new" else case["requests"] * (case["past"] + case["new"])
        return {"bytes": 2 * h * (written + read) * (2 * d + _row_bytes(case)) + 4 * (written + read), "flops": 2 * h * d * (4 * written + 2 * read)}
    b, lq, lk, hq = (case[x] for x in ("batch", "q_len", "kv_len", "q_heads"))
    keys = lk if case["lengths"] == "full" else (max(lq, lk // 2) + lk) / 2
    return {"bytes": int(b * (2 * h * keys * _row_bytes(case) + 4 * lq * hq * d + 4 * -(-lk // case["page"]))),
            "flops": int(4 * b * hq * d * lq * keys)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "attention": _exact_attention, "gemv": _exact_gemv}[case["op"]](case, s)


def _exact_values(x, bits):
    """What [rows, D] in 64 bits stand for once they have been through the cache."""
    if bits == 16:
        return x
    step = torch.empty_like(x)
    low = torch.zeros_like(x)
    for first in range(0, x.shape[1], x.shape[1] if bits == 8 else GROUP):
        part = x[:, first:] if bits == 8 else x[:, first:first + GROUP]
        least = part.min(1).values
        reach = part.abs().max(1).values / 127 if bits == 8 else (part.max(1).values - least) / 15
        exponent = torch.floor(torch.log2(torch.where(reach > 0, reach, 1.0)))
        unit = 2.0 ** (exponent - 7)  # a bf16's last place
        step[:, first:first + part.shape[1]] = (torch.ceil(reach / unit) * unit)[:, None]
        if bits == 4:
            low[:, first:first + part.shape[1]] = least[:, None]
    return torch.round((x - low) / torch.where(step > 0, step, 1.0)) * step + low


def _exact_row(case, s, name, slots, head):
    """The rows at these slots as 64-bit values [slots, D], element by element from the layout."""
    d, bits, page = case["head_dim"], case["bits"], case["page"]
    at, within = slots // page, slots % page
    cache = s[name + "_cache"]
    if bits == 16 and name == "k":
        return cache[at, head, within].double()
    unit = cache.flatten(2)[at, head]  # a page of the head: its units in order
    values = torch.empty(len(slots), d, dtype=torch.float64, device="cuda")
    row = d if bits >= 8 else d // 2
    for e in range(d):
        g, r = e // GROUP, e % GROUP
        high = 0
        if name == "k":
            place = within * row + e
            if bits == 4:
                nibble = r % 8 // 2 + 4 * (r % 2)
                place = within * row + r // 16 * (8 * d // GROUP) + 8 * g + r % 16 // 8 * 4 + nibble // 2
                high = nibble % 2
        else:
            piece = row // 16
            t = min(4, 16 // (piece * (2 if bits == 16 else 1)))
            lane, inside = (e // piece, e % piece) if bits >= 8 else (r // 4, 2 * g + r % 4 // 2)
            high = r % 2
            place = within // t * (t * row) + (lane * t + within % t) * piece + inside
        u = unit.gather(1, place[:, None])[:, 0]
        if bits == 4:
            u = u // 16 if high else u % 16
        values[:, e] = u.double()
    if bits == 16:
        return values
    scales = s[name + "_scales"][at, head, within].double()
    if bits == 8:
        return (values - 128) * scales[:, None]
    return values * scales[:, :, 0].repeat_interleave(GROUP, 1) + scales[:, :, 1].repeat_interleave(GROUP, 1)


def _exact_store(case, s):
    results = []
    read = s["read_slots"].long()
    new = torch.full((s["k_cache"].shape[0] * case["page"],), -1, dtype=torch.long, device="cuda")
    new[s["write_slots"].long()] = torch.arange(s["write_slots"].numel(), device="cuda")
    source = new[read]
    fresh = source >= 0
    for name in ("k", "v"):
        out = torch.empty(len(read), case["kv_heads"], case["head_dim"], dtype=torch.float64, device="cuda")
        for h in range(case["kv_heads"]):
            out[:, h] = _exact_row(case, s, name, read, h)
            out[fresh, h] = _exact_values(s[name][source[fresh], h].double(), case["bits"])
        results.append(out)
    return tuple(results)


def _exact_attention(case, s):
    b, lq, hq, hk, d, page = (case[x] for x in ("batch", "q_len", "q_heads", "kv_heads", "head_dim", "page"))
    out = torch.zeros(b, lq, hq, d, dtype=torch.float64, device="cuda")
    group = hq // hk
    trees = s["tree"].tolist() if s["tree"] is not None else [[(2 << t) - 1 for t in range(lq)]] * b
    for i, length in enumerate(s["lengths"].tolist()):
        key = torch.arange(length, device="cuda")
        slots = s["table"][i].long()[key // page] * page + key % page
        keep = torch.ones(lq, length, dtype=torch.bool, device="cuda")
        for t in range(lq):
            keep[t, length - lq:] = torch.tensor([trees[i][t] >> j & 1 for j in range(lq)], device="cuda").bool()
        for h in range(hk):
            k, v = _exact_row(case, s, "k", slots, h), _exact_row(case, s, "v", slots, h)
            for g in range(group):
                logits = (s["q"][i, :, h * group + g].double() @ k.T) * d ** -0.5
                out[i, :, h * group + g] = torch.softmax(logits.masked_fill(~keep, -math.inf), -1) @ v
    return out


def _exact_gemv(case, s):
    n, k, g = case["n"], case["k"], case["g"]
    unsigned = s["words"].long() & 0xFFFFFFFF
    w = torch.empty(unsigned.shape[0], k, dtype=torch.float64, device="cuda")
    for j in range(8):
        w[:, j::8] = (unsigned // 16 ** j % 16).double()
    for j in range(k // g):
        w[:, j * g:(j + 1) * g] = w[:, j * g:(j + 1) * g] * s["scales"][:, j:j + 1].double() + s["biases"][:, j:j + 1].double()
    y = s["x"].double() @ w.T
    if case["form"] == "swiglu":
        y = y[:, :n] * torch.sigmoid(y[:, :n]) * y[:, n:]
    return y if case["form"] != "residual" else y + s["residual"].double()
