"""The attention half of a block (examples/adapted_attention_block.py): adapters beside the packed QKV linear, norms and
rotation in place, joint attention with padding, gated output linear, against the same computation in 64 bits."""
import importlib.util
import os

import pytest
import torch

import binary_bit_gemm_amd as lb

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapted_attention_block.py")


def load():
    spec = importlib.util.spec_from_file_location("adapted_attention_block", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("requests,text,image,heads", [(4, 37, 100, 2), (1, 1, 1, 4), (2, 64, 577, 4)])
def test_the_block_in_one_piece(requests, text, image, heads):
    """Four tensors are rounded to bf16 on the way (QKV, the turned q and k, the mixed values, the result), each by 2^-8
    of its elements at most; normed q and k make scores of a few units, so an error of 2 * 2^-8 in each
    of them moves the probabilities by a few per cent at most.  As relative norms: 4 * 2^-8 for the
    roundings and as much again for the scores."""
    m = load()
    args = m.example(requests, text, image, heads)
    block = args[0]
    q = torch.empty(requests, text + image, heads, 128, dtype=torch.bfloat16, device="cuda")
    need = max(lb.attention_workspace_size(q, q, q), lb.lora_workspace_size(max(text, image), 16))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    got = m.attention_half(*args, ws)
    want = m.reference(*args)
    for s in ("text", "image"):
        assert bool(torch.isfinite(got[s]).all())
        assert float((got[s].double() - want[s]).norm() / want[s].norm()) <= 8 * 2.0 ** -8
    again = m.attention_half(*args, ws)
    assert all(torch.equal(again[s], got[s]) for s in got)
    assert block.dim == 128 * heads


@pytest.mark.parametrize("requests,capacity,heads,kv_heads", [(16, 700, 6, 2), (1, 3000, 4, 4), (5, 40, 4, 1), (33, 130, 2, 2)])
def test_a_decoded_token_of_many_requests(requests, capacity, heads, kv_heads):
    """One call per linear with every request's own adapter.  Rounded to bf16 on the way: QKV, the turned q and k, the mixed values,
    the output linear's result and the sum, each by 2^-8 at most; scores of a few units move the probabilities by a few
    per cent at most: 5 * 2^-8 for the roundings and as much again for the scores."""
    m = load()
    layer, x, adapter, filled = m.decode_example(requests, capacity, heads, kv_heads)
    assert requests == 1 or len(set(adapter.tolist())) > 1
    ws = m.decode_workspace(layer, requests)
    want = m.decode_reference(layer, x, adapter, filled)
    got = m.decode_step(layer, x, adapter, filled, ws)
    assert bool(torch.isfinite(got).all())
    assert float((got.double() - want).norm() / want.norm()) <= 10 * 2.0 ** -8
    assert torch.equal(m.decode_step(layer, x, adapter, filled, ws), got)
    for r in range(requests):  # a request by itself, from its own cache
        one = m.Layer.__new__(m.Layer)
        one.__dict__.update(layer.__dict__)
        one.keys, one.values = layer.keys[r:r + 1], layer.values[r:r + 1]
        alone = m.decode_step(one, x[r:r + 1], adapter[r:r + 1], filled[r:r + 1], m.decode_workspace(one, 1))
        assert float((alone.double() - want[r:r + 1]).norm() / want[r:r + 1].norm()) <= 10 * 2.0 ** -8
