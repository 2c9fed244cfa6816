"""Host-side checks of the operators around the packed linears (CPU only): every refusal comes before anything touches a
device, and the workspace sizes are what the calls document.  tests of the host code under sanitizers: the last test runs this file
against the sanitized library."""
import ctypes
import os
import subprocess
import sys

import pytest

import binary_bit_gemm_amd as lb
from binary_bit_gemm_amd import _lib

OK, INVALID, UNSUPPORTED, ALIGN = 0, 1, 2, 3
A = 0x10000  # a 16-byte-aligned fake address: never dereferenced by the host checks
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ---- lowbit_gemm_lora ----

def lora(**kw):
    d = dict(X=A, W=A, S=A, Y=A, M=64, N=256, K=256, g=64, bits=2, A=A, B=A, alpha=A, rows=A, adapters=4, rank=16, ws=A, bytes=1 << 30)
    d.update(kw)
    return _lib.lib().lowbit_gemm_lora(d["X"], d["W"], d["S"], d["Y"], d["M"], d["N"], d["K"], d["g"], d["bits"], d["A"], d["B"],
                                       d["alpha"], d["rows"], d["adapters"], d["rank"], d["ws"], d["bytes"], None)


@pytest.mark.parametrize("change,want", [
    (dict(N=250), INVALID), (dict(K=200), INVALID), (dict(M=-1), INVALID), (dict(X=0), INVALID), (dict(Y=0), INVALID),
    (dict(bits=3), UNSUPPORTED), (dict(g=32), UNSUPPORTED), (dict(g=32, bits=1), UNSUPPORTED), (dict(X=A + 8), ALIGN),
    (dict(rank=0), UNSUPPORTED), (dict(rank=12), UNSUPPORTED), (dict(rank=136), UNSUPPORTED), (dict(rank=-8), UNSUPPORTED),
    (dict(adapters=-1), INVALID), (dict(adapters=(1 << 16) + 1), UNSUPPORTED),
    (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(alpha=0), INVALID), (dict(rows=0), INVALID),
    (dict(ws=0), INVALID), (dict(bytes=100), INVALID), (dict(bytes=0), INVALID),
    (dict(A=A + 8), ALIGN), (dict(B=A + 2), ALIGN), (dict(alpha=A + 2), ALIGN), (dict(rows=A + 1), ALIGN), (dict(ws=A + 8), ALIGN),
    (dict(N=1 << 24, rank=128, K=64, M=1), UNSUPPORTED),  # B of one adapter: 4 GiB
    (dict(M=0, A=0, B=0, rows=0, ws=0), OK),
])
def test_lora_refusals(change, want):
    assert lora(**change) == want


def test_lora_workspace_size():
    size = lb.lora_workspace_size
    assert size(0, 16) == size(-1, 16) == size(16, 12) == size(16, 0) == size(16, 136) == size(1 << 31, 16) == 0
    for M in (1, 15, 16, 17, 500, 2048, 2049, 100000, (1 << 31) - 1):
        for rank in (8, 16, 24, 64, 128):
            assert size(M, rank) >= 4096 + 4 * M * rank
    for rank in (8, 16, 64, 128):  # a workspace for some rows serves fewer
        sizes = [size(M, rank) for M in range(1, 5000, 7)]
        assert sizes == sorted(sizes) and sizes[-1] <= 4096 + 4 * 5000 * rank + (9 << 20)
    n = size(64, 16)
    assert lora(bytes=n - 1) == INVALID
    assert size(509, 32, 3072, 9216, 128, 1) > size(509, 32)            # 192 tiles of 64 x 128: K is split
    assert size(4608, 32, 9216, 3072) == size(4608, 32)                 # enough tiles
    assert size(16, 32, 3072, 9216) == size(16, 32)                     # few rows
    assert size(64, 12, 256, 256) == size(64, 16, 250, 256) == size(64, 16, 256, 256, 32) == size(0, 16, 256, 256) == 0


# ---- lowbit_qk_norm_rope ----

def qk(**kw):
    d = dict(q=A, k=A, q_out=2 * A, k_out=2 * A, q_weight=A, k_weight=A, positions=A, freqs=A, tokens=10, q_token=1024, q_head=128,
             k_token=1024, k_head=128, q_out_token=1024, q_out_head=128, k_out_token=1024, k_out_head=128, q_heads=8, k_heads=2,
             head_dim=128, axes=2, dims=(64, 32), interleaved=1, eps=1e-6)
    d.update(kw)
    dims = tuple(d["dims"]) + (0,) * (4 - len(d["dims"]))
    p = lb._QK_PROBLEM.pack(*(d[n] for n in ("q", "k", "q_out", "k_out", "q_weight", "k_weight", "positions", "freqs", "tokens", "q_token",
                                             "q_head", "k_token", "k_head", "q_out_token", "q_out_head", "k_out_token", "k_out_head",
                                             "q_heads", "k_heads", "head_dim", "axes")), *dims, d["interleaved"], d["eps"])
    return _lib.lib().lowbit_qk_norm_rope(p, None)


@pytest.mark.parametrize("change,want", [
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED), (dict(axes=5), UNSUPPORTED), (dict(axes=-1), UNSUPPORTED),
    (dict(dims=(64, 31)), INVALID), (dict(dims=(64, 0)), INVALID), (dict(dims=(64, -2)), INVALID), (dict(dims=(130, 14)), INVALID),
    (dict(dims=(64, 34)), INVALID), (dict(dims=(128, 16)), INVALID), (dict(dims=(64, 8)), INVALID),
    (dict(tokens=-1), INVALID), (dict(q_heads=-1), INVALID), (dict(k_heads=1 << 17), UNSUPPORTED),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(q_token=1020), INVALID), (dict(k_head=-128), INVALID), (dict(q_out_token=1 << 41), INVALID),
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(q_out=0), INVALID), (dict(k_out=0), INVALID), (dict(positions=0), INVALID),
    (dict(freqs=0), INVALID), (dict(q=A + 8), ALIGN), (dict(k_out=A + 8), ALIGN), (dict(q_weight=A + 4), ALIGN),
    (dict(positions=A + 2), ALIGN), (dict(freqs=A + 1), ALIGN),
    (dict(q_out_token=512), INVALID), (dict(q_out_head=64), INVALID), (dict(k_out_token=0), INVALID),  # output rows that overlap
    (dict(q_out=A, q_out_token=2048), INVALID),  # in place with another order
    (dict(tokens=0, q=0, k=0, q_out=0, k_out=0, positions=0, freqs=0), OK), (dict(q_heads=0, k_heads=0, q=0, k=0), OK),
])
def test_qk_refusals(change, want):
    assert qk(**change) == want


# ---- lowbit_attention ----

def attention_problem(**kw):
    d = dict(q=A, k=A, v=A, o=2 * A, mask=0, lens=0, start=0, batch=2, q_len=10, kv_len=20, mask_batch=20, q_heads=8, kv_heads=2,
             head_dim=128, causal=0, scale=0.1)
    d.update(kw)
    D, hq, hk = d["head_dim"], d["q_heads"], d["kv_heads"]
    st = dict(q_batch=d["q_len"] * hq * D, q_token=hq * D, q_head=D, k_batch=d["kv_len"] * hk * D, k_token=hk * D, k_head=D,
              v_batch=d["kv_len"] * hk * D, v_token=hk * D, v_head=D, o_batch=d["q_len"] * hq * D, o_token=hq * D, o_head=D)
    st.update({n: d[n] for n in st if n in d})
    st = {n: min(max(v, -(1 << 62)), 1 << 62) for n, v in st.items()}
    return lb._ATTENTION_PROBLEM.pack(d["q"], d["k"], d["v"], d["o"], d["mask"], d["lens"], d["start"], d["batch"], d["q_len"],
                                      d["kv_len"], *st.values(), d["mask_batch"], hq, hk, D, d["causal"], d["scale"])


def attention(ws=0, nbytes=0, **kw):
    return _lib.lib().lowbit_attention(attention_problem(**kw), ws, nbytes, None)


@pytest.mark.parametrize("change,want", [
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(batch=-1), INVALID), (dict(q_len=-1), INVALID),
    (dict(kv_len=-1), INVALID), (dict(q_heads=-8), INVALID), (dict(q_heads=9), INVALID), (dict(kv_heads=3), INVALID),
    (dict(kv_heads=0), INVALID), (dict(kv_len=(1 << 31) - 1), UNSUPPORTED), (dict(q_len=1 << 31), UNSUPPORTED),
    (dict(q_len=1 << 30, q_heads=8), UNSUPPORTED), (dict(batch=1 << 16, q_heads=256, kv_heads=256), UNSUPPORTED),
    (dict(batch=1 << 17), UNSUPPORTED), (dict(q_heads=1 << 17, kv_heads=1 << 17), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q_token=1020), INVALID), (dict(k_head=-128), INVALID), (dict(v_batch=1 << 41), INVALID), (dict(mask_batch=-1), INVALID),
    (dict(k_token=64), INVALID), (dict(v_token=0), INVALID), (dict(k_token=(1 << 24) + 8), UNSUPPORTED),
    (dict(o_token=512), INVALID), (dict(o_head=64), INVALID), (dict(o_batch=0), INVALID),
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(o=0), INVALID),
    (dict(q=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(o=A + 8), ALIGN), (dict(lens=A + 2), ALIGN), (dict(start=A + 1), ALIGN),
    (dict(ws=A + 8, nbytes=100), ALIGN),
    (dict(batch=0, q=0), OK), (dict(q_len=0, q=0, o=0), OK), (dict(q_heads=0, kv_heads=0, q=0, k=0, v=0, o=0), OK),
])
def test_attention_refusals(change, want):
    assert attention(**change) == want


def test_attention_scale_limits():
    """scale * log2(e) is what the kernels multiply by: it has to be a number too."""
    assert attention(scale=3.0e38) == INVALID and attention(scale=2.0 ** 127 * 1.4) == INVALID
    # past the scale's check the next one answers
    assert attention(scale=2.0 ** 127, q=0) == INVALID and attention(scale=2.0 ** 127, q=A + 8) == ALIGN
    assert attention(scale=1e-38, q=A + 8) == ALIGN


def test_null_problems():
    L = _lib.lib()
    assert L.lowbit_qk_norm_rope(None, None) == INVALID and L.lowbit_attention(None, None, 0, None) == INVALID
    assert L.lowbit_attention_workspace_size(None) == 0


@pytest.mark.parametrize("kernel", [None, "few", "many", "many64", "many128"])
def test_attention_plans(kernel, monkeypatch):
    """Workspace sizes over many shapes: none where keys are not split, room for every split's rows otherwise."""
    if kernel:
        monkeypatch.setenv("LOWBIT_ATTENTION", kernel)
    L = _lib.lib()
    size = lambda **kw: int(L.lowbit_attention_workspace_size(attention_problem(**kw)))  # noqa: E731
    assert size(head_dim=96) == size(batch=0) == size(q_len=0) == 0
    assert size(kv_len=0) == size(kv_len=1) == 0
    for batch in (1, 3, 300):
        for q_len in (1, 2, 17, 128, 1000, 5000):
            for kv_len in (1, 31, 64, 500, 4096, 40007, 1 << 20):
                for hq, hk in ((1, 1), (32, 8), (24, 24), (64, 1)):
                    for D in (64, 128):
                        n = size(batch=batch, q_len=q_len, kv_len=kv_len, q_heads=hq, kv_heads=hk, head_dim=D)
                        assert n == size(batch=batch, q_len=q_len, kv_len=kv_len, q_heads=hq, kv_heads=hk, head_dim=D, causal=1)
                        if n:
                            rows = batch * hq * q_len
                            assert (n - 4096) % ((D + 2) * 4) == 0 and n >= 4096 + 2 * rows * (D + 2) * 4
                            assert n <= 4096 + 512 * 128 * (D + 2) * 4 * 2, (batch, q_len, kv_len, hq, hk, D, n)


def test_binding_refuses_before_the_device():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        lb.qk_norm_rope(x, x, None, None, ())
    with pytest.raises(TypeError):
        lb.qk_norm_rope(x.float(), x, None, None, ())
    with pytest.raises(ValueError, match="4-D"):
        lb.attention(x, x, x)
    with pytest.raises(TypeError):
        lb.attention(None, x, x)
    assert lb.rope_freqs((8, 4), 100.0, device="cpu").tolist() == pytest.approx([1, 100 ** -0.25, 0.1, 100 ** -0.75, 1, 0.1])


def test_binding_refuses_an_output_that_is_no_tensor():
    torch = pytest.importorskip("torch")
    like = torch.zeros(1, 2, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="out must be a torch.Tensor"):
        lb._output([[0.0, 0.0]], like.shape, like)
    with pytest.raises(ValueError, match="out must be"):
        lb._output(like, (2, 2), like)
    assert lb._output(like, like.shape, like) is like


def test_under_sanitizers():
    """This file's checks against the library built with AddressSanitizer and UndefinedBehaviorSanitizer on its host code."""
    from binary_bit_gemm_amd import build as B
    if os.environ.get("LOWBIT_LIBRARY") or not os.path.exists(B.HIPCC):
        pytest.skip("already the sanitized library, or no hipcc")
    from tests.test_host_sanitizers import _stale
    if _stale(B.LIB_SAN):
        B.build(jobs=min(8, os.cpu_count() or 1), sanitize=True)
    env = dict(os.environ, LD_PRELOAD=B.sanitizer_runtime(), LOWBIT_LIBRARY=B.LIB_SAN,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0:exitcode=97",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1:exitcode=98")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-k", "not sanitizers and not binding",
                        os.path.abspath(__file__)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert ctypes.sizeof(ctypes.c_void_p) == 8
