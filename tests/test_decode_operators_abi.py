"""Host-side checks of the decoding operators (CPU only): every refusal comes before anything touches a device, and the workspace
sizes are what the calls document.  The last test runs this file against the sanitized library."""
import os
import subprocess
import sys

import pytest

import binary_bit_gemm_amd as lb
from binary_bit_gemm_amd import _lib

OK, INVALID, UNSUPPORTED, ALIGN = 0, 1, 2, 3
A = 0x10000  # a 16-byte-aligned fake address: never dereferenced by the host checks
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CACHE = dict(ck=A, cv=A, ks=A, vs=A, pages=8, page=64, heads=2, dim=128, bits=8)


def cache_fields(d):
    return [d[n] for n in ("ck", "cv", "ks", "vs", "pages", "page", "heads", "dim", "bits")]


# ---- lowbit_cache_write, lowbit_cache_read ----

def rows(function, **kw):
    d = dict(CACHE, k=A, v=A, tokens=5, k_token=256, k_head=128, v_token=256, v_head=128, slots=A)
    d.update(kw)
    return getattr(_lib.lib(), function)(lb._CACHE.pack(*cache_fields(d)), d["k"], d["v"], d["tokens"], d["k_token"], d["k_head"], d["v_token"],
                                         d["v_head"], d["slots"], None)


SHAPE_REFUSALS = [
    (dict(bits=2), UNSUPPORTED), (dict(bits=0), UNSUPPORTED), (dict(bits=32), UNSUPPORTED), (dict(dim=96), UNSUPPORTED), (dict(dim=256), UNSUPPORTED),
    (dict(page=0), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(page=-16), UNSUPPORTED),
    (dict(pages=-1), INVALID), (dict(heads=-1), INVALID), (dict(heads=(1 << 16) + 1), UNSUPPORTED), (dict(pages=1 << 25), UNSUPPORTED),
    (dict(pages=1 << 62), UNSUPPORTED), (dict(ck=0), INVALID), (dict(cv=0), INVALID), (dict(ks=0), INVALID), (dict(vs=0), INVALID),
    (dict(ck=A + 8), ALIGN), (dict(cv=A + 4), ALIGN), (dict(ks=A + 2), ALIGN), (dict(vs=A + 8), ALIGN), (dict(bits=4, vs=0), INVALID),
]


@pytest.mark.parametrize("function", ["lowbit_cache_write", "lowbit_cache_read"])
@pytest.mark.parametrize("change,want", SHAPE_REFUSALS + [
    (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), UNSUPPORTED), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(slots=0), INVALID),
    (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(slots=A + 2), ALIGN), (dict(k_token=252), INVALID), (dict(v_head=-128), INVALID),
    (dict(v_token=1 << 41), INVALID), (dict(tokens=0, k=0, v=0, slots=0), OK), (dict(heads=0, k=0), OK),
    (dict(pages=0, ck=0, cv=0, ks=0, vs=0), OK),
])
def test_rows_refusals(function, change, want):
    assert rows(function, **change) == want


def test_rows_that_overlap():
    """Rows read back must lie apart; rows written may come from one place."""
    for change in (dict(k_head=64), dict(v_token=128), dict(k_token=0), dict(v_head=0)):
        assert rows("lowbit_cache_read", **change) == INVALID
        assert rows("lowbit_cache_write", slots=A + 1, **change) == ALIGN  # past its checks of strides, not on to the device


# ---- lowbit_cache_attention ----

def problem(**kw):
    d = dict(CACHE, q=A, o=2 * A, table=A, lens=A, q_lens=0, tree=0, batch=2, q_len=3, kv_len=500, q_heads=8, scale=0.1, stride=8)
    d.update(kw)
    st = dict(q_batch=d["q_len"] * d["q_heads"] * 128, q_token=d["q_heads"] * 128, q_head=128)
    st.update({n.replace("q_", "o_"): v for n, v in st.items()})
    st.update({n: d[n] for n in st if n in d})
    st = {n: min(max(v, -(1 << 62)), 1 << 62) for n, v in st.items()}
    return lb._CACHE_ATTENTION_PROBLEM.pack(*cache_fields(d), d["q"], d["o"], d["table"], d["lens"], d["q_lens"], d["tree"], d["batch"], d["q_len"],
                                            d["kv_len"], *st.values(), d["stride"], d["q_heads"], d["scale"])


def attention(ws=0, nbytes=0, **kw):
    return _lib.lib().lowbit_cache_attention(problem(**kw), ws, nbytes, None)


@pytest.mark.parametrize("change,want", SHAPE_REFUSALS + [
    (dict(batch=-1), INVALID), (dict(q_len=-1), INVALID), (dict(kv_len=-1), INVALID), (dict(q_heads=-8), INVALID), (dict(q_heads=9), INVALID),
    (dict(heads=0), INVALID), (dict(batch=1 << 17), UNSUPPORTED), (dict(q_heads=1 << 17), UNSUPPORTED), (dict(kv_len=(1 << 31) - 1), UNSUPPORTED),
    (dict(q_len=1 << 31), UNSUPPORTED), (dict(q_len=1 << 30), UNSUPPORTED), (dict(q_len=65, tree=A), UNSUPPORTED),
    (dict(batch=1 << 16, q_len=1 << 12), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=3.0e38), INVALID), (dict(q_token=1020), INVALID), (dict(o_head=-128), INVALID), (dict(q_batch=1 << 41), INVALID),
    (dict(stride=-1), INVALID), (dict(o_token=512), INVALID), (dict(o_head=64), INVALID), (dict(o_batch=0), INVALID),
    (dict(q=0), INVALID), (dict(o=0), INVALID), (dict(table=0), INVALID), (dict(lens=0), INVALID),
    (dict(q=A + 8), ALIGN), (dict(o=A + 2), ALIGN), (dict(table=A + 2), ALIGN), (dict(lens=A + 1), ALIGN), (dict(q_lens=A + 2), ALIGN),
    (dict(tree=A + 4), ALIGN), (dict(ws=A + 8, nbytes=100), ALIGN),
    (dict(batch=0, q=0), OK), (dict(q_len=0, q=0, o=0), OK), (dict(q_heads=0, heads=0, q=0, o=0, lens=0), OK),
])
def test_attention_refusals(change, want):
    assert attention(**change) == want


def test_null_problems():
    L = _lib.lib()
    assert L.lowbit_cache_attention(None, None, 0, None) == INVALID and L.lowbit_cache_attention_workspace_size(None) == 0
    assert L.lowbit_cache_write(None, A, A, 1, 128, 128, 128, 128, A, None) == INVALID
    assert L.lowbit_cache_read(None, A, A, 1, 128, 128, 128, 128, A, None) == INVALID


def test_attention_plans():
    """Workspace sizes over many shapes: none where keys are not split, room for every split's rows otherwise."""
    size = lambda **kw: int(_lib.lib().lowbit_cache_attention_workspace_size(problem(**kw)))  # noqa: E731
    assert size(dim=96) == size(batch=0) == size(q_len=0) == size(kv_len=0) == size(kv_len=1) == 0
    assert size(batch=1, q_len=1, kv_len=40007) > 0
    for batch in (1, 3, 300):
        for q_len in (1, 2, 17, 64, 1000):
            for kv_len in (1, 31, 500, 4099, 40007, 1 << 20):
                for hq, hk in ((1, 1), (32, 8), (24, 24), (64, 1)):
                    for dim in (64, 128):
                        for bits in (4, 8, 16):
                            n = size(batch=batch, q_len=q_len, kv_len=kv_len, q_heads=hq, heads=hk, dim=dim, bits=bits, q_head=128, o_head=128)
                            if n:
                                rows_all = batch * hq * q_len
                                assert (n - 4096) % ((dim + 2) * 4) == 0 and n >= 4096 + 2 * rows_all * (dim + 2) * 4
                                assert n <= 4096 + 1024 * 64 * (dim + 2) * 4, (batch, q_len, kv_len, hq, hk, dim, bits, n)


# ---- lowbit_gemv_affine ----

def gemv(**kw):
    d = dict(X=A, W=A, S=A, B=A, R=0, Y=A, M=1, N=256, K=256, g=64, swiglu=0)
    d.update(kw)
    return _lib.lib().lowbit_gemv_affine(*(d[n] for n in ("X", "W", "S", "B", "R", "Y", "M", "N", "K", "g", "swiglu")), None)


@pytest.mark.parametrize("change,want", [
    (dict(M=17), UNSUPPORTED), (dict(M=-1), INVALID), (dict(N=250), INVALID), (dict(N=-16), INVALID), (dict(K=200), INVALID), (dict(g=128, K=192), INVALID),
    (dict(g=32), UNSUPPORTED), (dict(g=96), UNSUPPORTED), (dict(K=(1 << 22) + 64), UNSUPPORTED), (dict(N=1 << 20, K=1 << 14), UNSUPPORTED),
    (dict(N=1 << 19, K=1 << 14, swiglu=1), UNSUPPORTED), (dict(N=1 << 19, K=1 << 13, swiglu=1, R=A + 2), UNSUPPORTED),  # 2N rows: 4 GiB
    (dict(N=(1 << 19) - 16, K=1 << 13, swiglu=1, R=A + 2), ALIGN), (dict(N=1 << 19, K=1 << 13, R=A + 2), ALIGN),
    (dict(X=0), INVALID), (dict(W=0), INVALID), (dict(S=0), INVALID), (dict(B=0), INVALID), (dict(Y=0), INVALID),
    (dict(X=A + 8), ALIGN), (dict(W=A + 4), ALIGN), (dict(S=A + 2), ALIGN), (dict(B=A + 2), ALIGN), (dict(Y=A + 8), ALIGN), (dict(R=A + 2), ALIGN),
    (dict(M=0, X=0, W=0, S=0, B=0, Y=0), OK), (dict(N=0, W=0, S=0, B=0, Y=0), OK),
])
def test_gemv_refusals(change, want):
    assert gemv(**change) == want


# ---- the binding ----

def test_binding_refuses_before_the_device():
    torch = pytest.importorskip("torch")
    u8 = torch.zeros(2, 1, 16, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="bits"):
        lb.KVCache(u8, u8, bits=2)
    with pytest.raises(ValueError, match="GPU"):
        lb.KVCache(u8, u8, bits=8)
    with pytest.raises(TypeError):
        lb.KVCache(u8.float(), u8, bits=16)
    with pytest.raises(TypeError):
        lb.KVCache(None, u8, bits=8)
    with pytest.raises(ValueError, match="bits"):
        lb.kv_cache(1, 1, 64, bits=3)
    with pytest.raises(ValueError, match="head_dim"):
        lb.kv_cache(1, 1, 96)
    x = torch.zeros(1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        lb.gemv_affine(x, None, None, None, 64)
    with pytest.raises(TypeError, match="key_lens"):
        lb.cache_attention(x, None, None, None)


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


def test_a_workspace_for_every_call():
    """LOWBIT_CACHE_ATTENTION_WORKSPACE_BYTES covers any call (the size that one call can use falls as a batch grows), and no more than that is asked for."""
    size = lambda **kw: int(_lib.lib().lowbit_cache_attention_workspace_size(problem(**kw)))  # noqa: E731
    most = 0
    for batch in (1, 2, 5, 8, 17, 31, 64, 128, 255, 256, 300):
        for q_len in (1, 2, 4, 5, 16, 17, 27, 32, 33, 64, 128, 500):
            for kv_len in (300, 1000, 2100, 16000, 40007, 1 << 22):
                for hq, hk in ((1, 1), (32, 8), (16, 2), (64, 1)):
                    for dim in (64, 128):
                        for bits in (4, 8, 16):
                            n = size(batch=batch, q_len=q_len, kv_len=kv_len, q_heads=hq, heads=hk, dim=dim, bits=bits, q_head=128, o_head=128)
                            assert n <= lb.CACHE_ATTENTION_WORKSPACE_BYTES, (batch, q_len, kv_len, hq, hk, dim, bits, n)
                            most = max(most, n)
    assert most == lb.CACHE_ATTENTION_WORKSPACE_BYTES
    with open(os.path.join(ROOT, "include", "lowbit.h")) as f:
        assert f"#define LOWBIT_CACHE_ATTENTION_WORKSPACE_BYTES {lb.CACHE_ATTENTION_WORKSPACE_BYTES}\n" in f.read()
