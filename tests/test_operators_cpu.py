"""The 8-bit product and the 4-bit cache without a GPU: the oracles' own pins,
the library's refusals (host checks, before any CUDA call) and the binding's."""
import ctypes

import numpy as np
import pytest
import torch

from bit_gemv_bcq_b200 import api
from bit_gemv_bcq_b200 import build as libbuild
from oracle import i8, kv4

P16 = 0x10000   # never dereferenced: every call below is refused first


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return api.lib()


# ------------------------------------------------------------------ oracles

def test_i8_oracle_by_hand():
    q, s = i8.quantize([[254.0, 1.0, 3.0, -5.0, 253.0], [0, 0, 0, 0, 0], [1, np.nan, 0, 0, 0]])
    assert q.tolist() == [[127, 0, 2, -2, 126], [0] * 5, [0] * 5]   # 0.5, 1.5, -2.5, 126.5 to even
    assert s[0] == 2 and s[1] == 0 and np.isnan(s[2])
    assert i8.gemm([[1, -2]], [0.5], [[3, 4], [127, -128]], [2.0, 1.0]).tolist() == [[-5.0, 191.5]]


def test_kv4_oracle_by_hand():
    x = np.zeros(128)
    x[:64] = np.arange(64) % 16 * 2.0 - 6.0          # z = -6, a = 2
    x[64:] = 5.0                                     # constant: a = 0
    code, param = kv4.quantize(x)
    assert param.tolist() == [[2.0, -6.0], [0.0, 5.0]]
    assert code[:16].tolist() == list(range(16)) and not code[64:].any()
    byte = kv4.pack(code)
    assert byte[0] == 0x10 and np.array_equal(kv4.unpack(byte), code)
    assert np.array_equal(kv4.values(byte, param), x)
    x[64] = 70000.0
    assert np.isnan(kv4.quantize(x)[1][1]).all()


def test_kv4_oracle_attention_by_brute_force():
    rng = np.random.default_rng(0)
    pages, heads, ps, D, lens, new = 4, 2, 16, 64, [20, 3], [3, 2]
    k, v = (rng.integers(0, 256, (pages, heads, ps, D // 2)).astype(np.uint8) for _ in "kv")
    kp, vp = (rng.uniform(-0.3, 0.3, (pages, heads, ps, 1, 2)).astype(np.float16) for _ in "kv")
    table = np.array([[2, 0], [3, 1]])
    cu = [0, 3, 5]
    q = rng.normal(size=(5, 4, D))
    out, lse, _ = kv4.attention(q, k, kp, v, vp, table, lens, cu, 0.1, window=4)
    for b in range(2):
        for i in range(new[b]):
            pos = lens[b] - new[b] + i
            for h in range(4):
                num, den = np.zeros(D), 0.0
                for j in range(max(0, pos - 3), pos + 1):
                    where = (table[b][j // ps], h // 2, j % ps)
                    K, V = kv4.values(k[where], kp[where]), kv4.values(v[where], vp[where])
                    e = np.exp(0.1 * (q[cu[b] + i, h] * K).sum())
                    num, den = num + e * V, den + e
                np.testing.assert_allclose(out[cu[b] + i, h], num / den, rtol=1e-12)
                np.testing.assert_allclose(lse[cu[b] + i, h], np.log(den), rtol=1e-12)
    out, lse, _ = kv4.attention(q[:2], k, kp, v, vp, table, [1], [0, 2], 0.1)
    assert not out[0].any() and np.isneginf(lse[0]).all() and out[1].any()


# -------------------------------------------------- refusals of the library

def test_quantize_i8_refusals(L):
    ok = dict(x=P16, dtype=0, M=2, K=40, ldx=40, q=P16, ldq=48, scale=P16)

    def call(**kw):
        a = {**ok, **kw}
        return L.bcq_quantize_i8(a["x"], a["dtype"], a["M"], a["K"], a["ldx"], a["q"], a["ldq"],
                                 a["scale"], None)
    for name in ("x", "q", "scale"):
        assert call(**{name: None}) == api.BCQ_ERR_NULL
    for kw in (dict(M=-1), dict(K=0), dict(K=65537, ldx=65537, ldq=65552), dict(ldx=39), dict(ldq=32)):
        assert call(**kw) == api.BCQ_ERR_SHAPE, kw
    for kw in (dict(x=P16 + 1), dict(q=P16 + 8), dict(ldq=56), dict(scale=P16 + 2)):
        assert call(**kw) == api.BCQ_ERR_ALIGN, kw
    assert call(dtype=2) == api.BCQ_ERR_UNSUPPORTED
    assert call(M=0, x=None, q=None, scale=None) == api.BCQ_OK


def _product(L, name, **kw):
    a = {**dict(x=P16, ldx=48, sx=P16, w=P16, ldw=48, sw=P16, M=2, N=3, K=40, y=P16, dtype=0, ldy=3,
                ws=P16, nws=1 << 20), **kw}
    if name == "gemm":
        return L.bcq_gemm_i8(a["x"], a["ldx"], a["sx"], a["w"], a["ldw"], a["sw"], a["M"], a["N"],
                             a["K"], a["y"], a["dtype"], a["ldy"], None)
    return L.bcq_linear_i8(a["x"], a["dtype"], a["ldx"], a["w"], a["ldw"], a["sw"], a["M"], a["N"],
                           a["K"], a["y"], a["ldy"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("name", ["gemm", "linear"])
def test_product_refusals(L, name):
    for p in ("x", "w", "sw", "y") + (("sx",) if name == "gemm" else ("ws",)):
        assert _product(L, name, **{p: None}) == api.BCQ_ERR_NULL, p
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(K=65537, ldx=65552, ldw=65552), dict(ldx=32),
               dict(ldw=32), dict(ldy=2)):
        assert _product(L, name, **kw) == api.BCQ_ERR_SHAPE, kw
    for kw in (dict(w=P16 + 8), dict(ldw=56), dict(sw=P16 + 2), dict(y=P16 + 1)):
        assert _product(L, name, **kw) == api.BCQ_ERR_ALIGN, kw
    assert _product(L, name, dtype=3) == api.BCQ_ERR_UNSUPPORTED
    assert _product(L, name, M=0, x=None, sx=None, y=None, ws=None) == api.BCQ_OK
    if name == "gemm":
        for kw in (dict(x=P16 + 8), dict(ldx=56), dict(sx=P16 + 1), dict(dtype=2, y=P16 + 2)):
            assert _product(L, name, **kw) == api.BCQ_ERR_ALIGN, kw
    else:
        assert _product(L, name, dtype=2) == api.BCQ_ERR_UNSUPPORTED
        assert _product(L, name, nws=L.bcq_linear_i8_workspace_bytes(2, 40) - 1) == api.BCQ_ERR_NULL
        assert _product(L, name, ws=P16 + 4) == api.BCQ_ERR_ALIGN


def test_linear_workspace(L):
    assert L.bcq_linear_i8_workspace_bytes(3, 40) == 3 * 48 + 16
    assert L.bcq_linear_i8_workspace_bytes(1 << 20, 65536) == (1 << 36) + (1 << 22)
    for bad in ((-1, 40), (3, 0), (3, 65537)):
        assert L.bcq_linear_i8_workspace_bytes(*bad) == 0


def _cache(**kw):
    a = {**dict(k=P16, k_param=P16, v=P16, v_param=P16, pages=4, heads=2, page_size=32, head_dim=128), **kw}
    return ctypes.byref(api._Kv4(*a.values()))


CACHE_FAULTS = [(dict(k=None), api.BCQ_ERR_NULL), (dict(v_param=None), api.BCQ_ERR_NULL),
                (dict(pages=0), api.BCQ_ERR_SHAPE), (dict(heads=0), api.BCQ_ERR_SHAPE),
                (dict(page_size=8), api.BCQ_ERR_SHAPE), (dict(page_size=40), api.BCQ_ERR_SHAPE),
                (dict(head_dim=96), api.BCQ_ERR_UNSUPPORTED), (dict(k=P16 + 8), api.BCQ_ERR_ALIGN),
                (dict(v_param=P16 + 4), api.BCQ_ERR_ALIGN)]
PLACE_FAULTS = [(dict(table=None), api.BCQ_ERR_NULL), (dict(kv_len=None), api.BCQ_ERR_NULL),
                (dict(cu=None), api.BCQ_ERR_SHAPE), (dict(T=-1), api.BCQ_ERR_SHAPE),
                (dict(B=0), api.BCQ_ERR_SHAPE), (dict(W=0), api.BCQ_ERR_SHAPE),
                (dict(W=1 << 27), api.BCQ_ERR_SHAPE), (dict(table=P16 + 2), api.BCQ_ERR_ALIGN),
                (dict(cu=P16 + 1), api.BCQ_ERR_ALIGN)]


def _kv4(L, name, cache=None, **kw):
    a = {**dict(x=P16, y=P16, ld=256, hd=128, dtype=0, T=5, table=P16, W=8, kv_len=P16, cu=P16, B=2,
                H=4, max_q=4, max_kv=100, window=0, scale=0.1, out=P16, ldo=512, hdo=128, lse=None,
                ws=P16, nws=1 << 30), **kw}
    c = cache if cache is not None else _cache()
    places = (a["table"], a["W"], a["kv_len"], a["cu"], a["B"])
    if name == "append":
        return L.bcq_kv4_append(c, a["x"], a["ld"], a["hd"], a["y"], a["ld"], a["hd"], a["dtype"],
                                a["T"], *places, None)
    if name == "read":
        return L.bcq_kv4_read(c, a["x"], a["y"], a["dtype"], a["T"], *places, None)
    return L.bcq_kv4_attention(c, a["x"], a["ld"], a["hd"], a["dtype"], a["T"], a["H"], *places,
                               a["max_q"], a["max_kv"], 1, a["window"], a["scale"], a["out"],
                               a["ldo"], a["hdo"], a["lse"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("name", ["append", "read", "attention"])
def test_kv4_refusals(L, name):
    for kw, want in CACHE_FAULTS:
        assert _kv4(L, name, cache=_cache(**kw)) == want, kw
    for kw, want in PLACE_FAULTS + [(dict(x=None), api.BCQ_ERR_NULL), (dict(x=P16 + 8), api.BCQ_ERR_ALIGN),
                                    (dict(dtype=3), api.BCQ_ERR_UNSUPPORTED)]:
        assert _kv4(L, name, **kw) == want, kw
    assert _kv4(L, name, T=0) == api.BCQ_OK
    if name != "attention":
        assert _kv4(L, name, y=None) == api.BCQ_ERR_NULL
    if name != "read":
        assert _kv4(L, name, dtype=2) == api.BCQ_ERR_UNSUPPORTED
        for kw in (dict(ld=260), dict(hd=4)):
            assert _kv4(L, name, **kw) == api.BCQ_ERR_ALIGN, kw
        assert _kv4(L, name, ld=-8) == api.BCQ_ERR_SHAPE


def test_kv4_attention_refusals(L):
    for kw in (dict(H=0), dict(H=3), dict(H=2 * 129), dict(max_q=0), dict(max_kv=0), dict(window=-1),
               dict(scale=float("inf")), dict(scale=float("nan"))):
        assert _kv4(L, "attention", **kw) == api.BCQ_ERR_SHAPE, kw
    assert _kv4(L, "attention", out=None) == api.BCQ_ERR_NULL
    assert _kv4(L, "attention", out=P16 + 4) == api.BCQ_ERR_ALIGN
    assert _kv4(L, "attention", hdo=4) == api.BCQ_ERR_ALIGN
    assert _kv4(L, "attention", lse=P16 + 2) == api.BCQ_ERR_ALIGN
    for kw in (dict(ldo=504), dict(ldo=128), dict(hdo=64), dict(ldo=0), dict(hdo=0), dict(ldo=64, hdo=512)):
        assert _kv4(L, "attention", **kw) == api.BCQ_ERR_SHAPE, kw        # vectors of out that overlap


@pytest.mark.parametrize("name", ["append", "read", "attention"])
def test_kv4_positions_are_counted_in_an_int(L, name):
    """At most 2^30 positions of a sequence; no GPU is needed to refuse more (T = 0 runs nothing)."""
    assert _kv4(L, name, T=0, W=1 << 25) == api.BCQ_OK
    assert _kv4(L, name, T=0, W=(1 << 25) + 1) == api.BCQ_ERR_SHAPE


# -------------------------------------------------------------- fast calls

def test_fast_module_leaves_other_calls_alone(L):
    """Bound to the library, and NotImplemented for whatever is no usual call:
    tensors that are not on a GPU, other objects, other numbers of arguments."""
    f = api._fast()
    h, i = torch.zeros(4, 64, dtype=torch.float16), torch.zeros(4, 64, dtype=torch.int8)
    for call in (f.quantize_i8, f.gemm_i8, f.linear_i8, f.kv4_append, f.kv4_read, f.kv4_attention):
        for n in range(16):
            assert call(*[h] * n) is NotImplemented
            assert call(*[None] * n) is NotImplemented
            assert call(*[i, "x", 1, None, 2.5][:n]) is NotImplemented
    with pytest.raises(TypeError):
        f.bind(1, 2)
    with pytest.raises(ValueError):
        f.bind(*[0] * 8)
    for n, call in (("quantize_i8", lambda: api.quantize_i8(h)),
                    ("linear_i8", lambda: api.linear_i8(h, i, h[0].float()))):
        with pytest.raises(ValueError):
            call()


def test_numbers_beyond_an_int_are_refused(L):
    """ctypes would take their low 32 bits: a window of 2^32 + 1 would be one of 1."""
    for big in ((1 << 32) + 1, 1 << 31, -(1 << 31) - 1):
        with pytest.raises(api.BcqError) as e:
            api._run("bcq_quantize_i8", 0, P16, 0, big, 16, 16, P16, 16, P16, None)
        assert e.value.status == api.BCQ_ERR_SHAPE


# -------------------------------------------------- refusals of the binding

@pytest.fixture
def host(monkeypatch):
    """CPU tensors pass for CUDA ones; a call that reaches the library fails the test."""
    class Cuda(torch.Tensor):
        is_cuda = True

    class NoLibrary:
        def __getattr__(self, name):
            def call(*a):
                if name.endswith("_bytes"):
                    return 0
                raise AssertionError(name + " was reached")
            return call
    libbuild.build()
    api._fast()
    monkeypatch.setattr(api, "lib", lambda: NoLibrary())
    return lambda *size, dtype=torch.float16: torch.zeros(*size, dtype=dtype).as_subclass(Cuda)


def _refused(calls):
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"case {i} was not refused")


def test_i8_binding_refusals(host):
    i8t, f32 = torch.int8, torch.float32
    x, s, w, sw = host(4, 64, dtype=i8t), host(4, dtype=f32), host(6, 64, dtype=i8t), host(6, dtype=f32)
    h = host(4, 64)
    _refused([
        lambda: api.quantize_i8(torch.zeros(4, 64, dtype=torch.float16)),
        lambda: api.quantize_i8(host(4, 64, dtype=f32)),
        lambda: api.quantize_i8(host(64)),
        lambda: api.quantize_i8(h.t()),
        lambda: api.quantize_i8(host(1, 64).expand(4, 64)),
        lambda: api.gemm_i8(x[:, 1:], s, w[:, 1:], sw),                # rows off 16 bytes
        lambda: api.gemm_i8(host(4, 40, dtype=i8t), s, host(6, 40, dtype=i8t), sw),
        lambda: api.gemm_i8(x, s[:3], w, sw),
        lambda: api.gemm_i8(x, s.half(), w, sw),
        lambda: api.gemm_i8(x, s, w[:, :48], sw),
        lambda: api.gemm_i8(x, s, w, s),
        lambda: api.gemm_i8(x, s, w, sw, dtype=torch.float64),
        lambda: api.gemm_i8(x, s, w, sw, out=host(4, 5)),
        lambda: api.gemm_i8(x, s, w, sw, out=host(4, 6, dtype=f32)),
        lambda: api.gemm_i8(x, s, w, sw, out=host(6, 4).t()),
        lambda: api.gemm_i8(x, s, w, sw, out=host(1, 6).expand(4, 6)),
        lambda: api.linear_i8(x, w, sw),
        lambda: api.linear_i8(h, w.half(), sw),
        lambda: api.linear_i8(h[:, :32], w, sw),
        lambda: api.linear_i8(h, w, sw, out=host(4, 6, dtype=torch.bfloat16)),
    ])


def test_kv4_binding_refusals(host):
    u8, i32 = torch.uint8, torch.int32

    def cache(page=16, D=128, heads=2, **kw):
        a = dict(k=host(4, heads, page, D // 2, dtype=u8), k_param=host(4, heads, page, D // 64, 2),
                 v=host(4, heads, page, D // 2, dtype=u8), v_param=host(4, heads, page, D // 64, 2))
        a.update(kw)
        return api.Kv4Cache(**a)
    c = cache()
    table, n, cu = host(2, 3, dtype=i32), host(2, dtype=i32), host(3, dtype=i32)
    k, q = host(5, 2, 128), host(5, 4, 128)
    _refused([
        lambda: cache(page=8), lambda: cache(page=24), lambda: cache(D=192),
        lambda: cache(k_param=host(4, 2, 16, 1, 2)),
        lambda: cache(k=host(4, 2, 16, 64)),
        lambda: cache(v=host(5, 2, 16, 64, dtype=u8), v_param=host(5, 2, 16, 2, 2)),
        lambda: cache(v=host(4, 2, 64, 16, dtype=u8).transpose(2, 3)),
        lambda: api.kv4_append(c, k, k[:4], table, n, cu),
        lambda: api.kv4_append(c, k, k.bfloat16(), table, n, cu),
        lambda: api.kv4_append(c, q, q, table, n, cu),
        lambda: api.kv4_append(c, k.float(), k.float(), table, n, cu),
        lambda: api.kv4_append(c, host(5, 2, 256)[..., ::2], k, table, n, cu),
        lambda: api.kv4_append(c, host(5, 2, 132)[..., :128], k, table, n, cu),
        lambda: api.kv4_append(c, host(5, 2, 136)[..., 4:132], k, table, n, cu),
        lambda: api.kv4_append(c, k, k, table, n),                     # 5 rows, 2 sequences
        lambda: api.kv4_append(c, k, k, table, n, n),
        lambda: api.kv4_append(c, k, k, table.long(), n, cu),
        lambda: api.kv4_append(c, k, k, table[:, ::2], n, cu),
        lambda: api.kv4_append(c, k, k, table, cu, cu),
        lambda: api.kv4_read(c, table, n, cu),
        lambda: api.kv4_read(c, table, n, cu, tokens=5, dtype=torch.float64),
        lambda: api.kv4_read(c, table, n, cu, k=k),
        lambda: api.kv4_read(c, table, n, cu, k=k, v=q),
        lambda: api.kv4_attention(host(5, 3, 128), c, table, n, cu),
        lambda: api.kv4_attention(host(5, 4, 64), c, table, n, cu),
        lambda: api.kv4_attention(host(20, 128), c, table, n, cu),
        lambda: api.kv4_attention(q, c, table, n),
        lambda: api.kv4_attention(q, c, table, n, cu, out=host(4, 4, 128)),
        lambda: api.kv4_attention(q, c, table, n, cu, out=host(5, 4, 128, dtype=torch.bfloat16)),
        lambda: api.kv4_attention(q, c, table, n, cu, out=host(5, 1, 128).expand(5, 4, 128)),
        lambda: api.kv4_attention(q, c, table, n, cu, out=host(1, 4, 128).expand(5, 4, 128)),
    ])


def test_impatience_is_a_switch():
    L = api.lib()
    assert L.bcq_debug_impatient(2) == api.BCQ_ERR_SHAPE and L.bcq_debug_impatient(-1) == api.BCQ_ERR_SHAPE
    assert L.bcq_debug_impatient(1) == api.BCQ_OK and L.bcq_debug_impatient(0) == api.BCQ_OK


def test_the_library_is_built_without_torch_or_a_compiler(monkeypatch, tmp_path, capsys):
    """The fast calls' module is left out, one of an older build with it; libbcq.so is not."""
    import importlib.util
    fast = tmp_path / "_fast.so"
    monkeypatch.setattr(libbuild, "FAST", str(fast))
    find = importlib.util.find_spec
    for change in ("torch", "compiler"):
        fast.write_bytes(b"old")
        with monkeypatch.context() as m:
            if change == "torch":
                m.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
            else:
                m.setenv("CXX", str(tmp_path / "no-such-compiler"))
            assert libbuild.build() == libbuild.LIB
        assert not fast.exists() and "left out" in capsys.readouterr().err


def test_the_binding_works_without_the_fast_calls(monkeypatch, L):
    import sys
    import bit_gemv_bcq_b200 as package
    monkeypatch.setattr(api, "_fast_module", None)
    monkeypatch.setitem(sys.modules, "bit_gemv_bcq_b200._fast", None)
    monkeypatch.delattr(package, "_fast", raising=False)
    with pytest.warns(RuntimeWarning, match="fast calls"):
        f = api._fast()
    assert f.quantize_i8(1) is NotImplemented and f.kv4_append(1, 2) is NotImplemented
    assert api._fast() is f
    with pytest.raises(ValueError, match="CUDA tensor"):       # the longer way refuses as ever
        api.quantize_i8(torch.zeros(2, 16, dtype=torch.float16))
