"""The 4-bit key/value cache on the GPU against the fp64 oracle (oracle/kv4.py).

Codes, scales and offsets have to be the oracle's, bit for bit, and what is
read back is a c + z in fp32 (one rounding) rounded to its type.

Attention's tolerance counts its roundings, each at most half a step of its
type, u = 2^-11 for fp16 and e = 2^-24 for fp32.  A value of K or V may be
rounded to fp16 once (u of its magnitude a c + |z|), and p or p a once (u):
  scores    ds <= S (u + 4 D e) with S = |scale| sum |q| (a c + |z|), the sums
            over D and the two scalings in fp32; exp2's argument, up to
            |s| log2 e < 2 S, is rounded to fp32 and its result is good to a
            few steps: 16 e (1 + S) more;
  weights   p is off by at most 2 ds of itself (numerator and sum), and by u;
  output    A (2 ds + 2 u + n 4 e) with A = sum p (a c + |z|), n positions
            summed in fp32, and half a step of the output's type;
  lse       ds, n 4 e and fp32's own step.
"""
import numpy as np
import pytest
import torch

from bit_gemv_bcq_b200 import api
from oracle import kv4

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()
    yield
    assert api.device_error() == api.BCQ_OK


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _f64(t):
    return t.double().cpu().numpy()


class Case:
    """A cache of drawn codes behind a shuffled table; NaN wherever no token is."""

    def __init__(self, lens, new, heads, D, page_size, seed=0, extra=0, spare=2):
        self.lens, self.new = list(lens), list(new)
        B = len(lens)
        rng = np.random.default_rng(seed)
        W = max(1, -(-max(max(lens), 1) // page_size)) + extra
        pages = W * B + spare
        self.table = rng.permutation(pages)[:W * B].reshape(B, W).astype(np.int32)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        shape = (pages, heads, page_size)
        self.arrays = {}
        for part in ("k", "v"):
            a = rng.uniform(0.05, 0.4, (*shape, D // 64)).astype(np.float16)
            z = (rng.normal(0, 0.5, a.shape) - 7.5 * a).astype(np.float16)
            param = np.stack([a, z], -1)
            live = np.zeros((pages, page_size), dtype=bool)
            for b, n in enumerate(lens):
                at = np.arange(n)
                live[self.table[b][at // page_size], at % page_size] = True
            param.transpose(0, 2, 1, 3, 4)[~live] = np.nan
            self.arrays[part] = rng.integers(0, 256, (*shape, D // 2)).astype(np.uint8)
            self.arrays[part + "_param"] = param
        self.cache = api.Kv4Cache(*(torch.from_numpy(self.arrays[n]).cuda()
                                    for n in ("k", "k_param", "v", "v_param")))
        self.t_table, self.t_len, self.t_cu = (torch.from_numpy(x).cuda() for x in (
            self.table, np.array(lens, dtype=np.int32), self.cu))

    @property
    def T(self):
        return int(self.cu[-1])


def _queries(T, H, D, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, D, generator=g) * scale).to(dtype).cuda()


U, E = 2.0 ** -11, 2.0 ** -24


def _tolerances(S, A, ref, n, D, dtype):
    """(ds, the output's tolerance) of the header, S [...], A and ref [..., D]."""
    ds = S * (U + 4 * D * E) + 16 * E * (1 + S)
    tol = A * (2 * ds + 2 * U + 4 * n * E)[..., None]
    return ds, tol + torch.finfo(dtype).eps / 2 * np.abs(ref) + 2.0 ** -25


def _check_attention(c, q, out, lse, scale=None, causal=True, window=0, what=""):
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    scale32 = float(np.float32(scale))
    ro, rl, mag = kv4.attention(_f64(q), c.arrays["k"], c.arrays["k_param"], c.arrays["v"],
                                c.arrays["v_param"], c.table, c.lens, c.cu, scale32, causal, window)
    n = max(c.lens)
    ds, tol = _tolerances(mag["s"], mag["v"], ro, n, D, q.dtype)
    err = np.abs(_f64(out) - ro)
    assert np.isfinite(_f64(out)).all(), what
    assert (err <= tol).all(), f"{what}: worst {err.max():.3e} of {tol.max():.3e}, {(err > tol).sum()} outside"
    if lse is not None:
        got = _f64(lse)
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(got), empty), what
        d = np.abs(got[~empty] - rl[~empty])
        t = (ds + 4 * n * E + 2 * E * np.abs(np.where(empty, 0, rl)))[~empty]
        assert (d <= t).all(), f"{what}: lse off by {d.max():.3e}"


# Hints for max_kv: what the case has (few positions: the kernel of few rows),
# and one under which the kernel of many rows runs wherever there are many.
HINTS = pytest.mark.parametrize("hint", [None, 4000])


def _run(c, q, hint=None, **kw):
    args = dict(max_q=max(c.new), max_kv=hint or max(max(c.lens), 1), return_lse=True)
    args.update(kw)
    return api.kv4_attention(q, c.cache, c.t_table, c.t_len, c.t_cu, **args)


# ------------------------------------------------------------------- append

def _append_case(lens, new, heads, D, page_size, dtype, seed=0, scale=1.0):
    c = Case(lens, new, heads, D, page_size, seed)
    g = torch.Generator().manual_seed(seed)
    row = torch.randn(c.T + 1, (4 + 2 * heads) * D + 8, generator=g) * scale  # a fused projection's rows
    row = row.to(dtype).cuda()
    k = row[:c.T, 4 * D:(4 + heads) * D].view(c.T, heads, D)
    v = row[:c.T, (4 + heads) * D:(4 + 2 * heads) * D].view(c.T, heads, D)
    return c, k, v


def _expect_append(c, k, v):
    page_size = c.arrays["k"].shape[2]
    want = {n: x.copy() for n, x in c.arrays.items()}
    for part, x in (("k", k), ("v", v)):
        code, param = kv4.quantize(_f64(x))
        for b, n in enumerate(c.lens):
            for i in range(c.new[b]):
                j = n - c.new[b] + i
                if j < 0:
                    continue
                p, o = c.table[b, j // page_size], j % page_size
                want[part][p, :, o] = kv4.pack(code[c.cu[b] + i])
                want[part + "_param"][p, :, o] = param[c.cu[b] + i]
    return want


def _check_cache(c, want):
    for n in ("k", "k_param", "v", "v_param"):
        got = getattr(c.cache, n).cpu().numpy()
        assert np.array_equal(got.view(np.uint8 if n in "kv" else np.uint16),
                              want[n].view(np.uint8 if n in "kv" else np.uint16)) or \
            np.array_equal(got, want[n], equal_nan=True), n


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,new,heads,D,page_size", [
    ([1], [1], 1, 64, 16), ([5, 40], [5, 1], 2, 128, 16), ([33, 16, 100], [17, 0, 64], 3, 64, 32),
    ([70, 3], [70, 2], 8, 128, 48), ([20], [20], 1, 256, 16), ([200, 1, 0], [129, 1, 0], 4, 128, 64)])
def test_append_writes_the_oracles_codes_and_nothing_else(lens, new, heads, D, page_size, dtype):
    c, k, v = _append_case(lens, new, heads, D, page_size, dtype)
    api.kv4_append(c.cache, k, v, c.t_table, c.t_len, c.t_cu)
    _check_cache(c, _expect_append(c, k, v))


@pytest.mark.parametrize("heads,D", [(1, 64), (1, 128), (1, 256), (2, 64), (3, 64), (5, 64), (2, 128), (3, 128), (7, 64),
                                     (8, 64)])
def test_many_rows_of_few_heads_in_and_out(heads, D):
    """Rows that share a block, some of them of no sequence, and a page that is missing."""
    lens, new = [2500, 0, 70, 1900], [2300, 0, 70, 1833]
    c, k, v = _append_case(lens, new, heads, D, 48, F16)
    T = c.T
    pad = lambda x: torch.cat([x[:5] * float("nan"), x, x[:9] * float("nan")])   # noqa: E731
    cu = c.t_cu + 5
    api.kv4_append(c.cache, pad(k), pad(v), c.t_table, c.t_len, cu)
    d, _, _ = _append_case(lens, new, heads, D, 48, F16)
    for b in range(4):                                        # the same, a few rows a call
        for i in range(0, new[b], 350):
            r = slice(int(c.cu[b]) + i, int(c.cu[b]) + min(i + 350, new[b]))
            n = r.stop - r.start
            api.kv4_append(d.cache, k[r], v[r], d.t_table[b:b + 1], _i32([lens[b] - new[b] + i + n]), _i32([0, n]))
    for n in ("k", "k_param", "v", "v_param"):
        assert torch.equal(getattr(c.cache, n).view(torch.uint8), getattr(d.cache, n).view(torch.uint8)), n
    for dtype in (F16, F32):
        rk, rv = (torch.full((T + 14, heads, D), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        api.kv4_read(c.cache, c.t_table, c.t_len, cu, dtype=dtype, k=rk, v=rv)
        assert (rk[:5] == 7).all() and (rk[T + 5:] == 7).all() and (rv[T + 5:] == 7).all()
        sk, sv = api.kv4_read(d.cache, d.t_table[3:], d.t_len[3:], _i32([0, 333]), tokens=333, dtype=dtype)
        assert torch.equal(rk[T + 5 - 333:T + 5], sk) and torch.equal(rv[T + 5 - 333:T + 5], sv)
    t = c.t_table.clone()
    t[0, 10] = -1                                             # positions 480..527: rows 280..327 of the first
    before = c.cache.k.clone()
    api.kv4_append(c.cache, pad(k), pad(v), t, c.t_len, cu)
    assert api.device_error() == api.BCQ_ERR_PAGE and torch.equal(before, c.cache.k)
    gk, _ = api.kv4_read(c.cache, t, c.t_len, cu, tokens=T + 14)
    assert api.device_error() == api.BCQ_ERR_PAGE
    ok, _ = api.kv4_read(c.cache, c.t_table, c.t_len, cu, tokens=T + 14)
    assert (gk[285:333] == 0).all() and torch.equal(gk[5:285], ok[5:285]) and torch.equal(gk[333:T + 5], ok[333:T + 5])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_append_one_row_each_without_cu(dtype):
    lens = [3, 17, 64, 1]
    c, k, v = _append_case(lens, [1] * 4, 2, 128, 16, dtype)
    api.kv4_append(c.cache, k, v, c.t_table, c.t_len)
    _check_cache(c, _expect_append(c, k, v))
    a = api.kv4_read(c.cache, c.t_table, c.t_len, dtype=dtype)
    b = api.kv4_read(c.cache, c.t_table, c.t_len, c.t_cu, tokens=4, dtype=dtype)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_groups_at_the_edge_of_the_format(dtype):
    D, rows = 128, []
    ramp = torch.linspace(-1, 1, 64, dtype=torch.float64)
    half = torch.arange(64, dtype=torch.float64) / 2          # steps of a half: every quotient a half or whole
    rows.append(torch.cat([torch.zeros(64), torch.full((64,), 3.25)]))           # constant: a = 0
    rows.append(torch.cat([half.clamp(max=15), -half.clamp(max=15)]))           # a = 1: halves to even
    rows.append(torch.cat([ramp * 59000, ramp * 60000]))
    rows.append(torch.cat([ramp * 1e-7, ramp * 6e-5]))                          # a is subnormal or zero
    rows.append(torch.cat([ramp * 61000, ramp]))                                # beyond the range: NaN
    rows.append(torch.cat([ramp, torch.where(ramp == 1, float("nan"), ramp)]))
    rows.append(torch.cat([torch.where(ramp == 1, float("inf"), ramp), ramp]))
    rows.append(torch.cat([1000 + ramp, 1e-3 * ramp - 500]))                    # a small range far from zero
    x = torch.stack([r.double() for r in rows]).to(dtype)
    T = len(rows)
    c = Case([T], [T], 1, D, 16)
    k = x.view(T, 1, D).cuda()
    v = k.flip(0).contiguous()
    api.kv4_append(c.cache, k, v, c.t_table, c.t_len, c.t_cu)
    _check_cache(c, _expect_append(c, k, v))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_halves_decided_exactly(dtype):
    # offsets and steps for which (x - z) / a is a half, or next to one, all over the range
    rng = np.random.default_rng(5)
    T, D = 2000, 64
    a = rng.uniform(0.01, 3, (T, 1)).astype(np.float16).astype(np.float64)
    z = rng.normal(0, 2, (T, 1)).astype(np.float16).astype(np.float64)
    c = np.concatenate([np.zeros((T, 1)), np.full((T, 1), 15.0),
                        rng.integers(0, 15, (T, D - 2)) + 0.5], 1)
    x = torch.from_numpy((z + a * c)[:, None, :]).to(dtype).cuda()
    k = Case([T], [T], 1, D, 64)
    api.kv4_append(k.cache, x, x, k.t_table, k.t_len, k.t_cu)
    _check_cache(k, _expect_append(k, x, x))


def test_rows_of_no_sequence_are_not_read_or_written():
    c, k, v = _append_case([20, 9], [4, 9], 2, 128, 16, F16)
    k2 = torch.cat([torch.full((3, 2, 128), float("nan"), dtype=F16, device="cuda"), k,
                    torch.full((5, 2, 128), float("nan"), dtype=F16, device="cuda")])
    v2 = torch.cat([k2[:3], v, k2[-5:]])
    cu = c.t_cu + 3
    api.kv4_append(c.cache, k2, v2, c.t_table, c.t_len, cu)
    want = _expect_append(c, k, v)
    _check_cache(c, want)
    c.arrays = want
    rk = torch.full((c.T + 8, 2, 128), 7.0, dtype=F16, device="cuda")
    rv = rk.clone()
    api.kv4_read(c.cache, c.t_table, c.t_len, cu, k=rk, v=rv)
    assert (rk[:3] == 7).all() and (rk[-5:] == 7).all() and (rv[:3] == 7).all() and (rv[-5:] == 7).all()
    wk, _ = api.kv4_read(c.cache, c.t_table, c.t_len, c.t_cu, tokens=c.T)
    assert torch.equal(rk[3:-5], wk)
    q = _queries(c.T + 8, 4, 128, F16)
    out = torch.full_like(q, 7.0)
    api.kv4_attention(q, c.cache, c.t_table, c.t_len, cu, max_q=9, out=out)
    assert (out[:3] == 7).all() and (out[-5:] == 7).all()
    _check_attention(c, q[3:-5], out[3:-5], None)


# --------------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_read_gives_the_values(D, dtype):
    c = Case([40, 7, 0, 129], [33, 7, 0, 50], 3, D, 32)
    k, v = api.kv4_read(c.cache, c.t_table, c.t_len, c.t_cu, tokens=c.T, dtype=dtype)
    for got, part in ((k, "k"), (v, "v")):
        for b, n in enumerate(c.lens):
            val = kv4.values(kv4.gather(c.arrays[part], c.table[b], n),
                             kv4.gather(c.arrays[part + "_param"], c.table[b], n))[n - c.new[b]:]
            # a c + z: its bits span less than fp64's, so fp32's rounding of it is the fused one
            want = torch.from_numpy(val.astype(np.float32)).to(dtype)
            assert torch.equal(got[c.cu[b]:c.cu[b + 1]].cpu(), want), (part, b)


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H,heads", [(1, 1), (4, 4), (8, 2), (8, 1), (7, 1), (12, 4), (32, 2), (20, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_token_each(D, H, heads, dtype):
    lens = [1, 2, 15, 16, 17, 63, 100, 0, 257]
    c = Case(lens, [1] * len(lens), heads, D, 16, seed=H)
    q = _queries(len(lens), H, D, dtype)
    out, lse = _run(c, q)
    _check_attention(c, q, out, lse, what=f"D={D} H={H}/{heads}")
    o2 = api.kv4_attention(q, c.cache, c.t_table, c.t_len)       # no cu, no hints
    _check_attention(c, q, o2, None)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,new,H,heads,D,page_size", [
    ([5], [5], 2, 1, 64, 16), ([40, 3, 77], [7, 3, 2], 8, 2, 128, 16), ([130, 64], [33, 64], 4, 4, 64, 32),
    ([300], [150], 12, 3, 128, 48), ([600, 530], [300, 1], 8, 2, 128, 16), ([520], [400], 7, 1, 256, 48),
    ([1100], [97], 2, 2, 64, 16), ([129, 5], [129, 5], 32, 2, 128, 16), ([70, 0, 71], [5, 0, 70], 6, 1, 256, 64), ([256], [256], 2, 2, 128, 128),
    ([1000, 513], [3, 129], 4, 1, 128, 64), ([260, 259], [1, 140], 5, 1, 64, 16)])
@HINTS
def test_several_rows(lens, new, H, heads, D, page_size, dtype, hint):
    c = Case(lens, new, heads, D, page_size, seed=sum(lens))
    q = _queries(c.T, H, D, dtype, seed=1)
    out, lse = _run(c, q, hint)
    _check_attention(c, q, out, lse)


@pytest.mark.parametrize("causal,window", [(True, 1), (True, 5), (True, 16), (True, 64), (True, 1000),
                                           (False, 0), (False, 9), (True, 512), (False, 600)])
@pytest.mark.parametrize("lens,new", [([33, 100], [1, 1]), ([50, 20], [20, 20]), ([200], [140]),
                                      ([700, 90], [150, 90])])
@HINTS
@pytest.mark.parametrize("D", [64, 128, 256])
def test_masks(lens, new, causal, window, hint, D):
    c = Case(lens, new, 2, D, 16, seed=window)
    q = _queries(c.T, 8, D, F16, seed=2)
    out, lse = _run(c, q, hint, causal=causal, window=window)
    _check_attention(c, q, out, lse, causal=causal, window=window)


@pytest.mark.parametrize("n,new,H", [(3, 8, 4), (0, 2, 8), (10, 200, 4), (0, 1, 1), (0, 300, 2), (70, 300, 4)])
@HINTS
def test_rows_that_see_nothing(n, new, H, hint):
    """More rows than tokens: the first rows lie before position 0."""
    c = Case([n, 40], [new, 1], 1, 128, 16)
    q = _queries(c.T, H, 128, F16)
    out, lse = _run(c, q, hint)
    _check_attention(c, q, out, lse)
    empty = max(0, new - n)
    assert (out[:empty] == 0).all() and torch.isneginf(lse[:empty]).all()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 30, 2 ** 20])
@pytest.mark.parametrize("new", [8, 300])
@HINTS
def test_widest_windows_hide_nothing(window, new, hint):
    """The first rows lie before position 0, from which the window is counted."""
    c = Case([3, 40], [new, 1], 1, 128, 16)
    q = _queries(c.T, 4, 128, F16)
    out, lse = _run(c, q, hint, window=window)
    _check_attention(c, q, out, lse)
    with pytest.raises(api.BcqError):
        _run(c, q, hint, window=2 ** 32 + 1)


@pytest.mark.parametrize("new", [1, 4, 160])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 4.0])
@HINTS
def test_scales_of_the_scores(scale, new, hint):
    c = Case([200, 30], [new, 1], 2, 64, 16)
    q = _queries(c.T, 4, 64, F16)
    out, lse = _run(c, q, hint, scale=scale)
    _check_attention(c, q, out, lse, scale=scale)


@pytest.mark.parametrize("new", [1, 150])
@pytest.mark.parametrize("dtype,mag", [(F16, 1e-4), (F16, 300.0), (F16, 3e4), (BF16, 1e-12), (BF16, 1e6), (BF16, 1e30)])
@HINTS
def test_queries_of_any_magnitude(dtype, mag, new, hint):
    """The factor keeps the scores where they are; fp16's and fp32's ranges must not matter in between."""
    c = Case([180, 9], [new, 1], 2, 128, 16)
    q = _queries(c.T, 4, 128, dtype).float().clamp(-2, 2).mul(mag).to(dtype)
    scale = 128 ** -0.5 / mag
    out, lse = _run(c, q, hint, scale=scale)
    _check_attention(c, q, out, lse, scale=scale)


@pytest.mark.parametrize("new", [1, 6, 140])
@pytest.mark.parametrize("D", [64, 128, 256])
@HINTS
def test_nan_stays_where_it_belongs(new, D, hint):
    c = Case([160, 50], [new, 1], 2, D, 16)
    q = _queries(c.T, 8, D, F16)
    ref, _ = _run(c, q, hint)
    q2 = q.clone()
    q2[0, 3, 5] = float("nan")
    q2[-1, 6, 0] = float("inf")
    out, _ = _run(c, q2, hint)
    assert torch.isnan(out[0, 3]).all() and torch.isnan(out[-1, 6]).all()
    keep = torch.ones(c.T, 8, dtype=torch.bool)
    keep[0, 3] = keep[-1, 6] = False
    assert torch.equal(out[keep], ref[keep])
    # a NaN group in the second sequence's key of head 1: that head's rows, nothing else
    p = int(c.table[1, 0])
    c.cache.k_param[p, 1, 3, 0] = float("nan")
    out, _ = _run(c, q, hint)
    assert torch.isnan(out[-1, 4:]).all()
    assert torch.equal(out[-1, :4], ref[-1, :4]) and torch.equal(out[:-1], ref[:-1])
    # NaN groups in the first sequence's values, at a position that only the rows
    # from it on see: that group's outputs of those rows
    j, g = 160 - new + new // 2, D // 64 - 1
    p, o = int(c.table[0, j // 16]), j % 16
    c.cache.v_param[p, 0, o, g, 0] = float("nan")
    out, lse = _run(c, q, hint)
    seen = out[new // 2:new, :4]
    assert torch.isnan(seen[..., 64 * g:]).all() and torch.equal(seen[..., :64 * g], ref[new // 2:new, :4, :64 * g])
    assert torch.equal(out[:new // 2, :4], ref[:new // 2, :4]) and torch.isfinite(lse[:new, :4]).all()
    assert torch.equal(out[:new, 4:], ref[:new, 4:])


@pytest.mark.parametrize("new", [1, 5, 200])
@HINTS
def test_strided_queries_and_outputs(new, hint):
    c = Case([300, 20], [new, 2], 2, 128, 32)
    q = _queries(c.T, 8, 128, BF16)
    ref, _ = _run(c, q, hint)
    fused = torch.full((c.T, 8 * 128 + 4 * 128 + 8), float("nan"), dtype=BF16, device="cuda")
    qs = fused[:, :1024].view(c.T, 8, 128)
    qs.copy_(q)
    buf = torch.full((8, c.T + 1, 136), 3.0, dtype=BF16, device="cuda")   # head-major, padded
    out = buf[:, :c.T, :128].transpose(0, 1)
    got, _ = _run(c, qs, hint, out=out)
    assert got is out and torch.equal(out, ref)
    buf[:, :c.T, :128] = 3.0
    assert (buf == 3.0).all()


def test_results_do_not_depend_on_the_hint_or_the_neighbours():
    lens = [1000, 3, 517, 64]
    c = Case(lens, [1] * 4, 2, 128, 16, extra=3)
    q = _queries(4, 8, 128, F16)
    ref, rl = _run(c, q)
    _check_attention(c, q, ref, rl)
    for hint in (1, 64, 100000):
        out, lse = _run(c, q, max_kv=hint)
        _check_attention(c, q, out, lse, what=f"hint {hint}")
    again, _ = _run(c, q)
    assert torch.equal(again, ref)


def test_bad_pages_lengths_and_row_counts_are_recorded():
    c = Case([40, 40], [1, 1], 1, 64, 16)
    q = _queries(2, 2, 64, F16)
    ref, _ = _run(c, q)
    for bad in (-1, 10 ** 6):
        t = c.t_table.clone()
        t[1, 1] = bad
        out = api.kv4_attention(q, c.cache, t, c.t_len, c.t_cu, max_q=1)
        assert api.device_error() == api.BCQ_ERR_PAGE
        assert torch.equal(out[0], ref[0]) and torch.isfinite(out[1]).all()
        k = torch.ones(2, 1, 64, dtype=F16, device="cuda")
        t[1, 1], t[1, 2] = c.t_table[1, 1], bad
        before = c.cache.k.clone()
        api.kv4_append(c.cache, k[:0], k[:0], t, c.t_len, torch.zeros_like(c.t_cu))
        assert api.device_error() == api.BCQ_OK and torch.equal(before, c.cache.k)
        api.kv4_append(c.cache, k[1:], k[1:], t, c.t_len, _i32([0, 0, 1]))
        assert api.device_error() == api.BCQ_ERR_PAGE and torch.equal(before, c.cache.k)
        rk, _ = api.kv4_read(c.cache, t, c.t_len, _i32([0, 0, 1]), tokens=1)
        assert api.device_error() == api.BCQ_ERR_PAGE and (rk == 0).all()
    long = _i32([40, 10 ** 6])
    out = api.kv4_attention(q, c.cache, c.t_table, long, c.t_cu, max_q=1)
    assert api.device_error() == api.BCQ_ERR_PAGE and torch.equal(out[0], ref[0])
    out = api.kv4_attention(q, c.cache, c.t_table, _i32([40, -7]), c.t_cu, max_q=1)
    assert api.device_error() == api.BCQ_ERR_PAGE
    assert torch.equal(out[0], ref[0]) and (out[1] == 0).all()
    out = torch.full_like(q, 5.0)
    api.kv4_attention(q, c.cache, c.t_table, c.t_len, _i32([0, 2, 2]), max_q=1, out=out)
    assert api.device_error() == api.BCQ_ERR_SHAPE and (out[1] == 5).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_missing_page_under_many_rows(D):
    """Its positions are left out, for every row, and it is recorded."""
    c = Case([200], [150], 1, D, 16)
    q = _queries(150, 4, D, F16)
    t = c.t_table.clone()
    t[0, 3] = -5                           # positions 48..63
    out, lse = api.kv4_attention(q, c.cache, t, c.t_len, c.t_cu, max_q=150, max_kv=4000, return_lse=True)
    assert api.device_error() == api.BCQ_ERR_PAGE
    ro, rl, mag = kv4.attention(_f64(q), *(c.arrays[n] for n in ("k", "k_param", "v", "v_param")), c.table, c.lens,
                                c.cu, float(np.float32(D ** -0.5)), hidden=range(48, 64))
    ds, tol = _tolerances(mag["s"], mag["v"], ro, 200, D, F16)
    assert (np.abs(_f64(out) - ro) <= tol).all() and (np.abs(_f64(lse) - rl) <= ds + 1e-4).all()
    few, _ = api.kv4_attention(q, c.cache, t, c.t_len, c.t_cu, max_q=150, max_kv=200, return_lse=True)
    assert api.device_error() == api.BCQ_ERR_PAGE
    assert (np.abs(_f64(few) - ro) <= tol).all()


def test_no_rows():
    c = Case([40], [1], 1, 64, 16)
    q = torch.empty(0, 2, 64, dtype=F16, device="cuda")
    zero = _i32([0, 0])
    assert api.kv4_attention(q, c.cache, c.t_table, c.t_len, zero).shape == (0, 2, 64)
    k, v = api.kv4_read(c.cache, c.t_table, c.t_len, zero, tokens=0)
    assert k.shape == (0, 1, 64)
    api.kv4_append(c.cache, k, v, c.t_table, c.t_len, zero)


@pytest.mark.parametrize("new", [1, 130])
def test_a_long_cache(new):
    """Offsets beyond 2^31 bytes: the sequence's pages are the last of a large cache."""
    pages, heads, page_size, D = 18000, 8, 256, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 8 << 30:
        pytest.skip("needs 8 GB")
    small = Case([700], [new], heads, D, page_size, seed=3)
    cache = api.Kv4Cache.empty(pages, heads, page_size, D)
    assert cache.k.numel() > 2 ** 31
    W = small.table.shape[1]
    far = torch.arange(pages - W, pages, dtype=torch.int32, device="cuda").flip(0)
    src = torch.from_numpy(small.table[0].astype(np.int64)).cuda()
    for n in ("k", "k_param", "v", "v_param"):
        getattr(cache, n)[far.long()] = getattr(small.cache, n)[src]
    q = _queries(new, 16, D, F16)
    ref, rl = _run(small, q)
    out, lse = api.kv4_attention(q, cache, far.view(1, W), small.t_len, small.t_cu, max_q=new, max_kv=700,
                                 return_lse=True)
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    k, v = api.kv4_read(cache, far.view(1, W), small.t_len, small.t_cu, tokens=new)
    api.kv4_append(cache, k, v, far.view(1, W), small.t_len, small.t_cu)
    k2, _ = api.kv4_read(small.cache, small.t_table, small.t_len, small.t_cu, tokens=new)
    assert torch.equal(k, k2)


@pytest.mark.parametrize("B,n,H,heads", [(1, 20000, 8, 1), (1, 5000, 32, 8), (40, 600, 8, 4), (300, 90, 4, 2)])
def test_long_and_many(B, n, H, heads):
    """Split sequences and full grids: some of the rows in fp64."""
    D, page_size = 128, 64
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(n // 2, n + 1, B)]
    c = Case(lens, [1] * B, heads, D, page_size, seed=B)
    q = _queries(B, H, D, F16)
    out, lse = _run(c, q)
    pick = sorted(set(int(x) for x in rng.integers(0, B, 6)))
    for b in pick:
        at = [(kv4.gather(c.arrays[p], c.table[b], lens[b]),
               kv4.gather(c.arrays[p + "_param"], c.table[b], lens[b])) for p in "kv"]
        K, V = (kv4.values(*x) for x in at)
        Km, Vm = (kv4.magnitudes(*x) for x in at)
        g = np.arange(H) // (H // heads)
        scale = float(np.float32(D ** -0.5))
        s = np.einsum("hd,nhd->hn", _f64(q[b]), K[:, g]) * scale
        S = (np.einsum("hd,nhd->hn", np.abs(_f64(q[b])), Km[:, g]) * scale).max(1)
        p = np.exp(s - s.max(1, keepdims=True))
        total = p.sum(1)
        ref = np.einsum("hn,nhd->hd", p / total[:, None], V[:, g])
        A = np.einsum("hn,nhd->hd", p / total[:, None], Vm[:, g])
        ds, tol = _tolerances(S, A, ref, lens[b], D, F16)
        assert (np.abs(_f64(lse[b]) - s.max(1) - np.log(total)) <= ds + 4 * lens[b] * E + 64 * E).all()
        assert (np.abs(_f64(out[b]) - ref) <= tol).all()


# ------------------------------------------------------------------ together

def test_a_decode_layer_as_it_is_used():
    """Projection in 8 bits, rows into the cache, attention, projection: prompt, then tokens."""
    torch.manual_seed(0)
    E, H, heads, D, page_size = 512, 4, 2, 128, 16
    wq, sq = api.quantize_i8((torch.randn((H + 2 * heads) * D, E) * E ** -0.5).half().cuda())
    wo, so = api.quantize_i8((torch.randn(E, H * D) * (H * D) ** -0.5).half().cuda())
    cache = api.Kv4Cache.empty(24, heads, page_size, D)
    table = torch.randperm(24, dtype=torch.int32).cuda()[:16].view(2, 8)
    lens = np.array([0, 0])
    seen = [[], []]
    for new in ([37, 20], [1, 1], [1, 1], [5, 3]):
        cu = np.concatenate([[0], np.cumsum(new)])
        T = int(cu[-1])
        lens = lens + np.array(new)
        x = torch.randn(T, E).half().cuda()
        qkv = api.linear_i8(x, wq, sq)
        q = qkv[:, :H * D].view(T, H, D)
        k = qkv[:, H * D:(H + heads) * D].view(T, heads, D)
        v = qkv[:, (H + heads) * D:].view(T, heads, D)
        t_len, t_cu = _i32(lens.tolist()), _i32(cu.tolist())
        api.kv4_append(cache, k, v, table, t_len, t_cu)
        o = api.kv4_attention(q, cache, table, t_len, t_cu, max_q=max(new))
        y = api.linear_i8(o.view(T, H * D), wo, so)
        assert torch.isfinite(y).all() and y.shape == (T, E)
        for b in range(2):
            held = [(kv4.pack(code), param) for code, param in (
                kv4.quantize(_f64(x[cu[b]:cu[b + 1]])) for x in (k, v))]
            seen[b].append([f(*h) for h in held for f in (kv4.values, kv4.magnitudes)])
            Kb, Km, Vb, Vm = (np.concatenate([s[i] for s in seen[b]]) for i in range(4))
            for i in range(new[b]):
                n = int(lens[b]) - new[b] + i + 1
                for h in range(H):
                    row = _f64(q[cu[b] + i, h])
                    s = Kb[:n, h // 2] @ row * D ** -0.5
                    S = (Km[:n, h // 2] @ np.abs(row) * D ** -0.5).max()
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    ref = p @ Vb[:n, h // 2]
                    _, tol = _tolerances(S, p @ Vm[:n, h // 2], ref, n, D, F16)
                    assert (np.abs(_f64(o[cu[b] + i, h]) - ref) <= tol).all()


def test_captured_and_replayed_with_other_lengths():
    """One graph, replayed as the sequences grow; two graphs of the same stream replayed at once."""
    lens = [30, 5]
    c = Case([64, 64], [1, 1], 2, 128, 16)
    q = _queries(2, 8, 128, F16)
    kv_len = _i32(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.kv4_attention(q, c.cache, c.t_table, kv_len, max_kv=64)
    side.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = api.kv4_attention(q, c.cache, c.t_table, kv_len, max_kv=64)
        graphs.append((g, out))
    for lens in ([30, 5], [33, 48], [64, 1], [0, 64]):
        kv_len.copy_(_i32(lens))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        c.lens = lens
        for _, out in graphs:
            _check_attention(c, q, out, None, what=str(lens))


def test_fast_calls_are_the_same_calls():
    """With the current stream named the binding takes its long way: the same bits."""
    st = torch.cuda.current_stream()
    c, k, v = _append_case([40, 70], [5, 70], 2, 128, 16, BF16)
    api.kv4_append(c.cache, k, v, c.t_table, c.t_len, c.t_cu)
    d = Case([40, 70], [5, 70], 2, 128, 16)
    api.kv4_append(d.cache, k, v, d.t_table, d.t_len, d.t_cu, stream=st)
    for n in ("k", "k_param", "v", "v_param"):
        a, b = getattr(c.cache, n), getattr(d.cache, n)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for dtype in (F16, BF16, F32):
        x = api.kv4_read(c.cache, c.t_table, c.t_len, c.t_cu, tokens=75, dtype=dtype)
        y = api.kv4_read(c.cache, c.t_table, c.t_len, c.t_cu, tokens=75, dtype=dtype, stream=st)
        assert x[0].dtype == dtype and all(torch.equal(a, b) for a, b in zip(x, y))
    row = torch.randn(75, 1024 + 8, device="cuda").half()
    q = row[:, :1024].view(75, 8, 128)
    for kw in (dict(), dict(max_q=70, max_kv=70), dict(window=5, scale=0.3, return_lse=True), dict(causal=False),
               dict(scale=1, return_lse=True, max_q=70)):
        x = api.kv4_attention(q, c.cache, c.t_table, c.t_len, c.t_cu, **kw)
        y = api.kv4_attention(q, c.cache, c.t_table, c.t_len, c.t_cu, stream=st, **kw)
        x, y = (z if isinstance(z, tuple) else (z,) for z in (x, y))
        assert len(x) == len(y) == 1 + bool(kw.get("return_lse"))
        assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_side_stream():
    c = Case([500, 30], [1, 1], 2, 128, 16)
    q = _queries(2, 8, 128, F16)
    ref, _ = _run(c, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = _run(c, q, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)


def _steps(c, queries, rows, w, w_scale, out):
    """Tokens one after the other with nothing between the calls; each call's inputs are written just before it
    and written over just after it."""
    q, k, n, x = queries[0].clone(), rows[0].clone(), torch.zeros_like(c.t_len), None
    for i, (qi, ki) in enumerate(zip(queries, rows)):
        q.copy_(qi), k.copy_(ki)
        n.fill_(i + 1)
        api.kv4_append(c.cache, k, k, c.t_table, n)
        k.zero_()
        out[i].copy_(api.kv4_attention(q, c.cache, c.t_table, n, max_kv=600).flatten(1))
        a = api.kv4_attention(q, c.cache, c.t_table, n, max_kv=600)
        n.zero_(), q.zero_()
        x = api.linear_i8(a.flatten(1), w, w_scale)
        a.zero_()
        codes, scale = api.quantize_i8(x)
        x.zero_()
        x = api.gemm_i8(codes, scale, w, w_scale, dtype=F32)
        out[i] += x.abs().clamp(max=1.0) * 2.0 ** -6


@pytest.mark.parametrize("captured", [False, True])
def test_calls_wait_for_what_came_before(captured):
    """Kernels that are set up early read nothing early: in a row, in a graph, behind a fork and a join and a memset."""
    g = torch.Generator().manual_seed(3)
    S, B, H, D = 40, 3, 4, 128
    c = Case([S] * B, [1] * B, H, D, 16)
    queries, rows = (torch.randn(S, B, H, D, generator=g).half().cuda() for _ in range(2))
    w, w_scale = api.quantize_i8(torch.randn(H * D, H * D, generator=g).half().cuda())
    want, got = (torch.zeros(S, B, H * D, device="cuda", dtype=F16) for _ in range(2))
    k, k_param = c.cache.k.clone(), c.cache.k_param.clone()
    for i in range(S):                      # each call alone
        n = torch.full((B,), i + 1, dtype=torch.int32, device="cuda")
        api.kv4_append(c.cache, rows[i], rows[i], c.t_table, n)
        torch.cuda.synchronize()
        a = api.kv4_attention(queries[i], c.cache, c.t_table, n, max_kv=600).flatten(1)
        torch.cuda.synchronize()
        x = api.linear_i8(a, w, w_scale)
        torch.cuda.synchronize()
        codes, scale = api.quantize_i8(x)
        torch.cuda.synchronize()
        want[i] = a + api.gemm_i8(codes, scale, w, w_scale, dtype=F32).abs().clamp(max=1.0) * 2.0 ** -6
    if not captured:
        for _ in range(3):
            c.cache.k.copy_(k), c.cache.k_param.copy_(k_param)
            _steps(c, queries, rows, w, w_scale, got)
            assert torch.equal(got, want)
        return
    side = torch.cuda.Stream()
    other = torch.zeros(1 << 20, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            other.add_(1)
            c.cache.k_param.copy_(k_param)
        c.cache.k.copy_(k)
        here.wait_stream(side)
        _steps(c, queries, rows, w, w_scale, got)
        side.wait_stream(here)
        with torch.cuda.stream(side):      # a call whose stream joins, and one behind a memset
            out = api.kv4_attention(queries[0], c.cache, c.t_table, c.t_len, max_kv=600)
        here.wait_stream(side)
        last = api.kv4_attention(queries[0], c.cache, c.t_table, c.t_len, max_kv=600)
    for _ in range(3):
        got.zero_(), c.cache.k.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert torch.equal(out, last) and not torch.isnan(out).any()


@pytest.mark.parametrize("B,n,L,H,heads,D", [(1, 1024, 2048, 16, 16, 64), (2, 300, 1500, 16, 4, 128),
                                             (3, 64, 900, 16, 2, 64), (2, 70, 1200, 16, 4, 256)])
def test_many_calls_in_a_row(B, n, L, H, heads, D):
    """No wait of any call runs out, and every call gives the same bits."""
    c = Case([L] * B, [n] * B, heads, D, 64)
    q = _queries(c.T, H, D, F16)
    ref, ref_lse = _run(c, q, 4000)
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(400):
        out, lse = _run(c, q, 4000)
        bad += (out != ref).sum() + (lse != ref_lse).sum()
    assert int(bad) == 0 and api.device_error() == api.BCQ_OK


@pytest.fixture(params=[(511, 0), (4000, 0)], ids=["short", "long"])
def as_if_large(request, monkeypatch):
    """Every call as if it might have thousands of rows: the kernel of many rows, with keys in two parts and in one."""
    run, attention = _run, api.kv4_attention
    args = dict(max_q=5000, max_kv=request.param[0])
    monkeypatch.setitem(globals(), "_run", lambda c, q, hint=None, **kw: run(c, q, **{**kw, **args}))
    monkeypatch.setattr(api, "kv4_attention", lambda *a, **kw: attention(*a, **{**kw, **args}))


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 64), (True, 600), (False, 0), (False, 9)])
@pytest.mark.parametrize("lens,new", [([33, 100], [1, 1]), ([200], [140]), ([700, 90, 0], [150, 90, 3])])
@pytest.mark.parametrize("D,H", [(64, 6), (128, 8), (256, 8)])
def test_large_masks(as_if_large, lens, new, causal, window, D, H):
    c = Case(lens, new, 2, D, 16, seed=window)
    q = _queries(c.T, H, D, BF16 if window == 64 else F16, seed=2)
    out, lse = _run(c, q, causal=causal, window=window)
    _check_attention(c, q, out, lse, causal=causal, window=window)


@pytest.mark.parametrize("lens,new,H,heads,D,page_size", [
    ([5], [5], 2, 1, 64, 16), ([1], [1], 1, 1, 128, 16), ([300], [150], 12, 3, 128, 48), ([520], [400], 7, 1, 256, 48),
    ([129, 5], [129, 5], 32, 2, 128, 16), ([70, 0, 71], [5, 0, 70], 6, 1, 256, 64), ([256], [256], 2, 2, 128, 128)])
def test_large_rows(as_if_large, lens, new, H, heads, D, page_size):
    test_several_rows(lens, new, H, heads, D, page_size, F16, None)


@pytest.mark.parametrize("new", [1, 6, 140])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_nan(as_if_large, new, D):
    test_nan_stays_where_it_belongs(new, D, None)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_strides_scales_and_missing_pages(as_if_large, D):
    test_strided_queries_and_outputs(200, None)
    test_rows_that_see_nothing(0, 300, 2, None)
    for scale in (0.0, -0.3, 4.0):
        test_scales_of_the_scores(scale, 160, None)
    for dtype, mag in ((F16, 1e-4), (F16, 3e4), (BF16, 1e-12), (BF16, 1e30)):
        test_queries_of_any_magnitude(dtype, mag, 150, None)
    test_a_missing_page_under_many_rows(D)


@pytest.mark.parametrize("B,n,L,H,heads,D", [(8, 100, 400, 16, 4, 64), (4, 150, 300, 16, 4, 128), (4, 100, 400, 8, 2, 256)])
def test_many_short_calls_in_a_row(B, n, L, H, heads, D):
    c = Case([L] * B, [n] * B, heads, D, 64)
    q = _queries(c.T, H, D, F16)
    kw = dict(max_q=5000)
    ref, ref_lse = _run(c, q, 500, **kw)
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(400):
        out, lse = _run(c, q, 500, **kw)
        bad += (out != ref).sum() + (lse != ref_lse).sum()
    assert int(bad) == 0 and api.device_error() == api.BCQ_OK


@pytest.mark.parametrize("B,n,L,H,heads,D", [(40, 64, 700, 16, 4, 128), (60, 40, 600, 12, 2, 64), (50, 32, 500, 8, 2, 256)])
@pytest.mark.parametrize("hint", [500, 4000])
def test_nan_values_in_every_step_of_a_full_grid(B, n, L, H, heads, D, hint):
    """V's groups that are no numbers reach the rows that see them and no others, however late V's codes
    come: a few at every 64 positions, more blocks of rows than SMs, the cache flushed from L2."""
    c = Case([L] * B, [n] * B, heads, D, 16, seed=D)
    rng = np.random.default_rng(D)
    G = D // 64
    param = c.arrays["v_param"].copy()
    odd = np.zeros((B, L, heads, G), dtype=bool)
    for b in range(B):
        for j0 in range(0, L, 64):
            for _ in range(2):
                j, h, g = rng.integers(j0, min(j0 + 64, L)), rng.integers(heads), rng.integers(G)
                if rng.integers(4):              # most of them where only some rows see them
                    j = max(j, L - n + rng.integers(n))
                odd[b, j, h, g] = True
                param[c.table[b, j // 16], h, j % 16, g, rng.integers(2)] = np.nan
    first = np.where(odd.any(1), odd.argmax(1), L)                            # [B][heads][G]
    pos = np.arange(L - n, L)
    want = pos[None, :, None, None] >= first[:, None]                          # [B][n][heads][G]
    want = np.repeat(np.repeat(want, H // heads, 2).reshape(B * n, H, G), 64, 2)
    assert want.any() and not want.all()
    want = torch.from_numpy(want).cuda()
    q = _queries(c.T, H, D, F16)
    kw = dict(max_q=5000)                                                       # the kernel of many rows
    clean, clean_lse = _run(c, q, hint, **kw)
    c.cache.v_param.copy_(torch.from_numpy(param))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(60):
        flush.fill_(i)
        out, lse = _run(c, q, hint, **kw)
        wrong += (torch.isnan(out) != want).sum() + (out != clean)[~want].sum() + (lse != clean_lse).sum()
    assert int(wrong) == 0 and api.device_error() == api.BCQ_OK


def _values_of_any_size(mag, peak, n, new, H, heads, D, seed=0):
    """A cache whose first position outweighs each other one e^peak times, for queries of ones and scale 1 / D,
    and whose V has scales about `mag` ("grows": from 1e-4 to 1 with the position)."""
    c = Case([n, 40], [new, 1], heads, D, 64, seed=seed)
    rng = np.random.default_rng(seed)
    shape = c.arrays["v_param"].shape[:-1]
    a = np.full(shape, 1e-4 if mag == "grows" else mag)
    if mag == "grows":
        at = np.arange(n)
        a.transpose(0, 2, 1, 3)[c.table[0][at // 64], at % 64] = (1e-4 * 1e4 ** (at / n))[:, None, None]
    a = (a * (1 + 0.01 * rng.integers(0, 2, shape))).astype(np.float16)
    v = np.stack([a, (-7.5 * a.astype(np.float64)).astype(np.float16)], -1)
    v[np.isnan(c.arrays["v_param"][..., 0])] = np.nan                          # where no token is
    k = np.zeros_like(c.arrays["k_param"])
    for b in range(2):
        k[c.table[b, 0], :, 0, :, 1] = peak
    c.arrays.update(k_param=k, v_param=v)
    c.cache.k_param.copy_(torch.from_numpy(k))
    c.cache.v_param.copy_(torch.from_numpy(v))
    return c


@pytest.mark.parametrize("dtype,new,H,heads,D", [(F16, 1, 4, 1, 128), (BF16, 1, 2, 2, 64), (F16, 3, 2, 1, 256),
                                                 (BF16, 3, 8, 2, 128), (F16, 1, 16, 1, 64)])
@pytest.mark.parametrize("peak", [0.0, 9.0])
@pytest.mark.parametrize("mag", [2000.0, 0.3, 6e-3, 3e-4, 3e-5, "grows"])
def test_values_of_any_magnitude(mag, peak, dtype, new, H, heads, D):
    """Few rows, positions in one part: each weight p and each p a is off by u of itself, whatever V's magnitude and
    however one position outweighs the rest.  The kernel's scores are products of exact operands summed in fp32 (the
    offsets' in two fp16 parts, 2^-22); p a c is rounded twice and p z once; and what lies 2^23 below the row's
    largest, or 2^13 below V's largest scale, adds a step of 2^-33 of the largest a position."""
    n = 8000
    c = _values_of_any_size(mag, peak, n, new, H, heads, D)
    q = torch.ones(c.T, H, D, dtype=dtype, device="cuda")
    out, lse = _run(c, q, max_kv=128, scale=1.0 / D)
    ro, rl, m = kv4.attention(_f64(q), *(c.arrays[x] for x in ("k", "k_param", "v", "v_param")), c.table, c.lens, c.cu,
                              1.0 / D)
    ds = m["s"] * (2.0 ** -22 + 4 * D * E) + 16 * E * (1 + m["s"])
    largest = np.nanmax(np.abs(c.arrays["v_param"].astype(np.float64)).sum(-1)) * 15
    tol = (m["v"] * (2 * ds + 2 * U + 4 * n * E)[..., None] + n * 2.0 ** -33 * largest +
           torch.finfo(dtype).eps / 2 * np.abs(ro) + 2.0 ** -25)
    err = np.abs(_f64(out) - ro)
    assert (err <= tol).all(), f"worst {(err / tol).max():.2f} of the tolerance, {err.max():.2e}"
    assert (np.abs(_f64(lse) - rl) <= ds + 4 * n * E + 2 * E * np.abs(rl)).all()


@pytest.mark.parametrize("new", [1, 6, 140])
@HINTS
def test_what_no_row_sees_has_no_effect(new, hint):
    """Finite numbers of any size behind a sequence's end, in front of its window and beside a hole change no bit."""
    c = Case([175, 50], [new, 1], 2, 128, 16)
    q = _queries(c.T, 8, 128, F16)
    c.cache.v_param.mul_(1e-3)
    for kw in (dict(), dict(window=21)):
        ref, ref_lse = _run(c, q, hint, **kw)
        keep = [getattr(c.cache, x).clone() for x in ("k_param", "v_param")]
        for b in range(2):
            first = max(0, c.lens[b] - c.new[b] - 20) if kw else 0
            for j in [*range(first), *range(c.lens[b], 16 * c.table.shape[1])]:
                for x in (c.cache.k_param, c.cache.v_param):
                    x[int(c.table[b, j // 16]), :, j % 16] = 6e4 * (-1) ** j
        out, lse = _run(c, q, hint, **kw)
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
        for x, y in zip((c.cache.k_param, c.cache.v_param), keep):
            x.copy_(y)


@pytest.mark.parametrize("kw,adds", [(dict(max_q=5000, max_kv=4000), 32), (dict(max_kv=128), 64), (dict(), 64)],
                         ids=["many", "few", "few, split"])
@pytest.mark.parametrize("peak", [12.5, 13.25, 13.5])
@pytest.mark.parametrize("D", [64, 256])
def test_a_long_tail_of_small_weights_counts(D, peak, kw, adds):
    """One position and, e^peak times lighter each, 2^18 others that weigh half as much together or more; V is 1.
    Weights are off by u, and fp32 sums of n positions, 16 at a time in two parts or by four warps, by 2 E each."""
    n = 2 ** 18
    c = Case([n], [1], 1, D, 256)
    c.cache.k_param.zero_()
    c.cache.v_param.zero_()
    c.cache.v_param[..., 1] = 1.0
    c.cache.k_param[int(c.table[0, 0]), :, 0, :, 1] = peak
    tol = U + 2 * E * (n / adds + 64)
    for dtype in (BF16, F16):
        q = torch.ones(1, 1, D, dtype=dtype, device="cuda")
        out, lse = _run(c, q, scale=1.0 / D, **kw)
        err = np.abs(_f64(out) - 1).max()
        assert err <= tol + torch.finfo(dtype).eps / 2, err
        want = peak + np.log1p((n - 1) * np.exp(-peak))
        assert abs(float(lse) - want) <= 2 * E * (n / adds + 64) + 64 * E * want


@pytest.mark.parametrize("B,n,L,H,heads,D", [(4, 300, 900, 16, 4, 128), (1, 200, 6000, 8, 2, 128), (40, 60, 300, 2, 2, 128)])
@pytest.mark.parametrize("hint", [500, 4000])
def test_waits_that_run_out_are_reported(B, n, L, H, heads, D, hint):
    """Whichever wait of the kernel of many rows gives up first, the call ends and says so."""
    c = Case([L] * B, [n] * B, heads, D, 64)
    q = _queries(c.T, H, D, F16)
    kw = dict(max_q=5000)
    ref, ref_lse = _run(c, q, hint, **kw)
    try:
        given_up = 0
        for _ in range(30):
            api.debug_impatient(True)
            out, lse = _run(c, q, hint, **kw)
            status = api.device_error()
            assert status == api.BCQ_ERR_TIMEOUT or (status == api.BCQ_OK and torch.equal(out, ref) and torch.equal(lse, ref_lse))
            given_up += status == api.BCQ_ERR_TIMEOUT
            api.debug_impatient(False)
            out, lse = _run(c, q, hint, **kw)
            assert api.device_error() == api.BCQ_OK and torch.equal(out, ref) and torch.equal(lse, ref_lse)
        assert given_up
    finally:
        api.debug_impatient(False)


@pytest.mark.parametrize("D,H,heads", [(64, 4, 1), (128, 8, 2), (256, 4, 2)])
@pytest.mark.parametrize("lens,new", [([700], [700]), ([1500, 40, 300], [200, 40, 150])])
@pytest.mark.parametrize("kw", [dict(), dict(window=400), dict(causal=False)])
def test_rows_that_see_few_positions_have_exact_scores(D, H, heads, lens, new, kw):
    """The kernel of many rows, whatever the call's other rows and its hint are: keys in two fp16 parts, 2^-22."""
    c = Case(lens, new, heads, D, 16, seed=D)
    q = _queries(c.T, H, D, F16, seed=4)
    _, lse = _run(c, q, max_q=5000, max_kv=4000, **kw)
    _, rl, m = kv4.attention(_f64(q), *(c.arrays[x] for x in ("k", "k_param", "v", "v_param")), c.table, c.lens, c.cu,
                             float(np.float32(D ** -0.5)), kw.get("causal", True), kw.get("window", 0))
    ds = m["s"] * (2.0 ** -22 + 4 * D * E) + 16 * E * (1 + m["s"])
    few = np.concatenate([[kv4.visible(n, r, i, **kw).sum() < 512 for i in range(r)] for n, r in zip(lens, new)])
    err = np.abs(_f64(lse) - rl)
    assert (err <= ds + 4 * 512 * E + 2 * E * np.abs(rl))[few].all(), f"{err[few].max():.1e} of {ds[few].max():.1e}"


@pytest.mark.parametrize("new,max_q", [(1, 1), (6, 6), (140, 140), (1, 5000), (140, 5000)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages_in_front_of_every_window_may_be_gone(new, max_q, D):
    """A table whose entries before the first row's window are no pages: nothing to record, and the same bits."""
    lens = [75 + new, 190 + new, 17 + new, 49 + new]
    c = Case(lens, [new] * 4, 2, D, 16)
    q = _queries(c.T, 8, D, F16)
    for window in (1, 16, 20, 33):
        ref, ref_lse = _run(c, q, 4000, max_q=max_q, window=window)
        assert api.device_error() == api.BCQ_OK
        t = c.t_table.clone()
        for b, n in enumerate(lens):
            t[b, :max(0, n - new - window + 1) // 16] = -1
        out, lse = api.kv4_attention(q, c.cache, t, c.t_len, c.t_cu, max_q=max_q, max_kv=4000, window=window,
                                     return_lse=True)
        assert api.device_error() == api.BCQ_OK, window
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse), window


@pytest.mark.parametrize("new,max_q", [(1, 1), (40, 40), (40, 5000)])
@pytest.mark.parametrize("scale", [0.1, -0.1, 0.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_with_an_infinity_are_nan(new, max_q, scale, D):
    """Also where every score is -infinity: that is no row which sees nothing."""
    c = Case([new], [new], 1, D, 16)
    c.cache.k_param[..., 0], c.cache.k_param[..., 1] = 0, 1      # K is 1
    c.cache.v_param.nan_to_num_()
    q = _queries(new, 4, D, F16)
    ref, ref_lse = _run(c, q, 4000, max_q=max_q, scale=scale)
    q[0, 1, 3], q[0, 2, 5], q[-1, 3, D - 1] = float("-inf"), float("inf"), float("-inf")
    out, lse = _run(c, q, 4000, max_q=max_q, scale=scale)
    odd = torch.zeros(new, 4, dtype=torch.bool)
    odd[0, 1] = odd[0, 2] = odd[-1, 3] = True
    assert torch.isnan(out[odd]).all() and torch.isnan(lse[odd]).all()
    assert torch.equal(out[~odd], ref[~odd]) and torch.equal(lse[~odd], ref_lse[~odd])


@pytest.mark.parametrize("heads,D", [(1, 64), (2, 128), (2, 256), (8, 128), (32, 128), (32, 256)])
def test_rows_in_and_out_whatever_shares_a_block(heads, D):
    """Each number of rows on both sides of where the kernels change: the same codes and values as 100 rows a call."""
    most = 10300 if heads * D <= 256 else 4100 if heads * D <= 1024 else 1190
    c, k, v = _append_case([most], [most], heads, D, 64, F16)
    for i in range(0, most, 100):
        r = slice(i, min(i + 100, most))
        api.kv4_append(c.cache, k[r], v[r], c.t_table, _i32([r.stop]), _i32([0, r.stop - i]))
    parts = ("k", "k_param", "v", "v_param")
    want = {n: getattr(c.cache, n).clone() for n in parts}
    ok, ov = (torch.cat(x) for x in zip(*(api.kv4_read(c.cache, c.t_table, _i32([min(i + 100, most)]),
                                                      _i32([0, min(100, most - i)]), tokens=min(100, most - i))
                                          for i in range(0, most, 100))))
    for T in (444, 445, 592, 593, 1184, 1185, 4095, 4096, 10239, 10240, 10300):
        if T > most:
            continue
        for n in parts:
            getattr(c.cache, n).zero_()
        api.kv4_append(c.cache, k[:T], v[:T], c.t_table, _i32([T]), _i32([0, T]))
        for i in range(T, most, 100):                            # the rest, as before
            r = slice(i, min(i + 100, most))
            api.kv4_append(c.cache, k[r], v[r], c.t_table, _i32([r.stop]), _i32([0, r.stop - i]))
        at = torch.arange(most, device="cuda")
        page, pos = c.t_table[0].long()[at // 64], at % 64
        for n in parts:
            a, b = (x.view(torch.uint8)[page, :, pos] for x in (getattr(c.cache, n), want[n]))
            assert torch.equal(a, b), (T, n)
        rk, rv = api.kv4_read(c.cache, c.t_table, _i32([T]), _i32([0, T]), tokens=T)
        assert torch.equal(rk, ok[:T]) and torch.equal(rv, ov[:T]), T


def test_both_ways_refuse_the_same_calls():
    """The fast calls' own checks let nothing through that the binding's longer way refuses."""
    h, f32, i8 = torch.float16, torch.float32, torch.int8
    Z = lambda *n, dtype=h: torch.zeros(*n, dtype=dtype, device="cuda")          # noqa: E731
    c = Case([40, 70], [2, 3], 2, 128, 16)
    cache, tab, n, cu = c.cache, c.t_table, c.t_len, c.t_cu
    q, k = Z(5, 8, 128), Z(5, 2, 128)
    x8, s8, w8, t8 = Z(4, 64, dtype=i8), Z(4, dtype=f32), Z(6, 64, dtype=i8), Z(6, dtype=f32)
    wide = Z(9, 1100)

    def att(q=q, t=tab, n=n, cu=cu, **kw):
        return lambda **s: api.kv4_attention(q, cache, t, n, cu, **kw, **s)

    def app(k=k, v=k, t=tab, n=n, cu=cu):
        return lambda **s: api.kv4_append(cache, k, v, t, n, cu, **s)

    def read(t=tab, n=n, cu=cu, **kw):
        return lambda **s: api.kv4_read(cache, t, n, cu, **kw, **s)

    def gemm(x=x8, s=s8, w=w8, t=t8, **kw):
        return lambda **st: api.gemm_i8(x, s, w, t, **kw, **st)

    def lin(x=Z(4, 64), w=w8, t=t8, **kw):
        return lambda **st: api.linear_i8(x, w, t, **kw, **st)

    bad = [
        att(q=q.float()), att(q=q[:, :, :64]), att(q=q[0]), att(q=Z(5, 7, 128)), att(q=Z(5, 0, 128)), att(q=Z(4, 8, 130)[:, :, 1:129]),
        att(q=wide[:5, 3:1027].view(5, 8, 128)), att(q=Z(128, 8, 5).permute(2, 1, 0)), att(q=Z(5, 512, 128)), att(cu=None),
        att(t=tab.long()), att(t=tab[0]), att(t=tab.t()), att(t=tab[:, :0]), att(n=n.long()), att(n=n[:1]), att(n=n[None]),
        att(cu=cu[:2]), att(cu=cu.long()), att(max_q=0), att(max_kv=0), att(max_q=-1), att(window=-1), att(max_q=2 ** 31),
        att(max_kv=2 ** 32 + 1), att(window=2 ** 33), att(scale=float("nan")), att(scale=float("inf")), att(scale=1e300),
        att(max_q=1.5), att(t=tab.cpu()), att(cu=cu.cpu()),
        app(k=k.float()), app(v=k.bfloat16()), app(v=k[:4]), app(k=Z(5, 3, 128)), app(k=k[..., :64], v=k[..., :64]), app(cu=None),
        app(k=Z(5, 2, 129)[..., :128]), app(t=tab.long()), app(n=n[:1]),
        read(tokens=5, dtype=torch.int8), read(), read(tokens=-1), read(cu=None, tokens=5), read(tokens=5, t=tab[0]),
        gemm(x=x8[:, :60]), gemm(x=x8.half()), gemm(w=w8[:, :48]), gemm(s=s8[:3]), gemm(s=s8.half()), gemm(t=t8[None]),
        gemm(x=Z(4, 72, dtype=i8)[:, 8:]), gemm(x=Z(4, 72, dtype=i8)[:, :64]), gemm(x=x8[:1].expand(4, 64)), gemm(dtype=torch.int8),
        gemm(out=Z(4, 5)), gemm(out=Z(4, 6, dtype=f32)), gemm(out=Z(6, 4).t()), gemm(out=Z(1, 6).expand(4, 6)),
        lin(x=Z(4, 64, dtype=f32)), lin(x=Z(4, 63)), lin(x=Z(64, 4).t()), lin(x=Z(64)), lin(out=Z(4, 6, dtype=f32)), lin(t=t8[:5]),
        lambda **s: api.quantize_i8(Z(4, 64, dtype=f32), **s), lambda **s: api.quantize_i8(Z(64, 4).t(), **s),
        lambda **s: api.quantize_i8(Z(4, 0), **s), lambda **s: api.quantize_i8(Z(2, 65537), **s),
        lambda **s: api.quantize_i8(Z(1, 8).expand(3, 8), **s),
    ]
    st = torch.cuda.current_stream()
    for i, call in enumerate(bad):
        raised = []
        for kw in ({}, {"stream": st}):
            try:
                call(**kw)
                raised.append(None)
            except Exception as e:
                raised.append((type(e), str(e)))
        assert raised[0] == raised[1], (i, raised)
        if raised[0] is None:            # taken by both: the same bits
            a, b = call(), call(stream=st)
            for x, y in zip(*((z if isinstance(z, tuple) else (z,)) for z in (a, b))):
                assert x is None or torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)), i
    assert api.device_error() == api.BCQ_OK


def test_tensors_let_go_at_once_outlive_a_call_on_another_stream():
    """Inputs that nobody holds when a call on a side stream returns: their memory is not written over before it runs."""
    side = torch.cuda.Stream()
    c, k, v = _append_case([40, 70], [5, 70], 2, 128, 16, F16)
    q, x = _queries(75, 8, 128, F16), _queries(75, 4, 128, F16).view(75, 512)
    w, ws = api.quantize_i8(torch.randn(384, 512, device="cuda").half())
    codes, scale = api.quantize_i8(x)
    parts = lambda: [getattr(c.cache, n) for n in ("k", "k_param", "v", "v_param")]   # noqa: E731
    places = [c.t_table, c.t_len, c.t_cu]
    before = [t.clone() for t in parts()]
    api.kv4_append(c.cache, k, v, *places)
    after = [t.clone() for t in parts()]
    calls = [(lambda q, *t, **s: api.kv4_attention(q, api.Kv4Cache(*t[:4]), *t[4:], max_q=70, **s), [q, *after, *places]),
             (lambda *t, **s: api.kv4_read(api.Kv4Cache(*t[:4]), *t[4:], tokens=75, **s)[0], [*after, *places]),
             (api.linear_i8, [x, w, ws]), (api.gemm_i8, [codes, scale, w, ws]),
             (lambda x, **s: api.quantize_i8(x, **s)[0], [x])]
    for i, (call, args) in enumerate(calls):
        want = call(*args)
        mine = [t.clone() for t in args]
        sizes = sorted({t.numel() * t.element_size() for t in mine})
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                                      # some 10 ms
        y = call(*mine, stream=side)
        del mine
        junk = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        del junk
    mine, into = [t.clone() for t in (k, v, *places)], [t.clone() for t in before]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    api.kv4_append(api.Kv4Cache(*into), *mine, stream=side)
    sizes = sorted({t.numel() * t.element_size() for t in mine})
    del mine
    junk = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(into, after))
    assert api.device_error() == api.BCQ_OK


@pytest.mark.parametrize("heads,D", [(1, 64), (2, 128), (3, 256)])
@pytest.mark.parametrize("B", [257, 700])
def test_more_sequences_than_a_block_has_threads(B, heads, D):
    """Their row offsets no longer lie in shared memory: in, out and attention, some sequences without rows or tokens."""
    rng = np.random.default_rng(B + D)
    new = [int(x) for x in rng.integers(0, 4, B)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 40, B))]
    new[5] = lens[5] = 0
    c, k, v = _append_case(lens, new, heads, D, 16, F16)
    api.kv4_append(c.cache, k, v, c.t_table, c.t_len, c.t_cu)
    want = _expect_append(c, k, v)
    _check_cache(c, want)
    c.arrays = want
    rk, rv = api.kv4_read(c.cache, c.t_table, c.t_len, c.t_cu, tokens=c.T, dtype=F32)
    for got, x in ((rk, k), (rv, v)):
        code, param = kv4.quantize(_f64(x))
        assert np.array_equal(got.cpu().numpy(), kv4.values(kv4.pack(code), param).astype(np.float32))
    q = _queries(c.T, 2 * heads, D, F16)
    out, lse = _run(c, q)
    _check_attention(c, q, out, lse)
    out, lse = _run(c, q, 4000, max_q=5000)
    _check_attention(c, q, out, lse)
