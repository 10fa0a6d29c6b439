"""The 8-bit product on the GPU against the fp64 oracle (oracle/i8.py).

Codes and scales have to be the oracle's, bit for bit.  Of a product, the sum
is exact and y = fp32(fp32(fp32(sum) sx) sw) rounded to its type, so with u =
2^-24 it is off by at most three roundings of u (relative: 3 u + 3 u^2 + u^3 <
3.01 u) and half a step of its type, and no more: the tolerance is that, plus
half of the type's smallest step where y is subnormal.
"""
import numpy as np
import pytest
import torch

from bit_gemv_bcq_b200 import api
from oracle import i8

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
SUBNORMAL = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()
    yield
    assert api.device_error() == api.BCQ_OK


def _f64(t):
    return t.double().cpu().numpy()


def _activations(M, K, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * scale
    x[:, torch.randperm(K, generator=g)[:max(1, K // 500)]] *= 20
    return x.to(dtype).cuda()


def _codes(M, K, seed, pad=0):
    """Codes -127..127 whose rows lie on 16 bytes, anything between them."""
    g = torch.Generator().manual_seed(seed)
    ld = -(-K // 16) * 16 + pad
    q = torch.randint(-127, 128, (M, ld), generator=g, dtype=torch.int8).cuda()
    return q[:, :K], (torch.rand(M, generator=g) * 0.01 + 1e-4).cuda()


def _check_product(y, ref, what):
    dtype = y.dtype
    rel = 3.01 * 2.0 ** -24 + (torch.finfo(dtype).eps / 2 if dtype != F32 else 0.0)
    err = np.abs(_f64(y) - ref)
    bad = ~(err <= rel * np.abs(ref) * (1 + 2.0 ** -10) + SUBNORMAL[dtype])
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {err.max():.3e}"


# ----------------------------------------------------------------- quantize

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (2, 8), (5, 128), (1, 4096), (17, 1003), (64, 2048),
                                 (2, 8192), (3, 8193), (2, 14336), (1, 65536), (300, 257)])
def test_codes_and_scales_are_the_oracles(M, K, dtype):
    x = _activations(M, K, dtype, 31 * M + K)
    q, s = api.quantize_i8(x)
    rq, rs = i8.quantize(_f64(x))
    assert q.shape == (M, K) and q.stride(0) % 16 == 0 or M == 1
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K,ld", [(2999, 72, 72), (3000, 72, 80), (8200, 1031, 1040), (1023, 5000, 5000),
                                    (1024, 5000, 5008), (1030, 16384, 16384), (1030, 4100, 4101)])
def test_many_rows(M, K, ld, dtype):
    """The other shapes of a block, and rows whose last eight values are fewer."""
    x = torch.full((M, ld), float("nan"), dtype=dtype, device="cuda")[:, :K]
    x.copy_(_activations(M, K, dtype, M + K))
    q, s = api.quantize_i8(x)
    rq, rs = i8.quantize(_f64(x))
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("K", [5, 40, 97, 4100])
@pytest.mark.parametrize("off", [0, 1])
def test_columns_beyond_a_row_are_left(K, off):
    x = _activations(3, K, F16, K)
    base = torch.empty(3 * K + 1, dtype=F16, device="cuda")
    view = base[off:off + 3 * K].view(3, K)
    view.copy_(x)
    ldq = -(-K // 16) * 16 + 16
    q = torch.full((3, ldq), 99, dtype=torch.int8, device="cuda")
    s = torch.zeros(3, device="cuda")
    assert api.lib().bcq_quantize_i8(view.data_ptr(), 0, 3, K, K, q.data_ptr(), ldq, s.data_ptr(), None) == api.BCQ_OK
    torch.cuda.synchronize()
    assert (q[:, K:] == 99).all()
    assert np.array_equal(q[:, :K].cpu().numpy(), i8.quantize(_f64(x))[0])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_halves_go_to_even_exactly(dtype):
    # max 254 u makes x = (2 j + 1) u the half j + 1/2 itself; its neighbours are not halves
    for u in (1.0, 2.0 ** -10, 2.0 ** -20 if dtype == BF16 else 2.0 ** -14):
        vals = [254.0 * u] + [s * (2 * j + 1) * u for j in range(127) for s in (1, -1)]
        x = torch.tensor([vals], dtype=torch.float64).to(dtype)
        x = torch.cat([x, torch.nextafter(x.float(), torch.tensor(0.0)).to(dtype)], 0).cuda()
        q, s = api.quantize_i8(x)
        rq, rs = i8.quantize(_f64(x))
        assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_every_mantissa_against_every_code(dtype):
    # each mantissa as a row's maximum, against a spread of values below it
    bits = 10 if dtype == F16 else 7
    top = 1.0 + torch.arange(2 ** bits, dtype=torch.float64) / 2 ** bits
    x = top[:, None] * torch.linspace(-1, 1, 515, dtype=torch.float64)[None]
    x = torch.cat([top[:, None], x], 1).to(dtype).cuda()
    q, s = api.quantize_i8(x)
    rq, rs = i8.quantize(_f64(x))
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("dtype,values", [
    (F16, [0.0, 6e-8, 6e-5, 65504.0]), (BF16, [0.0, 9.2e-41, 1e-38, 1e-20, 3.38e38])])
@pytest.mark.parametrize("K", [64, 100])
def test_extreme_rows(dtype, values, K):
    x = torch.zeros(len(values) + 4, K, dtype=torch.float64)
    ramp = torch.linspace(-1, 1, K, dtype=torch.float64)
    for i, v in enumerate(values):
        x[i] = ramp * v
    x = x.to(dtype)
    x[-4, 3], x[-3, 5], x[-2, K - 1], x[-1, 0] = float("nan"), float("inf"), float("-inf"), -0.0
    x = x.cuda()
    q, s = api.quantize_i8(x)
    rq, rs = i8.quantize(_f64(x))
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.isnan(rs[-4:-1]).all() and rs[-1] == 0


@pytest.mark.parametrize("M,K,ld,off", [(5, 96, 200, 0), (5, 96, 97, 0), (4, 40, 48, 1), (3, 33, 64, 8),
                                        (1, 100, 100, 3)])
def test_rows_apart_and_off_alignment(M, K, ld, off):
    base = torch.full((M * ld + off + 64,), float("nan"), dtype=F16, device="cuda")
    x = base[off:off + M * ld].view(M, ld)[:, :K]
    src = _activations(M, K, F16, 5)
    x.copy_(src)
    q, s = api.quantize_i8(x)
    rq, rs = i8.quantize(_f64(src))
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


# ------------------------------------------------------------------ product

SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 100, 48), (3, 33, 17), (7, 1000, 1003),
          (8, 256, 512), (16, 4096, 1024), (17, 130, 4096), (31, 1111, 257), (32, 96, 96),
          (33, 2048, 640), (64, 515, 2048), (65, 64, 31), (77, 1111, 1003), (127, 129, 255),
          (128, 128, 128), (129, 300, 1040), (200, 14336, 256), (256, 512, 4096), (257, 513, 130),
          (400, 777, 2064), (1000, 1000, 1000)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_product_matches_the_oracle(M, N, K, dtype):
    x, sx = _codes(M, K, 3 * M + K)
    w, sw = _codes(N, K, 5 * N + K + 1, pad=16)
    y = api.gemm_i8(x, sx, w, sw, dtype=dtype)
    assert y.dtype == dtype and y.shape == (M, N)
    _check_product(y, i8.gemm(x.cpu().numpy(), sx.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy()),
                   f"M={M} N={N} K={K} {dtype}")


@pytest.mark.parametrize("M,N,K", [(1, 14336, 4096), (16, 14336, 4096), (16, 4096, 14336), (48, 4096, 4096),
                                   (64, 14336, 4096), (100, 5000, 8192), (128, 14336, 2048), (144, 4096, 3000),
                                   (250, 9000, 4096), (333, 6000, 4000), (600, 8192, 4096), (1500, 4096, 1100),
                                   (333, 14336, 1024), (500, 9000, 2048), (512, 28672, 512), (700, 14336, 640)])
def test_long_sums_and_many_tiles(M, N, K):
    """Rings that wrap, tiles in several rounds: against fp64 on the GPU, three calls in a row."""
    x, sx = _codes(M, K, 3 * M + K)
    ws = [_codes(N, K, 7 * N + i) for i in range(3)]
    ys = [api.gemm_i8(x, sx, w, sw, dtype=F32) for w, sw in ws]
    for y, (w, sw) in zip(ys, ws):
        acc = x.double() @ w.double().t()          # exact: below 2^53
        ref = acc * sx.double()[:, None] * sw.double()[None]
        assert bool(((y.double() - ref).abs() <= 3.01 * 2.0 ** -24 * (1 + 2.0 ** -10) * ref.abs()).all())


@pytest.mark.parametrize("M", [1, 20, 300])
def test_largest_sums_do_not_wrap(M):
    K, N = 65536, 40
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one_m, one_n = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    y = api.gemm_i8(x, one_m, w, one_n, dtype=F32)
    assert torch.equal(y[:, 0], torch.full((M,), 2.0 ** 30, device="cuda"))
    assert torch.equal(y[:, 1], torch.full((M,), -128.0 * 127 * K, device="cuda"))


@pytest.mark.parametrize("M", [1, 5, 16, 40, 150])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_linear_is_quantize_and_product(M, dtype):
    N, K = 1030, 1544
    x = _activations(M, K, dtype, M)
    w, sw = api.quantize_i8(_activations(N, K, F16, 77, 0.02))
    y = api.linear_i8(x, w, sw)
    q, s = api.quantize_i8(x)
    assert torch.equal(y, api.gemm_i8(q, s, w, sw, dtype=dtype))
    rq, rs = i8.quantize(_f64(x))
    _check_product(y, i8.gemm(rq, rs, w.cpu().numpy(), sw.cpu().numpy()), f"linear M={M}")


@pytest.mark.parametrize("M", [2, 70])
def test_nan_and_zero_rows_stay_in_their_rows(M):
    N, K = 200, 160
    x = _activations(M, K, F16, 1)
    x[0, 7] = float("inf")
    x[1] = 0
    w, sw = api.quantize_i8(_activations(N, K, F16, 2, 0.02))
    y = api.linear_i8(x, w, sw)
    assert torch.isnan(y[0]).all() and (y[1] == 0).all()
    assert torch.isfinite(y[1:]).all()


@pytest.mark.parametrize("M,N,K", [(3, 70, 64), (40, 129, 100), (150, 300, 512)])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_output_rows_apart_leave_the_rest(M, N, K, dtype):
    x, sx = _codes(M, K, 1)
    w, sw = _codes(N, K, 2)
    big = torch.full((M + 2, N + 9), 7.0, dtype=dtype, device="cuda")
    out = big[1:M + 1, 3:N + 3]
    y = api.gemm_i8(x, sx, w, sw, dtype=dtype, out=out)
    assert y is out
    assert torch.equal(out, api.gemm_i8(x, sx, w, sw, dtype=dtype))
    big[1:M + 1, 3:N + 3] = 7.0
    assert (big == 7.0).all()


@pytest.mark.parametrize("M", [1, 24, 300])
def test_bytes_behind_a_row_are_not_data(M):
    N, K = 90, 45
    x, sx = _codes(M, K, 1)
    w, sw = _codes(N, K, 2)
    y = api.gemm_i8(x, sx, w, sw)
    for t in (x, w):   # other bytes between the rows
        full = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1))
        keep = t.clone()
        full.fill_(99)
        t.copy_(keep)
    assert torch.equal(api.gemm_i8(x, sx, w, sw), y)


def test_no_rows():
    w, sw = _codes(32, 64, 2)
    x = torch.empty(0, 64, dtype=F16, device="cuda")
    assert api.linear_i8(x, w, sw).shape == (0, 32)
    q, s = api.quantize_i8(x)
    assert q.shape == (0, 64) and s.shape == (0,)
    assert api.gemm_i8(q, s, w, sw).shape == (0, 32)


@pytest.mark.parametrize("M,K", [(1, 64), (5, 100), (40, 1000)])
def test_fast_calls_are_the_same_calls(M, K):
    """With the current stream named the binding takes its long way: the same bits."""
    st = torch.cuda.current_stream()
    x = _activations(M, K, BF16, 1)
    q, s = api.quantize_i8(x)
    q2, s2 = api.quantize_i8(x, stream=st)
    assert torch.equal(q, q2) and torch.equal(s, s2) and q.stride(0) == q2.stride(0)
    w, sw = _codes(70, K, 2)
    for dtype in (F16, BF16, F32):
        y = api.gemm_i8(q, s, w, sw, dtype=dtype)
        assert torch.equal(y, api.gemm_i8(q, s, w, sw, dtype=dtype, stream=st)) and y.dtype == dtype
        out = torch.empty_like(y)
        assert api.gemm_i8(q, s, w, sw, dtype=dtype, out=out) is out and torch.equal(out, y)
    y = api.linear_i8(x, w, sw)
    assert torch.equal(y, api.linear_i8(x, w, sw, stream=st)) and y.dtype == BF16


def test_side_stream_and_two_graphs_at_once():
    N, K = 600, 1024
    w, sw = api.quantize_i8(_activations(N, K, F16, 3, 0.02))
    xs = [_activations(m, K, F16, m) for m in (4, 90)]
    refs = [api.linear_i8(x, w, sw) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = api.linear_i8(xs[0], w, sw, stream=side)
    side.synchronize()
    assert torch.equal(y, refs[0])
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(api.linear_i8(x, w, sw))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)
    xs[0].copy_(_activations(4, K, F16, 99))     # replayed with other inputs
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], api.linear_i8(xs[0], w, sw))


@pytest.mark.parametrize("M,N,K", [(16, 60000, 4096), (3, 30000, 8192), (400, 16384, 4096), (1024, 8192, 2048), (77, 1111, 1003)])
def test_waits_that_run_out_are_reported(M, N, K):
    """Whichever wait of a kernel gives up first, in one CTA or in one of a pair, the call ends and says so."""
    x, sx = _codes(M, K, 1)
    w, sw = _codes(N, K, 2)
    ref = api.gemm_i8(x, sx, w, sw)
    try:
        given_up = 0
        for _ in range(30):
            api.debug_impatient(True)
            y = api.gemm_i8(x, sx, w, sw)
            status = api.device_error()
            assert status == api.BCQ_ERR_TIMEOUT or (status == api.BCQ_OK and torch.equal(y, ref))
            given_up += status == api.BCQ_ERR_TIMEOUT
            api.debug_impatient(False)
            y = api.gemm_i8(x, sx, w, sw)
            assert api.device_error() == api.BCQ_OK and torch.equal(y, ref)
        assert given_up
    finally:
        api.debug_impatient(False)


@pytest.mark.parametrize("N", [1, 3])
def test_as_many_rows_as_an_int_counts(N):
    M, K = 2 ** 31 - 1, 9
    if torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() < 80 << 30:
        pytest.skip("needs 80 GB")
    x = torch.empty(M, 16, dtype=torch.int8, device="cuda").random_(-127, 128)[:, :K]
    sx = torch.empty(M, device="cuda").uniform_(1e-3, 1e-2)
    w, sw = _codes(N, K, 2)
    y = api.gemm_i8(x, sx, w, sw)
    assert api.device_error() == api.BCQ_OK
    for part in (slice(0, 5000), slice(M // 2, M // 2 + 5000), slice(M - 5000, M)):
        ref = i8.gemm(_f64(x[part]), _f64(sx[part]), _f64(w), _f64(sw))
        _check_product(y[part], ref, part)
    del x, sx, y
    torch.cuda.empty_cache()
