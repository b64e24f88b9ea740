"""int8 rows and their product against plain forms in 64 bits.

Rows: codes and scales are exact by definition (rint of an exactly compared quotient, the
scale one correctly rounded division), so they are compared for equality.

Product: the integer sum is exact.  Converting it to binary32, two multiplications and an
addition round by at most 2^-24 each, relative to the value they give, and the type of y by
half its eps.  With p the scaled sum, v = p + bias:
    |y - v| <= 3.01 * 2^-24 |p| + 2^-24 |v| + eps/2 |v| (1 + 2^-22) + the type's smallest step.
"""
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
STEP = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}


@pytest.fixture(scope="module")
def iqq():
    import post_weight_quantization_rowwise_b200 as m
    return m


def _rows64(x):
    amax = x.double().abs().amax(1)
    d = torch.where(amax < 2.0 ** -119, 0.0, (amax / 127).float().double())
    q = torch.where(d[:, None] > 0, torch.round(x.double() / torch.where(d > 0, d, 1.0)[:, None]), 0.0)
    return q.to(torch.int8), d.float()


def _rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _codes(rows, n, seed, pad=0, lo=-127):
    """Random codes in rows of a multiple of 16 bytes, junk behind them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randint(lo, 128, (rows, (n + 15) // 16 * 16 + pad), generator=g, device="cuda").to(torch.int8)
    return buf[:, :n]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("nrows,n", [(1, 1), (1, 4096), (3, 7), (5, 129), (2, 11000), (700, 4096), (301, 333),
                                     (4, 20000), (400, 40000)])
def test_rows_exact(iqq, dtype, nrows, n):
    x = _rand((nrows, n), dtype, nrows * 31 + n)
    x[0, 0] = 40.0
    q, d = iqq.quantize_i8_rows(x)
    q0, d0 = _rows64(x)
    assert torch.equal(d, d0)
    assert torch.equal(q, q0)


def test_rows_ties_zeros_and_tiny(iqq):
    """Quotients on and next to a half, rows of zeros, and magnitudes around 2^-119 and the
    largest binary32."""
    n = 256
    d = torch.tensor([0.5, 3.0, 2.0 ** -60, 1.7e30, 0.0371], device="cuda")
    half = torch.arange(n, device="cuda") % 127 + 0.5
    x = d[:, None] * half
    x[:, 1::3] = torch.nextafter(x[:, 1::3], torch.zeros_like(x[:, 1::3]))
    x[:, 2::3] = torch.nextafter(x[:, 2::3], torch.full_like(x[:, 2::3], float("inf")))
    x[:, 5::7] *= -1
    x[:, 0] = 127 * d
    tiny = torch.zeros(6, n, device="cuda")
    tiny[1, 3] = 2.0 ** -119
    tiny[2, 3] = 2.0 ** -120
    tiny[3, 3] = 1e-45
    tiny[4, :] = torch.finfo(F32).max
    tiny[5, 1], tiny[5, 2] = 2.0 ** -118, -2.0 ** -119
    x = torch.cat([x, tiny])
    q, s = iqq.quantize_i8_rows(x)
    q0, s0 = _rows64(x)
    assert torch.equal(s, s0) and torch.equal(q, q0)


def test_rows_nonfinite_flagged_and_contained(iqq):
    x = _rand((5, 300), F32, 3)
    x[1, 299], x[3, 0], x[4, 5] = float("nan"), float("inf"), -float("inf")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, d = iqq.quantize_i8_rows(x, flags=flags)
    q0, d0 = _rows64(x[[0, 2]])
    assert int(flags.item()) == iqq.FLAG_NONFINITE_INPUT
    assert torch.equal(q[[0, 2]], q0) and torch.equal(d[[0, 2]], d0)
    assert torch.isnan(d[[1, 3, 4]]).all() and (q[[1, 3, 4]] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,ldx,off", [(100, 117, 1), (64, 64, 3), (4096, 4100, 0), (11000, 11008, 8)])
def test_rows_strides_and_alignment(iqq, dtype, n, ldx, off):
    """Rows apart and off 16-byte boundaries; bytes behind a row of codes stay as they were."""
    base = _rand((1, 9 * ldx + off), dtype, n)[0]
    x = torch.as_strided(base, (9, n), (ldx, 1), off)
    buf = torch.full((9, (n + 15) // 16 * 16 + 32), 77, dtype=torch.int8, device="cuda")
    d = torch.empty(9, device="cuda")
    iqq.iqq_quantize_i8_rows(x, buf[:, :n], d)
    q0, d0 = _rows64(x)
    assert torch.equal(buf[:, :n], q0) and torch.equal(d, d0)
    assert (buf[:, n:] == 77).all()


def _check(y, a, da, w, dw, bias):
    p = a.double() @ w.double().t() * (da.double()[:, None] * dw.double())
    v = p if bias is None else p + bias.double()
    half = torch.finfo(y.dtype).eps / 2 if y.dtype != F32 else 0.0
    bound = 3.01 * 2.0 ** -24 * p.abs() + 2.0 ** -24 * v.abs() + half * v.abs() * (1 + 2.0 ** -22) + STEP[y.dtype]
    off = (y.double() - v).abs() - bound
    assert off.max() <= 0, (float(off.max()), int((off > 0).sum()))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n_tok,n_out,k", [
    (1, 1, 1), (1, 4096, 4096), (1, 130, 11000), (2, 257, 129), (5, 64, 16), (8, 300, 4095), (16, 11008, 1024),
    (17, 1000, 640), (33, 129, 2048), (64, 512, 14336), (65, 511, 333), (100, 4099, 256), (128, 128, 128),
    (192, 640, 4096), (200, 300, 5000), (257, 513, 1000), (777, 1031, 2200), (1025, 260, 90), (3, 5, 131071),
    (2000, 3001, 300), (1100, 11008, 500), (5000, 2100, 140)])
def test_gemm_shapes(iqq, dtype, n_tok, n_out, k):
    a, w = _codes(n_tok, k, 1 + k), _codes(n_out, k, 2 + n_out, pad=32)
    da = _rand((n_tok, 1), F32, 3)[:, 0].abs() * 1e-3 + 1e-5
    dw = _rand((n_out, 1), F32, 4)[:, 0].abs() * 1e-3 + 1e-5
    bias = _rand((n_out, 1), F32, 5)[:, 0].contiguous() if (n_tok + n_out) % 2 else None
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = iqq.gemm_i8(a, da, w, dw, bias=bias, dtype=dtype, flags=flags)
    assert int(flags.item()) == 0
    _check(y, a, da, w, dw, bias)


@pytest.mark.parametrize("n_tok", [1, 6, 40, 300])
def test_gemm_extreme_codes(iqq, n_tok):
    """The largest sums 32 bits have to hold: -128 everywhere, at the largest k."""
    k = 131071
    a = torch.full((n_tok, 131072), -128, dtype=torch.int8, device="cuda")[:, :k]
    w = torch.full((70, 131072), -128, dtype=torch.int8, device="cuda")[:, :k]
    one = torch.ones(max(n_tok, 70), device="cuda")
    y = iqq.gemm_i8(a, one, w, one)
    assert (y == float(torch.tensor(float(16384 * k), dtype=F32))).all()


@pytest.mark.parametrize("n_tok,n_out", [(1, 300), (7, 300), (50, 257), (300, 259)])
def test_gemm_leaves_the_rest_of_y(iqq, n_tok, n_out):
    """A view of a wider y: what lies between and behind its rows stays as it was; offsets that
    leave y off any 16-byte boundary."""
    k = 500
    a, w = _codes(n_tok, k, 1), _codes(n_out, k, 2)
    da, dw = torch.full((n_tok,), 0.01, device="cuda"), torch.full((n_out,), 0.02, device="cuda")
    for dtype in (F32, BF16):
        buf = torch.full((n_tok + 2, n_out + 5), 7.0, dtype=dtype, device="cuda")
        iqq.iqq_gemm_i8(a, da, w, dw, buf[1:-1, 3:3 + n_out])
        _check(buf[1:-1, 3:3 + n_out], a, da, w, dw, None)
        rest = buf.clone()
        rest[1:-1, 3:3 + n_out] = 7.0
        assert (rest == 7.0).all()


def test_rows_of_no_values(iqq):
    """Rows of length 0 have the scale 0, and their product is the bias."""
    a, da = iqq.quantize_i8_rows(torch.empty(3, 0, device="cuda"))
    w, dw = iqq.quantize_i8_rows(torch.empty(40, 0, device="cuda"))
    bias = torch.arange(40.0, device="cuda")
    assert (da == 0).all() and a.shape == (3, 0)
    assert torch.equal(iqq.gemm_i8(a, da, w, dw, bias=bias), bias.expand(3, 40))


def test_gemm_empty_sum_and_nan_scale(iqq):
    a, w = _codes(3, 16, 1)[:, :0], _codes(40, 16, 2)[:, :0]
    one, bias = torch.ones(40, device="cuda"), torch.arange(40.0, device="cuda")
    assert torch.equal(iqq.gemm_i8(a, one, w, one, bias=bias), bias.expand(3, 40))
    a, w, da = _codes(3, 64, 1), _codes(40, 64, 2), torch.tensor([1.0, float("nan"), 1.0], device="cuda")
    y = iqq.gemm_i8(a, da, w, one)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2]]).all()


def test_gemm_same_value_however_split(iqq):
    """An output depends on its token and channel alone: one token by itself, within batches of
    every size class, and run after run."""
    k, n_out = 4096, 1000
    a, w = _codes(600, k, 8), _codes(n_out, k, 9)
    da, dw = _rand((600, 1), F32, 1)[:, 0].abs(), _rand((n_out, 1), F32, 2)[:, 0].abs()
    whole = iqq.gemm_i8(a, da, w, dw)
    assert torch.equal(whole, iqq.gemm_i8(a, da, w, dw))
    for n in (1, 2, 9, 20, 40, 70, 130, 200, 300):
        assert torch.equal(iqq.gemm_i8(a[:n], da, w, dw), whole[:n]), n
    assert torch.equal(iqq.gemm_i8(a, da, w[:130], dw), whole[:, :130])


def test_linear_on_a_side_stream_and_in_a_graph(iqq):
    """Rows and product together, as a layer runs them: on a stream of its own, and captured and
    replayed with new inputs."""
    x, w = _rand((24, 2000), BF16, 1), _rand((700, 2000), F32, 2)
    wc, dw = iqq.quantize_i8_rows(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, d = iqq.quantize_i8_rows(x, stream=side)
    y = iqq.gemm_i8(a, d, wc, dw, dtype=BF16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    q0, d0 = _rows64(x)
    _check(y, q0, d0, wc, dw, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, d = iqq.quantize_i8_rows(x)
        y2 = iqq.gemm_i8(a, d, wc, dw, dtype=BF16)
    for seed in (1, 5):
        x.copy_(_rand((24, 2000), BF16, seed))
        graph.replay()
        q0, d0 = _rows64(x)
        _check(y2, q0, d0, wc, dw, None)


def test_calls_in_turn_on_the_same_buffers(iqq):
    """Rows and product over and over into the same codes, scales and y with other data, and nothing that
    waits for the device between the calls: every call sees what the one before wrote."""
    xs = [_rand((40, 1000), F32, i) * 2.0 ** (i % 5 - 2) for i in range(24)]
    w, dw = iqq.quantize_i8_rows(_rand((300, 1000), F32, 99))
    codes, scales = torch.zeros(40, 1008, dtype=torch.int8, device="cuda")[:, :1000], torch.zeros(40, device="cuda")
    ys = [torch.zeros(40, 300, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        iqq.iqq_quantize_i8_rows(x, codes, scales)
        iqq.iqq_gemm_i8(codes, scales, w, dw, y)
    for x, y in zip(xs, ys):
        q0, d0 = _rows64(x)
        _check(y, q0, d0, w, dw, None)
