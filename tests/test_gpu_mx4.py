"""Microscaled 4-bit floating point (qamw_mx4_*) against the fp64 oracle.

Quantisation: codes and scale bytes equal the oracle's. Both sides rotate in
fp64 in different orders (matrix product and butterflies), so a value may be
decided differently only where it lies within 1e-12 (relative to the group's
unit) of a rounding border; those are counted and must be next to none.

Decode: fp32 butterflies. A chain of log2 b additions, the factor 1/sqrt(b)
(itself rounded) and the division by s, each rounding by at most 2^-24 of a
magnitude below A = sum_block |q| / sqrt(b) / s:
  |x - x_ref| <= (log2 b + 4) 2^-24 A, plus 2^-8 |x_ref| for bf16.

Product: every e2m1 product with its power-of-two scales is exact; the tensor
cores add 32 or 64 of them and the running fp32 sum, cutting bits below 2^-23
of the largest term, so K / 32 + 2 steps lose at most 2^-23 S each, S = sum
|x w| (doubled here for the alignment inside a step):
  |Y - Y_ref| <= (K / 32 + 2) 2^-22 S, plus 2^-8 |Y_ref| for bf16."""
import numpy as np
import pytest
import torch

import vector_codebook_codec_b200 as qamw
from oracle import mx4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    return lib


def _matrix(M, K, seed, dtype):
    g = np.random.default_rng(seed)
    W = g.standard_normal((M, K)) * 0.02 * np.exp(g.standard_normal((1, K)))
    if M >= 4:
        W[1] = 0.0                                 # a row of nothing
        W[2, : K // 2] = 0.0                       # groups of nothing
        W[3] = np.round(W[3] * 200) * 0.25         # values on the rounding borders
    t = torch.from_numpy(W.astype(np.float32)).to(dtype)
    return t, t.to(torch.float64).numpy()


def _scale(K, seed):
    return np.exp(0.5 * np.random.default_rng(seed + 1000).standard_normal(K)).astype(np.float32)


def _check_quantized(q, W64, s, divide, block, seed):
    code, byte, margin = mx4.quantize_rows(mx4.prepare_rows(W64, s, divide, block, seed))
    got = mx4.unpack_codes(q.codes.cpu().numpy())
    rows = qamw.mx4_scale_rows(q).cpu().numpy()
    assert np.array_equal(rows, byte)
    assert np.array_equal(q.scales.cpu().numpy(), mx4.tile_scales(byte))
    off = got != code
    # the sign of a value that rounds to zero may come from a cancellation's last bit
    off &= ~(((got & 7) == 0) & ((code & 7) == 0))
    assert not (off & (margin > 1e-12)).any(), int(off.sum())
    assert off.sum() <= 4


SHAPES = [(1, 32, 32), (1, 4096, 128), (3, 96, 32), (5, 1056, 0), (128, 1024, 1024), (129, 2048, 256),
          (37, 5120, 512), (64, 64, 2), (70, 160, 16), (33, 1024, 64), (2, 8192, 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", ["none", "multiply", "divide"])
@pytest.mark.parametrize("M,K,block", SHAPES)
def test_quantize(M, K, block, scale, dtype):
    t, W64 = _matrix(M, K, M + K, dtype)
    s = None if scale == "none" else _scale(K, K)
    sd = None if s is None else torch.from_numpy(s).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = qamw.mx4_quantize(t.cuda(), block, 77, sd, divide=scale == "divide", status=status)
    assert status.item() == 0
    _check_quantized(q, W64, s, scale == "divide", block, 77)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,shift", [(0, 1), (8, 0), (7, 3)])
def test_quantize_strided_and_unaligned(dtype, pad, shift):
    """A slice of a wider matrix: any leading dimension and any element alignment."""
    M, K = 35, 160
    t, _ = _matrix(M, K + pad + shift, 5, dtype)
    W = t.cuda()[:, shift:shift + K]
    q = qamw.mx4_quantize(W, 32, 4)
    _check_quantized(q, W.to(torch.float64).cpu().numpy(), None, False, 32, 4)


def test_quantize_special_values():
    """Subnormals, the largest values, negative zero, Inf and NaN groups."""
    rows = np.zeros((9, 64), dtype=np.float32)
    rows[0, 0] = 2.0 ** -149
    rows[1, 0], rows[1, 1] = 3.4e38, -3.0e38
    rows[2, 3] = np.nan
    rows[3, 40] = np.inf
    rows[4, :] = -0.0
    rows[5, :32] = np.linspace(-7.9, 7.9, 32)
    rows[6, 0], rows[6, 1:32] = 6.0, 2.0 ** -130
    rows[7, 0] = -np.inf
    rows[8, :] = 2.0 ** -126
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = qamw.mx4_quantize(torch.from_numpy(rows).cuda(), status=status)
    assert status.item() == qamw.STATUS_NONFINITE_INPUT
    _check_quantized(q, rows.astype(np.float64), None, False, 0, 0)
    v = qamw.mx4_decode(q, torch.float32).cpu().numpy()
    code, byte, _ = mx4.quantize_rows(rows.astype(np.float64))
    assert np.array_equal(v, mx4.values(code, byte).astype(np.float32), equal_nan=True)


def test_quantize_nan_spreads_over_its_block_only():
    t, W64 = _matrix(4, 256, 3, torch.float32)
    t[2, 70] = float("nan")
    W64[2, 70] = np.nan
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = qamw.mx4_quantize(t.cuda(), 64, 1, status=status)
    byte = qamw.mx4_scale_rows(q).cpu().numpy()
    assert status.item() == qamw.STATUS_NONFINITE_INPUT
    assert (byte[2, 2:4] == 255).all() and (byte == 255).sum() == 2


@pytest.mark.parametrize("M,K,block,scale,divide", [
    (1, 32, 0, False, False), (5, 96, 32, True, False), (129, 1024, 256, True, True), (3, 5120, 1024, True, False),
    (257, 2048, 64, False, False), (31, 160, 2, True, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode(M, K, block, scale, divide, dtype):
    t, _ = _matrix(M, K, K, torch.float32)
    s = _scale(K, 3) if scale else None
    sd = None if s is None else torch.from_numpy(s).cuda()
    q = qamw.mx4_quantize(t.cuda(), block, 5, sd, divide=divide)
    code, byte = mx4.unpack_codes(q.codes.cpu().numpy()), qamw.mx4_scale_rows(q).cpu().numpy()
    raw = qamw.mx4_decode(q, dtype, original=False).to(torch.float64).cpu().numpy()
    assert np.array_equal(raw, mx4.values(code, byte))
    wide = torch.full((M, K + 24), 7.0, dtype=dtype, device="cuda")
    got = qamw.mx4_decode(q, dtype, out=wide[:, 8:8 + K]).to(torch.float64).cpu().numpy()
    assert (wide[:, :8] == 7.0).all() and (wide[:, 8 + K:] == 7.0).all()
    ref = mx4.decode(code, byte, s, divide, block, 5)
    A = np.abs(mx4.values(code, byte))
    if block:
        A = np.repeat(A.reshape(M, K // block, block).sum(axis=2), block, axis=1) / np.sqrt(block)
    if s is not None:
        A = A * s if divide else A / s
    tol = (max(np.log2(max(block, 1)), 0) + 4) * 2.0 ** -24 * A
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(got - ref) <= tol).all()


def test_from_parts_round_trip():
    t, _ = _matrix(130, 416, 9, torch.bfloat16)
    q = qamw.mx4_quantize(t.cuda())
    rows = qamw.mx4_scale_rows(q)
    p = qamw.mx4_from_parts(q.codes, rows)
    assert torch.equal(p.scales, q.scales) and torch.equal(qamw.mx4_decode(p), qamw.mx4_decode(q))


PRODUCTS = [(1, 32, 1), (128, 256, 16), (129, 96, 17), (257, 1024, 33), (64, 160, 65), (300, 4096, 130),
            (200, 288, 257), (1000, 512, 300), (2048, 2080, 5), (77, 7424, 64), (640, 320, 1025)]


def _product_case(M, K, T, seed):
    W, _ = _matrix(M, K, seed, torch.bfloat16)
    X, _ = _matrix(T, K, seed + 1, torch.bfloat16)
    return qamw.mx4_quantize(W.cuda(), 32, 2), qamw.mx4_quantize(X.cuda(), 32, 2)


def _values(q):
    return qamw.mx4_decode(q, torch.float32, original=False).to(torch.float64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,T", PRODUCTS)
def test_matmul(M, K, T, dtype):
    Wq, Xq = _product_case(M, K, T, M + T)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = torch.full((T + 2, M + 3), 7.0, dtype=dtype, device="cuda")
    Y = qamw.mx4_matmul(Wq, Xq, dtype, status=status, out=wide[1:T + 1, 1:M + 1])
    assert status.item() == 0
    assert (wide[0] == 7.0).all() and (wide[T + 1] == 7.0).all()
    assert (wide[:, 0] == 7.0).all() and (wide[:, M + 1:] == 7.0).all()
    W, X = _values(Wq), _values(Xq)
    ref, S = X @ W.t(), X.abs() @ W.abs().t()
    tol = (K / 32 + 2) * 2.0 ** -22 * S
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    assert ((Y.to(torch.float64) - ref).abs() <= tol).all()


def test_matmul_extreme_scales():
    """Scale bytes over most of the exponent range, products kept inside fp32."""
    M, K, T = 130, 256, 20
    g = np.random.default_rng(0)
    wb = g.integers(127 - 60, 127 + 50, (M, K // 32)).astype(np.uint8)
    xb = g.integers(127 - 50, 127 + 60, (T, K // 32)).astype(np.uint8)
    wc = g.integers(0, 256, (M, K // 2)).astype(np.uint8)
    xc = g.integers(0, 256, (T, K // 2)).astype(np.uint8)
    Wq = qamw.mx4_from_parts(torch.from_numpy(wc).cuda(), torch.from_numpy(wb).cuda())
    Xq = qamw.mx4_from_parts(torch.from_numpy(xc).cuda(), torch.from_numpy(xb).cuda())
    Y = qamw.mx4_matmul(Wq, Xq).to(torch.float64).cpu().numpy()
    W, X = mx4.values(mx4.unpack_codes(wc), wb), mx4.values(mx4.unpack_codes(xc), xb)
    S = np.abs(X) @ np.abs(W).T
    assert (np.abs(Y - X @ W.T) <= (K / 32 + 2) * 2.0 ** -22 * S).all()


def test_matmul_nan_rows_stay_in_their_rows():
    Wq, Xq = _product_case(140, 128, 9, 3)
    clean = qamw.mx4_matmul(Wq, Xq)
    rows = qamw.mx4_scale_rows(Wq)
    rows[130, 1] = 255
    xr = qamw.mx4_scale_rows(Xq)
    xr[4, 0] = 255
    Wn = qamw.mx4_from_parts(Wq.codes, rows, 32, 2)
    Xn = qamw.mx4_from_parts(Xq.codes, xr, 32, 2)
    Y = qamw.mx4_matmul(Wn, Xn)
    nan = torch.isnan(Y)
    want = torch.zeros_like(nan)
    want[4, :] = True
    want[:, 130] = True
    assert torch.equal(nan, want)
    assert torch.equal(Y[~want], clean[~want])


@pytest.mark.parametrize("T", [1, 40, 300])
def test_linear_is_quantize_then_matmul(T):
    """The whole path as it is used: the product of the prepared rows, and the
    graph of it replayed on new activations, equal to the calls in turn."""
    M, K, block = 260, 1152, 128
    Wt, W64 = _matrix(M, K, 1, torch.bfloat16)
    s = _scale(K, 1)
    sd = torch.from_numpy(s).cuda()
    Wq = qamw.mx4_quantize(Wt.cuda(), block, 6, sd)
    X = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    X.normal_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qamw.mx4_linear(Wq, X)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = qamw.mx4_linear(Wq, X)
    for seed in (1, 2):
        Xt, X64 = _matrix(T, K, 50 + seed, torch.bfloat16)
        X.copy_(Xt)
        graph.replay()
        Xq = qamw.mx4_quantize(X, block, 6, sd, divide=True)
        _check_quantized(Xq, X64, s, True, block, 6)
        torch.cuda.synchronize()
        assert torch.equal(Y, qamw.mx4_matmul(Wq, Xq))


def test_linear_error_is_that_of_four_bits():
    """The 4-bit product against the unrounded one: an element is off by at most
    1/4 of a group's unit range, so the relative RMS error stays below 25%."""
    M, K, T = 256, 1024, 64
    g = torch.Generator().manual_seed(0)
    W = (torch.randn(M, K, generator=g) * 0.02).to(torch.bfloat16)
    W[:, 5] *= 20
    X = torch.randn(T, K, generator=g).to(torch.bfloat16)
    ref = X.double() @ W.double().t()
    Y = qamw.mx4_linear(qamw.mx4_quantize(W.cuda(), 128, 1), X.cuda()).double().cpu()
    assert (Y - ref).norm() / ref.norm() < 0.25


def test_runs_on_a_given_stream():
    t, W64 = _matrix(40, 512, 8, torch.bfloat16)
    W = t.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = qamw.mx4_quantize(W, 64, 3, stream=side)
    Y = qamw.mx4_linear(q, W, stream=side)
    side.synchronize()
    _check_quantized(q, W64, None, False, 64, 3)
    assert torch.equal(Y, qamw.mx4_linear(q, W))


def test_offsets_beyond_32_bits():
    """More than 2^32 bytes of input: the last rows equal those of a slice coded alone."""
    M, K, tail = 70000, 32768, 200
    W = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    W.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    q = qamw.mx4_quantize(W, 128, 5)
    part = qamw.mx4_quantize(W[M - tail:], 128, 5)
    assert torch.equal(q.codes[M - tail:], part.codes)
    assert torch.equal(qamw.mx4_scale_rows(q)[M - tail:], qamw.mx4_scale_rows(part))
    D = qamw.mx4_decode(q, out=W)
    assert torch.equal(D[M - tail:], qamw.mx4_decode(part))
    X = torch.randn((3, K), device="cuda").to(torch.bfloat16)
    Y, Yp = qamw.mx4_linear(q, X), qamw.mx4_linear(part, X)
    tol = (K / 32 + 2) * 2.0 ** -22 * (_values(qamw.mx4_quantize(X, 128, 5)).abs() @ _values(part).abs().t())
    assert ((Y[:, M - tail:] - Yp).abs() <= 2 * tol).all()


@pytest.mark.parametrize("kind", ["ties", "zeros", "constant", "tiny", "huge", "wide"])
@pytest.mark.parametrize("block", [0, 16, 64, 256])
def test_quantize_hard_rows(kind, block):
    """Rows that leave the fp32 decision open: exact ties of small integers, rows
    and groups of zeros, one rotated coefficient, magnitudes near the ends of
    fp32, and 2^40 between the columns."""
    M, K = 140, 1280
    g = np.random.default_rng(len(kind) + block)
    W = g.integers(-6, 7, (M, K)).astype(np.float64) * 0.25
    if kind == "zeros":
        W[g.random((M, K)) < 0.97] = 0.0
        W[:, 256:512] = 0.0
    elif kind == "constant":
        W[:] = g.standard_normal((M, 1))
    elif kind == "tiny":
        W = g.standard_normal((M, K)) * 2.0 ** -140
    elif kind == "huge":
        W = np.clip(g.standard_normal((M, K)), -3, 3) * 2.0 ** 124
    elif kind == "wide":
        W = g.standard_normal((M, K)) * 2.0 ** g.integers(-20, 21, (1, K))
    t = torch.from_numpy(W.astype(np.float32))
    s = _scale(K, 9)
    for sd, divide in ((None, False), (s, False), (s, True)):
        q = qamw.mx4_quantize(t.cuda(), block, 3, None if sd is None else torch.from_numpy(sd).cuda(), divide=divide)
        _check_quantized(q, t.to(torch.float64).numpy(), sd, divide, block, 3)


@pytest.mark.parametrize("value", [0.0, 2.0 ** -120, 2.0 ** 120, -1.5, float("inf")])
def test_quantize_unusual_scales(value):
    """Column scales far from 1, negative, zero or infinite: still the fp64 definition."""
    M, K = 9, 256
    t, W64 = _matrix(M, K, 5, torch.float32)
    s = _scale(K, 2)
    s[40:44] = value
    sd = torch.from_numpy(s).cuda()
    for divide in (False, True):
        for block in (0, 64):
            with np.errstate(all="ignore"):
                _check_quantized(qamw.mx4_quantize(t.cuda(), block, 1, sd, divide=divide), W64, s, divide, block, 1)


def test_many_streams_at_once():
    """Calls of every kernel on eight streams, interleaved: each as it is alone."""
    cases = []
    for i, (M, K, T) in enumerate([(300, 512, 1), (2048, 1024, 100), (640, 768, 20), (900, 512, 300), (4096, 512, 128),
                                   (77, 2048, 64), (1500, 1024, 128), (256, 4096, 3)]):
        W, _ = _matrix(M, K, i, torch.bfloat16)
        X, _ = _matrix(T, K, 50 + i, torch.bfloat16)
        q, x = qamw.mx4_quantize(W.cuda(), 64, i), X.cuda()
        cases.append((q, x, qamw.mx4_linear(q, x), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(20):
        for n, (q, x, _, stream) in enumerate(cases):
            got[n].append(qamw.mx4_linear(q, x, stream=stream))
    torch.cuda.synchronize()
    for n, (_, _, want, _) in enumerate(cases):
        assert all(torch.equal(y, want) for y in got[n])


def test_refusals():
    W = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    q = qamw.mx4_quantize(W)
    for bad in (dict(W=W.cpu()), dict(W=W.half()), dict(W=W.t()), dict(W=W[:, :48]), dict(W=W[0]),
                dict(col_scale=torch.ones(63, device="cuda")), dict(col_scale=torch.ones(64)),
                dict(col_scale=torch.ones(128, device="cuda")[::2]),
                dict(status=torch.zeros(1, device="cuda")),
                dict(out=(q.codes[:3], q.scales)), dict(out=(q.codes, q.scales[:-16]))):
        with pytest.raises(ValueError):
            qamw.mx4_quantize(**{"W": W, **bad})
    for block in (-1, 3, 128):
        with pytest.raises(qamw.QamwError):
            qamw.mx4_quantize(W, block)
    with pytest.raises(qamw.QamwError):
        qamw.mx4_quantize(W[:1].expand(4, 64))
    with pytest.raises(ValueError):
        qamw.mx4_decode(q, torch.float16)
    with pytest.raises(ValueError):
        qamw.mx4_decode(q, out=torch.empty((4, 32), dtype=torch.bfloat16, device="cuda"))
    other = qamw.mx4_quantize(torch.zeros((4, 96), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        qamw.mx4_matmul(q, other)
    with pytest.raises(ValueError):
        qamw.mx4_matmul(q, qamw.mx4_quantize(W, 32, 1))
    with pytest.raises(ValueError):
        qamw.mx4_linear(qamw.mx4_quantize(W, divide=True), W)
    with pytest.raises(ValueError):
        qamw.mx4_matmul(q, q, out=torch.empty((4, 5), device="cuda"))
    with pytest.raises(ValueError):
        qamw.mx4_from_parts(q.codes, torch.zeros((4, 3), dtype=torch.uint8, device="cuda"))
