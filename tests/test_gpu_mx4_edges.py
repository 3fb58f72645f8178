"""The microscaled 4-bit operators where they can go wrong at the ends of what
they take: groups that cancel against the rest of their block, the largest and
smallest scales of a decode, a quantisation that takes long.

Quantisation: the inputs are multiples of 2^-24 below 2^20, so a block's sums
are exact in fp64 in any order, and the codes have to be the oracle's.

Decode, as in test_gpu_mx4.py, with A = sum_block |q 2^e| / sqrt(b) / s:
  |x - x_ref| <= (log2 b + 4) 2^-24 A, plus half a step of the subnormal
numbers (2^-150) for fp32; for bf16 2^-8 |x_ref| and 2^-134 more. What the type
cannot hold (above its largest value by more than half a step) is Inf."""
import numpy as np
import pytest
import torch

import vector_codebook_codec_b200 as qamw
from oracle import codec, mx4
from test_gpu_mx4 import _check_quantized, _scale

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    return lib


def _grid(W, bits):
    return np.round(W * 2.0 ** bits) * 2.0 ** -bits


def _coefficient_rows(M, K, block, seed):
    """Rows that the rotation takes to one coefficient of each block and a residual of 2^-21 .. 2^-9 of it."""
    g = np.random.default_rng(seed)
    eps = 2.0 ** np.linspace(-21, -9, M)[:, None]
    return codec.sign_mask(seed, K) * _grid(1.0 + eps * g.standard_normal((M, K)), 23)


def _pair_rows(M, K, block, apart, seed):
    """N(0, 1) and two equal outliers of 3e3 .. 3e5 in each block, `apart` columns from one another: half of the
    block's groups see them cancel."""
    g = np.random.default_rng(seed)
    V = torch.from_numpy(g.standard_normal((M, K))).to(torch.bfloat16).double().numpy()
    V = _grid(V, 16)
    first = np.arange(0, K, block) + g.integers(0, 32)
    a = torch.from_numpy(10.0 ** np.linspace(3.5, 5.5, M)).to(torch.bfloat16).double().numpy()[:, None]
    V[:, first] = a
    V[:, first + apart] = a
    return codec.sign_mask(seed, K) * V


@pytest.mark.parametrize("block", [64, 128, 256, 1024])
def test_quantize_one_coefficient(block):
    W = _coefficient_rows(300, 2048, block, block)
    t = torch.from_numpy(W).float()
    assert np.array_equal(t.double().numpy(), W)
    _check_quantized(qamw.mx4_quantize(t.cuda(), block, block), W, None, False, block, block)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block,apart", [(64, 32), (128, 32), (128, 64), (256, 64), (256, 128), (1024, 32), (1024, 512)])
def test_quantize_equal_outliers(block, apart, dtype):
    W = _pair_rows(300, 2048, block, apart, block + apart)
    t = torch.from_numpy(W).to(dtype)
    assert np.array_equal(t.double().numpy(), W)
    for s, divide in ((None, False), (np.full(2048, 0.5, np.float32), False), (np.full(2048, 4.0, np.float32), True)):
        sd = None if s is None else torch.from_numpy(s).cuda()
        q = qamw.mx4_quantize(t.cuda(), block, block + apart, sd, divide=divide)
        _check_quantized(q, W, s, divide, block, block + apart)


def _check_decoded(q, dtype, code, byte, s, divide, block, seed):
    M, K = code.shape
    got = qamw.mx4_decode(q, dtype).double().cpu().numpy()
    with np.errstate(all="ignore"):
        ref = mx4.decode(code, byte, s, divide, block, seed)
        A = np.abs(mx4.values(code, byte))
        if block:
            A = np.repeat(A.reshape(M, K // block, block).sum(axis=2), block, axis=1) / np.sqrt(block)
        if s is not None:
            A = A * np.abs(s.astype(np.float64)) if divide else A / np.abs(s.astype(np.float64))
        tol = (np.log2(max(block, 1)) + 4) * 2.0 ** -24 * A + 2.0 ** -150
        if dtype == torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + 2.0 ** -134
        top = torch.finfo(dtype).max * (1 + torch.finfo(dtype).eps / 4)       # half a step above the largest value
        held, over = np.abs(ref) + tol < top, np.abs(ref) - tol > top
        assert (np.abs(got - ref) <= tol)[held].all()
        assert (got == np.sign(ref) * np.inf)[over].all()
        assert np.array_equal(np.isnan(got), np.isnan(ref))
    return held


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [0, 16, 32, 64, 256, 1024])
@pytest.mark.parametrize("power", [124, 100, -100, -126, -145])
def test_decode_magnitudes_near_the_ends_of_fp32(power, block, dtype):
    """Rows of 2^power, which the quantisation takes, come back: no Inf or 0 before the last rounding."""
    M, K = 140, 2048
    g = np.random.default_rng(block + power + 200)
    t = torch.from_numpy((np.clip(g.standard_normal((M, K)), -3, 3) * 2.0 ** power).astype(np.float32))
    for s, divide in ((None, False), (_scale(K, 9), False), (_scale(K, 9), True)):
        q = qamw.mx4_quantize(t.cuda(), block, 3, None if s is None else torch.from_numpy(s).cuda(), divide=divide)
        code, byte = mx4.unpack_codes(q.codes.cpu().numpy()), qamw.mx4_scale_rows(q).cpu().numpy()
        held = _check_decoded(q, dtype, code, byte, s, divide, block, 3)
        assert held.mean() > 0.9


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [0, 2, 32, 64, 128, 512, 1024])
def test_decode_any_scale_byte(block, dtype):
    """Scale bytes of the whole range beside one another, NaN and empty groups among them."""
    M, K = 90, 1056 if block <= 32 else 2048
    g = np.random.default_rng(block)
    byte = g.integers(0, 255, (M, K // 32)).astype(np.uint8)
    byte[:30] = g.integers(90, 160, (30, K // 32))
    byte[5, 3], byte[40, 7] = 255, 255
    codes = g.integers(0, 256, (M, K // 2)).astype(np.uint8)
    codes[20:25, 16:64] = 0
    byte[20:25, 1:4] = 0
    code = mx4.unpack_codes(codes)
    for s, divide in ((None, False), (_scale(K, 1), False), (_scale(K, 1), True)):
        q = qamw.mx4_from_parts(torch.from_numpy(codes).cuda(), torch.from_numpy(byte).cuda(), block, 11,
                                None if s is None else torch.from_numpy(s).cuda(), divide)
        _check_decoded(q, dtype, code, byte, s, divide, block, 11)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [0, 32, 256])
@pytest.mark.parametrize("value", [2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 2.0 ** 126, -2.0 ** 127])
def test_decode_extreme_column_scales(value, block, dtype):
    """Columns whose s lies at the ends of fp32, 1/s beyond them: x / s and x s as they are defined."""
    M, K = 70, 1024
    g = np.random.default_rng(block + 1)
    codes = g.integers(0, 256, (M, K // 2)).astype(np.uint8)
    byte = g.integers(60, 200, (M, 1)).astype(np.uint8).repeat(K // 32, axis=1)
    s = _scale(K, 2)
    s[40:44], s[700] = value, value
    code = mx4.unpack_codes(codes)
    for divide in (False, True):
        q = qamw.mx4_from_parts(torch.from_numpy(codes).cuda(), torch.from_numpy(byte).cuda(), block, 4,
                                torch.from_numpy(s).cuda(), divide)
        _check_decoded(q, dtype, code, byte, s, divide, block, 4)


@pytest.mark.parametrize("value", [0.0, float("inf"), float("nan")])
def test_decode_zero_and_infinite_column_scales(value):
    """x / 0, x / Inf, 0 Inf and their like (sums inside a group of 32 are exact, so a zero is one)."""
    M, K = 20, 256
    g = np.random.default_rng(3)
    codes = g.integers(0, 256, (M, K // 2)).astype(np.uint8)
    byte = g.integers(100, 150, (M, K // 32)).astype(np.uint8)
    s = _scale(K, 2)
    s[40:44] = value
    code = mx4.unpack_codes(codes)
    for block in (0, 32):
        for divide in (False, True):
            q = qamw.mx4_from_parts(torch.from_numpy(codes).cuda(), torch.from_numpy(byte).cuda(), block, 4,
                                    torch.from_numpy(s).cuda(), divide)
            got = qamw.mx4_decode(q, torch.float32).cpu().numpy()
            with np.errstate(all="ignore"):
                ref = mx4.decode(code, byte, s, divide, block, 4)
            odd = ~np.isfinite(ref)
            assert np.array_equal(got[odd], ref[odd].astype(np.float32), equal_nan=True)
            assert (got[:, 40:44][~odd[:, 40:44]] == 0).all() and np.isfinite(got[~odd]).all()


@pytest.mark.parametrize("T", [3, 100, 3000])
def test_linear_with_a_slow_quantisation(T):
    """Rows that rotate to one coefficient: all other groups are decided in fp64, some hundred times the usual
    work, and the product that has been launched beside it waits."""
    M, K, block = 200, 16384, 1024
    g = np.random.default_rng(T)
    X = codec.sign_mask(8, K) * torch.from_numpy(g.standard_normal((T, 1))).to(torch.bfloat16).double().numpy()
    t = torch.from_numpy(X).to(torch.bfloat16).cuda()
    W = qamw.mx4_quantize(torch.from_numpy(g.standard_normal((M, K)).astype(np.float32)).cuda(), block, 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Y = qamw.mx4_linear(W, t, status=status)
    Xq = qamw.mx4_quantize(t, block, 8, divide=True)
    assert torch.equal(Y, qamw.mx4_matmul(W, Xq)) and status.item() == 0
    assert (qamw.mx4_scale_rows(Xq).view(T, K // block, block // 32)[:, :, 1:] == 0).all()
