"""The microscaled 4-bit operators where they can go wrong at the ends of what
they take: groups that cancel against the rest of their block.

Quantisation: the inputs are multiples of 2^-24 below 2^20, so a block's sums
are exact in fp64 in any order, and the codes have to be the oracle's."""
import numpy as np
import pytest
import torch

import vector_codebook_codec_b200 as qamw
from oracle import codec
from test_gpu_mx4 import _check_quantized

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
