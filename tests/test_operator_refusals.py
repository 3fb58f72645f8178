"""Calls of the 4-bit and cross-entropy operators that are refused before anything reaches the GPU: no GPU needed."""
import types

import pytest
import torch

import vector_codebook_codec_b200 as qamw
from test_abi_host import (FAKE, ODD, QAMW_EINVAL, QAMW_EUNSUPPORTED, _cef, _ceg, _cep, _cew, _cgw, _mxd, _mxl, _mxq)


@pytest.fixture
def _host_tensors(lib, monkeypatch):
    """The checks of type and shape alone, so that tensors in host memory pass for device ones."""
    def need(name, t, dtype=None, ndim=None):
        if t is not None and ((dtype is not None and t.dtype != dtype) or (ndim is not None and t.dim() != ndim)):
            raise ValueError(name)
    monkeypatch.setattr(qamw, "_need_cuda", need)


def _encoded(V=512, K=256, bits=8):
    return qamw.Encoded(torch.zeros((V, qamw.words_per_row(K, bits)), dtype=torch.int32), torch.ones(V), torch.ones(K),
                        torch.ones(K // 2), V, K, 128, 1, 256, bits)


def test_encoded_head_is_taken(_host_tensors):
    h = qamw._Head(_encoded(), torch.zeros((256, 2)))
    assert (h.V, h.K, h.ld) == (512, 256, 256)


@pytest.mark.parametrize("field,value", [
    ("row_norm", torch.ones(1024)[::2]), ("row_norm", torch.ones(1).expand(512)), ("row_norm", torch.ones(511)),
    ("sigma", torch.ones(256)[::2]), ("sigma", torch.ones(1).expand(128)), ("sigma", torch.ones(256)),
    ("col_scale", torch.ones(512)[::2]), ("col_scale", torch.ones(1).expand(256)),
    ("packed", torch.zeros((512, 64), dtype=torch.int32)[:, :32]), ("packed", torch.zeros((1, 64), dtype=torch.int32).expand(512, 64)),
])
def test_encoded_head_with_a_strided_or_broadcast_part(_host_tensors, field, value):
    """The decode takes every part as contiguous: a view with another stride would be read past its end."""
    head = _encoded()
    setattr(head, field, value)
    with pytest.raises(ValueError):
        qamw._Head(head, torch.zeros((256, 2)))


@pytest.mark.parametrize("codebook", [torch.zeros((256, 1)), torch.zeros((256, 3)), torch.zeros((1, 512)), None])
def test_encoded_head_with_another_codebook_shape(_host_tensors, codebook):
    with pytest.raises(ValueError):
        qamw._Head(_encoded(), codebook)


def test_stream_of_another_device():
    """It would be passed over: the work would go to the current stream of the tensors' device."""
    with pytest.raises(ValueError):
        qamw._on(torch.device("cuda", 0), types.SimpleNamespace(device=torch.device("cuda", 1)))


@pytest.mark.parametrize("call,argument", [(_mxq, "s"), (_mxd, "s"), (_mxl, "s"), (_cew, "loss"), (_cew, "lse"),
                                           (_cef, "loss"), (_cef, "lse"), (_cef, "t"), (_cgw, "lse"), (_cgw, "g"),
                                           (_ceg, "lse"), (_ceg, "g")])
def test_misaligned_vectors(lib, call, argument):
    """A float or int64 vector off its element's alignment would be a misaligned access on the GPU."""
    assert call(lib, **{argument: ODD}) == QAMW_EINVAL
    assert lib.qamw_last_error()


@pytest.mark.parametrize("call,kw", [(_cep, dict(ldx=1 << 39)), (_cep, dict(ldw=1 << 39)), (_cew, dict(ldw=1 << 39)),
                                     (_cew, dict(ldx=1 << 39)), (_ceg, dict(ldw=1 << 39)), (_cgw, dict(ldw=1 << 39)),
                                     (_cgw, dict(dW=FAKE, lddw=1 << 39)), (_ceg, dict(dW=FAKE, lddw=1 << 39))])
def test_rows_further_apart_than_a_tensor_map_holds(lib, call, kw):
    """Strides of 2^40 bytes: refused as arguments, before the kernels that need no tensor map are launched."""
    assert call(lib, **kw) == QAMW_EUNSUPPORTED
    assert lib.qamw_last_error()
