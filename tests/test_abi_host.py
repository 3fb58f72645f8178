"""Host-only checks of the C ABI: the library loads, exports every function
``include/qamw.h`` declares, and rejects bad arguments on the host with the
documented status code before touching the GPU (these calls never reach a
CUDA API, so they run without a device)."""
import ctypes
import os
import re
import subprocess

import pytest

from vector_codebook_codec_b200 import (LIB_PATH, QAMW_EINVAL, QAMW_ENULL, QAMW_EUNSUPPORTED,
                                        QAMW_EWORKSPACE, QAMW_OK)

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qamw.h")
FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: validation fails first


def _declared_functions():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(qamw_\w+)\s*\(", text)))


def test_header_declares_the_codec_entry_points():
    names = _declared_functions()
    for n in ("qamw_calibrate_sigma", "qamw_encode", "qamw_decode", "qamw_words_per_row",
              "qamw_calibrate_workspace_bytes", "qamw_status_string", "qamw_last_error"):
        assert n in names


def test_library_exports_every_declared_symbol(lib):
    out = subprocess.run(["nm", "-D", "--defined-only", LIB_PATH], capture_output=True, text=True).stdout
    exported = set(re.findall(r"\bT (qamw_\w+)$", out, flags=re.M))
    missing = [n for n in _declared_functions() if n not in exported]
    assert not missing, missing
    for n in _declared_functions():
        getattr(lib, n)


def test_words_per_row(lib):
    assert lib.qamw_words_per_row(4096, 11) == 704
    assert lib.qamw_words_per_row(11008, 10) == 1720
    assert lib.qamw_words_per_row(13824, 11) == 2376
    assert lib.qamw_words_per_row(512, 8) == 64
    assert lib.qamw_words_per_row(12, 11) == 3
    assert lib.qamw_words_per_row(3, 8) == -1
    assert lib.qamw_words_per_row(8, 0) == -1
    assert lib.qamw_words_per_row(8, 17) == -1


def test_status_strings(lib):
    for code in range(6):
        assert lib.qamw_status_string(code)
    assert lib.qamw_status_string(99) == b"unknown status"


def test_calibrate_workspace_bytes(lib):
    """The layout the header states: s [K] and r [M] in fp32, then the fp64
    partial sums [ceil(M/28)][K/2], each section rounded up to 256 bytes."""
    def a256(n):
        return (n + 255) // 256 * 256
    for M, K in ((4096, 4096), (1, 2), (29, 1000), (11008, 4096), (4096, 11008)):
        groups = (M + 27) // 28
        assert lib.qamw_calibrate_workspace_bytes(M, K) == a256(4 * K) + a256(4 * M) + a256(groups * (K // 2) * 8)
    assert lib.qamw_calibrate_workspace_bytes(0, 8) == 0
    assert lib.qamw_calibrate_workspace_bytes(8, 1) == 0


def _enc(lib, **kw):
    a = dict(W=FAKE, wt=1, M=8, K=256, ldw=256, act=None, alpha=0.5, block=128, seed=1, sigma=FAKE,
             cb=FAKE, N=256, bits=8, table=None, packed=FAKE, r=FAKE, s=FAKE, status=None, stream=None)
    a.update(kw)
    return lib.qamw_encode(a["W"], a["wt"], a["M"], a["K"], a["ldw"], a["act"], a["alpha"], a["block"],
                           a["seed"], a["sigma"], a["cb"], a["N"], a["bits"], a["table"], a["packed"], a["r"],
                           a["s"], a["status"], a["stream"])


def _dec(lib, **kw):
    a = dict(packed=FAKE, r=FAKE, sigma=FAKE, s=None, M=8, K=256, block=128, seed=1, cb=FAKE, N=256,
             bits=8, out=FAKE, ot=1, ldo=256, status=None, stream=None)
    a.update(kw)
    return lib.qamw_decode(a["packed"], a["r"], a["sigma"], a["s"], a["M"], a["K"], a["block"], a["seed"],
                           a["cb"], a["N"], a["bits"], a["out"], a["ot"], a["ldo"], a["status"], a["stream"])


def _cal(lib, **kw):
    a = dict(W=FAKE, wt=1, M=8, K=256, ldw=256, act=None, alpha=0.5, block=128, seed=1, sigma=FAKE,
             ws=FAKE, wsb=1 << 30, status=None, stream=None)
    a.update(kw)
    return lib.qamw_calibrate_sigma(a["W"], a["wt"], a["M"], a["K"], a["ldw"], a["act"], a["alpha"],
                                    a["block"], a["seed"], a["sigma"], a["ws"], a["wsb"], a["status"],
                                    a["stream"])


@pytest.mark.parametrize("kw,code", [
    (dict(W=None), QAMW_ENULL), (dict(sigma=None), QAMW_ENULL), (dict(cb=None), QAMW_ENULL),
    (dict(packed=None), QAMW_ENULL), (dict(r=None), QAMW_ENULL), (dict(s=None), QAMW_ENULL),
    (dict(K=255, ldw=255), QAMW_EINVAL), (dict(K=192, ldw=192), QAMW_EINVAL),
    (dict(block=96), QAMW_EINVAL), (dict(block=1), QAMW_EINVAL), (dict(block=2048, K=2048, ldw=2048), QAMW_EUNSUPPORTED),
    (dict(M=0), QAMW_EINVAL), (dict(ldw=128), QAMW_EINVAL), (dict(bits=0), QAMW_EINVAL),
    (dict(bits=17), QAMW_EINVAL), (dict(N=257), QAMW_EINVAL), (dict(N=0), QAMW_EINVAL),
    (dict(N=16384, bits=16), QAMW_EUNSUPPORTED), (dict(alpha=float("nan")), QAMW_EINVAL),
    (dict(alpha=float("inf")), QAMW_EINVAL), (dict(wt=7), QAMW_EINVAL),
    (dict(table=ctypes.c_void_p(0x10008)), QAMW_EINVAL),
])
def test_encode_rejects_on_host(lib, kw, code):
    assert _enc(lib, **kw) == code
    assert lib.qamw_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(packed=None), QAMW_ENULL), (dict(r=None), QAMW_ENULL), (dict(sigma=None), QAMW_ENULL),
    (dict(cb=None), QAMW_ENULL), (dict(out=None), QAMW_ENULL), (dict(K=7), QAMW_EINVAL),
    (dict(block=3), QAMW_EINVAL), (dict(ldo=100), QAMW_EINVAL), (dict(N=300), QAMW_EINVAL),
    (dict(ot=5), QAMW_EINVAL), (dict(bits=20, N=4), QAMW_EINVAL),
])
def test_decode_rejects_on_host(lib, kw, code):
    assert _dec(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(W=None), QAMW_ENULL), (dict(sigma=None), QAMW_ENULL), (dict(ws=None), QAMW_EWORKSPACE),
    (dict(wsb=16), QAMW_EWORKSPACE), (dict(ws=ctypes.c_void_p(0x10010)), QAMW_EINVAL),
    (dict(K=100, ldw=100), QAMW_EINVAL), (dict(alpha=float("nan")), QAMW_EINVAL), (dict(ldw=3), QAMW_EINVAL),
])
def test_calibrate_rejects_on_host(lib, kw, code):
    assert _cal(lib, **kw) == code


def _cal_enc(lib, **kw):
    a = dict(W=FAKE, wt=1, M=8, K=256, ldw=256, act=None, alpha=0.5, block=128, seed=1, cb=FAKE, N=256,
             bits=8, table=None, sigma=FAKE, packed=FAKE, r=FAKE, s=FAKE, ws=FAKE, wsb=1 << 30, status=None,
             stream=None)
    a.update(kw)
    return lib.qamw_calibrate_encode(a["W"], a["wt"], a["M"], a["K"], a["ldw"], a["act"], a["alpha"],
                                     a["block"], a["seed"], a["cb"], a["N"], a["bits"], a["table"], a["sigma"],
                                     a["packed"], a["r"], a["s"], a["ws"], a["wsb"], a["status"], a["stream"])


@pytest.mark.parametrize("kw,code", [
    (dict(W=None), QAMW_ENULL), (dict(cb=None), QAMW_ENULL), (dict(sigma=None), QAMW_ENULL),
    (dict(packed=None), QAMW_ENULL), (dict(r=None), QAMW_ENULL), (dict(s=None), QAMW_ENULL),
    (dict(ws=None), QAMW_EWORKSPACE), (dict(wsb=16), QAMW_EWORKSPACE),
    (dict(ws=ctypes.c_void_p(0x10010)), QAMW_EINVAL), (dict(K=255, ldw=255), QAMW_EINVAL),
    (dict(block=96), QAMW_EINVAL), (dict(M=0), QAMW_EINVAL), (dict(ldw=128), QAMW_EINVAL),
    (dict(N=257), QAMW_EINVAL), (dict(bits=17), QAMW_EINVAL), (dict(alpha=float("nan")), QAMW_EINVAL),
    (dict(wt=7), QAMW_EINVAL), (dict(table=ctypes.c_void_p(0x10008)), QAMW_EINVAL),
    (dict(block=2048, K=2048, ldw=2048), QAMW_EUNSUPPORTED),
])
def test_calibrate_encode_rejects_on_host(lib, kw, code):
    assert _cal_enc(lib, **kw) == code
    assert lib.qamw_last_error()


def test_rotate_and_scale_reject_on_host(lib):
    assert lib.qamw_rotate_rows(None, FAKE, 2, 8, 4, 0, 0, None) == QAMW_ENULL
    assert lib.qamw_rotate_rows(FAKE, FAKE, 2, 12, 8, 0, 0, None) == QAMW_EINVAL
    assert lib.qamw_channel_scale(None, 0.5, 8, None, None, None) == QAMW_ENULL
    assert lib.qamw_channel_scale(None, float("nan"), 8, FAKE, None, None) == QAMW_EINVAL


def test_error_message_cleared_on_next_rejection(lib):
    assert _enc(lib, W=None) == QAMW_ENULL
    first = lib.qamw_last_error()
    assert _enc(lib, K=255, ldw=255) == QAMW_EINVAL
    assert lib.qamw_last_error() != first and b"K" in lib.qamw_last_error()
    assert QAMW_OK == 0


def test_lloyd_entry_points_reject_on_host(lib):
    ws = 1 << 30
    assert lib.qamw_lloyd_workspace_bytes(0, 16) == 0
    assert lib.qamw_lloyd_workspace_bytes(1000, 16) >= 3 * 8 * 16 + 8
    assert lib.qamw_lloyd_assign(None, 10, FAKE, 4, FAKE, None, None) == QAMW_ENULL
    assert lib.qamw_lloyd_assign(FAKE, 10, FAKE, 4, None, None, None) == QAMW_ENULL
    assert lib.qamw_lloyd_assign(FAKE, 0, FAKE, 4, FAKE, None, None) == QAMW_EINVAL
    assert lib.qamw_lloyd_assign(FAKE, 10, FAKE, 0, FAKE, None, None) == QAMW_EINVAL
    assert lib.qamw_lloyd_assign(FAKE, 10, FAKE, 8193, FAKE, None, None) == QAMW_EINVAL
    assert lib.qamw_lloyd_assign(ctypes.c_void_p(0x10008), 10, FAKE, 4, FAKE, None, None) == QAMW_EINVAL
    assert lib.qamw_lloyd_update(FAKE, 10, FAKE, 4, FAKE, None, ws, None) == QAMW_EWORKSPACE
    assert lib.qamw_lloyd_update(FAKE, 10, FAKE, 4, FAKE, FAKE, 8, None) == QAMW_EWORKSPACE
    assert lib.qamw_lloyd_update(FAKE, 10, None, 4, FAKE, FAKE, ws, None) == QAMW_ENULL
    assert lib.qamw_lloyd_update(FAKE, 10, FAKE, 4, FAKE, ctypes.c_void_p(0x10010), ws, None) == QAMW_EINVAL
    it, conv = ctypes.c_int32(-5), ctypes.c_int32(-5)
    assert lib.qamw_lloyd_train(FAKE, 10, FAKE, 4, -1, FAKE, FAKE, ws, ctypes.byref(it), ctypes.byref(conv),
                                None) == QAMW_EINVAL
    assert lib.qamw_lloyd_train(FAKE, 10, FAKE, 4, 5, None, FAKE, ws, None, None, None) == QAMW_ENULL
    assert it.value == -5 and conv.value == -5   # untouched on a rejected call


def test_encode_polar_rejects_on_host(lib):
    def call(**kw):
        a = dict(W=FAKE, wt=1, M=8, K=256, ldw=256, act=None, alpha=0.5, block=128, seed=1, sigma=FAKE,
                 amps=FAKE, A=8, P=32, bits=8, packed=FAKE, r=FAKE, s=FAKE)
        a.update(kw)
        return lib.qamw_encode_polar(a["W"], a["wt"], a["M"], a["K"], a["ldw"], a["act"], a["alpha"], a["block"],
                                     a["seed"], a["sigma"], a["amps"], a["A"], a["P"], a["bits"], a["packed"],
                                     a["r"], a["s"], None, None)
    assert call(amps=None) == QAMW_ENULL
    assert call(A=0) == QAMW_EINVAL
    assert call(P=0) == QAMW_EINVAL
    assert call(A=16, P=32) == QAMW_EINVAL          # 512 points > 2^8
    assert call(amps=ctypes.c_void_p(0x10004)) == QAMW_EINVAL
    assert call(block=1024, K=1024, ldw=1024) == QAMW_EUNSUPPORTED


def test_selftest_rejects_on_host(lib):
    assert lib.qamw_selftest_wait_timeout(5, None, None) == QAMW_ENULL
    assert lib.qamw_selftest_wait_timeout(0, FAKE, None) == QAMW_EINVAL
    assert lib.qamw_selftest_wait_timeout((1 << 20) + 1, FAKE, None) == QAMW_EINVAL


def test_sharded_calibration_rejects_on_host(lib):
    assert lib.qamw_sigma_from_partial_sums(None, 1, 8, 8, FAKE, None) == QAMW_ENULL
    assert lib.qamw_sigma_from_partial_sums(FAKE, 0, 8, 8, FAKE, None) == QAMW_EINVAL
    assert lib.qamw_sigma_from_partial_sums(FAKE, 1, 8, 0, FAKE, None) == QAMW_EINVAL
    assert lib.qamw_calibrate_partial_sums(FAKE, 1, 8, 256, 256, None, 0.5, 128, 1, None, FAKE, 1 << 30, None,
                                           None) == QAMW_ENULL
    assert lib.qamw_calibrate_partial_sums(FAKE, 1, 8, 256, 256, None, 0.5, 128, 1, FAKE, None, 0, None,
                                           None) == QAMW_EWORKSPACE


def test_encode_prepared_rejects_on_host(lib):
    def call(**kw):
        a = dict(W=FAKE, wt=1, M=8, K=256, ldw=256, s=FAKE, r=FAKE, block=128, seed=1, sigma=FAKE, cb=FAKE,
                 N=256, bits=8, table=None, packed=FAKE, status=None, stream=None)
        a.update(kw)
        return lib.qamw_encode_prepared(a["W"], a["wt"], a["M"], a["K"], a["ldw"], a["s"], a["r"], a["block"],
                                        a["seed"], a["sigma"], a["cb"], a["N"], a["bits"], a["table"],
                                        a["packed"], a["status"], a["stream"])
    for kw in (dict(W=None), dict(s=None), dict(r=None), dict(sigma=None), dict(cb=None), dict(packed=None)):
        assert call(**kw) == QAMW_ENULL
    for kw in (dict(K=255, ldw=255), dict(block=96), dict(ldw=128), dict(bits=0), dict(N=257), dict(wt=7),
               dict(table=ctypes.c_void_p(0x10008))):
        assert call(**kw) == QAMW_EINVAL
    assert call(N=16384, bits=16) == QAMW_EUNSUPPORTED


def test_decode_matmul_rejects_on_host(lib):
    ws = lib.qamw_decode_matmul_workspace_bytes(128, 256, 16)
    assert ws >= 16 * 256 * 2 + 16 * 4 and ws % 256 == 0
    assert lib.qamw_decode_matmul_workspace_bytes(128, 256, 0) == 0
    assert lib.qamw_decode_matmul_workspace_bytes(0, 256, 16) == 0
    assert lib.qamw_decode_matmul_workspace_bytes(128, 256, (1 << 24) + 1) == 0

    def call(**kw):
        a = dict(packed=FAKE, r=FAKE, sigma=FAKE, s=None, M=128, K=256, block=128, seed=1, cb=FAKE, N=2048,
                 bits=11, X=FAKE, T=16, ldx=256, Y=FAKE, ldy=128, ws=FAKE, nws=ws, status=None, stream=None)
        a.update(kw)
        return lib.qamw_decode_matmul(a["packed"], a["r"], a["sigma"], a["s"], a["M"], a["K"], a["block"],
                                      a["seed"], a["cb"], a["N"], a["bits"], a["X"], a["T"], a["ldx"], a["Y"],
                                      a["ldy"], a["ws"], a["nws"], a["status"], a["stream"])
    for kw in (dict(packed=None), dict(r=None), dict(sigma=None), dict(cb=None), dict(X=None), dict(Y=None),
               dict(ws=None)):
        assert call(**kw) == QAMW_ENULL
    for kw in (dict(T=0), dict(T=(1 << 24) + 1), dict(ldx=255), dict(ldy=127), dict(X=ctypes.c_void_p(0x10008)), dict(ldx=260),
               dict(packed=ctypes.c_void_p(0x10004)), dict(sigma=ctypes.c_void_p(0x10008)),
               dict(ws=ctypes.c_void_p(0x10080)), dict(nws=ws - 1),
               dict(block=96), dict(N=2049)):
        assert call(**kw) == QAMW_EINVAL
    assert call(K=384 - 128 + 64, ldx=384) == QAMW_EINVAL               # K = 320: not a multiple of the block
    assert call(K=192, block=64, ldx=192) == QAMW_EUNSUPPORTED          # K not a multiple of 128
    big = lib.qamw_decode_matmul_workspace_bytes(128, 32768 + 128, 16)
    assert call(K=32768 + 128, ldx=32768 + 128, nws=big) == QAMW_EUNSUPPORTED


def test_mx4_scale_bytes(lib):
    """Tiles of 128 rows x 128 columns, 512 bytes each; 0 for an invalid shape."""
    assert lib.qamw_mx4_scale_bytes(1, 32) == 512
    assert lib.qamw_mx4_scale_bytes(129, 160) == 4 * 512
    assert lib.qamw_mx4_scale_bytes(11008, 4096) == 86 * 32 * 512
    for M, K in ((0, 32), (1, 0), (1, 31), (1, 48), (1 << 31, 32)):
        assert lib.qamw_mx4_scale_bytes(M, K) == 0


def _mxq(lib, **kw):
    a = dict(W=FAKE, wt=1, M=8, K=256, ldw=256, s=None, divide=0, block=128, seed=1, codes=FAKE, scales=FAKE)
    a.update(kw)
    return lib.qamw_mx4_quantize(*a.values(), None, None)


def _mxd(lib, **kw):
    a = dict(codes=FAKE, scales=FAKE, M=8, K=256, s=None, divide=0, block=128, seed=1, out=FAKE, ot=1, ldo=256)
    a.update(kw)
    return lib.qamw_mx4_decode(*a.values(), None)


def _mxm(lib, **kw):
    a = dict(wc=FAKE, ws=FAKE, M=8, xc=FAKE, xs=FAKE, T=4, K=256, Y=FAKE, ot=0, ldy=8)
    a.update(kw)
    return lib.qamw_mx4_matmul(*a.values(), None, None)


def _mxl(lib, **kw):
    a = dict(wc=FAKE, ws=FAKE, M=8, X=FAKE, xt=1, T=4, K=256, ldx=256, s=None, block=128, seed=1, Y=FAKE, ot=0, ldy=8,
             work=FAKE, wb=1 << 40)
    a.update(kw)
    return lib.qamw_mx4_linear(*a.values(), None, None)


ODD = ctypes.c_void_p(0x10001)


@pytest.mark.parametrize("call,kw,rc", [
    (_mxq, dict(W=None), QAMW_ENULL), (_mxq, dict(codes=None), QAMW_ENULL), (_mxq, dict(scales=None), QAMW_ENULL),
    (_mxq, dict(wt=7), QAMW_EINVAL), (_mxq, dict(M=0), QAMW_EINVAL), (_mxq, dict(K=240), QAMW_EINVAL),
    (_mxq, dict(K=0), QAMW_EINVAL), (_mxq, dict(ldw=255), QAMW_EINVAL), (_mxq, dict(block=1), QAMW_EINVAL),
    (_mxq, dict(block=96), QAMW_EINVAL), (_mxq, dict(block=512), QAMW_EINVAL),
    (_mxq, dict(block=2048, K=2048, ldw=2048), QAMW_EUNSUPPORTED), (_mxq, dict(W=ODD), QAMW_EINVAL),
    (_mxq, dict(codes=ODD), QAMW_EINVAL), (_mxq, dict(M=(1 << 30) + 1), QAMW_EUNSUPPORTED),
    (_mxq, dict(K=(1 << 24) + 32, ldw=1 << 25, block=32), QAMW_EUNSUPPORTED),
    (_mxd, dict(codes=None), QAMW_ENULL), (_mxd, dict(out=None), QAMW_ENULL), (_mxd, dict(ot=9), QAMW_EINVAL),
    (_mxd, dict(ldo=200), QAMW_EINVAL), (_mxd, dict(block=-2), QAMW_EINVAL), (_mxd, dict(scales=ODD), QAMW_EINVAL),
    (_mxd, dict(out=ODD), QAMW_EINVAL),
    (_mxm, dict(wc=None), QAMW_ENULL), (_mxm, dict(xs=None), QAMW_ENULL), (_mxm, dict(Y=None), QAMW_ENULL),
    (_mxm, dict(T=0), QAMW_EINVAL), (_mxm, dict(ldy=7), QAMW_EINVAL), (_mxm, dict(ot=2), QAMW_EINVAL),
    (_mxm, dict(K=100), QAMW_EINVAL), (_mxm, dict(xc=ODD), QAMW_EINVAL),
    (_mxl, dict(X=None), QAMW_ENULL), (_mxl, dict(Y=None), QAMW_ENULL), (_mxl, dict(wc=None), QAMW_ENULL),
    (_mxl, dict(T=0), QAMW_EINVAL), (_mxl, dict(ldx=255), QAMW_EINVAL), (_mxl, dict(ldy=7), QAMW_EINVAL),
    (_mxl, dict(block=6), QAMW_EINVAL), (_mxl, dict(xt=5), QAMW_EINVAL), (_mxl, dict(X=ODD), QAMW_EINVAL),
    (_mxl, dict(work=None), QAMW_EWORKSPACE), (_mxl, dict(wb=64), QAMW_EWORKSPACE), (_mxl, dict(work=ODD), QAMW_EINVAL),
])
def test_mx4_rejects_bad_arguments(lib, call, kw, rc):
    assert call(lib, **kw) == rc
    assert lib.qamw_last_error()


def test_mx4_linear_workspace_bytes(lib):
    from vector_codebook_codec_b200 import mx4_scale_bytes
    for T, K in ((1, 32), (37, 5120), (300, 4096)):
        assert lib.qamw_mx4_linear_workspace_bytes(T, K) == (T * K // 2 + 255) // 256 * 256 + mx4_scale_bytes(T, K)
        assert mx4_scale_bytes(T, K) == lib.qamw_mx4_scale_bytes(T, K)
    assert lib.qamw_mx4_linear_workspace_bytes(3, 40) == 0


def test_mx4_scale_layout_rejects_bad_arguments(lib):
    for f in (lib.qamw_mx4_pack_scales, lib.qamw_mx4_unpack_scales):
        assert f(None, 4, 64, FAKE, None) == QAMW_ENULL
        assert f(FAKE, 4, 64, None, None) == QAMW_ENULL
        assert f(FAKE, 4, 65, FAKE, None) == QAMW_EINVAL
        assert f(FAKE, 0, 64, FAKE, None) == QAMW_EINVAL


def test_cross_entropy_workspace_bytes(lib):
    """A maximum and a sum per token and 128 entries, then a logit per token."""
    def a256(n):
        return (n + 255) // 256 * 256
    for T, V in ((1, 1), (300, 50021), (4096, 65536)):
        assert lib.qamw_cross_entropy_workspace_bytes(T, V) == a256(8 * T * ((V + 127) // 128)) + a256(4 * T)
    for T, V in ((0, 5), (5, 0), ((1 << 24) + 1, 5)):
        assert lib.qamw_cross_entropy_workspace_bytes(T, V) == 0
    assert lib.qamw_cross_entropy_grad_workspace_bytes(4, 8, 256) >= 4 * 256 * 2 + 4 * 8 * 6
    for T, K, p in ((0, 8, 256), (4, 12, 256), (4, 8, 0)):
        assert lib.qamw_cross_entropy_grad_workspace_bytes(T, K, p) == 0


BIG = 1 << 40


def _cep(lib, **kw):
    a = dict(X=FAKE, T=8, K=64, ldx=64, W=FAKE, n=300, ldw=64, v0=0, V=300, t=FAKE, ignore=-100, ws=FAKE, wb=BIG)
    a.update(kw)
    return lib.qamw_cross_entropy_piece(*a.values(), None, None)


def _cef(lib, **kw):
    a = dict(T=8, V=300, t=FAKE, ignore=-100, ws=FAKE, wb=BIG, loss=FAKE, lse=FAKE)
    a.update(kw)
    return lib.qamw_cross_entropy_finish(*a.values(), None, None)


def _ceg(lib, **kw):
    a = dict(X=FAKE, T=8, K=64, ldx=64, W=FAKE, n=300, ldw=64, v0=0, V=300, t=FAKE, ignore=-100, lse=FAKE, g=FAKE,
             piece=300, first=1, dW=None, lddw=0, ws=FAKE, wb=BIG)
    a.update(kw)
    return lib.qamw_cross_entropy_grad_piece(*a.values(), None, None)


def _cex(lib, **kw):
    a = dict(T=8, K=64, piece=300, dX=FAKE, lddx=64, ws=FAKE, wb=BIG)
    a.update(kw)
    return lib.qamw_cross_entropy_grad_finish(*a.values(), None)


def _cew(lib, **kw):
    a = dict(X=FAKE, T=8, K=64, ldx=64, W=FAKE, V=300, ldw=64, t=FAKE, ignore=-100, loss=FAKE, lse=FAKE, ws=FAKE, wb=BIG)
    a.update(kw)
    return lib.qamw_cross_entropy(*a.values(), None, None)


def _cgw(lib, **kw):
    a = dict(X=FAKE, T=8, K=64, ldx=64, W=FAKE, V=300, ldw=64, t=FAKE, ignore=-100, lse=FAKE, g=FAKE, piece=300, dX=FAKE,
             lddx=64, dW=None, lddw=0, ws=FAKE, wb=BIG)
    a.update(kw)
    return lib.qamw_cross_entropy_grad(*a.values(), None, None)


@pytest.mark.parametrize("call", [_cew, _cgw])
@pytest.mark.parametrize("kw,rc", [
    (dict(X=None), QAMW_ENULL), (dict(W=None), QAMW_ENULL), (dict(t=None), QAMW_ENULL), (dict(lse=None), QAMW_ENULL),
    (dict(T=0), QAMW_EINVAL), (dict(K=60), QAMW_EINVAL), (dict(V=0), QAMW_EINVAL), (dict(ldx=60), QAMW_EINVAL),
    (dict(ldw=68), QAMW_EINVAL), (dict(X=ODD), QAMW_EINVAL), (dict(ws=None), QAMW_EWORKSPACE),
    (dict(wb=100), QAMW_EWORKSPACE), (dict(ws=ODD), QAMW_EINVAL), (dict(V=1 << 31), QAMW_EUNSUPPORTED),
])
def test_whole_cross_entropy_rejects_bad_arguments(lib, call, kw, rc):
    assert call(lib, **kw) == rc
    assert lib.qamw_last_error()


@pytest.mark.parametrize("kw,rc", [
    (dict(dX=None), QAMW_ENULL), (dict(g=None), QAMW_ENULL), (dict(lddx=63), QAMW_EINVAL), (dict(piece=0), QAMW_EINVAL),
    (dict(piece=200), QAMW_EINVAL), (dict(dW=FAKE, lddw=63), QAMW_EINVAL), (dict(dW=ODD, lddw=64), QAMW_EINVAL),
])
def test_whole_gradient_rejects_bad_arguments(lib, kw, rc):
    assert _cgw(lib, **kw) == rc
    assert lib.qamw_last_error()


@pytest.mark.parametrize("call", [_cep, _ceg])
@pytest.mark.parametrize("kw,rc", [
    (dict(X=None), QAMW_ENULL), (dict(W=None), QAMW_ENULL), (dict(t=None), QAMW_ENULL), (dict(T=0), QAMW_EINVAL),
    (dict(T=(1 << 24) + 1), QAMW_EINVAL), (dict(K=60), QAMW_EINVAL), (dict(ldx=60), QAMW_EINVAL),
    (dict(ldx=68), QAMW_EINVAL), (dict(ldw=56), QAMW_EINVAL), (dict(v0=100, V=1000), QAMW_EINVAL),
    (dict(v0=256), QAMW_EINVAL), (dict(n=300, V=1000), QAMW_EINVAL), (dict(n=0), QAMW_EINVAL),
    (dict(v0=-256), QAMW_EINVAL), (dict(X=ODD), QAMW_EINVAL), (dict(W=ODD), QAMW_EINVAL), (dict(t=ODD), QAMW_EINVAL),
    (dict(ws=None), QAMW_EWORKSPACE), (dict(wb=100), QAMW_EWORKSPACE), (dict(ws=ODD), QAMW_EINVAL),
    (dict(V=1 << 31, n=256), QAMW_EUNSUPPORTED),
])
def test_cross_entropy_pieces_reject_bad_arguments(lib, call, kw, rc):
    assert call(lib, **kw) == rc
    assert lib.qamw_last_error()


@pytest.mark.parametrize("call,kw,rc", [
    (_cef, dict(t=None), QAMW_ENULL), (_cef, dict(loss=None), QAMW_ENULL), (_cef, dict(lse=None), QAMW_ENULL),
    (_cef, dict(T=0), QAMW_EINVAL), (_cef, dict(V=0), QAMW_EINVAL), (_cef, dict(wb=16), QAMW_EWORKSPACE),
    (_ceg, dict(lse=None), QAMW_ENULL), (_ceg, dict(g=None), QAMW_ENULL), (_ceg, dict(piece=299), QAMW_EINVAL),
    (_ceg, dict(dW=FAKE, lddw=63), QAMW_EINVAL), (_ceg, dict(dW=ODD, lddw=64), QAMW_EINVAL),
    (_cex, dict(dX=None), QAMW_ENULL), (_cex, dict(lddx=63), QAMW_EINVAL), (_cex, dict(piece=0), QAMW_EINVAL),
    (_cex, dict(wb=16), QAMW_EWORKSPACE), (_cex, dict(K=12), QAMW_EINVAL),
])
def test_cross_entropy_rejects_bad_arguments(lib, call, kw, rc):
    assert call(lib, **kw) == rc
    assert lib.qamw_last_error()
