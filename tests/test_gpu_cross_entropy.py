"""The head's cross entropy and its gradient (qamw_cross_entropy_*) against
the formulas in fp64.

Logits: bf16 products are exact in fp32; the tensor cores add 16 of them and
the running sum, cutting below 2^-23 of the largest term, doubled for the
alignment inside a step: |dl_tv| <= (K / 16 + 2) 2^-22 S_tv, S = sum |x w|.
With E_t = max_v |dl_tv|:
  lse : E_t, plus the exponentials (2^-21 relative each) and their sums (256
        columns in order, the tiles in 8 chains): (256 + tiles + 32) 2^-24,
        plus 2^-22 |lse| for its arithmetic in units of log 2;
  loss: twice E_t plus the same;
  G   : g (p (E_t + the error of the given lse + 2^-20) ) and its bf16 rounding
        2^-8 |G| (p - 1 near p = 1 included: it is exact to 2^-24);
  dX  : sum_v |dG| |W| + (V / 16 + 2) 2^-22 sum |G W|, and 2^-8 |dX| for bf16;
  dW  : sum_t |dG| |X| + (T / 16 + 2) 2^-22 sum |G X|, and 2^-8 |dW|."""
import numpy as np
import pytest
import torch

import synth
import vector_codebook_codec_b200 as qamw

pytestmark = pytest.mark.gpu
IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    return lib


def _case(T, K, V, seed, std=0.05, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    W = (torch.randn(V, K, generator=g) * std).to(torch.bfloat16).cuda()
    t = torch.randint(0, V, (T,), generator=g)
    if T > 2:
        t[torch.rand(T, generator=g) < ignored] = IGNORE
        t[0], t[-1] = 0, V - 1
    return X, W, t.cuda(), torch.rand(T, generator=g).cuda() - 0.25


def _forward64(X, W, t):
    z = X.double() @ W.double().t()
    lse = torch.logsumexp(z, dim=1)
    live = t != IGNORE
    at = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    E = ((X.shape[1] / 16 + 2) * 2.0 ** -22 * (X.double().abs() @ W.double().abs().t())).amax(dim=1)
    return z, lse, torch.where(live, lse - at, torch.zeros_like(lse)), live, E


def _tail(V, lse):
    return (256 + V / 256 + 32) * 2.0 ** -24 + 2.0 ** -22 * lse.abs()


def _check_forward(X, W, t, loss, lse):
    z, lse64, loss64, live, E = _forward64(X, W, t)
    tail = _tail(W.shape[0], lse64) + 2.0 ** -21
    assert ((lse.double() - lse64).abs() <= E + tail).all()
    assert ((loss.double() - loss64).abs() <= 2 * E + tail + 2.0 ** -23 * loss64.abs()).all()
    assert (loss[~live] == 0).all()


def _check_grad(X, W, t, lse, g, dX, dW):
    z, lse64, _, live, E = _forward64(X, W, t)
    p = torch.exp(z - lse64[:, None])
    G = p.clone()
    G.scatter_add_(1, t.clamp(min=0)[:, None], -live.double()[:, None])
    gl = torch.where(live, g.double(), torch.zeros_like(lse64))[:, None]
    G = G * gl
    dG = gl.abs() * p * (E + (lse.double() - lse64).abs() + 2.0 ** -20)[:, None] + 2.0 ** -8 * G.abs()
    dG = dG + gl.abs() * 2.0 ** -23
    X64, W64 = X.double(), W.double()
    if dX is not None:
        ref = G @ W64
        tol = dG @ W64.abs() + (W.shape[0] / 16 + 2) * 2.0 ** -22 * (G.abs() @ W64.abs())
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
        assert ((dX.double() - ref).abs() <= tol).all()
        assert (dX[~live] == 0).all()
    if dW is not None:
        ref = G.t() @ X64
        tol = dG.t() @ X64.abs() + (X.shape[0] / 16 + 2) * 2.0 ** -22 * (G.abs().t() @ X64.abs())
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
        assert ((dW.double() - ref).abs() <= tol).all()


SHAPES = [(1, 8, 1), (1, 64, 300), (3, 72, 257), (128, 256, 512), (129, 128, 1000), (300, 64, 777),
          (257, 2048, 2049), (16, 2048, 5000), (513, 200, 4100), (2, 4096, 32000), (1025, 1024, 6007)]


@pytest.mark.parametrize("T,K,V", SHAPES)
def test_forward(T, K, V):
    X, W, t, _ = _case(T, K, V, T + K + V)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse = qamw.cross_entropy(X, W, t, status=status)
    assert status.item() == 0
    _check_forward(X, W, t, loss, lse)


@pytest.mark.parametrize("T,K,V", SHAPES)
def test_gradient(T, K, V):
    X, W, t, g = _case(T, K, V, T + K + V + 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, lse = qamw.cross_entropy(X, W, t, status=status)
    dX, dW = qamw.cross_entropy_grad(X, W, t, lse, g, status=status)
    assert status.item() == 0
    _check_grad(X, W, t, lse, g, dX, dW)


@pytest.mark.parametrize("T,K,V,piece", [(70, 96, 1000, 256), (300, 512, 3000, 512), (40, 64, 513, 256)])
def test_pieces_of_the_vocabulary(T, K, V, piece):
    """Pieces give the forward pass bit for bit, and the gradients within the bound."""
    X, W, t, g = _case(T, K, V, V)
    whole = qamw.cross_entropy(X, W, t)
    parts = qamw.cross_entropy(X, W, t, piece=piece)
    assert torch.equal(whole[0], parts[0]) and torch.equal(whole[1], parts[1])
    dX, dW = qamw.cross_entropy_grad(X, W, t, whole[1], g, piece=piece)
    _check_grad(X, W, t, whole[1], g, dX, dW)
    again = qamw.cross_entropy_grad(X, W, t, whole[1], g, piece=piece)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW)


def test_equal_weights_lose_nothing_to_the_rounding_of_g():
    """With the mean's equal g_t the gradients are as near as their bf16 outputs
    allow: the RMS error stays within 1.2 times that of rounding the exact ones."""
    T, K, V = 333, 256, 4000
    X, W, t, _ = _case(T, K, V, 17)
    g = torch.full((T,), 1.0 / 301.0, device="cuda")
    _, lse = qamw.cross_entropy(X, W, t)
    dX, dW = qamw.cross_entropy_grad(X, W, t, lse, g)
    z, lse64, _, live, _ = _forward64(X, W, t)
    G = torch.exp(z - lse64[:, None])
    G.scatter_add_(1, t.clamp(min=0)[:, None], -live.double()[:, None])
    G = G * (g.double() * live)[:, None]
    for got, ref in ((dX, G @ W.double()), (dW, G.t() @ X.double())):
        own = (ref.to(torch.bfloat16).double() - ref).norm()
        assert (got.double() - ref).norm() <= 1.2 * own


def test_a_bad_weight_stays_in_its_token():
    """A NaN g_t reaches its own row of dX only; zero weights give zero gradients."""
    X, W, t, g = _case(50, 64, 300, 18, ignored=0.0)
    _, lse = qamw.cross_entropy(X, W, t)
    g[7] = float("nan")
    dX, _ = qamw.cross_entropy_grad(X, W, t, lse, g)
    bad = torch.isnan(dX).any(dim=1)
    assert bad[7] and bad.sum() == 1
    dX, dW = qamw.cross_entropy_grad(X, W, t, lse, torch.zeros_like(g))
    assert (dX == 0).all() and (dW == 0).all()


def test_gradient_against_differences():
    """The directional derivative of the summed loss (fp64) along random directions."""
    X, W, t, g = _case(60, 128, 700, 4)
    loss, lse = qamw.cross_entropy(X, W, t)
    dX, dW = qamw.cross_entropy_grad(X, W, t, lse, g)
    gen = torch.Generator().manual_seed(9)
    U = torch.randn(X.shape, generator=gen, dtype=torch.float64).cuda()
    R = torch.randn(W.shape, generator=gen, dtype=torch.float64).cuda()

    def total(e):
        z = (X.double() + e * U) @ (W.double() + e * R).t()
        live = t != IGNORE
        at = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
        return (g.double() * torch.where(live, torch.logsumexp(z, dim=1) - at, torch.zeros_like(at))).sum()

    h = 1e-5
    diff = (total(h) - total(-h)) / (2 * h)
    got = (dX.double() * U).sum() + (dW.double() * R).sum()
    # every entry of dX and dW is off by two bf16 roundings at most, in random directions
    scale = ((dX.double() * U) ** 2).sum().sqrt() + ((dW.double() * R) ** 2).sum().sqrt()
    assert (got - diff).abs() <= 8 * 2.0 ** -7 * scale


def _coded_heads(V, K, seed):
    g = np.random.default_rng(seed)
    N, bits = 256, 8
    enc = qamw.Encoded(None, torch.from_numpy(synth.make_row_norms(V, seed)).cuda(),
                       torch.from_numpy(synth.make_act_rms(K, 0.5, seed)).cuda(),
                       torch.from_numpy(synth.make_sigma(K // 2, seed)).cuda(), V, K, 128, seed, N, bits)
    words = g.integers(-2 ** 31, 2 ** 31, (V, qamw.words_per_row(K, bits)), dtype=np.int64).astype(np.int32)
    enc.packed = torch.from_numpy(words).cuda()
    W = torch.from_numpy((g.standard_normal((V, K)) * 0.05).astype(np.float32)).cuda()
    s = torch.from_numpy(synth.make_act_rms(K, 0.5, seed + 1)).cuda()
    return enc, torch.from_numpy(qamw.load_codebook(N)).cuda(), qamw.mx4_quantize(W, 64, seed, s)


@pytest.mark.parametrize("piece", [None, 256, 512])
def test_coded_heads(piece):
    """A coded head gives what its decoded matrix gives, bit for bit."""
    V, K, T = 1200, 384, 150
    enc, C, mx = _coded_heads(V, K, 3)
    X, _, t, g = _case(T, K, V, 8)
    for head, cb, W in ((enc, C, qamw.decode(enc, C)), (mx, None, qamw.mx4_decode(mx))):
        loss, lse = qamw.cross_entropy(X, head, t, codebook=cb, piece=piece)
        ref = qamw.cross_entropy(X, W, t)
        assert torch.equal(loss, ref[0]) and torch.equal(lse, ref[1])
        _check_forward(X, W, t, loss, lse)
        dX, none = qamw.cross_entropy_grad(X, head, t, lse, g, codebook=cb, piece=piece)
        assert none is None
        dX2, dW2 = qamw.cross_entropy_grad(X, head, t, lse, g, codebook=cb, piece=piece, weight_grad=True)
        rX, rW = qamw.cross_entropy_grad(X, W, t, lse, g, piece=piece)
        assert torch.equal(dX, rX) and torch.equal(dX2, rX) and torch.equal(dW2, rW)


def test_perplexity_of_a_coded_head():
    """The set as it is used: code a head in both forms, score tokens drawn from
    the unrounded head, and follow the gradient: the loss of a coded head is
    above the original's on its own samples, and a step against dX lowers it."""
    V, K, T = 2048, 512, 256
    gen = torch.Generator().manual_seed(1)
    W = (torch.randn(V, K, generator=gen) * 0.1).to(torch.bfloat16)
    X = torch.randn(T, K, generator=gen).to(torch.bfloat16)
    t = torch.distributions.Categorical(logits=X.double() @ W.double().t()).sample().cuda()
    W, X = W.cuda(), X.cuda()
    C = torch.from_numpy(qamw.load_codebook(2048)).cuda()
    enc = qamw.calibrate_encode(W, None, 0.5, 128, 1, C, bits=11, search_table=qamw.build_search_table(C))
    mx = qamw.mx4_quantize(W, 128, 1)
    base = qamw.cross_entropy(X, W, t)[0].double().mean()
    for head, cb in ((enc, C), (mx, None)):
        loss, lse = qamw.cross_entropy(X, head, t, codebook=cb)
        dX, _ = qamw.cross_entropy_grad(X, head, t, lse, torch.full((T,), 1.0 / T, device="cuda"), codebook=cb)
        assert torch.isfinite(loss).all() and abs(loss.double().mean() - base) < 1.0
        Xn = (X.float() - 0.05 * T * dX.float()).to(torch.bfloat16)
        assert qamw.cross_entropy(Xn, head, t, codebook=cb)[0].mean() < loss.mean()


def test_large_logits_and_empty_rows():
    """Logits of some hundreds, equal logits, and a batch in which no token counts."""
    X, W, t, g = _case(140, 64, 600, 2, std=8.0)
    loss, lse = qamw.cross_entropy(X, W, t)
    assert lse.abs().max() > 100
    _check_forward(X, W, t, loss, lse)
    dX, dW = qamw.cross_entropy_grad(X, W, t, lse, g)
    _check_grad(X, W, t, lse, g, dX, dW)
    zero = torch.zeros_like(X)
    loss, lse = qamw.cross_entropy(zero, W, t)
    _check_forward(zero, W, t, loss, lse)
    none = torch.full_like(t, IGNORE)
    loss, lse = qamw.cross_entropy(X, W, none)
    dX, dW = qamw.cross_entropy_grad(X, W, none, lse, g)
    assert (loss == 0).all() and (dX == 0).all() and (dW == 0).all()


def test_padded_rows_may_hold_anything():
    """NaN and Inf in the rows of ignored tokens reach nothing but their own lse."""
    X, W, t, g = _case(200, 128, 900, 6)
    clean = X.clone()
    clean[t == IGNORE] = 0
    X[t == IGNORE] = float("nan")
    X[(t == IGNORE).nonzero()[0, 0]] = float("inf")
    g[t == IGNORE] = float("nan")
    loss, lse = qamw.cross_entropy(X, W, t)
    assert (loss[t == IGNORE] == 0).all() and torch.isfinite(loss).all()
    dX, dW = qamw.cross_entropy_grad(X, W, t, lse, g)
    ref = qamw.cross_entropy(clean, W, t)
    gz = torch.where(t == IGNORE, torch.zeros_like(g), g)
    rX, rW = qamw.cross_entropy_grad(clean, W, t, ref[1], gz)
    assert torch.equal(dX, rX) and torch.equal(dW, rW) and torch.equal(loss, ref[0])


def test_nan_stays_in_its_token():
    X, W, t, g = _case(40, 64, 500, 12, ignored=0.0)
    ref = qamw.cross_entropy(X, W, t)
    X[7, 3] = float("nan")
    loss, lse = qamw.cross_entropy(X, W, t)
    bad = torch.isnan(loss)
    assert bad.sum() == 1 and bad[7] and torch.equal(loss[~bad], ref[0][~bad])


def test_targets_out_of_range_are_reported_and_ignored():
    X, W, t, g = _case(40, 64, 500, 13, ignored=0.0)
    t2 = t.clone()
    t2[5], t2[6] = 500, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse = qamw.cross_entropy(X, W, t2, status=status)
    assert status.item() == qamw.STATUS_BAD_INDEX
    t3 = t.clone()
    t3[5], t3[6] = IGNORE, IGNORE
    assert torch.equal(loss, qamw.cross_entropy(X, W, t3)[0])
    for a, b in zip(qamw.cross_entropy_grad(X, W, t2, lse, g), qamw.cross_entropy_grad(X, W, t3, lse, g)):
        assert torch.equal(a, b)
    # another ignore_index, inside the vocabulary's range
    assert (qamw.cross_entropy(X, W, t, ignore_index=int(t[3]))[0][t == t[3]] == 0).all()


def test_strided_inputs():
    """Slices of wider matrices: leading dimensions that are multiples of 8."""
    X, W, t, g = _case(50, 96, 400, 21)
    Xw = torch.zeros((50, 128), dtype=torch.bfloat16, device="cuda")
    Ww = torch.zeros((400, 112), dtype=torch.bfloat16, device="cuda")
    Xw[:, 16:112] = X
    Ww[:, 8:104] = W
    a = qamw.cross_entropy(X, W, t)
    b = qamw.cross_entropy(Xw[:, 16:112], Ww[:, 8:104], t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for p, q in zip(qamw.cross_entropy_grad(X, W, t, a[1], g),
                    qamw.cross_entropy_grad(Xw[:, 16:112], Ww[:, 8:104], t, a[1], g)):
        assert torch.equal(p, q)


def test_captured_and_replayed():
    """Forward and backward in one graph, replayed on new inputs; two graphs in turn."""
    X, W, t, g = _case(150, 128, 700, 31)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _, l0 = qamw.cross_entropy(X, W, t)
        qamw.cross_entropy_grad(X, W, t, l0, g)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            loss, lse = qamw.cross_entropy(X, W, t)
            dX, dW = qamw.cross_entropy_grad(X, W, t, lse, g)
        graphs.append((gr, loss, lse, dX, dW))
    for k in range(2):
        Xn, Wn, tn, gn = _case(150, 128, 700, 40 + k)
        X.copy_(Xn), W.copy_(Wn), t.copy_(tn), g.copy_(gn)
        for gr, loss, lse, dX, dW in graphs:
            gr.replay()
        torch.cuda.synchronize()
        ref = qamw.cross_entropy(X, W, t)
        rX, rW = qamw.cross_entropy_grad(X, W, t, ref[1], g)
        for gr, loss, lse, dX, dW in graphs:
            assert torch.equal(loss, ref[0]) and torch.equal(lse, ref[1])
            assert torch.equal(dX, rX) and torch.equal(dW, rW)


def test_runs_on_a_given_stream():
    X, W, t, g = _case(64, 64, 300, 41)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    loss, lse = qamw.cross_entropy(X, W, t, stream=side)
    dX, dW = qamw.cross_entropy_grad(X, W, t, lse, g, stream=side)
    side.synchronize()
    ref = qamw.cross_entropy(X, W, t)
    rX, rW = qamw.cross_entropy_grad(X, W, t, ref[1], g)
    assert torch.equal(loss, ref[0]) and torch.equal(dX, rX) and torch.equal(dW, rW)


def test_offsets_beyond_32_bits():
    """A head of more than 2^32 bytes: the normaliser, targets at its end, and the last rows of dW."""
    T, K, V, tail = 3, 4096, 600000, 500
    gen = torch.Generator(device="cuda").manual_seed(1)
    W = torch.empty((V, K), dtype=torch.bfloat16, device="cuda")
    W.normal_(std=0.02, generator=gen)
    X = torch.randn((T, K), device="cuda", generator=gen).to(torch.bfloat16)
    t = torch.tensor([V - 1, V - 200, 5], device="cuda")
    g = torch.tensor([0.5, 0.25, -0.5], device="cuda")
    z = torch.cat([X.double() @ W[i:i + 50000].double().t() for i in range(0, V, 50000)], dim=1)
    lse64 = torch.logsumexp(z, dim=1)
    loss, lse = qamw.cross_entropy(X, W, t)
    # |logits| < 8, |x w| sums below 100: the bounds of the header with S = 100
    E = (K / 16 + 2) * 2.0 ** -22 * 100 + _tail(V, lse64) + 2.0 ** -21
    assert ((lse - lse64).abs() <= E).all()
    assert ((loss - (lse64 - z.gather(1, t[:, None])[:, 0])).abs() <= 2 * E).all()
    dX, dW = qamw.cross_entropy_grad(X, W, t, lse, g)
    G = torch.exp(z[:, V - tail:] - lse64[:, None])
    G[0, tail - 1] -= 1
    G[1, tail - 200] -= 1
    G = G * g.double()[:, None]
    tol = 2.0 ** -7 * (G.abs().t() @ X.double().abs()) + 2.0 ** -20 * X.double().abs().sum(0)
    assert ((dW[V - tail:].double() - G.t() @ X.double()).abs() <= tol).all()


def test_two_streams_at_once():
    """Forward and backward of two batches on two streams, beside 4-bit products on a third."""
    a, b = _case(300, 256, 2000, 61), _case(40, 128, 3000, 62)
    W = qamw.mx4_quantize(a[1], 64, 1)
    streams = [torch.cuda.Stream() for _ in range(3)]
    want = []
    for X, H, t, g in (a, b):
        loss, lse = qamw.cross_entropy(X, H, t)
        want.append((loss, lse) + qamw.cross_entropy_grad(X, H, t, lse, g))
    wanted = qamw.mx4_linear(W, a[0][:60])
    torch.cuda.synchronize()
    got, ys = [[], []], []
    for _ in range(10):
        for n, (X, H, t, g) in enumerate((a, b)):
            loss, lse = qamw.cross_entropy(X, H, t, stream=streams[n])
            got[n].append((loss, lse) + qamw.cross_entropy_grad(X, H, t, lse, g, stream=streams[n]))
        ys.append(qamw.mx4_linear(W, a[0][:60], stream=streams[2]))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for n in range(2) for r in got[n] for p, q in zip(r, want[n]))
    assert all(torch.equal(y, wanted) for y in ys)


def test_refusals():
    X, W, t, g = _case(8, 64, 300, 51)
    lse = torch.zeros(8, device="cuda")
    for bad in (dict(X=X.float()), dict(X=X.cpu()), dict(head=W.float()), dict(head=W[:, :56]), dict(targets=t[:7]),
                dict(targets=t.int()), dict(targets=t.cpu()), dict(piece=100), dict(piece=0),
                dict(targets=t.repeat(2)[::2]), dict(status=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            qamw.cross_entropy(**{"X": X, "head": W, "targets": t, **bad})
    for bad in (dict(lse=lse[:7]), dict(lse=lse.double()), dict(grad_loss=g.cpu()), dict(grad_loss=g[:, None])):
        with pytest.raises(ValueError):
            qamw.cross_entropy_grad(**{"X": X, "head": W, "targets": t, "lse": lse, "grad_loss": g, **bad})
    for Xb, Wb in ((X[:, :60], W[:, :60]), (X[:, 4:60], W[:, :56]), (X[:0], W)):
        with pytest.raises(qamw.QamwError):
            qamw.cross_entropy(Xb, Wb, t[:Xb.shape[0]])
    enc, C, mx = _coded_heads(256, 128, 1)
    with pytest.raises(ValueError):
        qamw.cross_entropy(X[:, :64], enc, t, codebook=C)
    with pytest.raises(ValueError):
        qamw.cross_entropy(torch.zeros((8, 128), dtype=torch.bfloat16, device="cuda"), enc, t)
