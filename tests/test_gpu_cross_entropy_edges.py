"""The head's cross entropy and its gradient at the ends of what they take:
tokens that the model is sure of, logits near the largest fp32 number, targets
out of range, gradients of a few tokens, and the same call again.

Logits here are products of one term, so they are exact. A loss is
(max - l_target) + log(sum): the difference of two logits, rounded once
(2^-24 of it), and the logarithm of a sum that starts at 1. Its error: two
or three roundings of 2^-24 where the sum is near 1 (a warp's, and the tiles'),
(12 + 4) 2^-24 + 12 x 1.3e-8 < 2^-19 of every other term (its argument's
rounding, the exponential, and log2 e in fp32), a step of the logarithm:
  |loss - loss64| <= 4 2^-24 + 2^-19 loss64."""
import math

import pytest
import torch

import vector_codebook_codec_b200 as qamw
from test_gpu_cross_entropy import _case, _coded_heads, _forward64

pytestmark = pytest.mark.gpu
IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    return lib


@pytest.mark.parametrize("top", [15.0, 30.0, 100.0, 300.0, 4096.0, -300.0])
@pytest.mark.parametrize("V", [2, 700, 5000])
def test_loss_of_a_sure_token(top, V):
    """A second logit 12 below the first: the loss of 6.1e-6 is far below a step of the normaliser."""
    W = torch.full((V, 16), 0.0, dtype=torch.bfloat16)
    X = torch.zeros((9, 16), dtype=torch.bfloat16)
    X[:, 0] = 1
    for t in torch.randint(0, V, (6,), generator=torch.Generator().manual_seed(V)).tolist():
        W[:, 0] = top - 80
        W[t, 0] = top
        W[(t + 1) % V, 0] = top - 12
        z = W[:, 0].double()
        ref = torch.log1p(torch.exp(z - z[t]).sum() - 1).item()
        loss, _ = qamw.cross_entropy(X.cuda(), W.cuda(), torch.full((9,), t, device="cuda"))
        assert ref > 0 and ((loss.double() - ref).abs() <= 4 * 2.0 ** -24 + 2.0 ** -19 * ref).all(), (loss, ref)


def _lowest_and_largest():
    V, K, low = 600, 8, torch.finfo(torch.bfloat16).min
    X = torch.zeros((4, K), dtype=torch.bfloat16)
    W = torch.zeros((V, K), dtype=torch.bfloat16)
    X[0, 0] = 1                      # every logit at the lowest value
    W[:, 0] = low
    X[1, 1] = 1                      # half of them, the others small
    W[::2, 1] = low
    W[1::2, 1] = torch.linspace(-2, 2, V // 2)
    X[2, 2] = 1                      # one at the largest
    W[:, 2] = 1
    W[7, 2] = -low
    X[3, 3] = 1                      # the lowest and the largest together
    W[:, 3] = low
    W[9, 3] = -low
    t = torch.tensor([5, 11, 7, 9])
    z = X.double() @ W.double().t()
    return X.cuda(), W.cuda(), t.cuda(), z.cuda()


def test_logits_near_the_largest_number():
    """Entries masked with the type's lowest value, tokens for which nothing else is left, and a logit near the top."""
    X, W, t, z = _lowest_and_largest()
    loss, lse = qamw.cross_entropy(X, W, t)
    lse64 = torch.logsumexp(z, dim=1)
    assert ((lse.double() - lse64).abs() <= 2.0 ** -21 * (1 + lse64.abs())).all()
    want = torch.tensor([math.log(W.shape[0]), (lse64[1] - z[1, 11]).item(), 0.0, 0.0], dtype=torch.float64, device="cuda")
    assert ((loss.double() - want).abs() <= 2.0 ** -20 * (1 + want)).all()


def test_gradient_of_logits_near_the_largest_number():
    """exp(l - lse) of the same: the entries of G and dW stay finite (dX sums products beyond fp32)."""
    X, W, t, z = _lowest_and_largest()
    lse = torch.logsumexp(z, dim=1).float()
    g = torch.tensor([1.0, 0.5, 0.25, 2.0], device="cuda")
    _, dW = qamw.cross_entropy_grad(X, W, t, lse, g)
    G = torch.exp(z - lse.double()[:, None])
    G.scatter_add_(1, t[:, None], -torch.ones_like(z[:, :1]))
    ref = (G * g.double()[:, None]).t() @ X.double()
    assert ((dW.double() - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -22).all()


def test_gradient_reports_targets_out_of_range():
    """qamw.h: another target outside [0, V) is left out and sets the status, in the gradient's calls too."""
    X, W, t, g = _case(40, 64, 500, 13, ignored=0.0)
    _, lse = qamw.cross_entropy(X, W, t)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qamw.cross_entropy_grad(X, W, t, lse, g, status=status)
    assert status.item() == 0
    for bad in (500, -1, 2 ** 40):
        for piece in (None, 256):
            u = t.clone()
            u[39] = bad
            status.zero_()
            qamw.cross_entropy_grad(X, W, u, lse, g, piece=piece, status=status)
            assert status.item() == qamw.STATUS_BAD_INDEX
    enc, C, mx = _coded_heads(500, 64 * 2, 5)
    X, _, t, g = _case(40, 128, 500, 14, ignored=0.5)
    _, lse = qamw.cross_entropy(X, mx, t)
    status.zero_()
    qamw.cross_entropy_grad(X, mx, t, lse, g, piece=256, status=status)
    assert status.item() == 0
    t[3] = 501
    qamw.cross_entropy_grad(X, mx, t, lse, g, piece=256, status=status)
    assert status.item() == qamw.STATUS_BAD_INDEX


@pytest.mark.parametrize("T,K,V", [(1, 64, 500), (1, 2048, 1504), (2, 512, 3000), (3, 72, 257), (5, 1024, 4100), (7, 256, 777),
                                   (16, 200, 1000), (16, 136, 2049)])
@pytest.mark.parametrize("piece", [None, 256])
def test_gradient_of_few_tokens_is_rounded_once(T, K, V, piece):
    """With few tokens the rounding of G does not average out: up to 16 of them G is held to 2^-16 (two bf16
    terms), and the outputs are rounded once. Logits wide enough that target probabilities spread over (0, 1).
    The bounds are those of test_gpu_cross_entropy.py with 2^-16 |G| in place of 2^-8 |G|."""
    X, W, t, g = _case(T, K, V, T + K + V, std=3.0 / K ** 0.5)
    with torch.no_grad():                      # the target's logit among the largest
        z = X.double() @ W.double().t()
        t = torch.where(t == IGNORE, t, z.topk(3, dim=1).indices[:, 1])
    _, lse = qamw.cross_entropy(X, W, t)
    dX, dW = qamw.cross_entropy_grad(X, W, t, lse, g, piece=piece)
    z, lse64, _, live, E = _forward64(X, W, t)
    p = torch.exp(z - lse64[:, None])
    G = p.clone()
    G.scatter_add_(1, t.clamp(min=0)[:, None], -live.double()[:, None])
    gl = torch.where(live, g.double(), torch.zeros_like(lse64))[:, None]
    G = G * gl
    dG = gl.abs() * (p * (E + (lse.double() - lse64).abs() + 2.0 ** -20)[:, None] + 2.0 ** -23) + 2.0 ** -16 * G.abs()
    X64, W64 = X.double(), W.double()
    for got, ref, tol in (
            (dX, G @ W64, dG @ W64.abs() + (V / 16 + 2) * 2.0 ** -22 * (G.abs() @ W64.abs())),
            (dW, G.t() @ X64, dG.t() @ X64.abs() + (T / 8 + 3) * 2.0 ** -22 * (G.abs().t() @ X64.abs()))):
        assert ((got.double() - ref).abs() <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()).all()
    assert (dX[~live] == 0).all()


def test_gradient_of_few_tokens_with_an_infinite_weight():
    """An infinite g_t: its own entries are Inf or NaN, the other tokens' rows of dX are what they were."""
    X, W, t, g = _case(20, 64, 300, 18, ignored=0.0)
    _, lse = qamw.cross_entropy(X, W, t)
    g[7] = float("inf")
    dX, _ = qamw.cross_entropy_grad(X, W, t, lse, g)
    g[7] = 0
    ref, _ = qamw.cross_entropy_grad(X, W, t, lse, g)
    assert not torch.isfinite(dX[7]).any()
    # their G is not scaled by max |g| then: other roundings
    rest = torch.arange(20, device="cuda") != 7
    assert ((dX - ref)[rest].abs().double() <= 2.0 ** -7 * ref[rest].abs().double() + 2.0 ** -15 * W.abs().sum(0).double()).all()


@pytest.mark.parametrize("T,V,K", [(1, 1000, 256), (16, 3001, 1024), (301, 5021, 512), (700, 9000, 1024)])
def test_the_same_call_gives_the_same_bits(T, V, K):
    """Alone, and with another batch's passes before and after that nothing waits for."""
    X, W, t, g = _case(T, K, V, 70)
    Y, _, u, h = _case(T, K, V, 71)
    loss, lse = qamw.cross_entropy(X, W, t)
    want = (loss, lse) + qamw.cross_entropy_grad(X, W, t, lse, g)
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for Z, v, w in ((X, t, g), (Y, u, h), (X, t, g)):
            loss, l = qamw.cross_entropy(Z, W, v)
            got.append((loss, l) + qamw.cross_entropy_grad(Z, W, v, l, w))
        torch.cuda.synchronize()
        for r in (got[0], got[2]):
            assert all(torch.equal(a, b) for a, b in zip(r, want))


@pytest.mark.parametrize("T", [1, 9, 16, 17])
def test_few_tokens_in_every_form(T):
    """Around the border of the two-term gradient: coded heads by pieces, slices of wider matrices, a replayed graph."""
    V, K = 900, 256
    enc, C, mx = _coded_heads(V, K, T)
    X, _, t, g = _case(T, K, V, 80 + T)
    W = qamw.mx4_decode(mx)
    for head, cb, rows in ((enc, C, qamw.decode(enc, C)), (mx, None, W)):
        for piece in (None, 256):
            _, lse = qamw.cross_entropy(X, head, t, codebook=cb, piece=piece)
            got = qamw.cross_entropy_grad(X, head, t, lse, g, codebook=cb, piece=piece, weight_grad=True)
            want = qamw.cross_entropy_grad(X, rows, t, lse, g, piece=piece)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    wide = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + K] = X
    got = qamw.cross_entropy_grad(wide[:, 8:8 + K], W, t, lse, g)
    want = qamw.cross_entropy_grad(X, W, t, lse, g)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dX, dW = qamw.cross_entropy_grad(X, W, t, lse, g)
    for seed in (1, 2):
        Y, _, u, h = _case(T, K, V, 90 + seed)
        X.copy_(Y), t.copy_(u), g.copy_(h)
        lse.copy_(qamw.cross_entropy(X, W, t)[1])
        graph.replay()
        torch.cuda.synchronize()
        want = qamw.cross_entropy_grad(X, W, t, lse, g)
        assert torch.equal(dX, want[0]) and torch.equal(dW, want[1])


def test_few_and_many_tokens_on_two_streams():
    """Two-term and one-term gradients and decodes that need fp64, at once."""
    a, b = _case(11, 512, 3000, 91), _case(200, 256, 2000, 92)
    streams = [torch.cuda.Stream() for _ in range(3)]
    big = qamw.mx4_quantize(torch.randn((300, 1024), device="cuda").clamp(-3, 3) * 2.0 ** 124, 64, 1)
    want = []
    for X, W, t, g in (a, b):
        loss, lse = qamw.cross_entropy(X, W, t)
        want.append((loss, lse) + qamw.cross_entropy_grad(X, W, t, lse, g))
    decoded = qamw.mx4_decode(big)
    assert torch.isfinite(decoded).all()
    torch.cuda.synchronize()
    got, ds = [[], []], []
    for _ in range(10):
        for n, (X, W, t, g) in enumerate((a, b)):
            loss, lse = qamw.cross_entropy(X, W, t, stream=streams[n])
            got[n].append((loss, lse) + qamw.cross_entropy_grad(X, W, t, lse, g, stream=streams[n]))
        ds.append(qamw.mx4_decode(big, stream=streams[2]))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for n in range(2) for r in got[n] for p, q in zip(r, want[n]))
    assert all(torch.equal(d, decoded) for d in ds)
