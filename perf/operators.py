"""What is measured of the microscaled 4-bit operators and of the head's cross entropy.

Two families, five operators:

* microscaled 4-bit floating point (OCP MX: e2m1 elements, one e8m0 scale per
  32 columns), after the codec's own channel scale and sign-masked block
  Hadamard rotation: ``mx4_quantize``, ``mx4_decode`` and the product
  ``mx4_linear`` (quantise the activations, multiply on the tensor cores);
* the cross entropy of a model's head, without keeping the logits, and its
  gradient: ``cross_entropy`` and ``cross_entropy_grad``.

``run`` holds the plain forms (elementary torch operations) and the calls a
user makes; ``exact`` restates each operator in 64 bits in another way.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
IGNORE = -100
# e2m1: the magnitudes of codes 0..7, and the borders between neighbours
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one token's activations on their way into a coded layer: latency
        {"name": "quantize_token_1x4096", "op": "quantize", "M": 1, "K": 4096, "dtype": "bf16", "block": 128,
         "scale": "divide", "pad": 0},
        # a whole MLP projection, coded once per checkpoint
        {"name": "quantize_11008x4096", "op": "quantize", "M": 11008, "K": 4096, "dtype": "bf16", "block": 128,
         "scale": "multiply", "pad": 0},
        # plain microscaling of an fp32 master copy, a slice of a wider matrix, an odd number of rows
        {"name": "quantize_f32_1003x5632", "op": "quantize", "M": 1003, "K": 5632, "dtype": "f32", "block": 0,
         "scale": "none", "pad": 32},
        # the coded matrix back as the bf16 weights of a library product
        {"name": "decode_5120x13824", "op": "decode", "M": 5120, "K": 13824, "dtype": "bf16", "block": 256,
         "scale": "multiply"},
        # a small coded matrix back in fp32, to measure its error
        {"name": "decode_f32_257x2048", "op": "decode", "M": 257, "K": 2048, "dtype": "f32", "block": 64,
         "scale": "none"},
        # one token through an attention projection: generation
        {"name": "linear_t1_4096x4096", "op": "linear", "T": 1, "M": 4096, "K": 4096, "dtype": "f32", "block": 128,
         "scale": "multiply"},
        # a ragged batch of requests through a 13B MLP projection
        {"name": "linear_t37_13824x5120", "op": "linear", "T": 37, "M": 13824, "K": 5120, "dtype": "bf16",
         "block": 128, "scale": "multiply"},
        # a prompt through an MLP projection
        {"name": "linear_t4096_11008x4096", "op": "linear", "T": 4096, "M": 11008, "K": 4096, "dtype": "bf16",
         "block": 128, "scale": "multiply"},
        # the scores of a few continuations: the head's weights are all there is to read
        {"name": "ce_t16_v32000_k2048", "op": "ce", "T": 16, "V": 32000, "K": 2048, "ignored": 0.0},
        # perplexity over one sequence
        {"name": "ce_t4096_v32000_k4096", "op": "ce", "T": 4096, "V": 32000, "K": 4096, "ignored": 0.1},
        # sensitivities from a short text, ragged in every size
        {"name": "ce_grad_t301_v50021_k2048", "op": "ce_grad", "T": 301, "V": 50021, "K": 2048, "ignored": 0.1},
        # a training step of a large head
        {"name": "ce_grad_t4096_v65536_k4096", "op": "ce_grad", "T": 4096, "V": 65536, "K": 4096, "ignored": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "decode", "linear", "linear", "ce", "ce_grad"])
    if op in ("ce", "ce_grad"):
        return {"op": op, "T": _log(rng, 1, 4096), "V": _log(rng, 1000, 65536), "K": 8 * _log(rng, 32, 512),
                "ignored": rng.choice([0.0, 0.1, 0.5])}
    block = rng.choice([0, 32, 64, 128, 256])
    step = max(block, 32)
    K = step * max(1, _log(rng, 256, 13824) // step)
    c = {"op": op, "K": K, "block": block}
    if op == "linear":
        c.update(T=_log(rng, 1, 4096), M=_log(rng, 64, 13824), dtype=rng.choice(["bf16", "f32"]),
                 scale=rng.choice(["none", "multiply"]))
    elif op == "decode":
        c.update(M=_log(rng, 64, 13824), dtype=rng.choice(["bf16", "f32"]), scale=rng.choice(["none", "multiply"]))
    else:
        c.update(M=_log(rng, 1, 13824), dtype=rng.choice(["bf16", "f32"]),
                 scale=rng.choice(["none", "multiply", "divide"]), pad=rng.choice([0, 0, 32]))
    return c


def work(case):
    op, K = case["op"], case["K"]
    if op in ("ce", "ce_grad"):
        T, V = case["T"], case["V"]
        if op == "ce":
            return {"bytes": 2 * (T + V) * K + 8 * T + 8 * T, "flops": 2 * T * V * K}
        # the logits again (they are not kept), dX and dW: the products
        return {"bytes": 2 * 2 * (T + V) * K + 16 * T, "flops": 6 * T * V * K}
    coded = 17 / 32
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "linear":
        T, M = case["T"], case["M"]
        return {"bytes": int(coded * M * K + 2 * T * K + size * T * M), "flops": 2 * T * M * K}
    M = case["M"]
    rot = M * K * int(math.log2(case["block"])) if case["block"] else 0
    if op == "decode":
        return {"bytes": int((coded + size) * M * K), "flops": rot}
    # the matrix, its coded form and the values that it stands for
    return {"bytes": int((size + coded + 2) * M * K), "flops": rot + M * K}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, device=DEV, dtype=torch.float32, generator=g)


def _weights(g, M, K):
    """N(0, 0.02), a few outlier columns."""
    w = _normal(g, M, K) * 0.02
    cols = torch.rand(K, device=DEV, generator=g) < 0.005
    return torch.where(cols, w * 20.0, w)


def _col_scale(g, K):
    """sqrt of the activations' RMS per channel (lognormal)."""
    return torch.exp(0.5 * _normal(g, K))


def prepare(case, seed):
    g = _gen(seed)
    op, K = case["op"], case["K"]
    st = {"case": case}
    if op in ("ce", "ce_grad"):
        T, V = case["T"], case["V"]
        st["X"] = _normal(g, T, K).to(torch.bfloat16)
        st["W"] = (_normal(g, V, K) * 0.02).to(torch.bfloat16)
        t = torch.randint(0, V, (T,), device=DEV, generator=g)
        skip = torch.rand(T, device=DEV, generator=g) < case["ignored"]
        st["targets"] = torch.where(skip, torch.full_like(t, IGNORE), t)
        if op == "ce_grad":
            live = (st["targets"] != IGNORE).to(torch.float32)
            st["g"] = live / live.sum().clamp(min=1.0)
            # the forward pass has run: its normaliser is in hand
            st["lse"] = _plain_ce(st["X"], st["W"], st["targets"])[1]
        return st
    M, block = case["M"], case["block"]
    st["seed"] = int(seed) * 7 + 1
    s = None if case["scale"] == "none" else _col_scale(g, K)
    st["scale"] = s
    if op == "quantize":
        wide = K + case["pad"]
        w = _weights(g, M, wide).to(DTYPES[case["dtype"]])
        st["W"] = w[:, :K]
        return st
    # a coded matrix, as a checkpoint holds it: packed codes and one scale byte per 32 columns
    W = _weights(g, M, K).to(torch.bfloat16)
    codes, scales = _plain_quantize(W, s, False, block, st["seed"])
    st["codes"], st["scales"] = codes, scales
    if op == "linear":
        x = _normal(g, case["T"], K)
        st["X"] = (x if s is None else x * s * s).to(torch.bfloat16)
    if own:
        import vector_codebook_codec_b200 as q
        st["coded"] = q.mx4_from_parts(codes, scales, block=block, seed=st["seed"], col_scale=s)
    return st


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _signs(seed, K):
    """d_j = -1 where bit 63 of SplitMix64's output j + 1 for the seed is set."""
    with np.errstate(over="ignore"):
        z = np.uint64(seed) + np.arange(1, K + 1, dtype=np.uint64) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z = z ^ (z >> np.uint64(31))
    return torch.from_numpy(np.where(z >> np.uint64(63), -1.0, 1.0)).to(DEV)


def _hadamard(block, dtype):
    """Sylvester's matrix, entry (i, j) = (-1)^popcount(i & j), over sqrt(b)."""
    i = np.arange(block)
    odd = np.bitwise_count(i[:, None] & i[None, :]) % 2
    return torch.from_numpy(np.where(odd, -1.0, 1.0) / math.sqrt(block)).to(DEV, dtype)


def _blocks(y, block):
    """H_b y / sqrt(b) for every block of b columns."""
    return (y.reshape(-1, block) @ _hadamard(block, y.dtype)).reshape(y.shape)


def _plain_quantize(W, s, divide, block, seed):
    """Packed e2m1 codes [M, K/2] (the even column in the low half) and e8m0 scales [M, K/32]."""
    M, K = W.shape
    y = W.to(torch.float64)
    if s is not None:
        y = y / s.to(torch.float64) if divide else y * s.to(torch.float64)
    if block:
        y = _blocks(y * _signs(seed, K), block)
    y = y.reshape(M, K // 32, 32)
    amax = y.abs().amax(dim=2, keepdim=True)
    e = torch.frexp(amax)[1].to(torch.int32) - 3          # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    a = torch.ldexp(y.abs(), -e)
    # ties to even: a border belongs to its neighbour with the even code
    borders = torch.tensor(BORDERS, dtype=torch.float64, device=DEV)
    lo = torch.bucketize(a, borders, right=False)
    code = torch.where(lo % 2 == 0, lo, torch.bucketize(a, borders, right=True)).to(torch.uint8)
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).reshape(M, K // 2, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), (e.squeeze(2) + 127).to(torch.uint8)


def _plain_values(codes, scales):
    """The fp32 values that codes and scales stand for."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=torch.float32, device=DEV)
    M, half = codes.shape
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), dim=2).reshape(M, half // 16, 32)
    e = scales.to(torch.int32) - 127
    return torch.ldexp(v, e.unsqueeze(2)).reshape(M, 2 * half)


def _plain_decode(codes, scales, s, block, seed, dtype):
    y = _plain_values(codes, scales)
    if block:
        y = _blocks(y, block) * _signs(seed, y.shape[1]).to(torch.float32)
    if s is not None:
        y = y / s
    return y.to(dtype)


def _plain_ce(X, W, targets):
    """Loss and normaliser of each token."""
    z = X.float() @ W.float().t()
    m = z.amax(dim=1, keepdim=True)
    lse = m.squeeze(1) + torch.log(torch.exp(z - m).sum(dim=1))
    live = targets != IGNORE
    at = z.gather(1, torch.where(live, targets, torch.zeros_like(targets)).unsqueeze(1)).squeeze(1)
    return torch.where(live, lse - at, torch.zeros_like(lse)), lse


def _plain_ce_grad(X, W, targets, lse, g):
    X32, W32 = X.float(), W.float()
    live = targets != IGNORE
    p = torch.exp(X32 @ W32.t() - lse.unsqueeze(1))
    t = torch.where(live, targets, torch.zeros_like(targets)).unsqueeze(1)
    p.scatter_add_(1, t, torch.where(live, -1.0, 0.0).unsqueeze(1).to(torch.float32))
    p *= torch.where(live, g, torch.zeros_like(g)).unsqueeze(1)
    return (p @ W32).to(torch.bfloat16), (p.t() @ X32).to(torch.bfloat16)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import vector_codebook_codec_b200 as q
        if op == "quantize":
            m = q.mx4_quantize(state["W"], block=c["block"], seed=state["seed"], col_scale=state["scale"],
                               divide=c["scale"] == "divide")
            return q.mx4_decode(m, original=False)
        if op == "decode":
            return q.mx4_decode(state["coded"], out_dtype=DTYPES[c["dtype"]])
        if op == "linear":
            return q.mx4_linear(state["coded"], state["X"], out_dtype=DTYPES[c["dtype"]])
        if op == "ce":
            loss, lse = q.cross_entropy(state["X"], state["W"], state["targets"], ignore_index=IGNORE)
            return {"loss": loss, "lse": lse}
        dX, dW = q.cross_entropy_grad(state["X"], state["W"], state["targets"], state["lse"], state["g"],
                                      ignore_index=IGNORE)
        return {"dX": dX, "dW": dW}
    if op == "quantize":
        codes, scales = _plain_quantize(state["W"], state["scale"], c["scale"] == "divide", c["block"],
                                        state["seed"])
        return _plain_values(codes, scales).to(torch.bfloat16)
    if op == "decode":
        return _plain_decode(state["codes"], state["scales"], state["scale"], c["block"], state["seed"],
                             DTYPES[c["dtype"]])
    if op == "linear":
        xc, xs = _plain_quantize(state["X"], state["scale"], True, c["block"], state["seed"])
        return (_plain_values(xc, xs) @ _plain_values(state["codes"], state["scales"]).t()).to(DTYPES[c["dtype"]])
    if op == "ce":
        loss, lse = _plain_ce(state["X"], state["W"], state["targets"])
        return {"loss": loss, "lse": lse}
    dX, dW = _plain_ce_grad(state["X"], state["W"], state["targets"], state["lse"], state["g"])
    return {"dX": dX, "dW": dW}


# --------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------

def _exact_blocks(v, block):
    """The block Hadamard rotation by butterflies (adds and subtracts), in 64 bits."""
    rows, K = v.shape
    h = 1
    while h < block:
        v = v.reshape(rows, K // (2 * h), 2, h)
        v = torch.stack((v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]), dim=2)
        h *= 2
    return v.reshape(rows, K) * (1.0 / math.sqrt(block))


def _exact_quantized(W, s, divide, block, seed):
    """The values of the quantised matrix: each the closest multiple that its group's scale allows."""
    out = []
    rows = max(1, (1 << 23) // W.shape[1])
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=DEV)
    for i in range(0, W.shape[0], rows):
        y = W[i:i + rows].double()
        if s is not None:
            y = y / s.double() if divide else y * s.double()
        if block:
            y = _exact_blocks(y * _signs(seed, y.shape[1]), block)
        y = y.reshape(y.shape[0], -1, 32)
        top = y.abs().amax(dim=2, keepdim=True)
        # the binary exponent from the bits of the double
        e = ((top.view(torch.int64) >> 52) & 0x7FF) - 1023 - 2
        e = e.clamp(-127, 127)
        unit = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=DEV), e.double())
        a = y.abs() / unit
        best = torch.zeros_like(a)
        dist = a.clone()
        for k in range(1, 8):
            dk = (a - grid[k]).abs()
            take = (dk < dist) | ((dk == dist) & (k % 2 == 0))
            best = torch.where(take, grid[k], best)
            dist = torch.where(take, dk, dist)
        out.append((torch.where(y < 0, -best, best) * unit).reshape(y.shape[0], -1))
    return torch.cat(out)


def _exact_values(codes, scales):
    both = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], -1).to(torch.int64)
    mant, ex = both & 1, (both >> 1) & 3
    mag = torch.where(ex == 0, 0.5 * mant.double(), (1.0 + 0.5 * mant.double()) * torch.exp2(ex.double() - 1.0))
    unit = torch.exp2(scales.double() - 127.0).repeat_interleave(32, dim=1)
    return torch.where((both >> 3) == 1, -mag, mag) * unit


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantized(st["W"], st["scale"], case["scale"] == "divide", case["block"], st["seed"])
    if op == "decode":
        y = _exact_values(st["codes"], st["scales"])
        if case["block"]:
            y = _exact_blocks(y, case["block"]) * _signs(st["seed"], y.shape[1])
        return y if st["scale"] is None else y / st["scale"].double()
    if op == "linear":
        x = _exact_quantized(st["X"], st["scale"], True, case["block"], st["seed"])
        return x @ _exact_values(st["codes"], st["scales"]).t()
    X, W, t = st["X"].double(), st["W"].double(), st["targets"]
    live = t != IGNORE
    if op == "ce":
        loss, lse = [], []
        for i in range(0, X.shape[0], 1024):
            z = X[i:i + 1024] @ W.t()
            n = torch.logsumexp(z, dim=1)
            at = z[torch.arange(z.shape[0], device=DEV), t[i:i + 1024].clamp(min=0)]
            loss.append(torch.where(live[i:i + 1024], n - at, torch.zeros_like(n)))
            lse.append(n)
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    lse, g = st["lse"].double(), torch.where(live, st["g"].double(), torch.zeros_like(st["g"].double()))
    dX = torch.zeros_like(X)
    dW = torch.empty_like(W)
    for v in range(0, W.shape[0], 8192):
        Wv = W[v:v + 8192]
        G = torch.exp(X @ Wv.t() - lse[:, None])
        hit = (t[:, None] == torch.arange(v, v + Wv.shape[0], device=DEV)[None, :]) & live[:, None]
        G = (G - hit.double()) * g[:, None]
        dX += G @ Wv
        dW[v:v + 8192] = G.t() @ X
    return {"dX": dX, "dW": dW}
