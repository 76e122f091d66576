"""The soft-assignment operators, as measured: 8-bit points (quantize and
dequantize), scores of points against centroids (the product of two 8-bit
operands with one scale per block of 128), the gradients of those scores, taken
from the 8-bit points kept from the forward pass, and the balance loss of a
soft assignment with the members counted per cluster and its gradient.

``run`` computes them in plain torch operations (``own`` false) or through
the library (``own`` true), on the same inputs.

Layouts, for both sides.  Points (N, D) or (B, N, D); an 8-bit operand is the
pair (data float8_e4m3fn (..., N, D) with rows ceil(D / 16) * 16 bytes apart,
scale float8_e8m0fnu (..., N, ceil(D / 128))) and stands for data * scale, one
scale for each 128 consecutive coordinates of a row.  The scale of a block is the
smallest power of two 2^e with max|x| <= 448 * 2^e, e >= -117; data is
x / 2^e rounded to nearest even.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128
MIN_EXP = -117
# work caps of a drawn case; the listed 1m cases are at or above each of them
MAX_ELEMS = 1 << 28      # N * D of points, N * K of scores
MAX_MACS = 1 << 36       # N * D * K of products


# ------------------------------------------------------------------ cases
def listed():
    return [
        # points of the small fp32 workload kept in 8 bits: a latency-sized call
        dict(name="quantize_16k_f32", op="quantize", B=1, N=16384, D=32, dtype="f32"),
        # the largest in-core workload's points (4M x 128 bf16), kept in 8 bits
        # between a forward and a backward pass
        dict(name="quantize_4m", op="quantize", B=1, N=1 << 22, D=128, dtype="bf16"),
        # one new point against a large codebook (serving: a single token)
        dict(name="scores_one_row", op="scores", B=1, N=1, D=128, K=16384, dtype="f32", bias=True),
        # every point of the 1M workload against its 1024 centroids
        dict(name="scores_1m", op="scores", B=1, N=1 << 20, D=128, K=1024, dtype="bf16", bias=True),
        # ragged sizes: a width that ends inside a block, an odd number of centroids
        dict(name="scores_odd", op="scores", B=1, N=99991, D=200, K=777, dtype="f32", bias=True),
        # the batched vector-quantization workload: one small codebook per instance
        dict(name="scores_batch", op="scores", B=512, N=4096, D=64, K=256, dtype="bf16", bias=False),
        # wide features (a router over hidden states): the product itself bounds it
        dict(name="scores_wide", op="scores", B=1, N=8192, D=4096, K=1024, dtype="bf16", bias=True),
        # gradients of one training step on the 1M workload
        dict(name="grad_1m", op="grad", B=1, N=1 << 20, D=128, K=1024, dtype="bf16"),
        # gradients in fp32 at the small workload's shape
        dict(name="grad_16k_f32", op="grad", B=1, N=16384, D=32, K=64, dtype="f32"),
        # ragged gradients
        dict(name="grad_odd", op="grad", B=1, N=30011, D=200, K=777, dtype="bf16"),
        # balance loss, member counts and gradient over the 1M workload's scores
        dict(name="balance_1m", op="balance", B=1, N=1 << 20, K=1024, T=1, dtype="bf16", masked=False),
        # two picks per point among 64 clusters, a padded batch (some rows off)
        dict(name="balance_16k_pad", op="balance", B=4, N=4099, K=64, T=2, dtype="f32", masked=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One case of the ranges behind the listed ones: from single rows to a
    million, widths from 1 to 4096, 1 to 16384 centroids, batches, both types."""
    op = rng.choice(("quantize", "scores", "grad", "balance"))
    dtype = rng.choice(("bf16", "f32"))
    B = rng.choice((1, 1, 1, _log_int(rng, 2, 64)))
    N = _log_int(rng, 1, 1 << 20)
    case = dict(op=op, B=B, dtype=dtype)
    if op == "quantize":
        D = _log_int(rng, 1, 4096)
        case.update(N=max(1, min(N, MAX_ELEMS // (B * D))), D=D)
        return case
    K = _log_int(rng, 1, 16384)
    N = max(1, min(N, MAX_ELEMS // (B * K)))
    if op == "balance":
        case.update(N=N, K=K, T=rng.choice((1, 1, 2, min(K, rng.randint(1, 8)))), masked=rng.random() < 0.5)
        return case
    D = _log_int(rng, 1, 4096 if op == "scores" else 1024)
    N = max(1, min(N, MAX_MACS // (B * K * D), MAX_ELEMS // (B * D)))
    case.update(N=N, D=D, K=K)
    if op == "scores":
        case["bias"] = rng.random() < 0.5
    return case


# ----------------------------------------------------------------- inputs
def _points(gen, B, N, D, dtype):
    """Points of a Gaussian mixture (centres N(0, 4I), sigma 1)."""
    comps = min(N, 256)
    centres = 2 * torch.randn(B * comps, D, generator=gen, device=DEV)
    label = torch.randint(comps, (B, N), generator=gen, device=DEV)
    label += comps * torch.arange(B, device=DEV)[:, None]
    x = torch.randn(B, N, D, generator=gen, device=DEV)
    for b in range(0, B, 64):
        x[b:b + 64] += centres[label[b:b + 64]]
    return x.to(TYPES[dtype])


def _squeeze(t, B):
    return t[0] if B == 1 else t


def _scores_like(gen, B, N, K, dtype, make):
    """make(chunk of normal scores (B, n, K) float32, its first row) over the rows in chunks,
    so that float32 copies of the whole never exist."""
    out = torch.empty(B, N, K, dtype=TYPES[dtype], device=DEV)
    step = max(1, (1 << 27) // (B * K))
    for i in range(0, N, step):
        n = min(step, N - i)
        out[:, i:i + n] = make(torch.randn(B, n, K, generator=gen, device=DEV), i)
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, B, N = case["op"], case["B"], case["N"]
    st = dict(case=case)
    if op == "quantize":
        st["X"] = _squeeze(_points(gen, B, N, case["D"], case["dtype"]), B)
        return st
    K = case["K"]
    if op == "balance":
        T = case["T"]
        # cluster popularity, from rare to common, under the points' own scores
        pop = torch.randn(B, 1, K, generator=gen, device=DEV)
        S = _scores_like(gen, B, N, K, case["dtype"], lambda s, i: 2 * s + pop)
        idx = torch.empty(B, N, T, dtype=torch.int32, device=DEV)
        step = max(1, (1 << 26) // (B * K))
        for i in range(0, N, step):
            idx[:, i:i + step] = S[:, i:i + step].float().topk(T, dim=-1).indices.int()
        st["valid"] = None
        if case["masked"]:
            # a padded batch: each instance's tail is off, and what stands there is not data
            lens = torch.randint(0, N + 1, (B, 1), generator=gen, device=DEV)
            st["valid"] = torch.arange(N, device=DEV)[None, :] < lens
            S.masked_fill_(~st["valid"][:, :, None], float("nan"))
            st["valid"] = _squeeze(st["valid"], B)
        st["S"] = _squeeze(S, B)
        st["idx"] = _squeeze(idx if T > 1 else idx[:, :, 0].contiguous(), B)
        st["coef"] = torch.full((B,), 0.01, device=DEV)   # the loss's weight in the training loss
        return st
    D = case["D"]
    X = _points(gen, B, N, D, "bf16")
    # centroids: points of the set, moved a little
    pick = torch.randint(N, (B, K), generator=gen, device=DEV)
    C = torch.gather(X.float(), 1, pick[:, :, None].expand(B, K, D)) + 0.1 * torch.randn(
        B, K, D, generator=gen, device=DEV)
    st["X"] = tuple(_squeeze(t, B) for t in _quantize(X))
    st["C"] = tuple(_squeeze(t, B) for t in _quantize(C))
    # logits of -||x - c||^2 / D up to a term of the row: (2 x.c - ||c||^2) / D
    st["alpha"] = 2.0 / D
    if op == "scores":
        st["bias"] = _squeeze(-(C * C).sum(-1) / D, B) if case["bias"] else None
    else:
        hit = torch.randint(K, (B, N, 1), generator=gen, device=DEV)

        def grad_of(s, i):  # softmax cross-entropy's gradient, mean over the points
            p = torch.softmax(2 * s, dim=-1)
            n = p.shape[1]
            p.scatter_add_(-1, hit[:, i:i + n], -torch.ones(B, n, 1, device=DEV))
            return p / N
        st["dS"] = _squeeze(_scores_like(gen, B, N, K, case["dtype"], grad_of), B)
    return st


# ------------------------------------------------------------ plain forms
def _quantize(X):
    """8-bit blocks of X (..., N, D): (data, scale)."""
    D = X.shape[-1]
    nb = -(-D // BLOCK)
    lead = X.shape[:-1]
    # rows in pieces, so that a large X needs no float32 copy of all of it
    flat = X.reshape(-1, D)
    ld = -(-D // 16) * 16
    data = torch.zeros(flat.shape[0], ld, dtype=torch.uint8, device=X.device).view(torch.float8_e4m3fn)
    scale = torch.empty(flat.shape[0], nb, dtype=torch.uint8, device=X.device)
    step = max(1, (1 << 26) // D)
    for i in range(0, flat.shape[0], step):
        x = torch.nn.functional.pad(flat[i:i + step].float(), (0, nb * BLOCK - D)).view(-1, nb, BLOCK)
        amax = x.abs().amax(-1)
        # amax = f * 2^k with f in [0.5, 1), and 448 = 0.875 * 2^9
        f, k = torch.frexp(amax)
        e = torch.where(f <= 0.875, k - 9, k - 8).clamp_min(MIN_EXP)
        e = torch.where(amax == 0, torch.full_like(e, MIN_EXP), e)
        q = torch.ldexp(x, -e[:, :, None]).to(torch.float8_e4m3fn)
        data[i:i + step, :D] = q.view(-1, nb * BLOCK)[:, :D]
        scale[i:i + step] = (e + 127).to(torch.uint8)
    return data.view(*lead, ld)[..., :D], scale.view(torch.float8_e8m0fnu).view(*lead, nb)


def _values(q, dtype=torch.float32):
    """The values an 8-bit operand stands for."""
    data, scale = q
    D = data.shape[-1]
    s = torch.ldexp(torch.ones((), device=DEV), scale.view(torch.uint8).int() - 127)
    return (data.float() * s.repeat_interleave(BLOCK, dim=-1)[..., :D]).to(dtype)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        return _values(_quantize(st["X"]), TYPES[case["dtype"]])
    if op == "scores":
        S = torch.matmul(_values(st["X"]), _values(st["C"]).transpose(-1, -2)) * st["alpha"]
        if st["bias"] is not None:
            S += st["bias"].unsqueeze(-2)
        return S.to(TYPES[case["dtype"]])
    if op == "grad":
        X, C, dS = _values(st["X"]), _values(st["C"]), st["dS"]
        N, K = dS.shape[-2:]
        dX = torch.empty_like(X, dtype=TYPES[case["dtype"]])
        dC = torch.zeros(C.shape, dtype=torch.float64, device=DEV)
        db = torch.zeros(C.shape[:-1], dtype=torch.float64, device=DEV)
        step = max(1, (1 << 28) // (case["B"] * K))  # long sums over the rows: float32 pieces, joined in 64 bits
        for i in range(0, N, step):
            g = dS[..., i:i + step, :].float()
            dX[..., i:i + step, :] = torch.matmul(g, C) * st["alpha"]
            dC += torch.matmul(g.transpose(-1, -2), X[..., i:i + step, :]) * st["alpha"]
            db += g.sum(-2, dtype=torch.float64)
        return dX, dC.float(), db.float()
    S, idx, valid = st["S"], st["idx"], st["valid"]
    B, N, K, T = case["B"], case["N"], case["K"], case["T"]
    S, idx = S.view(B, N, K), idx.view(B, N, T)
    rows = torch.full((B,), N, device=DEV, dtype=torch.float64)
    ok = None
    if valid is not None:
        ok = valid.view(B, N)
        rows = ok.sum(-1).double()
        idx = torch.where(ok[:, :, None], idx, torch.full_like(idx, K))
    slot = idx.long() + (K + 1) * torch.arange(B, device=DEV)[:, None, None]
    counts = torch.bincount(slot.view(-1), minlength=B * (K + 1)).view(B, K + 1)[:, :K].int()
    share = (counts / (rows.clamp_min(1) * T)[:, None]).float()
    dS = torch.empty_like(S)
    sum_r = torch.zeros(B, dtype=torch.float64, device=DEV)
    coef = (st["coef"].double() * K / rows.clamp_min(1)).float()
    step = max(1, (1 << 28) // (B * K))
    for i in range(0, N, step):
        p = torch.softmax(S[:, i:i + step].float(), dim=-1)
        if ok is not None:
            p = torch.where(ok[:, i:i + step, None], p, torch.zeros((), device=DEV))
        r = (p * share[:, None, :]).sum(-1, keepdim=True)
        sum_r += r.sum((1, 2), dtype=torch.float64)
        dS[:, i:i + step] = coef[:, None, None] * p * (share[:, None, :] - r)
    loss = (K * sum_r / rows.clamp_min(1)).float()
    return loss, _squeeze(counts, B), _squeeze(dS, B)


# ------------------------------------------------- through the library
def _own(st):
    import means_clustering_flashassign_b200 as km
    case = st["case"]
    op, dt = case["op"], TYPES[case["dtype"]]
    if op == "quantize":
        return km.dequantize(km.quantize(st["X"]), dt)
    if op == "balance":
        bal = km.balance(st["S"], st["idx"], valid=st["valid"])
        dS = km.balance_grad(st["S"], bal, grad=st["coef"], valid=st["valid"])
        return bal.loss, bal.counts, dS
    X, C = km.Quantized(*st["X"]), km.Quantized(*st["C"])
    if op == "scores":
        return km.scores(X, C, bias=st["bias"], alpha=st["alpha"], dtype=dt)
    return km.scores_grad(st["dS"], X, C, alpha=st["alpha"], dtype=dt)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    """Inputs read once, outputs written once; products at two operations a term."""
    B, N = case["B"], case["N"]
    s = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "quantize":   # read X, write the 8-bit form, read it, write X
        nb = -(-case["D"] // BLOCK)
        return dict(bytes=B * N * (2 * s * case["D"] + 2 * (case["D"] + nb)), flops=4 * B * N * case["D"])
    K = case["K"]
    if case["op"] == "balance":    # forward: S and the picks; backward: S again and dS
        return dict(bytes=B * N * (3 * s * K + 4 * case["T"]) + 4 * B * K, flops=10 * B * N * K)
    D = case["D"]
    nb = -(-D // BLOCK)
    ops = B * (N + K) * (D + nb)
    if case["op"] == "scores":
        return dict(bytes=ops + B * N * K * s + (4 * B * K if case["bias"] else 0), flops=2 * B * N * D * K)
    return dict(bytes=ops + B * N * K * s + B * N * D * s + 4 * B * K * (D + 1), flops=4 * B * N * D * K)


# ------------------------------------------- the definition, in 64 bits
def _exact_scale(amax):
    """2^e, e the smallest integer >= -117 with amax <= 448 * 2^e (float64)."""
    e = torch.floor(torch.log2(amax.clamp_min(2.0 ** -140))) - 10
    for _ in range(4):
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    return torch.exp2(e.clamp_min(MIN_EXP))


def _exact_blocks(x):
    """float64 rows (n, D) rounded to the 8-bit format's values: sign, 3 mantissa
    bits, exponents from 2^-6, multiples of 2^-9 below."""
    out = torch.empty_like(x)
    for j in range(0, x.shape[1], BLOCK):
        b = x[:, j:j + BLOCK]
        s = _exact_scale(b.abs().amax(1, keepdim=True))
        y = b / s
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        out[:, j:j + BLOCK] = torch.round(y / step) * step * s
    return out


def _exact_values(q):
    data, scale = (t.reshape(-1, t.shape[-1]) for t in q)
    v = data.double()
    e = scale.view(torch.uint8).double() - 127
    for j in range(scale.shape[1]):
        v[:, j * BLOCK:(j + 1) * BLOCK] *= torch.exp2(e[:, j:j + 1])
    return v.view(q[0].shape)


def exact(case, seed):
    st = prepare(case, seed)
    op, B, N = case["op"], case["B"], case["N"]
    if op == "quantize":
        X = st["X"].view(-1, case["D"])
        out = torch.empty(X.shape, dtype=torch.float64, device=DEV)
        step = max(1, (1 << 26) // case["D"])
        for i in range(0, X.shape[0], step):
            out[i:i + step] = _exact_blocks(X[i:i + step].double())
        return out.view(st["X"].shape)
    K = case["K"]
    if op == "scores":
        X, C = _exact_values(st["X"]), _exact_values(st["C"])
        S = X @ C.mT
        S *= st["alpha"]
        if st["bias"] is not None:
            S += st["bias"].double()[..., None, :]
        return S
    if op == "grad":
        X, C, dS = _exact_values(st["X"]), _exact_values(st["C"]), st["dS"]
        dX = torch.empty_like(X)
        dC = torch.zeros_like(C)
        db = torch.zeros(C.shape[:-1], dtype=torch.float64, device=DEV)
        step = max(1, (1 << 27) // (B * K))
        for i in range(0, N, step):
            g = dS[..., i:i + step, :].double()
            dX[..., i:i + step, :] = st["alpha"] * (g @ C)
            dC += st["alpha"] * (g.mT @ X[..., i:i + step, :])
            db += g.sum(-2)
        return dX, dC, db
    T = case["T"]
    S, idx = st["S"].view(B, N, K), st["idx"].view(B, N, T).long()
    on = torch.ones(B, N, dtype=torch.bool, device=DEV) if st["valid"] is None else st["valid"].view(B, N)
    loss = torch.zeros(B, dtype=torch.float64, device=DEV)
    counts = torch.zeros(B, K, dtype=torch.int32, device=DEV)
    dS = torch.zeros(B, N, K, dtype=torch.float64, device=DEV)
    for b in range(B):
        m = int(on[b].sum())
        if m == 0:
            continue
        counts[b] = torch.zeros(K, dtype=torch.int32, device=DEV).index_add_(
            0, idx[b][on[b]].reshape(-1), torch.ones(m * T, dtype=torch.int32, device=DEV))
        f = counts[b].double() / (m * T)
        step = max(1, (1 << 27) // K)
        for i in range(0, N, step):
            here = on[b, i:i + step]
            s = torch.where(here[:, None], S[b, i:i + step].double(), 0.0)
            w = torch.exp(s - s.amax(1, keepdim=True))
            w /= w.sum(1, keepdim=True)
            w *= here[:, None]
            r = w @ f
            loss[b] += K * r.sum() / m
            dS[b, i:i + step] = st["coef"][b].double() * K / m * w * (f - r[:, None])
    return loss, _squeeze(counts, B), _squeeze(dS, B)
