"""The soft-assignment operators on the GPU against float64 computations of
their definitions: 8-bit points, scores, gradients of the scores, and the
balance loss with its member counts and gradient.

Tolerances count roundings: half a step relative for each rounding to the
output type (bf16 2^-8, float32 2^-24), and for a sum of n terms accumulated
by the tensor cores in float32, steps of at most 2^-22 of the sum of
magnitudes per accumulation (a bound for any internal alignment that keeps 24
bits), one accumulation per 32 (8-bit) or 16 (bf16) terms.  Products of small
integers are exact and are compared exactly."""

import pytest
import torch

import means_clustering_flashassign_b200 as km

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ACC = 2.0 ** -22


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def lead(B, *shape):
    return (B, *shape) if B > 1 else shape


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def values(q):
    """float64 values of 8-bit points, by arithmetic on the stored bytes."""
    bits = q.data.contiguous().view(torch.uint8).long()
    sign = 1.0 - 2.0 * (bits >> 7)
    ex, man = (bits >> 3) & 15, bits & 7
    v = torch.where(ex > 0, (8 + man).double() * torch.exp2(ex.double() - 10), man.double() * 2.0 ** -9)
    v = torch.where((bits & 127) == 127, torch.full_like(v, float("nan")), v * sign)
    s = q.scale.view(torch.uint8).double()
    s = torch.where(s == 255, torch.full_like(s, float("nan")), torch.exp2(s - 127))
    return v * s.repeat_interleave(128, dim=-1)[..., :v.shape[-1]]


def ref_quantize(X):
    """float64 values of X's 8-bit form, from the definition."""
    out = torch.empty(X.shape, dtype=torch.float64, device=X.device)
    for j in range(0, X.shape[-1], 128):
        b = X[..., j:j + 128].double()
        a = b.abs().amax(-1, keepdim=True)
        e = torch.full_like(a, -117)
        for k in range(-117, 121):
            e = torch.where(a > 448 * 2.0 ** k, torch.full_like(a, k + 1.0), e)
        y = b / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        v = torch.round(y / step) * step * torch.exp2(e)
        out[..., j:j + 128] = torch.where(torch.isfinite(a), v, torch.full_like(v, float("nan")))
    return out


# --------------------------------------------------------------- 8-bit points
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,D", [(1, 1, 1), (1, 5, 8), (1, 33, 16), (1, 1000, 32), (2, 77, 40), (1, 257, 64),
                                   (3, 50, 72), (1, 513, 128), (1, 100, 129), (1, 64, 200), (2, 9, 777), (1, 7, 4096),
                                   (1, 70000, 24)])
def test_quantize_is_the_definition(B, N, D, dtype):
    g = gen(N + D)
    X = randn(g, *lead(B, N, D)) * torch.exp2(torch.randint(-60, 60, lead(B, N, 1), generator=g, device=DEV).float())
    X = X.to(dtype)
    q = km.quantize(X)
    assert q.data.shape == X.shape and q.data.stride(-2) == (D + 15) // 16 * 16
    ref = ref_quantize(X)
    assert torch.equal(values(q), ref)
    for dt in (torch.bfloat16, torch.float32):
        assert torch.equal(km.dequantize(q, dt).double(), ref)


def test_quantize_edges_of_the_scale():
    """Powers of two and 448 times them (exact), the next floats above, zeros,
    the largest and the smallest floats, and ties of the rounding."""
    rows = []
    for v in (1.0, 448.0, 448.00003, 447.99997, 0.0, 3.4e38, 2.0 ** -110, 2.0 ** -126, 1e-45, 2.0 ** -117 * 448):
        r = torch.zeros(128)
        r[3] = v
        r[70] = -v / 3
        r[100] = v * 2.0 ** -9
        rows.append(r)
    tie = torch.zeros(128)
    tie[0] = 448.0
    tie[1:9] = torch.tensor([17.0, 19.0, 21.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, -17.0])
    X = torch.stack(rows + [tie]).to(DEV)
    q = km.quantize(X)
    assert torch.equal(values(q), ref_quantize(X))
    assert values(q)[-1, 1:9].tolist() == [16.0, 20.0, 20.0, 1.0, 1.25, 0.0, 2.0 ** -8, -16.0]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_marks_blocks_that_are_not_finite(bad):
    X = randn(gen(1), 4, 300)
    X[1, 130] = bad
    X[3, 299] = bad
    v = km.dequantize(km.quantize(X), torch.float32)
    nan = torch.zeros(4, 300, dtype=torch.bool, device=DEV)
    nan[1, 128:256] = True
    nan[3, 256:] = True
    assert torch.equal(torch.isnan(v), nan)
    assert torch.equal(torch.where(nan, 0.0, v.double()), torch.where(nan, 0.0, ref_quantize(X)))


def test_quantize_of_no_points():
    q = km.quantize(torch.empty(0, 40, device=DEV))
    assert q.data.shape == (0, 40) and q.scale.shape == (0, 1)
    assert km.dequantize(q).shape == (0, 40)


def test_quantize_misaligned_points():
    buf = randn(gen(2), 100 * 64 + 1, dtype=torch.bfloat16)
    X = buf[1:].view(100, 64)
    assert X.data_ptr() % 16
    assert torch.equal(values(km.quantize(X)), ref_quantize(X))
    out = torch.empty(100 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(100, 64)
    assert torch.equal(km.dequantize(km.quantize(X), out=out).double(), ref_quantize(X))


# --------------------------------------------------------------------- scores
SHAPES = [(1, 1, 128, 16384), (1, 128, 128, 128), (1, 300, 32, 64), (3, 131, 200, 77), (2, 64, 1, 1), (1, 1, 1, 1),
          (1, 257, 640, 129), (1, 500, 4096, 100), (5, 129, 513, 257), (1, 1000, 40, 1000), (1, 20000, 128, 264),
          (40, 70, 64, 256), (1, 33, 2065, 8)]


def int_points(g, B, N, D):
    """Small integers times a power of two per block: exact in 8 bits."""
    nb = (D + 127) // 128
    X = torch.randint(-3, 4, lead(B, N, D), generator=g, device=DEV).float()
    s = torch.exp2(torch.randint(-2, 3, lead(B, N, nb), generator=g, device=DEV).float())
    return X * s.repeat_interleave(128, dim=-1)[..., :D]


@pytest.mark.parametrize("B,N,D,K", SHAPES)
def test_scores_of_small_integers_are_exact(B, N, D, K):
    """Sums below 2^24 of multiples of 2^-4: exact in float32 in any order."""
    g = gen(7 * N + D)
    X, C = int_points(g, B, N, D), int_points(g, B, K, D)
    qx, qc = km.quantize(X), km.quantize(C)
    assert torch.equal(values(qx), X.double()) and torch.equal(values(qc), C.double())
    bias = torch.randint(-5, 6, lead(B, K), generator=g, device=DEV).float()
    S = km.scores(qx, qc, bias=bias, alpha=2.0)
    assert torch.equal(S.double(), 2 * X.double() @ C.double().mT + bias.double()[..., None, :])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,D,K", SHAPES)
def test_scores_against_float64(B, N, D, K, dtype):
    g = gen(N + 3 * D)
    qx, qc = km.quantize(randn(g, *lead(B, N, D)) * 3), km.quantize(randn(g, *lead(B, K, D)))
    bias = randn(g, *lead(B, K))
    alpha = 1.7
    x, c = values(qx), values(qc)
    for bb in (None, bias):
        S = km.scores(qx, qc, bias=bb, alpha=alpha, dtype=dtype)
        assert S.dtype == dtype
        alpha32 = float(torch.tensor(alpha, dtype=torch.float32))
        ref = alpha32 * (x @ c.mT) + (0 if bb is None else bb.double()[..., None, :])
        mag = alpha32 * (x.abs() @ c.abs().mT)
        tol = ACC * (D // 32 + 2) * mag + 2 * HALF[dtype] * ref.abs() + 2.0 ** -24 * mag + 1e-30
        assert ((S.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,D,K", [(1, 40011, 200, 777), (1, 40011, 40, 129), (3, 9000, 128, 300), (2, 15001, 130, 552),
                                     (1, 33000, 16, 1128)])
def test_scores_of_many_points_with_a_short_last_tile(B, N, D, K, dtype):
    """Shares cut by work: every score is written, whatever the last tile holds."""
    g = gen(K)
    X, C = int_points(g, B, N, D), int_points(g, B, K, D)
    S = torch.full(lead(B, N, K), float("nan"), dtype=dtype, device=DEV)
    km.scores(km.quantize(X), km.quantize(C), out=S, dtype=dtype)
    # exact in float32 (as above); bf16 rounds once
    assert torch.equal(S, (X.double() @ C.double().mT).to(dtype))


def test_scores_of_a_block_that_is_not_finite():
    g = gen(5)
    X, C = randn(g, 200, 300), randn(g, 150, 300)
    X[17, 200] = float("nan")
    C[33, 5] = float("inf")
    S = km.scores(km.quantize(X), km.quantize(C))
    nan = torch.zeros(200, 150, dtype=torch.bool, device=DEV)
    nan[17], nan[:, 33] = True, True
    assert torch.equal(torch.isnan(S), nan)


def test_scores_write_only_their_rows():
    """The buffer before and behind S stays as it was, for aligned and odd widths."""
    g = gen(6)
    for K in (64, 77, 130):
        for dtype in (torch.bfloat16, torch.float32):
            N = 150
            buf = torch.full((N + 16, K), 7.0, dtype=dtype, device=DEV)
            S = buf[8:8 + N]
            km.scores(km.quantize(randn(g, N, 48)), km.quantize(randn(g, K, 48)), out=S, dtype=dtype)
            assert (buf[:8] == 7).all() and (buf[8 + N:] == 7).all()
            assert not (S == 7).all()


def test_scores_of_no_points():
    q = km.quantize(torch.empty(0, 40, device=DEV))
    c = km.quantize(torch.ones(5, 40, device=DEV))
    assert km.scores(q, c).shape == (0, 5)


# ------------------------------------------------------------ score gradients
GSHAPES = [(1, 1, 1, 1), (1, 64, 64, 64), (1, 128, 128, 128), (1, 300, 32, 64), (3, 131, 200, 77), (2, 65, 8, 1000),
           (1, 3000, 128, 264), (1, 257, 520, 129), (1, 1, 128, 2048), (1, 5000, 24, 3), (7, 129, 65, 40),
           (1, 1100, 300, 136)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,D,K", GSHAPES)
def test_scores_grad_of_small_integers_is_exact(B, N, D, K, dtype):
    g = gen(11 * N + D)
    X, C = int_points(g, B, N, D), int_points(g, B, K, D)
    dS = torch.randint(-2, 3, lead(B, N, K), generator=g, device=DEV).to(dtype)
    if dtype == torch.float32:
        dS += 2.0 ** -9 * torch.randint(-1, 2, dS.shape, generator=g, device=DEV)
    dX, dC, db = km.scores_grad(dS, km.quantize(X), km.quantize(C), alpha=0.5, dtype=torch.float32)
    d = dS.double()
    assert torch.equal(db.double(), d.sum(-2))
    assert torch.equal(dX.double(), 0.5 * d @ C.double())
    assert torch.equal(dC.double(), 0.5 * d.mT @ X.double())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,D,K", GSHAPES)
def test_scores_grad_against_float64(B, N, D, K, dtype):
    g = gen(13 * N + D)
    qx, qc = km.quantize(randn(g, *lead(B, N, D)) * 3), km.quantize(randn(g, *lead(B, K, D)))
    dS = randn(g, *lead(B, N, K), dtype=dtype) * 1e-3
    x, c, d = values(qx), values(qc), dS.double()
    f32 = torch.float32
    for want in (dtype, f32):
        dX, dC, db = km.scores_grad(dS, qx, qc, alpha=0.25, dtype=want)
        assert dX.dtype == want and dC.dtype == f32 and db.dtype == f32
        # float32 dS: three times the accumulations (one per piece), 2^-24 for what the pieces leave
        n = 3 if dtype == f32 else 1
        for got, ref, mag, terms in (
                (dX, 0.25 * d @ c, 0.25 * d.abs() @ c.abs(), K),
                (dC, 0.25 * d.mT @ x, 0.25 * d.abs().mT @ x.abs(), N)):
            half = HALF[got.dtype]
            tol = (ACC * (n * terms / 16 + 4) + 2.0 ** -24) * mag + 2 * half * ref.abs() + 1e-30
            assert ((got.double() - ref).abs() <= tol).all()
        tol = 2.0 ** -24 * (16 + 4) * d.abs().sum(-2) + 2.0 ** -24 * d.sum(-2).abs() + 1e-30
        assert ((db.double() - d.sum(-2)).abs() <= tol).all()


def test_scores_grad_parts_and_repeats():
    g = gen(3)
    qx, qc = km.quantize(randn(g, 3000, 128)), km.quantize(randn(g, 200, 128))
    dS = randn(g, 3000, 200, dtype=torch.bfloat16)
    dX, dC, db = km.scores_grad(dS, qx, qc)
    a = km.scores_grad(dS, qx, qc, want_dC=False, want_dbias=False)
    b = km.scores_grad(dS, qx, qc, want_dX=False, want_dbias=False)
    c = km.scores_grad(dS, qx, qc, want_dX=False, want_dC=False)
    assert a[1] is None and a[2] is None and b[0] is None and b[2] is None and c[0] is None and c[1] is None
    assert torch.equal(a[0], dX) and torch.equal(b[1], dC) and torch.equal(c[2], db)
    for _ in range(3):
        r = km.scores_grad(dS, qx, qc)
        assert torch.equal(r[0], dX) and torch.equal(r[1], dC) and torch.equal(r[2], db)


def test_scores_grad_of_no_points():
    q = km.quantize(torch.empty(0, 40, device=DEV))
    c = km.quantize(torch.ones(5, 40, device=DEV))
    dX, dC, db = km.scores_grad(torch.empty(0, 5, device=DEV), q, c)
    assert dX.shape == (0, 40) and not dC.any() and not db.any() and dC.shape == (5, 40)


def test_scores_grad_against_differences():
    """Moving one coordinate of a point or centroid by a step of its 8-bit
    value moves sum(dS * S) by the gradient times the step (S is linear in
    each).  Integer data: every number here is exact."""
    g = gen(9)
    X, C = int_points(g, 1, 140, 136), int_points(g, 1, 90, 136)
    dS = torch.randint(-2, 3, (140, 90), generator=g, device=DEV).float()
    dX, dC, db = km.scores_grad(dS, km.quantize(X), km.quantize(C), alpha=0.5)
    bias = torch.zeros(90, device=DEV)

    def f(x, c, b):
        return (dS.double() * km.scores(km.quantize(x), km.quantize(c), bias=b, alpha=0.5).double()).sum()
    f0 = f(X, C, bias)
    for i, d in ((0, 0), (139, 135), (77, 128)):
        X2 = X.clone()
        X2[i, d] = 0.0
        assert f(X2, C, bias) - f0 == dX[i, d].double() * (0.0 - X[i, d].double())
        j = i % 90
        C2 = C.clone()
        C2[j, d] = 0.0
        assert f(X, C2, bias) - f0 == dC[j, d].double() * (0.0 - C[j, d].double())
        b2 = bias.clone()
        b2[j] = 2.0
        assert f(X, C, b2) - f0 == 2 * db[j].double()


# -------------------------------------------------------------------- balance
def ref_balance(S, idx, valid, grad):
    """float64 loss, counts, dS of one instance."""
    N, K = S.shape
    idx = idx.reshape(N, -1).long()
    on = torch.ones(N, dtype=torch.bool, device=DEV) if valid is None else valid.bool()
    M, T = int(on.sum()), idx.shape[1]
    picks = idx[on].reshape(-1)
    picks = picks[(picks >= 0) & (picks < K)]
    counts = torch.bincount(picks, minlength=K)[:K].int()
    p = torch.zeros(N, K, dtype=torch.float64, device=DEV)
    s = S[on].double()
    if s.numel():
        m = s.amax(1, keepdim=True)
        w = torch.exp(s - torch.where(m == -float("inf"), torch.zeros_like(m), m))
        tot = w.sum(1, keepdim=True)
        p[on] = torch.where(tot == 0, torch.zeros_like(w), w / tot)
    f = counts.double() / max(M * T, 1)
    r = p @ f
    loss = K * r.sum() / max(M, 1)
    return loss, counts, grad * K / max(M, 1) * p, f, r


def check_balance(S, idx, valid=None, grad=None):
    bal = km.balance(S, idx, valid=valid)
    dS = km.balance_grad(S, bal, grad=grad, valid=valid)
    assert dS.dtype == S.dtype and dS.shape == S.shape
    B = S.shape[0] if S.dim() == 3 else 1
    for b in range(B):
        def one(t):
            return t[b] if t is not None and S.dim() == 3 else t
        gr = 1.0 if grad is None else float(grad[b])
        s = one(S)
        K = s.shape[1]
        loss, counts, cp, f, r = ref_balance(s, one(idx), one(valid), gr)
        d = cp * (f - r[:, None])
        assert torch.equal(one(bal.counts), counts)
        M = int(one(valid).sum()) if valid is not None else s.shape[0]
        assert int(bal.rows[b]) == M
        # p = exp(s - lse): lse and the difference are rounded to half a step of their size (terms
        # with |s - lse| above 30 vanish beside the largest), expf and logf are within 2 steps; the
        # row sums of K float32 terms add at most K / 32 + 5 + 8 steps to numerator and denominator
        top = s.double().amax(1)
        top = top[torch.isfinite(top)].abs().max().item() if torch.isfinite(top).any() else 0.0
        rel = (top + 8 + 30 + 8 + 2 * (K / 32 + 13)) * 2.0 ** -24
        # the loss is the mean of 1 + r, r = sum p u, u = K f - 1: r's magnitudes sum to at most loss + 1
        assert (bal.loss[b].double() - loss).abs() <= (rel + 2.0 ** -22) * (loss + 1)
        # d = (cp / K) * (u - r'), u = K f - 1 and r' = sum p u: cp is known to rel, u to 2 half steps of
        # K f + 1, r' to rel of its magnitudes, at most K r + 1; their difference keeps the absolute
        # errors of both (also where it is exactly 0), the product rounds to the type
        tol = (HALF[S.dtype] + rel + 2.0 ** -22) * d.abs() \
            + cp.abs() * (f + r[:, None] + 2.0 / K) * (rel + 2.0 ** -22) + 1e-37
        assert ((one(dS).double() - d).abs() <= tol).all()
    return bal, dS


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,K,T", [(1, 1, 1, 1), (1, 7, 3, 1), (1, 1000, 64, 2), (2, 333, 77, 1), (1, 50, 1024, 8),
                                     (3, 129, 256, 1), (1, 20000, 128, 1), (1, 9, 10007, 3), (1, 5, 20000, 1),
                                     (64, 4, 16, 1), (1, 4097, 8, 2), (1, 300, 2500, 1), (1, 700, 33, 4)])
def test_balance_against_float64(B, N, K, T, dtype):
    g = gen(N + K)
    S = (randn(g, *lead(B, N, K)) * 3).to(dtype)
    idx = torch.randint(0, K, lead(B, N, T) if T > 1 else lead(B, N), generator=g, device=DEV, dtype=torch.int32)
    check_balance(S, idx)
    valid = torch.rand(lead(B, N), generator=g, device=DEV) < 0.6
    grad = randn(g, B)
    S2 = torch.where(valid[..., None], S, torch.full_like(S, float("nan")))   # what is off is not looked at
    idx2 = torch.where((valid if T == 1 else valid[..., None]), idx, torch.full_like(idx, 1 << 30))
    check_balance(S2, idx2, valid, grad)


def test_balance_of_even_picks_has_no_gradient():
    """Every cluster picked as often as every other: u is exactly 0, and so is the
    gradient; the loss is 1."""
    g = gen(29)
    for K, T in ((3, 3), (8, 1), (77, 7), (64, 2)):
        N = 11 * K
        idx = (torch.arange(N * T, device=DEV) % K).int().view(N, T)
        S = randn(g, N, K) * 3
        bal = km.balance(S, idx)
        assert (bal.counts == 11 * T).all() and not km.balance_grad(S, bal).any() and not bal.dot.any() and bal.loss == 1


def test_balance_masks():
    """Columns of -inf, of the type's lowest value, rows of nothing but -inf,
    picks that are none, no valid point."""
    g = gen(4)
    for dtype in (torch.bfloat16, torch.float32):
        for K in (16, 77, 600):
            S = (randn(g, 90, K) * 2).to(dtype)
            S[:, 1::3] = -float("inf")
            S[5] = -float("inf")
            S[7, :] = -float("inf")
            S[7, K - 1] = 3.0
            S[8, :-1] = torch.finfo(dtype).min
            idx = torch.randint(-2, K + 2, (90, 2), generator=g, device=DEV, dtype=torch.int32)
            bal, dS = check_balance(S, idx)
            assert not dS[5].any() and bal.dot[5] == 0 and bal.lse[5] == -float("inf")
            off = torch.zeros(90, dtype=torch.uint8, device=DEV)
            bal, dS = check_balance(S, idx, off)
            assert not dS.any() and bal.loss == 0 and not bal.counts.any() and bal.rows == 0


def test_balance_of_a_row_that_is_not_a_number():
    S = randn(gen(8), 40, 50)
    idx = torch.zeros(40, dtype=torch.int32, device=DEV)
    for bad in (float("nan"), float("inf")):
        S2 = S.clone()
        S2[13, 20] = bad
        bal = km.balance(S2, idx)
        dS = km.balance_grad(S2, bal)
        assert torch.isnan(bal.loss).all()
        assert torch.isnan(dS[13]).any() and torch.isfinite(dS[:13]).all() and torch.isfinite(dS[14:]).all()


def test_balance_of_no_points():
    bal = km.balance(torch.empty(0, 5, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV))
    assert bal.loss == 0 and not bal.counts.any() and bal.rows == 0
    assert km.balance_grad(torch.empty(0, 5, device=DEV), bal).shape == (0, 5)


def test_balance_gradient_against_differences():
    """Central differences of the float64 loss (counts fixed) with step h =
    2^-10: their own error is h^2 / 6 of a third derivative, itself at most
    K / M * f <= K / M here."""
    g = gen(12)
    N, K, h = 20, 12, 2.0 ** -10
    S = randn(g, N, K)
    idx = torch.randint(0, K, (N,), generator=g, device=DEV, dtype=torch.int32)
    bal = km.balance(S, idx)
    dS = km.balance_grad(S, bal)
    for i in range(0, N, 7):
        for k in range(K):
            lo, hi = S.double(), S.double()
            lo[i, k] -= h
            hi[i, k] += h
            d = (ref_balance(hi, idx, None, 1.0)[0] - ref_balance(lo, idx, None, 1.0)[0]) / (2 * h)
            assert abs(float(dS[i, k]) - float(d)) <= K / N * h * h + 1e-6 * K / N


def test_balance_repeats_bit_for_bit():
    g = gen(2)
    S = randn(g, 50000, 100, dtype=torch.bfloat16)
    idx = torch.randint(0, 100, (50000, 3), generator=g, device=DEV, dtype=torch.int32)
    a = km.balance(S, idx)
    da = km.balance_grad(S, a)
    for _ in range(3):
        b = km.balance(S, idx)
        assert all(torch.equal(x, y) for x, y in zip(a[:5], b[:5]))
        assert torch.equal(km.balance_grad(S, b), da)


# ---------------------------------------------------------------- as a whole
def train_step(X, C, t):
    """Forward and backward of a balance-regularised soft assignment."""
    qx, qc = km.quantize(X), km.quantize(C)
    bias = -(C * C).sum(-1) / t
    S = km.scores(qx, qc, bias=bias, alpha=2.0 / t, dtype=torch.bfloat16)
    idx, _, _ = km.assign(X, C.to(X.dtype), want_mindist=False, want_objective=False)
    bal = km.balance(S, idx)
    dS = km.balance_grad(S, bal)
    dX, dC, db = km.scores_grad(dS, qx, qc, alpha=2.0 / t)
    return bal.loss, bal.counts, dX, dC, db


def test_the_run_of_them_together():
    g = gen(21)
    X = randn(g, 5000, 128, dtype=torch.bfloat16)
    C = X[:200].float() + 0.1 * randn(g, 200, 128)
    loss, counts, dX, dC, db = train_step(X, C, 64.0)
    idx, _, _ = km.assign(X, C.to(X.dtype))
    _, fit_counts = km.update(X, idx, C.clone())
    assert torch.equal(counts, fit_counts)      # the members the centroid update counts
    xd, cd = values(km.quantize(X)).requires_grad_(), values(km.quantize(C)).requires_grad_()
    bias = (-(C * C).sum(-1) / 64.0).double().requires_grad_()
    S = 2.0 / 64 * (xd @ cd.T) + bias
    f = counts.double() / 5000
    ref = 200 * (torch.softmax(S, -1) @ f).mean()
    ref.backward()
    # S and dS are rounded to bf16 (2^-8 each): S of size up to a few makes exp err by |S| 2^-8
    smax = float(S.detach().abs().max())
    rel = 2 * (smax + 1) * 2.0 ** -8
    ref = float(ref.detach())
    assert abs(float(loss) - ref) <= rel * ref
    for got, want in ((dX, xd.grad), (dC, cd.grad), (db, bias.grad)):
        err = (got.double() - want).norm() / want.norm()
        assert err <= 2 * rel


def test_together_in_a_graph_and_on_another_stream():
    g = gen(22)
    X = randn(g, 3000, 64, dtype=torch.bfloat16)
    C = X[:96].float().contiguous()
    ref = train_step(X, C, 32.0)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = train_step(X, C, 32.0)
    other.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    Xs = X.clone()
    with torch.cuda.graph(graph):
        out = train_step(Xs, C, 32.0)
    for seed in (30, 31):
        Xs.copy_(randn(gen(seed), 3000, 64, dtype=torch.bfloat16))
        graph.replay()
        want = train_step(Xs, C, 32.0)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_stream_argument_and_two_calls_at_once():
    g = gen(23)
    qx, qc = km.quantize(randn(g, 40000, 128)), km.quantize(randn(g, 500, 128))
    ref = km.scores(qx, qc)
    dS = randn(g, 40000, 500, dtype=torch.bfloat16)
    rg = km.scores_grad(dS, qx, qc)
    idx = torch.randint(0, 500, (40000,), generator=g, device=DEV, dtype=torch.int32)
    rb = km.balance(ref, idx)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(3):
        for s in (s1, s2):
            outs.append((km.scores(qx, qc, stream=s), km.scores_grad(dS, qx, qc, stream=s),
                         km.balance(ref, idx, stream=s)))
    torch.cuda.synchronize()
    for a, b, c in outs:
        assert torch.equal(a, ref)
        assert all(torch.equal(x, y) for x, y in zip(b, rg))
        assert all(torch.equal(x, y) for x, y in zip(c[:5], rb[:5]))


def test_workspaces_report_no_timeout():
    g = gen(24)
    qx, qc = km.quantize(randn(g, 1000, 200)), km.quantize(randn(g, 300, 200))
    ws = torch.empty(km.soft_workspace_size(km.SOFT_SCORES_GRAD, 1, 1000, 200, 300, km.BF16), dtype=torch.uint8,
                     device=DEV)
    km.scores(qx, qc, workspace=ws)
    assert km.workspace_status(ws) == 0
    km.scores_grad(randn(g, 1000, 300, dtype=torch.bfloat16), qx, qc, workspace=ws)
    assert km.workspace_status(ws) == 0
    for n in (1000, 50000):   # both ways of counting
        ws.fill_(255)
        km.balance(randn(g, n, 30), torch.zeros(n, dtype=torch.int32, device=DEV), workspace=ws)
        assert km.workspace_status(ws) == 0


def test_bytes_behind_the_rows_do_not_matter():
    g = gen(26)
    for D in (40, 129, 200):
        X, C = randn(g, 300, D), randn(g, 70, D)
        qx, qc = km.quantize(X), km.quantize(C)
        ld = (D + 15) // 16 * 16
        dS = randn(g, 300, 70, dtype=torch.bfloat16)
        ref = (km.scores(qx, qc), *km.scores_grad(dS, qx, qc), km.dequantize(qx))

        def dirty(q):
            data = torch.full((q.data.shape[0], ld), 0x7f, dtype=torch.uint8, device=DEV)   # NaN bytes
            data[:, :D] = q.data.view(torch.uint8)
            return km.Quantized(data.view(torch.float8_e4m3fn)[:, :D], q.scale)
        got = (km.scores(dirty(qx), dirty(qc)), *km.scores_grad(dS, dirty(qx), dirty(qc)), km.dequantize(dirty(qx)))
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_gradients_of_blocks_that_are_not_finite():
    """A point's NaN block reaches dC's columns of that block, a centroid's NaN
    block dX's; nothing else."""
    g = gen(27)
    X, C = randn(g, 300, 300), randn(g, 90, 300)
    X[7, 130] = float("inf")
    C[5, 299] = float("nan")
    dX, dC, db = km.scores_grad(randn(g, 300, 90), km.quantize(X), km.quantize(C))
    assert torch.isnan(dC[:, 128:256]).all() and torch.isfinite(dC[:, :128]).all() and torch.isfinite(dC[:, 256:]).all()
    assert torch.isnan(dX[:, 256:]).all() and torch.isfinite(dX[:, :256]).all()
    assert torch.isfinite(db).all()


@pytest.mark.parametrize("N,D,K,dtype", [(40000, 64, 300, torch.bfloat16), (9000, 32, 5000, torch.float32),
                                         (2000, 24, 40000, torch.float32), (300000, 16, 8, torch.float32)])
def test_long_sums_keep_their_precision(N, D, K, dtype):
    """Sums over many points and many centroids: chains of at most 32 MMAs, each losing at most 2^-23 of its magnitudes, joined by
    rounded adds of which there are at most sqrt(terms / 512) + 40 in effect
    (rounding errors of either sign); the error of the whole result, in norms,
    against the size of its terms."""
    g = gen(N)
    X, C = randn(g, N, D) + 1.0, randn(g, K, D) - 1.0
    qx, qc = km.quantize(X), km.quantize(C)
    dS = (torch.rand(N, K, generator=g, device=DEV) * 1e-4).to(dtype)   # all of one sign: no cancellation to hide behind
    dX, dC, _ = km.scores_grad(dS, qx, qc, dtype=torch.float32)
    x, c, d = values(qx), values(qc), dS.double()
    for got, ref, terms in ((dX, d @ c, K), (dC, d.mT @ x, N)):
        chain = min(32, terms // 16 * (3 if dtype == torch.float32 else 1) + 1)
        tol = (chain * 2.0 ** -23 + ((terms / 512) ** 0.5 + 40) * 2.0 ** -24)
        assert (got.double() - ref).norm() <= tol * ref.norm()


@pytest.mark.parametrize("call,spec", [("quantize", "launch"), ("scores", "launch"), ("grad", "launch"),
                                       ("grad", "launch:3"), ("balance", "launch:2"), ("balance_grad", "launch")])
def test_injected_launch_failures(call, spec, monkeypatch):
    g = gen(25)
    X = randn(g, 700, 72)
    qx, qc = km.quantize(X), km.quantize(randn(g, 40, 72))
    S = km.scores(qx, qc)
    idx = torch.zeros(700, dtype=torch.int32, device=DEV)
    bal = km.balance(S, idx)
    fns = {"quantize": lambda: km.quantize(X), "scores": lambda: km.scores(qx, qc),
           "grad": lambda: km.scores_grad(S, qx, qc), "balance": lambda: km.balance(S, idx),
           "balance_grad": lambda: km.balance_grad(S, bal)}
    monkeypatch.setenv("KM_FAULT", spec)
    with pytest.raises(km.KMError) as e:
        fns[call]()
    assert e.value.status == 6
    monkeypatch.delenv("KM_FAULT")
    fns[call]()
    torch.cuda.synchronize()


def test_every_8_bit_value_under_every_kind_of_scale():
    """All 256 bytes (NaN among them) under the scales 2^-127, 2^-117, 1, 2^7, 2^8,
    2^120, 2^127 and NaN: what dequantize gives, and what the gradients multiply
    by (dS = 1 at one centroid or point each)."""
    scales = torch.tensor([0, 10, 127, 134, 135, 247, 254, 255], dtype=torch.uint8, device=DEV)
    data = torch.arange(256, dtype=torch.uint8, device=DEV).view(2, 128).repeat(8, 1).view(torch.float8_e4m3fn)
    q = km.Quantized(data, scales.repeat_interleave(2)[:, None].contiguous().view(torch.float8_e8m0fnu))
    v = values(q)

    def same(got, dtype):
        # one rounding to the type, which some scales need (an overflow rounds to infinity)
        want = v.to(torch.float32).to(dtype)
        return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    big = scales.repeat_interleave(2) == 0   # products below 2^-126 may leave bf16's or the MMA's range
    assert same(km.dequantize(q, torch.float32), torch.float32)
    got = km.dequantize(q, torch.bfloat16)
    keep = ~big
    assert torch.equal(got[keep].nan_to_num(7.0), v.float().bfloat16()[keep].nan_to_num(7.0))
    eye = torch.eye(16, dtype=torch.bfloat16, device=DEV)
    finite = (scales.repeat_interleave(2) > 0) & (scales.repeat_interleave(2) < 247)
    f = km.Quantized(q.data[finite].contiguous(), q.scale[finite].contiguous())
    n = int(finite.sum())
    w = values(f)
    nan = torch.isnan(w)
    one = km.quantize(torch.ones(n, 128, device=DEV))
    dX, _, _ = km.scores_grad(eye[:n, :n].contiguous(), one, f, dtype=torch.float32)
    _, dC, _ = km.scores_grad(eye[:n, :n].contiguous(), f, one, dtype=torch.float32)
    # a NaN in a column of the operand reaches every row of it through 0 * NaN
    col = nan.any(0)
    for got in (dX, dC):
        assert torch.isnan(got[:, col]).all()
        assert torch.equal(got[:, ~col].double(), w[:, ~col])


def test_scores_captured_first_and_called_after():
    """The status word that calls without a workspace share is not a graph's memory."""
    saved = dict(km._status_words)
    km._status_words.clear()
    g = gen(28)
    qx, qc = km.quantize(randn(g, 500, 64)), km.quantize(randn(g, 60, 64))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = km.scores(qx, qc)
    assert not km._status_words
    graph.replay()
    ref = km.scores(qx, qc)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and len(km._status_words) == 1
    del graph, out
    assert torch.equal(km.scores(qx, qc), ref)
    km._status_words.update(saved)
