"""The soft-assignment operators over the whole range of their inputs, against
float64 computations of their definitions: scores far from 0 and masked to
finite values.

Tolerances count roundings in units of 2^-24 (U), half a float32 step of
relative error; every one is derived beside its use, row by row."""

import pytest
import torch

import means_clustering_flashassign_b200 as km

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# ---------------------------------------------- balance far from 0 and masked
FINE = 16.0   # |logsumexp| up to which one float32 of it is enough


def far_rows(g, K, dtype):
    """Rows of scores as callers have them: with an offset of either sign that
    the softmax does not see, and rows that a finite mask fills, whole or in
    part; rows near 0 between them (threads of one warp then differ)."""
    base = torch.randn(40, K, generator=g, device=DEV)
    off = torch.tensor([0, 1e3, 0, -1e4, 20, -20, 1e4, 1e6, 0, -1e6], device=DEV).repeat(4)[:, None]
    S = (base + off).to(dtype)
    low = torch.finfo(dtype).min
    S[20], S[21], S[22], S[23], S[24] = low, -1e9, 1e8, -1e4, -1e30
    S[25] = torch.where(torch.arange(K, device=DEV) % 3 == 1, -float("inf"), low)
    S[26] = torch.where(torch.arange(K, device=DEV) % 3 == 1, -float("inf"), -1e9)
    S[27] = -float("inf")
    S[28, 1:] = low            # one ordinary score
    S[29] = torch.finfo(dtype).max
    S[30] = -1e9
    S[30, K // 2:] = -2e9
    return S


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [3, 8, 16, 77, 256, 300, 1024, 1500, 1504, 4101, 5000, 8192, 20000])
def test_balance_gradient_of_rows_far_from_zero(K, dtype):
    """Every form of the rows: 1 to 256 threads a row, 16-byte and single loads,
    and the wide one."""
    g = gen(K)
    S = far_rows(g, K, dtype)
    N = S.shape[0]
    valid = torch.ones(N, dtype=torch.bool, device=DEV)
    valid[[4, 30, 39]] = False
    Sv = torch.where(valid[:, None], S, torch.full_like(S, float("nan")))
    idx = torch.randint(0, K, (N, 2), generator=g, device=DEV, dtype=torch.int32)
    grad = torch.tensor([0.7], device=DEV)
    bal = km.balance(Sv, idx, valid=valid)
    dS = km.balance_grad(Sv, bal, grad=grad, valid=valid)
    assert not dS[~valid].any() and not dS[27].any()

    M = int(valid.sum())
    counts = torch.bincount(idx[valid].view(-1).long(), minlength=K)
    assert torch.equal(bal.counts.long(), counts)
    s = S.double()
    m = s.amax(1, keepdim=True).clamp_min(-1e300)        # (the row of -inf)
    w = torch.exp(s - m)
    tot = w.sum(1, keepdim=True)
    p = torch.where(tot > 0, w / tot.clamp_min(1e-300), torch.zeros_like(w))
    u = K * counts.double() / (2 * M) - 1
    r = (p * u).sum(1, keepdim=True)
    coef = float(grad) / M
    ref = coef * p * (u - r) * valid[:, None]
    # d = s - logsumexp: float32 rounds the difference and its product with log2 e, whose
    # constant is rounded too (3 |d|), ex2 is off by 4; the row's sum takes K / 32 + 13 adds of terms
    # off by that (the mean of |d| under p); what one float32 leaves of the logsumexp shifts d by
    # at most half a step of it, and not by more than log K
    lse = torch.where(tot > 0, m + torch.log(tot.clamp_min(1e-300)), torch.zeros_like(m))
    d = (s - lse).abs().clamp_max(200)                   # (p is 0 in float32 from 104 on)
    left = (lse.abs() * U).clamp_max(torch.log(torch.tensor(float(K))).item() + 0.1)
    mean = (p * (d + left)).sum(1, keepdim=True)
    rel = 3 * (d + left) + 4 + K / 32 + 13 + 3 * mean + 4 + 3 * left + 2
    # rows near 0 take p = exp(s - lse): its rounding (8 half units of 2^-24 at 16) and logf's (a step of at most 16)
    rel = (rel + torch.where(lse.abs() <= FINE + 1e-3, 8.0 + 16.0, 0.0)) * U
    assert float(rel[d < 20].max()) <= (3 * 20 + 35 + 24 + 16 * 3 * 11 + K / 32 + 40) * U   # no tolerance grows with the scores
    err_r = (p * u.abs() * (rel + (K / 32 + 13) * U)).sum(1, keepdim=True) + 4 * U * r.abs()
    tol = HALF[dtype] * ref.abs() + coef * p * ((u - r).abs() * (rel + 6 * U) + 4 * U * u.abs() + err_r + 4 * U * r.abs()) + 1e-37
    err = (dS.double() - ref).abs()
    assert (err <= tol).all(), (err - tol).max(1).values.argmax()
    # the loss's own gradient: every row's sums to 0, and the loss itself is the same rows'
    want = ((p.sum(1) + r[:, 0])[valid]).sum() / M
    assert (bal.loss[0].double() - want).abs() <= (err_r[valid].sum() / M + 2 ** -20 * (want.abs() + 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [8, 77, 300, 1024, 1504, 4101, 8192, 20000])
def test_balance_gradient_of_many_rows_far_from_zero(K, dtype):
    """The same 40 rows 60 times over, each time the same gradient bit for bit,
    whichever threads take them and whatever rows they took before."""
    g = gen(K + 1)
    S = far_rows(g, K, dtype).repeat(60, 1)
    idx = torch.randint(0, K, (S.shape[0],), generator=g, device=DEV, dtype=torch.int32)
    bal = km.balance(S, idx)
    dS = km.balance_grad(S, bal).view(60, 40, K)
    assert torch.isfinite(dS).all() and (dS[0, 20] != 0).any()
    assert torch.equal(dS, dS[:1].expand(60, 40, K).contiguous())
    # a row's gradient sums to 0: p is off by (K / 32 + 250) U at most (above: |d| of the probable
    # clusters below 40) and r by as much of its terms; where one cluster has all of the row, u - r
    # cancels and leaves the rounding of both, of size up to 32 here, over M
    if dtype == torch.float32:
        scale = dS.double().abs().sum(-1)
        assert (dS.double().sum(-1).abs() <= scale * (K / 32 + 250) * 2 * U + 2.0 ** -18 / S.shape[0]).all()


# ------------------------------------------------- float32 dS as bf16 pieces
def signs(g, *shape):
    """+-2^-10: exact in 8 bits, products with them exact."""
    return (torch.randint(0, 2, shape, generator=g, device=DEV) * 2 - 1).float() * 2.0 ** -10


@pytest.mark.parametrize("N,D,K", [(300, 64, 90), (257, 130, 64), (70, 16, 33)])
@pytest.mark.parametrize("v", [3.4e38, -3.4e38, torch.finfo(torch.float32).max, 3.3961775e38, 3.3961773e38,
                               float("inf"), -float("inf"), float("nan")])
def test_gradients_of_the_largest_floats_and_of_infinities(N, D, K, v):
    """One such entry of dS: its row of dX, its row of dC and its dbias are its
    products (exact: powers of two), every other sum is as without it."""
    g = gen(K)
    X, C = signs(g, N, D), signs(g, K, D)
    dS = torch.zeros(N, K, device=DEV)
    i, k = N - 2, K - 3
    dS[i, k] = v
    dS[i, 0] = dS[0, k] = 3.0
    dS[1, 1] = 2.0 ** -100
    dX, dC, db = km.scores_grad(dS, km.quantize(X), km.quantize(C))
    d = dS.double()
    for got, ref in ((dX, d @ C.double()), (dC, d.mT @ X.double()), (db, d.sum(0))):
        # 3 beside 3.4e38 vanishes in float32, in the reference's rounding too
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(got.nan_to_num(nan=0.0, posinf=1.0, neginf=-1.0), ref.float().nan_to_num(nan=0.0, posinf=1.0, neginf=-1.0))
        assert torch.equal(torch.isinf(got), torch.isinf(ref.float()))


def test_an_infinity_times_zero_is_not_a_number():
    X, C = torch.ones(9, 32, device=DEV), torch.ones(20, 32, device=DEV)
    C[4, 7], X[2, 3] = 0.0, 0.0
    dS = torch.zeros(9, 20, device=DEV)
    dS[2, 4] = float("inf")
    dX, dC, db = km.scores_grad(dS, km.quantize(X), km.quantize(C))
    assert torch.isnan(dX[2, 7]) and torch.isnan(dC[4, 3]) and db[4] == float("inf")
    dX[2, 7], dC[4, 3] = float("inf"), float("inf")
    assert (dX[2] == float("inf")).all() and (dC[4] == float("inf")).all()
    dX[2], dC[4] = 0.0, 0.0
    assert not dX.any() and not dC.any()


# ---------------------------------------------------- a bf16 dX of many terms
@pytest.mark.parametrize("B,N,D,K,dtype", [
    (1, 70, 136, 1 << 20, torch.bfloat16), (1, 70, 40, 1 << 20, torch.float32), (1, 300, 64, 32768, torch.bfloat16),
    (1, 300, 65, 32769, torch.bfloat16), (2, 257, 8, 40001, torch.bfloat16), (1, 600, 130, 10880, torch.float32),
    (3, 100, 24, 10881, torch.float32), (1, 1, 5, 70000, torch.float32), (1, 4000, 130, 33000, torch.bfloat16)])
def test_bf16_gradient_of_many_terms(B, N, D, K, dtype):
    """Terms of one sign, so that what the tensor core cuts off adds up: at most
    2048 MMAs in one float32 chain, each losing up to 2^-23 of the sum, then one
    rounding to bf16 (2^-8 at most, of either sign: the mean over all elements
    falls with their number)."""
    g = gen(K + N)
    shape = (B,) if B > 1 else ()
    qx = km.quantize(torch.rand(*shape, N, D, generator=g, device=DEV))
    qc = km.quantize(torch.rand(*shape, K, D, generator=g, device=DEV) + 0.5)
    dS = torch.rand(*shape, N, K, generator=g, device=DEV).to(dtype)
    dX, dC, db = km.scores_grad(dS, qx, qc, dtype=torch.bfloat16, alpha=0.5)
    assert dX.dtype == torch.bfloat16
    c, x = km.dequantize(qc, torch.float32).double(), km.dequantize(qx, torch.float32).double()
    ref = 0.5 * (dS.double() @ c)
    err = (dX.double() - ref) / ref
    assert err.abs().max() <= 2.0 ** -8 + 2048 * 2.0 ** -23
    assert err.mean().abs() <= 2048 * 2.0 ** -23 + 4 * 2.0 ** -8 / err.numel() ** 0.5
    # alone, and beside no dC, the same bits; dC and dbias as ever
    assert torch.equal(km.scores_grad(dS, qx, qc, dtype=torch.bfloat16, alpha=0.5, want_dC=False, want_dbias=False)[0], dX)
    assert ((dC.double() - 0.5 * dS.double().mT @ x).norm() <= 1e-5 * dC.double().norm())
    assert (db.double() - dS.double().sum(-2)).norm() <= 1e-6 * db.double().norm()


# -------------------------------------------------- counts above float32's 24 bits
@pytest.mark.parametrize("K,T,count", [(3, 3, (1 << 24) + 1), (77, 1, (1 << 24) + 3), (5000, 128, 386544), (10007, 1024, 174080),
                                       (2500, 8, 800002)])
def test_balance_of_even_picks_in_any_number(K, T, count):
    """Counts as a long accumulation leaves them, given to the gradient: even ones
    give exactly 0, and one more pick than that is seen (u to 3 roundings)."""
    g = gen(K)
    S = torch.randn(6, K, generator=g, device=DEV)
    M = K * count // T
    assert M * T == K * count < 1 << 31
    bal = km.balance(S, torch.zeros(6, dtype=torch.int32, device=DEV))
    even = bal._replace(counts=torch.full((K,), count, dtype=torch.int32, device=DEV), picks=T,
                        rows=torch.tensor([M], dtype=torch.int32, device=DEV), dot=torch.zeros(6, device=DEV))
    dS = km.balance_grad(S, even)
    assert not dS.any()
    p = torch.softmax(S.double(), 1)
    one = even._replace(counts=even.counts.clone())
    one.counts[1] += 1
    u = torch.zeros(K, dtype=torch.float64, device=DEV)
    u[1] = K / (M * T)
    ref = p * u / M
    # p: |logsumexp| and |d| below 16, K / 32 + 13 adds of the row's sum (above); u and the products 8
    tol = ref.abs() * (3 * 16 + 24 + 2 * (K / 32 + 13) + 3 * 16 + 12) * U + 1e-37
    assert ((km.balance_grad(S, one).double() - ref).abs() <= tol).all()


# ------------------------------------------------------- scores of long points
@pytest.mark.parametrize("N,D,K", [(300, 65536, 200), (130, 65536, 77), (33, 8192, 129), (257, 4097, 64), (1, 20000, 5), (150, 12289, 131)])
def test_scores_of_long_points(N, D, K):
    """Terms of one sign: a chain of at most 128 MMAs, each cutting off up to 2^-23
    of a sum that grows evenly (64 of them in effect), the D / 4096 chains added
    with half a step each, and the result's two roundings."""
    g = gen(D + K)
    qx, qc = (km.quantize(torch.rand(n, D, generator=g, device=DEV) + 0.1) for n in (N, K))
    x, c = (km.dequantize(q, torch.float32).double() for q in (qx, qc))
    bias = torch.randn(K, generator=g, device=DEV)
    ref = 0.5 * (x @ c.T) + bias.double()
    S = km.scores(qx, qc, alpha=0.5, bias=bias)
    rel = 65 * 2 * U + (D / 4096 + 3) * U
    assert ((S.double() - ref).abs() <= rel * (ref.abs() + bias.abs())).all()
    assert torch.equal(km.scores(qx, qc, alpha=0.5, bias=bias), S)
    # a bf16 result takes one chain: D / 32 of them, half of which count, beside its rounding
    S16 = km.scores(qx, qc, alpha=0.5, bias=bias, dtype=torch.bfloat16)
    assert ((S16.double() - ref).abs() <= (HALF[torch.bfloat16] + D / 32 * U + 3 * U) * (ref.abs() + bias.abs())).all()


@pytest.mark.parametrize("N,D,K", [(300, 65536, 200), (130, 65536, 77), (33, 8192, 129), (257, 4097, 64), (70, 12300, 260), (3, 40000, 2),
                                   (9000, 8192, 1100), (5000, 4100, 1301)])
def test_scores_of_long_points_of_small_integers_are_exact(N, D, K):
    g = gen(D + K + 1)
    X, C = (torch.randint(-1, 2, (n, D), generator=g, device=DEV).float() for n in (N, K))
    bias = torch.randint(-5, 6, (K,), generator=g, device=DEV).float()
    buf = torch.full((N + 16, K), 7.0, device=DEV)
    S = km.scores(km.quantize(X), km.quantize(C), bias=bias, alpha=2.0, out=buf[8:8 + N])
    assert torch.equal(S.double(), 2 * X.double() @ C.double().T + bias.double())
    assert (buf[:8] == 7).all() and (buf[8 + N:] == 7).all()
