"""Host-side checks of the soft-assignment operators, no GPU needed: shapes,
types, layouts and workspaces are refused before any launch, by the binding
(tensors) and by the C entry points (sizes and pointers)."""

import ctypes

import pytest
import torch

import means_clustering_flashassign_b200 as km

F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def q_cpu(N, D):
    return km.Quantized(torch.zeros(N, (D + 15) // 16 * 16, dtype=torch.uint8).view(F8)[..., :D],
                        torch.zeros(N, (D + 127) // 128, dtype=torch.uint8).view(E8))


@pytest.mark.parametrize("call", [
    lambda: km.quantize(torch.zeros(4, 8)),
    lambda: km.dequantize(q_cpu(4, 8)),
    lambda: km.scores(q_cpu(4, 8), q_cpu(2, 8)),
    lambda: km.scores_grad(torch.zeros(4, 2), q_cpu(4, 8), q_cpu(2, 8)),
    lambda: km.balance(torch.zeros(4, 2), torch.zeros(4, dtype=torch.int32)),
    lambda: km.balance_grad(torch.zeros(4, 2), None),
])
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA"):
        call()


class FakeCuda:
    """Just enough of a CUDA tensor for the layout checks."""

    def __init__(self, t, device="cuda:0"):
        self.t, self.is_cuda, self.device = t, True, torch.device(device)

    def __getattr__(self, name):
        return getattr(self.t, name)


def fake_q(data, scale, device="cuda:0"):
    return km.Quantized(FakeCuda(data, device), FakeCuda(scale, device))


def test_layout_of_8_bit_points():
    good = q_cpu(6, 40)
    assert km._check_quantized(fake_q(*good), "X") == (1, 6, 40, False)
    b = torch.zeros(2, 6, 48, dtype=torch.uint8).view(F8)[..., :40]
    s = torch.zeros(2, 6, 1, dtype=torch.uint8).view(E8)
    assert km._check_quantized(fake_q(b, s), "X") == (2, 6, 40, True)
    one = km.Quantized(torch.zeros(1, 16, dtype=torch.uint8).view(F8)[..., :3], torch.zeros(1, 1, dtype=torch.uint8).view(E8))
    assert km._check_quantized(fake_q(*one), "X") == (1, 1, 3, False)


@pytest.mark.parametrize("data,scale,error,msg", [
    (torch.zeros(6, 40, dtype=torch.uint8).view(F8), None, ValueError, "48 bytes apart"),       # rows not padded
    (torch.zeros(12, 48, dtype=torch.uint8).view(F8)[::2, :40], None, ValueError, "48 bytes"),   # strided rows
    (torch.zeros(6, 48, dtype=torch.uint8)[:, :40], None, TypeError, "float8_e4m3fn"),
    (None, torch.zeros(6, 1, dtype=torch.uint8), TypeError, "float8_e8m0fnu"),
    (None, torch.zeros(5, 1, dtype=torch.uint8).view(E8), ValueError, "must have shape"),
    (None, torch.zeros(6, 2, dtype=torch.uint8).view(E8), ValueError, "must have shape"),
    (torch.zeros(6 * 48 - 8, dtype=torch.uint8).view(F8).as_strided((6, 40), (48, 1)), None, ValueError, "last row"),
    (torch.zeros(6 * 48 + 1, dtype=torch.uint8).view(F8)[1:].as_strided((6, 40), (48, 1), 1), None, ValueError, "aligned"),
    (torch.zeros(48, dtype=torch.uint8).view(F8), None, ValueError, "must be"),
])
def test_other_layouts_are_refused(data, scale, error, msg):
    good = q_cpu(6, 40)
    q = fake_q(good.data if data is None else data, good.scale if scale is None else scale)
    with pytest.raises(error, match=msg):
        km._check_quantized(q, "X")


def test_operands_on_two_devices_are_refused():
    with pytest.raises(ValueError, match="the points are on"):
        km._check_quantized(fake_q(*q_cpu(6, 40), device="cuda:1"), "C", torch.device("cuda:0"))
    with pytest.raises(TypeError, match="Quantized"):
        km._check_quantized(torch.zeros(3), "X")


def test_validity_masks():
    dev = torch.device("cpu")
    assert km._valid_mask(None, (3,), dev) is None
    km._valid_mask(torch.ones(3, dtype=torch.bool), (3,), dev)
    for bad in (torch.ones(3), torch.ones(4, dtype=torch.bool), torch.ones(6, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            km._valid_mask(bad, (3,), dev)


BIG = 1 << 31


@pytest.mark.parametrize("args", [
    (km.SOFT_SCORES, 0, 10, 8, 4, km.BF16), (km.SOFT_SCORES, 1, -1, 8, 4, km.BF16), (km.SOFT_SCORES, 1, 10, 0, 4, km.BF16),
    (km.SOFT_SCORES, 1, 10, 8, 0, km.BF16), (km.SOFT_SCORES, 1, BIG, 8, 4, km.BF16), (km.SOFT_SCORES, 1, 10, 65537, 4, km.F32),
    (km.SOFT_SCORES, 1, 10, 8, (1 << 20) + 1, km.F32), (km.SOFT_SCORES, 65537, 10, 8, 4, km.F32),
    (km.SOFT_SCORES_GRAD, 1, 10, 8, 4, 2), (3, 1, 10, 8, 4, km.BF16), (-1, 1, 10, 8, 4, km.BF16),
])
def test_sizes_out_of_range_have_no_workspace(args):
    assert km.library().km_soft_workspace_size(*args) == 0
    assert km.library().km_last_error()
    with pytest.raises(km.KMError):
        km.soft_workspace_size(*args)


def test_workspaces_are_not_scores_sized():
    # no N x K term where dS is used as it lies
    w = km.soft_workspace_size(km.SOFT_SCORES_GRAD, 1, 1 << 20, 128, 1024, km.BF16)
    assert w < (1 << 20) * 1024 * 2 / 4
    assert km.soft_workspace_size(km.SOFT_SCORES, 1, 1 << 20, 128, 1024, km.BF16) <= 1 << 16
    assert km.soft_workspace_size(km.SOFT_BALANCE, 1, 1 << 20, 128, 1024, km.F32) <= 1 << 17
    for N in (0, 1, 5):
        assert km.soft_workspace_size(km.SOFT_SCORES_GRAD, 2, N, 3, 5, km.F32) > 0


def test_c_entries_refuse_bad_calls_before_the_device():
    L = km.library()
    buf = (ctypes.c_uint8 * 8192)()
    a = (ctypes.addressof(buf) + 255) // 256 * 256
    p, odd, sz = ctypes.c_void_p(a), ctypes.c_void_p(a + 8), 4096
    INVALID, WORKSPACE, UNSUPPORTED = 1, 4, 2
    assert L.km_quantize(None, 1, 4, 8, km.F32, p, p, None) == INVALID
    assert L.km_quantize(p, 1, 4, 8, 9, p, p, None) == INVALID
    assert L.km_quantize(p, 1, 4, 8, km.F32, odd, p, None) == INVALID
    assert L.km_dequantize(p, None, 1, 4, 8, km.F32, p, None) == INVALID
    assert L.km_dequantize(odd, p, 1, 4, 8, km.F32, p, None) == INVALID
    assert L.km_quantize(p, 1, BIG, 8, km.F32, p, p, None) == UNSUPPORTED
    scores = lambda x=p, c=p, s=p, n=4, d=8, k=4, ws=p, wsb=sz, dt=km.F32: L.km_scores(  # noqa: E731
        x, p, c, p, None, 1.0, 1, n, d, k, dt, s, ws, wsb, None)
    assert scores(x=None) == INVALID and scores(c=None) == INVALID and scores(s=None) == INVALID
    assert scores(x=odd) == INVALID and scores(c=odd) == INVALID and scores(dt=7) == INVALID
    assert scores(ws=None) == WORKSPACE and scores(ws=odd) == WORKSPACE and scores(wsb=16) == WORKSPACE
    assert scores(d=1 << 17) == UNSUPPORTED
    grad = lambda ds=p, dx=p, dc=p, db=p, dt=km.BF16, dxt=km.BF16, wsb=sz: L.km_scores_grad(  # noqa: E731
        ds, p, p, p, p, 1.0, 1, 4, 8, 4, dt, dxt, dx, dc, db, p, wsb, None)
    assert grad(ds=None) == INVALID and grad(ds=odd) == INVALID and grad(dx=None, dc=None, db=None) == INVALID
    assert grad(dt=3) == INVALID and grad(dxt=3) == INVALID and grad(wsb=256) == WORKSPACE
    bal = lambda s=p, i=p, t=1, loss=p, cnt=p, n=4, wsb=sz: L.km_balance(  # noqa: E731
        s, i, None, 1, n, 4, t, km.F32, loss, cnt, p, p, p, p, wsb, None)
    assert bal(s=None) == INVALID and bal(i=None) == INVALID and bal(loss=None) == INVALID and bal(cnt=None) == INVALID
    assert bal(t=0) == INVALID and bal(t=1025) == INVALID and bal(s=odd) == INVALID and bal(wsb=8) == WORKSPACE
    assert bal(n=1 << 22, t=1024) == UNSUPPORTED
    bgrad = lambda s=p, ds=p, r=p, t=1: L.km_balance_grad(s, None, p, r, p, p, None, 1, 4, 4, t, km.F32, ds, None)  # noqa: E731
    assert bgrad(s=None) == INVALID and bgrad(ds=None) == INVALID and bgrad(r=None) == INVALID
    assert bgrad(ds=odd) == INVALID and bgrad(t=0) == INVALID
    one = ctypes.c_void_p(a + 1)   # between elements
    assert L.km_quantize(one, 1, 4, 8, km.BF16, p, p, None) == INVALID
    assert L.km_dequantize(p, p, 1, 4, 8, km.F32, ctypes.c_void_p(a + 2), None) == INVALID
    assert scores(s=one) == INVALID and grad(dx=one) == INVALID and grad(dc=one) == INVALID
    assert bal(i=one) == INVALID and bal(loss=one) == INVALID and bgrad(r=one) == INVALID


def test_valid_calls_without_a_gpu_report_the_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    L = km.library()
    buf = (ctypes.c_uint8 * 8192)()
    p = ctypes.c_void_p((ctypes.addressof(buf) + 255) // 256 * 256)
    assert L.km_quantize(p, 1, 4, 8, km.F32, p, p, None) == 3
    assert L.km_scores(p, p, p, p, None, 1.0, 1, 4, 8, 4, km.F32, p, p, 4096, None) == 3


@pytest.mark.parametrize("kernel", ["k_grad_prep", "k_grad", "k_grad_join", "k_bal_zero", "k_bal_count", "k_bal_rows",
                                    "k_bal_rows_wide"])
def test_chained_kernels_wait_before_they_touch_the_chains_data(kernel):
    """The same rule as for the kernels of a Lloyd iteration: every kernel that
    may be launched with programmatic stream serialization waits on the device
    before it can return."""
    import test_chain_rule as rule
    bodies = rule._kernel_bodies(kernel)
    assert bodies
    for fname, body in bodies:
        w = body.find("pdl_wait();")
        assert w >= 0 and "return;" not in body[:w], (kernel, fname)


def test_the_rounding_of_a_long_gradient_waits_and_has_room():
    """k_grad_round is chained like the kernels above; its sums are a float32 dX of
    workspace where the terms of an element pass 512 slices of 64, and none below."""
    import test_chain_rule as rule
    (_, body), = rule._kernel_bodies("k_grad_round")
    assert body.find("pdl_wait();") < body.find("sums +")
    for dtype, last in ((km.BF16, 512 * 64), (km.F32, 170 * 64)):
        size = [km.soft_workspace_size(km.SOFT_SCORES_GRAD, 2, 50, 72, K, dtype) for K in (last, last + 8)]
        assert size[1] - size[0] >= 2 * 50 * 72 * 4
        # and no more beyond it than 8 centroids take: their operand, planes and pieces
        assert size[1] - size[0] <= 2 * 50 * 72 * 4 + 8 * 2 * (72 * 2 + 3 * 50 * 2 + 148 * 4 * 80) + 4096


@pytest.mark.parametrize("B,N,D,K,dtype", [(65536, BIG - 1, 65536, 1 << 20, km.F32), (65536, BIG - 1, 65536, 1, km.BF16),
                                           (65536, BIG - 1, 1, 1 << 20, km.F32), (64, BIG - 1, 65536, 1 << 20, km.F32),
                                           (63, BIG - 1, 65536, 1 << 20, km.F32), (65536, (1 << 21) - 1, 65536, 1 << 20, km.F32),
                                           (65536, 1 << 21, 8, 8, km.BF16)])
def test_workspace_sizes_do_not_wrap(B, N, D, K, dtype):
    """No size, or one that holds the operands it stands for (in whole numbers of any length)."""
    ldd, ldk = (D + 7) // 8 * 8, (K + 7) // 8 * 8
    least = 2 * B * (N + K) * ldd + (6 * B * N * ldk if dtype == km.F32 else 0)
    got = km.library().km_soft_workspace_size(km.SOFT_SCORES_GRAD, B, N, D, K, dtype)
    assert got == 0 if B * N >= 1 << 37 else got >= least
    L = km.library()
    buf = (ctypes.c_uint8 * 512)()
    p = ctypes.c_void_p((ctypes.addressof(buf) + 255) // 256 * 256)
    if B * N >= 1 << 37:   # and no call of such a shape
        assert L.km_quantize(p, B, N, D, dtype, p, p, None) == 2
        assert L.km_scores(p, p, p, p, None, 1.0, B, N, D, K, dtype, p, p, 256, None) == 2


@pytest.mark.parametrize("dtype,es", [(km.F32, 4), (km.BF16, 2)])
def test_a_balance_gradient_over_its_own_scores_is_refused(dtype, es):
    """Rows are read ahead of the rows written: dS anywhere on S would change what
    later rows are taken from."""
    L = km.library()
    buf = (ctypes.c_uint8 * 8192)()
    a = (ctypes.addressof(buf) + 255) // 256 * 256
    size = 2 * 20 * 16 * es                # B = 2, N = 20, K = 16
    call = lambda s, ds: L.km_balance_grad(ctypes.c_void_p(s), None, a, a, a, a, None, 2, 20, 16, 1, dtype, ctypes.c_void_p(ds), None)  # noqa: E731
    for off in (0, 16, 16 * es, size - 16):
        assert call(a, a + off) == 1 and call(a + off, a) == 1
        assert b"overlap" in L.km_last_error()
    if not torch.cuda.is_available():      # side by side they get as far as the device
        assert call(a, a + size) == 3 and call(a + size, a) == 3
