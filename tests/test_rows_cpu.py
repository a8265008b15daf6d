"""What the layer norm, backward and checkpoint calls refuse, without a GPU:
every case returns before the library touches HIP."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

gn = pytest.importorskip("groupnorm_silu_normalization_amd")
from groupnorm_silu_normalization_amd import GnStatus  # noqa: E402

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(16)]
ODD = ctypes.c_void_p(0x10001)
I64 = ctypes.c_int64


def layer_norm(x=P[0], xs=64, g=P[1], b=P[2], y=P[3], ys=64, M=4, C=64, eps=1e-6, dtype=0,
               mean=None, rstd=None, codes=None, scales=None):
    return gn.gn_layer_norm_rows(x, xs, g, b, y, ys, M, C, eps, dtype, mean, rstd, codes, scales,
                                 None)


def layer_norm_backward(dy=P[0], dys=64, x=P[1], xs=64, codes=None, scales=None, mean=P[2],
                        rstd=P[3], g=P[4], dx=P[5], dxs=64, dg=P[6], db=P[7], M=4, C=64, dtype=0,
                        ws=P[8], size=1 << 30):
    return gn.gn_layer_norm_rows_backward(dy, dys, x, xs, codes, scales, mean, rstd, g, dx, dxs,
                                          dg, db, M, C, dtype, ws, size, None)


def group_backward(dy=P[0], x=P[1], codes=None, scales=None, mean=P[2], rstd=P[3], g=P[4], b=P[5],
                   dx=P[6], dg=P[7], db=P[8], N=1, L=4, C=64, G=8, silu=1, dtype=0, ws=P[9],
                   size=1 << 30):
    return gn.gn_silu_rows_backward(dy, x, codes, scales, mean, rstd, g, b, dx, dg, db, N, L, C, G,
                                    silu, dtype, ws, size, None)


def apply_save(x=P[0], mean=P[1], rstd=P[2], g=P[3], b=P[4], y=P[5], codes=P[6], scales=P[7], N=1,
               L=4, C=64, G=8, silu=1, dtype=0):
    return gn.gn_apply_rows_save(x, mean, rstd, g, b, y, codes, scales, N, L, C, G, silu, dtype,
                                 None)


def save(x=P[0], xs=64, codes=P[1], scales=P[2], M=4, C=64, dtype=0):
    return gn.gn_checkpoint_rows(x, xs, codes, scales, M, C, dtype, None)


def restore(codes=P[1], scales=P[2], x=P[0], xs=64, M=4, C=64, dtype=0):
    return gn.gn_restore_rows(codes, scales, x, xs, M, C, dtype, None)


BIG = 1 << 61


@pytest.mark.parametrize("fn,kw", [
    (layer_norm, dict(x=None)), (layer_norm, dict(y=None)), (layer_norm, dict(M=-1)),
    (layer_norm, dict(C=0)), (layer_norm, dict(eps=-1.0)), (layer_norm, dict(eps=float("nan"))),
    (layer_norm, dict(eps=float("inf"))), (layer_norm, dict(dtype=3)),
    (layer_norm, dict(dtype=0x40)), (layer_norm, dict(xs=-1)), (layer_norm, dict(ys=63)),
    (layer_norm, dict(ys=-64, M=1)), (layer_norm, dict(codes=P[5])),
    (layer_norm, dict(scales=P[5])), (layer_norm, dict(M=BIG)), (layer_norm, dict(xs=BIG)),
    (layer_norm, dict(ys=BIG)), (layer_norm, dict(M=1 << 40, C=1 << 30)),
    (layer_norm_backward, dict(dy=None)), (layer_norm_backward, dict(dx=None)),
    (layer_norm_backward, dict(mean=None)), (layer_norm_backward, dict(rstd=None)),
    (layer_norm_backward, dict(x=None)), (layer_norm_backward, dict(codes=P[9], scales=P[10])),
    (layer_norm_backward, dict(x=None, codes=P[9])), (layer_norm_backward, dict(scales=P[9])),
    (layer_norm_backward, dict(dys=-1)), (layer_norm_backward, dict(xs=-1)),
    (layer_norm_backward, dict(dxs=8)), (layer_norm_backward, dict(ws=None, M=5000)),
    (layer_norm_backward, dict(M=-4)), (layer_norm_backward, dict(C=-64)),
    (layer_norm_backward, dict(dtype=0x13)),
    (group_backward, dict(dy=None)), (group_backward, dict(dx=None)),
    (group_backward, dict(mean=None)), (group_backward, dict(rstd=None)),
    (group_backward, dict(x=None)), (group_backward, dict(codes=P[10], scales=P[11])),
    (group_backward, dict(G=0)), (group_backward, dict(G=7)), (group_backward, dict(G=-8)),
    (group_backward, dict(silu=2)), (group_backward, dict(N=-1)), (group_backward, dict(L=-1)),
    (group_backward, dict(ws=None, L=50000)), (group_backward, dict(N=1 << 40, L=1 << 30)),
    (group_backward, dict(dtype=9)),
    (apply_save, dict(x=None)), (apply_save, dict(y=None)), (apply_save, dict(codes=None)),
    (apply_save, dict(scales=None)), (apply_save, dict(mean=None)), (apply_save, dict(rstd=None)),
    (apply_save, dict(G=5)), (apply_save, dict(silu=-1)), (apply_save, dict(C=0)),
    (save, dict(x=None)), (save, dict(codes=None)), (save, dict(scales=None)),
    (save, dict(M=-1)), (save, dict(C=0)), (save, dict(xs=-8)), (save, dict(dtype=4)),
    (save, dict(M=BIG)), (save, dict(xs=BIG, M=2)),
    (restore, dict(x=None)), (restore, dict(codes=None)), (restore, dict(scales=None)),
    (restore, dict(xs=63)), (restore, dict(xs=0)), (restore, dict(M=-1)),
])
def test_invalid(fn, kw):
    assert fn(**kw) == GnStatus.INVALID_ARGUMENT


@pytest.mark.parametrize("fn,kw", [
    (layer_norm, dict(C=16385, xs=16385, ys=16385)), (layer_norm, dict(x=ODD)),
    (layer_norm, dict(y=ODD)), (layer_norm, dict(g=ODD)), (layer_norm, dict(b=ODD)),
    (layer_norm, dict(mean=ODD)), (layer_norm, dict(rstd=ODD)),
    (layer_norm, dict(x=ctypes.c_void_p(0x10002), dtype=2)),
    (layer_norm_backward, dict(C=16385, xs=16385, dys=16385, dxs=16385)),
    (layer_norm_backward, dict(dy=ODD)), (layer_norm_backward, dict(x=ODD)),
    (layer_norm_backward, dict(dx=ODD)), (layer_norm_backward, dict(mean=ODD)),
    (layer_norm_backward, dict(dg=ODD)), (layer_norm_backward, dict(db=ODD)),
    (layer_norm_backward, dict(ws=ODD)),
    (group_backward, dict(C=8200, G=8)), (group_backward, dict(dy=ODD)),
    (group_backward, dict(x=ODD)), (group_backward, dict(dx=ODD)),
    (group_backward, dict(rstd=ODD)), (group_backward, dict(dg=ODD)),
    (group_backward, dict(ws=ODD)), (group_backward, dict(N=1 << 24, L=1)),
    (apply_save, dict(C=8200, G=8)), (apply_save, dict(x=ODD)), (apply_save, dict(y=ODD)),
    (apply_save, dict(N=1 << 24, L=1)),
    (save, dict(C=16385, xs=16385)), (save, dict(x=ODD)),
    (restore, dict(C=16385, xs=16385)), (restore, dict(x=ODD)),
])
def test_unsupported(fn, kw):
    assert fn(**kw) == GnStatus.UNSUPPORTED


def test_empty_input_is_ok_without_gpu():
    assert layer_norm(M=0) == GnStatus.OK
    assert layer_norm_backward(M=0, dg=None, db=None) == GnStatus.OK
    assert group_backward(L=0, dg=None, db=None) == GnStatus.OK
    assert group_backward(N=0, dg=None, db=None) == GnStatus.OK
    assert apply_save(N=0) == GnStatus.OK and apply_save(L=0) == GnStatus.OK
    assert save(M=0) == GnStatus.OK and restore(M=0) == GnStatus.OK


def workspace(fn, *a):
    out = I64(-7)
    return fn(*a, ctypes.byref(out)), out.value


def test_workspace_sizes():
    ln, gb = gn.gn_layer_norm_rows_backward_workspace, gn.gn_silu_rows_backward_workspace
    for M, C, dt in ((5000, 1, 0), (2000, 64, 1), (70000, 4096, 0), (9000, 16384, 2),
                     (1 << 40, 8, 0)):
        st, n = workspace(ln, M, C, dt)
        assert st == GnStatus.OK and 0 < n < 1 << 30 and n % (8 * C) == 0
        if M * C < 1 << 40:
            assert layer_norm_backward(M=M, C=C, xs=C, dys=C, dxs=C, dtype=dt,
                                       size=n - 1) == GnStatus.SCRATCH_TOO_SMALL
    for M in (0, 1, 1000):      # few rows need none
        assert workspace(ln, M, 64, 0) == (GnStatus.OK, 0)
    assert workspace(ln, 4, 16385, 0)[0] == GnStatus.UNSUPPORTED
    assert workspace(ln, -1, 64, 0)[0] == GnStatus.INVALID_ARGUMENT
    assert ln(4, 64, 0, None) == GnStatus.INVALID_ARGUMENT
    for N, L, C, G, dt in ((1, 1, 1, 1, 0), (3, 7, 96, 8, 1), (1, 1 << 20, 256, 32, 0),
                           (2, 5, 8192, 1, 2), (2, 5, 64, 8, 0)):
        st, n = workspace(gb, N, L, C, G, dt)
        assert st == GnStatus.OK and 0 < n < 1 << 30
        assert group_backward(N=N, L=L, C=C, G=G, dtype=dt,
                              size=n - 1) == GnStatus.SCRATCH_TOO_SMALL
        assert group_backward(N=N, L=L, C=C, G=G, dtype=dt, size=-1) == GnStatus.SCRATCH_TOO_SMALL
        assert group_backward(N=N, L=L, C=C, G=G, dtype=dt,
                              ws=None) == GnStatus.INVALID_ARGUMENT
    assert workspace(gb, 1, 0, 64, 8, 0) == (GnStatus.OK, 0)
    assert workspace(gb, 1, 100, 64, 8, 0) == (GnStatus.OK, 0)     # one launch, one sample
    assert workspace(gb, 1, 4, 64, 7, 0)[0] == GnStatus.INVALID_ARGUMENT
    assert workspace(gb, 1, 4, 8200, 8, 0)[0] == GnStatus.UNSUPPORTED
    assert gb(1, 4, 64, 8, 0, None) == GnStatus.INVALID_ARGUMENT


# ---- the binding ---------------------------------------------------------------
def test_binding_declines_what_is_not_on_a_gpu_or_under_autograd():
    x = torch.ones(4, 64)
    st = torch.ones(4)
    with torch.no_grad():
        assert gn.layer_norm_rows(x) is None
        assert gn.checkpoint_rows(x) is None
        assert gn.layer_norm_rows_backward(x, x, st, st) is None
        r = torch.ones(1, 4, 64)
        assert gn.group_norm_silu_rows_backward(r, r, torch.ones(1, 8), torch.ones(1, 8)) is None
        ck = gn.Checkpoint8(torch.zeros(4, 64, dtype=torch.int8),
                            torch.zeros(4, 2, dtype=torch.uint8), torch.bfloat16)
        assert gn.restore_rows(ck) is None


def test_checkpoint_object():
    codes, scales = torch.zeros(3, 70, dtype=torch.int8), torch.zeros(3, 3, dtype=torch.uint8)
    ck = gn.Checkpoint8(codes, scales, torch.float16)
    assert ck.shape == (3, 70) and ck.dtype == torch.float16 and ck.device.type == "cpu"
    with pytest.raises(TypeError):
        gn.Checkpoint8(codes.float(), scales, torch.float16)
    with pytest.raises(TypeError):
        gn.Checkpoint8(codes, scales.to(torch.int8), torch.float16)
    with pytest.raises(TypeError):
        gn.Checkpoint8(codes, scales, torch.float64)
    for bad in (scales[:, :2], scales[:2], scales.reshape(-1)):
        with pytest.raises(ValueError):
            gn.Checkpoint8(codes, bad, torch.float16)
    with pytest.raises(ValueError):
        gn.Checkpoint8(torch.zeros(70, 3, dtype=torch.int8).t(), scales, torch.float16)


def test_row_strides():
    rs = gn.binding._row_stride
    x = torch.zeros(6, 4, 10)
    assert rs(x) == 10 and rs(x[..., 2:7]) == 10 and rs(x[0, 0]) == 10
    assert rs(x[:, ::2, 1:]) == 20 and rs(x[::2, :, 1:]) is None and rs(x[::2, 0]) == 80
    assert rs(x[..., ::2]) is None and rs(x[0, 0].expand(5, 10)) == 0
    assert rs(x.transpose(0, 1)) is None and rs(torch.zeros(3, 1).expand(3, 1)) == 1
    assert rs(torch.zeros(7)[3:4]) == 1


def test_calls_without_a_device_check_name_the_cause_on_cpu_tensors():
    """Steps that take any tensor's address report what torch says of its
    device (ValueError) or of the missing GPU, not of a stream."""
    x, st = torch.zeros(1, 4, 64), torch.zeros(1, 8)
    for call in (lambda: gn.group_stats_rows(x, 8), lambda: gn.apply_rows(x, st, st),
                 lambda: gn.profile_rows(x, 8, None, None, 1e-6, True, x, 1)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)) as e:
            with torch.no_grad():
                call()
        assert "Stream" not in str(e.value)
