"""What the root-mean-square norm, the 8-bit rows and their product refuse,
without a GPU: every case returns before the library touches HIP."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

gn = pytest.importorskip("groupnorm_silu_normalization_amd")
from groupnorm_silu_normalization_amd import GnStatus  # noqa: E402

import rows8_reference as ref  # noqa: E402

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(16)]
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)
EIGHT = ctypes.c_void_p(0x10008)
I64 = ctypes.c_int64
BIG = 1 << 61


def norm(x=P[0], xs=64, res=P[1], rs=64, g=P[2], h=P[3], hs=64, y=P[4], ys=64, codes=None, cs=64,
         scales=None, rstd=P[5], M=4, C=64, eps=1e-6, dtype=0):
    return gn.gn_rms_norm_rows(x, xs, res, rs, g, h, hs, y, ys, codes, cs, scales, rstd, M, C, eps,
                               dtype, None)


def norm8(codes=P[6], scales=P[7], **kw):
    return norm(y=None, codes=codes, scales=scales, **kw)


def grad(dy=P[0], dys=64, x=P[1], xs=64, codes=None, scales=None, rstd=P[2], g=P[3], dh=P[4],
         dhs=64, dx=P[5], dxs=64, dg=P[6], M=4, C=64, dtype=0, ws=P[7], size=1 << 30):
    return gn.gn_rms_norm_rows_backward(dy, dys, x, xs, codes, scales, rstd, g, dh, dhs, dx, dxs,
                                        dg, M, C, dtype, ws, size, None)


def quantize(x=P[0], xs=64, codes=P[1], cs=64, scales=P[2], M=4, C=64, dtype=0):
    return gn.gn_quantize_rows(x, xs, codes, cs, scales, M, C, dtype, None)


def widen(codes=P[0], cs=64, scales=P[1], x=P[2], xs=64, M=4, C=64, dtype=0):
    return gn.gn_dequantize_rows(codes, cs, scales, x, xs, M, C, dtype, None)


def pack(codes=P[0], cs=64, packed=P[1], N=32, K=64):
    return gn.gn_int8_pack_weights(codes, cs, packed, N, K, None)


def product(a=P[0], as_=64, sa=P[1], w=P[2], sw=P[3], bias=P[4], res=P[5], rs=32, z=P[6], zs=32,
            M=4, N=32, K=64, dtype=0):
    return gn.gn_int8_matmul(a, as_, sa, w, sw, bias, res, rs, z, zs, M, N, K, dtype, None)


@pytest.mark.parametrize("fn,kw", [
    (norm, dict(x=None)), (norm, dict(y=None)), (norm, dict(codes=P[6], scales=P[7])),
    (norm, dict(res=None)), (norm, dict(h=None)), (norm, dict(h=P[4])), (norm8, dict(scales=None)),
    (norm8, dict(codes=None)), (norm, dict(scales=P[7])), (norm, dict(eps=-1.0)),
    (norm, dict(eps=float("nan"))), (norm, dict(eps=float("inf"))), (norm, dict(dtype=3)),
    (norm, dict(dtype=0x40)), (norm, dict(xs=-1)), (norm, dict(rs=-1)), (norm, dict(hs=63)),
    (norm, dict(ys=63)), (norm8, dict(cs=63)), (norm8, dict(cs=-64, M=1)), (norm, dict(M=-1)),
    (norm, dict(C=0)), (norm, dict(M=BIG)), (norm, dict(xs=BIG)), (norm, dict(rs=BIG)),
    (norm, dict(hs=BIG)), (norm8, dict(cs=BIG)),
    (grad, dict(dy=None)), (grad, dict(dx=None)), (grad, dict(rstd=None)), (grad, dict(x=None)),
    (grad, dict(codes=P[8], scales=P[9])), (grad, dict(x=None, codes=P[8])),
    (grad, dict(scales=P[9])), (grad, dict(dys=-1)), (grad, dict(xs=-1)), (grad, dict(dhs=-1)),
    (grad, dict(dxs=8)), (grad, dict(ws=None, M=5000)), (grad, dict(M=-4)), (grad, dict(C=-64)),
    (grad, dict(dtype=0x13)), (grad, dict(dhs=BIG)),
    (quantize, dict(x=None)), (quantize, dict(codes=None)), (quantize, dict(scales=None)),
    (quantize, dict(M=-1)), (quantize, dict(C=0)), (quantize, dict(xs=-8)),
    (quantize, dict(cs=63)), (quantize, dict(dtype=4)), (quantize, dict(M=BIG)),
    (widen, dict(x=None)), (widen, dict(codes=None)), (widen, dict(scales=None)),
    (widen, dict(xs=63)), (widen, dict(cs=-1)), (widen, dict(M=-1)), (widen, dict(dtype=-1)),
    (pack, dict(codes=None)), (pack, dict(packed=None)), (pack, dict(N=0)), (pack, dict(K=0)),
    (pack, dict(N=-5)), (pack, dict(cs=-1)), (pack, dict(cs=BIG)),
    (product, dict(a=None)), (product, dict(sa=None)), (product, dict(w=None)),
    (product, dict(sw=None)), (product, dict(z=None)), (product, dict(M=-1)),
    (product, dict(N=0)), (product, dict(K=-1)), (product, dict(dtype=3)),
    (product, dict(zs=31)), (product, dict(as_=-16)), (product, dict(rs=-1)),
    (product, dict(as_=BIG)),
])
def test_invalid(fn, kw):
    assert fn(**kw) == GnStatus.INVALID_ARGUMENT


@pytest.mark.parametrize("fn,kw", [
    (norm, dict(C=16385, xs=16385, rs=16385, hs=16385, ys=16385)), (norm, dict(x=ODD)),
    (norm, dict(res=ODD)), (norm, dict(h=ODD)), (norm, dict(y=ODD)), (norm, dict(g=ODD)),
    (norm, dict(rstd=TWO)), (norm8, dict(scales=TWO)), (norm, dict(x=TWO, dtype=2)),
    (grad, dict(C=16385, xs=16385, dys=16385, dxs=16385)), (grad, dict(dy=ODD)),
    (grad, dict(x=ODD)), (grad, dict(dh=ODD)), (grad, dict(dx=ODD)), (grad, dict(rstd=TWO)),
    (grad, dict(dg=ODD)), (grad, dict(g=ODD)), (grad, dict(ws=TWO)),
    (quantize, dict(C=16385, xs=16385, cs=16385)), (quantize, dict(x=ODD)),
    (quantize, dict(scales=TWO)),
    (widen, dict(C=16385, xs=16385)), (widen, dict(x=ODD)), (widen, dict(scales=TWO)),
    (pack, dict(packed=EIGHT)), (pack, dict(K=65537)), (pack, dict(N=(1 << 20) + 1)),
    (product, dict(w=EIGHT)), (product, dict(sa=TWO)),
    (product, dict(sw=TWO)), (product, dict(bias=TWO)), (product, dict(bias=ODD, dtype=0x20)),
    (product, dict(res=ODD)), (product, dict(z=ODD)), (product, dict(K=65537, as_=65552)),
    (product, dict(N=(1 << 20) + 1, zs=1 << 21)), (product, dict(M=(1 << 20) + 1)),
])
def test_unsupported(fn, kw):
    assert fn(**kw) == GnStatus.UNSUPPORTED


def test_empty_input_is_ok_without_gpu():
    assert norm(M=0) == GnStatus.OK and norm8(M=0) == GnStatus.OK
    assert grad(M=0, dg=None) == GnStatus.OK
    assert quantize(M=0) == GnStatus.OK and widen(M=0) == GnStatus.OK
    assert product(M=0) == GnStatus.OK


def size_of(fn, *a):
    out = I64(-7)
    return fn(*a, ctypes.byref(out)), out.value


def test_workspace_sizes():
    rb = gn.gn_rms_norm_rows_backward_workspace
    for M, C, dt in ((5000, 1, 0), (2000, 64, 1), (70000, 4096, 0), (9000, 16384, 2)):
        st, n = size_of(rb, M, C, dt)
        assert st == GnStatus.OK and 0 < n < 1 << 30 and n % (4 * C) == 0
        assert grad(M=M, C=C, xs=C, dys=C, dxs=C, dhs=C, dtype=dt,
                    size=n - 1) == GnStatus.SCRATCH_TOO_SMALL
    for M in (0, 1, 1000):
        assert size_of(rb, M, 64, 0) == (GnStatus.OK, 0)
    assert size_of(rb, 4, 16385, 0)[0] == GnStatus.UNSUPPORTED
    assert size_of(rb, -1, 64, 0)[0] == GnStatus.INVALID_ARGUMENT
    assert rb(4, 64, 0, None) == GnStatus.INVALID_ARGUMENT

    pb = gn.gn_int8_packed_bytes
    for N, K in ((1, 1), (16, 64), (17, 129), (4096, 4096), (1 << 20, 65536)):
        st, n = size_of(pb, N, K)
        assert st == GnStatus.OK and n >= N * K and n % 1024 == 0
        assert n <= (N + 15) * (K + 127)
    assert size_of(pb, 0, 4)[0] == GnStatus.INVALID_ARGUMENT
    assert size_of(pb, 4, 65537)[0] == GnStatus.UNSUPPORTED
    assert pb(4, 4, None) == GnStatus.INVALID_ARGUMENT


def test_product_plan():
    plan = gn.int8_matmul_plan
    for M, N, K in ((1, 1, 1), (1, 4096, 4096), (300, 500, 700), (1 << 20, 17, 65536),
                    (4096, 1 << 20, 1)):
        p = plan(M, N, K)
        assert p["workgroups"] == -(-M // p["rows"]) * -(-N // p["channels"]) < 1 << 23
    assert plan(1, 4096, 4096) == dict(rows=16, channels=16, tiles_kernel=0, workgroups=256)
    assert plan(16384, 4096, 4096)["tiles_kernel"] == 1
    # rows too far apart for 32-bit distances within a tile
    assert plan(16384, 4096, 4096, 1 << 24)["tiles_kernel"] == 0
    assert plan(1 << 20, 1 << 20, 64) is None       # more workgroups than a launch holds
    fn, out = gn.gn_int8_matmul_plan, (ctypes.c_int64 * 4)()
    assert fn(1, 1, 1, 1, None) == GnStatus.INVALID_ARGUMENT
    assert fn(-1, 1, 1, 1, out) == fn(1, 0, 1, 1, out) == GnStatus.INVALID_ARGUMENT
    assert fn(1, 1, 1, -1, out) == GnStatus.INVALID_ARGUMENT
    assert fn(1, 1, 65537, 1, out) == GnStatus.UNSUPPORTED


# ---- the binding ---------------------------------------------------------------
def rows8(*shape, dtype=torch.bfloat16):
    return gn.Rows8(torch.zeros(*shape, dtype=torch.int8), torch.zeros(*shape[:-1]), dtype)


def test_binding_declines_what_is_not_on_a_gpu_or_under_autograd():
    x = torch.ones(4, 64)
    with torch.no_grad():
        assert gn.rms_norm_rows(x) is None
        assert gn.rms_norm_rows(x, quantize=True) is None
        assert gn.rms_norm_rows_backward(x, x, torch.ones(4)) is None
        assert gn.quantize_rows(x) is None
        assert gn.dequantize_rows(rows8(4, 64)) is None
        assert gn.pack_int8_weight(rows8(32, 64)) is None
        assert gn.int8_matmul(rows8(4, 64), rows8(32, 64)) is None


def test_binding_refuses_what_is_no_input():
    x = torch.ones(4, 64)
    with torch.no_grad():
        for call in (lambda: gn.rms_norm_rows([1.0]), lambda: gn.quantize_rows(None),
                     lambda: gn.dequantize_rows(x), lambda: gn.pack_int8_weight(x),
                     lambda: gn.int8_matmul(x, rows8(32, 64)),
                     lambda: gn.int8_matmul(rows8(4, 64), x),
                     lambda: gn.int8_matmul(rows8(4, 64), rows8(32, 64), dtype=torch.int8)):
            with pytest.raises(TypeError):
                call()
        for call in (lambda: gn.pack_int8_weight(rows8(2, 32, 64)),
                     lambda: gn.int8_matmul(rows8(4, 64), rows8(32, 65)),
                     lambda: gn.int8_matmul(rows8(4, 64), rows8(2, 32, 64))):
            with pytest.raises(ValueError):
                call()


def test_rows8_object():
    codes, scales = torch.zeros(3, 70, dtype=torch.int8), torch.zeros(3)
    q = gn.Rows8(codes, scales, torch.float16)
    assert q.shape == (3, 70) and q.dtype == torch.float16 and q.device.type == "cpu"
    assert gn.Rows8(torch.zeros(3, 80, dtype=torch.int8)[:, :70], scales, torch.float16)
    for bad in ((codes.float(), scales), (codes, scales.double()), (codes, None)):
        with pytest.raises(TypeError):
            gn.Rows8(*bad, torch.float16)
    with pytest.raises(TypeError):
        gn.Rows8(codes, scales, torch.float64)
    for bad in (scales[:2], scales.reshape(3, 1)):
        with pytest.raises(ValueError):
            gn.Rows8(codes, bad, torch.float16)
    with pytest.raises(ValueError):
        gn.Rows8(torch.zeros(70, 3, dtype=torch.int8).t(), scales, torch.float16)
    with pytest.raises(ValueError):
        gn.Rows8(codes, torch.zeros(6)[::2], torch.float16)


def test_packed_weight_object():
    size = size_of(gn.gn_int8_packed_bytes, 20, 70)[1]
    data, scales = torch.zeros(size, dtype=torch.int8), torch.zeros(20)
    assert gn.PackedInt8Weight(data, scales, 20, 70).shape == (20, 70)
    for bad in ((data.float(), scales), (data, scales.double())):
        with pytest.raises(TypeError):
            gn.PackedInt8Weight(*bad, 20, 70)
    for bad in ((data[:-1], scales, 20, 70), (data, scales[:19], 20, 70), (data, scales, 20, 700),
                (data, scales, 33, 70), (data, torch.zeros(40)[::2], 20, 70),
                (data, scales, 0, 70)):
        with pytest.raises(ValueError):
            gn.PackedInt8Weight(*bad)


def test_reference_codes_are_nearest_and_ties_even():
    g = torch.Generator().manual_seed(3)
    t = torch.randn(50, 200, generator=g)
    t[1] = 0.0
    t[2] = 254.0
    t[2, :5] = torch.tensor([1.0, 3.0, 5.0, -1.0, -3.0])    # halves of 254 / 127
    q, top = ref.codes_of(t)
    assert torch.equal(q[2, :5], torch.tensor([0, 2, 2, 0, -2]))
    assert int(q.abs().max()) == 127 and not q[1].any()
    off = (127 * t.double() - q * top.unsqueeze(-1)).abs()
    assert bool((off <= 0.5 * top.unsqueeze(-1)).all())
