"""The binding looks at what elements are, not at their size alone: a tensor of
another type of the same size is refused before its pointer is passed on.
Calls without rows launch nothing and need no GPU."""
import pytest
import torch

import activation_sparse_feedforward_gate_amd as tw

F32, BF16, MX8 = tw.TWELL_F32, tw.TWELL_BF16, tw.TWELL_MXFP8
f16, bf16, f32, u8 = torch.float16, torch.bfloat16, torch.float32, torch.uint8
e4m3, e8m0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def e(*size, dt):
    return torch.zeros(*size, dtype=dt)


def weights():
    return tw.TwellW4(e(8, 32, dt=u8), e(8, 2, dt=u8))


def refused(name, f, *args):
    """The type of argument `name` is what the call refuses."""
    with pytest.raises(ValueError, match=rf"^{name}: expected .*(float|int)\d+.* elements"):
        f(*args)


@pytest.fixture
def norm():
    """Arguments of a forward of no rows; a dict that a test changes."""
    def call(mx=False, fwd=True, **k):
        sh = tw.norm_shape(0, 64, BF16, F32, MX8 if mx else BF16, BF16, 1e-5, 0.1)
        a = dict(x=e(0, 64, dt=bf16), res=e(0, 64, dt=f32), w=None, rng=None, sum=e(0, 64, dt=f32),
                 y=e(0, 64, dt=u8 if mx else bf16), ys=e(0, 2, dt=u8) if mx else None, rstd=e(0, dt=f32),
                 dw=None, ws=None)
        a.update(k)
        if fwd:
            return tw.twell_add_rmsnorm_fwd, (sh, a["x"], a["res"], a["w"], a["rng"], a["sum"], a["y"], a["ys"], a["rstd"])
        return tw.twell_add_rmsnorm_bwd, (sh, a["y"], a["res"], a["sum"], a["w"], a["rstd"], a["rng"], a["res"],
                                          a["x"], a["dw"], a["ws"])
    return call


@pytest.fixture(autouse=True)
def stream(monkeypatch):
    """A stream to launch nothing on, where there is no GPU to ask for one."""
    class Null:
        cuda_stream = 0
    for name in ("twell_add_rmsnorm_fwd", "twell_add_rmsnorm_bwd", "twell_dropout_add", "twell_w4_matvec",
                 "twell_ffn_fwd_w4"):
        f = getattr(tw, name)
        monkeypatch.setattr(tw, name, lambda *a, f=f: f(*a, stream=Null()))


def test_norm_types(norm):
    for mx in (False, True):
        f, a = norm(mx)
        f(*a)
    f, a = norm(fwd=False)
    f(*a)
    f, a = norm(True, y=e(0, 64, dt=e4m3), ys=e(0, 2, dt=e8m0))
    f(*a)
    for fwd in (True, False):
        refused("x" if fwd else "dx", *flat(norm(fwd=fwd, x=e(0, 64, dt=f16))))
        refused("y" if fwd else "dy", *flat(norm(fwd=fwd, y=e(0, 64, dt=torch.int16))))
        refused("residual" if fwd else "dsum", *flat(norm(fwd=fwd, res=e(0, 64, dt=torch.int32))))
        refused("sum", *flat(norm(fwd=fwd, sum=e(0, 64, dt=torch.int32))))
        refused("w", *flat(norm(fwd=fwd, w=e(64, dt=f16))))
        refused("rng", *flat(norm(fwd=fwd, rng=e(2, dt=torch.float64))))
        refused("rstd", *flat(norm(fwd=fwd, rstd=e(0, dt=torch.int32))))
    refused("dw", *flat(norm(fwd=False, dw=e(64, dt=torch.int32))))
    for dt in (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int8, torch.bool):
        refused("y", *flat(norm(True, y=e(0, 64, dt=dt))))
        refused("y_scale", *flat(norm(True, ys=e(0, 2, dt=dt))))


def flat(call):
    return call[0], *call[1]


def test_dropout_types():
    sh = tw.norm_shape(0, 8, F32, BF16, BF16, F32, 0.0, 0.1)
    x, res, y = e(0, 8, dt=f32), e(0, 8, dt=bf16), e(0, 8, dt=bf16)
    tw.twell_dropout_add(sh, x, res, None, y)
    refused("x", tw.twell_dropout_add, sh, e(0, 8, dt=torch.int32), res, None, y)
    refused("residual", tw.twell_dropout_add, sh, x, e(0, 8, dt=f16), None, y)
    refused("y", tw.twell_dropout_add, sh, x, res, None, e(0, 8, dt=f16))
    refused("rng", tw.twell_dropout_add, sh, x, res, e(2, dt=torch.float64), y)


@pytest.mark.gpu
def test_product_types():
    """Types that a product takes, and others of their size."""
    def g(*size, dt):
        return e(*size, dt=dt).cuda()

    W = tw.TwellW4(g(8, 32, dt=u8), g(8, 2, dt=u8))
    y = g(3, 8, dt=f32)
    for x, xs in ((g(3, 64, dt=bf16), None), (g(3, 64, dt=u8), g(3, 2, dt=u8)), (g(3, 64, dt=e4m3), g(3, 2, dt=e8m0))):
        y.fill_(1.0)
        tw.twell_w4_matvec(x, xs, W, None, y)
        torch.cuda.synchronize()
        assert (y == 0).all()
    for dt in (f16, torch.int16):
        refused("x", tw.twell_w4_matvec, g(3, 64, dt=dt), None, W, None, y)
        refused("bias", tw.twell_w4_matvec, g(3, 64, dt=bf16), None, W, g(8, dt=dt), y)
    for dt in (torch.float8_e5m2, torch.int8):
        refused("x", tw.twell_w4_matvec, g(3, 64, dt=dt), g(3, 2, dt=u8), W, None, y)
        refused("x_scale", tw.twell_w4_matvec, g(3, 64, dt=u8), g(3, 2, dt=dt), W, None, y)


def test_layer_types():
    sh, mx = tw.ffn_shape(0, 64, 64, BF16, F32), tw.ffn_shape(0, 64, 64, MX8, F32)
    x, q, y = e(0, 64, dt=bf16), e(0, 64, dt=u8), e(0, 64, dt=f32)
    W = tw.TwellW4(e(64, 32, dt=u8), e(64, 2, dt=u8))
    refused("x", tw.twell_ffn_fwd_w4, sh, e(0, 64, dt=f16), None, W, None, W, W, y, None)
    refused("x", tw.twell_ffn_fwd_w4, mx, e(0, 64, dt=torch.int8), e(0, 2, dt=u8), W, None, W, W, y, None)
    refused("x_scale", tw.twell_ffn_fwd_w4, mx, q, e(0, 2, dt=torch.int8), W, None, W, W, y, None)
    with pytest.raises(ValueError, match="^Wg: .*on the GPU"):             # the tokens pass
        tw.twell_ffn_fwd_w4(sh, x, None, W, None, W, W, y, None)


def test_weight_types():
    for dt in (torch.int8, e4m3, torch.bool):
        with pytest.raises(ValueError):
            tw.TwellW4(e(8, 32, dt=dt), e(8, 2, dt=u8))
        with pytest.raises(ValueError):
            tw.TwellW4(e(8, 32, dt=u8), e(8, 2, dt=dt))
    tw.TwellW4(e(8, 32, dt=u8).view(torch.float4_e2m1fn_x2), e(8, 2, dt=e8m0))
    W = weights()
    object.__setattr__(W, "scales", e(8, 2, dt=torch.int8))        # what the native module is given, whatever made it
    refused("W", tw.twell_w4_matvec, e(0, 64, dt=bf16), None, W, None, e(0, 8, dt=f32))
