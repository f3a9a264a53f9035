"""Host-side refusals of the calls on 4-bit weights and their binding; nothing
is launched, so no GPU is needed."""
import ctypes

import pytest

import activation_sparse_feedforward_gate_amd as tw

F32, BF16, MX8 = tw.TWELL_F32, tw.TWELL_BF16, tw.TWELL_MXFP8
A = 4096          # any aligned address


def _w(N=64, K=64, codes=A, scales=A):
    return tw.c_twell_w4(N, K, codes, scales)


def _matvec(W, **k):
    a = dict(T=2, x=A, dt=BF16, ldx=64, xs=None, bias=A, y=A, ydt=F32, ldy=64)
    a.update(k)
    return tw.lib().twell_w4_matvec(a["T"], a["x"], a["dt"], a["ldx"], a["xs"],
                                    ctypes.byref(W) if W is not None else None, a["bias"], a["y"], a["ydt"], a["ldy"],
                                    None)


def test_matvec_refusals():
    E, UN = tw.TWELL_EINVAL, tw.TWELL_EUNSUPPORTED
    assert _matvec(None) == E
    for w in (_w(N=0), _w(N=-1), _w(K=0), _w(K=-32), _w(codes=None), _w(scales=None), _w(codes=A + 8)):
        assert _matvec(w) == E
    assert _matvec(_w(K=48), ldx=48) == UN and _matvec(_w(K=33)) == UN
    for k in (dict(T=-1), dict(x=None), dict(y=None), dict(dt=F32), dict(dt=9), dict(dt=MX8), dict(xs=A), dict(ydt=MX8),
              dict(ydt=5), dict(ldx=63), dict(ldy=63), dict(ldx=-64), dict(x=A + 1), dict(y=A + 2), dict(bias=A + 1),
              dict(ydt=BF16, y=A + 1)):
        assert _matvec(_w(), **k) == E, k
    assert tw.twell_last_error()
    assert _matvec(_w(), T=0, x=None, y=None) == tw.TWELL_OK


def _ffn(sh, **k):
    a = dict(x=A, xs=None, Wg=_w(128, 64), bg=A, Wu=_w(128, 64), Wd=_w(128, 64), y=A, ws=A, wsb=1 << 30)
    a.update(k)

    def p(w):
        return ctypes.byref(w) if w is not None else None
    return tw.lib().twell_ffn_fwd_w4(sh, a["x"], a["xs"], p(a["Wg"]), a["bg"], p(a["Wu"]), p(a["Wd"]), a["y"], a["ws"],
                                     a["wsb"], None)


def _sh(T=2, d=64, F=128, in_dt=BF16, out_dt=F32):
    return tw.ffn_shape(T, d, F, in_dt, out_dt)


def test_layer_refusals():
    E, UN = tw.TWELL_EINVAL, tw.TWELL_EUNSUPPORTED
    assert _ffn(None) == E
    for bad in (_sh(T=-1), _sh(d=0), _sh(F=-64), _sh(in_dt=F32), _sh(in_dt=7), _sh(out_dt=MX8), _sh(out_dt=4)):
        assert _ffn(bad) == E and tw.twell_ffn_fwd_w4_workspace(bad) == 0
    for bad in (_sh(d=96), _sh(F=100), _sh(T=1 << 25), _sh(T=1 << 20, F=2048), _sh(d=1 << 16, F=1 << 15)):
        assert _ffn(bad) == UN and tw.twell_ffn_fwd_w4_workspace(bad) == 0
    sh = _sh()
    for k in (dict(x=None), dict(y=None), dict(xs=A), dict(Wg=None), dict(Wu=None), dict(Wd=None), dict(x=A + 1),
              dict(y=A + 2), dict(bg=A + 1), dict(Wg=_w(64, 64)), dict(Wu=_w(128, 128)), dict(Wd=_w(64, 128)),
              dict(Wd=_w(128, 64, codes=None)), dict(Wu=_w(128, 64, codes=A + 4)), dict(ws=A + 8)):
        assert _ffn(sh, **k) == E, k
    assert _ffn(_sh(in_dt=MX8)) == E                                         # scales missing
    need = tw.twell_ffn_fwd_w4_workspace(sh)
    assert need > 0
    assert _ffn(sh, wsb=need - 1) == _ffn(sh, ws=None) == tw.TWELL_EWORKSPACE
    assert _ffn(_sh(T=0), x=None, y=None, ws=None, wsb=0) == tw.TWELL_OK
    assert tw.twell_ffn_fwd_w4_workspace(_sh(T=0)) == 0


def test_the_layer_on_dense_weights_refuses_mxfp8():
    sh = _sh(in_dt=MX8)
    L = tw.lib()
    assert L.twell_ffn_fwd(ctypes.byref(sh), A, A, None, A, A, A, None, -1, A, 1 << 30, None) == tw.TWELL_EINVAL
    assert tw.twell_ffn_fwd_workspace(sh) == 0
    sh = _sh(out_dt=MX8)
    assert L.twell_ffn_fwd(ctypes.byref(sh), A, A, None, A, A, A, None, -1, A, 1 << 30, None) == tw.TWELL_EINVAL


def test_binding_checks_tensors():
    import torch
    u8 = torch.uint8
    codes, scales = torch.zeros(8, 32, dtype=u8), torch.zeros(8, 2, dtype=u8)
    W = tw.TwellW4(codes, scales)
    assert (W.N, W.K) == (8, 64)
    for c, s in ((codes[:, :16], scales), (codes, torch.zeros(7, 2, dtype=u8)), (codes, torch.zeros(8, 3, dtype=u8)),
                 (codes.float(), scales), (codes, torch.zeros(16, dtype=u8))):
        with pytest.raises(ValueError):
            tw.TwellW4(c, s)
    x, y, b = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(3, 8), torch.zeros(8, dtype=torch.bfloat16)
    q, qs = torch.zeros(3, 64, dtype=u8), torch.zeros(3, 2, dtype=u8)
    for args in ((x.float(), None, W, b, y), (x[:, :32], None, W, b, y), (x, qs, W, b, y), (q, None, W, b, y),
                 (q, qs[:2], W, b, y), (x, None, W, b[:7], y), (x, None, W, b.float(), y), (x, None, W, b, y[:2]),
                 (x, None, W, b, torch.zeros(3, 9)), (x, None, W, b, torch.zeros(8, 3).t())):
        with pytest.raises(ValueError):
            tw.twell_w4_matvec(*args)
    with pytest.raises(TypeError):
        tw.twell_w4_matvec(x, None, W, b, y.double())


def test_matvec_refuses_rows_past_32_bit_offsets():
    assert _matvec(_w(K=1 << 30), ldx=1 << 30) == tw.TWELL_EUNSUPPORTED


def test_no_tokens_is_no_error_in_either_type():
    """A tensor of no elements has no address; nothing is read or written."""
    for k in (dict(dt=BF16), dict(dt=MX8), dict(dt=MX8, xs=A)):
        assert _matvec(_w(), T=0, x=None, y=None, **k) == tw.TWELL_OK, k
    assert _matvec(_w(), T=0, x=None, y=None, dt=F32) == tw.TWELL_EINVAL     # a type that no product takes
