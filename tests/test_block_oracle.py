"""The oracle of the operators around the layer, pinned on the CPU: published
known answers of the random generator, formats by brute force, gradients by
central differences; and the host-side refusals of those operators' entry
points, which need no GPU."""
import ctypes

import numpy as np
import pytest

import activation_sparse_feedforward_gate_amd as tw
import oracle as O

F32, BF16, MX8 = tw.TWELL_F32, tw.TWELL_BF16, tw.TWELL_MXFP8


# ---------------------------------------------------------------- generator and formats

@pytest.mark.parametrize("counter,key,words", [
    ([0] * 4, [0] * 2, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]),
])
def test_philox_known_answers(counter, key, words):
    assert [int(v) for v in O.philox4x32_10(counter, key)] == words


def test_dropout_rate_and_scale():
    x = np.ones((400, 501))
    y = O.dropout(x, 0.25, seed=(7 << 40) + 3, offset=5)
    n = x.size
    assert abs((y == 0).mean() - 0.25) < 5 * np.sqrt(0.25 * 0.75 / n)
    assert set(np.unique(y)) == {0.0, 1 / 0.75}
    assert (O.dropout(x, 0.25, seed=(7 << 40) + 3, offset=6) != y).any()
    assert (O.dropout(x, 1.0, seed=1, offset=0) == 0).all()
    assert (O.dropout(x, 0.0) == x).all()


def test_e4m3_round_is_nearest():
    table = np.unique(O.e4m3_value(np.arange(128))[:127])
    assert table[0] == 0 and table[-1] == 448 and len(table) == 127
    v = np.random.default_rng(0).uniform(-448, 448, 4000) * 2.0 ** -np.random.default_rng(1).integers(0, 18, 4000)
    got = O.e4m3_round(v)
    best = np.abs(np.abs(v)[:, None] - table).min(axis=1)
    np.testing.assert_allclose(np.abs(np.abs(v) - np.abs(got)), best, rtol=0, atol=0)
    assert np.isin(np.abs(got), table).all()


@pytest.mark.parametrize("top", [448.0, 6.0])
def test_mx_scale_is_smallest(top):
    g = np.random.default_rng(2).normal(size=(50, 70)) * 2.0 ** np.random.default_rng(3).integers(-140, 120, (50, 1))
    g[0] = 0
    g[1, :32] = top * 2.0 ** 3            # exactly representable top
    g[2, 5] = np.inf
    s = O.mx_scale(g, top)
    pad = np.zeros((50, 96))
    pad[:, :70] = np.abs(g)
    m = pad.reshape(50, 3, 32).max(axis=2)
    assert s[2, 0] == 255 and (s[0] == 0).all() and s[1, 0] == 130
    fin = np.isfinite(m)
    assert (m[fin] <= top * 2.0 ** (s[fin] - 127.0)).all()
    more = fin & (s > 0)
    assert (m[more] > top * 2.0 ** (s[more] - 128.0)).all()


def test_mxfp4_values():
    codes = np.arange(16)
    assert list(O.e2m1_value(codes)) == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    w = np.zeros((1, 32))
    w[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5]      # ties go to the even code
    c, s = O.mxfp4(w)
    assert s[0, 0] == 127
    assert list(c[0, :9]) == [7, 0, 2, 2, 4, 4, 6, 6, 14]
    assert list(O.mxfp4_value(c, s)[0, :9]) == [6, 0, 1, 1, 2, 2, 4, 4, -4]


def test_rmsnorm_gradients_by_differences():
    r = np.random.default_rng(4)
    T, d, eps, p, h = 3, 10, 1e-3, 0.25, 1e-5
    x, res, w, dy, ds = (r.normal(size=s) for s in ((T, d), (T, d), (d,), (T, d), (T, d)))

    def loss(x, res, w):
        s, y, _ = O.add_rmsnorm_fwd(x, res, w, eps, p, 11, 12)
        return (y * dy).sum() + (s * ds).sum()

    s, _, rstd = O.add_rmsnorm_fwd(x, res, w, eps, p, 11, 12)
    dres, dx, dw = O.add_rmsnorm_bwd(dy, ds, s, w, rstd, p, 11, 12)
    for v, g, at in ((x, dx, 0), (res, dres, 1), (w, dw, 2)):
        for i in np.ndindex(v.shape):
            a = [x.copy(), res.copy(), w.copy()]
            a[at][i] += h
            up = loss(*a)
            a[at][i] -= 2 * h
            # central differences: O(h^2) truncation and 2^-53 / h rounding of a loss of about 30
            assert abs((up - loss(*a)) / (2 * h) - g[i]) < 1e-7


# ---------------------------------------------------------------- refusals of the norm and dropout calls

A = 4096          # any aligned address: nothing is launched in these tests


def _fwd(sh, **k):
    a = dict(x=A, ldx=64, res=A, ldres=64, w=A, rng=A, sum=A, ldsum=64, y=A, ldy=64, ys=None, rstd=A)
    a.update(k)
    return tw.lib().twell_add_rmsnorm_fwd(sh, a["x"], a["ldx"], a["res"], a["ldres"], a["w"], a["rng"], a["sum"],
                                          a["ldsum"], a["y"], a["ldy"], a["ys"], a["rstd"], None)


def _bwd(sh, **k):
    a = dict(dy=A, lddy=64, ds=A, ldds=64, sum=A, ldsum=64, w=A, rstd=A, rng=A, dres=A, lddres=64, dx=A, lddx=64,
             dw=A, ws=A, wsb=1 << 30)
    a.update(k)
    return tw.lib().twell_add_rmsnorm_bwd(sh, a["dy"], a["lddy"], a["ds"], a["ldds"], a["sum"], a["ldsum"], a["w"],
                                          a["rstd"], a["rng"], a["dres"], a["lddres"], a["dx"], a["lddx"], a["dw"],
                                          a["ws"], a["wsb"], None)


def _drop(sh, **k):
    a = dict(x=A, ldx=64, res=A, ldres=64, rng=A, y=A, ldy=64)
    a.update(k)
    return tw.lib().twell_dropout_add(sh, a["x"], a["ldx"], a["res"], a["ldres"], a["rng"], a["y"], a["ldy"], None)


def _shape(**k):
    a = dict(T=8, d=64, x_dt=F32, res_dt=BF16, y_dt=BF16, w_dt=BF16, eps=1e-6, p=0.1)
    a.update(k)
    return tw.norm_shape(**a)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(d=0), dict(d=-3), dict(x_dt=MX8), dict(res_dt=7), dict(w_dt=MX8),
                                 dict(y_dt=3), dict(p=-0.1), dict(p=1.5), dict(p=float("nan")), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(eps=float("inf"))])
def test_bad_norm_shapes(bad):
    for f in (_fwd, _bwd, _drop):
        assert f(_shape(**bad)) == tw.TWELL_EINVAL
    if bad != dict(T=-1):
        assert tw.twell_last_error()
    assert tw.twell_add_rmsnorm_bwd_workspace(_shape(**bad)) == 0


def test_norm_refusals():
    L = tw.lib()
    sh = _shape()
    assert _fwd(None) == _bwd(None) == _drop(None) == tw.TWELL_EINVAL
    for f in (_fwd, _bwd, _drop):
        assert f(_shape(d=65537)) == tw.TWELL_EUNSUPPORTED
        assert f(sh, rng=None) == tw.TWELL_EINVAL
        assert b"rng" in L.twell_last_error()
        assert f(sh, rng=A + 4) == tw.TWELL_EINVAL
    for k in (dict(x=None), dict(y=None), dict(sum=None), dict(x=A + 2), dict(res=A + 1), dict(y=A + 1), dict(w=A + 1),
              dict(ldx=63), dict(ldres=63), dict(ldsum=0), dict(ldy=-64), dict(rstd=A + 2), dict(ys=A)):
        assert _fwd(sh, **k) == tw.TWELL_EINVAL, k
    assert _fwd(_shape(y_dt=MX8)) == tw.TWELL_EINVAL                        # scales missing
    assert _bwd(_shape(y_dt=MX8)) == tw.TWELL_EINVAL
    assert _drop(_shape(y_dt=MX8)) == tw.TWELL_EINVAL
    for k in (dict(dy=None), dict(sum=None), dict(rstd=None), dict(dres=None, dx=None), dict(lddy=63), dict(ldds=1),
              dict(ldsum=63), dict(lddres=63), dict(lddx=63), dict(dy=A + 1), dict(dx=A + 2), dict(dw=A + 2),
              dict(ws=A + 8)):
        assert _bwd(sh, **k) == tw.TWELL_EINVAL, k
    need = tw.twell_add_rmsnorm_bwd_workspace(sh)
    assert need > 0
    assert _bwd(sh, wsb=need - 1) == tw.TWELL_EWORKSPACE
    assert _bwd(sh, ws=None) == tw.TWELL_EWORKSPACE
    for k in (dict(x=None), dict(y=None), dict(ldx=63), dict(ldres=63), dict(ldy=63), dict(x=A + 1), dict(y=A + 1)):
        assert _drop(sh, **k) == tw.TWELL_EINVAL, k


def test_norm_without_rows_launches_nothing():
    sh = _shape(T=0)
    assert _fwd(sh, x=None, y=None) == _drop(sh, x=None, y=None) == tw.TWELL_OK
    assert _bwd(sh, dy=None, sum=None, rstd=None, dres=None, dx=None, dw=None, ws=None, wsb=0) == tw.TWELL_OK


def test_binding_checks_tensors():
    """The binding refuses tensors whose shape, element size or column stride
    differ from the shape struct's before it passes a pointer on."""
    import torch
    sh = tw.norm_shape(4, 8, F32, F32, F32, F32)
    ok = torch.zeros(4, 8)
    for bad in (torch.zeros(4, 9), torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 4).t(),
                torch.zeros(4, 16)[:, ::2]):
        for pos in range(2):
            args = [ok, ok]
            args[pos] = bad
            with pytest.raises(ValueError):
                tw.twell_dropout_add(sh, args[0], None, None, args[1])
    with pytest.raises(ValueError):
        tw.twell_dropout_add(sh, ok, None, torch.zeros(3, dtype=torch.int64), ok)
    assert isinstance(sh, ctypes.Structure)
