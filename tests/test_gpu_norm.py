"""GPU parity of the residual sum, norm and dropout calls against the float64
oracle.

Tolerances (u = 2^-24, half a step of fp32; H = half a step of the output's
dtype: 2^-8 bf16, u fp32; a row's sum of d values loses at most n u of the sum
of its terms' magnitudes, n = d / 64 + 16 additions on the longest way through
64 or more lanes):
  sum    3 u (|x / (1-p)| + |residual|) + H |sum|
  rstd   (n + 4) u, relative
  y      (n + 8) u |y| + H |y|, from the sum as stored
  dres   (n + 12) u (rstd (|dy w| + |xh| mean|dy w xh|) + |dsum|) + H |dres|
  dw     (T + 8) u sum_t |dy xh|
"""
import numpy as np
import pytest

import oracle as O

from gpu_util import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}
EPS = 1e-5
SEED, OFFSET = (123 << 33) + 77, (5 << 32) + 9


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    assert _t.cuda.is_available(), "GPU tests need a GPU"
    return _t


@pytest.fixture(scope="module")
def tw():
    import activation_sparse_feedforward_gate_amd as _tw
    _tw.lib()
    return _tw


def dts(torch, tw):
    return {"f32": (torch.float32, tw.TWELL_F32), "bf16": (torch.bfloat16, tw.TWELL_BF16)}


def values(t):
    return t.detach().to("cpu").double().numpy()


def make(torch, rng, T, d, dt, scale=1.0):
    return torch.from_numpy((scale * rng.normal(size=(T, d))).astype(np.float32)).to("cuda").to(dt)


def rng_tensor(torch):
    return torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda")


def check_sum(got, x, res, p, half):
    ref = O.dropout(x, p, SEED, OFFSET)
    mag = np.abs(ref)
    if res is not None:
        ref, mag = ref + res, mag + np.abs(res)
    assert (np.abs(got - ref) <= 3 * U * mag + half * np.abs(ref)).all()


def check_norm(y, rstd, s, w, half):
    n = s.shape[1] / 64 + 16
    _, ref, r = O.add_rmsnorm_fwd(s, None, w, EPS)
    if rstd is not None:
        assert (np.abs(rstd - r) <= (n + 4) * U * r).all()
    assert (np.abs(y - ref) <= ((n + 8) * U + half) * np.abs(ref)).all()


SIZES = [(1, 1), (1, 2304), (3, 7), (5, 64), (130, 72), (33, 513), (17, 1000), (9, 1001), (64, 2048), (40, 2304),
         (7, 4097), (5, 8192), (3, 12345), (2, 20000), (2, 32768), (1, 65536), (2, 65535), (1500, 96), (4100, 250)]


@pytest.mark.parametrize("T,d", SIZES)
def test_norm_fwd_sizes(torch, tw, T, d):
    r = np.random.default_rng(T * 7 + d)
    for xd, rd, yd, p in (("f32", "bf16", "bf16", 0.1), ("bf16", "f32", "f32", 0.0)):
        log(f"[norm fwd] T={T} d={d} {xd} {rd} {yd} p={p}")
        D = dts(torch, tw)
        x, res, w = make(torch, r, T, d, D[xd][0]), make(torch, r, T, d, D[rd][0], 3.0), make(torch, r, 1, d, D[rd][0])
        s, y = torch.empty(T, d, dtype=D[rd][0], device="cuda"), torch.empty(T, d, dtype=D[yd][0], device="cuda")
        rstd = torch.empty(T, device="cuda")
        sh = tw.norm_shape(T, d, D[xd][1], D[rd][1], D[yd][1], D[rd][1], EPS, p)
        tw.twell_add_rmsnorm_fwd(sh, x, res, w, rng_tensor(torch), s, y, None, rstd)
        check_sum(values(s), values(x), values(res), p, HALF[rd])
        check_norm(values(y), values(rstd), values(s), values(w)[0], HALF[yd])


@pytest.mark.parametrize("T,d", [(515, 40), (601, 129), (515, 257), (514, 520), (601, 1001), (513, 1032), (515, 1999),
                                 (514, 2304), (513, 2560), (515, 2567), (513, 4090), (514, 5001), (513, 9000),
                                 (513, 17000)])
def test_norm_fwd_many_rows(torch, tw, T, d):
    """Widths of every lane layout with more rows than the latency-bound calls
    have, the last workgroup partly filled."""
    test_norm_fwd_sizes(torch, tw, T, d)


@pytest.mark.parametrize("T,d", [(1283 * 16, 24), (1281 * 8 + 3, 200), (1281 * 4 + 1, 300), (1024 * 2 + 3, 1001),
                                 (768 * 2 + 1, 1999), (1030, 2304), (515, 4100), (513, 9000), (1025, 16500)])
def test_norm_bwd_many_rows(torch, tw, T, d):
    """More rows than one round of the workgroups takes, at every lane layout."""
    bwd_case(torch, tw, T, d, "f32", "bf16", "bf16", 0.1)


@pytest.mark.parametrize("xd", ["f32", "bf16"])
@pytest.mark.parametrize("rd", ["f32", "bf16"])
@pytest.mark.parametrize("yd", ["f32", "bf16", "mx8"])
def test_norm_fwd_types(torch, tw, xd, rd, yd):
    """Every dtype combination, with and without each optional argument."""
    T, d = 21, 300
    D = dts(torch, tw)
    r = np.random.default_rng(5)
    x, res, w = make(torch, r, T, d, D[xd][0]), make(torch, r, T, d, D[rd][0]), make(torch, r, 1, d, D[rd][0])
    for has_res, has_sum, has_w, p in ((1, 1, 1, 0.25), (1, 1, 0, 0.0), (0, 1, 1, 0.5), (0, 1, 1, 0.0), (0, 0, 0, 0.0),
                                       (1, 1, 1, 1.0)):
        log(f"[norm fwd] {xd} {rd} {yd} res={has_res} sum={has_sum} w={has_w} p={p}")
        s = torch.empty(T, d, dtype=D[rd][0], device="cuda") if has_sum else None
        ys = torch.empty(T, -(-d // 32), dtype=torch.uint8, device="cuda") if yd == "mx8" else None
        y = torch.empty(T, d, dtype=torch.uint8 if yd == "mx8" else D[yd][0], device="cuda")
        sh = tw.norm_shape(T, d, D[xd][1], D[rd][1], tw.TWELL_MXFP8 if yd == "mx8" else D[yd][1], D[rd][1], EPS, p)
        tw.twell_add_rmsnorm_fwd(sh, x, res if has_res else None, w if has_w else None, rng_tensor(torch) if p else None,
                                 s, y, ys)
        if has_sum:
            check_sum(values(s), values(x), values(res) if has_res else None, p, HALF[rd])
        stored = values(s) if has_sum else values(x)
        wv = values(w)[0] if has_w else None
        if yd == "mx8":
            check_mx(y.cpu().numpy(), ys.cpu().numpy(), O.add_rmsnorm_fwd(stored, None, wv, EPS)[1])
        else:
            check_norm(values(y), None, stored, wv, HALF[yd])


def check_mx(codes, scale, v):
    """Codes and scales against the values v, which the kernel holds in fp32 to
    `off`: scales are the oracle's unless the group's largest value lies within
    `off` of a border, and each value is off by half an e4m3 step (2^-4 of it,
    or 2^-10 below the smallest normal, in units of the scale)."""
    d = v.shape[1]
    off = (d / 64 + 24) * U
    want = O.mx_scale(v, 448.0)
    lo, hi = O.mx_scale(v * (1 - off), 448.0), O.mx_scale(v * (1 + off), 448.0)
    assert ((scale == want) | (scale == lo) | (scale == hi)).all()
    s = np.repeat(2.0 ** (scale.astype(np.float64) - 127), 32, axis=1)[:, :d]
    got = O.e4m3_value(codes) * s
    assert (np.abs(got - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s) + 2 * off * np.abs(v)).all()


@pytest.mark.parametrize("T,d", [(1, 2304), (1, 1), (5, 31), (6, 33), (9, 1001), (64, 2048), (3, 5000), (2, 20001),
                                 (1, 65536), (1200, 80)])
def test_norm_to_mxfp8(torch, tw, T, d):
    D = dts(torch, tw)
    r = np.random.default_rng(d)
    x = make(torch, r, T, d, torch.float32) * torch.exp(2 * make(torch, r, 1, d, torch.float32))
    x[0, : min(d, 40)] = 0.0                                    # a group of zeros
    res = make(torch, r, T, d, torch.bfloat16, 0.0)
    s, y = torch.empty_like(res), torch.empty(T, d, dtype=torch.uint8, device="cuda")
    ys = torch.full((T, -(-d // 32)), 9, dtype=torch.uint8, device="cuda")
    sh = tw.norm_shape(T, d, D["f32"][1], D["bf16"][1], tw.TWELL_MXFP8, D["bf16"][1], EPS)
    log(f"[norm mx8] T={T} d={d}")
    tw.twell_add_rmsnorm_fwd(sh, x, res, None, None, s, y, ys)
    v = O.add_rmsnorm_fwd(values(s), None, None, EPS)[1]
    check_mx(y.cpu().numpy(), ys.cpu().numpy(), v)


def test_norm_of_unusual_rows(torch, tw):
    """Rows of zeros, of one value, with infinities and NaN, and of values near
    the type's limits follow the formula in fp32."""
    D = dts(torch, tw)
    d = 96
    x = torch.ones(6, d, device="cuda")
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 40] = float("nan")
    x[3] = 1e-30
    x[4] = 3e38
    y, rstd = torch.empty_like(x), torch.empty(6, device="cuda")
    sh = tw.norm_shape(6, d, D["f32"][1], D["f32"][1], D["f32"][1], D["f32"][1], EPS)
    tw.twell_add_rmsnorm_fwd(sh, x, None, None, None, None, y, None, rstd)
    y, rstd = y.cpu(), rstd.cpu()
    assert (y[0] == 0).all() and abs(rstd[0].item() * np.sqrt(EPS) - 1) < 1e-6
    assert rstd[1] == 0 and torch.isnan(y[1, 5]) and (y[1, :5] == 0).all()
    assert torch.isnan(y[2]).all() and torch.isnan(rstd[2])
    assert torch.isfinite(y[3]).all() and rstd[4] == 0 and (y[4] == 0).all()
    codes, ys = torch.empty(6, d, dtype=torch.uint8, device="cuda"), torch.empty(6, 3, dtype=torch.uint8, device="cuda")
    sh = tw.norm_shape(6, d, D["f32"][1], D["f32"][1], tw.TWELL_MXFP8, D["f32"][1], EPS)
    tw.twell_add_rmsnorm_fwd(sh, x, None, None, None, None, codes, ys)
    codes, ys = codes.cpu().numpy(), ys.cpu().numpy()
    assert (codes[0] == 0).all() and (ys[0] == 0).all()
    assert ys[1, 0] == 255 and (ys[1, 1:] == 0).all() and (codes[1, :32] == 0x7f).all() and (codes[1, 32:] == 0).all()
    assert (ys[2] == 255).all() and (codes[2] == 0x7f).all()


def test_norm_strided_in_place(torch, tw):
    """Rows inside wider buffers at odd offsets; sum over residual; neighbours
    stay as they were."""
    D = dts(torch, tw)
    T, d = 37, 501
    r = np.random.default_rng(9)
    xb, rb = make(torch, r, T, d + 11, torch.bfloat16), make(torch, r, T, d + 7, torch.bfloat16)
    yb = torch.full((T, d + 5), 7.0, device="cuda")
    x0, r0 = values(xb), values(rb)
    x, res, y = xb[:, 3:3 + d], rb[:, 1:1 + d], yb[:, 2:2 + d]
    sh = tw.norm_shape(T, d, D["bf16"][1], D["bf16"][1], D["f32"][1], D["bf16"][1], EPS, 0.1)
    tw.twell_add_rmsnorm_fwd(sh, x, res, None, rng_tensor(torch), res, y)
    check_sum(values(res), x0[:, 3:3 + d], r0[:, 1:1 + d], 0.1, HALF["bf16"])
    check_norm(values(y), None, values(res), None, HALF["f32"])
    got = values(rb)
    assert (got[:, 0] == r0[:, 0]).all() and (got[:, d + 1:] == r0[:, d + 1:]).all() and (values(xb) == x0).all()
    assert (yb[:, :2] == 7).all() and (yb[:, d + 2:] == 7).all()


def bwd_case(torch, tw, T, d, yd, rd, xd, p, has=(1, 1, 1, 1, 1), seed=3):
    """Runs the backward; has = (dsum, w, dres, dx, dw)."""
    D = dts(torch, tw)
    r = np.random.default_rng(seed + d)
    dy, ds, s = make(torch, r, T, d, D[yd][0]), make(torch, r, T, d, D[rd][0]), make(torch, r, T, d, D[rd][0], 2.0)
    w = make(torch, r, 1, d, D[rd][0])
    rstd = torch.from_numpy(O.add_rmsnorm_fwd(values(s), None, None, EPS)[2].astype(np.float32)).cuda()
    sh = tw.norm_shape(T, d, D[xd][1], D[rd][1], D[yd][1], D[rd][1], EPS, p)
    dres = torch.full((T, d), 5.0, dtype=D[rd][0], device="cuda") if has[2] else None
    dx = torch.full((T, d), 5.0, dtype=D[xd][0], device="cuda") if has[3] else None
    dw = torch.full((d,), 5.0, device="cuda") if has[4] else None
    ws = torch.empty(max(16, tw.twell_add_rmsnorm_bwd_workspace(sh)), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    log(f"[norm bwd] T={T} d={d} {yd} {rd} {xd} p={p} {has}")
    tw.twell_add_rmsnorm_bwd(sh, dy, ds if has[0] else None, s, w if has[1] else None, rstd,
                             rng_tensor(torch) if p else None, dres, dx, dw, ws if has[4] else None)
    dyv, sv, rv = values(dy), values(s), values(rstd)
    wv = values(w)[0] if has[1] else np.ones(d)
    dsv = values(ds) if has[0] else np.zeros((T, d))
    ref, refx, refw = O.add_rmsnorm_bwd(dyv, dsv, sv, wv, rv, p, SEED, OFFSET)
    xh = sv * rv[:, None]
    n = d / 64 + 16
    mag = rv[:, None] * (np.abs(dyv * wv) + np.abs(xh) * np.abs(dyv * wv * xh).mean(axis=1, keepdims=True)) + np.abs(dsv)
    if has[2]:
        assert (np.abs(values(dres) - ref) <= (n + 12) * U * mag + HALF[rd] * np.abs(ref)).all()
    if has[3]:
        kept = O.dropout_keep(T, d, p, SEED, OFFSET) / max(1 - np.rint(p * 65536) / 65536, 1e-9) if p else 1.0
        assert (np.abs(values(dx) - refx) <= kept * (n + 14) * U * mag + HALF[xd] * np.abs(refx)).all()
    if has[4]:
        assert (np.abs(values(dw) - refw) <= (T + 8) * U * np.abs(dyv * xh).sum(axis=0)).all()


@pytest.mark.parametrize("T,d", SIZES + [(3000, 1024)])
def test_norm_bwd_sizes(torch, tw, T, d):
    bwd_case(torch, tw, T, d, "f32", "bf16", "bf16", 0.1)
    bwd_case(torch, tw, T, d, "bf16", "f32", "f32", 0.0)


@pytest.mark.parametrize("yd", ["f32", "bf16"])
@pytest.mark.parametrize("rd", ["f32", "bf16"])
@pytest.mark.parametrize("xd", ["f32", "bf16"])
def test_norm_bwd_types(torch, tw, yd, rd, xd):
    for has, p in (((1, 1, 1, 1, 1), 0.25), ((0, 1, 1, 0, 1), 0.0), ((1, 0, 0, 1, 0), 0.5), ((0, 0, 1, 1, 1), 1.0)):
        bwd_case(torch, tw, 23, 304, yd, rd, xd, p, has)


def test_norm_bwd_without_rows_clears_dw(torch, tw):
    sh = tw.norm_shape(0, 100, 0, 0, 0, 0, EPS)
    e, dw = torch.empty(0, 100, device="cuda"), torch.full((100,), 3.0, device="cuda")
    tw.twell_add_rmsnorm_bwd(sh, e, None, e, None, torch.empty(0, device="cuda"), None, e, None, dw, None)
    assert (dw == 0).all()


def test_norm_grad_by_differences(torch, tw):
    """Central differences of the GPU forward in fp32 against its backward.
    The oracle's quotient at the same step h takes the truncation out, so what
    is left is the forward's rounding, 2 * 24 u sum|terms| / (2 h)."""
    T, d, p, h = 4, 96, 0.25, 2.0 ** -6
    r = np.random.default_rng(1)
    x, res, w, dy, ds, dirx, dirr = (make(torch, r, T, d, torch.float32) for _ in range(7))
    w, rng = w[:1].contiguous(), rng_tensor(torch)
    sh = tw.norm_shape(T, d, 0, 0, 0, 0, EPS, p)

    def fwd(x, res):
        s, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
        tw.twell_add_rmsnorm_fwd(sh, x, res, w, rng, s, y, None, rstd)
        return s, y, rstd

    def loss(x, res):
        s, y, _ = fwd(x, res)
        return (values(y) * values(dy)).sum() + (values(s) * values(ds)).sum()

    def loss64(x, res):
        s, y, _ = O.add_rmsnorm_fwd(x, res, values(w)[0], EPS, p, SEED, OFFSET)
        return (y * values(dy)).sum() + (s * values(ds)).sum()

    s, y, rstd = fwd(x, res)
    dres, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(tw.twell_add_rmsnorm_bwd_workspace(sh), dtype=torch.uint8, device="cuda")
    tw.twell_add_rmsnorm_bwd(sh, dy, ds, s, w, rstd, rng, dres, dx, dw, ws)
    slope = (values(dx) * values(dirx)).sum() + (values(dres) * values(dirr)).sum()
    up, dn = (x + h * dirx, res + h * dirr), (x - h * dirx, res - h * dirr)
    q = (loss(*up) - loss(*dn)) / (2 * h)
    q64 = (loss64(*(values(v) for v in up)) - loss64(*(values(v) for v in dn))) / (2 * h)
    terms = (np.abs(values(y) * values(dy)) + np.abs(values(s) * values(ds))).sum()
    assert abs(q - q64) <= 24 * U * terms * 2 / h
    # O(h^2) of the oracle's own quotient, from its value at h / 2
    up, dn = (x + h / 2 * dirx, res + h / 2 * dirr), (x - h / 2 * dirx, res - h / 2 * dirr)
    q2 = (loss64(*(values(v) for v in up)) - loss64(*(values(v) for v in dn))) / h
    assert abs(q64 - slope) <= 2 * abs(q64 - q2) + 64 * U * terms / h


@pytest.mark.parametrize("xd,rd,yd", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"),
                                      ("bf16", "f32", "bf16"), ("bf16", "bf16", "f32"), ("f32", None, "bf16"),
                                      ("f32", "bf16", "f32"), ("bf16", "f32", "f32"), ("bf16", None, "f32")])
@pytest.mark.parametrize("T,d", [(1, 1), (33, 1001), (5, 9000), (2100, 64)])
def test_dropout_add(torch, tw, T, d, xd, rd, yd):
    D = dts(torch, tw)
    r = np.random.default_rng(d)
    x, res = make(torch, r, T, d, D[xd][0]), make(torch, r, T, d, D[rd][0]) if rd else None
    for p in (0.0, 2.0 ** -16, 0.3, 1.0):
        y = torch.empty(T, d, dtype=D[yd][0], device="cuda")
        sh = tw.norm_shape(T, d, D[xd][1], D[rd or "f32"][1], D[yd][1], 0, 0.0, p)
        tw.twell_dropout_add(sh, x, res, rng_tensor(torch) if p else None, y)
        check_sum(values(y), values(x), values(res) if rd else None, p, HALF[yd])


def test_dropped_values_are_zero_whatever_they_were(torch, tw):
    T, d, p = 8, 64, 0.5
    x = torch.full((T, d), float("nan"), device="cuda")
    y = torch.empty_like(x)
    tw.twell_dropout_add(tw.norm_shape(T, d, 0, 0, 0, 0, 0.0, p), x, None, rng_tensor(torch), y)
    keep = O.dropout_keep(T, d, p, SEED, OFFSET)
    got = y.cpu().numpy()
    assert np.isnan(got[keep]).all() and (got[~keep] == 0).all()


def test_dropout_is_its_own_backward_in_place(torch, tw):
    """y = dropout(x) with a weight on every value: the gradient of sum(g y) is
    dropout(g), here written over g."""
    T, d, p = 61, 333, 0.25
    r = np.random.default_rng(2)
    g = make(torch, r, T, d, torch.float32)
    g0 = values(g)
    tw.twell_dropout_add(tw.norm_shape(T, d, 0, 0, 0, 0, 0.0, p), g, None, rng_tensor(torch), g)
    check_sum(values(g), g0, None, p, U)


def test_offsets_beyond_32_bits(torch, tw):
    """More than 2^31 elements: the last rows are normed and dropped as any."""
    T, d = 33000, 65536
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    r = np.random.default_rng(0)
    x[-3:] = make(torch, r, 3, d, torch.bfloat16)
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    sh = tw.norm_shape(T, d, 1, 1, 1, 1, EPS)
    tw.twell_add_rmsnorm_fwd(sh, x, None, None, None, None, y, None, rstd)
    check_norm(values(y[-4:]), values(rstd[-4:]), values(x[-4:]), None, HALF["bf16"])
    assert (y[0] == 1).all()
    sh = tw.norm_shape(T, d, 1, 1, 1, 1, EPS, 0.5)
    tw.twell_dropout_add(sh, x, None, rng_tensor(torch), y)
    blocks = np.arange((T - 1) * (d // 8), T * (d // 8), dtype=np.uint64)
    w = O.philox4x32_10([blocks & np.uint64(0xFFFFFFFF), blocks >> np.uint64(32),
                         np.full_like(blocks, OFFSET & 0xFFFFFFFF), np.full_like(blocks, OFFSET >> 32)],
                        [SEED & 0xFFFFFFFF, SEED >> 32])
    half = np.stack([v for k in w for v in (k & np.uint64(0xFFFF), k >> np.uint64(16))], axis=1).reshape(-1)
    want = np.where(half >= 32768, 2 * values(x[-1]), 0.0)
    assert (values(y[-1]) == want).all()


def test_norm_on_another_stream_and_in_a_graph(torch, tw):
    """Forward and backward on a side stream, then captured into a graph and
    replayed with other inputs and random state."""
    T, d, p = 50, 520, 0.25
    r = np.random.default_rng(6)
    sh = tw.norm_shape(T, d, 0, 1, 1, 1, EPS, p)
    shb = tw.norm_shape(T, d, 0, 1, 0, 1, EPS, p)
    x, dy = make(torch, r, T, d, torch.float32), make(torch, r, T, d, torch.float32)
    res, w = make(torch, r, T, d, torch.bfloat16), make(torch, r, 1, d, torch.bfloat16)
    rng = rng_tensor(torch)
    s, y, rstd = torch.empty_like(res), torch.empty_like(res), torch.empty(T, device="cuda")
    dres, dx, dw = torch.empty_like(res), torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(tw.twell_add_rmsnorm_bwd_workspace(shb), dtype=torch.uint8, device="cuda")
    out = (s, y, rstd, dres, dx, dw)

    def step(stream=None):
        tw.twell_add_rmsnorm_fwd(sh, x, res, w, rng, s, y, None, rstd, stream)
        tw.twell_add_rmsnorm_bwd(shb, dy, res, s, w, rstd, rng, dres, dx, dw, ws, stream)

    step()
    torch.cuda.synchronize()
    eager = [t.clone() for t in out]
    for t in out:
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        x.copy_(make(torch, r, T, d, torch.float32))
        rng[1] += 1
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, got)), k


@pytest.mark.parametrize("T,d", [(1024, 40), (1025, 40), (1024, 4096), (1024, 4104), (1025, 5000), (1024, 8), (65, 1003)])
def test_norm_bwd_both_ways_to_dw(torch, tw, T, d):
    """Sizes on both sides of the rule that takes dw from workgroups of its own."""
    bwd_case(torch, tw, T, d, "f32", "bf16", "bf16", 0.1)
    bwd_case(torch, tw, T, d, "bf16", "f32", "f32", 0.0)


@pytest.mark.parametrize("T,d", [(70, 1003), (1100, 45)])
def test_norm_bwd_strided_and_in_place(torch, tw, T, d):
    """Rows inside wider buffers and dres written over dsum: the same bits as
    from rows side by side."""
    r = np.random.default_rng(11)
    sh = tw.norm_shape(T, d, 1, 1, 0, 1, EPS, 0.25)
    dy, ds, s = (make(torch, r, T, d, t) for t in (torch.float32, torch.bfloat16, torch.bfloat16))
    w, rstd, rng = make(torch, r, 1, d, torch.bfloat16), torch.rand(T, device="cuda") + 0.5, rng_tensor(torch)
    ws = torch.empty(tw.twell_add_rmsnorm_bwd_workspace(sh), dtype=torch.uint8, device="cuda")

    def wide(t, at, more):
        b = torch.full((T, d + more), 7.0, dtype=t.dtype, device="cuda")
        b[:, at:at + d] = t
        return b, b[:, at:at + d]

    got = []
    for strided in (False, True):
        log(f"[norm bwd strided] T={T} d={d} strided={strided}")
        (yb, y), (db, dres), (sb, sv), (xb, dx) = ((t, t) if not strided else wide(t, at, more) for t, at, more in (
            (dy, 3, 8), (ds.clone(), 1, 3), (s, 5, 6), (torch.zeros_like(ds), 2, 9)))
        dw = torch.empty(d, device="cuda")
        tw.twell_add_rmsnorm_bwd(sh, y, dres, sv, w, rstd, rng, dres, dx, dw, ws)
        got.append((dres.clone(), dx.clone(), dw))
        if strided:
            assert (db[:, :1] == 7).all() and (db[:, 1 + d:] == 7).all()
            assert (xb[:, :2] == 7).all() and (xb[:, 2 + d:] == 7).all()
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,d", [(1024, 9), (130, 1009), (1000, 2041), (300, 2500)])
def test_norm_bwd_fp32_columns_of_dw(torch, tw, T, d):
    bwd_case(torch, tw, T, d, "f32", "f32", "f32", 0.1)
