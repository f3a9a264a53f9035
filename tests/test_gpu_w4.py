"""GPU parity of the products with MXFP4 weights and of the layer on them
against the float64 oracle.

Tolerances (u = 2^-24; H = half a step of y's dtype: 2^-8 bf16, u fp32; the
matrix instructions may cut rather than round a partial sum, so an addition
counts 2 u; operands are exact in every format):
  product  (2 K + 4) u (sum |x w| + |bias|) + H |y|
  layer    eg, eu: the same for the gate and up products;
           ea = eg (|u| + eu) + h eu + u |a|;
           sum ea |wd| + (2 F + 4) u sum (|a| + ea) |wd| + H |y|
"""
import numpy as np
import pytest

import oracle as O

from gpu_util import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}


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


def values(t):
    return t.detach().to("cpu").double().numpy()


def make_w(torch, tw, r, N, K, std=1.0):
    """Random codes with scales of a normal weight's spread: (TwellW4, values)."""
    codes = r.integers(0, 16, (N, K))
    scale = (np.round(np.log2(std / 3)) + r.integers(-1, 2, (N, K // 32)) + 127).astype(np.uint8)
    return pack_w(torch, tw, codes, scale)


def pack_w(torch, tw, codes, scale):
    b = torch.from_numpy((codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)).cuda()
    return tw.TwellW4(b, torch.from_numpy(scale).cuda()), O.mxfp4_value(codes, scale)


def make_x(torch, r, T, K, kind):
    """(x, x_scale, values)."""
    if kind == "bf16":
        x = torch.from_numpy(r.normal(size=(T, K)).astype(np.float32)).bfloat16()
        return x.cuda(), None, values(x)
    codes = r.integers(0, 256, (T, K)).astype(np.uint8)
    codes[(codes & 127) == 127] = 0
    scale = r.integers(118, 122, (T, K // 32)).astype(np.uint8)
    v = O.e4m3_value(codes) * np.repeat(O.e8m0_value(scale), 32, axis=1)
    return torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda(), v


def out(torch, T, N, yd):
    return torch.full((T, N), 7.0, dtype=torch.float32 if yd == "f32" else torch.bfloat16, device="cuda")


def check_product(y, x, w, bias, yd):
    ref = x @ w.T + (0 if bias is None else bias)
    mag = np.abs(x) @ np.abs(w).T + (0 if bias is None else np.abs(bias))
    err = np.abs(y - ref)
    assert (err <= (2 * x.shape[1] + 4) * U * mag + HALF[yd] * np.abs(ref)).all(), float(err.max())


@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (1, 16, 128), (2, 17, 32), (3, 5, 96), (1, 9216, 2304), (1, 2049, 4128),
                                   (4, 300, 160), (15, 63, 1024), (16, 4001, 2048), (17, 130, 224), (33, 1000, 512),
                                   (48, 64, 544), (64, 515, 2304), (65, 40, 256), (131, 100, 128), (7, 257, 16384),
                                   (64, 20011, 256), (32, 9001, 320)])
@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_matvec(torch, tw, T, N, K, kind):
    r = np.random.default_rng(T * 1000 + N + K)
    W, w = make_w(torch, tw, r, N, K, K ** -0.5)
    x, xs, xv = make_x(torch, r, T, K, kind)
    bias = torch.from_numpy(r.normal(size=N).astype(np.float32)).bfloat16().cuda()
    for yd, b in (("f32", bias), ("bf16", None)):
        log(f"[w4 matvec] T={T} N={N} K={K} {kind} {yd}")
        y = out(torch, T, N, yd)
        tw.twell_w4_matvec(x, xs, W, b, y)
        check_product(values(y), xv, w, None if b is None else values(b), yd)


@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_matvec_strided(torch, tw, kind):
    """x and y inside wider buffers at odd offsets; neighbours stay."""
    r = np.random.default_rng(3)
    for T, N, K in ((5, 37, 160), (20, 130, 256)):
        W, w = make_w(torch, tw, r, N, K)
        x, xs, xv = make_x(torch, r, T, K, kind)
        xb = torch.zeros(T, K + 13, dtype=x.dtype, device="cuda")
        xb[:, 3:3 + K] = x
        for yd in ("f32", "bf16"):
            log(f"[w4 matvec strided] T={T} {kind} {yd}")
            yb = out(torch, T, N + 9, yd)
            tw.twell_w4_matvec(xb[:, 3:3 + K], xs, W, None, yb[:, 5:5 + N])
            got = values(yb)
            check_product(got[:, 5:5 + N], xv, w, None, yd)
            assert (got[:, :5] == 7).all() and (got[:, 5 + N:] == 7).all()


def test_matvec_every_code_and_scale(torch, tw):
    """One weight row per code and one per scale byte, against one-hot tokens:
    single products, exact in fp32."""
    K = 256
    codes = np.zeros((16 + 256, K), dtype=np.int64)
    scale = np.full((16 + 256, K // 32), 127, dtype=np.uint8)
    for c in range(16):
        codes[c] = c
    codes[16:, :] = 2                       # 1.0
    scale[16:, :] = np.arange(256)[:, None]
    W, w = pack_w(torch, tw, codes, scale)
    for kind in ("bf16", "mx8"):
        log(f"[w4 codes] {kind}")
        for k in (0, 31, 32, 77, 255):
            x = torch.zeros(2, K, dtype=torch.bfloat16, device="cuda")
            x[0, k], x[1, k] = 1.0, -2.0
            if kind == "bf16":
                y = out(torch, 2, 272, "f32")
                tw.twell_w4_matvec(x, None, W, None, y)
            else:
                q = torch.zeros(2, K, dtype=torch.uint8, device="cuda")
                q[0, k], q[1, k] = 0x38, 0xc0
                y = out(torch, 2, 272, "f32")
                tw.twell_w4_matvec(q, torch.full((2, K // 32), 127, dtype=torch.uint8, device="cuda"), W, None, y)
            got = values(y)
            assert (got[0, :16] == w[:16, k]).all() and (got[1, :16] == -2 * w[:16, k]).all()
            # 2^-127 .. 2^127 and NaN; the smallest may be flushed with the fp32 subnormals
            assert (got[0, 18:271] == 2.0 ** (np.arange(2, 255) - 127.0)).all()
            assert np.isnan(got[:, 271]).all() and (np.abs(got[0, 16:18]) <= 2.0 ** -126).all()


def test_matvec_token_scales(torch, tw):
    """Every scale byte of an MXFP8 token against weights of one."""
    K = 8192
    W, _ = pack_w(torch, tw, np.full((3, K), 2), np.full((3, K // 32), 127, dtype=np.uint8))
    x = torch.zeros(256, K, dtype=torch.uint8, device="cuda")
    s = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(256, 1)
    for t in range(256):
        x[t, 32 * t + t % 32] = 0x3a                      # 1.25
    y = out(torch, 256, 3, "f32")
    log("[w4 token scales]")
    tw.twell_w4_matvec(x, s, W, None, y)
    got = values(y)
    assert np.isnan(got).all()                           # 0 * NaN of the last block's scale
    s[:, 255] = 127
    s[255, 255] = 255
    tw.twell_w4_matvec(x, s, W, None, y)
    got = values(y)
    assert (got[3:255] == (1.25 * 2.0 ** (np.arange(3, 255) - 127.0))[:, None]).all() and np.isnan(got[255]).all()


@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_bad_values_stay_in_their_row(torch, tw, kind):
    """A NaN token, or a NaN weight scale, reaches its own row or column only."""
    r = np.random.default_rng(8)
    T, N, K = 19, 70, 352
    W, w = make_w(torch, tw, r, N, K)
    x, xs, xv = make_x(torch, r, T, K, kind)
    if kind == "bf16":
        x[4, 340] = float("nan")
        x[17, 0] = float("inf")
    else:
        x[4, 340] = 0x7f
        xs[17, 0] = 255
    W.scales[33, 10] = 255
    y = out(torch, T, N, "f32")
    log(f"[w4 nan] {kind}")
    tw.twell_w4_matvec(x, xs, W, None, y)
    got = values(y)
    assert np.isnan(got[4]).all() and np.isnan(got[:, 33]).all() and not np.isfinite(got[17]).any()
    t, n = np.setdiff1d(np.arange(T), [4, 17]), np.setdiff1d(np.arange(N), [33])
    check_product(got[np.ix_(t, n)], xv[t], w[n], None, "f32")


def test_weights_beyond_32_bits(torch, tw):
    """More than 2^31 bytes of codes: the last rows are read as any."""
    N, K = 280000, 16384
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    codes[-20:] = torch.randint(0, 256, (20, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.full((N, K // 32), 120, dtype=torch.uint8, device="cuda")
    c = codes[-20:].cpu().numpy().astype(np.int64)
    full = np.stack((c & 15, c >> 4), axis=2).reshape(20, K)
    w = O.mxfp4_value(full, np.full((20, K // 32), 120))
    for kind, T in (("bf16", 1), ("mx8", 3)):
        x, xs, xv = make_x(torch, np.random.default_rng(1), T, K, kind)
        y = out(torch, T, N, "f32")
        log(f"[w4 large] {kind}")
        tw.twell_w4_matvec(x, xs, tw.TwellW4(codes, scales), None, y)
        check_product(values(y[:, -20:]), xv, w, None, "f32")
        assert (y[:, :-20] == 0).all()


# ---------------------------------------------------------------- the layer

def layer(torch, tw, r, T, d, F, kind, yd, bg=None, use_bias=True):
    Wg, wg = make_w(torch, tw, r, F, d, d ** -0.5)
    Wu, wu = make_w(torch, tw, r, F, d, d ** -0.5)
    Wd, wd = make_w(torch, tw, r, F, d, F ** -0.5)
    x, xs, xv = make_x(torch, r, T, d, kind)
    if bg is None:
        bg = r.normal(size=F) * 1.5 - 3.0
    b = torch.from_numpy(np.asarray(bg, dtype=np.float32)).bfloat16().cuda() if use_bias else None
    y = run_layer(torch, tw, T, d, F, kind, yd, x, xs, Wg, b, Wu, Wd)
    check_layer(values(y), xv, wg, 0.0 if b is None else values(b), wu, wd, yd)
    return y


def run_layer(torch, tw, T, d, F, kind, yd, x, xs, Wg, b, Wu, Wd, stream=None):
    sh = tw.ffn_shape(T, d, F, tw.TWELL_BF16 if kind == "bf16" else tw.TWELL_MXFP8,
                      tw.TWELL_F32 if yd == "f32" else tw.TWELL_BF16)
    y = out(torch, T, d, yd)
    ws = torch.full((tw.twell_ffn_fwd_w4_workspace(sh),), 255, dtype=torch.uint8, device="cuda")
    tw.twell_ffn_fwd_w4(sh, x, xs, Wg, b, Wu, Wd, y, ws, stream)
    return y


def check_layer(y, x, wg, b, wu, wd, yd):
    d, F = x.shape[1], wg.shape[0]
    n = (2 * d + 4) * U
    g, u = x @ wg.T + b, x @ wu.T
    h = np.maximum(g, 0)
    eg, eu = n * (np.abs(x) @ np.abs(wg).T + np.abs(b)), n * (np.abs(x) @ np.abs(wu).T)
    near = g > -eg                                      # neurons that may fire
    a = h * u
    ea = np.where(near, eg * (np.abs(u) + eu) + h * eu + U * np.abs(a), 0)
    ref = O.ffn_w4(x, wg, b, wu, wd)
    tol = ea @ np.abs(wd) + (2 * F + 4) * U * ((np.abs(a) + ea) @ np.abs(wd)) + HALF[yd] * np.abs(ref)
    err = np.abs(y - ref)
    assert (err <= tol).all(), (float(err.max()), float((err - tol).max()))


@pytest.mark.parametrize("T,d,F", [(1, 64, 64), (1, 2304, 9216), (2, 128, 192), (7, 320, 64), (16, 256, 512),
                                   (17, 64, 576), (33, 192, 128), (64, 2048, 1408), (65, 128, 320), (130, 64, 256),
                                   (5, 4096, 512), (300, 64, 64), (48, 576, 16384)])
@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_layer(torch, tw, T, d, F, kind):
    r = np.random.default_rng(T + d + F)
    for yd, use_bias in (("f32", True), ("bf16", False)):
        log(f"[w4 layer] T={T} d={d} F={F} {kind} {yd} bias={use_bias}")
        layer(torch, tw, r, T, d, F, kind, yd, use_bias=use_bias)


@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_layer_no_neuron_and_all_neurons(torch, tw, kind):
    r = np.random.default_rng(11)
    for T in (1, 20, 70):
        log(f"[w4 layer empty/full] T={T} {kind}")
        y = layer(torch, tw, r, T, 192, 256, kind, "f32", bg=np.full(256, -1e4))
        assert (y == 0).all()
        layer(torch, tw, r, T, 192, 256, kind, "f32", bg=np.full(256, 100.0))


@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_layer_rows_that_fire_differently(torch, tw, kind):
    """One token fires every neuron, one none, one only the last; NaN scales of
    Wu and Wd on a neuron that never fires, and a NaN token, reach nothing."""
    r = np.random.default_rng(12)
    T, d, F = 18, 128, 320
    Wg, wg = make_w(torch, tw, r, F, d, 0.1)
    Wu, wu = make_w(torch, tw, r, F, d, 0.1)
    Wd, wd = make_w(torch, tw, r, F, d, 0.1)
    x, xs, xv = make_x(torch, r, T, d, "bf16")
    wgc, wgs = np.zeros((F, d), dtype=np.int64), np.full((F, d // 32), 127, dtype=np.uint8)
    wgc[:, 0] = 2                                       # g = x[t, 0] + bg
    Wg, wg = pack_w(torch, tw, wgc, wgs)
    bg = np.zeros(F)
    bg[-1], bg[7] = 4.0, -1000.0
    x[:, 0] = -4.0
    x[0, 0], x[1, 0] = 8.0, -2.0                        # every neuron but 7; only the last
    xs = None
    if kind == "mx8":
        q = torch.clamp(x.float(), -448, 448).to(torch.float8_e4m3fn)
        x, xs = q.view(torch.uint8), torch.full((T, d // 32), 127, dtype=torch.uint8, device="cuda")
        xv = values(q.float())
    else:
        xv = values(x)
    Wu.scales[7] = 255
    Wd.scales[7] = 255
    if kind == "bf16":
        x[9, 3] = float("nan")
    else:
        x[9, 3] = 0x7f
    wu[7] = wd[7] = 0
    b = torch.from_numpy(bg.astype(np.float32)).bfloat16().cuda()
    log(f"[w4 layer rows] {kind}")
    y = values(run_layer(torch, tw, T, d, F, kind, "f32", x, xs, Wg, b, Wu, Wd))
    live = np.setdiff1d(np.arange(T), [9])
    check_layer(y[live], xv[live], wg, bg, wu, wd, "f32")
    assert (y[2:] == 0).all()                           # no neuron fires; g of the NaN token is NaN, not > 0
    assert (y[0] != 0).any() and (y[1] != 0).any()


@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_layer_repeats_on_a_stream_and_in_a_graph(torch, tw, kind):
    r = np.random.default_rng(13)
    T, d, F = 9, 256, 1024
    Wg, _ = make_w(torch, tw, r, F, d, d ** -0.5)
    Wu, _ = make_w(torch, tw, r, F, d, d ** -0.5)
    Wd, _ = make_w(torch, tw, r, F, d, F ** -0.5)
    x, xs, _ = make_x(torch, r, T, d, kind)
    b = torch.full((F,), -2.0, dtype=torch.bfloat16, device="cuda")
    sh = tw.ffn_shape(T, d, F, tw.TWELL_BF16 if kind == "bf16" else tw.TWELL_MXFP8, tw.TWELL_F32)
    ws = torch.empty(tw.twell_ffn_fwd_w4_workspace(sh), dtype=torch.uint8, device="cuda")
    y, z = out(torch, T, d, "f32"), out(torch, T, F, "f32")

    def step(stream=None):
        tw.twell_w4_matvec(x, xs, Wg, b, z, stream)
        tw.twell_ffn_fwd_w4(sh, x, xs, Wg, b, Wu, Wd, y, ws, stream)

    log(f"[w4 stream, graph] {kind}")
    step()
    torch.cuda.synchronize()
    want = y.clone(), z.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(z, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        x.copy_(make_x(torch, r, T, d, kind)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), z.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(y, got[0]) and torch.equal(z, got[1]), k


@pytest.mark.parametrize("T,N,K", [(5, 4500, 4192), (33, 2200, 4128), (3, 8200, 4096), (20, 17000, 96), (3, 4200, 64),
                                   (50, 300, 8288), (9, 33000, 672), (16, 4097, 32)])
@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_matvec_splits(torch, tw, T, N, K, kind):
    """The splits of K over a workgroup's waves: one to eight of them, runs of
    chunks that are no multiple of four, and rows of fewer than four blocks."""
    r = np.random.default_rng(T + N + K)
    W, w = make_w(torch, tw, r, N, K, K ** -0.5)
    x, xs, xv = make_x(torch, r, T, K, kind)
    log(f"[w4 splits] T={T} N={N} K={K} {kind}")
    y = out(torch, T, N, "f32")
    tw.twell_w4_matvec(x, xs, W, None, y)
    check_product(values(y), xv, w, None, "f32")


@pytest.mark.parametrize("T,N,K", [(17, 10241, 416), (64, 10300, 1184), (33, 16384, 96), (17, 10240, 416), (70, 12001, 512)])
@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_matvec_middle_sizes(torch, tw, T, N, K, kind):
    test_matvec_splits(torch, tw, T, N, K, kind)
