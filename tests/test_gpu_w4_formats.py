"""Every code and scale byte of MXFP4 weights and MXFP8 tokens through every
path that decodes them, and odd places and bad values at one and two tokens.

A single product at a time, so results are exact.  Operands of magnitude below
2^-126 may be taken as 0 or lose their last bits, those of 2^128 and more are
infinities (a NaN where a zero meets them)."""
import numpy as np
import pytest

import oracle as O

from test_gpu_w4 import check_product, log, make_w, make_x, out, pack_w, run_layer, torch, tw, values  # noqa: F401

pytestmark = pytest.mark.gpu

LOW, HIGH = 2.0 ** -126, 2.0 ** 128


def check_single(got, operand, factor, nan):
    """got against operand * factor, where `operand` is what was decoded."""
    v = np.abs(operand)
    with np.errstate(invalid="ignore", over="ignore"):
        want = operand * factor
        plain = ~nan & ((v == 0) | ((v >= LOW) & (v < HIGH))) & ((want == 0) | ((np.abs(want) >= LOW) & (np.abs(want) < HIGH)))
        low = ~nan & (v > 0) & (v < LOW)
    assert plain.any() and (got[plain] == want[plain]).all()
    assert np.isnan(got[nan]).all()
    assert not np.isfinite(got[~nan & (v >= HIGH)]).any()
    assert (np.abs(got[low]) <= LOW * np.abs(factor[low] if np.ndim(factor) else factor)).all()


@pytest.mark.parametrize("T,copies", [(1, 1), (2, 1), (3, 1), (3, 2), (17, 3), (17, 5)],
                         ids=["one", "two", "narrow", "small", "middle", "large"])
@pytest.mark.parametrize("K", [32, 96, 288])
@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_weight_codes_and_scales(torch, tw, T, copies, K, kind):
    """A row for every code and scale byte, in one of the row's blocks; the
    other blocks hold zeros of other scales."""
    r = np.random.default_rng(K + T)
    blocks, N = K // 32, 4096 * copies
    n = np.arange(N)
    code, byte, at = n % 16, n // 16 % 256, (n // 7) % blocks
    codes, scale = np.zeros((N, blocks, 32), dtype=np.int64), r.integers(0, 255, (N, blocks)).astype(np.uint8)
    codes[n, at] = code[:, None]
    scale[n, at] = byte
    W, _ = pack_w(torch, tw, codes.reshape(N, K), scale)
    x = np.zeros((T, blocks, 32))
    for t in range(T):
        x[t, :, (7 * t + 5) % 32] = 1.0 if t % 2 == 0 else -0.5
    x = x.reshape(T, K)
    if kind == "bf16":
        xt, xs = torch.from_numpy(x).to(torch.bfloat16).cuda(), None
    else:
        xt = torch.from_numpy(x * 4).to(torch.float8_e4m3fn).cuda()
        xs = torch.full((T, blocks), 125, dtype=torch.uint8, device="cuda")
    log(f"[w4 codes] T={T} N={N} K={K} {kind}")
    y = out(torch, T, N, "f32")
    tw.twell_w4_matvec(xt, xs, W, None, y)
    got = values(y)
    with np.errstate(invalid="ignore"):
        w = O.e2m1_value(code) * O.e8m0_value(byte)
    for t in range(T):
        check_single(got[t], w, 1.0 if t % 2 == 0 else -0.5, byte == 255)


@pytest.mark.parametrize("T,N", [(1, 40), (2, 40), (256, 40), (256, 300), (256, 10400), (256, 16400)],
                         ids=["one", "two", "narrow", "small", "middle", "large"])
@pytest.mark.parametrize("K", [64, 160])
def test_token_codes_and_scales(torch, tw, T, N, K):
    """A token for every code, at scales that cover every byte, in one of its
    blocks; the other blocks hold zeros of other scales."""
    r = np.random.default_rng(K + N)
    blocks = K // 32
    W, _ = pack_w(torch, tw, np.full((N, K), 2), np.full((N, blocks), 127, dtype=np.uint8))
    i = np.arange(4096)
    code, byte, at = i % 256, (i % 256 * 37 + i // 256 * 16 + i // 16 % 16) % 256, i % blocks
    q, s = np.zeros((4096, blocks, 32), dtype=np.uint8), r.integers(0, 255, (4096, blocks)).astype(np.uint8)
    q[i, at, (5 * i + 3) % 32] = code
    s[i, at] = byte
    q, s = torch.from_numpy(q.reshape(4096, K)).cuda(), torch.from_numpy(s).cuda()
    log(f"[w4 token codes] T={T} N={N} K={K}")
    got = torch.empty(4096, N, device="cuda")
    for t in range(0, 4096, T):
        tw.twell_w4_matvec(q[t:t + T], s[t:t + T], W, None, got[t:t + T])
    got = values(got[:, [0, 1, 15, N // 2, N - 1]])
    with np.errstate(invalid="ignore"):
        v = O.e4m3_value(code) * O.e8m0_value(byte)
    assert len(np.unique(byte)) == 256
    for n in range(got.shape[1]):
        check_single(got[:, n], v, 1.0, np.isnan(v))


@pytest.mark.parametrize("T", [1, 2, 3, 9, 40])
def test_down_product_codes_and_scales(torch, tw, T):
    """One neuron fires with a = 1: y is its row of Wd, which holds every code
    and scale byte."""
    d, F = 8192, 64
    zero, one = np.zeros((F, d), dtype=np.int64), np.full((F, d // 32), 127, dtype=np.uint8)
    up = zero.copy()
    up[:, 9] = 2
    down, scale = np.tile(np.arange(d) % 16, (F, 1)), np.tile(np.arange(256).astype(np.uint8), (F, 1))
    Wg, Wu, Wd = (pack_w(torch, tw, c, s)[0] for c, s in ((zero, one), (up, one), (down, scale)))
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    x[:, 9] = 1.0
    b = torch.full((F,), -1.0, dtype=torch.bfloat16, device="cuda")
    b[37] = 1.0
    log(f"[w4 down codes] T={T}")
    y = values(run_layer(torch, tw, T, d, F, "bf16", "f32", x, None, Wg, b, Wu, Wd))
    byte = np.arange(d) // 32
    with np.errstate(invalid="ignore"):
        w = O.e2m1_value(np.arange(d) % 16) * O.e8m0_value(byte)
    for t in range(T):
        check_single(y[t], w, 1.0, byte == 255)


@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("kind", ["bf16", "mx8"])
@pytest.mark.parametrize("N,K", [(37, 160), (130, 1056), (16, 4128)])
def test_few_tokens_at_odd_places(torch, tw, T, kind, N, K):
    """x, x_scale and y at odd offsets, x and y in wider rows; neighbours stay."""
    r = np.random.default_rng(N + T)
    W, w = make_w(torch, tw, r, N, K)
    x, xs, xv = make_x(torch, r, T, K, kind)
    xb = torch.zeros(T, K + 13, dtype=x.dtype, device="cuda")
    xb[:, 3:3 + K] = x
    if xs is not None:
        flat = torch.zeros(xs.numel() + 1, dtype=torch.uint8, device="cuda")
        flat[1:] = xs.reshape(-1)
        xs = flat[1:].view(xs.shape)
    for yd in ("f32", "bf16"):
        log(f"[w4 odd places] T={T} {kind} {yd} N={N} K={K}")
        yb = out(torch, T, N + 9, yd)
        tw.twell_w4_matvec(xb[:, 3:3 + K], xs, W, None, yb[:, 5:5 + N])
        got = values(yb)
        check_product(got[:, 5:5 + N], xv, w, None, yd)
        assert (got[:, :5] == 7).all() and (got[:, 5 + N:] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "mx8"])
@pytest.mark.parametrize("bad", [0, 1])
def test_bad_values_of_two_tokens(torch, tw, kind, bad):
    """A token with a NaN or an infinity leaves the other as it is, and a NaN
    scale reaches its row of weights only."""
    r = np.random.default_rng(8 + bad)
    N, K = 70, 1376
    W, w = make_w(torch, tw, r, N, K)
    x, xs, xv = make_x(torch, r, 2, K, kind)
    if kind == "bf16":
        x[bad, K - 1] = float("nan") if bad else float("inf")
    elif bad:
        x[bad, K - 1] = 0x7f
    else:
        xs[bad, 0] = 255
    W.scales[33, 42] = 255
    rows = np.setdiff1d(np.arange(N), [33])
    log(f"[w4 bad values of two tokens] {kind} {bad}")
    y = out(torch, 2, N, "f32")
    tw.twell_w4_matvec(x, xs, W, None, y)
    got = values(y)
    assert not np.isfinite(got[bad]).any() and np.isnan(got[:, 33]).all()
    check_product(got[1 - bad:2 - bad][:, rows], xv[1 - bad:2 - bad], w[rows], None, "f32")
    y = out(torch, 1, N, "f32")
    one = slice(1 - bad, 2 - bad)
    tw.twell_w4_matvec(x[one], None if xs is None else xs[one], W, None, y)
    got = values(y)
    assert np.isnan(got[0, 33])
    check_product(got[:, rows], xv[one], w[rows], None, "f32")
