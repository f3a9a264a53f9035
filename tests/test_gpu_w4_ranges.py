"""Products with MXFP4 weights at the ends of their ranges."""
import numpy as np
import pytest

from test_gpu_w4 import check_product, log, make_w, make_x, torch, tw, values  # noqa: F401

pytestmark = pytest.mark.gpu

PIECE = 1 << 24


def pieces(n, borders):
    """Runs of 0..n around its ends and the borders, and all of it in pieces."""
    near = [(max(0, b - 20), min(n, b + 20)) for b in sorted({0, n, *[b for b in borders if b < n]})]
    assert all(a[1] <= b[0] for a, b in zip(near, near[1:]))
    return near, [(i, min(n, i + PIECE)) for i in range(0, n, PIECE)]


def filled(torch, value, dt, n, *size):
    t = torch.empty(n, *size, dtype=dt, device="cuda")
    for i in range(0, n, PIECE):
        t[i:i + PIECE].fill_(value)
    return t


def put(big, runs, few):
    at = 0
    for lo, hi in runs:
        big[lo:hi].copy_(few[at:at + hi - lo])
        at += hi - lo


@pytest.mark.parametrize("T,N", [(1, (1 << 26) + 45), (2, (1 << 30) + 47), (3, (1 << 26) + 45), (20, (1 << 26) + 60)])
def test_rows_of_more_than_one_launch(torch, tw, T, N):
    """More rows than a grid takes: those around each launch's border, the first
    and the last are as any, with their bias; the others are 0."""
    K = 32
    r = np.random.default_rng(N)
    near, every = pieces(N, range(1 << 26, N, 1 << 26))
    n = sum(hi - lo for lo, hi in near)
    few, w = make_w(torch, tw, r, n, K)
    b = torch.from_numpy(r.normal(size=n).astype(np.float32)).bfloat16().cuda()
    codes, scales = filled(torch, 0, torch.uint8, N, K // 2), filled(torch, 120, torch.uint8, N, 1)
    bias = filled(torch, 0, torch.bfloat16, N)
    for big, part in ((codes, few.codes), (scales, few.scales), (bias, b)):
        put(big, near, part)
    for kind in ("bf16", "mx8"):
        log(f"[w4 many rows] T={T} N={N} {kind}")
        x, xs, xv = make_x(torch, r, T, K, kind)
        y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        for t in range(T):
            for lo, hi in every:
                y[t, lo:hi].fill_(7.0)
        tw.twell_w4_matvec(x, xs, tw.TwellW4(codes, scales), bias, y)
        check_product(np.concatenate([values(y[:, lo:hi]) for lo, hi in near], axis=1), xv, w, values(b), "bf16")
        for lo, hi in near:
            y[:, lo:hi].zero_()
        assert not any(bool(y[t, lo:hi].any()) for t in range(T) for lo, hi in every)
    del codes, scales, bias, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,kind", [((1 << 24) + 41, "bf16"), ((1 << 24) + 55, "mx8"), ((1 << 31) - 1, "mx8")])
def test_tokens_of_more_than_one_launch(torch, tw, T, kind):
    """More tokens than 32-bit token indexes take beside a tile."""
    N, K = 3, 32
    r = np.random.default_rng(T % 1000)
    W, w = make_w(torch, tw, r, N, K)
    near, every = pieces(T, [1 << 24, 5 << 24])
    few, fs, xv = make_x(torch, r, sum(hi - lo for lo, hi in near), K, kind)
    log(f"[w4 many tokens] T={T} {kind}")
    x, xs = filled(torch, 0, few.dtype, T, K), None
    put(x, near, few)
    if kind == "mx8":
        xs = filled(torch, 120, torch.uint8, T, 1)
        put(xs, near, fs)
    y = filled(torch, 7.0, torch.bfloat16, T, N)
    tw.twell_w4_matvec(x, xs, W, None, y)
    check_product(np.concatenate([values(y[lo:hi]) for lo, hi in near]), xv, w, None, "bf16")
    for lo, hi in near:
        y[lo:hi].zero_()
    assert not any(bool(y[lo:hi].any()) for lo, hi in every)
    del x, xs, y
    torch.cuda.empty_cache()
