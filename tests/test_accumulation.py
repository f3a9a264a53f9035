"""Products and column sums lose no more than additions in fp32 on the ways that
the kernels add them; and the bounds tell that from coarser or longer ways."""
import numpy as np
import pytest

from accumulation import INNER, column_error, product_error

SIZES = [(1, 2304), (2, 16384), (1, 4096), (3, 1024), (16, 2304), (20, 5632), (64, 16384)]


def f32(v):
    return np.asarray(v, dtype=np.float32).astype(np.float64)


def operands(r, T, N, K):
    x = f32(r.normal(size=(T, K)))
    return x, np.array([0, .5, 1, 1.5, 2, 3, 4, 6])[r.integers(0, 8, (N, K))] * r.choice([-1, 1], (N, K)) * K ** -0.5


def instructions(x, w, K, coarse=None):
    """A K loop in steps of one instruction; coarse: each cuts its sum to that share
    of the magnitudes it adds, otherwise it cuts to fp32's 24 bits."""
    acc = np.zeros((x.shape[0], w.shape[0]))
    for k in range(0, K, INNER):
        a, b = x[:, k:k + INNER], w[:, k:k + INNER]
        s = acc + a @ b.T
        if coarse:
            unit = coarse * (np.abs(a) @ np.abs(b).T)
        else:
            unit = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(s), 1e-30))) - 23)
        acc = np.trunc(s / unit) * unit
    return acc


@pytest.mark.parametrize("T,K", SIZES)
def test_product_bounds(T, K):
    """Every term after the other, cut to fp32, in as many waves as the bound
    counts stays within; a loop that adds at 2^-16 of an instruction's terms does not."""
    r = np.random.default_rng(K)
    n = max(T, 3)
    x, w = operands(r, n, 600, K)
    waves = 1 if K <= 512 else 2 if K <= 1024 else 4
    runs = np.array_split(np.arange(K // 128), waves)
    cols = [np.concatenate([np.arange(128 * c, 128 * c + 128) for c in run]) for run in runs]
    got = f32(sum(instructions(x[:, c], w[:, c], len(c)) for c in cols))
    worst, rms = product_error(got, x, w, n, K)
    assert worst <= 1 and rms <= 1
    for parts in (cols, [np.arange(K)]):
        got = sum(instructions(x[:, c], w[:, c], len(c), 2.0 ** -16) for c in parts)
        assert product_error(got, x, w, T, K)[1] > 1


@pytest.mark.parametrize("T,parts", [(5000, 1024), (20000, 512), (32768, 256)])
def test_column_bounds(T, parts):
    r = np.random.default_rng(T)
    terms = r.normal(size=(T, 200))
    assert max(column_error(f32(terms).sum(axis=0), terms, T, parts)) <= 1
    part = np.zeros((parts, 200), dtype=np.float32)
    for t in range(0, T, parts):
        rows = terms[t:t + parts].astype(np.float32)
        part[:len(rows)] += rows
    total = np.zeros(200, dtype=np.float32)
    for p in part:                                          # more in a row than the kernels', and still less than T
        total += p
    serial = np.zeros(200, dtype=np.float32)
    for row in terms.astype(np.float32):
        serial += row
    assert column_error(serial.astype(np.float64), terms, T, parts)[1] > 1
    assert column_error(total.astype(np.float64), terms, T, parts)[1] < column_error(serial.astype(np.float64), terms, T, parts)[1]


# ---------------------------------------------------------------- the kernels

@pytest.mark.gpu
@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("N", [1000, 10250, 16400])
@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_products(T, K, N, kind):
    import torch

    import activation_sparse_feedforward_gate_amd as tw
    from test_gpu_w4 import make_w, make_x, values
    r = np.random.default_rng(T + N + K)
    few = 300
    W, w = make_w(torch, tw, r, few, K, K ** -0.5)
    at = torch.linspace(0, N - 1, few, device="cuda").long()
    codes, scales = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"), torch.full((N, K // 32), 120, dtype=torch.uint8, device="cuda")
    codes[at], scales[at] = W.codes, W.scales
    x, xs, xv = make_x(torch, r, T, K, kind)
    y = torch.empty(T, N, device="cuda")
    print(f"[w4 accumulation] T={T} N={N} K={K} {kind}", flush=True)
    tw.twell_w4_matvec(x, xs, tw.TwellW4(codes, scales), None, y)
    worst, rms = product_error(values(y[:, at]), xv, w, T, K)
    print(f"   of the bounds: largest {worst:.3f}, mean {rms:.3f}", flush=True)
    assert worst <= 1 and rms <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(777, 1001), (1024, 2304), (1025, 520), (5000, 250), (20000, 1001), (32768, 512), (3000, 4100),
                                 (2000, 9000), (1500, 17000)])
def test_columns_of_dw(T, d):
    import torch

    import activation_sparse_feedforward_gate_amd as tw
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    dy, s = (torch.randn(T, d, generator=g, device="cuda") for _ in range(2))
    rstd = torch.rand(T, generator=g, device="cuda") + 0.5
    sh = tw.norm_shape(T, d, 0, 0, 0, 0, 1e-5)
    size = tw.twell_add_rmsnorm_bwd_workspace(sh)
    ws, dw, dres = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty(d, device="cuda"), torch.empty_like(s)
    print(f"[dw accumulation] T={T} d={d}", flush=True)
    tw.twell_add_rmsnorm_bwd(sh, dy, None, s, None, rstd, None, dres, None, dw, ws)
    n = min(d, 1001)
    f = [v[:, :n].double().cpu().numpy() for v in (dy, s)]
    worst, rms = column_error(dw[:n].double().cpu().numpy(), f[0] * f[1] * rstd.double().cpu().numpy()[:, None], T,
                              size // (4 * d))
    print(f"   of the bounds: largest {worst:.3f}, mean {rms:.3f}", flush=True)
    assert worst <= 1 and rms <= 1
