"""The norm's forward at more rows than the latency-bound calls have (1024), in
every lane layout of the widths between 513 and 4096 and every type, the last
workgroup partly filled; tolerances are those of test_gpu_norm."""
import numpy as np
import pytest

import oracle as O

from test_gpu_norm import EPS, HALF, check_mx, check_norm, check_sum, dts, log, make, rng_tensor, torch, tw, values  # noqa: F401

pytestmark = pytest.mark.gpu

# the layouts for 513..1024, 1025..2048, 2049..2560 and 2561..4096 columns
SIZES = [(1027, 1001), (1025, 516), (1025, 1999), (1026, 1032), (1027, 2305), (1029, 2560), (1025, 2567), (1031, 4090)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("xd", ["f32", "bf16"])
@pytest.mark.parametrize("rd", ["f32", "bf16"])
@pytest.mark.parametrize("yd", ["f32", "bf16", "mx8"])
def test_many_rows(torch, tw, T, d, xd, rd, yd):
    r = np.random.default_rng(T + d)
    D = dts(torch, tw)
    for has_res, p, wide in ((1, 0.25, 0), (0, 0.0, 5)):
        log(f"[norm layouts] T={T} d={d} {xd} {rd} {yd} res={has_res} p={p}")
        x, w = make(torch, r, T, d + wide, D[xd][0])[:, wide:], make(torch, r, 1, d, D[rd][0])
        res = make(torch, r, T, d, D[rd][0], 3.0) if has_res else None
        s = torch.empty(T, d, dtype=D[rd][0], device="cuda")
        mx = yd == "mx8"
        yb = torch.full((T, d + wide), 7, dtype=torch.uint8 if mx else D[yd][0], device="cuda")
        y, ys = yb[:, :d], torch.empty(T, -(-d // 32), dtype=torch.uint8, device="cuda") if mx else None
        rstd = torch.empty(T, device="cuda")
        sh = tw.norm_shape(T, d, D[xd][1], D[rd][1], tw.TWELL_MXFP8 if mx else D[yd][1], D[rd][1], EPS, p)
        tw.twell_add_rmsnorm_fwd(sh, x, res, w, rng_tensor(torch) if p else None, s, y, ys, rstd)
        check_sum(values(s), values(x), None if res is None else values(res), p, HALF[rd])
        assert (yb[:, d:] == 7).all()
        if mx:
            check_mx(y.cpu().numpy(), ys.cpu().numpy(), O.add_rmsnorm_fwd(values(s), None, values(w)[0], EPS)[1])
        else:
            check_norm(values(y), values(rstd), values(s), values(w)[0], HALF[yd])
