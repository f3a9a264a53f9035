"""Outputs of the norm's backward that share memory with its other arguments:
refused on the host where they are not written in place, and in place the same
bits as into memory of their own, on both sides of 1024 rows."""
import numpy as np
import pytest

import activation_sparse_feedforward_gate_amd as tw

F32, BF16 = tw.TWELL_F32, tw.TWELL_BF16
T, D = 8, 64
FAR = 1 << 24                           # addresses of arguments that share nothing; nothing is launched


def bwd(ld=D, dtypes=(F32, F32, F32), rows=T, **k):
    a = {n: FAR * (i + 1) for i, n in enumerate(("dy", "dsum", "sum", "dres", "dx"))}
    lds = {n: ld for n in a}
    for n, v in k.items():
        a[n], lds[n] = v if isinstance(v, tuple) else (v, ld)
    y, r, x = dtypes
    sh = tw.norm_shape(rows, D, x, r, y, F32, 1e-5, 0.0)
    return tw.lib().twell_add_rmsnorm_bwd(sh, a["dy"], lds["dy"], a["dsum"], lds["dsum"], a["sum"], lds["sum"], None,
                                          64, None, a["dres"], lds["dres"], a["dx"], lds["dx"], 1 << 30, 1 << 31,
                                          1 << 30, None)


@pytest.mark.parametrize("rows", [T, 5000])
@pytest.mark.parametrize("out,other", [("dx", "dy"), ("dx", "sum"), ("dx", "dsum"), ("dres", "dy"), ("dres", "sum"),
                                       ("dres", "dsum"), ("dx", "dres")])
def test_overlap_that_is_not_in_place_is_refused(out, other, rows):
    at = FAR * (("dy", "dsum", "sum", "dres", "dx").index(other) + 1)
    E = tw.TWELL_EINVAL
    for by in (4, D * 4, (rows - 1) * D * 4 + 252, -4, -D * 4 * (rows - 1)):      # shifted by a value, by rows
        assert bwd(rows=rows, **{out: at + by}) == E, by
        assert b"overlap" in tw.lib().twell_last_error()
    assert bwd(rows=rows, **{out: (at, D + 8)}) == E                       # another stride
    wide = 2 * D                                                           # columns of one wider buffer
    for by in (4 * (D - 1), 4 * (wide - D + 1), 4 * (wide + D - 1)):
        assert bwd(ld=wide, rows=rows, **{out: at + by}) == E, by
    for dtypes in ((BF16, F32, BF16), (F32, BF16, F32), (BF16, BF16, F32), (F32, F32, BF16)):
        size = {"dy": dtypes[0], "dx": dtypes[2]}
        if size.get(out, dtypes[1]) != size.get(other, dtypes[1]):
            assert bwd(dtypes=dtypes, rows=rows, **{out: at}) == E         # another element type at the same place


def test_both_outputs_in_one_place_are_refused():
    assert bwd(dres=FAR, dx=FAR) == tw.TWELL_EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(9, 5), (70, 1003), (1100, 1003), (1025, 45), (300, 4100), (3, 20000)])
def test_in_place(rows, d):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + d)

    def rand(*size):
        return torch.randn(*size, generator=g, device="cuda")

    sh = tw.norm_shape(rows, d, F32, F32, F32, F32, 1e-5, 0.25)
    src = {n: rand(rows, d) for n in ("dy", "dsum", "sum")}
    w, rstd, rng = rand(d), torch.rand(rows, generator=g, device="cuda") + 0.5, torch.tensor([3, 4], device="cuda")
    ws = torch.empty(tw.twell_add_rmsnorm_bwd_workspace(sh), dtype=torch.uint8, device="cuda")

    def run(dres, dx, wide=0):
        """Results with dres and dx over the named inputs, or in memory of their own."""
        buf = torch.full((len(src) + 2, rows, d + wide), 7.0, device="cuda")
        m = {n: buf[i][:, :d] for i, n in enumerate((*src, "dres", "dx"))}
        for n, v in src.items():
            m[n].copy_(v)
        dw = torch.empty(d, device="cuda")
        o, x = m[dres], m[dx]
        tw.twell_add_rmsnorm_bwd(sh, m["dy"], m["dsum"], m["sum"], w, rstd, rng, o, x, dw, ws)
        torch.cuda.synchronize()
        assert (buf[:, :, d:] == 7.0).all()
        return o.clone(), x.clone(), dw.double().cpu().numpy()

    want = run("dres", "dx")
    mag = (src["dy"] * src["sum"] * rstd[:, None]).double().abs().sum(dim=0).cpu().numpy()
    for dres, dx in (("dsum", "dx"), ("dsum", "dy"), ("sum", "dx"), ("dres", "sum"), ("sum", "dy"), ("dy", "dsum"),
                     ("dres", "dsum"), ("dy", "dx")):
        for wide in (0, 3):
            got = run(dres, dx, wide)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (dres, dx, wide)
            # dw in one of two orders, each of at most `rows` additions and two products a term
            assert (np.abs(got[2] - want[2]) <= 2 * (rows + 2) * 2.0 ** -24 * mag).all(), (dres, dx, wide)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [70, 1100])
def test_columns_of_one_buffer_are_no_overlap(rows):
    """dy, sum and the outputs as neighbouring columns of one matrix."""
    import torch
    d = 72
    sh = tw.norm_shape(rows, d, F32, F32, F32, F32, 1e-5, 0.0)
    buf = torch.randn(rows, 4 * d, device="cuda")
    dy, s, dres, dx = (buf[:, i * d:(i + 1) * d] for i in range(4))
    rstd, dw = torch.rand(rows, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(tw.twell_add_rmsnorm_bwd_workspace(sh), dtype=torch.uint8, device="cuda")
    a, b, c, e = dy.clone(), s.clone(), torch.empty(rows, d, device="cuda"), torch.empty(rows, d, device="cuda")
    dw1 = torch.empty_like(dw)
    tw.twell_add_rmsnorm_bwd(sh, a, None, b, None, rstd, None, c, e, dw1, ws)
    tw.twell_add_rmsnorm_bwd(sh, dy, None, s, None, rstd, None, dres, dx, dw, ws)
    assert torch.equal(dres, c) and torch.equal(dx, e) and torch.equal(dw, dw1)
    assert torch.equal(dy, a) and torch.equal(s, b)
