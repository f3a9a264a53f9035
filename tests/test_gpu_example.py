"""The example's stack: its gradients against the float64 oracle with the same
roundings to bf16, a training run, and its decoding step against the oracle,
eager and from a graph.

Tolerances (relative Frobenius): a bf16 value rounds by at most 2^-8 of itself,
the oracle at the same places, so that a value differs where the two sides
round one number to different neighbours (one step, 2^-7) or a gate changes
sign: 1e-2 for gradients.  The decoding step's activations are in e4m3 (one
step 2^-3): 5e-2 where a few of the values take the other neighbour."""
import importlib.util
import os

import numpy as np
import pytest

import oracle as O
from workloads.synth import round_bf16

from gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "residual_stack.py")
    spec = importlib.util.spec_from_file_location("residual_stack", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().to("cpu").double().numpy()


def bf(v):
    return round_bf16(np.asarray(v, dtype=np.float32)).astype(np.float64)


def rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


@pytest.mark.parametrize("threshold", [-1, 40, 192])
def test_gradients(ex, threshold):
    import torch
    T, d, f, L, p = 90, 64, 192, 2, 0.25
    stack = ex.Stack(L, d, f, 50, seed=3)
    t = ex.Trainer(stack, T, p, threshold)
    t.rng[:, 1] = 5
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    emb = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    dout = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    log(f"[example gradients] threshold={threshold}")
    out = f64(t.forward(emb))
    din = f64(t.backward(dout))

    q = [{k: bf(f64(v)) for k, v in layer.items()} for layer in stack.layers]
    s, x, r, y = [f64(emb)], [], [], None
    for i in range(L):
        if i:
            s.append(bf(O.dropout(y.astype(np.float32), p, i, 5) + s[i - 1]))
        _, xi, ri = O.add_rmsnorm_fwd(s[i], None, q[i]["w"], ex.EPS)
        x.append(bf(xi))
        r.append(ri)
        y = O.ffn_dense_fwd(x[i], q[i]["Wg"], q[i]["bg"], q[i]["Wu"], q[i]["Wd"])["y"]
    ref = O.dropout(y, p, L, 5) + s[L - 1]
    assert rel(out, ref) <= 1e-2, rel(out, ref)
    dsum = f64(dout)
    dy = bf(O.dropout(dsum, p, L, 5))
    for i in reversed(range(L)):
        b = O.ffn_dense_bwd(x[i], q[i]["Wg"], q[i]["bg"], q[i]["Wu"], q[i]["Wd"], dy)
        dres, dx, dw = O.add_rmsnorm_bwd(b["dX"], dsum, s[i], q[i]["w"], r[i], p if i else 0.0, i, 5)
        dsum, dy = bf(dres), bf(dx)
        for k, v in (("Wg", b["dWgT"]), ("Wu", b["dWuT"]), ("Wd", b["dWd"]), ("bg", b["dbg"]), ("w", dw)):
            e = rel(f64(t.grads[i][k]), v)
            log(f"   layer {i} {k} {e:.2e}")
            assert e <= 1e-2, (i, k, e)
    assert rel(din, dsum) <= 1e-2, rel(din, dsum)


def test_training_learns_and_serving_answers(ex):
    import torch
    stack = ex.Stack(2, 128, 512, 60)
    losses, follow = ex.train(stack, 256, 60)
    log(f"[example] loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    assert losses[-1] < 0.5 * losses[0]
    server = ex.Server(stack, 7)
    ids = torch.arange(7, device="cuda") + 3
    for k in range(4):                                  # replays after the first, eager work between them
        got = server.step(ids).clone()
        logits = server.logits.clone()
        server.ids.copy_(ids)
        server._step()
        torch.cuda.synchronize()
        assert torch.equal(server.logits, logits) and torch.equal(server.ids, got), k
        ids = follow[ids]


def dequantised(W):
    codes = W.codes.cpu().numpy().astype(np.int64)
    c = np.stack((codes & 15, codes >> 4), axis=2).reshape(codes.shape[0], -1)
    return c, W.scales.cpu().numpy().astype(np.int64)


def test_decoding_step(ex):
    import torch
    T, d, f = 5, 128, 320
    stack = ex.Stack(2, d, f, 75, seed=8)
    server = ex.Server(stack, T)
    ids = torch.tensor([3, 0, 74, 9, 3], device="cuda")
    log("[example decoding step]")
    server.step(ids)
    quantise = []
    for q, p in zip(server.layers, stack.layers):
        w = {}
        for k in ("Wg", "Wu", "Wd"):
            c, s = dequantised(q[k])
            rc, rs = O.mxfp4(f64(p[k]))
            quantise.append((c == rc).all() and (s == rs).all())
            w[k] = O.mxfp4_value(c, s)
        w["bg"] = bf(f64(p["bg"]))
        w["w"] = bf(f64(p["w"]))
        q["ref"] = w
    assert all(quantise)

    def x8(s, w):
        _, v, _ = O.add_rmsnorm_fwd(s, None, w, ex.EPS)
        v, scale = O.mxfp8(v)
        return v * np.repeat(O.e8m0_value(scale), 32, axis=1)

    s = bf(f64(stack.E))[ids.cpu().numpy()]
    for q in server.layers:
        w = q.pop("ref")
        s = bf(s + O.ffn_w4(x8(s, w["w"]), w["Wg"], w["bg"], w["Wu"], w["Wd"]))
    ref = x8(s, bf(f64(stack.w))) @ O.mxfp4_value(*dequantised(server.out)).T
    e = rel(f64(server.logits), ref)
    log(f"   logits {e:.2e}")
    assert e <= 5e-2
