#!/usr/bin/env python3
"""A stack of sparse feed-forward layers on a residual stream, trained and then
served on 4-bit weights.

    python examples/residual_stack.py [--layers 2] [--d 256] [--f 1024] [--tokens 512] [--steps 60]

Training (bf16 weights), per layer: the residual sum with dropout and norm
(twell_add_rmsnorm_fwd), the layer with its saved TwELL of h (twell_ffn_fwd);
after the last one, twell_dropout_add.  The backward runs twell_dropout_add,
twell_ffn_bwd_hybrid and twell_add_rmsnorm_bwd; no mask is stored, the random
numbers are drawn again.  The task is synthetic: next-token targets of a fixed
permutation, so the loss falls.

Serving: the trained weights become MXFP4 once; a step takes one token per
sequence through norms that write MXFP8, layers on 4-bit weights
(twell_ffn_fwd_w4) and a 4-bit output product (twell_w4_matvec), captured in a
graph.
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import activation_sparse_feedforward_gate_amd as tw  # noqa: E402

BF16, F32, MX8 = tw.TWELL_BF16, tw.TWELL_F32, tw.TWELL_MXFP8
EPS = 1e-5


def empty(*size, dt=torch.bfloat16):
    return torch.empty(*size, dtype=dt, device="cuda")


def space(n):
    return empty(max(16, n), dt=torch.uint8)


def mxfp4(w):
    """TwellW4 of a weight matrix [N][K]: per 32 columns the smallest power of
    two that holds them within +-6 and the nearest code (ties to even)."""
    N, K = w.shape
    v = w.float().view(N, K // 32, 32)
    m, e = torch.frexp(v.abs().amax(dim=2))
    e = torch.where(m <= 0.75, e - 3, e - 2).clamp(-127, 127)
    e = torch.where(m == 0, -127, e)
    a = torch.ldexp(v, -e.unsqueeze(2)).abs()
    code = sum((a >= t if i % 2 else a > t).to(torch.uint8) for i, t in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    code = (code | ((v < 0).to(torch.uint8) << 3)).view(N, K)
    return tw.TwellW4((code[:, 0::2] | code[:, 1::2] << 4).contiguous(), (e + 127).to(torch.uint8).contiguous())


class Stack:
    """Weights of the stack: per layer norm, gate, up, down and gate bias; the
    tied embedding and the last norm."""

    def __init__(self, layers, d, f, vocab, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(std, *size):
            return torch.randn(*size, generator=g, device="cuda") * std

        self.d, self.f, self.vocab = d, f, vocab
        self.E = normal(1.0, vocab, d)
        self.layers = [{"w": torch.ones(d, device="cuda"), "Wg": normal(d ** -0.5, f, d), "Wu": normal(d ** -0.5, f, d),
                        "Wd": normal(f ** -0.5, f, d), "bg": torch.full((f,), -1.0, device="cuda")}
                       for _ in range(layers)]
        self.w = torch.ones(d, device="cuda")

    def parameters(self):
        """The fp32 weights, by (layer, name); layer None: the last norm."""
        return {**{(i, k): v for i, p in enumerate(self.layers) for k, v in p.items()}, (None, "w"): self.w}


class Trainer:
    """Buffers of T tokens for forward and backward, kept from step to step."""

    def __init__(self, stack, T, p=0.1, threshold=None):
        self.stack, self.T, self.p = stack, T, p
        d, f, L = stack.d, stack.f, len(stack.layers)
        self.threshold = f // 4 if threshold is None else threshold
        # forward: x is the layer's fp32 output; backward: its gradient goes into the layer as bf16
        self.fwd = tw.norm_shape(T, d, F32, BF16, BF16, BF16, EPS, p)
        self.first = tw.norm_shape(T, d, BF16, BF16, BF16, BF16, EPS)
        self.bwd = tw.norm_shape(T, d, BF16, BF16, F32, BF16, EPS, p)
        self.last = tw.norm_shape(T, d, F32, BF16, BF16, BF16, EPS, p)
        self.dlast = tw.norm_shape(T, d, BF16, BF16, BF16, BF16, EPS, p)
        self.ffn = tw.ffn_shape(T, d, f, BF16, F32)
        self.sum = [empty(T, d) for _ in range(L + 1)]
        self.x = [empty(T, d) for _ in range(L)]
        self.rstd = [empty(T, dt=torch.float32) for _ in range(L)]
        self.h = [tw.alloc_twell_mat(T, f) for _ in range(L)]
        self.y, self.dx32 = empty(T, d, dt=torch.float32), empty(T, d, dt=torch.float32)
        self.dy, self.dsum = empty(T, d), empty(T, d)
        self.rng = torch.zeros(L, 2, dtype=torch.int64, device="cuda")
        self.rng[:, 0] = torch.arange(L, device="cuda") + 1                  # a seed per layer; the offset counts steps
        self.ws = space(max(tw.twell_ffn_fwd_workspace(self.ffn, True),
                            tw.twell_ffn_bwd_workspace(self.ffn, self.threshold),
                            tw.twell_add_rmsnorm_bwd_workspace(self.bwd)))
        self.grads = [{"w": empty(d, dt=torch.float32), "Wg": empty(f, d, dt=torch.float32),
                       "Wu": empty(f, d, dt=torch.float32), "Wd": empty(f, d, dt=torch.float32),
                       "bg": empty(f, dt=torch.float32)} for _ in range(L)]

    def forward(self, emb):
        """The residual stream [T][d] after the layers, for bf16 inputs."""
        self.q = [{k: v.bfloat16() for k, v in p.items()} for p in self.stack.layers]
        self.sum[0].copy_(emb)
        for i, q in enumerate(self.q):
            if i == 0:
                tw.twell_add_rmsnorm_fwd(self.first, self.sum[0], None, q["w"], None, None, self.x[0], None, self.rstd[0])
            else:
                tw.twell_add_rmsnorm_fwd(self.fwd, self.y, self.sum[i - 1], q["w"], self.rng[i - 1], self.sum[i],
                                         self.x[i], None, self.rstd[i])
            tw.twell_ffn_fwd(self.ffn, self.x[i], q["Wg"], q["bg"], q["Wu"], q["Wd"], self.y, self.h[i],
                             self.threshold, self.ws)
        L = len(self.q)
        tw.twell_dropout_add(self.last, self.y, self.sum[L - 1], self.rng[L - 1], self.sum[L])
        return self.sum[L]

    def backward(self, dout):
        """Gradients of the weights for the gradient of forward's result;
        returns that of its input."""
        L = len(self.q)
        self.dsum.copy_(dout)
        tw.twell_dropout_add(self.dlast, self.dsum, None, self.rng[L - 1], self.dy)
        for i in reversed(range(L)):
            q, g = self.q[i], self.grads[i]
            tw.twell_ffn_bwd_hybrid(self.ffn, self.x[i], q["Wg"], q["bg"], q["Wu"], q["Wd"], self.dy, self.h[i],
                                    self.threshold, self.dx32, g["Wg"], g["Wu"], g["Wd"], g["bg"], None, self.ws)
            # dres over dsum: the gradient of the stream, and dropped that of the layer below
            shape = self.bwd if i else tw.norm_shape(self.T, self.stack.d, BF16, BF16, F32, BF16, EPS)
            tw.twell_add_rmsnorm_bwd(shape, self.dx32, self.dsum, self.sum[i], q["w"], self.rstd[i],
                                     self.rng[i - 1] if i else None, self.dsum, self.dy if i else None, g["w"], self.ws)
        return self.dsum

    def next_masks(self):
        self.rng[:, 1] += 1


def loss_of(stack, stream, targets):
    """Mean cross-entropy of the tied output product over the last norm, and the
    gradient of the stream and of the last norm's weights (plain torch)."""
    s = stream.float().requires_grad_(True)
    w = stack.w.clone().requires_grad_(True)
    y = s * torch.rsqrt(s.square().mean(dim=1, keepdim=True) + EPS) * w
    loss = torch.nn.functional.cross_entropy(y @ stack.E.t() * stack.d ** -0.5, targets)
    loss.backward()
    return loss.detach(), s.grad, w.grad


def train(stack, tokens, steps, lr=3e-3, p=0.1, seed=1):
    """Trains on next-token pairs of a fixed permutation (Adam over the fp32
    weights); returns the losses."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    follow = torch.randperm(stack.vocab, generator=g, device="cuda")
    t = Trainer(stack, tokens, p)
    weights = stack.parameters()
    opt = torch.optim.Adam(list(weights.values()), lr=lr)
    losses = []
    for _ in range(steps):
        ids = torch.randint(0, stack.vocab, (tokens,), generator=g, device="cuda")
        out = t.forward(stack.E[ids].bfloat16())
        loss, dout, dw = loss_of(stack, out, follow[ids])
        t.backward(dout)
        for (i, k), v in weights.items():
            v.grad = dw if i is None else t.grads[i][k]
        opt.step()
        t.next_masks()
        losses.append(loss)
    return [float(v) for v in losses], follow


class Server:
    """A decoding step of T sequences on MXFP4 weights."""

    def __init__(self, stack, T):
        self.stack, self.T = stack, T
        d, f = stack.d, stack.f
        self.layers = [{k: mxfp4(p[k]) for k in ("Wg", "Wu", "Wd")} for p in stack.layers]
        self.w = [p["w"].bfloat16() for p in stack.layers] + [stack.w.bfloat16()]
        self.bg = [p["bg"].bfloat16() for p in stack.layers]
        self.E, self.out = stack.E.bfloat16(), mxfp4(stack.E * d ** -0.5)
        self.first = tw.norm_shape(T, d, BF16, BF16, MX8, BF16, EPS)
        self.next = tw.norm_shape(T, d, F32, BF16, MX8, BF16, EPS)
        self.ffn = tw.ffn_shape(T, d, f, MX8, F32)
        self.ids = torch.zeros(T, dtype=torch.int64, device="cuda")
        self.sum, self.y = empty(T, d), empty(T, d, dt=torch.float32)
        self.x, self.scale = empty(T, d, dt=torch.float8_e4m3fn), empty(T, -(-d // 32), dt=torch.uint8)
        self.logits = empty(T, stack.vocab, dt=torch.float32)
        self.ws = space(tw.twell_ffn_fwd_w4_workspace(self.ffn))
        self.graph = None

    def _step(self):
        self.sum.copy_(self.E[self.ids])
        tw.twell_add_rmsnorm_fwd(self.first, self.sum, None, self.w[0], None, None, self.x, self.scale)
        for i, q in enumerate(self.layers):
            tw.twell_ffn_fwd_w4(self.ffn, self.x, self.scale, q["Wg"], self.bg[i], q["Wu"], q["Wd"], self.y, self.ws)
            tw.twell_add_rmsnorm_fwd(self.next, self.y, self.sum, self.w[i + 1], None, self.sum, self.x, self.scale)
        tw.twell_w4_matvec(self.x, self.scale, self.out, None, self.logits)
        self.ids.copy_(self.logits.argmax(dim=1))

    def step(self, ids=None):
        """The next token of each sequence (after ids, or the last result)."""
        if ids is not None:
            self.ids.copy_(ids)
        if self.graph is None:
            first = self.ids.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self._step()
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._step()
            self.ids.copy_(first)
        self.graph.replay()
        return self.ids


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--d", type=int, default=256, help="a multiple of 64")
    ap.add_argument("--f", type=int, default=1024, help="a multiple of 64")
    ap.add_argument("--vocab", type=int, default=250)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--sequences", type=int, default=16)
    a = ap.parse_args()
    stack = Stack(a.layers, a.d, a.f, a.vocab)
    losses, follow = train(stack, a.tokens, a.steps)
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps of {a.tokens} tokens")
    s = Server(stack, a.sequences)
    ids, right = torch.arange(a.sequences, device="cuda") % a.vocab, 0
    for _ in range(20):
        want = follow[ids]
        right += int((s.step(ids) == want).sum())
        ids = want                                      # each step from the right token
    print(f"serving on 4-bit weights: {right} of {20 * a.sequences} tokens as taught")


if __name__ == "__main__":
    main()
