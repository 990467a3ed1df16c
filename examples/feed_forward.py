"""A gated feed-forward block on the operators of hierarchical_gemm_gb300.tsffn.

    y = x + (silu(x Wg) * (x Wu)) Wd

Training: `Block.step` runs the forward pass (the gated projection, then the
down projection with the residual in its epilogue), the backward pass, the
clipping of the two weight gradients by their global norm, and a plain
gradient-descent update.  Serving: `Block.decode` runs the same block on the
few rows of a decoding step, into buffers that are kept, so that a step can
be captured into a CUDA graph.

    python examples/feed_forward.py [--tokens 2048] [--hidden 1024] [--width 2816] [--steps 20]

trains the block towards a fixed random target and then times decoding.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from hierarchical_gemm_gb300 import tsffn  # noqa: E402


class Block:
    """The block's weights, stored as layers usually hold them (outputs x
    inputs): w_gu (2 F x K), gate rows first, and w_down (K x F)."""

    def __init__(self, hidden, width, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(rows, cols):
            return torch.randn((rows, cols), generator=g, device="cuda").mul_(cols ** -0.5).to(dtype)
        self.w_gu, self.w_down = normal(2 * width, hidden), normal(hidden, width)
        self.master = [self.w_gu.float(), self.w_down.float()]
        self.grads = [torch.empty_like(self.w_gu), torch.empty_like(self.w_down)]

    def forward(self, x, save=False):
        h = tsffn.gated(x, self.w_gu.t(), act="silu", save=save)
        h, saved = h if save else (h, None)
        y = tsffn.linear(h, self.w_down.t(), residual=x)
        return (y, h, saved) if save else y

    def backward(self, dy, x, h, saved):
        """Weight gradients into self.grads; returns the gradient at x."""
        dh, _, _ = tsffn.linear_backward(dy, h, self.w_down.t(), dW=self.grads[1].t(), need=("dX",))
        dx, _ = tsffn.gated_backward(dh, x, self.w_gu.t(), saved, act="silu", dW=self.grads[0].t(), need=("dX",))
        return dx.add_(dy)  # the residual branch

    def step(self, x, target, lr, max_norm=1.0):
        """One step of gradient descent on the mean square error; returns
        (loss, gradient norm before clipping), on the device."""
        y, h, saved = self.forward(x, save=True)
        diff = y.float() - target
        loss = diff.square().mean()
        dy = (diff * (2.0 / diff.numel())).to(x.dtype)
        self.backward(dy, x, h, saved)
        norm = tsffn.clip_grad_norm(self.grads, max_norm)
        for w, m, g in zip((self.w_gu, self.w_down), self.master, self.grads):
            m.sub_(g, alpha=lr)
            w.copy_(m)
        return loss, norm

    def decode(self, x, h, y, handle=None):
        """The block on x (a few rows) into y, h between."""
        tsffn.gated(x, self.w_gu.t(), act="silu", H=h, handle=handle)
        return tsffn.linear(h, self.w_down.t(), residual=x, C=y, handle=handle)


def decode_graph(block, x):
    """(graph, y): replaying the graph runs the block on x's contents."""
    h = torch.empty((x.shape[0], block.w_down.shape[1]), dtype=x.dtype, device="cuda")
    y = torch.empty_like(x)
    handle = tsffn.Handle()  # the graph's own: it may be replayed on any stream
    block.decode(x, h, y, handle)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.decode(x, h, y, handle)
    graph.handle, graph.buffers = handle, (x, h, y)  # live as long as the graph
    return graph, y


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--width", type=int, default=2816)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    block = Block(a.hidden, a.width)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    target = x.float() + torch.randn((a.tokens, a.hidden), device="cuda") * 0.1
    losses = []
    for i in range(a.steps):
        loss, norm = block.step(x, target, lr=5.0, max_norm=0.05)
        losses.append(loss)
        if i % 5 == 0 or i == a.steps - 1:
            print("step %3d  loss %.4f  gradient norm %.4f" % (i, float(loss), float(norm)))
    graph, _ = decode_graph(block, x[:1].clone())
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(10):
        graph.replay()
    start.record()
    for _ in range(200):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print("decoding one token: %.2f us" % (start.elapsed_time(end) * 1e3 / 200))
    assert tsffn.status() == 0 and graph.handle.status() == 0
    return [float(v) for v in losses]


if __name__ == "__main__":
    main()
