"""What a rank computes on its own block between a reduce-scatter and an all-gather, in one training step
of a sharded model on P virtual ranks of one GPU:

  forward    the ranks' partial sums of a layer's output are reduce-scattered; each rank adds its rows of
             the residual stream, norms them and writes 8-bit rows and their scales straight into its
             part of the gathered buffers; an all-gather sends both to every rank (half the bytes of bf16);
  backward   the partial gradients of the normed rows are reduce-scattered; each rank works out the
             gradient of its rows of the stream and its part of the weight's gradient;
  update     the gradients of the weight matrices are reduce-scattered, whole matrices to a rank; each rank
             orthogonalises its own through the momentum that it keeps, and an all-gather sends the
             updates to every rank.

    python examples/sharded_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import device_triggered_transfers_gb300 as D  # noqa: E402

CODES = torch.float8_e4m3fn


class ReduceScatter:
    """Rank b of P gets the sum of every rank's [P * rows, cols] bf16 partial over its block b of rows."""

    def __init__(self, P: int, rows: int, cols: int):
        self.P, self.rows, self.cols = P, rows, cols
        size = 2 * P * rows * cols * 2                     # the vector, then the slots
        self.bufs = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(P)]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.rs = D.AllReduce(self.bufs, size, "bf16", rows, cols, gather=False)

    def vector(self, r: int) -> torch.Tensor:
        n = self.P * self.rows * self.cols
        return self.bufs[r].view(torch.bfloat16)[:n].view(self.P * self.rows, self.cols)

    def __call__(self, partials, stream):
        """partials: a [P * rows, cols] tensor of every rank; returns rank b's block of the sum, a view."""
        for r, t in enumerate(partials):
            self.vector(r).copy_(t)
        torch.cuda.synchronize()         # a round's copiers take every SM: nothing else is to start during one
        handles = self.rs.start(stream)
        D.dtt_publish(handles, 0, self.P * self.P, stream=stream)
        self.rs.reduce(self.err, stream)
        self.rs.wait()
        self.rs.next_round()
        assert int(self.err.item()) == 0
        return [self.vector(b)[b * self.rows:(b + 1) * self.rows] for b in range(self.P)]


class AllGather:
    """Rank r's rows of its [P * rows, cols] output, to every rank."""

    def __init__(self, P: int, rows: int, cols: int, dtype: torch.dtype):
        self.P, self.rows = P, rows
        self.outs = [torch.zeros(P * rows, cols, device="cuda").to(dtype) for _ in range(P)]
        self.plan = D.prepare_all_gather(self.outs)

    def mine(self, r: int) -> torch.Tensor:
        return self.outs[r][r * self.rows:(r + 1) * self.rows]

    def __call__(self, stream) -> None:
        stream.synchronize()
        handles = self.plan.start(stream)
        D.dtt_publish(handles, 0, self.P, stream=stream)
        self.plan.wait()
        self.plan.next_round()


class ShardedStep:
    """P ranks with `rows` rows of the residual stream each, and `matrices` weight matrices of m x n each."""

    def __init__(self, P: int, rows: int, cols: int, matrices: int, m: int, n: int, group: int = 128, mu: float = 0.95):
        self.P, self.matrices, self.m, self.n = P, matrices, m, n
        self.stream = torch.cuda.Stream()
        self.norm = D.RMSNorm(cols, y="e4m3", group=group)
        self.scatter = ReduceScatter(P, rows, cols)
        self.codes = AllGather(P, rows, cols, CODES)
        self.scales = AllGather(P, rows, self.norm.scale_cols, torch.float32)
        self.ortho = D.Orthogonalizer(m, n, batch=matrices, mu=mu, nesterov=True)
        self.scatter_w = ReduceScatter(P, matrices * m, n)
        self.updates = AllGather(P, matrices * m, n, torch.bfloat16)
        self.momentum = [torch.zeros(matrices, m, n, device="cuda") for _ in range(P)]
        self.weight = torch.ones(cols, dtype=torch.bfloat16, device="cuda")

    def forward(self, partials, stream_rows):
        """partials: the ranks' bf16 partial outputs; stream_rows[r]: rank r's rows of the residual stream,
        updated in place.  Returns what the backward pass needs: every rank's rstd."""
        blocks = self.scatter(partials, self.stream)
        rstd = [torch.empty(b.shape[0], device="cuda") for b in blocks]
        for r, x in enumerate(blocks):
            self.norm.forward(x, self.weight, self.codes.mine(r), residual=stream_rows[r], residual_out=stream_rows[r],
                              scales=self.scales.mine(r), rstd=rstd[r], stream=self.stream)
        self.codes(self.stream)
        self.scales(self.stream)
        return rstd

    def backward(self, partials, stream_rows, rstd, dres):
        """partials: the ranks' bf16 partial gradients of the normed rows; dres[r]: the gradient that reaches
        rank r's rows of the stream from further on, replaced by theirs.  Returns the weight's gradient."""
        blocks = self.scatter(partials, self.stream)
        dweight = [torch.empty(self.norm.cols, device="cuda") for _ in blocks]
        for r, dy in enumerate(blocks):
            self.norm.backward(dy, stream_rows[r], self.weight, rstd[r], dres[r], dweight[r], dres=dres[r], stream=self.stream)
        self.stream.synchronize()
        return sum(dweight)

    def update(self, grads):
        """grads: the ranks' bf16 gradients of all P * matrices weights, [P * matrices * m, n].  Returns the
        orthogonalised updates of all of them as rank 0 has them."""
        blocks = self.scatter_w(grads, self.stream)
        for r, g in enumerate(blocks):
            shape = (self.matrices, self.m, self.n)
            self.ortho.run(g.view(shape), self.updates.mine(r).view(shape), momentum=self.momentum[r], stream=self.stream)
        self.updates(self.stream)
        assert self.ortho.errors == 0
        return self.updates.outs[0].view(self.P * self.matrices, self.m, self.n)


def main() -> None:
    P, rows, cols, matrices, m, n = 4, 1024, 4096, 2, 512, 1024
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    step = ShardedStep(P, rows, cols, matrices, m, n)
    stream_rows, dres = [normal(rows, cols) for _ in range(P)], [normal(rows, cols) for _ in range(P)]
    rstd = step.forward([normal(P * rows, cols) for _ in range(P)], stream_rows)
    y = step.codes.outs[1].float().view(P * rows, -1, 128) * step.scales.outs[1].unsqueeze(-1)
    print("normed rows as rank 1 has them: rms %.4f" % y.square().mean().sqrt())
    dweight = step.backward([normal(P * rows, cols) for _ in range(P)], stream_rows, rstd, dres)
    print("gradient of the weight: norm %.1f" % dweight.norm())
    u = step.update([normal(P * matrices * m, n) for _ in range(P)])
    s = torch.linalg.svdvals(u.float())
    print("singular values of the updates: %.3f to %.3f" % (s.min(), s.max()))


if __name__ == "__main__":
    main()
