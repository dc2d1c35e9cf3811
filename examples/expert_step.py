"""A training step of a layer of experts, which are spread over P virtual ranks of one GPU:

  forward    each rank layer-norms its rows of the residual stream into its part of a gathered buffer and picks
             each row's experts; all-gathers send rows, choices and weights to every rank, which sorts the rows of
             its own experts, runs them, and adds the weighted results to its partial sum; a reduce-scatter
             returns the sums, which each rank adds to its rows;
  backward   an all-gather sends the rows' gradients to every rank, which works out those of its experts' rows
             and weights, runs its experts backwards, and brings its partial gradient of the normed rows back the
             same way; each rank then works out the gradient of its rows of the stream;
  update     AdamW on what each rank holds: its experts, whose weights no other rank has, with 8-bit states and bf16
             weights rounded at random; and its share of the norm's parameters, with f32 weights whose bf16 copy
             goes straight into an all-gather's buffer.

The router is given: its scores come from a fixed matrix, and its gradient stops at the weights.

    python examples/expert_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import device_triggered_transfers_gb300 as D  # noqa: E402
from examples.sharded_step import AllGather, ReduceScatter  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class ExpertStep:
    """P ranks with `rows` rows of `cols` columns each, and `experts` experts each, of cols x cols: y = x W."""

    def __init__(self, P: int, rows: int, cols: int, experts: int, top_k: int, align: int = 16, seed: int = 0):
        self.P, self.rows, self.cols, self.experts, self.top_k = P, rows, cols, experts, top_k
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.stream = torch.cuda.Stream()
        self.norm = D.LayerNorm(cols)
        self.sort = [D.ExpertRows(experts, top_k, first=r * experts, align=align) for r in range(P)]
        self.normed, self.dout = AllGather(P, rows, cols, BF16), AllGather(P, rows, cols, BF16)
        self.ids, self.weights = AllGather(P, rows, top_k, torch.int32), AllGather(P, rows, top_k, F32)
        self.scatter = ReduceScatter(P, rows, cols)
        self.router = torch.randn(cols, P * experts, generator=g, device="cuda")
        self.matrices = [(torch.randn(experts, cols, cols, generator=g, device="cuda") / cols ** 0.5).to(BF16) for _ in range(P)]
        # weight and bias in one row of 2 cols, a part of it each rank's, as all ranks have them and as f32
        share = 2 * cols // P
        self.params = AllGather(P, 1, share, BF16)
        for out in self.params.outs:
            out.view(-1)[:cols] = 1.0
        self.master = [self.params.mine(r).float().view(-1) for r in range(P)]
        self.optimizers = []
        for r in range(P):
            n = experts * cols * cols
            states = [torch.zeros(n, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
            scales = [torch.zeros(D.AdamW.blocks(n), device="cuda") for _ in range(2)]
            flat = [torch.zeros(share, device="cuda") for _ in range(3)]
            matrix = self.matrices[r]
            self.optimizers.append((
                D.AdamW([matrix], [torch.zeros_like(matrix, dtype=F32)], [states[0]], [states[1]], m_scales=[scales[0]],
                        v_scales=[scales[1]], seed=seed + r),
                D.AdamW([self.master[r]], [flat[0]], [flat[1]], [flat[2]], copies=[self.params.mine(r).view(-1)], weight_decay=0.0)))

    def parameters(self):
        """(weight, bias) as every rank has them."""
        both = self.params.outs[0].view(-1)
        return both[:self.cols], both[self.cols:]

    def experts_of(self, r: int, rows: torch.Tensor, counts, offsets, backward=None):
        """Rank r's experts, one after the other; with `backward`, its rows' gradients and the matrices'."""
        out = torch.zeros_like(rows)
        grads = torch.zeros(self.matrices[r].shape, device="cuda") if backward is not None else None
        for e, (at, n) in enumerate(zip(offsets.tolist(), counts.tolist())):
            x = rows[at:at + n]
            if backward is None:
                out[at:at + n] = x @ self.matrices[r][e]
            else:
                out[at:at + n] = backward[at:at + n] @ self.matrices[r][e].t()
                grads[e] = x.float().t() @ backward[at:at + n].float()
        return out if backward is None else (out, grads)

    def forward(self, stream_rows):
        """stream_rows[r]: rank r's bf16 rows of the residual stream, updated in place.  Returns what the backward pass
        needs, among it the rows as they were."""
        weight, bias = self.parameters()
        saved = {"h": [h.clone() for h in stream_rows], "mean": [], "rstd": [], "plan": [], "rows": [], "results": []}
        with torch.cuda.stream(self.stream):
            self.stream.wait_stream(torch.cuda.default_stream())
            for r, h in enumerate(saved["h"]):
                mean, rstd = torch.empty(self.rows, device="cuda"), torch.empty(self.rows, device="cuda")
                self.norm.forward(h, weight, bias, self.normed.mine(r), mean=mean, rstd=rstd, stream=self.stream)
                saved["mean"].append(mean)
                saved["rstd"].append(rstd)
                scores, ids = (self.normed.mine(r).float() @ self.router).topk(self.top_k, dim=1)
                self.ids.mine(r).copy_(ids)
                self.weights.mine(r).copy_(torch.softmax(scores, dim=1))
        for gather in (self.normed, self.ids, self.weights):
            gather(self.stream)
        partials = []
        for r, sort in enumerate(self.sort):
            tokens = self.P * self.rows
            position = torch.empty(tokens, self.top_k, dtype=torch.int32, device="cuda")
            offsets, counts = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (self.experts + 1, self.experts))
            rows = torch.zeros(sort.most_rows(tokens), self.cols, dtype=BF16, device="cuda")
            sort.route(self.ids.outs[r], position, offsets, counts)
            sort.dispatch(self.normed.outs[r], position, offsets, counts, rows)
            results = self.experts_of(r, rows, counts, offsets)
            partial = torch.empty(tokens, self.cols, dtype=BF16, device="cuda")
            sort.combine(results, position, partial, weights=self.weights.outs[r])
            partials.append(partial)
            saved["plan"].append((position, offsets, counts))
            saved["rows"].append(rows)
            saved["results"].append(results)
        saved["partials"] = partials
        for h, block in zip(stream_rows, self.scatter(partials, self.stream)):
            h.add_(block)
        return saved

    def backward(self, saved, dstream):
        """dstream[r]: the gradient that reaches rank r's rows of the stream, replaced by that of the rows before the layer.
        Returns the gradients of every rank's matrices, of the weight and of the bias (these two added over ranks), and of the
        pairs' weights as each rank has its part of them."""
        weight, _ = self.parameters()
        torch.cuda.synchronize()
        for r, d in enumerate(dstream):
            self.dout.mine(r).copy_(d)
        torch.cuda.synchronize()
        self.dout(self.stream)
        partials, matrices, pairs = [], [], []
        for r, sort in enumerate(self.sort):
            position, offsets, counts = saved["plan"][r]
            drows = torch.zeros_like(saved["rows"][r])
            dweights = torch.empty(self.P * self.rows, self.top_k, device="cuda")
            sort.combine_backward(self.dout.outs[r], saved["results"][r], position, self.weights.outs[r], offsets, counts, drows, dweights)
            dx, grads = self.experts_of(r, saved["rows"][r], counts, offsets, backward=drows)
            partial = torch.empty(self.P * self.rows, self.cols, dtype=BF16, device="cuda")
            sort.combine(dx, position, partial)
            partials.append(partial)
            matrices.append(grads)
            pairs.append(dweights)
        saved["dpartials"] = partials
        blocks = self.scatter(partials, self.stream)
        sums = torch.zeros(2, self.cols, device="cuda")
        for r, (d, block) in enumerate(zip(dstream, blocks)):
            mine = torch.empty(2, self.cols, device="cuda")
            self.norm.backward(block, saved["h"][r], weight, saved["mean"][r], saved["rstd"][r], d, mine[0], mine[1], dres=d)
            sums += mine
        return matrices, sums[0], sums[1], pairs

    def update(self, matrices, dweight, dbias, step: int, lr: float):
        """One step of every rank's optimizers; the norm's new parameters go to every rank."""
        both = torch.cat([dweight, dbias]).chunk(self.P)
        torch.cuda.synchronize()
        for r, (own, shared) in enumerate(self.optimizers):
            own.run(lr, step, grads=[matrices[r]], stream=self.stream)
            shared.run(lr, step, grads=[both[r].contiguous()], stream=self.stream)
        self.params(self.stream)


def main() -> None:
    P, rows, cols, experts, top_k = 4, 512, 1024, 4, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    step = ExpertStep(P, rows, cols, experts, top_k)
    for t in range(1, 4):
        stream_rows = [torch.randn(rows, cols, generator=g, device="cuda").to(BF16) for _ in range(P)]
        dstream = [(0.1 * torch.randn(rows, cols, generator=g, device="cuda")).to(BF16) for _ in range(P)]
        saved = step.forward(stream_rows)
        matrices, dweight, dbias, _ = step.backward(saved, dstream)
        step.update(matrices, dweight, dbias, t, 1e-3)
        loads = torch.cat([plan[2] for plan in saved["plan"]])
        print("step %d: rows of an expert %d to %d, gradient of the norm's weight %.3f, of the matrices %.3f" % (
            t, loads.min(), loads.max(), dweight.norm(), torch.stack([m.norm() for m in matrices]).norm()))


if __name__ == "__main__":
    main()
