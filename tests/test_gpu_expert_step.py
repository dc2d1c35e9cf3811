"""GPU: the step of a layer of experts (examples/expert_step.py) on small sizes, each of its operators against the oracle's 64 bits
on what reached it, and the gradients of the whole against the formula and its differences."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from conftest import ROOT
from oracle import adamw as OA
from oracle import experts as OE
from oracle import norm as ON

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from conftest import ensure_built
    ensure_built()
    spec = importlib.util.spec_from_file_location("expert_step", os.path.join(ROOT, "examples", "expert_step.py"))
    S = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(S)

E = 2.0 ** -24
BF16 = torch.bfloat16


def f64(t):
    return t.float().double().cpu().numpy()


def half(v):
    """Half of bf16's spacing around v."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 1e-37))) - 8)


def test_steps_match_the_oracle():
    P, rows, cols, experts, k, align = 2, 24, 64, 3, 2, 8
    g = torch.Generator(device="cuda").manual_seed(5)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(BF16)

    step = S.ExpertStep(P, rows, cols, experts, k, align=align)
    for t in (1, 2):
        stream_rows, dstream = [normal(rows, cols) for _ in range(P)], [normal(rows, cols) for _ in range(P)]
        before, dbefore = [f64(h) for h in stream_rows], [f64(d) for d in dstream]
        weight, bias = (f64(x) for x in step.parameters())
        saved = step.forward(stream_rows)
        torch.cuda.synchronize()
        tokens = P * rows
        for r in range(P):
            _, mean, rstd, y = ON.layer_forward(before[r], None, weight, bias, 1e-5)
            # h is 1 to 4 in size: the mean's 41 e of it times rstd times the weight, and 32 e of the rest
            slack = 200 * E * (np.abs(y) + np.abs(weight) + np.abs(bias))
            for q in range(P):
                assert (np.abs(f64(step.normed.outs[q][r * rows:(r + 1) * rows]) - y) <= half(y) + slack).all()
        everything = f64(step.normed.outs[0])
        ids, w = step.ids.outs[0].cpu().numpy(), f64(step.weights.outs[0])
        total = np.zeros((tokens, cols))
        for r in range(P):
            position, offsets, counts = (x.cpu().numpy() for x in saved["plan"][r])
            want = OE.route(ids, experts, r * experts, align, step.sort[r].most_rows(tokens))
            for got, x in zip((position, offsets, counts), want):
                assert np.array_equal(got, x)
            assert np.array_equal(f64(saved["rows"][r]), OE.dispatch(everything, position, offsets, counts, np.zeros(saved["rows"][r].shape)))
            out, size = OE.combine(f64(saved["results"][r]), position, w)
            assert (np.abs(f64(saved["partials"][r]) - out) <= half(out) * (out != 0) + (k + 1) * E * size).all()
            total += f64(saved["partials"][r])
        for r in range(P):                       # the reduce-scatter's sum of two bf16 is exact in f32, then rounded; so is h + sum
            new = before[r] + f64(torch.from_numpy(total[r * rows:(r + 1) * rows]).float().to(BF16))
            assert (np.abs(f64(stream_rows[r]) - new) <= half(new) * (new != 0)).all()

        matrices, dweight, dbias, pairs = step.backward(saved, dstream)
        torch.cuda.synchronize()
        dall = f64(step.dout.outs[0])
        dnormed = np.zeros((tokens, cols))
        for r in range(P):
            position, offsets, counts = (x.cpu().numpy() for x in saved["plan"][r])
            drows, dw, size = OE.combine_backward(dall, f64(saved["results"][r]), position, w, offsets, counts, np.zeros(saved["rows"][r].shape))
            assert (np.abs(f64(pairs[r]) - dw) <= 60 * E * size).all()
            # the matrices' gradient, from rows that were rounded to bf16 once more (2^-8 of each term)
            for e in range(experts):
                cut = slice(offsets[e], offsets[e] + counts[e])
                x = f64(saved["rows"][r])[cut]
                grad = x.T @ drows[cut]
                assert (np.abs(f64(matrices[r][e]) - grad) <= (2.0 ** -8 + 2.0 ** -10) * (np.abs(x).T @ np.abs(drows[cut])) + 1e-30).all()
            dnormed += f64(saved["dpartials"][r])
        total_w, total_b, size_w, size_b = (np.zeros(cols) for _ in range(4))
        for r in range(P):
            dy = f64(torch.from_numpy(dnormed[r * rows:(r + 1) * rows]).float().to(BF16))
            mean, rstd = f64(saved["mean"][r]), f64(saved["rstd"][r])
            dx, dw, db = ON.layer_backward(dy, before[r], weight, mean, rstd, dbefore[r])
            assert (np.abs(f64(dstream[r]) - dx) <= half(dx) + 50 * E * 100).all()      # terms are below 100
            total_w, total_b = total_w + dw, total_b + db
            size_w += np.abs(dy * (before[r] - mean[:, None]) * rstd[:, None]).sum(0)
            size_b += np.abs(dy).sum(0)
        assert (np.abs(f64(dweight) - total_w) <= 500 * E * size_w).all() and (np.abs(f64(dbias) - total_b) <= 500 * E * size_b).all()

        lr = 1e-2
        master = [f64(m) for m in step.master]
        old = [f64(m) for m in step.matrices]
        states = [[f64(x[0]).reshape(-1) for x in (own._lists["m"], own._lists["v"], own._lists["m_scales"], own._lists["v_scales"])]
                  for own, _ in step.optimizers]
        flats = [[f64(x[0]) for x in (shared._lists["m"], shared._lists["v"])] for _, shared in step.optimizers]
        step.update(matrices, dweight, dbias, t, lr)
        torch.cuda.synchronize()
        both = np.concatenate([f64(dweight), f64(dbias)]).reshape(P, -1)
        n = experts * cols * cols
        for r in range(P):
            p, _, _ = OA.step(master[r], both[r], *flats[r], t, lr, (0.9, 0.999), 1e-8, 0.0)
            assert (np.abs(f64(step.master[r]) - p) <= 3 * E * np.abs(p) + 60 * E * lr).all()
            assert torch.equal(step.params.outs[0][r], step.master[r].to(BF16))
            m, v = states[r][0] * OA.spread(states[r][2], n), (states[r][1] * OA.spread(states[r][3], n)) ** 2
            p, _, _ = OA.step(old[r].reshape(-1), f64(matrices[r]).reshape(-1), m, v, t, lr, (0.9, 0.999), 1e-8, 0.01)
            bits = OA.noise(r, t, 0, np.arange(n))[2]
            off = 3 * E * np.abs(p) + 200 * E * lr
            lo, hi = (OA.stochastic(p + s * off, bits, 8, 2.0 ** -126) for s in (-1, 1))
            got = f64(step.matrices[r]).reshape(-1)
            assert ((lo <= got) & (got <= hi)).all()
        for q in range(1, P):
            assert torch.equal(step.params.outs[q], step.params.outs[0])


def test_the_layer_s_gradient_is_that_of_the_formula():
    """Of the whole layer, with the choices and weights held, by autograd in 64 bits: what the bf16 values between the operators
    leave.  Each of the five on the way (normed rows, results, their gradients twice, the sums) is rounded by at most 2^-8 of itself, of
    which a row's product of 64 sees independent ones: a few 2^-8 / sqrt(3) together of a gradient's size; 0.02 of its norm is allowed."""
    P, rows, cols, experts, k = 2, 32, 64, 2, 2
    g = torch.Generator(device="cuda").manual_seed(6)
    step = S.ExpertStep(P, rows, cols, experts, k, align=4)
    stream_rows = [torch.randn(rows, cols, generator=g, device="cuda").to(BF16) for _ in range(P)]
    dstream = [torch.randn(rows, cols, generator=g, device="cuda").to(BF16) for _ in range(P)]
    x = torch.cat(stream_rows).double().requires_grad_()
    weight, bias = (p.double().requires_grad_() for p in step.parameters())
    matrices = [m.double().requires_grad_() for m in step.matrices]
    d = torch.cat(dstream).double()
    saved = step.forward(stream_rows)
    ids, pair_weights = step.ids.outs[0].long(), step.weights.outs[0].double()
    mean, var = x.mean(1, keepdim=True), x.var(1, keepdim=True, unbiased=False)
    y = (x - mean) / torch.sqrt(var + 1e-5) * weight + bias
    every = torch.cat(matrices)
    out = x + (torch.einsum("tc,tkcd->tkd", y, every[ids]) * pair_weights[:, :, None]).sum(1)
    out.backward(d)
    got, dweight, dbias, _ = step.backward(saved, dstream)

    def near(a, b):
        assert float((a.double() - b).norm() / b.norm()) < 0.02

    near(torch.cat(stream_rows), out.detach())
    near(torch.cat(dstream), x.grad)
    near(dweight, weight.grad)
    near(dbias, bias.grad)
    for a, b in zip(got, matrices):
        near(a, b.grad)


def test_the_example_runs():
    S.main()
