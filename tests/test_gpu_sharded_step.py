"""GPU: the sharded step (examples/sharded_step.py) on small sizes against the oracle's 64 bits, with the
tolerances of test_gpu_ops.py (bf16 sums of the P partials are exact in f32 before their one rounding)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from conftest import ROOT
from oracle import norm as ON
from oracle import ortho as OO

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from conftest import ensure_built
    ensure_built()
    spec = importlib.util.spec_from_file_location("sharded_step", os.path.join(ROOT, "examples", "sharded_step.py"))
    S = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(S)


def test_two_steps_match_the_oracle():
    P, rows, cols, matrices, m, n, mu = 2, 32, 256, 2, 48, 96, 0.95
    g = torch.Generator(device="cuda").manual_seed(11)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    def f64(t):
        return t.float().double().cpu().numpy()

    step = S.ShardedStep(P, rows, cols, matrices, m, n, mu=mu)
    step.weight.copy_(1 + 0.2 * normal(cols))
    want_m = np.zeros((P, matrices, m, n))
    stream_rows = [normal(rows, cols) for _ in range(P)]
    for _ in range(2):
        before = [f64(t) for t in stream_rows]
        partials = [normal(P * rows, cols) for _ in range(P)]
        rstd = step.forward(partials, stream_rows)
        x = sum(t.float() for t in partials).to(torch.bfloat16)          # the reduce-scatter's own rounding
        for r in range(P):
            h, s, y = ON.forward(f64(x[r * rows:(r + 1) * rows]), before[r], f64(step.weight), 1e-6)
            np.testing.assert_allclose(f64(rstd[r]), s, rtol=2e-6)
            assert (np.abs(f64(stream_rows[r]) - h) <= np.abs(h) * 2.0 ** -8 + 1e-30).all()
            for q in range(P):                                           # every rank has every block
                codes, scales = (f64(t.outs[q][r * rows:(r + 1) * rows]) for t in (step.codes, step.scales))
                np.testing.assert_allclose(scales, ON.scales(y, 128), rtol=3e-6)
                spread = ON.spread(scales, 128, cols)
                assert (np.abs(codes * spread - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * spread) * 1.001).all()
        grads = [normal(P * rows, cols) for _ in range(P)]
        dres = [normal(rows, cols) for _ in range(P)]
        want = [f64(t) for t in dres]
        dweight = step.backward(grads, stream_rows, rstd, dres)
        dy = sum(t.float() for t in grads).to(torch.bfloat16)
        total, size = np.zeros(cols), np.zeros(cols)
        for r in range(P):
            mine = f64(dy[r * rows:(r + 1) * rows])
            dx, dw = ON.backward(mine, f64(stream_rows[r]), f64(step.weight), f64(rstd[r]), want[r])
            # bf16 rounding, and f32 errors of the terms (values here are below 100)
            assert (np.abs(f64(dres[r]) - dx) <= np.abs(dx) * 2.0 ** -8 + 100 * 50 * 2.0 ** -24).all()
            total += dw
            size += np.abs(mine * f64(stream_rows[r]) * f64(rstd[r])[:, None]).sum(axis=0)
        assert (np.abs(f64(dweight) - total) <= 500 * 2.0 ** -24 * size).all()
        wgrads = [normal(P * matrices * m, n) for _ in range(P)]
        u = step.update(wgrads)
        gsum = f64(sum(t.float() for t in wgrads).to(torch.bfloat16)).reshape(P, matrices, m, n)
        for r in range(P):
            for k in range(matrices):
                up, want_m[r, k] = OO.momentum_step(gsum[r, k], want_m[r, k], np.float32(mu), True)
                ref = OO.orthogonalize(up, 5, [(3.4445, -4.7750, 2.0315)] * 5, 1e-7)
                got = f64(u[r * matrices + k])
                assert np.linalg.norm(got - ref) < 9e-3 * np.linalg.norm(ref)
        for q in range(1, P):
            assert torch.equal(step.updates.outs[q], step.updates.outs[0])
