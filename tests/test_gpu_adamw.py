"""GPU: AdamW over lists of tensors against the oracle's 64 bits, a step at a time from the states as they were.

Tolerances, from the arithmetic (e = 2^-24): m and v are two products and a fused sum of the inputs, which with the
gradient's scale, a code's scale and beta's own rounding are within 5 e and 9 e (v squares the gradient, and a root's code)
of the terms' magnitudes.  The root is half of v's error and an ulp, the quotient's sum, reciprocal and products 8 e: the
change of p is off by 20 e of its own size and by m's error over the denominator; p itself takes 3 e.  A code is the
value by the block's scale, to the nearest within half a spacing (e4m3: 4 significant bits, smallest normal 2^-6), or what
stochastic rounding makes of some value within that error."""
import sys

import numpy as np
import pytest
import torch

from oracle import adamw as OA

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from conftest import ensure_built
    ensure_built()
    import device_triggered_transfers_gb300 as D

E = 2.0 ** -24
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = {"bf16": BF16, "f32": F32, "e4m3": E4M3}
LR, BETAS, EPS = 1e-2, (0.9, 0.99), 1e-8


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def f64(t):
    return t.to(F32).double().cpu().numpy()


class Lists:
    """Tensors of the given sizes inside buffers with sevens around them, `shift` elements off their alignment."""

    def __init__(self, sizes, param="f32", grad="bf16", state="f32", copy=False, seed=None, shift=0, decay=0.1, zero=False, gap=16, one_seed=0):
        self.sizes, self.small, self.seed, self.gap = sizes, state == "e4m3", seed, gap
        g = gen(one_seed)
        self.buffers = {}

        def lists(name, kind, make, count=lambda n: n):
            starts, at = [], gap + shift
            for n in sizes:
                starts.append(at)
                at += -(-count(n) // 16) * 16 + gap
            flat = torch.full((at + gap,), 7.0, device="cuda").to(TYPES[kind])
            views = []
            for a, n in zip(starts, sizes):
                v = flat[a:a + count(n)]
                v.copy_(make(count(n)).to(TYPES[kind]))
                views.append(v)
            self.buffers[name] = (flat, starts, [count(n) for n in sizes])
            return views

        rand = lambda n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
        # gradients over a few orders of magnitude, some of them zero
        grads = lambda n: 1e-3 * rand(n) * torch.exp(2 * rand(n)) * (torch.rand(n, generator=g, device="cuda") > 0.1)  # noqa: E731
        none = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
        self.p = lists("param", param, lambda n: 0.1 * rand(n))
        self.g = lists("grad", grad, grads)
        self.copies = lists("copy", "bf16", rand) if copy else None
        self.ms = self.vs = None
        if self.small:
            self.m = lists("m", "e4m3", none if zero else lambda n: 100 * rand(n))
            self.v = lists("v", "e4m3", none if zero else lambda n: 100 * rand(n).abs())
            self.ms = lists("m_scales", "f32", none if zero else lambda n: 1e-6 * (1 + torch.rand(n, generator=g, device="cuda")), D.AdamW.blocks)
            self.vs = lists("v_scales", "f32", none if zero else lambda n: 1e-5 * (1 + torch.rand(n, generator=g, device="cuda")), D.AdamW.blocks)
        else:
            self.m = lists("m", "f32", none if zero else lambda n: 1e-3 * rand(n))
            self.v = lists("v", "f32", none if zero else lambda n: 1e-6 * rand(n).square())
        self.decay = [decay * (i % 3) for i in range(len(sizes))]
        self.op = D.AdamW(self.p, self.g, self.m, self.v, m_scales=self.ms, v_scales=self.vs, copies=self.copies, betas=BETAS, eps=EPS,
                          weight_decay=self.decay, seed=seed)

    def state(self):
        return [{k: None if t is None else t[i].clone() for k, t in (("p", self.p), ("g", self.g), ("m", self.m), ("v", self.v), ("ms", self.ms), ("vs", self.vs))}
                for i in range(len(self.sizes))]

    def check_gaps(self):
        for name, (flat, starts, counts) in self.buffers.items():
            left = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
            for a, n in zip(starts, counts):
                left[a:a + n] = False
            assert (flat[left].float() == 7).all(), name

    def check(self, before, t, scale=1.0, lr=LR):
        """The tensors against one step from `before`."""
        self.check_gaps()
        for i, n in enumerate(self.sizes):
            if n:
                self.check_one(i, n, before[i], t, scale, lr)

    def check_one(self, i, n, b, t, scale, lr):
        p, g, m, v = (f64(b[k]) for k in "pgmv")
        if self.small:
            m, v = m * OA.spread(f64(b["ms"]), n), (v * OA.spread(f64(b["vs"]), n)) ** 2
        want_p, want_m, want_v = OA.step(p, g, m, v, t, lr, BETAS, EPS, self.decay[i], scale)
        size_m = BETAS[0] * np.abs(m) + (1 - BETAS[0]) * np.abs(g * scale)
        off_m = 5 * E * size_m
        change = np.abs(want_p - p * (1 - lr * self.decay[i]))
        denom = np.sqrt(want_v) / np.sqrt(1 - BETAS[1] ** t) + EPS
        off_p = 3 * E * np.abs(p) + 20 * E * change + lr / (1 - BETAS[0] ** t) * off_m / denom
        noise = [None] * 3 if self.seed is None else OA.noise(self.seed, t, i, np.arange(n))
        got, nan = f64(self.p[i]), np.isnan(want_p)          # random codes of m, a standard deviation of 100, now and then
        if self.p[i].dtype == F32:                           # one past 448, which is NaN
            lo, hi = want_p - off_p, want_p + off_p
            if self.copies is not None:
                assert torch.equal(self.copies[i], self.p[i].to(BF16))
        elif self.seed is None:
            half = OA.spacing(want_p, 8, 1e-37) / 2
            lo, hi = want_p - half - off_p, want_p + half + off_p
        else:
            lo, hi = (OA.stochastic(want_p + s * off_p, noise[2], 8, 2.0 ** -126) for s in (-1, 1))
        assert np.array_equal(np.isnan(got), nan) and ((lo <= got) & (got <= hi))[~nan].all()
        if not self.small:
            assert (np.abs(f64(self.m[i]) - want_m) <= off_m).all()
            assert (np.abs(f64(self.v[i]) - want_v) <= 9 * E * want_v).all()
            return
        for codes, scales, x, off, bits in ((self.m[i], self.ms[i], want_m, off_m, noise[0]), (self.v[i], self.vs[i], np.sqrt(want_v), 7 * E * np.sqrt(want_v), noise[1])):
            c, s = f64(codes), f64(scales)
            pad = lambda a: np.concatenate([a, np.zeros(-n % OA.BLOCK)]).reshape(-1, OA.BLOCK).max(1)  # noqa: E731
            nan = np.isnan(pad(x))                           # a block with a NaN is NaN
            assert np.array_equal(np.isnan(s), nan) and (np.abs(s - OA.scales(x)) <= (pad(off) / 448 + 4 * E * s))[~nan].all()
            s, fine = OA.spread(s, n), ~OA.spread(nan, n)
            assert np.isnan(c[~fine]).all()
            c, s, x, off, bits = (None if a is None else a[fine] for a in (c, s, x, off, bits))
            x, off = x / s, off / s + 4 * E * np.abs(x / s)
            if bits is None:
                lo, hi = x - off - OA.spacing(np.abs(x) - off, 4, 2.0 ** -6) / 2, x + off + OA.spacing(np.abs(x) + off, 4, 2.0 ** -6) / 2
            else:
                # below 2^-6 the value is moved to [2^-6, 2^-5) and rounded there once: half an ulp of that
                off = np.maximum(off, 2.0 ** -29)
                lo, hi = (OA.stochastic(np.sign(x) * np.maximum(np.abs(x) + k * off, 0), bits, 4, 2.0 ** -6) for k in (-1, 1))
                lo, hi = np.minimum(lo, hi), np.maximum(lo, hi)
            if codes is self.v[i]:
                assert ((c > 0) == (x > 0)).all()
                hi = np.maximum(hi, 2.0 ** -9)
                lo = np.where(x > 0, np.maximum(lo, 2.0 ** -9), 0)
            lo, hi = np.clip(lo, -448, 448), np.clip(hi, -448, 448)
            assert ((lo <= c) & (c <= hi)).all()


SIZES = [1, 2, 7, 8, 9, 127, 128, 129, 255, 257, 2047, 2048, 2049, 4096, 5000, 10001, 131]
KINDS = [(p, g, s, seed) for p in ("f32", "bf16") for g in ("f32", "bf16") for s in ("f32", "e4m3") for seed in (None, 77)]


@pytest.mark.parametrize("param,grad,state,seed", KINDS)
@pytest.mark.parametrize("shift", [0, 8, 1])
def test_steps(param, grad, state, seed, shift):
    """Tensors that are 16-byte aligned, all 8 elements off it (f32 still is), and not at all."""
    a = Lists(SIZES, param, grad, state, copy=param == "f32" and shift != 8, seed=seed, shift=shift)
    for t in (1, 2, 1000):
        before = a.state()
        a.op.run(LR, t)
        a.check(before, t)


@pytest.mark.parametrize("param,state,seed", [("f32", "f32", None), ("bf16", "e4m3", 5), ("f32", "e4m3", None)])
def test_tensors_back_to_back(param, state, seed):
    """Views of flat buffers, all of one offset, as a rank's share of a model's weights has them."""
    sizes, copy = [4096, 4097, 3, 20000, 12, 5000, 4095, 8], param == "f32"
    a = Lists([sum(sizes)], param, "bf16", state if state == "f32" else "f32", copy=copy, seed=seed)
    starts = np.cumsum([0] + sizes)
    cut = lambda flat: [flat[s:s + n] for s, n in zip(starts, sizes)]  # noqa: E731
    a.p, a.g, a.copies = cut(a.p[0]), cut(a.g[0]), cut(a.copies[0]) if copy else None
    a.sizes, a.decay = sizes, [0.1 * (i % 3) for i in range(len(sizes))]
    if state == "e4m3":
        a.small = True
        a.m, a.v = (cut(torch.zeros(sum(sizes), device="cuda").to(E4M3)) for _ in range(2))
        a.ms, a.vs = ([torch.zeros(D.AdamW.blocks(n), device="cuda") for n in sizes] for _ in range(2))
    else:
        a.m, a.v = cut(a.m[0]), cut(a.v[0])
    a.op = D.AdamW(a.p, a.g, a.m, a.v, m_scales=a.ms, v_scales=a.vs, copies=a.copies, betas=BETAS, eps=EPS, weight_decay=a.decay, seed=seed)
    for t in (1, 2):
        before = a.state()
        a.op.run(LR, t)
        a.check(before, t)


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_from_nothing(state):
    """States and their scales all zero: elements without a gradient keep their weight and stay zero."""
    a = Lists(SIZES, "f32", "f32", state, zero=True, decay=0.0)
    before = a.state()
    a.op.run(LR, 1)
    a.check(before, 1)
    for p, g, m, v, b in zip(a.p, a.g, a.m, a.v, before):
        idle = g == 0
        assert torch.equal(p[idle], b["p"][idle]) and not m.float()[idle].any() and not v.float()[idle].any()


@pytest.mark.parametrize("count", [49, 384, 385, 1000])
@pytest.mark.parametrize("state,seed", [("f32", None), ("e4m3", 9)])
def test_many_tensors_and_empty_ones(count, state, seed):
    """More than one launch's table holds, empty tensors among them: numbers, and so the random bits, go by the list."""
    sizes = [0 if i % 7 == 3 else 1 + (i * 37) % 300 for i in range(count)]
    a = Lists(sizes, "bf16", "f32", state, seed=seed)
    before = a.state()
    a.op.run(LR, 4)
    a.check(before, 4)


@pytest.mark.parametrize("state,seed", [("f32", None), ("e4m3", 3)])
def test_scale_of_the_gradients_and_other_gradients(state, seed):
    a = Lists([5000, 77], "bf16", "bf16", state, seed=seed)
    scale = torch.full((1,), 0.25, device="cuda")
    before = a.state()
    a.op.run(LR, 3, grad_scale=scale)
    a.check(before, 3, scale=0.25)
    before = a.state()
    others = [torch.randn(n + 1, generator=gen(n), device="cuda").to(BF16)[1:] for n in a.sizes]
    for b, g in zip(before, others):
        b["g"] = g
    a.op.run(LR, 4, grads=others)
    a.check(before, 4)
    for bad in (others[:1], [others[0], others[1].float()], [others[0], others[1][:-1]], [others[0].cpu(), others[1]]):
        with pytest.raises(D.DttError):
            a.op.run(LR, 5, grads=bad)


@pytest.mark.parametrize("state,seed", [("f32", None), ("e4m3", 3)])
def test_a_captured_step_counts_and_takes_the_rate_from_the_device(state, seed):
    a = Lists([5000, 77, 2048], "bf16", "bf16", state, seed=seed)
    lr, step, scale = torch.full((1,), LR, device="cuda"), torch.full((1,), 5, dtype=torch.int32, device="cuda"), torch.full((1,), 0.5, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        a.op.run(lr, step, grad_scale=scale, stream=stream)
    for t, rate in ((6, LR), (7, 3 * LR), (8, 0.0)):
        lr.fill_(rate)
        before = a.state()
        graph.replay()
        torch.cuda.synchronize()
        assert int(step) == t
        # the device's own 1 - beta^t is within a few ulp of the host's
        a.check(before, t, scale=0.5, lr=float(lr))
    # and uncaptured, back to back
    for t in (9, 10):
        before = a.state()
        a.op.run(lr, step)
        assert int(step) == t
        a.check(before, t, lr=0.0)


def test_the_same_call_gives_the_same_bits_and_another_seed_others():
    runs = []
    for seed in (4, 4, 5):
        a = Lists([10001], "bf16", "bf16", "e4m3", seed=seed)
        for t in (1, 2, 3):
            a.op.run(LR, t)
        runs.append([t.view(torch.uint8).clone() for t in (a.p[0], a.m[0], a.v[0])])
    assert all(torch.equal(x, y) for x, y in zip(runs[0], runs[1]))
    assert not any(torch.equal(x, y) for x, y in zip(runs[0], runs[2]))


def test_a_shift_of_the_tensor_changes_nothing():
    """The aligned and the element path give the same bits."""
    for param, grad, state, seed in KINDS:
        runs = []
        for shift in (0, 1):
            a = Lists([5000, 129], param, grad, state, seed=seed, shift=shift)
            a.op.run(LR, 2)
            runs.append([t.clone() for k in (a.p, a.m, a.v, a.ms or [], a.vs or []) for t in k])
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(*runs)), (param, grad, state, seed)


def test_rounding_at_random_keeps_the_mean_where_nearest_stands_still():
    """A weight of 1 in bf16 and changes of 2^-11 (a sixteenth of its spacing below): nearest never moves, at random 4000 weights move
    by 30 such changes on average.  One step up or down of 2^-8 has a variance of at most 2^-8 x 2^-11 a step: the mean of 4000 after
    30 steps is within six of sqrt(30 x 2^-19 / 4000) = 1.2e-4 of it; the moments' own rounding moves the changes by a few per cent."""
    n, steps = 4000, 30
    moved = {}
    for seed in (None, 11):
        p, g = torch.ones(n, dtype=BF16, device="cuda"), torch.ones(n, device="cuda")
        m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        op = D.AdamW([p], [g], [m], [v], betas=(0.0, 0.0), eps=1e-12, weight_decay=0.0, seed=seed)
        for t in range(1, steps + 1):
            op.run(2.0 ** -11, t)
        moved[seed] = float((1 - p.double()).mean())
    assert moved[None] == 0
    assert abs(moved[11] - steps * 2.0 ** -11) < 6 * 1.2e-4


def test_codes_rounded_at_random_follow_a_slow_average():
    """v of beta2 = 0.999 falls by 0.1 % a step without gradients: a root's code is to fall on average as it does, where nearest stands
    still but for the block's largest.  1000 steps take the root to 0.606 of itself.  A code's rounding is off by at most a spacing,
    an eighth of the value, a step with probability 0.0005 x 8: a variance of 0.0005 / 8 of the value squared a step, together 0.06, so the
    mean of 12700 elements is within six of 0.25 / sqrt(12700) = 0.0022."""
    n = 12800
    for seed in (None, 13):
        p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        x = 1 + torch.rand(n, generator=gen(1), device="cuda")
        x[::128] = 448.0                                        # each block's largest keeps the scale
        m, v = torch.zeros(n, device="cuda").to(E4M3), (16 * x).clamp(max=448).to(E4M3)
        start = v.double()
        ms, vs = torch.zeros(n // 128, device="cuda"), torch.ones(n // 128, device="cuda")
        op = D.AdamW([p], [g], [m], [v], m_scales=[ms], v_scales=[vs], betas=(0.9, 0.999), weight_decay=0.0, seed=seed)
        g[::128] = 448.0                                        # holds its v where it is
        for t in range(1, 1001):
            op.run(0.0, t)
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        rest[::128] = False
        ratio = float(((v.double() * vs.double().repeat_interleave(128)) / start)[rest].mean())
        assert abs(ratio - (1.0 if seed is None else 0.999 ** 500)) < (1e-3 if seed is None else 6 * 0.0022)


def alike_blocks(n):
    """(gradient, code of m, of v, scale of m, of v) that a block's elements share, of n / 128 blocks, f32."""
    rng, blocks = np.random.default_rng(3), n // OA.BLOCK
    f = lambda x: x.astype(np.float32)  # noqa: E731
    codes = np.concatenate([np.arange(8, 16) * 2.0 ** e for e in range(-3, 5)])
    return (f(1e-3 * rng.standard_normal(blocks)), f(rng.choice(codes, blocks) * rng.choice([-1, 1], blocks)), f(rng.choice(codes, blocks)),
            f(1e-6 * (1 + rng.random(blocks))), f(1e-5 * (1 + rng.random(blocks))))


def largest_code(x):
    """Of a block's largest x by its scale, rounded down, each operation of f32 by itself."""
    f = np.float32
    return np.where(x * (f(1) / (x * f(1 / 448))) < f(448), 0x7D, 0x7E)


@pytest.mark.parametrize("shift", [0, 1])
def test_a_blocks_largest_with_a_noise_of_0_has_the_formulas_code(shift):
    """It is 448 or an ulp below, and 448's code or the one below, by the formula's roundings alone.  Elements of a block are alike,
    so that each is its largest; one in 65536 has a noise of 0."""
    n, seed, f = 1 << 21, 5, np.float32
    g, m, v, ms, vs = alike_blocks(n)
    a = Lists([n], "bf16", "f32", "e4m3", seed=seed, shift=shift)
    for name, x in (("g", g), ("m", m), ("v", v)):
        t = getattr(a, name)[0]
        t.copy_(torch.from_numpy(OA.spread(x, n)).cuda().to(t.dtype))
    a.ms[0].copy_(torch.from_numpy(ms))
    a.vs[0].copy_(torch.from_numpy(vs))
    a.op.run(LR, 3)
    noise_m, noise_v, _ = OA.noise(seed, 3, 0, np.arange(n))
    new_m = f(BETAS[0]) * (m * ms) + f(1 - BETAS[0]) * g
    root = v * vs
    new_root = np.sqrt(f(BETAS[1]) * (root * root) + f(1 - BETAS[1]) * g * g)
    for got, new, noise in ((a.m[0], new_m, noise_m), (a.v[0], new_root, noise_v)):
        code = largest_code(np.abs(new))
        assert len(set(code)) == 2 and (noise == 0).sum() > 16
        want = np.where(noise == 0, OA.spread(code, n), 0x7E) | np.where(OA.spread(new, n) < 0, 0x80, 0)
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), want)


@pytest.mark.parametrize("shift", [0, 1])
def test_blocks_of_zeros_stay_zero_with_any_noise(shift):
    a = Lists([1 << 21], "bf16", "f32", "e4m3", seed=5, shift=shift, zero=True)
    a.g[0].zero_()
    a.op.run(LR, 1)
    for t in (a.m[0], a.v[0]):
        assert not t.view(torch.uint8).any()
    for t in (a.ms[0], a.vs[0]):
        assert (t == OA.SCALE_MIN).all()


def test_a_small_decay_is_that_of_its_size():
    """Of 1e-6, where 1 - 1e-6 in f32 is 1.3 % off: weights without gradients shrink by 1e-6 on average, each product and sum
    rounded by half an ulp (2^-24 of the weight) at random, of which a million's mean keeps a thousandth; six of that is allowed."""
    n = 1 << 20
    p = 1 + torch.rand(n, generator=gen(3), device="cuda")
    before = p.double()
    zeros = [torch.zeros(n, device="cuda") for _ in range(3)]
    D.AdamW([p], zeros[:1], zeros[1:2], zeros[2:], weight_decay=0.1).run(1e-5, 1)
    assert abs(float(((before - p.double()) / before).mean()) - 1e-6) < 6 * 2 * E / 1024


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("state,seed", [("f32", None), ("e4m3", None), ("e4m3", 3)])
def test_nan_and_infinity_stay_in_their_element_or_block(state, seed, shift):
    a = Lists([1000], "f32", "f32", state, shift=shift, seed=seed)
    a.g[0][200] = float("nan")
    a.g[0][700] = float("inf")
    before = a.p[0].clone()
    a.op.run(LR, 1)
    p, m, v = a.p[0], a.m[0].float(), a.v[0].float()
    assert torch.isnan(p[200]) and torch.isfinite(p).sum() >= 998
    if state == "f32":
        assert torch.isnan(m[200]) and torch.isnan(v[200]) and torch.isinf(v[700])
        assert torch.isfinite(torch.cat([m[:200], m[201:700], m[701:], v[:200], v[201:700], v[701:]])).all()
    else:
        assert torch.isnan(a.ms[0][1]) and torch.isnan(a.vs[0][1]) and torch.isnan(m[128:256]).all() and torch.isnan(v[128:256]).all()
        assert torch.isinf(a.ms[0][5]) and torch.isinf(a.vs[0][5])
        for s in (a.ms[0], a.vs[0]):
            assert torch.isfinite(s).sum() == 6
        for q in (m, v):
            assert torch.isfinite(q[:128]).all() and torch.isfinite(q[256:640]).all() and torch.isfinite(q[768:]).all()
    assert torch.isfinite(before).all()
    a.g[0].fill_(1e-3)
    a.op.run(LR, 2)
    if state == "e4m3":
        assert torch.isnan(a.p[0][128:256]).all() and torch.isnan(a.p[0][640:768]).all()
        assert torch.isfinite(a.p[0][:128]).all() and torch.isfinite(a.p[0][768:]).all()


def test_tiny_and_huge_gradients():
    """v is f32: a gradient below 1e-22 leaves no root, one above 1e19 an infinite one, whose step is zero."""
    for state in ("f32", "e4m3"):
        a = Lists([256], "f32", "f32", state, zero=True, decay=0.0)
        a.g[0].fill_(1e-25)
        a.g[0][128:] = 1e25
        before = a.p[0].clone()
        a.op.run(LR, 1)
        # 1e-26 / 1e-8 of the rate
        assert (a.p[0][:128] - before[:128]).abs().max() < 1e-6 and torch.equal(a.p[0][128:], before[128:])


def between(got, lo, hi):
    assert ((lo <= got) & (got <= hi)).all()


def tiny(n, grad):
    """Gradients from 1e-21 to 1e-17, some zero, both signs."""
    g = 10 ** (-21 + 4 * torch.rand(n, generator=gen(n), device="cuda")) * torch.randn(n, generator=gen(n + 1), device="cuda").sign()
    return (g * (torch.rand(n, generator=gen(n + 2), device="cuda") > 0.1)).to(TYPES[grad])


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_a_subnormal_v_has_its_root(grad, shift, monkeypatch):
    """Gradients that leave v = (1 - beta2) g^2 below 2^-126, with an eps that does not hide its root.  v's square and sum are each rounded
    to a multiple of 2^-149, half of that off at most, beside the 9 e of normal values; the step lies between those of the least and
    the largest such v."""
    monkeypatch.setattr(sys.modules[__name__], "EPS", 1e-25)
    a = Lists([5000, 129, 3], "f32", grad, "f32", shift=shift, zero=True, decay=0.0)
    for t in (1, 2, 1000):
        for i, n in enumerate(a.sizes):
            a.g[i].copy_(tiny(n + t, grad)[:n])
        before = a.state()
        a.op.run(LR, t)
        a.check_gaps()
        for i, b in enumerate(before):
            p, g, m, v = (f64(b[k]) for k in "pgmv")
            _, want_m, want_v = OA.step(p, g, m, v, t, LR, BETAS, EPS, 0.0)
            off_m = 5 * E * (BETAS[0] * np.abs(m) + (1 - BETAS[0]) * np.abs(g))
            assert (np.abs(f64(a.m[i]) - want_m) <= off_m).all()
            off = 9 * E * want_v + 2 * 2.0 ** -150
            between(f64(a.v[i]), want_v - off, want_v + off)
            assert t > 1 or i > 0 or ((want_v > 0) & (want_v < 2.0 ** -126)).sum() > 0.5 * len(p)
            most, least = (LR / (1 - BETAS[0] ** t) / (np.sqrt(np.maximum(want_v + k * off, 0)) / np.sqrt(1 - BETAS[1] ** t) + EPS) for k in (-1, 1))
            lo, hi = least * np.abs(want_m), most * np.abs(want_m)
            change = (p - f64(a.p[i])) * np.where(want_m < 0, -1, 1)
            few = np.where(want_v > 0, 3 * E * np.abs(p) + 20 * E * hi + most * off_m, 0)
            between(change, lo - few, hi + few)


@pytest.mark.parametrize("param,grad,seed", [("f32", "f32", None), ("bf16", "bf16", 3), ("f32", "bf16", 5)])
@pytest.mark.parametrize("shift", [0, 1])
def test_roots_of_subnormal_squares_keep_their_codes(param, grad, seed, shift, monkeypatch):
    """8-bit states: the root's block has its scale, a root above zero a code above zero, and the step is the formula's."""
    monkeypatch.setattr(sys.modules[__name__], "EPS", 1e-25)
    a = Lists([5000, 129, 3], param, grad, "e4m3", seed=seed, shift=shift, zero=True, decay=0.0)
    for t in (1, 2, 1000):
        for i, n in enumerate(a.sizes):
            a.g[i].copy_(tiny(n + t, grad)[:n])
        before = a.state()
        a.op.run(LR, t)
        a.check(before, t)
        assert max(float(s.max()) for s in a.vs) < 1e-18


@pytest.mark.parametrize("param,grad,seed", [("f32", "f32", None), ("bf16", "bf16", 3), ("f32", "bf16", 5)])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("n", [5000, 5100000])
def test_large_and_tiny_gradients_side_by_side(param, grad, seed, shift, n, monkeypatch):
    """8-bit states: up to 1e18, so that v passes 2^104, beside 1e-20 in one block, one group and one chunk; large ones come and go."""
    monkeypatch.setattr(sys.modules[__name__], "EPS", 1e-25)
    a = Lists([n, 333], param, grad, "e4m3", seed=seed, shift=shift, zero=True, decay=0.0)
    for t in (1, 2, 3):
        for i, size in enumerate(a.sizes):
            g = tiny(size + t, "f32")[:size].clone()
            block = torch.arange(size, device="cuda") // 128
            some = (block % 5 == t % 3) & (torch.rand(size, generator=gen(t), device="cuda") < 0.1)
            g[some] = (10 ** (12 + 6 * torch.rand(size, generator=gen(t + 9), device="cuda")))[some]
            a.g[i].copy_(g.to(TYPES[grad]))
        before = a.state()
        a.op.run(LR, t)
        a.check(before, t)
        assert max(float(s.max()) for s in a.vs) * 448 > 2.0 ** 52


@pytest.mark.parametrize("param,grad,state,seed", [k for k in KINDS if k[2] == "e4m3"])
@pytest.mark.parametrize("shift", [0, 1])
def test_several_chunks_a_cta(param, grad, state, seed, shift):
    """From some five million elements on, 8-bit states: tensors that end in a CTA's first, second, third and last chunk, at its end and
    just past it, with neighbours on both sides."""
    a = Lists([129, 5000001, 6145, 2049, 4097, 8191, 8192, 8193, 1], param, grad, state, copy=param == "f32", seed=seed, shift=shift)
    before = a.state()
    a.op.run(LR, 3)
    copies, a.copies = a.copies, None
    a.check(before, 3)
    for copy, p in zip(copies or [], a.p):                   # NaN, of a random code of m past 448, is not equal to itself
        assert torch.equal(torch.nan_to_num(copy), torch.nan_to_num(p.to(BF16))) and torch.equal(torch.isnan(copy), torch.isnan(p))


@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_a_blocks_largest_in_every_chunk_of_a_cta(grad):
    """With a noise of 0 it has the formula's code there too."""
    n, seed, f = 6 << 20, 5, np.float32
    g, m, v, ms, vs = alike_blocks(n)
    a = Lists([n], "bf16", grad, "e4m3", seed=seed)
    for name, x in (("g", g), ("m", m), ("v", v)):
        t = getattr(a, name)[0]
        t.copy_(torch.from_numpy(OA.spread(x, n)).cuda().to(t.dtype))
    g = a.g[0][::128].float().cpu().numpy()                  # as rounded to its type
    a.ms[0].copy_(torch.from_numpy(ms))
    a.vs[0].copy_(torch.from_numpy(vs))
    a.op.run(LR, 3)
    noise_m, noise_v, _ = OA.noise(seed, 3, 0, np.arange(n))
    new_m = f(BETAS[0]) * (m * ms) + f(1 - BETAS[0]) * g
    root = v * vs
    new_root = np.sqrt(f(BETAS[1]) * (root * root) + f(1 - BETAS[1]) * g * g)
    chunk = np.arange(n) // 2048 % 4
    for got, new, noise in ((a.m[0], new_m, noise_m), (a.v[0], new_root, noise_v)):
        code = largest_code(np.abs(new))
        for k in range(4):
            assert (noise[chunk == k] == 0).sum() > 8 and len(set(OA.spread(code, n)[(chunk == k) & (noise == 0)])) == 2
        want = np.where(noise == 0, OA.spread(code, n), 0x7E) | np.where(OA.spread(new, n) < 0, 0x80, 0)
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), want)


@pytest.mark.parametrize("shift", [0, 1])
def test_a_tensor_past_32_bits(shift):
    """2^32 + 5 elements of 8-bit states: byte offsets, element numbers and the random bits beyond 32 bits."""
    n = 2 ** 32 + 5
    p, g = (torch.zeros(n + shift, dtype=BF16, device="cuda")[shift:] for _ in range(2))
    m, v = (torch.zeros(n + shift, dtype=torch.uint8, device="cuda").view(E4M3)[shift:] for _ in range(2))
    ms, vs = (torch.zeros(D.AdamW.blocks(n), device="cuda") for _ in range(2))
    spots = [slice(0, 300), slice(2 ** 31 - 128, 2 ** 31 + 256), slice(2 ** 32 - 256, n)]
    for s in spots:
        p[s] = torch.randn(p[s].numel(), generator=gen(1), device="cuda").to(BF16)
        g[s] = torch.randn(p[s].numel(), generator=gen(2), device="cuda").to(BF16)
    before = [(f64(p[s]), f64(g[s])) for s in spots]
    op = D.AdamW([p], [g], [m], [v], m_scales=[ms], v_scales=[vs], betas=BETAS, eps=EPS, weight_decay=0.0, seed=21)
    op.run(LR, 1)
    for s, (p0, g0) in zip(spots, before):
        want, want_m, want_v = OA.step(p0, g0, 0 * p0, 0 * p0, 1, LR, BETAS, EPS, 0.0)
        off = 3 * E * np.abs(p0) + 30 * E * LR
        bits = OA.noise(21, 1, 0, np.arange(s.start, s.stop, dtype=np.uint64))
        lo, hi = (OA.stochastic(want + k * off, bits[2], 8, 2.0 ** -126) for k in (-1, 1))
        assert ((lo <= f64(p[s])) & (f64(p[s]) <= hi)).all()
        blocks = slice(s.start // 128, -(-s.stop // 128))
        x = want_m / OA.spread(f64(ms[blocks]), len(want_m))
        off = np.maximum(9 * E * np.abs(x), 2.0 ** -29)
        lo, hi = (OA.stochastic(np.sign(x) * np.maximum(np.abs(x) + k * off, 0), bits[0], 4, 2.0 ** -6) for k in (-1, 1))
        c = f64(m[s])
        assert ((np.minimum(lo, hi) <= c) & (c <= np.clip(np.maximum(lo, hi), -448, 448))).all()
    untouched = p[300:2 ** 31 - 128]
    assert not untouched.any()


def test_the_binding_refuses_what_does_not_fit():
    a = Lists([64, 65], "f32", "bf16", "e4m3", copy=True)
    ok = dict(params=a.p, grads=a.g, m=a.m, v=a.v, m_scales=a.ms, v_scales=a.vs, copies=a.copies)
    strided = torch.zeros(64, 2, device="cuda")[:, 0]
    for bad in (dict(params=a.p[:1]), dict(params=[a.p[0], a.p[1].double()]), dict(params=[strided, a.p[1]]), dict(params=[a.p[0].half(), a.p[1].half()]),
                dict(grads=[a.g[0], a.g[1].float()]), dict(grads=[a.g[0], a.g[0]]), dict(m=[a.m[0].float(), a.m[1].float()]), dict(m_scales=None),
                dict(v_scales=[a.vs[0], a.ms[1][:0]]), dict(copies=[a.p[0], a.p[1]]), dict(copies=a.copies[:1]), dict(weight_decay=[0.1]),
                dict(params=[a.p[0].cpu(), a.p[1]]), dict(seed=-1), dict(seed=2 ** 32), dict(betas=(1.0, 0.9)), dict(eps=0.0), dict(weight_decay=float("nan"))):
        with pytest.raises(D.DttError):
            D.AdamW(**{**ok, **bad})
    D.AdamW(**{**ok, "copies": [None, a.copies[1]]}).run(LR, 1)
    for bad in (dict(step=0), dict(step=2 ** 32), dict(step=torch.zeros(1, device="cuda")), dict(step=torch.zeros(1, dtype=torch.int32)), dict(lr=float("inf")),
                dict(lr=torch.zeros(2, device="cuda")), dict(grad_scale=torch.zeros(1, dtype=BF16, device="cuda"))):
        with pytest.raises(D.DttError):
            a.op.run(**{**dict(lr=LR, step=1), **bad})
