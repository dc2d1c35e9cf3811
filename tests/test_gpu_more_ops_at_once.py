"""GPU: layer norm, expert rows and AdamW beside one another: passes of two objects at once on two streams, called and replayed, give
the bits that they give alone; and an expert that a token chooses more than once."""
import numpy as np
import pytest
import torch

from oracle import experts as OE

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from conftest import ensure_built
    ensure_built()
    import device_triggered_transfers_gb300 as D

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Pass:
    """Norm, sort, rows there and back, their gradients, and AdamW on what is left, with buffers and objects of its own."""

    def __init__(self, seed, tokens, cols, k=4, experts=12, align=8):
        g = gen(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.norm, self.sort = D.LayerNorm(cols), D.ExpertRows(experts, k, first=2, align=align)
        self.x, self.h, self.y, self.dy, self.dx = (rand(tokens, cols).to(BF16) for _ in range(5))
        self.weight, self.bias = rand(cols).to(BF16), rand(cols).to(BF16)
        self.mean, self.rstd = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        self.dweight, self.dbias = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        self.ids = torch.randint(0, experts + 4, (tokens, k), generator=g, device="cuda", dtype=torch.int32)
        self.weights, self.dweights = torch.rand(tokens, k, generator=g, device="cuda"), torch.empty(tokens, k, device="cuda")
        ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.plan = ints(tokens, k), ints(experts + 1), ints(experts)
        self.rows, self.drows = (torch.zeros(self.sort.most_rows(tokens), cols, dtype=BF16, device="cuda") for _ in range(2))
        self.out = torch.empty(tokens, cols, dtype=BF16, device="cuda")
        n = tokens * cols
        self.p = rand(n).to(BF16)
        self.m, self.v = (torch.zeros(n, device="cuda").to(E4M3) for _ in range(2))
        self.ms, self.vs = (torch.zeros(D.AdamW.blocks(n), device="cuda") for _ in range(2))
        self.step = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.adamw = D.AdamW([self.p], [self.dx.view(-1)], [self.m], [self.v], m_scales=[self.ms], v_scales=[self.vs], seed=seed)

    def run(self, stream):
        self.norm.forward(self.x, self.weight, self.bias, self.y, residual=self.h, residual_out=self.h, mean=self.mean, rstd=self.rstd, stream=stream)
        self.sort.route(self.ids, *self.plan, stream=stream)
        self.sort.dispatch(self.y, *self.plan, self.rows, stream=stream)
        self.sort.combine(self.rows, self.plan[0], self.out, weights=self.weights, stream=stream)
        self.sort.combine_backward(self.out, self.rows, self.plan[0], self.weights, *self.plan[1:], self.drows, dweights=self.dweights, stream=stream)
        self.sort.combine(self.drows, self.plan[0], self.dy, stream=stream)
        self.norm.backward(self.dy, self.h, self.weight, self.mean, self.rstd, self.dx, dweight=self.dweight, dbias=self.dbias, stream=stream)
        self.adamw.run(1e-3, self.step, stream=stream)

    def results(self):
        return [t.clone() for t in (self.h, self.y, *self.plan, self.rows, self.out, self.drows, self.dweights, self.dy, self.dx, self.dweight, self.dbias, self.p,
                                    self.m.view(torch.uint8), self.v.view(torch.uint8), self.ms, self.vs, self.step)]


SIZES = [((3, 700, 1024), (4, 900, 4096)), ((5, 61, 999), (6, 1300, 2056)), ((7, 2000, 128), (8, 5, 8064))]


def alone(sizes, times):
    p = Pass(*sizes)
    for _ in range(times):
        p.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    return p.results()


def same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("sizes", SIZES)
def test_two_at_once_on_two_streams(sizes):
    want = [alone(s, 3) for s in sizes]
    passes, streams = [Pass(*s) for s in sizes], [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s in zip(passes, streams):
            p.run(s)
    torch.cuda.synchronize()
    for p, w in zip(passes, want):
        same(p.results(), w)


@pytest.mark.parametrize("sizes", SIZES)
def test_two_graphs_replayed_at_once(sizes):
    """Captured by the first call of each object, workspaces included."""
    want = [alone(s, 3) for s in sizes]
    passes, streams, graphs = [Pass(*s) for s in sizes], [torch.cuda.Stream() for _ in sizes], [torch.cuda.CUDAGraph() for _ in sizes]
    torch.cuda.synchronize()
    for p, s, g in zip(passes, streams, graphs):
        with torch.cuda.graph(g, stream=s):
            p.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for p, w in zip(passes, want):
        same(p.results(), w)


@pytest.mark.parametrize("tokens,cols,k", [(50, 100, 6), (700, 4096, 8), (1300, 2056, 3)])
def test_an_expert_chosen_more_than_once_by_a_token(tokens, cols, k):
    """Each choice has a row of its own.  Whole numbers: exactly."""
    g, op = gen(9), D.ExpertRows(3, k, first=1, align=4)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float()  # noqa: E731
    ids = torch.randint(0, 5, (tokens, k), generator=g, device="cuda")
    position, offsets, counts = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((tokens, k), (4,), (3,)))
    op.route(ids, position, offsets, counts)
    plan = OE.route(ids.cpu().numpy(), 3, 1, 4, 1 << 30)
    for got, want in zip((position, offsets, counts), plan):
        assert np.array_equal(got.cpu().numpy(), want)
    n = int(plan[1][-1])
    x, weights, dout = ints(tokens, cols), ints(tokens, k), ints(tokens, cols)
    rows, drows, out, dweights = (torch.zeros(n, cols, device="cuda"), torch.zeros(n, cols, device="cuda"), torch.zeros(tokens, cols, device="cuda"),
                                  torch.zeros(tokens, k, device="cuda"))
    op.dispatch(x, position, offsets, counts, rows)
    op.combine(rows, position, out, weights=weights)
    op.combine_backward(dout, rows, position, weights, offsets, counts, drows, dweights)
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    assert np.array_equal(host(rows), OE.dispatch(host(x), *plan, np.zeros((n, cols))))
    assert np.array_equal(host(out), OE.combine(host(rows), plan[0], host(weights))[0])
    want, want_dw, _ = OE.combine_backward(host(dout), host(rows), plan[0], host(weights), plan[1], plan[2], np.zeros((n, cols)))
    assert np.array_equal(host(drows), want) and np.array_equal(host(dweights), want_dw)
