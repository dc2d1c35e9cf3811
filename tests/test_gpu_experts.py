"""GPU: tokens' rows sorted by expert, and back, against the oracle.  Positions, counts and moved rows are exact.  A
combined row adds at most top_k products in f32: each product and each sum rounds once, within (top_k + 1) e of the terms'
magnitudes (e = 2^-24), before the one rounding to its type; a weight's gradient sums a row, at most ~60 roundings on
any path (a thread's columns, then two trees)."""
import numpy as np
import pytest
import torch

from oracle import experts as OE

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from conftest import ensure_built
    ensure_built()
    import device_triggered_transfers_gb300 as D

E = 2.0 ** -24
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
BITS = {BF16: 8, F32: 24}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def f64(t):
    return None if t is None else t.to(F32).double().cpu().numpy()


def half_spacing(v, kind):
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 1e-37))) - BITS[kind])


def routed(op, ids, max_rows=None, stream=None):
    tokens = ids.shape[0]
    position = torch.full((tokens, op.top_k), -7, dtype=torch.int32, device="cuda")
    offsets, counts = (torch.full((n,), -7, dtype=torch.int32, device="cuda") for n in (op.experts + 1, op.experts))
    op.route(ids, position, offsets, counts, max_rows=max_rows, stream=stream)
    return position, offsets, counts


def choices(tokens, k, of, seed=0, dtype=torch.int64, none=0.02):
    g = gen(seed)
    ids = torch.cat([torch.rand(min(4096, tokens - i), of, generator=g, device="cuda").topk(k, dim=1).indices for i in range(0, tokens, 4096)] or
                    [torch.zeros(0, k, dtype=torch.int64, device="cuda")])
    ids[torch.rand(tokens, generator=g, device="cuda") < none] = -1
    return ids.to(dtype)


ROUTES = [(0, 2, 4, 4, 0, 1), (1, 1, 1, 1, 0, 1), (1, 8, 8, 8, 0, 16), (5, 3, 9, 4, 3, 1), (37, 8, 128, 16, 32, 1), (100, 2, 1024, 1024, 0, 1),
          (255, 8, 60, 60, 0, 128), (257, 8, 60, 15, 45, 8), (1000, 32, 64, 64, 0, 1), (3001, 4, 7, 7, 0, 5), (4096, 8, 256, 256, 0, 128),
          (20011, 6, 160, 40, 120, 16), (40000, 8, 256, 256, 0, 1), (9, 1, 1024, 1000, 24, 7), (70001, 1, 3, 2, 1, 1)]


@pytest.mark.parametrize("tokens,k,of,experts,first,align", ROUTES)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_route(tokens, k, of, experts, first, align, dtype):
    op = D.ExpertRows(experts, k, first=first, align=align)
    ids = choices(tokens, k, of, seed=tokens, dtype=dtype)
    want = OE.route(ids.cpu().numpy(), experts, first, align, op.most_rows(tokens))
    for _ in range(2):
        for got, w in zip(routed(op, ids), want):
            assert np.array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("tokens", [1, 300, 9000])
def test_route_of_one_expert_of_none_and_of_ids_that_are_nobody_s(tokens):
    op = D.ExpertRows(5, 3, first=2, align=4)
    same = torch.full((tokens, 3), 4, dtype=torch.int64, device="cuda")
    none = torch.full((tokens, 3), -1, dtype=torch.int32, device="cuda")
    odd = torch.tensor([2 ** 40 + 3, -2 ** 63, 2 ** 63 - 1, 7, 1, 6, -2 ** 31, 2 ** 32 + 4, 2], device="cuda")
    odd = odd[torch.randint(0, 9, (tokens, 3), generator=gen(1), device="cuda")]
    low = torch.tensor([-2 ** 31, 2 ** 31 - 1, 3, 6], dtype=torch.int32, device="cuda")[torch.randint(0, 4, (tokens, 3), generator=gen(2), device="cuda")]
    for ids in (same, none, odd, low):
        for got, w in zip(routed(op, ids), OE.route(ids.cpu().numpy(), 5, 2, 4, op.most_rows(tokens))):
            assert np.array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("tokens", [50, 5000])
@pytest.mark.parametrize("room", [0, 1, 37, 130, 9000])
def test_route_stops_where_the_rows_end(tokens, room):
    op = D.ExpertRows(12, 4, align=8)
    ids = choices(tokens, 4, 12, seed=5)
    for got, w in zip(routed(op, ids, max_rows=room), OE.route(ids.cpu().numpy(), 12, 0, 8, room)):
        assert np.array_equal(got.cpu().numpy(), w)


def test_route_writes_nothing_beside_its_outputs():
    op = D.ExpertRows(12, 4, first=3, align=8)
    for tokens in (50, 5000):
        ids = choices(tokens, 4, 20, seed=6, dtype=torch.int32)
        wide = [torch.full((n + 8,), -7, dtype=torch.int32, device="cuda") for n in (tokens * 4, 13, 12)]
        op.route(ids, wide[0][4:-4].view(tokens, 4), wide[1][4:-4], wide[2][4:-4])
        for t, w in zip(wide, OE.route(ids.cpu().numpy(), 12, 3, 8, 1 << 30)):
            assert (t[:4] == -7).all() and (t[-4:] == -7).all() and np.array_equal(t[4:-4].cpu().numpy(), w.reshape(-1))


# tokens, cols, k, of, experts, first, align, padding columns of x and of rows
ROWS = [(1, 1, 1, 1, 1, 0, 1, 0, 0), (1, 4096, 8, 128, 16, 0, 1, 0, 0), (37, 4096, 8, 128, 16, 32, 1, 0, 0), (40, 136, 2, 8, 8, 0, 16, 8, 24), (64, 1001, 4, 16, 16, 0, 1, 0, 0),
        (33, 999, 3, 9, 4, 2, 5, 1, 3), (300, 8064, 4, 64, 16, 16, 128, 0, 0), (129, 64, 6, 12, 12, 0, 128, 0, 0), (50, 20000, 2, 4, 2, 1, 1, 0, 0), (9, 30, 32, 40, 40, 0, 7, 2, 2)]


# many tokens of long rows come through shared memory: parts of a tile, whole ones, more choices than a batch has
RING = [(610, 1024, 2, 8, 8, 0, 1, 0, 0), (700, 1032, 9, 16, 16, 0, 8, 8, 8), (650, 8064, 4, 64, 16, 16, 16, 0, 0), (613, 4096, 8, 32, 32, 0, 128, 0, 0),
        (609, 2056, 32, 40, 30, 5, 4, 0, 16), (1301, 2048, 1, 4, 1, 2, 1, 0, 0), (200, 4104, 20, 40, 30, 5, 4, 0, 16), (1300, 2056, 32, 40, 30, 5, 4, 8, 0),
        (500, 6000, 8, 64, 2, 7, 1, 0, 0)]
ROWS += RING


def batch(tokens, cols, k, of, experts, first, align, pad_x, pad_r, dtype, spare=3):
    """A sorted batch, x, and a buffer of sevens with some rows more than are needed."""
    op = D.ExpertRows(experts, k, first=first, align=align)
    ids = choices(tokens, k, of, seed=cols, none=0.1)
    plan = routed(op, ids)
    rows = int(plan[1][-1]) + spare
    x = (torch.randn(tokens, cols + pad_x, generator=gen(tokens), device="cuda") * 3).to(dtype)[:, :cols]
    buffer = torch.full((rows, cols + pad_r), 7.0, device="cuda").to(dtype)
    return op, plan, x, buffer


def host(t):
    """Its bytes: rows are moved as they are."""
    return t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("shape", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32, E4M3])
@pytest.mark.parametrize("scaled", [0, 1, 8, 33])
def test_dispatch(shape, dtype, scaled):
    op, (position, offsets, counts), x, buffer = batch(*shape, dtype)
    cols, before = shape[1], buffer.clone()
    rows = buffer[:, :cols]
    more = {}
    if scaled:
        more = dict(scales=torch.rand(shape[0], scaled, generator=gen(3), device="cuda"), row_scales=torch.full((rows.shape[0], scaled + 1), 7.0, device="cuda")[:, :scaled])
    op.dispatch(x, position, offsets, counts, rows, **more)
    plan = [t.cpu().numpy() for t in (position, offsets, counts)]
    assert np.array_equal(host(rows), OE.dispatch(host(x), *plan, host(before[:, :cols])))
    assert np.array_equal(host(buffer[:, cols:]), host(before[:, cols:]))
    if scaled:
        want = OE.dispatch(f64(more["scales"]), *plan, np.full((rows.shape[0], scaled), 7.0))
        assert np.array_equal(f64(more["row_scales"]), want)


def test_dispatch_looks_at_positions_before_it_uses_them():
    """Positions past the buffer have no row; the buffer's own are written."""
    op = D.ExpertRows(2, 2, align=4)
    offsets, counts = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 4, 8], [1, 1]))
    position = torch.tensor([[0, 8], [2 ** 31 - 1, 4], [-2 ** 31, -1]], dtype=torch.int32, device="cuda")
    x = torch.arange(3 * 64, device="cuda").view(3, 64).to(F32) + 1
    buffer = torch.full((10, 64), 7.0, device="cuda")
    op.dispatch(x, position, offsets, counts, buffer[1:9])
    want = torch.full((10, 64), 7.0, device="cuda")
    want[1:9] = 0
    want[1], want[5] = x[0], x[1]
    assert torch.equal(buffer, want)


def poisoned(rows, used, dtype):
    """NaN in the rows that no pair goes to."""
    rows = rows.clone()
    unused = torch.ones(rows.shape[0], dtype=torch.bool, device="cuda")
    unused[used[used >= 0].long()] = False
    rows[unused] = float("nan")
    return rows


@pytest.mark.parametrize("shape", ROWS)
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(shape, dtype, out_dtype, weighted):
    tokens, cols, k = shape[:3]
    op, (position, _, _), _, buffer = batch(*shape, dtype)
    buffer = poisoned(torch.randn(buffer.shape, generator=gen(8), device="cuda").to(dtype), position, dtype)
    weights = torch.softmax(torch.randn(tokens, k, generator=gen(4), device="cuda"), 1) if weighted else None
    out = torch.full((tokens + 2, cols + shape[7]), 7.0, device="cuda").to(out_dtype)
    op.combine(buffer[:, :cols], position, out[1:-1, :cols], weights=weights)
    want, size = OE.combine(f64(buffer[:, :cols]), position.cpu().numpy(), f64(weights))
    got = f64(out[1:-1, :cols])
    assert (np.abs(got - want) <= half_spacing(want, out_dtype) * (want != 0) + (k + 1) * E * size).all()
    assert (out[0] == 7).all() and (out[-1] == 7).all() and (out[:, cols:] == 7).all()
    assert (got[(position < 0).all(1).cpu().numpy()] == 0).all()


@pytest.mark.parametrize("shape", ROWS)
@pytest.mark.parametrize("dtype,dout_dtype", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_combine_backward(shape, dtype, dout_dtype):
    tokens, cols, k = shape[:3]
    op, (position, offsets, counts), _, buffer = batch(*shape, dtype)
    drows = buffer[:, :cols]
    rows = poisoned(torch.randn(buffer.shape[0], cols + shape[7], generator=gen(8), device="cuda").to(dtype), position, dtype)[:, :cols]
    weights = torch.softmax(torch.randn(tokens, k, generator=gen(4), device="cuda"), 1)
    dout = torch.randn(tokens, cols + shape[8], generator=gen(5), device="cuda").to(dout_dtype)[:, :cols]
    dweights = torch.full((tokens, k), 7.0, device="cuda")
    before = buffer.clone()
    op.combine_backward(dout, rows, position, weights, offsets, counts, drows, dweights)
    plan = [t.cpu().numpy() for t in (position, offsets, counts)]
    want, want_dw, size = OE.combine_backward(f64(dout), f64(rows), plan[0], f64(weights), plan[1], plan[2], f64(before[:, :cols]))
    assert (np.abs(f64(drows) - want) <= (half_spacing(want, dtype) + E * np.abs(want)) * (want != 0)).all()
    assert (np.abs(f64(dweights) - want_dw) <= 60 * E * size).all()
    assert torch.equal(buffer[:, cols:], before[:, cols:])
    # the same bits again; and without the weights' gradient, in place too
    again, dw2 = before[:, :cols], torch.zeros_like(dweights)
    op.combine_backward(dout, rows, position, weights, offsets, counts, again, dw2)
    assert torch.equal(again, drows) and torch.equal(dw2, dweights)
    alone = torch.full_like(before, 7.0)[:, :cols]
    op.combine_backward(dout, alone, position, weights, offsets, counts, alone)
    assert torch.equal(alone, drows)


@pytest.mark.parametrize("shape", ROWS)
def test_dispatch_and_combine_are_each_other_s_gradients(shape):
    """<dispatch(x), r> = <x, combine(r)>: in whole numbers, exactly."""
    tokens, cols = shape[:2]
    op, plan, _, buffer = batch(*shape, F32)
    g = gen(11)
    x = torch.randint(-8, 9, (tokens, cols), generator=g, device="cuda").float()
    r = torch.randint(-8, 9, (buffer.shape[0], cols), generator=g, device="cuda").float()
    rows, dx = torch.zeros_like(r), torch.zeros_like(x)
    op.dispatch(x, *plan, rows)
    op.combine(r, plan[0], dx)
    assert (rows.double() * r.double()).sum() == (x.double() * dx.double()).sum()


def test_gradients_are_differences():
    """Of combine on the GPU, which is linear in each argument: whole numbers, exactly."""
    op = D.ExpertRows(3, 2, align=4)
    plan = routed(op, choices(6, 2, 3, seed=3))
    n, g = int(plan[1][-1]), gen(12)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").float()  # noqa: E731
    rows, weights, dout = ints(n, 16), ints(6, 2), ints(6, 16)
    drows, dweights = torch.zeros_like(rows), torch.zeros_like(weights)
    op.combine_backward(dout, rows, plan[0], weights, *plan[1:], drows, dweights)

    def loss(rows, weights):
        out = torch.zeros(6, 16, device="cuda")
        op.combine(rows, plan[0], out, weights=weights)
        return float((out * dout).sum())

    base = loss(rows, weights)
    for t, grad in ((rows, drows), (weights, dweights)):
        for i in np.ndindex(*t.shape):
            t[i] += 1
            assert loss(rows, weights) - base == float(grad[i])
            t[i] -= 1


def test_infinities_and_nan_stay_in_their_token():
    op = D.ExpertRows(4, 2)
    plan = routed(op, choices(20, 2, 4, seed=2, none=0))
    rows = torch.randn(40, 64, generator=gen(1), device="cuda")
    rows[int(plan[0][3, 1]), 5] = float("nan")
    rows[int(plan[0][4, 0]), 6] = float("inf")
    weights = torch.ones(20, 2, device="cuda")
    weights[7, 0] = 0.0                         # 0 x inf is NaN: a weight of zero is still a weight
    rows[int(plan[0][7, 0]), 9] = float("inf")
    out = torch.zeros(20, 64, device="cuda")
    op.combine(rows, plan[0], out, weights=weights)
    assert torch.isnan(out[3, 5]) and torch.isinf(out[4, 6]) and torch.isnan(out[7, 9])
    assert torch.isfinite(out).sum() == 20 * 64 - 3


def test_tokens_of_no_batch():
    op = D.ExpertRows(4, 2, align=8)
    ids = torch.zeros(0, 2, dtype=torch.int64, device="cuda")
    plan = routed(op, ids)
    assert not plan[1].any() and not plan[2].any()
    rows = torch.full((5, 64), 7.0, device="cuda")
    x = torch.zeros(0, 64, device="cuda")
    op.dispatch(x, *plan, rows)
    op.combine(rows, plan[0], x)
    op.combine_backward(x, rows, plan[0], torch.zeros(0, 2, device="cuda"), *plan[1:], rows.clone(), torch.zeros(0, 2, device="cuda"))
    torch.cuda.synchronize()
    assert (rows == 7).all()



def test_no_tokens_and_no_rows_with_scales():
    """Rows that fill an expert up are zeros, their scales too; nothing else is written."""
    op = D.ExpertRows(2, 2, align=4)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x, scales = torch.zeros(0, 64, device="cuda").to(E4M3), torch.zeros(0, 3, device="cuda")
    rows, row_scales = torch.full((10, 64), 7.0, device="cuda").to(E4M3), torch.full((10, 3), 7.0, device="cuda")
    op.dispatch(x, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), ints(0, 4, 8), ints(1, 4), rows, scales=scales, row_scales=row_scales)
    for t in (rows.float(), row_scales):
        assert not t[1:4].any() and (t[0] == 7).all() and (t[4:] == 7).all()
    plan = routed(op, choices(6, 2, 2), max_rows=0)
    op.dispatch(torch.zeros(6, 64, device="cuda").to(E4M3), *plan, rows[:0], scales=torch.zeros(6, 3, device="cuda"), row_scales=row_scales[:0])
    torch.cuda.synchronize()
    assert (row_scales[0] == 7).all()
    with pytest.raises(D.DttError):
        op.dispatch(x, plan[0][:0], *plan[1:], rows, scales=scales)


def test_a_captured_pass_replays_with_other_choices():
    """The whole way there and back in a graph whose first call allocates the workspace; then other ids in place."""
    tokens, cols, k = 300, 512, 4
    op = D.ExpertRows(16, k, first=8, align=16)
    ids = choices(tokens, k, 32, seed=1)
    x = torch.randn(tokens, cols, generator=gen(1), device="cuda")
    weights = torch.rand(tokens, k, generator=gen(2), device="cuda")
    position = torch.zeros(tokens, k, dtype=torch.int32, device="cuda")
    offsets, counts = torch.zeros(17, dtype=torch.int32, device="cuda"), torch.zeros(16, dtype=torch.int32, device="cuda")
    rows, out = torch.zeros(op.most_rows(tokens), cols, device="cuda"), torch.zeros(tokens, cols, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        op.route(ids, position, offsets, counts, stream=stream)
        op.dispatch(x, position, offsets, counts, rows, stream=stream)
        op.combine(rows, position, out, weights=weights, stream=stream)
    for seed in (1, 2, 3):
        ids.copy_(choices(tokens, k, 32, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        want = OE.route(ids.cpu().numpy(), 16, 8, 16, op.most_rows(tokens))
        for got, w in zip((position, offsets, counts), want):
            assert np.array_equal(got.cpu().numpy(), w)
        total = (weights * (position >= 0)).sum(1, keepdim=True)
        assert ((out - x * total).abs() <= 6 * E * (x * total).abs() + 1e-30).all()


def test_calls_that_read_what_the_call_before_wrote_need_no_wait_between_them():
    tokens, cols, k = 3000, 1024, 4
    op = D.ExpertRows(32, k, align=16)
    x = torch.randn(tokens, cols, generator=gen(1), device="cuda").to(BF16)
    weights = torch.rand(tokens, k, generator=gen(2), device="cuda")
    ids = choices(tokens, k, 32)

    def chain(wait):
        y = x.clone()
        results = []
        for _ in range(6):
            plan = routed(op, ids)
            if wait:
                torch.cuda.synchronize()
            rows = torch.zeros(op.most_rows(tokens), cols, dtype=BF16, device="cuda")
            op.dispatch(y, *plan, rows)
            if wait:
                torch.cuda.synchronize()
            out, drows, dw = torch.zeros_like(y), torch.zeros_like(rows), torch.zeros_like(weights)
            op.combine(rows, plan[0], out, weights=weights)
            if wait:
                torch.cuda.synchronize()
            op.combine_backward(out, rows, plan[0], weights, *plan[1:], drows, dw)
            if wait:
                torch.cuda.synchronize()
            op.combine(drows, plan[0], y)
            results += [out, dw, y.clone()]
            ids.copy_((ids + 1) % 32)
        ids.copy_((ids - 6) % 32)
        torch.cuda.synchronize()
        return results

    ids.clamp_(min=0)
    for a, b in zip(chain(True), chain(False)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("late", ["true", "t == 37", "t % 7 == 3 && ring.at == 1"])
def test_a_wait_that_is_given_up_changes_nothing(late, tmp_path):
    """Threads that give an item up, all of them or some, take it and the later ones from global memory: the same bits."""
    from test_gpu_ops_edges import library_with
    L = library_with("experts.cu", [f"-DDTT_EXPERTS_LATE=({late})"], str(tmp_path))
    for shape in RING:
        tokens, cols, k = shape[:3]
        for dtype, other_dtype in ((BF16, BF16), (F32, BF16)):
            op, plan, _, buffer = batch(*shape, dtype)
            rows = torch.randn(buffer.shape[0], cols, generator=gen(1), device="cuda").to(dtype)
            dout = torch.randn(tokens, cols, generator=gen(2), device="cuda").to(other_dtype)
            weights = torch.rand(tokens, k, generator=gen(3), device="cuda")
            got = []
            for other in (False, True):
                if other:
                    op._combine, op._combine_backward = L.dtt_experts_combine, L.dtt_experts_combine_backward
                out, drows, dweights = torch.zeros_like(dout), torch.full_like(rows, 7.0), torch.zeros_like(weights)
                op.combine(rows, plan[0], out, weights=weights)
                op.combine_backward(dout, rows, plan[0], weights, *plan[1:], drows, dweights)
                got.append((out, drows, dweights))
            for a, b in zip(*got):
                assert torch.equal(a, b)



@pytest.mark.parametrize("late", ["t / 32 == 3", "t / 32 != 5", "t / 32 == 3 && ring.at == 2", "t / 64 == blockIdx.x % 4 && ring.at == 7"])
def test_warps_that_give_up_run_ahead_of_the_others(late, tmp_path):
    """All lanes of a warp give an item up, and from there on wait for nothing while other warps still read from the slots: no slot is
    filled again under them, and the results keep their bits.  Waits that nothing ends are cut short."""
    from test_gpu_ops_edges import library_with
    L = library_with("experts.cu", [f"-DDTT_EXPERTS_LATE=({late})", "-DDTT_EXPERTS_WAIT_LIMIT=4096u"], str(tmp_path))
    for shape in [(9000, 4096, 8, 32, 32, 0, 1, 0, 0), *RING]:
        tokens, cols, k = shape[:3]
        for dtype, other_dtype in ((BF16, BF16), (F32, BF16)):
            op, plan, _, buffer = batch(*shape, dtype)
            rows = torch.randn(buffer.shape[0], cols, generator=gen(1), device="cuda").to(dtype)
            dout = torch.randn(tokens, cols, generator=gen(2), device="cuda").to(other_dtype)
            weights = torch.rand(tokens, k, generator=gen(3), device="cuda")
            got = []
            for other in (False, True):
                if other:
                    op._combine, op._combine_backward = L.dtt_experts_combine, L.dtt_experts_combine_backward
                out, drows, dweights, alone = torch.zeros_like(dout), torch.full_like(rows, 7.0), torch.zeros_like(weights), torch.full_like(rows, 7.0)
                op.combine(rows, plan[0], out, weights=weights)
                op.combine_backward(dout, rows, plan[0], weights, *plan[1:], drows, dweights)
                op.combine_backward(dout, None, plan[0], weights, *plan[1:], alone)          # no barrier among the warps
                got.append((out, drows, dweights, alone))
            for a, b in zip(*got):
                assert torch.equal(a, b)


@pytest.mark.parametrize("late", ["true", "oldest.at == 3", "lane == 0 && oldest.at == 9", "lane % 2 && blockIdx.x % 3 == 1"])
def test_a_fetching_warp_that_gives_up_leaves_no_copy_behind(late, tmp_path):
    """It starts no more items, waits for those under way, the one it gave up among them, and the other warps take what is left from
    global memory: the same bits, launch after launch."""
    from test_gpu_ops_edges import library_with
    L = library_with("experts.cu", [f"-DDTT_EXPERTS_FETCH_LATE=({late})", "-DDTT_EXPERTS_WAIT_LIMIT=4096u"], str(tmp_path))
    for shape in [(9000, 4096, 8, 32, 32, 0, 1, 0, 0), *RING]:
        tokens, cols, k = shape[:3]
        op, plan, _, buffer = batch(*shape, BF16)
        rows = torch.randn(buffer.shape[0], cols, generator=gen(1), device="cuda").to(BF16)
        dout = torch.randn(tokens, cols, generator=gen(2), device="cuda").to(BF16)
        weights = torch.rand(tokens, k, generator=gen(3), device="cuda")
        got = []
        for other in (False, True, True):
            if other:
                op._combine, op._combine_backward = L.dtt_experts_combine, L.dtt_experts_combine_backward
            out, drows, dweights = torch.zeros_like(dout), torch.full_like(rows, 7.0), torch.zeros_like(weights)
            op.combine(rows, plan[0], out, weights=weights)
            op.combine_backward(dout, rows, plan[0], weights, *plan[1:], drows, dweights)
            got.append((out, drows, dweights))
        for a, *others in zip(*got):
            assert all(torch.equal(a, b) for b in others)


def test_rows_past_four_gigabytes():
    tokens, cols, k = 20011, 32768, 4              # 80044 rows of 64 KiB: 5.2 GB
    op = D.ExpertRows(8, k)
    plan = routed(op, choices(tokens, k, 8, none=0))
    x = torch.randint(-4, 5, (tokens, cols), generator=gen(1), device="cuda", dtype=torch.int8).to(BF16)
    rows = torch.zeros(op.most_rows(tokens), cols, dtype=BF16, device="cuda")
    op.dispatch(x, *plan, rows)
    out = torch.zeros_like(x)
    op.combine(rows, plan[0], out)
    assert torch.equal(out, x * 4)
    dw = torch.zeros(tokens, k, device="cuda")
    op.combine_backward(x, rows, plan[0], torch.full((tokens, k), 2.0, device="cuda"), *plan[1:], rows.clone(), dw)
    want = torch.cat([p.float().square().sum(1) for p in x.split(1000)])
    assert torch.equal(dw, want[:, None].expand(-1, k))          # sums of whole numbers below 2^24


def test_the_binding_refuses_what_does_not_fit():
    op = D.ExpertRows(4, 2, align=8)
    ids = choices(10, 2, 4)
    position, offsets, counts = routed(op, ids)
    x, rows = torch.zeros(10, 64, device="cuda"), torch.zeros(60, 64, device="cuda")
    w = torch.zeros(10, 2, device="cuda")
    ok = dict(ids=ids, position=position, offsets=offsets, counts=counts)
    for bad in (dict(ids=ids[:, :1]), dict(ids=ids.float()), dict(ids=ids.cpu()), dict(position=position[:9]), dict(offsets=offsets[:4]),
                dict(counts=counts.long()), dict(max_rows=-1), dict(max_rows=2 ** 31)):
        with pytest.raises(D.DttError):
            op.route(**{**ok, **bad})
    ok = dict(x=x, position=position, offsets=offsets, counts=counts, rows=rows)
    for bad in (dict(x=x[:9]), dict(rows=rows[:, :32]), dict(rows=rows.half()), dict(x=x.t().contiguous().t()), dict(scales=w), dict(row_scales=w),
                dict(scales=w, row_scales=torch.zeros(59, 2, device="cuda")), dict(position=position.long()), dict(rows=rows.cpu())):
        with pytest.raises(D.DttError):
            op.dispatch(**{**ok, **bad})
    for bad in (dict(weights=w.double()), dict(weights=w[:9]), dict(rows=rows.half()), dict(out=x[:9]), dict(out=x.cpu())):
        with pytest.raises(D.DttError):
            op.combine(**{**dict(rows=rows, position=position, out=x), **bad})
    ok = dict(dout=x, rows=rows, position=position, weights=w, offsets=offsets, counts=counts, drows=rows.clone(), dweights=w.clone())
    for bad in (dict(rows=rows[:59]), dict(rows=None), dict(weights=None), dict(dweights=w[:9]), dict(drows=rows.to(BF16)), dict(dout=x[:9])):
        with pytest.raises(D.DttError):
            op.combine_backward(**{**ok, **bad})
