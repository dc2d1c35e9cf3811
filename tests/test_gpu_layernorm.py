"""GPU: the layer norm and its backward pass against the oracle's 64 bits.

Tolerances, from the arithmetic: e = 2^-24 is half an f32 ulp, and a row's sum goes through at most ~40 roundings on any
path (a thread's columns, then two butterfly trees).  The mean is therefore within 41 e of the row's mean magnitude
A; each h - mean is off by that and half an ulp of its own, and their mean of squares, to which the mean's error
adds its square alone, is within 45 e + (41 e A / std)^2: half of that and a 2-ulp reciprocal square root reach rstd.
y = (h - mean) rstd weight + bias: the mean's error times rstd weight, 30 e of the product, 2 e of the sum.  h itself is
one rounded addition.  Roundings to bf16 and e4m3 as test_gpu_ops.py has them."""
import numpy as np
import pytest
import torch

from oracle import norm as ON

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from conftest import ensure_built
    ensure_built()
    import device_triggered_transfers_gb300 as D

E = 2.0 ** -24
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BITS = {"bf16": 8, "f32": 24}                # significant bits


def f64(t):
    return None if t is None else t.to(torch.float32).double().cpu().numpy()


def half_spacing(v, kind):
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 1e-37))) - BITS[kind])


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def slab(rows, cols, kind, pad, g, spread=1.0, shift=0.0):
    return (torch.randn(rows, cols + pad, generator=g, device="cuda") * spread + shift).to(TYPES[kind])[:, :cols]


def case(rows, cols, x="bf16", residual="bf16", weight="bf16", bias=True, y="bf16", group=0, pad=0, shift=1.0, seed=0):
    g = gen(seed)
    op = D.LayerNorm(cols, x=x, residual=residual or x, weight=weight or "bf16", y=y, group=group, eps=EPS)
    a = dict(x=slab(rows, cols, x, pad, g, 0.5), weight=slab(1, cols, weight, 0, g, 0.3, 1.0)[0] if weight else None,
             bias=slab(1, cols, weight or "bf16", 0, g, 0.2)[0] if bias else None)
    more = dict(residual=slab(rows, cols, residual, pad, g, 3.0, shift) if residual else None)
    out = dict(y=torch.zeros(rows, cols + pad, device="cuda").to(TYPES[y])[:, :cols], residual_out=slab(rows, cols, residual or x, pad, g),
               scales=torch.full((rows, op.scale_cols), -1.0, device="cuda") if y == "e4m3" else None,
               mean=torch.full((rows,), -1.0, device="cuda"), rstd=torch.full((rows,), -1.0, device="cuda"))
    return op, a, more, out


def forward(op, a, more, out):
    op.forward(a["x"], a["weight"], a["bias"], **more, **out)


def check(a, more, out, y, group):
    h, mean, rstd, want = ON.layer_forward(f64(a["x"]), f64(more["residual"]), f64(a["weight"]), f64(a["bias"]), EPS)
    kind = "bf16" if out["residual_out"].dtype == torch.bfloat16 else "f32"
    assert (np.abs(f64(out["residual_out"]) - h) <= half_spacing(h, kind) + 2 * E * np.abs(h)).all()
    size = np.abs(h).mean(axis=1)
    off = 41 * E * size
    assert (np.abs(f64(out["mean"]) - mean) <= off + E * np.abs(mean)).all()
    assert (np.abs(f64(out["rstd"]) / rstd - 1) <= 30 * E + (off * rstd) ** 2).all()
    w = np.ones(h.shape[1]) if a["weight"] is None else np.abs(f64(a["weight"]))
    b = np.zeros(h.shape[1]) if a["bias"] is None else np.abs(f64(a["bias"]))
    n = np.abs((h - mean[:, None]) * rstd[:, None]) * w
    slack = (off[:, None] + 2 * E * np.abs(h)) * rstd[:, None] * w + (30 * E + (off * rstd)[:, None] ** 2) * n + 2 * E * (n + b)
    got = f64(out["y"])
    if y != "e4m3":
        assert (np.abs(got - want) <= half_spacing(want, y) + slack).all()
        return
    s = ON.scales(want, group)
    assert (np.abs(f64(out["scales"]) - s) <= 3e-6 * s + slack.max(axis=1, keepdims=True) / 448).all()
    s = ON.spread(f64(out["scales"]), group, want.shape[1])
    assert (np.abs(got) <= 448).all()
    assert (np.abs(got * s - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s) * 1.001 + slack).all()


# every form: parts of a warp, the ring's three, chunks, rows read again, elements, the ring of elements
SHAPES = [
    (1, 1, {}), (3, 5, {}), (2, 8, dict(y="f32")), (5, 31, dict(pad=1)), (9, 256, {}), (7, 257, {}), (33, 16, dict(y="e4m3", group=128)),
    (1000, 24, dict(y="e4m3", group=32)), (10001, 128, dict(y="e4m3")), (513, 200, dict(weight=None, bias=False)), (40, 136, dict(residual=None, weight="f32", y="f32")),
    (1, 4096, dict(y="e4m3")), (37, 8064, dict(y="e4m3", group=128)), (300, 64, dict(y="e4m3", group=32)), (5, 200, dict(y="e4m3", group=64)),
    (3, 4097, dict(y="e4m3", group=128, pad=7)), (64, 4096, dict(x="f32", residual="f32", weight="f32", y="f32")), (64, 1000, dict(residual="f32", pad=8)),
    (11, 2048, dict(x="f32", residual="bf16", y="e4m3")), (130, 5001, dict(residual="f32", pad=7)), (20, 4096, dict(residual=None)),
    (20, 4096, dict(weight=None)), (20, 4096, dict(bias=False)), (4, 16384, {}), (3, 32768, dict(y="e4m3")), (2, 32769, dict(y="e4m3")),
    (2, 70000, dict(y="e4m3", group=128)), (2, 40000, dict(residual="f32", y="f32", pad=3)), (700, 4096, dict(y="e4m3")), (700, 4096, {}),
    (1000, 8064, dict(y="e4m3", group=128)), (999, 1024, dict(x="f32", residual="f32", y="f32")), (2500, 512, dict(y="e4m3", group=64)),
    (611, 12288, {}), (1217, 1001, dict(y="e4m3", group=64)), (1300, 264, dict(y="f32")), (1300, 4000, dict(pad=1)),
    (2, 65536, dict(x="f32", residual="f32", y="f32")), (100, 2056, dict(y="e4m3", group=128, weight="f32")),
]


@pytest.mark.parametrize("rows,cols,over", SHAPES)
def test_forward(rows, cols, over):
    op, a, more, out = case(rows, cols, **over)
    forward(op, a, more, out)
    again = {k: None if v is None else torch.zeros_like(v) for k, v in out.items()}
    forward(op, a, more, again)
    check(a, more, out, over.get("y", "bf16"), over.get("group", 0))
    for k, v in out.items():
        assert v is None or torch.equal(v.contiguous().view(torch.uint8), again[k].contiguous().view(torch.uint8)), k


@pytest.mark.parametrize("rows,cols,pad", [(40, 128, 0), (700, 4096, 0), (40, 8192, 0), (3, 40000, 0), (40, 1001, 1), (1300, 1001, 1)])
def test_a_mean_far_larger_than_the_rest(rows, cols, pad):
    """A mean 3000 times the spread: a variance from squares of h would have one or two digits left."""
    op, a, more, out = case(rows, cols, x="f32", residual="f32", weight="f32", y="f32", pad=pad, shift=9000.0)
    forward(op, a, more, out)
    check(a, more, out, "f32", 0)


@pytest.mark.parametrize("rows,cols,pad", [(9, 128, 0), (700, 1024, 0), (9, 16384, 0), (9, 40000, 0), (9, 1001, 1), (1300, 1001, 1)])
def test_constant_rows_give_the_bias_and_nan_and_infinity_stay_in_their_row(rows, cols, pad):
    op, a, more, out = case(rows, cols, y="f32", pad=pad)
    more["residual"][0] = 2.5
    a["x"][0] = 1.0
    a["x"][1, cols // 2] = float("nan")
    a["x"][2, cols - 1] = float("inf")
    forward(op, a, more, out)
    assert torch.equal(out["y"][0], a["bias"].float()) and out["mean"][0] == 3.5
    for r in (1, 2):
        assert torch.isnan(out["y"][r]).all() and torch.isnan(out["rstd"][r])
    assert torch.isnan(out["mean"][1]) and torch.isinf(out["mean"][2])
    keep = slice(3, None)
    check({"x": a["x"][keep], "weight": a["weight"], "bias": a["bias"]}, {"residual": more["residual"][keep]},
          {k: None if v is None else v[keep] for k, v in out.items()}, "f32", 0)



@pytest.mark.parametrize("rows,cols,pad", [(9, 128, 0), (700, 1024, 0), (700, 8192, 0), (9, 16384, 0), (9, 40000, 0), (9, 1001, 1), (1300, 1001, 1), (2, 40003, 1)])
def test_rows_whose_squares_or_sum_leave_f32(rows, cols, pad):
    """Squares about a mean of 0 that overflow: rstd 0, and so the bias; a sum that does: an infinite mean, and NaN."""
    op, a, more, out = case(rows, cols, x="f32", residual="f32", weight="f32", y="f32", pad=pad)
    more["residual"][:2] = 0
    a["x"][0] = 1e30 * (1 - 2 * (torch.arange(cols, device="cuda") % 2))
    a["x"][1] = 3e38
    forward(op, a, more, out)
    assert out["rstd"][0] == 0 and torch.equal(out["y"][0], a["bias"]) and out["mean"][0].abs() <= 1e30 / cols * 1.001
    assert torch.isinf(out["mean"][1]) and torch.isnan(out["y"][1]).all()
    keep = slice(2, None)
    if rows > 2:
        check({"x": a["x"][keep], "weight": a["weight"], "bias": a["bias"]}, {"residual": more["residual"][keep]},
              {k: None if v is None else v[keep] for k, v in out.items()}, "f32", 0)


@pytest.mark.parametrize("rows,cols", [(5, 128), (5, 4096), (700, 4096), (5, 40000), (3, 1001), (1300, 1001)])
def test_in_place_and_without_the_optional_outputs(rows, cols):
    op, a, more, out = case(rows, cols, y="e4m3")
    forward(op, a, more, out)
    r, y, scales = more["residual"].clone(), torch.zeros_like(out["y"]), torch.zeros_like(out["scales"])
    op.forward(a["x"], a["weight"], a["bias"], y, residual=r, residual_out=r, scales=scales)
    assert torch.equal(r, out["residual_out"]) and torch.equal(scales, out["scales"])
    assert torch.equal(y.view(torch.uint8), out["y"].view(torch.uint8))


@pytest.mark.parametrize("rows,cols,pad,group", [(37, 104, 16, 32), (700, 1000, 24, 128), (33, 1001, 7, 128), (1300, 1001, 7, 64), (2, 40000, 8, 0)])
def test_outputs_are_written_exactly(rows, cols, pad, group):
    op, a, more, out = case(rows, cols, y="e4m3", group=group)
    wide = {k: torch.full((rows + 2, cols + pad), 7.0, device="cuda").to(t) for k, t in (("y", TYPES["e4m3"]), ("r", TYPES["bf16"]))}
    flat = {k: torch.full((n + 8,), 7.0, device="cuda") for k, n in (("scales", rows * op.scale_cols), ("mean", rows), ("rstd", rows))}
    out.update(y=wide["y"][1:-1, :cols], residual_out=wide["r"][1:-1, :cols], scales=flat["scales"][4:-4].view(rows, -1), mean=flat["mean"][4:-4],
               rstd=flat["rstd"][4:-4])
    forward(op, a, more, out)
    check(a, more, out, "e4m3", group)
    for t in wide.values():
        assert (t[:, cols:].float() == 7).all() and (t[0].float() == 7).all() and (t[-1].float() == 7).all()
    for t in flat.values():
        assert (t[:4] == 7).all() and (t[-4:] == 7).all()


# ---- backward -------------------------------------------------------------------------------------
def grad_case(rows, cols, x="bf16", residual="bf16", weight="bf16", pad=0, dres=True, shift=1.0, seed=1):
    g = gen(seed)
    op = D.LayerNorm(cols, x=x, residual=residual, weight=weight or "bf16", eps=EPS)
    h = slab(rows, cols, residual, pad, g, 3.0, shift)
    a = dict(dy=slab(rows, cols, x, pad, g, 0.1), h=h, weight=slab(1, cols, weight, 0, g, 0.3, 1.0)[0] if weight else None,
             mean=h.float().mean(-1), rstd=(h.float().var(-1, unbiased=False) + EPS).rsqrt())
    return op, a, slab(rows, cols, residual, pad, g, 0.1) if dres else None, slab(rows, cols, residual, pad, g)


def check_backward(a, dres, dx, dw, db, residual):
    dy, h, w, mu, s = (f64(a[k]) for k in ("dy", "h", "weight", "mean", "rstd"))
    want, want_dw, want_db = ON.layer_backward(dy, h, w, mu, s, f64(dres))
    # f32 errors are relative to the terms: the row's means go through ~45 roundings, the rest a few
    n, g = (h - mu[:, None]) * s[:, None], dy if w is None else dy * w
    terms = s[:, None] * (np.abs(g) + np.abs(g).mean(axis=1, keepdims=True) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
    slack = 50 * E * (terms + (0 if dres is None else np.abs(f64(dres))))
    assert (np.abs(f64(dx) - want) <= half_spacing(want, residual) + slack).all()
    # each partial row adds its rows one after the other, then the partial rows are added
    depth = len(dy) / min(len(dy), 100) + 400
    if dw is not None:
        assert (np.abs(f64(dw) - want_dw) <= depth * E * np.abs(dy * n).sum(axis=0)).all()
    if db is not None:
        assert (np.abs(f64(db) - want_db) <= depth * E * np.abs(dy).sum(axis=0)).all()


GRADS = [(1, 1, {}), (3, 5, dict(x="f32", residual="f32")), (2, 64, {}), (17, 256, {}), (16, 4096, {}), (700, 4096, {}), (2000, 1024, dict(dres=False)),
         (1021, 5001, dict(x="f32", residual="f32", weight="f32", pad=3)), (50, 8064, dict(residual="f32")), (300, 8064, {}), (9, 12288, {}),
         (5, 16384, {}), (700, 16385, {}), (3, 20000, dict(pad=1)), (611, 4104, dict(weight="f32")), (640, 8192, dict(residual="f32", weight="f32")),
         (33, 16, {}), (10001, 128, {}), (5003, 104, dict(residual="f32")), (257, 40, dict(pad=8)), (96, 1000, {}), (97, 1000, {}), (5, 40000, {}),
         (200, 40000, dict(x="f32", residual="f32")), (63, 5001, dict(pad=3)), (300, 101, dict(pad=1)), (9000, 31, dict(pad=1)), (1, 64, {}), (120, 4000, dict(pad=1)),
         (200, 1024, dict(shift=500.0, residual="f32"))]


@pytest.mark.parametrize("rows,cols,over", GRADS)
def test_backward(rows, cols, over):
    op, a, dres, dx = grad_case(rows, cols, **over)
    wide = [torch.full((cols + 9,), 7.0, device="cuda") for _ in range(2)]
    dw, db = (t[4:4 + cols] for t in wide)
    op.backward(**a, dx=dx, dweight=dw, dbias=db, dres=dres)
    check_backward(a, dres, dx, dw, db, over.get("residual", "bf16"))
    assert all((t[:4] == 7).all() and (t[4 + cols:] == 7).all() for t in wide)
    # the same bits again, each gradient alone, neither, and in place
    one, two, again = torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda"), torch.zeros_like(dx)
    op.backward(**a, dx=again, dweight=one, dres=dres)
    assert torch.equal(again, dx) and torch.equal(one, dw)
    op.backward(**a, dx=again, dbias=two, dres=dres)
    assert torch.equal(again, dx) and torch.equal(two, db)
    if dres is not None:
        keep = dres.clone()
        op.backward(**a, dx=keep, dres=keep)
        assert torch.equal(keep, dx)


@pytest.mark.parametrize("rows,cols,over", [(40, 128, {}), (700, 4096, dict(residual="f32")), (120, 1001, dict(pad=1)), (3, 40000, {})])
def test_backward_without_a_weight(rows, cols, over):
    op, a, dres, dx = grad_case(rows, cols, weight=None, **over)
    db = torch.zeros(cols, device="cuda")
    op.backward(**a, dx=dx, dbias=db, dres=dres)
    check_backward(a, dres, dx, None, db, over.get("residual", "bf16"))
    with pytest.raises(D.DttError):
        op.backward(**a, dx=dx, dweight=db, dres=dres)


def test_backward_of_no_rows_zeroes_the_gradients():
    op, a, dres, dx = grad_case(0, 100)
    dw, db = (torch.full((100,), 7.0, device="cuda") for _ in range(2))
    op.backward(**a, dx=dx, dweight=dw, dbias=db, dres=dres)
    assert (dw == 0).all() and (db == 0).all()


def test_backward_is_the_forward_s_difference_quotient():
    """On the GPU's own forward in f32: central differences of step 2^-7 over sums of 64 terms."""
    op, a, _, dx = grad_case(2, 32, x="f32", residual="f32", weight="f32")
    dw, db = torch.empty(32, device="cuda"), torch.empty(32, device="cuda")
    op.backward(**a, dx=dx, dweight=dw, dbias=db)
    f32 = D.LayerNorm(32, x="f32", residual="f32", weight="f32", y="f32", eps=EPS)
    at = dict(h=a["h"], weight=a["weight"], bias=torch.zeros(32, device="cuda"))

    def loss(h, weight, bias):
        y = torch.empty_like(h)
        f32.forward(h, weight, bias, y)
        return float((a["dy"].double() * y.double()).sum())

    step = 2.0 ** -7
    for t, grad in (("h", dx), ("weight", dw), ("bias", db)):
        for i in np.ndindex(*at[t].shape):
            d = torch.zeros_like(at[t])
            d[i] = step
            up, down = (loss(**{**at, t: at[t] + s * d}) for s in (1, -1))
            # y is ~1, its rounding 2e-6 of it, dy 0.1: 64 x 0.1 x 2e-6 / 2^-6 at most 1e-3 (seen as a sum
            # of independent roundings 1e-4); the third derivative adds step^2 of the gradient's size
            assert abs((up - down) / (2 * step) - float(grad[i])) < 1e-3


@pytest.mark.parametrize("rows,cols", [(64, 4096), (700, 4096), (40, 1001)])
def test_a_captured_pass_replays_and_another_stream_takes_it(rows, cols):
    """Forward and backward in one graph, whose first call allocates the workspace, on a stream of its own."""
    op, a, more, out = case(rows, cols, y="bf16", residual="f32")
    grads = D.LayerNorm(cols, residual="f32", eps=EPS)
    dy, dx = slab(rows, cols, "bf16", 0, gen(3), 0.1), torch.zeros(rows, cols, device="cuda")
    dw, db = torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        op.forward(a["x"], a["weight"], a["bias"], **more, **out, stream=stream)
        grads.backward(dy, out["residual_out"], a["weight"], out["mean"], out["rstd"], dx, dw, db, stream=stream)
    for shift in (0.0, 1.0):
        a["x"].add_(shift)
        graph.replay()
        torch.cuda.synchronize()
        check(a, more, out, "bf16", 0)
        check_backward(dict(dy=dy, h=out["residual_out"], weight=a["weight"], mean=out["mean"], rstd=out["rstd"]), None, dx, dw, db, "f32")


@pytest.mark.parametrize("late", ["true", "r % 5 == 3", "r % 5 == 3 && t == 37"])
def test_rows_that_do_not_arrive_in_time_are_nan_and_so_are_the_parameters_gradients(late, tmp_path):
    """As test_gpu_ops_edges.py has it for the other norm: every value is right or NaN, whoever gives a row up."""
    from test_gpu_ops_edges import library_with
    L = library_with("norm.cu", [f"-DDTT_NORM_ROW_LATE=({late})"], str(tmp_path))
    for rows, cols, pad, kind in ((2000, 1024, 0, "bf16"), (1000, 4096, 0, "bf16"), (1000, 4096, 0, "f32"), (400, 12288, 0, "bf16"), (1300, 1001, 1, "f32"), (1300, 5001, 3, "f32")):
        op, a, more, _ = case(rows, cols, x=kind, residual=kind, weight=kind, y=kind, pad=pad)
        back, b, dres, _ = grad_case(rows, cols, x=kind, residual=kind, weight=kind, pad=pad)
        got = []
        for other in (False, True):
            if other:
                op._forward, back._backward = L.dtt_layernorm_forward, L.dtt_layernorm_backward
            y, h, dx = (torch.full((rows, cols + pad), 7.0, device="cuda").to(TYPES[kind])[:, :cols] for _ in range(3))
            mean, rstd, dw, db = (torch.full((n,), 7.0, device="cuda") for n in (rows, rows, cols, cols))
            forward(op, a, more, dict(y=y, residual_out=h, mean=mean, rstd=rstd))
            back.backward(**b, dx=dx, dweight=dw, dbias=db, dres=dres)
            got.append((y, h, mean, rstd, dx, dw, db))
        for right, seen in zip(*got):
            assert not torch.isnan(right).any()
            gone = torch.isnan(seen)
            assert gone.all() if late == "true" else (gone | (seen == right)).all()
        y, h, mean, rstd, dx, dw, db = got[1]
        assert torch.isnan(rstd[3::5]).all() and torch.isnan(mean[3::5]).all() and torch.isnan(h[3::5]).any(-1).all() and torch.isnan(dx[3::5]).all()
        assert torch.equal(torch.isnan(rstd), torch.isnan(y).all(-1)) and torch.equal(torch.isnan(rstd), torch.isnan(y).any(-1))
        assert torch.equal(torch.isnan(dx).any(-1), torch.isnan(dx).all(-1)) and torch.isnan(dw).any() and torch.isnan(db).any()


def test_rows_past_four_gigabytes():
    rows, cols = 70000, 32768                  # 4.6 GB of bf16
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-2:] = slab(2, cols, "bf16", 0, gen(9), 1.0, 3.0)
    y = torch.ones_like(x)
    out = dict(mean=torch.zeros(rows, device="cuda"), rstd=torch.zeros(rows, device="cuda"))
    D.LayerNorm(cols).forward(x, None, None, y, **out)
    tail = {k: v[-2:] for k, v in out.items()}
    check(dict(x=x[-2:], weight=None, bias=None), dict(residual=None), dict(y=y[-2:], residual_out=x[-2:], scales=None, **tail), "bf16", 0)
    assert not y[:-2].any()


def test_the_binding_refuses_what_does_not_fit():
    op, a, more, out = case(4, 64)
    for bad in (dict(bias=a["bias"].float()), dict(bias=a["bias"][:63]), dict(x=a["x"].float()), dict(x=a["x"].cpu()), dict(x=a["x"].t()[:4])):
        with pytest.raises(D.DttError):
            forward(op, {**a, **bad}, more, out)
    with pytest.raises(D.DttError):
        op.forward(a["x"], a["weight"], a["bias"], **more, **{**out, "mean": out["mean"].double()})
