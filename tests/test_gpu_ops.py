"""GPU: the norm, its backward pass and the orthogonalisation against the oracle's 64 bits.

Tolerances, from the arithmetic: e = 2^-24 is half an f32 ulp.  A row's sum of squares goes through at
most ~40 roundings on any path (a thread's columns, then two butterfly trees), all terms positive, so
it is within 40 e; half of that and a 2-ulp reciprocal square root reach rstd, and two products y:
30 e < 2e-6 in all.  Rounding to nearest moves a value by at most half the spacing of its binade:
2^-8 of the power of two below it in bf16 (8 significant bits), 2^-4 in e4m3 (4), where values below
2^-6 are 2^-9 apart."""
import numpy as np
import pytest
import torch

from oracle import norm as ON
from oracle import ortho as OO

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from conftest import ensure_built
    ensure_built()
    import device_triggered_transfers_gb300 as D

E = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BITS = {"bf16": 8, "f32": 24}                # significant bits
COEFFS = (3.4445, -4.7750, 2.0315)


def f64(t):
    return t.to(torch.float32).double().cpu().numpy() if t.dtype != torch.float32 else t.double().cpu().numpy()


def half_spacing(v, kind):
    """Half the distance between neighbours of `kind` around v (f64)."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 1e-37))) - BITS[kind])


def slab(rows, cols, kind, pad, gen, spread=1.0):
    """rows x cols values as a view of a buffer `pad` columns wider."""
    t = torch.randn(rows, cols + pad, generator=gen, device="cuda") * spread
    return t.to(TYPES[kind])[:, :cols]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def norm_case(rows, cols, x="bf16", residual="bf16", weight="bf16", y="bf16", group=0, pad=0, seed=0):
    g = gen(seed)
    op = D.RMSNorm(cols, x=x, residual=residual or x, weight=weight or "bf16", y=y, group=group, eps=1e-5)
    a = dict(x=slab(rows, cols, x, pad, g, 0.5),
             residual=slab(rows, cols, residual, pad, g, 3.0) if residual else None,
             weight=(1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(TYPES[weight]) if weight else None)
    out = dict(y=torch.zeros(rows, cols + pad, device="cuda").to(TYPES[y])[:, :cols],
               residual_out=slab(rows, cols, residual or x, pad, g),
               scales=torch.full((rows, op.scale_cols), -1.0, device="cuda") if y == "e4m3" else None,
               rstd=torch.full((rows,), -1.0, device="cuda"))
    return op, a, out


def check_forward(a, out, y, group, eps=1e-5):
    none = lambda t: None if t is None else f64(t)  # noqa: E731
    h, rstd, want = ON.forward(f64(a["x"]), none(a["residual"]), none(a["weight"]), eps)
    if out["residual_out"] is not None:
        kind = "bf16" if out["residual_out"].dtype == torch.bfloat16 else "f32"
        assert (np.abs(f64(out["residual_out"]) - h) <= half_spacing(h, kind) + 2 * E * np.abs(h)).all()
    if out["rstd"] is not None:
        np.testing.assert_allclose(f64(out["rstd"]), rstd, rtol=2e-6)
    got = f64(out["y"])
    # h itself is one rounded addition: where x and residual cancel its error is that of the larger
    slack = 2e-6 * np.abs(want) + 2 * E * np.abs(want / np.where(h == 0, 1, h)) * np.abs(f64(a["x"]))
    if y != "e4m3":
        assert (np.abs(got - want) <= half_spacing(want, y) + slack).all()
        return
    s = ON.scales(want, group)
    np.testing.assert_allclose(f64(out["scales"]), s, rtol=3e-6, atol=1e-35)
    s = ON.spread(f64(out["scales"]), group, want.shape[1])
    assert (np.abs(got) <= 448).all()
    assert (np.abs(got * s - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s) * 1.001 + slack).all()


NORMS = [
    (1, 1, {}), (3, 5, {}), (2, 8, dict(y="f32")), (5, 31, dict(pad=1)), (9, 256, {}), (7, 257, {}),
    (1, 4096, dict(y="e4m3")), (37, 8064, dict(y="e4m3", group=128)), (300, 64, dict(y="e4m3", group=32)),
    (5, 200, dict(y="e4m3", group=64)), (3, 4097, dict(y="e4m3", group=128, pad=7)),
    (64, 4096, dict(x="f32", residual="f32", weight="f32", y="f32")),
    (64, 1000, dict(residual="f32", pad=8)), (11, 2048, dict(x="f32", residual="bf16", y="e4m3")),
    (130, 5001, dict(residual="f32", pad=7)), (20, 4096, dict(residual=None)), (20, 4096, dict(weight=None)),
    (4, 16384, {}), (3, 32768, dict(y="e4m3")), (2, 32769, dict(y="e4m3")), (2, 70000, dict(y="e4m3", group=128)),
    (2, 40000, dict(residual="f32", y="f32", pad=3)), (700, 4096, dict(y="e4m3")), (700, 4096, {}),
    (1000, 8064, dict(y="e4m3", group=128)), (999, 1024, dict(x="f32", residual="f32", y="f32")),
    (2500, 512, dict(y="e4m3", group=64)), (611, 12288, {}),
]


@pytest.mark.parametrize("rows,cols,over", NORMS)
def test_forward(rows, cols, over):
    op, a, out = norm_case(rows, cols, **over)
    before = out["y"].clone() if over.get("pad") else None
    op.forward(**a, **out)
    torch.cuda.synchronize()
    check_forward(a, out, over.get("y", "bf16"), over.get("group", 0))
    assert before is None or before.shape == out["y"].shape


def test_forward_writes_nothing_beside_its_rows():
    rows, cols = 33, 1000
    op = D.RMSNorm(cols, y="e4m3", group=128)
    g = gen(3)
    wide = {k: torch.full((rows, 1024), 7.0, device="cuda").to(TYPES[t]) for k, t in (("y", "e4m3"), ("r", "bf16"))}
    op.forward(slab(rows, cols, "bf16", 0, g), None, wide["y"][:, :cols], residual_out=wide["r"][:, :cols],
               scales=torch.empty(rows, 8, device="cuda"))
    torch.cuda.synchronize()
    assert (wide["y"][:, cols:].float() == 7).all() and (wide["r"][:, cols:] == 7).all()


@pytest.mark.parametrize("rows,cols", [(5, 4096), (5, 40000), (700, 4096), (3, 1001)])
def test_forward_in_place(rows, cols):
    """residual_out = residual gives the same bits as apart; so does leaving the optional outputs out."""
    op, a, out = norm_case(rows, cols, y="e4m3")
    op.forward(**a, **out)
    b = {k: v if v is None else v.clone() for k, v in out.items()}
    r = a["residual"].clone()
    op.forward(a["x"], a["weight"], b["y"], residual=r, residual_out=r, scales=b["scales"])
    torch.cuda.synchronize()
    assert torch.equal(r, out["residual_out"]) and torch.equal(b["scales"], out["scales"])
    assert torch.equal(b["y"].view(torch.uint8), out["y"].view(torch.uint8))


@pytest.mark.parametrize("rows", [4, 700])
@pytest.mark.parametrize("group", [0, 128])
def test_forward_zeros_infinities_and_nan_stay_in_their_row(rows, group):
    op, a, out = norm_case(rows, 1024, y="e4m3", group=group)
    a["x"][0] = 0
    a["residual"][0] = 0
    a["x"][1, 7] = float("nan")
    a["x"][2, 1023] = float("inf")
    op.forward(**a, **out)
    torch.cuda.synchronize()
    assert (out["y"][0].float() == 0).all() and (out["scales"][0] == ON.SCALE_MIN).all()
    assert torch.isnan(out["rstd"][1]) and torch.isnan(out["scales"][1]).all() and torch.isnan(out["y"][1].float()).all()
    # an infinity: rstd 0, its own element 0 x inf, everything of its group NaN, other groups zeros
    assert out["rstd"][2] == 0 and torch.isnan(out["y"][2].float())[-1]
    assert (out["y"][2, :896].float() == 0).all() or group == 0
    keep = {k: (v[3:] if v is not None and v.dim() and v.shape[0] == rows else v) for k, v in {**a, **out}.items()}
    check_forward({k: keep[k] for k in a}, {k: keep[k] for k in out}, "e4m3", group)


def test_forward_past_four_gigabytes():
    rows, cols = 70000, 32768                  # 4.6 GB of bf16: byte offsets beyond 32 bits
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = gen(9)
    x[-2:] = torch.randn(2, cols, generator=g, device="cuda").to(torch.bfloat16)
    y = torch.ones_like(x)
    D.RMSNorm(cols, eps=1e-5).forward(x, None, y)
    torch.cuda.synchronize()
    check_forward(dict(x=x[-2:], residual=None, weight=None), dict(y=y[-2:], residual_out=None, rstd=None, scales=None),
                  "bf16", 0)
    assert not y[:-2].any()


def grad_case(rows, cols, x="bf16", residual="bf16", weight="bf16", pad=0, dres=True, seed=1):
    g = gen(seed)
    op = D.RMSNorm(cols, x=x, residual=residual, weight=weight, eps=1e-5)
    h = slab(rows, cols, residual, pad, g, 3.0)
    a = dict(dy=slab(rows, cols, x, pad, g, 0.1), h=h,
             weight=(1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(TYPES[weight]),
             rstd=(h.float().square().mean(-1) + 1e-5).rsqrt())
    return op, a, slab(rows, cols, residual, pad, g, 0.1) if dres else None, slab(rows, cols, residual, pad, g)


def check_backward(a, dres, dx, dw, residual):
    dy, h, w, s = (f64(a[k]) for k in ("dy", "h", "weight", "rstd"))
    want, want_dw = ON.backward(dy, h, w, s, None if dres is None else f64(dres))
    # f32 errors are relative to the terms: the row's mean goes through ~45 roundings, the rest a few
    n, g = h * s[:, None], dy * w
    terms = s[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
    slack = 50 * E * (terms + (0 if dres is None else np.abs(f64(dres))))
    assert (np.abs(f64(dx) - want) <= half_spacing(want, residual) + slack).all()
    if dw is not None:
        # each partial row adds its rows one after the other, then the partial rows are added
        depth = len(dy) / min(len(dy), 100) + 400
        assert (np.abs(f64(dw) - want_dw) <= depth * E * np.abs(dy * n).sum(axis=0)).all()


GRADS = [(1, 1, {}), (3, 5, dict(x="f32", residual="f32")), (2, 64, {}), (17, 256, {}), (16, 4096, {}),
         (700, 4096, {}), (2000, 1024, dict(dres=False)), (1021, 5001, dict(x="f32", residual="f32", weight="f32", pad=3)),
         (50, 8064, dict(residual="f32")), (300, 8064, {}), (9, 12288, {}), (5, 16384, {}), (700, 16385, {}),
         (3, 20000, dict(pad=1)), (611, 4104, dict(weight="f32")), (640, 8192, dict(residual="f32", weight="f32"))]


@pytest.mark.parametrize("rows,cols,over", GRADS)
def test_backward(rows, cols, over):
    op, a, dres, dx = grad_case(rows, cols, **over)
    dw = torch.full((cols,), 7.0, device="cuda")
    op.backward(**a, dx=dx, dweight=dw, dres=dres)
    torch.cuda.synchronize()
    check_backward(a, dres, dx, dw, over.get("residual", "bf16"))
    again, dw2 = dx.clone(), torch.zeros_like(dw)
    op.backward(**a, dx=again, dweight=dw2, dres=dres)
    if dres is not None:                        # in place, and without the weight's gradient
        keep = dres.clone()
        op.backward(**a, dx=keep, dres=keep)
        assert torch.equal(keep, dx)
    torch.cuda.synchronize()
    assert torch.equal(again, dx) and torch.equal(dw, dw2)


def test_backward_of_no_rows_zeroes_the_weight_s_gradient():
    op, a, dres, dx = grad_case(0, 100)
    dw = torch.full((100,), 7.0, device="cuda")
    op.backward(**a, dx=dx, dweight=dw, dres=dres)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_backward_is_the_forward_s_difference_quotient():
    """On the GPU's own forward in f32: central differences of step 2^-7 over sums of 64 terms."""
    op, a, _, dx = grad_case(2, 32, x="f32", residual="f32", weight="f32")
    dw = torch.empty(32, device="cuda")
    op.backward(**a, dx=dx, dweight=dw)
    f32 = D.RMSNorm(32, x="f32", residual="f32", weight="f32", y="f32", eps=1e-5)

    def loss(h, w):
        y = torch.empty_like(h)
        f32.forward(h, w, y)
        return float((a["dy"].double() * y.double()).sum())

    step = 2.0 ** -7
    for t, grad in (("h", dx), ("weight", dw)):
        for i in np.ndindex(*a[t].shape):
            d = torch.zeros_like(a[t])
            d[i] = step
            up, down = (loss(a["h"] + s * d, a["weight"]) if t == "h" else loss(a["h"], a["weight"] + s * d) for s in (1, -1))
            # y is ~1, its rounding 2e-6 of it, dy 0.1: 64 x 0.1 x 2e-6 / 2^-6 at most 1e-3 (seen as a sum
            # of independent roundings 1e-4); the third derivative adds step^2 of the gradient's size
            assert abs((up - down) / (2 * step) - float(grad[i])) < 1e-3


# rows of a part of a warp; and the ring where a CTA has no row, or one row, and room for two stages alone
SHORT = [(1, 8, dict(y="e4m3")), (33, 16, dict(y="e4m3", group=128)), (1000, 24, dict(y="e4m3", group=32)),
         (70, 40, dict(y="e4m3", group=32)), (257, 64, dict(y="e4m3", group=64)), (10001, 128, dict(y="e4m3")),
         (5003, 128, dict(residual="f32", y="e4m3", group=64)), (77, 200, dict(x="f32", residual="f32", y="e4m3", group=128)),
         (513, 256, dict(weight=None)), (40, 136, dict(residual=None, weight="f32", y="f32")), (65, 128, dict(pad=8)),
         (2, 264, dict(y="e4m3", group=64)), (151, 12288, dict(x="f32", residual="f32", y="e4m3", group=128)),
         (1217, 1001, dict(y="e4m3", group=64)), (1215, 1001, dict(y="e4m3", group=64))]


@pytest.mark.parametrize("rows,cols,over", SHORT)
def test_short_rows_and_small_rings(rows, cols, over):
    op, a, out = norm_case(rows, cols, **over)
    op.forward(**a, **out)
    torch.cuda.synchronize()
    check_forward(a, out, over.get("y", "bf16"), over.get("group", 0))
    kinds = {k: over[k] for k in ("x", "pad") if k in over}
    kinds["residual"] = over.get("residual") or "bf16"
    for dres in (True, False):
        op, a, dres, dx = grad_case(rows, cols, dres=dres, **kinds)
        dw, again = torch.full((cols,), 7.0, device="cuda"), torch.zeros(cols, device="cuda")
        op.backward(**a, dx=dx, dweight=dw, dres=dres)
        op.backward(**a, dx=torch.empty_like(dx), dweight=again, dres=dres)
        torch.cuda.synchronize()
        check_backward(a, dres, dx, dw, kinds["residual"])
        assert torch.equal(dw, again)


@pytest.mark.parametrize("rows,cols,over", [
    (96, 1000, {}), (97, 1000, {}), (96, 4096, dict(residual="f32")), (5, 40000, {}), (63, 5001, dict(x="f32", residual="f32", pad=3)),
    (95, 30000, dict(pad=1)), (96, 128, {}), (97, 128, {}), (1, 64, {}), (33, 31, dict(pad=1)), (2, 19500, {})])
def test_weight_gradient_of_few_rows(rows, cols, over):
    op, a, dres, dx = grad_case(rows, cols, **over)
    dw, again = torch.full((cols + 9,), 7.0, device="cuda"), torch.zeros(cols, device="cuda")
    op.backward(**a, dx=dx, dweight=dw[4:4 + cols], dres=dres)
    op.backward(**a, dx=torch.empty_like(dx), dweight=again, dres=dres)
    torch.cuda.synchronize()
    check_backward(a, dres, dx, dw[4:4 + cols], over.get("residual", "bf16"))
    assert torch.equal(dw[4:4 + cols], again) and (dw[:4] == 7).all() and (dw[4 + cols:] == 7).all()


def test_short_rows_keep_nan_to_themselves_and_their_slices():
    """NaN in a row that shares its warp with others; nothing beside the rows is written."""
    rows, cols, pad = 37, 104, 16
    op, a, out = norm_case(rows, cols, y="e4m3", group=32)
    a["x"][3, 50] = float("nan")
    a["x"][4], a["residual"][4] = 0, 0
    wide = torch.full((rows, cols + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    out["residual_out"] = wide[:, 8:8 + cols]
    op.forward(**a, **out)
    torch.cuda.synchronize()
    assert torch.isnan(out["rstd"][3]) and torch.isnan(out["y"][3].float()).all() and torch.isnan(out["scales"][3]).all()
    assert (out["y"][4].float() == 0).all() and (out["scales"][4] == ON.SCALE_MIN).all()
    keep = [i for i in range(rows) if i not in (3, 4)]
    check_forward({k: v if k == "weight" else v[keep] for k, v in a.items()}, {k: v[keep] for k, v in out.items()}, "e4m3", 32)
    assert (wide[:, :8] == 7).all() and (wide[:, 8 + cols:] == 7).all()
    op, a, dres, dx = grad_case(rows, cols)
    a["dy"][3, 50] = float("nan")
    op.backward(**a, dx=dx, dres=dres)
    torch.cuda.synchronize()
    assert torch.isnan(dx[3]).all()
    check_backward({k: v if k == "weight" else v[keep] for k, v in a.items()}, dres[keep], dx[keep], None, "bf16")


# ---- orthogonalisation ----------------------------------------------------------------------------
# The result's bf16 rounding is 1.7e-3 of its norm (half a spacing at most, uniform).  Operands rounded to f16
# (2^-12 of the value, uniform: 1.4e-4) enter a step through b A + c A A, at most 2.9 in norm, three of
# them: 7e-4 a step as independent errors, which the next steps' slopes (at most 1.7 near 1)
# multiply by 1, 1.7, 2.9, 4.9: 4.2e-3.  Together 4.5e-3; twice that is the bound.
ORTHO_TOL = 9e-3
# a rank-1 update: rounding noise of X in the directions it lacks would be 1e-1
RANK1_TOL = 5e-3


def rel(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


ORTHOS = [(1, 1, 1), (1, 3, 1), (2, 1, 100), (1, 8, 8), (3, 17, 33), (1, 64, 64), (1, 127, 129), (2, 128, 256),
          (1, 300, 200), (1, 1000, 256), (2, 200, 1111), (1, 512, 512), (3, 129, 640), (1, 640, 1920)]


@pytest.mark.parametrize("batch,rows,cols", ORTHOS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_orthogonalize(batch, rows, cols, dtype):
    x = (torch.randn(batch, rows, cols, generator=gen(rows + cols), device="cuda") * 1e-3).to(TYPES[dtype])
    out = torch.zeros(batch, rows, cols, dtype=torch.bfloat16, device="cuda")
    with D.Orthogonalizer(rows, cols, batch=batch, dtype=dtype, scale=0.5) as op:
        op.run(x, out)
        again = torch.zeros_like(out)
        op.run(x, again)
        assert op.errors == 0
    assert torch.equal(out, again)
    for i in range(batch):
        assert rel(f64(out[i]), OO.orthogonalize(f64(x[i]), 5, [COEFFS] * 5, 1e-7, 0.5)) < ORTHO_TOL


def orthogonalized(x, steps=5):
    """The formula in 64 bits on the device, for matrices that take the host too long."""
    x = x.double()
    if x.shape[0] > x.shape[1]:
        return orthogonalized(x.T, steps).T
    x = x / (x.norm() + 1e-7)
    a, b, c = COEFFS
    for _ in range(steps):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x


# one cluster a matrix, up to its longest row and one past it; the second product within the third; its limit
# and one past it; a product by CTA pairs; everything in one launch, with a last row block of 1, 2 or 64 rows
LARGE = [(2, 128, 4096), (1, 128, 4097), (1, 4096, 100), (5, 129, 1000), (9, 256, 700), (1, 2000, 250), (1, 257, 3000),
         (3, 1024, 1500), (4, 700, 4000), (1, 1500, 3500),
         (1, 8192, 2048), (1, 2048, 2048), (3, 2050, 2049), (1, 2300, 1900), (1, 1600, 5000), (5, 1025, 1100), (40, 257, 600)]


@pytest.mark.parametrize("batch,rows,cols", LARGE)
def test_orthogonalize_large(batch, rows, cols):
    x = torch.randn(batch, rows, cols, generator=gen(rows + cols), device="cuda").to(torch.bfloat16)
    if batch > 2:
        x[1, 5, 7] = float("nan")               # spoils its own matrix alone
    out, again = (torch.zeros(batch, rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with D.Orthogonalizer(rows, cols, batch=batch) as op:
        op.run(x, out)
        op.run(x, again)
        assert op.errors == 0
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    for i in range(batch):
        if batch > 2 and i == 1:
            assert torch.isnan(out[i]).all()
            continue
        want = orthogonalized(x[i])
        assert float((out[i].double() - want).norm() / want.norm()) < ORTHO_TOL


def test_orthogonalize_large_in_a_graph_beside_strided_arguments():
    """Everything in one launch: captured, replayed on new values, the result by columns and by rows into slices."""
    s = torch.cuda.Stream()
    for rows, cols in ((2100, 2501), (2501, 2100)):
        g = gen(rows)
        x = torch.randn(rows, cols, generator=g, device="cuda")
        res = torch.full((rows + 2, cols + 3), 7.0, dtype=torch.bfloat16, device="cuda")
        m = torch.zeros(rows, cols, device="cuda")
        out = res[1:rows + 1, 2:cols + 2]
        with D.Orthogonalizer(rows, cols, dtype="f32", mu=0.5, steps=3, coeffs=[COEFFS] * 3) as op:
            s.wait_stream(torch.cuda.current_stream())
            op.run(x, out, momentum=m, stream=s)
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                op.run(x, out, momentum=m, stream=s)
            x.normal_(generator=g)
            before = m.clone()
            out.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert op.errors == 0
        want_m = 0.5 * before.double() + x.double()
        assert float((m.double() - want_m).abs().max()) < 1e-5
        want = orthogonalized(want_m, 3)
        assert float((out.double() - want).norm() / want.norm()) < ORTHO_TOL
        out.fill_(7)
        assert (res == 7).all()


@pytest.mark.parametrize("rank", [1, 4])
def test_orthogonalize_large_of_low_rank(rank):
    g = gen(rank)
    x = torch.randn(2048, rank, generator=g, device="cuda") @ torch.randn(rank, 2304, generator=g, device="cuda")
    out = torch.empty(2048, 2304, dtype=torch.bfloat16, device="cuda")
    with D.Orthogonalizer(2048, 2304, dtype="f32") as op:
        op.run(x, out)
        assert op.errors == 0
    want = orthogonalized(x)
    assert float((out.double() - want).norm() / want.norm()) < RANK1_TOL


@pytest.mark.parametrize("nesterov", [False, True])
def test_orthogonalize_with_momentum_over_steps(nesterov):
    rows, cols, mu = 96, 160, 0.95
    g = gen(4)
    m = torch.zeros(2, rows, cols, device="cuda")
    want_m = np.zeros((2, rows, cols))
    out = torch.empty(2, rows, cols, dtype=torch.bfloat16, device="cuda")
    with D.Orthogonalizer(rows, cols, batch=2, mu=mu, nesterov=nesterov) as op:
        for step in range(3):
            x = torch.randn(2, rows, cols, generator=g, device="cuda").to(torch.bfloat16)
            op.run(x, out, momentum=m)
            u, want_m = OO.momentum_step(f64(x), want_m, np.float32(mu), nesterov)
            assert op.errors == 0
            assert np.abs(f64(m) - want_m).max() < 4 * E * (step + 1) * 20
            for i in range(2):
                assert rel(f64(out[i]), OO.orthogonalize(u[i], 5, [COEFFS] * 5, 1e-7)) < ORTHO_TOL


@pytest.mark.parametrize("rows,cols", [(65, 130), (130, 65)])
def test_orthogonalize_strided_arguments(rows, cols):
    """Slices of wider, taller buffers at odd offsets; nothing beside them is written."""
    g = gen(8)
    wide = torch.randn(2, rows + 3, cols + 5, generator=g, device="cuda").to(torch.bfloat16)
    mom = torch.randn(2, rows + 1, cols + 1, generator=g, device="cuda")
    res = torch.full((2, rows + 2, cols + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    x, m, out = wide[:, 1:rows + 1, 3:cols + 3], mom[:, 1:, 1:], res[:, 1:rows + 1, 1:cols + 1]
    before = f64(m)
    kept = mom[:, 0].clone()
    with D.Orthogonalizer(rows, cols, batch=2, mu=0.9, nesterov=True) as op:
        op.run(x, out, momentum=m)
        assert op.errors == 0
    u, want_m = OO.momentum_step(f64(x), before, np.float32(0.9), True)
    np.testing.assert_allclose(f64(m), want_m, rtol=1e-6, atol=1e-6)
    for i in range(2):
        assert rel(f64(out[i]), OO.orthogonalize(u[i], 5, [COEFFS] * 5, 1e-7)) < ORTHO_TOL
    res[:, 1:rows + 1, 1:cols + 1] = 7
    assert (res == 7).all() and torch.equal(mom[:, 0], kept)


@pytest.mark.parametrize("rank", [1, 4])
@pytest.mark.parametrize("rows,cols", [(256, 512), (700, 300)])
def test_orthogonalize_of_low_rank(rows, cols, rank):
    g = gen(rank)
    x = torch.randn(rows, rank, generator=g, device="cuda") @ torch.randn(rank, cols, generator=g, device="cuda")
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    with D.Orthogonalizer(rows, cols, dtype="f32") as op:
        op.run(x, out)
        assert op.errors == 0
    assert rel(f64(out), OO.orthogonalize(f64(x), 5, [COEFFS] * 5, 1e-7)) < RANK1_TOL


def test_orthogonalize_other_steps():
    """Steps with coefficients of their own, and one step alone; 1.5 s - 0.5 s^3 keeps values below 1."""
    x = torch.randn(96, 224, generator=gen(2), device="cuda")
    out = torch.empty(96, 224, dtype=torch.bfloat16, device="cuda")
    for coeffs in ([(4.0, -6.0, 3.0), (3.0, -3.0, 1.0), (1.5, -0.5, 0.0)], [(1.5, -0.5, 0.0)], [COEFFS] * 6):
        with D.Orthogonalizer(96, 224, dtype="f32", steps=len(coeffs), coeffs=coeffs) as op:
            op.run(x, out)
            assert op.errors == 0
        assert rel(f64(out), OO.orthogonalize(f64(x), len(coeffs), coeffs, 1e-7)) < 2 * ORTHO_TOL


def test_orthogonalize_zeros_and_nan():
    x = torch.zeros(3, 70, 90, device="cuda")
    x[1, 3, 4] = float("nan")
    x[2] = torch.randn(70, 90, generator=gen(1), device="cuda")
    out = torch.ones(3, 70, 90, dtype=torch.bfloat16, device="cuda")
    with D.Orthogonalizer(70, 90, batch=3, dtype="f32") as op:
        op.run(x, out)
        assert op.errors == 0
    assert (out[0] == 0).all() and torch.isnan(out[1]).all()
    assert rel(f64(out[2]), OO.orthogonalize(f64(x[2]), 5, [COEFFS] * 5, 1e-7)) < ORTHO_TOL


# ---- streams, graphs, refusals -----------------------------------------------------------------------
def test_on_another_stream_and_in_a_graph():
    """The operators on a stream of the caller's, captured once and replayed on new values."""
    op, a, out = norm_case(64, 4096, y="e4m3", group=128)
    gop, ga, dres, dx = grad_case(64, 4096)
    dw = torch.empty(4096, device="cuda")
    x = torch.randn(100, 200, generator=gen(6), device="cuda")
    o = torch.empty(100, 200, dtype=torch.bfloat16, device="cuda")
    ortho = D.Orthogonalizer(100, 200, dtype="f32")
    s = torch.cuda.Stream()

    def all_three():
        op.forward(**a, **out, stream=s)
        gop.backward(**ga, dx=dx, dweight=dw, dres=dres, stream=s)
        ortho.run(x, o, stream=s)

    s.wait_stream(torch.cuda.current_stream())
    all_three()                                 # kernels loaded, workspaces there
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        all_three()
    a["x"].normal_(generator=gen(77))
    ga["dy"].normal_(generator=gen(78))
    x.normal_(generator=gen(79))
    for t in (out["y"].view(torch.uint8), dx, dw, o):
        t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check_forward(a, out, "e4m3", 128)
    check_backward(ga, dres, dx, dw, "bf16")
    assert rel(f64(o), OO.orthogonalize(f64(x), 5, [COEFFS] * 5, 1e-7)) < ORTHO_TOL and ortho.errors == 0
    ortho.close()


def test_refuses_wrong_tensors():
    op, a, out = norm_case(4, 64, y="e4m3")
    bad = [dict(x=a["x"].float()), dict(x=a["x"][:, :32]), dict(x=a["x"].cpu()), dict(weight=a["weight"][:32]),
           dict(weight=a["weight"].float()), dict(residual=a["residual"][:2]), dict(y=out["y"].float()),
           dict(scales=None), dict(scales=out["scales"][:2]), dict(rstd=out["rstd"].double()),
           dict(x=torch.empty(64, 4, dtype=torch.bfloat16, device="cuda").T)]
    for over in bad:
        with pytest.raises(D.DttError) as e:
            op.forward(**{**a, **out, **over})
        assert e.value.code == D.EINVAL
    x = torch.zeros(8, 16, device="cuda")
    o = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    with D.Orthogonalizer(8, 16, dtype="f32") as plain, D.Orthogonalizer(8, 16, dtype="f32", mu=0.9) as mom:
        for call in (lambda: plain.run(x, x), lambda: plain.run(o, o), lambda: plain.run(x.T, o), lambda: plain.run(x, o, momentum=x),
                     lambda: mom.run(x, o), lambda: plain.run(x, None), lambda: mom.run(x, o, momentum=o)):
            with pytest.raises(D.DttError) as e:
                call()
            assert e.value.code == D.EINVAL
    for kw in (dict(coeffs=[(1, 2)]), dict(steps=2, coeffs=[(1, 0, 0)]), dict(dtype="u8"), dict(dtype="e4m3"), dict(eps=0.0)):
        with pytest.raises(D.DttError) as e:
            D.Orthogonalizer(8, 16, **kw)
        assert e.value.code == D.EINVAL
