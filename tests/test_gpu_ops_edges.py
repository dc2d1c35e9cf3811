"""GPU: where the operators can go wrong though ordinary values do not show it."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from conftest import ensure_built
    ensure_built()
    import device_triggered_transfers_gb300 as D

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def slab(rows, cols, pad, make, kind="f32"):
    """rows x cols of a buffer `pad` columns wider, filled by make(rows, cols + pad)."""
    return make(rows, cols + pad).to(TYPES[kind])[:, :cols]


# a case of each form of the forward pass: short rows, the ring's three, chunks, rows read again, and the same of
# single elements (few and many rows)
FORWARD = [(40, 128, 32, 0), (40, 256, 0, 0), (1300, 1024, 64, 0), (40, 4096, 128, 0), (40, 8192, 0, 0), (3, 16384, 0, 0), (3, 32768, 128, 0),
           (2, 65536, 128, 0), (40, 128, 32, 1), (40, 4096, 0, 1), (3, 16384, 64, 1), (2, 32768, 0, 1), (1300, 1024, 128, 1), (1300, 4096, 0, 1)]


@pytest.mark.parametrize("rows,cols,group,pad", FORWARD)
def test_codes_are_the_quotients_nearest_even(rows, cols, group, pad):
    """y is the weight (the rows are +-1), most of it midway between two codes times a scale of few bits: the
    f32 quotient is exactly midway and the code the even one."""
    g = gen(rows + cols)
    x = slab(rows, cols, pad, lambda *s: torch.where(torch.rand(*s, generator=g, device="cuda") < 0.5, -1.0, 1.0))
    width = group or cols
    mid = (2.0 * torch.randint(8, 16, (cols,), generator=g, device="cuda") + 1) / 16 * 2.0 ** torch.randint(-6, 9, (cols,), generator=g, device="cuda")
    mid = torch.where(mid > 448, 17.0, mid)
    mid[::width] = 448.0
    t = 1 + torch.randint(0, 1300, (cols // width,), generator=g, device="cuda") / 4096.0
    weight = mid * t.repeat_interleave(width)
    kinds = dict(x="f32", residual="f32", weight="f32", eps=0.0)
    op = D.RMSNorm(cols, y="e4m3", group=group, **kinds)
    codes = slab(rows, cols, pad, lambda *s: torch.zeros(*s, device="cuda"), "e4m3")
    y = slab(rows, cols, pad, lambda *s: torch.zeros(*s, device="cuda"))
    scales = torch.zeros(rows, op.scale_cols, device="cuda")
    op.forward(x, weight, codes, scales=scales)
    D.RMSNorm(cols, y="f32", **kinds).forward(x, weight, y)
    quotient = y / scales.repeat_interleave(width, 1)
    want = quotient.to(TYPES["e4m3"])
    # 4 significant bits of e4m3, so a value midway has its fifth bit set and none after it
    assert ((quotient.view(torch.int32) & 0xFFFFF) == 0x80000).float().mean() > 0.2
    assert torch.equal(codes.contiguous().view(torch.uint8), want.view(torch.uint8))


def test_codes_of_many_values_are_the_quotients():
    for rows, cols, group, pad in ((16384, 4096, 128, 0), (100000, 128, 32, 0), (4000, 1001, 64, 1), (64, 40000, 0, 0)):
        g = gen(cols)
        x = slab(rows, cols, pad, lambda *s: torch.randn(*s, generator=g, device="cuda"))
        weight = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
        op = D.RMSNorm(cols, x="f32", residual="f32", weight="f32", y="e4m3", group=group)
        codes = torch.zeros(rows, cols + pad, device="cuda").to(TYPES["e4m3"])[:, :cols]
        y = torch.zeros(rows, cols + pad, device="cuda")[:, :cols]
        scales = torch.zeros(rows, op.scale_cols, device="cuda")
        op.forward(x, weight, codes, scales=scales)
        D.RMSNorm(cols, x="f32", residual="f32", weight="f32", y="f32").forward(x, weight, y)
        want = (y / scales.repeat_interleave(group or cols, 1)[:, :cols]).to(TYPES["e4m3"])
        assert torch.equal(codes.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8)), (rows, cols)


@pytest.mark.parametrize("rows,cols,group,pad", FORWARD)
def test_rows_of_small_values_under_a_large_weight(rows, cols, group, pad):
    """rstd weight is beyond f32, h rstd weight is not (and in reverse, where it would be 0)."""
    for size, weight, dtype in ((1e-18, 1e21, "f32"), (1e15, 1e-32, "f32")):
        x = slab(rows, cols, pad, lambda *s: size * (1 + torch.rand(*s, generator=gen(cols), device="cuda")))
        y = slab(rows, cols, pad, lambda *s: torch.zeros(*s, device="cuda"), dtype)
        w = torch.full((cols,), weight, device="cuda")
        D.RMSNorm(cols, x="f32", residual="f32", weight="f32", y=dtype, eps=0.0).forward(x, w, y)
        h = x.double()
        want = h * (h.square().mean(-1, keepdim=True)).rsqrt() * w.double()
        # the row's error as in test_gpu_ops.py; a sum of squares around 1e-36 has all of f32's bits
        assert ((y.double() - want).abs() <= 2e-6 * want.abs()).all()


# ---- orthogonalisation ----------------------------------------------------------------------------
COEFFS = (3.4445, -4.7750, 2.0315)
ORTHO_TOL = 9e-3                             # as test_gpu_ops.py derives it


def orthogonalized(u, steps=5, eps=1e-7):
    """The formula in 64 bits on the device; one matrix."""
    u = u.double()
    if u.shape[0] > u.shape[1]:
        return orthogonalized(u.T, steps, eps).T
    u = u / (u.norm() + eps)
    a, b, c = COEFFS
    for _ in range(steps):
        g = u @ u.T
        u = a * u + (b * g + c * (g @ g)) @ u
    return u


@pytest.mark.parametrize("batch,rows,cols", [(1, 512, 8192), (4, 700, 4000), (1, 2048, 8192)])
def test_parts_of_the_first_product_are_all_there(batch, rows, cols):
    """Large matrices whose first product is worked out in parts that other CTAs add: the same bits every time."""
    x = torch.randn(batch, rows, cols, generator=gen(rows), device="cuda").to(torch.bfloat16)
    out, again = (torch.zeros(batch, rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with D.Orthogonalizer(rows, cols, batch=batch) as op:
        op.run(x, out)
        for _ in range(20):
            again.zero_()
            op.run(x, again)
            assert torch.equal(out.view(torch.int16), again.view(torch.int16))
        assert op.errors == 0
    for i in range(batch):
        want = orthogonalized(x[i])
        assert float((out[i].double() - want).norm() / want.norm()) < ORTHO_TOL


# a form each: one cluster, the second product within the third, a product a launch, everything in one launch
FORMS = [(3, 96, 160), (2, 256, 512), (2, 520, 1032), (2, 2048, 2056), (3, 65, 130), (2, 700, 300), (2, 1201, 2049)]


@pytest.mark.parametrize("batch,rows,cols", FORMS)
def test_matrices_whose_rows_alternate(batch, rows, cols):
    """A batch as the middle dimension: the same bits as one matrix after the other."""
    g = gen(rows)
    x = torch.randn(batch, rows, cols, generator=g, device="cuda")
    m = torch.randn(batch, rows, cols, generator=g, device="cuda")
    out = torch.zeros(batch, rows, cols, dtype=torch.bfloat16, device="cuda")
    x2, m2 = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (x, m))
    out2 = torch.zeros(rows, batch, cols, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert x2.stride(0) == cols and x2.stride(1) == batch * cols
    with D.Orthogonalizer(rows, cols, batch=batch, dtype="f32", mu=0.9, nesterov=True) as op:
        op.run(x, out, momentum=m)
        op.run(x2, out2, momentum=m2)
        assert op.errors == 0
        for shared in (x[:1].expand(batch, rows, cols), x.as_strided((batch, rows, cols), (cols - 1, batch * cols, 1)),
                       x.as_strided((batch, rows, cols), (cols, batch * cols - 1, 1))):
            with pytest.raises(D.DttError) as e:
                op.run(shared, out, momentum=m)
            assert e.value.code == D.EINVAL
    assert torch.equal(out2, out) and torch.equal(m2, m) and out.any()


def momentum_of(x, m, mu, nesterov):
    """(u, the new momentum) in 64 bits on the device."""
    m = float(np.float32(mu)) * m + x.double()
    return (x.double() + float(np.float32(mu)) * m if nesterov else m), m


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,rows,cols", [(2, 256, 512), (2, 512, 1024), (2, 512, 264), (1, 2048, 2048), (2, 1024, 4096), (2, 300, 501), (2, 501, 300)])
def test_momentum_over_steps_in_every_form(batch, rows, cols, dtype, nesterov):
    """Updates too large for one cluster: by chunks and by elements, wide and tall.  Each step adds two roundings of
    values below 16 to the momentum, 2^-21 each at most."""
    g = gen(rows + cols)
    m = torch.zeros(batch, rows, cols, device="cuda")
    want_m = m.double()
    out = torch.zeros(batch, rows, cols, dtype=torch.bfloat16, device="cuda")
    with D.Orthogonalizer(rows, cols, batch=batch, dtype=dtype, mu=0.95, nesterov=nesterov) as op:
        for step in range(3):
            x = torch.randn(batch, rows, cols, generator=g, device="cuda").to(TYPES[dtype])
            op.run(x, out, momentum=m)
            assert op.errors == 0
            u, want_m = momentum_of(x, want_m, 0.95, nesterov)
            assert want_m.abs().max() < 16
            assert (m.double() - want_m).abs().max() <= 2 * (step + 1) * 2.0 ** -21
            for i in range(batch):
                want = orthogonalized(u[i])
                assert float((out[i].double() - want).norm() / want.norm()) < ORTHO_TOL


def modelled(u, terms, steps=5):
    """The arithmetic that dtt_ops.h describes, in 64 bits but for the roundings it names: X in two f16 halves, the
    products' operands in f16, b A + c A A in one or two f16 terms, the result in bf16."""
    def f16(x):
        return x.to(torch.float16).double()

    def halves(x):
        x = x.float().double()
        return f16(x), f16((x - f16(x)) * 2048) / 2048

    a, b, c = COEFFS
    hi, lo = halves(u.double() / (u.double().norm() + 1e-7))
    for _ in range(steps):
        gram = f16(hi @ hi.T)
        poly = (b * gram + c * (gram @ gram)).float().double()
        operand = f16(poly)
        if terms == 2:
            operand = operand + f16(poly - operand)
        x = a * (hi + lo) + operand @ hi
        hi, lo = halves(x)
    return x.float().to(torch.bfloat16).double()


@pytest.mark.parametrize("terms,rows,cols", [(2, 96, 160), (2, 128, 512), (2, 128, 2048), (2, 200, 1000), (2, 256, 512), (1, 512, 512), (1, 520, 1032),
                                             (1, 1024, 2048), (1, 2048, 2048)])
def test_the_error_is_that_of_the_documented_roundings(terms, rows, cols):
    """Against 64 bits, no further off than a model with those roundings alone; one f16 term where there are two would
    be 1.12 to 1.18 times as far off.  Beside them are the f32 sums' errors, 2^-11 of the f16 operands': 8 % is for
    the rounding errors that fall otherwise."""
    u = torch.randn(rows, cols, generator=gen(cols), device="cuda")
    out = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    with D.Orthogonalizer(rows, cols, dtype="f32") as op:
        op.run(u, out)
        assert op.errors == 0
    want = orthogonalized(u)
    error, model = (float((t - want).norm() / want.norm()) for t in (out.double(), modelled(u, terms)))
    assert 1.6e-3 < model < 2.7e-3              # bf16's own is 1.66e-3
    assert error < 1.08 * model


@pytest.mark.parametrize("batch,rows,cols", [f for f in FORMS if f[0] > 1])
def test_huge_tiny_and_infinite_updates(batch, rows, cols):
    """A sum of squares beyond f32: zeros.  Far below eps: zeros.  An infinity: NaN.  The other matrices as ever, and
    the same for 1e15 and 1e-5 times an update."""
    g = gen(cols)
    u = torch.randn(rows, cols, generator=g, device="cuda")
    x = torch.stack([u] + [torch.randn(rows, cols, generator=g, device="cuda") for _ in range(batch - 1)])
    want = [orthogonalized(t) for t in x]
    out = torch.zeros(batch, rows, cols, dtype=torch.bfloat16, device="cuda")
    with D.Orthogonalizer(rows, cols, batch=batch, dtype="f32") as op:
        for value in ("huge", "tiny", "infinite", 2.0 ** 50, 2.0 ** -3):
            x[0] = u * {"huge": 1e19, "tiny": 1e-22, "infinite": 1.0}.get(value, value)
            if value == "infinite":
                x[0, rows // 2, cols // 3] = float("inf")
            out.fill_(7)
            op.run(x, out)
            assert op.errors == 0
            if value in ("huge", "tiny"):
                assert not out[0].any()
            elif value == "infinite":
                assert torch.isnan(out[0]).all()
            else:
                assert float((out[0].double() - want[0]).norm() / want[0].norm()) < ORTHO_TOL
            for i in range(1, batch):
                assert float((out[i].double() - want[i]).norm() / want[i].norm()) < ORTHO_TOL


# ---- streams ---------------------------------------------------------------------------------------
def test_a_workspace_is_not_given_away_while_a_call_on_the_default_stream_may_use_it():
    """Built under a side stream, used on the default one and dropped while that call waits: the side stream's
    next allocation of the size is another block."""
    s = torch.cuda.Stream()
    x = torch.randn(300, 500, generator=gen(1), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        op = D.Orthogonalizer(300, 500)
        address, size = op._workspace.address, op._workspace.buffer.numel()
    op.run(x, out)                              # the default stream; kernels loaded
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)              # some 0.2 s
    op.run(x, out)
    op.close()
    del op
    with torch.cuda.stream(s):
        other = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert other.data_ptr() != address
    torch.cuda.synchronize()
    want = orthogonalized(x)
    assert float((out.double() - want).norm() / want.norm()) < ORTHO_TOL


# ---- rows that do not arrive -------------------------------------------------------------------------
def library_with(source, defines, tmp):
    """The library, beside the one under test, with one source built for late arrivals."""
    import ctypes as C
    import os
    import subprocess
    from device_triggered_transfers_gb300 import build as B
    obj, lib = os.path.join(tmp, "late.o"), os.path.join(tmp, "libdtt_late.so")
    subprocess.run([B.nvcc(), *B.ARCH, *B.COMMON, *defines, "-c", os.path.join(B.CSRC, source), "-o", obj], check=True)
    others = [os.path.join(B.OBJ, f + ".o") for f in B.sources() if f != source]
    subprocess.run([B.nvcc(), *B.ARCH, "-shared", "-Xcompiler", "-fPIC", obj, *others, "-o", lib], check=True)
    L = C.CDLL(lib)
    for name, (restype, argtypes) in D._SIGS.items():
        getattr(L, name).restype, getattr(L, name).argtypes = restype, argtypes
    return L


@pytest.mark.parametrize("late", ["true", "r % 5 == 3", "r % 5 == 3 && t == 37"])
def test_rows_that_do_not_arrive_in_time_are_nan_and_so_is_the_weight_s_gradient(late, tmp_path):
    """Every value is right or NaN, never something else, whether all threads give up, at once or in the middle, or one
    of them does (thread t gives up row r where `late` says so); the CTAs wait for their copies before they leave."""
    L = library_with("norm.cu", [f"-DDTT_NORM_ROW_LATE=({late})"], str(tmp_path))
    for rows, cols, pad, kind in ((2000, 1024, 0, "bf16"), (1000, 4096, 0, "bf16"), (400, 12288, 0, "bf16"), (1300, 1001, 0, "f32"), (1300, 3001, 3, "f32")):
        g = gen(rows)
        x, res, dres = (slab(rows, cols, pad, lambda *s: torch.randn(*s, generator=g, device="cuda"), kind) for _ in range(3))
        w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(TYPES[kind])
        got = []
        for other in (False, True):
            op = D.RMSNorm(cols, x=kind, residual=kind, weight=kind, y=kind)
            back = D.RMSNorm(cols, x=kind, residual=kind, weight=kind)
            if other:
                op._forward, back._backward = L.dtt_rmsnorm_forward, L.dtt_rmsnorm_backward
            y, h, dx = (slab(rows, cols, pad, lambda *s: torch.full(s, 7.0, device="cuda"), kind) for _ in range(3))
            rstd, dw = torch.full((rows,), 7.0, device="cuda"), torch.full((cols,), 7.0, device="cuda")
            op.forward(x, w, y, residual=res, residual_out=h, rstd=rstd)
            back.backward(x, res, w, (x.float() + res.float()).square().mean(-1).rsqrt(), dx, dw, dres=dres)
            torch.cuda.synchronize()
            got.append((y, h, rstd, dx, dw))
        for right, seen in zip(*got):
            assert not torch.isnan(right).any()
            gone = torch.isnan(seen)
            assert gone.all() if late == "true" else (gone | (seen == right)).all()
        y, h, rstd, dx, dw = got[1]
        assert torch.isnan(rstd[3::5]).all() and torch.isnan(h[3::5]).any(-1).all() and torch.isnan(dx[3::5]).all()
        assert torch.equal(torch.isnan(rstd), torch.isnan(y).all(-1)) and torch.equal(torch.isnan(rstd), torch.isnan(y).any(-1))
        assert torch.equal(torch.isnan(dx).any(-1), torch.isnan(dx).all(-1)) and torch.isnan(dw).any()


def test_an_orthogonalisation_that_gives_up_its_waits_counts_an_error_and_ends(tmp_path, monkeypatch):
    """CTAs that give up at once, and others that wait in vain for them for 16 ms: all end soon, the error word says
    so, and the GPU does the next call as ever.  One cluster of 1, 4 and 16 CTAs, the second product within the
    third, a product a launch."""
    import time
    L = library_with("ortho.cu", ["-DDTT_ORTHO_LATE=(blockIdx.x == 0 || blockIdx.x == 5)", "-DDTT_ORTHO_WAIT_LIMIT=4096u"], str(tmp_path))
    for batch, rows, cols in ((3, 64, 64), (2, 100, 600), (1, 128, 4096), (1, 256, 512), (1, 1000, 200), (1, 512, 512)):
        x = torch.randn(batch, rows, cols, generator=gen(rows), device="cuda").to(torch.bfloat16)
        out = torch.zeros(batch, rows, cols, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        with monkeypatch.context() as m:
            m.setattr(D, "lib", lambda: L)
            with D.Orthogonalizer(rows, cols, batch=batch) as op:
                began = time.time()
                op.run(x, out)
                assert op.errors > 0 and time.time() - began < 5
        with D.Orthogonalizer(rows, cols, batch=batch) as op:
            op.run(x, out)
            assert op.errors == 0
        for i in range(batch):
            want = orthogonalized(x[i])
            assert float((out[i].double() - want).norm() / want.norm()) < ORTHO_TOL


# ---- the backward pass's first call ------------------------------------------------------------------
def gradients(rows, cols, seed=3):
    g = gen(seed)
    x, h, dx = (torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(torch.bfloat16)
    return dict(dy=x, h=h, weight=w, rstd=h.float().square().mean(-1).rsqrt(), dx=dx), torch.full((cols,), 7.0, device="cuda")


@pytest.mark.parametrize("rows", [40, 500])
def test_an_object_s_first_backward_pass_may_be_captured(rows):
    cols = 1000
    a, dw = gradients(rows, cols)
    D.RMSNorm(cols).backward(**a, dweight=dw)
    want, want_dx = dw.clone(), a["dx"].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    op, graph = D.RMSNorm(cols), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        op.backward(**a, dweight=dw, stream=s)
    dw.zero_()
    a["dx"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dw, want) and torch.equal(a["dx"], want_dx)
    # later calls outside the graph, on other streams
    other = torch.cuda.Stream()
    for stream in (None, other, other.cuda_stream):
        dw.zero_()
        torch.cuda.synchronize()
        op.backward(**a, dweight=dw, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(dw, want)


def test_an_object_s_first_backward_pass_does_not_wait_for_its_stream():
    rows, cols = 500, 1000
    a, dw = gradients(rows, cols)
    op, s, done = D.RMSNorm(cols), torch.cuda.Stream(), torch.cuda.Event()
    D.RMSNorm(cols).backward(**a, dweight=dw)
    want = dw.clone()
    with torch.cuda.stream(s):
        torch.empty(op.workspace_bytes, dtype=torch.uint8, device="cuda")     # the stream's pool has the room now
        torch.cuda.synchronize()
        torch.cuda._sleep(400_000_000)
        done.record()
        op.backward(**a, dweight=dw, stream=s)
        assert not done.query()
    torch.cuda.synchronize()
    assert torch.equal(dw, want)


# ---- the error word ----------------------------------------------------------------------------------
def test_errors_waits_for_the_last_call_whatever_its_stream():
    x = torch.randn(64, 64, generator=gen(1), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        with D.Orthogonalizer(64, 64) as op:
            assert op.errors == 0
            op.run(x, out, stream=stream)
            torch.cuda.synchronize()
            with torch.cuda.stream(torch.cuda.default_stream() if stream is None else side):
                torch.cuda._sleep(200_000_000)
                op._err.fill_(3)                # as if the call had counted, late
            with torch.cuda.stream(torch.cuda.Stream()):
                assert op.errors == 3


# ---- nothing beside the outputs ----------------------------------------------------------------------
def guarded(rows, cols, kind, aligned):
    """(a buffer full of sevens, its rows x cols in the middle: 16-byte aligned or not at all)"""
    left, right = (16, 16) if aligned else (3, 4)
    wide = torch.full((rows + 2, left + cols + right), 7.0, device="cuda").to(TYPES[kind])
    return wide, wide[1:rows + 1, left:left + cols]


def untouched(wide, view):
    """Whether everything of the buffer but the view is still sevens (the view is overwritten with them)."""
    view.view(torch.uint8 if view.dtype == TYPES["e4m3"] else view.dtype).copy_(
        torch.full(view.shape, 7.0, device="cuda").to(view.dtype).view(torch.uint8 if view.dtype == TYPES["e4m3"] else view.dtype))
    return bool((wide.float() == 7).all())


@pytest.mark.parametrize("rows,cols,group,pad", FORWARD + [(40, 136, 64, 0), (700, 264, 128, 0), (33, 1001, 32, 1), (1300, 101, 0, 1), (1217, 4001, 64, 1), (5, 9001, 128, 1)])
def test_outputs_are_written_exactly(rows, cols, group, pad):
    g = gen(rows)
    for y, residual in (("e4m3", "bf16"), ("bf16", "f32"), ("f32", "bf16")):
        x, res = (torch.randn(rows, cols, generator=g, device="cuda").to(TYPES[k]) for k in ("bf16", residual))
        (wy, vy), (wr, vr) = guarded(rows, cols, y, not pad), guarded(rows, cols, residual, not pad)
        op = D.RMSNorm(cols, x="bf16", residual=residual, y=y, group=group if y == "e4m3" else 0)
        count = rows * op.scale_cols
        ws, wd = torch.full((count + 8,), 7.0, device="cuda"), torch.full((rows + 8,), 7.0, device="cuda")
        op.forward(x, None, vy, residual=res, residual_out=vr, scales=ws[4:4 + count] if y == "e4m3" else None, rstd=wd[4:4 + rows])
        torch.cuda.synchronize()
        h = x.float() + res.float()
        assert torch.equal(vr, h.to(TYPES[residual])) and (wd[4:4 + rows] != 7).all()
        assert untouched(wy, vy) and untouched(wr, vr)
        for w, n in ((ws, count if y == "e4m3" else 0), (wd, rows)):
            assert (w[:4] == 7).all() and (w[4 + n:] == 7).all()
        # and the gradient
        dy, dres = (torch.randn(rows, cols, generator=g, device="cuda").to(TYPES[k]) for k in ("bf16", residual))
        rstd = h.square().mean(-1).rsqrt()
        wx, vx = guarded(rows, cols, residual, not pad)
        plain = torch.zeros(rows, cols, device="cuda").to(TYPES[residual])
        weight = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
        back = D.RMSNorm(cols, x="bf16", residual=residual)
        dws = [torch.full((cols + 8,), 7.0, device="cuda") for _ in range(2)]
        back.backward(dy, res, weight, rstd, vx, dws[0][4:4 + cols], dres=dres)
        back.backward(dy, res, weight, rstd, plain, dws[1][4:4 + cols], dres=dres)
        torch.cuda.synchronize()
        assert (vx.float() - plain.float()).abs().max() <= 2.0 ** -6 * plain.float().abs().max()     # other forms round otherwise
        assert untouched(wx, vx)
        for dw in dws:
            assert (dw[:4] == 7).all() and (dw[4 + cols:] == 7).all() and (dw[4:4 + cols] != 7).all()


# ---- one after the other ------------------------------------------------------------------------------
def test_calls_that_read_what_the_call_before_wrote_need_no_wait_between_them():
    """Launches begin before the one before them has ended.  Two norms, the gradient and an orthogonalisation of it on
    one stream, new values every time, against the same with the GPU idle between any two."""
    rows, cols = 1536, 1024
    kinds = dict(x="bf16", residual="bf16")
    first, second, back = D.RMSNorm(cols, **kinds), D.RMSNorm(cols, y="f32", **kinds), D.RMSNorm(cols, **kinds)
    ortho = [D.Orthogonalizer(rows // n, cols // n, batch=n * n, mu=0.9, nesterov=True) for n in (1, 4, 8)]
    s = torch.cuda.Stream()
    n_rounds = 25
    g = gen(5)
    inputs = [torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16) for _ in range(n_rounds)]
    weight = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(torch.bfloat16)

    def chain(wait):
        def done():
            if wait:
                torch.cuda.synchronize()
        x, h, y, dx = (torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(4))
        z, dw, rstd = torch.zeros(rows, cols, device="cuda"), torch.zeros(cols, device="cuda"), torch.zeros(rows, device="cuda")
        moms = [torch.zeros(rows * cols, device="cuda") for _ in ortho]
        outs = [torch.zeros(rows * cols, dtype=torch.bfloat16, device="cuda") for _ in ortho]
        kept = [[torch.zeros_like(t) for _ in range(n_rounds)] for t in (z, dx, dw, *outs)]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for k in range(n_rounds):
                x.copy_(inputs[k])
                done()
                first.forward(x, weight, y, residual=h, residual_out=h, stream=s)
                done()
                second.forward(y, weight, z, residual=h, residual_out=h, rstd=rstd, stream=s)
                done()
                back.backward(y, h, weight, rstd, dx, dw, stream=s)
                done()
                for op, m, o in zip(ortho, moms, outs):
                    shape = (op.batch, op.rows, op.cols)
                    op.run(dx.view(shape), o.view(shape), momentum=m.view(shape), stream=s)
                    done()
                first.forward(outs[0].view(rows, cols), weight, y, residual=h, residual_out=h, stream=s)
                done()
                back.backward(outs[1].view(rows, cols), h, weight, rstd, dx, dw, dres=dx, stream=s)
                done()
                for t, keep in zip((z, dx, dw, *outs), kept):
                    keep[k].copy_(t)
                done()
        torch.cuda.synchronize()
        return kept

    for fast, slow in zip(chain(False), chain(True)):
        for k in range(n_rounds):
            assert torch.equal(fast[k], slow[k]) and slow[k].any()
    for op in ortho:
        assert op.errors == 0
        op.close()


# ---- beyond four gigabytes -----------------------------------------------------------------------------
# aligned rows of a ring, short rows, rows of single elements in a ring; then few rows very far apart
@pytest.mark.parametrize("rows,cols,apart", [(600000, 4096, 0), (20_000_000, 128, 0), (600000, 4001, 0), (40, 4096, 60_000_000), (40, 1001, 60_000_001),
                                             (200, 1001, 12_000_001), (40, 40000, 60_000_000)])
def test_offsets_past_32_bits(rows, cols, apart):
    """More than 4 GB from the first to the last row: the last rows' values, zeros elsewhere."""
    def big(fill=0.0):
        if not apart:
            return torch.full((rows, cols), fill, dtype=torch.bfloat16, device="cuda")
        return torch.full((rows * apart,), fill, dtype=torch.bfloat16, device="cuda").as_strided((rows, cols), (apart, 1))

    g = gen(cols)
    small = {k: torch.randn(3, cols, generator=g, device="cuda").to(torch.bfloat16) for k in ("x", "res", "dres")}
    x, y = big(), big(7.0)
    x[-3:] = small["x"]
    rstd = torch.zeros(rows, device="cuda")
    weight = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(torch.bfloat16)
    op = D.RMSNorm(cols, eps=1e-5)
    op.forward(x, weight, y, rstd=rstd)
    torch.cuda.synchronize()
    h = small["x"].double()
    s = (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    want = h * s * weight.double()
    assert ((y[-3:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-30).all() and not y[:-3].any()
    assert ((rstd[-3:, None].double() - s).abs() <= 2e-6 * s).all()
    del y
    dx, dw = big(7.0), torch.zeros(cols, device="cuda")
    op.backward(x, x, weight, rstd, dx, dw, dres=x)
    torch.cuda.synchronize()
    s = rstd[-3:, None].double()
    n, gr = h * s, h * weight.double()
    want = s * (gr - n * (gr * n).mean(-1, keepdim=True)) + h
    # bf16's half spacing and 50 f32 roundings of terms below 100
    assert ((dx[-3:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 100 * 50 * 2.0 ** -24).all() and not dx[:-3].any()
    assert ((dw.double() - (h * n).sum(0)).abs() <= 500 * 2.0 ** -24 * (h * n).abs().sum(0) + 1e-30).all()


@pytest.mark.parametrize("batch,rows,cols", [(3, 96, 160), (3, 300, 512), (3, 301, 511), (3, 512, 300), (1, 1536, 1600)])
def test_matrices_past_32_bits(batch, rows, cols):
    """Matrices, or rows, more than 4 GB apart."""
    strides = (1_200_000_000, cols, 1) if batch > 1 else (0, 1_000_000, 1)
    size = (batch - 1) * strides[0] + (rows - 1) * strides[1] + cols
    x, m = (torch.zeros(size, device="cuda").as_strided((batch, rows, cols), strides) for _ in range(2))
    out = torch.zeros(size, dtype=torch.bfloat16, device="cuda").as_strided((batch, rows, cols), strides)
    x.copy_(torch.randn(batch, rows, cols, generator=gen(rows), device="cuda"))
    with D.Orthogonalizer(rows, cols, batch=batch, dtype="f32", mu=0.9, nesterov=True) as op:
        op.run(x, out, momentum=m)
        assert op.errors == 0
    assert torch.equal(m, x)
    for i in range(batch):
        want = orthogonalized(1.9 * x[i].double())
        assert float((out[i].double() - want).norm() / want.norm()) < ORTHO_TOL
