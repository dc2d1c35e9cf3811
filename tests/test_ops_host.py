"""What the operators of include/dtt_ops.h refuse, checked in the library before anything is launched
(no GPU needed), and their workspaces' sizes."""
import ctypes as C

import pytest

from conftest import ensure_built

ensure_built()

import device_triggered_transfers_gb300 as D  # noqa: E402

NAN, INF = float("nan"), float("inf")


def norm_desc(**over):
    d = D.dtt_rmsnorm_desc(D.BF16, D.BF16, D.BF16, D.BF16, 0, 1e-6, 64)
    for k, v in over.items():
        setattr(d, k, v)
    return d


def ortho_desc(**over):
    d = D.dtt_ortho_desc()
    d.x_dtype, d.batch, d.rows, d.cols, d.steps, d.eps, d.scale = D.BF16, 1, 64, 100, 2, 1e-7, 1.0
    for k in range(D.ORTHO_MAX_STEPS):
        d.coeffs[k][:] = (3.4445, -4.7750, 2.0315)
    for k, v in over.items():
        if k == "coeffs":
            d.coeffs[0][:] = v
        else:
            setattr(d, k, v)
    return d


@pytest.mark.parametrize("over", [dict(x_dtype=D.U8), dict(x_dtype=D.E4M3), dict(residual_dtype=D.U8),
                                  dict(weight_dtype=7), dict(y_dtype=D.U8), dict(group=128),
                                  dict(y_dtype=D.E4M3, group=16), dict(y_dtype=D.E4M3, group=256), dict(eps=-1e-9),
                                  dict(eps=NAN), dict(eps=INF), dict(cols=0), dict(cols=(1 << 24) + 1)])
def test_norm_refuses_a_bad_desc(over):
    n, d = C.c_uint64(), norm_desc(**over)
    L = D.lib()
    assert L.dtt_rmsnorm_workspace(C.byref(d), C.byref(n)) == D.EINVAL
    assert L.dtt_rmsnorm_forward(C.byref(d), 1, 256, 128, 0, 0, 0, 0, 0, 512, 128, 0, 0, 0) == D.EINVAL
    assert L.dtt_rmsnorm_backward(C.byref(d), 1, 256, 128, 512, 128, 0, 1024, 0, 0, 2048, 128, 0, 0, 0, 0) == D.EINVAL
    assert L.dtt_last_error()


FWD = dict(rows=2, x=256, x_pitch=128, residual=512, residual_pitch=128, weight=1024, residual_out=2048,
           residual_out_pitch=128, y=4096, y_pitch=128, scales=0, rstd=8192)


@pytest.mark.parametrize("over", [dict(rows=1 << 31), dict(x=0), dict(y=0), dict(x=257), dict(x_pitch=126), dict(x_pitch=129),
                                  dict(residual=513), dict(residual_pitch=0), dict(weight=1025),
                                  dict(residual_out=2049), dict(y_pitch=64), dict(rstd=8193), dict(scales=16384),
                                  dict(residual_out=512, residual_out_pitch=256)])
def test_forward_refuses(over):
    a = dict(FWD, **over)
    d = norm_desc()
    assert D.lib().dtt_rmsnorm_forward(C.byref(d), *a.values(), 0) == D.EINVAL


def test_forward_needs_scales_for_8_bits():
    d = norm_desc(y_dtype=D.E4M3)
    assert D.lib().dtt_rmsnorm_forward(C.byref(d), *dict(FWD, y_pitch=64).values(), 0) == D.EINVAL


BWD = dict(rows=2, dy=256, dy_pitch=128, h=512, h_pitch=128, weight=1024, rstd=2048, dres=4096, dres_pitch=128,
           dx=8192, dx_pitch=128, dweight=16384, workspace=32768, workspace_bytes=1 << 40)


@pytest.mark.parametrize("over", [dict(rows=1 << 31), dict(dy=0), dict(h=0), dict(rstd=0), dict(dx=0), dict(dy=257), dict(h=513),
                                  dict(dres=4097), dict(dx=8193), dict(dy_pitch=2), dict(dx_pitch=127), dict(weight=0),
                                  dict(weight=1), dict(dweight=16386), dict(workspace=0), dict(workspace=32776),
                                  dict(workspace_bytes=64), dict(dx=4096, dx_pitch=256)])
def test_backward_refuses(over):
    a = dict(BWD, **over)
    d = norm_desc()
    assert D.lib().dtt_rmsnorm_backward(C.byref(d), *a.values(), 0) == D.EINVAL


def test_no_rows_is_no_work():
    d = norm_desc()
    assert D.lib().dtt_rmsnorm_forward(C.byref(d), 0, *[0] * 12) == D.OK
    assert D.lib().dtt_rmsnorm_backward(C.byref(d), 0, *[0] * 14) == D.OK


@pytest.mark.parametrize("over", [dict(x_dtype=D.U8), dict(x_dtype=D.E4M3), dict(batch=0), dict(batch=65536), dict(rows=0), dict(cols=0),
                                  dict(rows=65537), dict(cols=65537), dict(steps=0), dict(steps=33),
                                  dict(rows=65536, cols=65536, batch=65535),
                                  dict(momentum=2), dict(nesterov=1), dict(momentum=1, nesterov=2), dict(mu=NAN),
                                  dict(scale=INF), dict(eps=0.0), dict(eps=NAN), dict(coeffs=(NAN, 0, 0)),
                                  dict(coeffs=(17.0, 0, 0)), dict(coeffs=(0, 2000.0, 0))])
def test_ortho_refuses_a_bad_desc(over):
    n, d, out = C.c_uint64(), ortho_desc(**over), C.c_void_p()
    L = D.lib()
    assert L.dtt_ortho_workspace(C.byref(d), C.byref(n)) == D.EINVAL
    assert L.dtt_ortho_create(C.byref(d), 256, 1 << 60, C.byref(out)) == D.EINVAL and not out.value
    assert L.dtt_last_error()


def test_ortho_refuses_a_bad_workspace():
    d, n, out = ortho_desc(), C.c_uint64(), C.c_void_p()
    L = D.lib()
    assert L.dtt_ortho_workspace(C.byref(d), C.byref(n)) == D.OK and n.value > 64 * 128 * 8
    for ws, size in ((0, n.value), (128, n.value), (256, n.value - 1)):
        assert L.dtt_ortho_create(C.byref(d), ws, size, C.byref(out)) == D.EINVAL and not out.value
    assert L.dtt_ortho_run(None, 256, 200, 0, None, 0, 0, 512, 200, 0, 256, None) == D.EINVAL
    L.dtt_ortho_destroy(None)


def test_workspaces_follow_the_sizes():
    n = C.c_uint64()
    D._check(D.lib().dtt_rmsnorm_workspace(C.byref(norm_desc(cols=100)), C.byref(n)))
    one = n.value
    D._check(D.lib().dtt_rmsnorm_workspace(C.byref(norm_desc(cols=200)), C.byref(n)))
    assert n.value == 2 * one > 0
    D._check(D.lib().dtt_ortho_workspace(C.byref(ortho_desc()), C.byref(n)))
    one = n.value
    D._check(D.lib().dtt_ortho_workspace(C.byref(ortho_desc(rows=100, cols=64)), C.byref(n)))
    assert n.value == one                       # the smaller side comes first either way
    D._check(D.lib().dtt_ortho_workspace(C.byref(ortho_desc(batch=3)), C.byref(n)))
    assert n.value > one


def test_binding_refuses_names_and_step_lists():
    for bad in (lambda: D.RMSNorm(64, x="f16"), lambda: D.RMSNorm(64, y="u8"), lambda: D.RMSNorm(64, x="e4m3"),
                lambda: D.RMSNorm(64, group=32)):
        with pytest.raises(D.DttError) as e:
            bad()
        assert e.value.code == D.EINVAL
