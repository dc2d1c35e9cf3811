"""What the layer norm, the expert rows and AdamW refuse, checked in the library before anything is launched (no GPU
needed), and their workspaces' sizes."""
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


FWD = dict(rows=2, x=256, x_pitch=128, residual=512, residual_pitch=128, weight=1024, bias=1280, residual_out=2048,
           residual_out_pitch=128, y=4096, y_pitch=128, scales=0, mean=16384, rstd=8192)


@pytest.mark.parametrize("over", [dict(rows=1 << 31), dict(x=0), dict(y=0), dict(x=257), dict(x_pitch=126), dict(x_pitch=129), dict(residual=513),
                                  dict(residual_pitch=0), dict(weight=1025), dict(bias=1281), dict(residual_out=2049), dict(y_pitch=64),
                                  dict(mean=16386), dict(rstd=8193), dict(scales=16384), dict(residual_out=512, residual_out_pitch=256)])
def test_layer_norm_s_forward_refuses(over):
    d = norm_desc()
    assert D.lib().dtt_layernorm_forward(C.byref(d), *dict(FWD, **over).values(), 0) == D.EINVAL
    assert b"layernorm" in D.lib().dtt_last_error()


BWD = dict(rows=2, dy=256, dy_pitch=128, h=512, h_pitch=128, weight=1024, mean=1536, rstd=2048, dres=4096, dres_pitch=128,
           dx=8192, dx_pitch=128, dweight=16384, dbias=65536, workspace=32768, workspace_bytes=1 << 40)


@pytest.mark.parametrize("over", [dict(rows=1 << 31), dict(dy=0), dict(h=0), dict(mean=0), dict(mean=1538), dict(rstd=0), dict(dx=0), dict(dy=257),
                                  dict(dres=4097), dict(dx=8193), dict(dy_pitch=2), dict(dx_pitch=127), dict(weight=0), dict(dweight=16386),
                                  dict(dbias=65538), dict(workspace=0), dict(workspace=32776), dict(workspace_bytes=64),
                                  dict(dweight=0, workspace=0), dict(dbias=0, workspace_bytes=64), dict(dx=4096, dx_pitch=256)])
def test_layer_norm_s_backward_refuses(over):
    d = norm_desc()
    assert D.lib().dtt_layernorm_backward(C.byref(d), *dict(BWD, **over).values(), 0) == D.EINVAL


def test_layer_norm_refuses_a_bad_desc_and_takes_no_rows():
    n, L = C.c_uint64(), D.lib()
    for over in (dict(x_dtype=D.U8), dict(weight_dtype=D.E4M3), dict(group=128), dict(eps=-1.0), dict(eps=NAN), dict(cols=0), dict(cols=(1 << 24) + 1)):
        d = norm_desc(**over)
        assert L.dtt_layernorm_workspace(C.byref(d), C.byref(n)) == D.EINVAL
        assert L.dtt_layernorm_forward(C.byref(d), *FWD.values(), 0) == D.EINVAL
        assert L.dtt_layernorm_backward(C.byref(d), *BWD.values(), 0) == D.EINVAL
    assert L.dtt_layernorm_forward(None, *FWD.values(), 0) == D.EINVAL
    assert L.dtt_layernorm_backward(None, *BWD.values(), 0) == D.EINVAL
    d = norm_desc()
    assert L.dtt_layernorm_forward(C.byref(d), 0, *[0] * 14) == D.OK
    assert L.dtt_layernorm_backward(C.byref(d), 0, *[0] * 16) == D.OK
    one = C.c_uint64()
    assert L.dtt_layernorm_workspace(C.byref(d), C.byref(n)) == D.OK == L.dtt_rmsnorm_workspace(C.byref(d), C.byref(one))
    assert n.value == 2 * one.value > 0


# ---- expert rows ----------------------------------------------------------------------------------
def experts_desc(**over):
    d = D.dtt_experts_desc(8, 0, 2, 4)
    for k, v in over.items():
        setattr(d, k, v)
    return d


ROUTE = dict(tokens=3, ids=256, id_bytes=4, max_rows=64, position=512, offsets=1024, counts=2048, workspace=4096, workspace_bytes=1 << 30)
DISPATCH = dict(tokens=3, position=512, offsets=1024, counts=2048, x=4096, x_pitch=128, row_bytes=128, rows=8192, rows_pitch=128,
                max_rows=64, scales=0, scales_pitch=0, scale_count=0, row_scales=0, row_scales_pitch=0)
COMBINE = dict(tokens=3, cols=64, position=512, rows=8192, rows_dtype=D.BF16, rows_pitch=128, max_rows=64, weights=1024, out=4096,
               out_dtype=D.BF16, out_pitch=128)
BACKWARD = dict(tokens=3, cols=64, position=512, offsets=1024, counts=2048, dout=4096, dout_dtype=D.BF16, dout_pitch=128, rows=8192,
                rows_dtype=D.BF16, rows_pitch=128, max_rows=64, weights=16384, drows=32768, drows_pitch=128, dweights=65536)
SCALED = dict(scales=256, scales_pitch=16, scale_count=4, row_scales=640, row_scales_pitch=16)


@pytest.mark.parametrize("over", [dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=33), dict(align=0), dict(align=65537), dict(first=1 << 31)])
def test_expert_rows_refuse_a_bad_desc(over):
    d, n, L = experts_desc(**over), C.c_uint64(), D.lib()
    assert L.dtt_experts_workspace(C.byref(d), C.byref(n)) == D.EINVAL
    assert L.dtt_experts_route(C.byref(d), *ROUTE.values(), 0) == D.EINVAL
    assert L.dtt_experts_dispatch(C.byref(d), *DISPATCH.values(), 0) == D.EINVAL
    assert L.dtt_experts_combine(C.byref(d), *COMBINE.values(), 0) == D.EINVAL
    assert L.dtt_experts_combine_backward(C.byref(d), *BACKWARD.values(), 0) == D.EINVAL


@pytest.mark.parametrize("over", [dict(tokens=1 << 30), dict(max_rows=1 << 31), dict(id_bytes=2), dict(ids=0), dict(ids=258), dict(ids=260, id_bytes=8),
                                  dict(position=0), dict(position=514), dict(offsets=0), dict(offsets=1026), dict(counts=0), dict(counts=2049),
                                  dict(workspace=0), dict(workspace=4104), dict(workspace_bytes=64 * 8 * 4 - 1)])
def test_route_refuses(over):
    assert D.lib().dtt_experts_route(C.byref(experts_desc()), *dict(ROUTE, **over).values(), 0) == D.EINVAL


@pytest.mark.parametrize("over", [dict(tokens=1 << 30), dict(max_rows=1 << 31), dict(row_bytes=0), dict(row_bytes=(1 << 26) + 1), dict(position=0), dict(offsets=0),
                                  dict(counts=0), dict(x=0), dict(rows=0), dict(x_pitch=127), dict(rows_pitch=64), dict(scales=256),
                                  dict(row_scales=256), dict(SCALED, scale_count=0), dict(SCALED, scales=258), dict(SCALED, scales_pitch=12),
                                  dict(SCALED, row_scales_pitch=18), dict(SCALED, row_scales_pitch=12), dict(SCALED, scale_count=(1 << 24) + 1)])
def test_dispatch_refuses(over):
    assert D.lib().dtt_experts_dispatch(C.byref(experts_desc()), *dict(DISPATCH, **over).values(), 0) == D.EINVAL


@pytest.mark.parametrize("over", [dict(tokens=1 << 30), dict(cols=0), dict(cols=(1 << 24) + 1), dict(rows_dtype=D.E4M3), dict(out_dtype=D.U8), dict(position=0),
                                  dict(rows=0), dict(rows=8193), dict(rows_pitch=126), dict(rows_pitch=129), dict(weights=1026), dict(out=0),
                                  dict(out_pitch=126), dict(out_dtype=D.F32), dict(out=4097)])
def test_combine_refuses(over):
    assert D.lib().dtt_experts_combine(C.byref(experts_desc()), *dict(COMBINE, **over).values(), 0) == D.EINVAL


@pytest.mark.parametrize("over", [dict(tokens=1 << 30), dict(cols=0), dict(rows_dtype=D.U8), dict(dout_dtype=D.E4M3), dict(position=0), dict(offsets=0), dict(counts=0),
                                  dict(dout=0), dict(dout=4097), dict(rows=0), dict(rows_pitch=126), dict(weights=0), dict(weights=16385),
                                  dict(drows=0), dict(drows_pitch=64), dict(drows_pitch=129), dict(dweights=65537)])
def test_combine_s_backward_refuses(over):
    assert D.lib().dtt_experts_combine_backward(C.byref(experts_desc()), *dict(BACKWARD, **over).values(), 0) == D.EINVAL


def test_expert_rows_of_nothing_are_no_work():
    d, L = experts_desc(align=1), D.lib()
    assert L.dtt_experts_dispatch(C.byref(d), 0, 0, 1024, 2048, 0, 0, 128, 8192, 128, 64, 0, 0, 0, 0, 0, 0) == D.OK
    assert L.dtt_experts_combine(C.byref(d), 0, 64, 0, 0, D.BF16, 0, 0, 0, 0, D.BF16, 0, 0) == D.OK


def test_dispatch_takes_no_tokens_and_no_rows_with_scales():
    """An empty tensor has no address; the other one of the two does."""
    d, L = experts_desc(align=1), D.lib()
    nothing = dict(tokens=0, x=0, x_pitch=0, position=0, scales=0, scales_pitch=0)
    for over in (dict(SCALED, **nothing), dict(SCALED, rows=0, rows_pitch=0, max_rows=0, row_scales=0, row_scales_pitch=0),
                 dict(SCALED, **nothing, rows=0, rows_pitch=0, max_rows=0, row_scales=0, row_scales_pitch=0)):
        assert L.dtt_experts_dispatch(C.byref(d), *dict(DISPATCH, **{**SCALED, **over}).values(), 0) == D.OK, over
    for over in (dict(SCALED, scales=0), dict(SCALED, row_scales=0), dict(SCALED, **nothing, scale_count=0)):
        assert L.dtt_experts_dispatch(C.byref(d), *dict(DISPATCH, **{**SCALED, **over}).values(), 0) == D.EINVAL, over


def test_the_sort_s_workspace_follows_the_experts():
    n = C.c_uint64()
    D._check(D.lib().dtt_experts_workspace(C.byref(experts_desc()), C.byref(n)))
    one = n.value
    D._check(D.lib().dtt_experts_workspace(C.byref(experts_desc(experts=16, top_k=32)), C.byref(n)))
    assert n.value == 2 * one > 0
    assert D.lib().dtt_experts_workspace(C.byref(experts_desc()), None) == D.EINVAL


# ---- AdamW ----------------------------------------------------------------------------------------
def adam_desc(**over):
    d = D.dtt_adamw_desc(D.F32, D.BF16, D.F32, 0, 0.9, 0.999, 1e-8, 0)
    for k, v in over.items():
        setattr(d, k, v)
    return d


def adam_tensor(**over):
    t = D.dtt_adamw_tensor(256, 512, 1024, 2048, None, None, None, 10, 0.01, 0)
    for k, v in over.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("over", [dict(param_dtype=D.E4M3), dict(grad_dtype=D.U8), dict(state_dtype=D.BF16), dict(stochastic=2), dict(beta1=1.0),
                                  dict(beta1=-0.1), dict(beta2=NAN), dict(beta2=1.5), dict(eps=0.0), dict(eps=NAN), dict(eps=INF), dict(eps=1e-31)])
def test_adamw_refuses_a_bad_desc(over):
    out = C.c_void_p()
    assert D.lib().dtt_adamw_create(C.byref(adam_desc(**over)), C.byref(adam_tensor()), 1, C.byref(out)) == D.EINVAL and not out.value


CODES = dict(m_scales=4096, v_scales=8192)


@pytest.mark.parametrize("desc,over", [
    ({}, dict(param=None)), ({}, dict(grad=None)), ({}, dict(m=None)), ({}, dict(v=None)), ({}, dict(param=258)), ({}, dict(grad=513)),
    ({}, dict(m=1026)), ({}, dict(v=2049)), ({}, dict(copy=4097)), ({}, CODES), ({}, dict(m_scales=4096)), ({}, dict(n=1 << 40)),
    ({}, dict(weight_decay=NAN)), ({}, dict(weight_decay=INF)), (dict(param_dtype=D.BF16), dict(copy=4096)),
    (dict(state_dtype=D.E4M3), {}), (dict(state_dtype=D.E4M3), dict(m_scales=4096)), (dict(state_dtype=D.E4M3), dict(CODES, m_scales=4098)),
    (dict(state_dtype=D.E4M3), dict(CODES, v_scales=8193))])
def test_adamw_refuses_a_bad_tensor(desc, over):
    """In any place of the list."""
    out, L = C.c_void_p(), D.lib()
    fine = CODES if desc.get("state_dtype") == D.E4M3 else {}
    bad = (D.dtt_adamw_tensor * 2)(adam_tensor(**fine), adam_tensor(**over))
    assert L.dtt_adamw_create(C.byref(adam_desc(**desc)), bad, 2, C.byref(out)) == D.EINVAL and not out.value
    assert b"tensor 1" in L.dtt_last_error()


@pytest.mark.parametrize("over", [dict(param=256), dict(m=1024), dict(v=1024 + 36), dict(grad=2048 + 36), dict(v=512 + 16), dict(param=1020)])
def test_adamw_refuses_buffers_that_overlap(over):
    """Ten elements: the first tensor has its param (f32) at 256, grad (bf16) at 512, m and v at 1024 and 2048."""
    out, L = C.c_void_p(), D.lib()
    apart = dict(param=1 << 16, grad=1 << 17, m=1 << 18, v=1 << 19)
    both = (D.dtt_adamw_tensor * 2)(adam_tensor(), adam_tensor(**{**apart, **over}))
    assert L.dtt_adamw_create(C.byref(adam_desc()), both, 2, C.byref(out)) == D.EINVAL and not out.value
    assert b"overlaps" in L.dtt_last_error()


def test_adamw_takes_gradients_that_overlap_and_neighbours():
    """As far as a GPU: the list is fine."""
    out, L = C.c_void_p(), D.lib()
    both = (D.dtt_adamw_tensor * 2)(adam_tensor(), adam_tensor(param=256 + 40, m=1024 + 40, v=2048 + 40))
    rc = L.dtt_adamw_create(C.byref(adam_desc()), both, 2, C.byref(out))
    assert rc == D.OK if out.value else b"overlaps" not in L.dtt_last_error()
    L.dtt_adamw_destroy(out)


def test_adamw_refuses_what_is_null():
    out, L = C.c_void_p(), D.lib()
    assert L.dtt_adamw_create(None, C.byref(adam_tensor()), 1, C.byref(out)) == D.EINVAL
    assert L.dtt_adamw_create(C.byref(adam_desc()), None, 1, C.byref(out)) == D.EINVAL
    assert L.dtt_adamw_create(C.byref(adam_desc()), C.byref(adam_tensor()), 1, None) == D.EINVAL
    assert L.dtt_adamw_run(None, None, 1e-3, 1, None, None, None, None) == D.EINVAL
    L.dtt_adamw_destroy(None)


def test_binding_refuses_names_and_sizes():
    for bad in (lambda: D.LayerNorm(64, x="f16"), lambda: D.LayerNorm(64, y="u8"), lambda: D.LayerNorm(64, group=32), lambda: D.ExpertRows(0, 1),
                lambda: D.ExpertRows(8, 0), lambda: D.ExpertRows(8, -1), lambda: D.ExpertRows(2000, 1), lambda: D.ExpertRows(8, 2, first=1 << 31),
                lambda: D.ExpertRows(8, 2, align=0), lambda: D.ExpertRows(8, 2 ** 32 + 2), lambda: D.AdamW([], [], [], [])):
        with pytest.raises(D.DttError) as e:
            bad()
        assert e.value.code == D.EINVAL
    assert D.ExpertRows(8, 2, align=4).most_rows(10) == 20 + 24 and D.AdamW.blocks(129) == 2
