"""Refusals of the dispatch, combine and 4-bit operators on the host (no GPU): every
invalid call returns its status before any HIP call, and the Python functions refuse
what the C functions cannot see."""
import pytest
import torch

import block_fp8_routed_amd as moe

P = 0x1000  # never dereferenced: validation fails, or there is nothing to do
OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE = (moe.MOE_OK, moe.MOE_ERR_NULL, moe.MOE_ERR_SHAPE,
                                           moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE)


def dispatch(x=P, ld_x=64, dtype=1, idx=P, tokens=4, hidden=64, k=2, experts=8, rows=P, ld_rows=64,
             offsets=P, pair=P, inv=P, ws=None, ws_bytes=0):
    return moe.load().moe_dispatch(x, ld_x, dtype, idx, tokens, hidden, k, experts, rows, ld_rows,
                                   offsets, pair, inv, ws, ws_bytes, None)


def dispatch_backward(d_rows=P, ld_rows=64, rows=8, dtype=1, inv=P, tokens=0, hidden=64, k=2, dx=P,
                      ld_dx=64, dx_dtype=1):
    return moe.load().moe_dispatch_backward(d_rows, ld_rows, rows, dtype, inv, tokens, hidden, k,
                                            dx, ld_dx, dx_dtype, None)


def combine(y=P, ld_y=64, rows=8, dtype=1, gates=P, inv=P, shared=None, ld_shared=0, tokens=0,
            hidden=64, k=2, out=P, ld_out=64, out_dtype=0):
    return moe.load().moe_combine(y, ld_y, rows, dtype, gates, inv, shared, ld_shared, tokens,
                                  hidden, k, out, ld_out, out_dtype, None)


def combine_backward(d_out=P, ld_d=64, d_dtype=0, y=P, ld_y=64, rows=8, dtype=1, gates=P, inv=P,
                     tokens=0, hidden=64, k=2, d_y=P, ld_dy=64, d_gates=P):
    return moe.load().moe_combine_backward(d_out, ld_d, d_dtype, y, ld_y, rows, dtype, gates, inv,
                                           tokens, hidden, k, d_y, ld_dy, d_gates, None)


def w4(x=P, ld_x=256, w=P, ws=P, st=0, wz=None, bias=None, rows=0, n=64, k=256, group=64, swiglu=0,
       out=P, ld_out=64, out_dtype=1, work=None, work_bytes=0):
    return moe.load().moe_linear_w4(x, ld_x, w, ws, st, wz, bias, rows, n, k, group, swiglu, out,
                                    ld_out, out_dtype, work, work_bytes, None)


def grouped(x=P, ld_x=256, offsets=P, w=P, ws=P, st=0, wz=None, bias=None, rows=0, experts=4, n=64,
            k=256, group=64, swiglu=0, out=P, ld_out=64, out_dtype=1, work=None, work_bytes=0):
    return moe.load().moe_grouped_linear_w4(x, ld_x, offsets, w, ws, st, wz, bias, rows, experts, n,
                                            k, group, swiglu, out, ld_out, out_dtype, work,
                                            work_bytes, None)


def test_no_rows_enqueue_nothing():
    assert [f() for f in (dispatch_backward, combine, combine_backward, w4, grouped)] == [OK] * 5


@pytest.mark.parametrize("f,names", [
    (dispatch, "x idx rows offsets pair inv"), (dispatch_backward, "d_rows inv dx"),
    (combine, "y gates inv out"), (combine_backward, "d_out y gates inv d_y d_gates"),
    (w4, "x w ws out"), (grouped, "x offsets w ws out")])
def test_required_pointers(f, names):
    for name in names.split():
        assert f(**{name: None}) == NULL, name


@pytest.mark.parametrize("f", [dispatch, dispatch_backward, combine, combine_backward])
@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), SHAPE), (dict(hidden=0), SHAPE), (dict(k=0), SHAPE), (dict(k=17), UNSUPPORTED),
    (dict(dtype=2), SHAPE), (dict(dtype=-1), SHAPE),
    (dict(tokens=1 << 24), UNSUPPORTED), (dict(tokens=(1 << 23) + 1, k=16), UNSUPPORTED),
    (dict(tokens=1 << 40), UNSUPPORTED), (dict(tokens=1 << 62), UNSUPPORTED)])
def test_refusals_of_the_row_operators(f, kw, status):
    assert f(**kw) == status


@pytest.mark.parametrize("f,lds", [(dispatch, "ld_x ld_rows"), (dispatch_backward, "ld_rows ld_dx"),
                                   (combine, "ld_y ld_out"),
                                   (combine_backward, "ld_d ld_y ld_dy")])
def test_row_distances_and_widths(f, lds):
    for ld in lds.split():
        assert f(**{ld: 63}) == SHAPE
    big = (1 << 20) + 1
    assert f(hidden=big, **{ld: big for ld in lds.split()}) == UNSUPPORTED
    wide = 1 << 20
    for tokens in (1 << 12, (1 << 12) - 1):
        assert f(hidden=wide, tokens=tokens, **{ld: wide for ld in lds.split()}) == UNSUPPORTED


@pytest.mark.parametrize("f,kw,status", [
    (dispatch, dict(experts=0), SHAPE), (dispatch, dict(experts=1025), UNSUPPORTED),
    (dispatch, dict(x=P + 1), UNSUPPORTED), (dispatch, dict(rows=P + 1), UNSUPPORTED),
    (dispatch, dict(x=P + 2, dtype=0), UNSUPPORTED), (dispatch, dict(idx=P + 2), UNSUPPORTED),
    (dispatch, dict(tokens=4096, k=2), NULL),
    (dispatch, dict(tokens=4096, k=2, ws=P, ws_bytes=255), WORKSPACE),
    (dispatch, dict(tokens=4096, k=2, ws=P + 16, ws_bytes=1 << 20), WORKSPACE),
    (dispatch_backward, dict(rows=-1), SHAPE), (dispatch_backward, dict(dx_dtype=3), SHAPE),
    (dispatch_backward, dict(dx=P + 1), UNSUPPORTED),
    (combine, dict(rows=-1), SHAPE), (combine, dict(out_dtype=7), SHAPE),
    (combine, dict(shared=P, ld_shared=63), SHAPE),
    (combine, dict(shared=P + 1, ld_shared=64), UNSUPPORTED), (combine, dict(gates=P + 2), UNSUPPORTED),
    (combine_backward, dict(rows=-1), SHAPE), (combine_backward, dict(d_dtype=2), SHAPE),
    (combine_backward, dict(d_out=P + 2), UNSUPPORTED), (combine_backward, dict(d_gates=P + 1), UNSUPPORTED),
])
def test_refusals_of_one_row_operator(f, kw, status):
    assert f(**kw) == status


def test_dispatch_workspace():
    assert moe.dispatch_workspace_bytes(1, 10, 512) == 0
    assert moe.dispatch_workspace_bytes(0, 10, 512) == 0
    n = moe.dispatch_workspace_bytes(4096, 10, 512)
    assert n > 0 and n % 256 == 0
    for bad in ((-1, 4, 8), (4096, 0, 8), (4096, 17, 8), (4096, 4, 0), (4096, 4, 1025)):
        assert moe.dispatch_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("f", [w4, grouped])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(n=0), SHAPE), (dict(k=0, ld_x=0), SHAPE), (dict(group=0), SHAPE),
    (dict(group=-64), SHAPE), (dict(k=250), SHAPE), (dict(group=16), UNSUPPORTED),
    (dict(group=256), UNSUPPORTED), (dict(swiglu=2), SHAPE), (dict(n=63, ld_out=63, swiglu=1), SHAPE),
    (dict(st=2), SHAPE), (dict(out_dtype=-1), SHAPE), (dict(ld_x=255), SHAPE), (dict(ld_out=63), SHAPE),
    (dict(ld_out=31, swiglu=1), SHAPE), (dict(rows=1 << 21), UNSUPPORTED),
    (dict(n=1 << 21, ld_out=1 << 21), UNSUPPORTED), (dict(k=1 << 21, ld_x=1 << 21), UNSUPPORTED),
    (dict(rows=1 << 20, n=1 << 20, ld_out=1 << 20), UNSUPPORTED),
    (dict(rows=4, x=P + 8), UNSUPPORTED), (dict(rows=4, w=P + 8), UNSUPPORTED),
    (dict(rows=4, ld_x=260), UNSUPPORTED), (dict(rows=4, ws=P + 2), UNSUPPORTED),
    (dict(rows=4, ws=P + 1, st=1), UNSUPPORTED), (dict(rows=4, bias=P + 2), UNSUPPORTED),
    (dict(rows=4, out=P + 1), UNSUPPORTED), (dict(rows=4, out=P + 2, out_dtype=0), UNSUPPORTED),
    (dict(rows=50000, n=1024, ld_out=1024), NULL),
    (dict(rows=50000, n=1024, ld_out=1024, work=P, work_bytes=1000), WORKSPACE),
    (dict(rows=50000, n=1024, ld_out=1024, work=P + 16, work_bytes=1 << 30), WORKSPACE)])
def test_refusals_of_the_products(f, kw, status):
    assert f(**kw) == status


def test_product_workspace():
    assert moe.linear_w4_workspace_bytes(1, 1, 4096, 4096, moe.MOE_BF16) == 0
    n = moe.linear_w4_workspace_bytes(5000, 1, 4096, 4000, moe.MOE_BF16)
    assert n >= 5000 * 4000 * 2 and n % 256 == 0
    for bad in ((-1, 1, 4096, 256, 1), (0, 1, 4096, 256, 1), (5000, 0, 4096, 256, 1),
                (5000, 1025, 4096, 256, 1), (5000, 1, 4096, 0, 1), (1 << 21, 1, 4096, 256, 1),
                (5000, 1, 4096, 1 << 21, 1), (5000, 1, 0, 256, 1), (5000, 1, 1 << 21, 256, 1)):
        assert moe.linear_w4_workspace_bytes(*bad) == 0


def test_refusals_of_the_grouped_product():
    assert grouped(experts=0) == SHAPE
    assert grouped(experts=1025) == UNSUPPORTED
    assert grouped(rows=4, offsets=P + 2) == UNSUPPORTED


def test_python_refuses_tensors_off_the_gpu():
    x, idx = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32)
    gates, codes = torch.zeros(4, 2), torch.zeros(8, 32, dtype=torch.uint8)
    for call in (lambda: moe.moe_dispatch(x, idx, 8), lambda: moe.moe_dispatch_backward(x, idx),
                 lambda: moe.moe_combine(x, gates, idx),
                 lambda: moe.moe_combine_backward(x, x, gates, idx),
                 lambda: moe.moe_linear_w4(x.bfloat16(), codes, torch.zeros(8, 1)),
                 lambda: moe.moe_grouped_linear_w4(x.bfloat16(), idx[0], codes[None],
                                                   torch.zeros(1, 8, 1))):
        with pytest.raises(ValueError):
            call()


@pytest.fixture
def off_gpu(monkeypatch):
    """The Python checks on CPU tensors, the C call replaced by one that must not run."""
    from block_fp8_routed_amd import _lib
    monkeypatch.setattr(_lib, "_place", lambda *a: 0)

    def no_call(*a):
        raise AssertionError("the call went through")
    monkeypatch.setattr(_lib, "_enqueue", no_call)
    return moe


def test_python_refuses_shapes_and_types(off_gpu):
    f, b, i, u = torch.float32, torch.bfloat16, torch.int32, torch.uint8
    z = torch.zeros
    bad = [
        lambda: moe.moe_dispatch(z(4, 64, dtype=torch.float16), z(4, 2, dtype=i), 8),
        lambda: moe.moe_dispatch(z(64, 4).t(), z(4, 2, dtype=i), 8),
        lambda: moe.moe_dispatch(z(64), z(4, 2, dtype=i), 8),
        lambda: moe.moe_dispatch(z(4, 64), z(4, 2, dtype=torch.int64), 8),
        lambda: moe.moe_dispatch(z(4, 64), z(5, 2, dtype=i), 8),
        lambda: moe.moe_dispatch(z(4, 64), z(2, 4, dtype=i).t(), 8),
        lambda: moe.moe_dispatch(z(4, 64), z(4, 2, dtype=i), 8, out=z(8, 64, dtype=b)),
        lambda: moe.moe_dispatch(z(4, 64), z(4, 2, dtype=i), 8, out=z(7, 64)),
        lambda: moe.moe_dispatch(z(4, 64), z(4, 2, dtype=i), 8, out=z(8, 65)),
        lambda: moe.moe_dispatch_backward(z(8, 64), z(8, dtype=i)),
        lambda: moe.moe_dispatch_backward(z(8, 64), z(4, 2, dtype=i), out_dtype=torch.float16),
        lambda: moe.moe_combine(z(8, 64), z(4, 3), z(4, 2, dtype=i)),
        lambda: moe.moe_combine(z(8, 64), z(4, 2, dtype=b), z(4, 2, dtype=i)),
        lambda: moe.moe_combine(z(8, 64), z(4, 2), z(4, 2, dtype=i), shared=z(4, 64, dtype=b)),
        lambda: moe.moe_combine(z(8, 64), z(4, 2), z(4, 2, dtype=i), shared=z(3, 64)),
        lambda: moe.moe_combine(z(8, 64), z(4, 2), z(4, 2, dtype=i), out=z(4, 63)),
        lambda: moe.moe_combine_backward(z(3, 64), z(8, 64), z(4, 2), z(4, 2, dtype=i)),
        lambda: moe.moe_combine_backward(z(4, 60), z(8, 64), z(4, 2), z(4, 2, dtype=i)),
        lambda: moe.moe_combine_backward(z(4, 64), z(8, 64), z(4, 2), z(4, 2, dtype=i),
                                         out=z(8, 64, dtype=b)),
        lambda: moe.moe_linear_w4(z(4, 64), z(8, 32, dtype=u), z(8, 1)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(8, 31, dtype=u), z(8, 1)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(8, 32, dtype=torch.int8), z(8, 1)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(8, 32, dtype=u), z(8, 3)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(8, 32, dtype=u), z(8, 0)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(8, 32, dtype=u), z(8, 1, dtype=torch.float16)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(8, 32, dtype=u), z(7, 1)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(8, 32, dtype=u), z(8, 1), z(8, 1)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(8, 32, dtype=u), z(8, 1), bias=z(7)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(8, 32, dtype=u), z(8, 1), out=z(4, 7)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(8, 32, dtype=u), z(8, 1), swiglu=True, out=z(4, 8)),
        lambda: moe.moe_linear_w4(z(4, 64, dtype=b), z(1, 8, 32, dtype=u), z(8, 1)),
        lambda: moe.moe_grouped_linear_w4(z(4, 64, dtype=b), z(2, dtype=i), z(8, 32, dtype=u), z(8, 1)),
        lambda: moe.moe_grouped_linear_w4(z(4, 64, dtype=b), z(3, dtype=i), z(1, 8, 32, dtype=u), z(1, 8, 1)),
        lambda: moe.moe_grouped_linear_w4(z(4, 64, dtype=b), z(2, dtype=torch.int64),
                                          z(1, 8, 32, dtype=u), z(1, 8, 1)),
        lambda: moe.moe_grouped_linear_w4(z(4, 64, dtype=b), z(2, dtype=i), z(1, 8, 32, dtype=u), z(8, 1)),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {n} was not refused")


def test_python_passes_what_the_header_allows(off_gpu):
    """The calls beside the refused ones do get as far as the library."""
    z, i = torch.zeros, torch.int32
    for call in (lambda: moe.moe_dispatch(z(4, 70)[:, 3:67], z(4, 2, dtype=i), 8),
                 lambda: moe.moe_combine(z(8, 64), z(4, 2), z(4, 2, dtype=i), out_dtype=torch.bfloat16),
                 lambda: moe.moe_linear_w4(z(4, 64).bfloat16(), z(8, 32).byte(), z(8, 1).bfloat16()),
                 lambda: moe.moe_grouped_linear_w4(z(4, 64).bfloat16(), z(2, dtype=i),
                                                   z(1, 8, 32).byte(), z(1, 8, 2))):
        with pytest.raises(AssertionError, match="went through"):
            call()
