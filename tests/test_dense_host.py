"""Host-side checks of the dense operators' C ABI and binding: no GPU work is
launched here (every call fails validation or has nothing to do)."""

import ctypes

import pytest
import torch

import virtual_noise_perturbed_amd as vn
from virtual_noise_perturbed_amd import _lib as E

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced
ODD = ctypes.c_void_p(0x10002)    # aligned to 2, not to 4


@pytest.fixture(scope="module")
def lib():
    return E.load()


def size_of(fn, *a):
    n = ctypes.c_int64(-1)
    return fn(*a, ctypes.byref(n)), n.value


def linear(lib, **kw):
    a = dict(x=FAKE, w=FAKE, dtype=E.VN_F32, b=None, r=None, rows=4, i=64, o=8, act=0, odt=E.VN_F32, y=FAKE, pre=None,
             ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.vn_linear(a["x"], a["w"], a["dtype"], a["b"], a["r"], a["rows"], a["i"], a["o"], a["act"], a["odt"],
                         a["y"], a["pre"], a["ws"], a["wsb"], None)


def test_linear_validation(lib):
    assert linear(lib, dtype=5) == E.VN_ERR_DTYPE
    assert linear(lib, odt=2) == E.VN_ERR_DTYPE
    for name in ("rows", "i", "o"):
        assert linear(lib, **{name: -1}) == E.VN_ERR_SHAPE
        assert linear(lib, **{name: 1 << 31}) == E.VN_ERR_OVERFLOW
        assert linear(lib, **{name: 1 << 30}) == E.VN_ERR_OVERFLOW   # threads past 32 bits
    assert linear(lib, rows=(1 << 31) - 1, o=(1 << 31) - 1) == E.VN_ERR_OVERFLOW    # tiles past 31 bits
    assert linear(lib, act=5) == E.VN_ERR_VALUE
    assert linear(lib, act=-1) == E.VN_ERR_VALUE
    assert linear(lib, wsb=-1) == E.VN_ERR_SHAPE
    for name in ("x", "w", "y"):
        assert linear(lib, **{name: None}) == E.VN_ERR_NULL
    for name in ("x", "w", "y", "b", "r", "pre", "ws"):
        assert linear(lib, **{name: ODD}) == E.VN_ERR_ALIGN
    # (a size whose few tiles share out k, with partial sums in the workspace)
    st, need = size_of(lib.vn_linear_workspace_size, E.VN_F32, 100, 4096, 100)
    assert st == E.VN_OK and need > 0
    assert linear(lib, rows=100, i=4096, o=100, wsb=need - 1) == E.VN_ERR_SHAPE
    assert linear(lib, rows=100, i=4096, o=100, ws=None, wsb=need) == E.VN_ERR_NULL
    # nothing to write
    assert linear(lib, rows=0, x=None, y=None) == E.VN_OK
    assert linear(lib, o=0, w=None, y=None) == E.VN_OK


def test_linear_workspace_size(lib):
    f = lib.vn_linear_workspace_size
    assert f(E.VN_F32, 1, 1, 1, None) == E.VN_ERR_NULL
    assert size_of(f, 7, 1, 1, 1)[0] == E.VN_ERR_DTYPE
    assert size_of(f, E.VN_BF16, -1, 1, 1)[0] == E.VN_ERR_SHAPE
    assert size_of(f, E.VN_BF16, 1, 1 << 40, 1)[0] == E.VN_ERR_OVERFLOW
    assert size_of(f, E.VN_BF16, 0, 64, 64) == (E.VN_OK, 0)
    # whole stages of bf16 that fill the GPU are read where they are
    assert size_of(f, E.VN_BF16, 4096, 4096, 4096) == (E.VN_OK, 0)


def backward(lib, **kw):
    a = dict(dy=FAKE, dydt=E.VN_F32, x=FAKE, w=FAKE, dtype=E.VN_F32, pre=FAKE, rows=4, i=64, o=8, act=2, dx=FAKE,
             dw=FAKE, dwdt=E.VN_F32, db=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.vn_linear_backward(a["dy"], a["dydt"], a["x"], a["w"], a["dtype"], a["pre"], a["rows"], a["i"], a["o"],
                                  a["act"], a["dx"], a["dw"], a["dwdt"], a["db"], a["ws"], a["wsb"], None)


def test_linear_backward_validation(lib):
    for name in ("dydt", "dtype", "dwdt"):
        assert backward(lib, **{name: 4}) == E.VN_ERR_DTYPE
    for name in ("rows", "i", "o"):
        assert backward(lib, **{name: -1}) == E.VN_ERR_SHAPE
        assert backward(lib, **{name: 1 << 31}) == E.VN_ERR_OVERFLOW
    assert backward(lib, act=9) == E.VN_ERR_VALUE
    for name in ("dy", "x", "w", "pre"):
        assert backward(lib, **{name: None}) == E.VN_ERR_NULL
    for name in ("dy", "x", "w", "pre", "dx", "dw", "db", "ws"):
        assert backward(lib, **{name: ODD}) == E.VN_ERR_ALIGN
    f = lib.vn_linear_backward_workspace_size
    st, need = size_of(f, E.VN_F32, E.VN_F32, 1000, 64, 8, 2, 7)
    assert st == E.VN_OK and need > 0
    assert backward(lib, rows=1000, wsb=need - 1) == E.VN_ERR_SHAPE
    assert backward(lib, rows=1000, ws=None, wsb=need) == E.VN_ERR_NULL
    assert size_of(f, E.VN_F32, E.VN_F32, 4, 64, 8, 2, 7) == (E.VN_OK, 0)   # (one launch, nothing between)
    assert size_of(f, E.VN_F32, E.VN_F32, 4, 64, 8, 2, 8)[0] == E.VN_ERR_VALUE
    assert size_of(f, E.VN_F32, E.VN_F32, 4, 64, 8, 7, 7)[0] == E.VN_ERR_VALUE
    assert f(E.VN_F32, E.VN_F32, 4, 64, 8, 2, 7, None) == E.VN_ERR_NULL
    # no output wanted
    assert backward(lib, dx=None, dw=None, db=None, ws=None, wsb=0) == E.VN_OK


def norm(lib, **kw):
    a = dict(x=FAKE, xdt=E.VN_F32, w=FAKE, b=FAKE, rows=3, n=8, eps=1e-5, y=FAKE, ydt=E.VN_F32, mean=FAKE, rstd=FAKE)
    a.update(kw)
    return lib.vn_layer_norm(a["x"], a["xdt"], a["w"], a["b"], a["rows"], a["n"], a["eps"], a["y"], a["ydt"],
                             a["mean"], a["rstd"], None)


def test_layer_norm_validation(lib):
    assert norm(lib, xdt=2) == E.VN_ERR_DTYPE
    assert norm(lib, ydt=-1) == E.VN_ERR_DTYPE
    assert norm(lib, rows=-1) == E.VN_ERR_SHAPE
    assert norm(lib, n=-1) == E.VN_ERR_SHAPE
    assert norm(lib, n=0) == E.VN_ERR_SHAPE          # the mean of nothing
    assert norm(lib, rows=1 << 40, n=1 << 40) == E.VN_ERR_OVERFLOW
    for eps in (float("nan"), float("inf"), -1e-5):
        assert norm(lib, eps=eps) == E.VN_ERR_VALUE
    assert norm(lib, x=None) == E.VN_ERR_NULL
    assert norm(lib, y=None) == E.VN_ERR_NULL
    for name in ("x", "y", "w", "b", "mean", "rstd"):
        assert norm(lib, **{name: ODD}) == E.VN_ERR_ALIGN
    assert norm(lib, rows=0, n=0, x=None, y=None) == E.VN_OK


def norm_backward(lib, **kw):
    a = dict(dy=FAKE, dydt=E.VN_F32, x=FAKE, xdt=E.VN_F32, w=FAKE, mean=FAKE, rstd=FAKE, rows=3, n=8, dx=FAKE,
             dw=FAKE, db=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.vn_layer_norm_backward(a["dy"], a["dydt"], a["x"], a["xdt"], a["w"], a["mean"], a["rstd"], a["rows"],
                                      a["n"], a["dx"], a["dw"], a["db"], a["ws"], a["wsb"], None)


def test_layer_norm_backward_validation(lib):
    assert norm_backward(lib, dydt=3) == E.VN_ERR_DTYPE
    assert norm_backward(lib, xdt=3) == E.VN_ERR_DTYPE
    assert norm_backward(lib, rows=-1) == E.VN_ERR_SHAPE
    assert norm_backward(lib, n=0) == E.VN_ERR_SHAPE
    assert norm_backward(lib, rows=1 << 40, n=1 << 40) == E.VN_ERR_OVERFLOW
    for name in ("dy", "x", "mean", "rstd"):
        assert norm_backward(lib, **{name: None}) == E.VN_ERR_NULL
    for name in ("dy", "x", "w", "mean", "rstd", "dx", "dw", "db", "ws"):
        assert norm_backward(lib, **{name: ODD}) == E.VN_ERR_ALIGN
    f = lib.vn_layer_norm_backward_workspace_size
    st, need = size_of(f, 3000, 8)
    assert st == E.VN_OK and need > 0
    assert norm_backward(lib, rows=3000, wsb=need - 1) == E.VN_ERR_SHAPE
    assert norm_backward(lib, rows=3000, ws=None, wsb=need) == E.VN_ERR_NULL
    assert size_of(f, 3, 8) == (E.VN_OK, 0)   # (one workgroup: no partial sums)
    assert f(3, 8, None) == E.VN_ERR_NULL
    assert size_of(f, -1, 8)[0] == E.VN_ERR_SHAPE
    assert norm_backward(lib, rows=0, n=0, dy=None, x=None) == E.VN_OK


def adamw(lib, count=1, **kw):
    i64, i32, dbl, vp = ctypes.c_int64 * 1, ctypes.c_int32 * 1, ctypes.c_double * 1, ctypes.c_void_p * 1
    a = dict(n=i64(5), p=vp(0x10000), pdt=i32(0), g=vp(0x10000), gdt=i32(0), c=None, wd=dbl(0.0), at=i64(0), total=128,
             bits=32, m=FAKE, v=FAKE, ms=FAKE, vs=FAKE, step=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, up=0, coef=None)
    a.update(kw)
    return lib.vn_adamw_step(count, a["n"], a["p"], a["pdt"], a["g"], a["gdt"], a["c"], a["wd"], a["at"], a["total"],
                             a["bits"], a["m"], a["v"], a["ms"], a["vs"], a["step"], a["lr"], a["b1"], a["b2"],
                             a["eps"], a["up"], a["coef"], None)


def test_adamw_validation(lib):
    i64, i32, dbl, vp = ctypes.c_int64 * 1, ctypes.c_int32 * 1, ctypes.c_double * 1, ctypes.c_void_p * 1
    assert adamw(lib, count=-1) == E.VN_ERR_SHAPE
    assert adamw(lib, count=0, n=None) == E.VN_OK
    assert adamw(lib, bits=16) == E.VN_ERR_VALUE
    assert adamw(lib, total=100) == E.VN_ERR_SHAPE           # not whole blocks
    assert adamw(lib, total=-128) == E.VN_ERR_SHAPE
    assert adamw(lib, n=i64(129)) == E.VN_ERR_SHAPE          # past the state
    assert adamw(lib, n=i64(-1)) == E.VN_ERR_SHAPE
    assert adamw(lib, n=i64(2**63 - 1)) == E.VN_ERR_SHAPE
    assert adamw(lib, at=i64(128)) == E.VN_ERR_SHAPE
    assert adamw(lib, at=i64(64), total=256) == E.VN_ERR_SHAPE
    assert adamw(lib, at=i64(-128)) == E.VN_ERR_SHAPE
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0), dict(b2=-0.1), dict(b2=float("nan")),
               dict(eps=-1.0), dict(step=0), dict(wd=dbl(float("inf")))):
        assert adamw(lib, **kw) == E.VN_ERR_VALUE
    assert adamw(lib, pdt=i32(2)) == E.VN_ERR_DTYPE
    assert adamw(lib, gdt=i32(-1)) == E.VN_ERR_DTYPE
    assert adamw(lib, pdt=i32(1), c=vp(0x10000)) == E.VN_ERR_DTYPE     # a copy of a bf16 parameter
    for name in ("n", "p", "pdt", "g", "gdt", "wd", "at", "m", "v"):
        assert adamw(lib, **{name: None}) == E.VN_ERR_NULL
    assert adamw(lib, p=vp(0)) == E.VN_ERR_NULL
    assert adamw(lib, bits=8, ms=None) == E.VN_ERR_NULL
    assert adamw(lib, p=vp(0x10002)) == E.VN_ERR_ALIGN
    assert adamw(lib, g=vp(0x10002)) == E.VN_ERR_ALIGN
    assert adamw(lib, c=vp(0x10001)) == E.VN_ERR_ALIGN
    assert adamw(lib, m=ODD) == E.VN_ERR_ALIGN
    assert adamw(lib, coef=ODD) == E.VN_ERR_ALIGN
    assert adamw(lib, n=i64(0), p=vp(0)) == E.VN_OK          # nothing to update
    f = lib.vn_adamw_coefficients
    assert f(None, 1e-3, 0.9, 0.999, FAKE, None) == E.VN_ERR_NULL
    assert f(FAKE, 1e-3, 0.9, 0.999, ODD, None) == E.VN_ERR_ALIGN
    assert f(FAKE, -1.0, 0.9, 0.999, FAKE, None) == E.VN_ERR_VALUE


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(2, 4), torch.zeros(3, 4)
    with pytest.raises(ValueError, match="no CPU path"):
        vn.linear(x, w)
    with pytest.raises(ValueError, match="no CPU path"):
        vn.linear_backward(torch.zeros(2, 3), x, w)
    with pytest.raises(ValueError, match="no CPU path"):
        vn.layer_norm(x)
    with pytest.raises(ValueError, match="no CPU path"):
        vn.layer_norm_backward(x, x, torch.zeros(2), torch.zeros(2))
    with pytest.raises(ValueError, match="no CPU path"):
        vn.AdamW([x], [x])
    with pytest.raises(ValueError):
        vn.AdamW([], [])
    with pytest.raises(TypeError):
        vn.linear(x, "w")


def test_sizes_of_zero_need_no_products(lib):
    for sizes in ((0, 8, 6), (3, 0, 6), (3, 8, 0), (0, 0, 0), (0, 0, 6)):
        for dtype in (E.VN_F32, E.VN_BF16):
            st, need = size_of(lib.vn_linear_backward_workspace_size, dtype, dtype, *sizes, 2, 7)
            assert st == E.VN_OK and need >= 0
            assert size_of(lib.vn_linear_workspace_size, dtype, *sizes)[0] == E.VN_OK
