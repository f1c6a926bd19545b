"""The dense operators (linear layer with epilogue, layer norm, their gradients,
AdamW) against their definitions in 64 bits, within bounds derived from their
operation counts; refusals; graphs; streams."""

import math

import pytest
import torch

import dense_ref as ref
import virtual_noise_perturbed_amd as vn
from gpu_util import device

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}


def rand(gen, *shape, scale=1.0, mean=0.0, dtype=F32):
    return (torch.randn(shape, generator=gen) * scale + mean).to(dtype)


def dev(t):
    return None if t is None else t.to(device())


def within(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if got.numel():
        worst = ((got - want).abs() / bound).max().item()
        assert worst <= 1.0, f"{what}: error is {worst:.3g} of its bound"


# (rows, in, out): one row, fewer than a tile, ragged in every direction, one off each tile, split sums
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 130), (2, 7, 300), (3, 100, 5), (5, 72, 16), (16, 512, 100),
          (17, 256, 33), (33, 65, 63), (64, 128, 64), (65, 191, 257), (100, 784, 256), (128, 64, 129),
          (127, 1000, 384), (300, 40, 700), (513, 320, 520), (1024, 256, 1100), (40, 8200, 24)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_shapes(shape, dtype):
    print("linear", shape, dtype, flush=True)
    m, k, n = shape
    dt = TYPES[dtype]
    gen = torch.Generator().manual_seed(m * 7 + k * 3 + n)
    x, w, b, r = (rand(gen, m, k, dtype=dt), rand(gen, n, k, scale=k ** -0.5, dtype=dt), rand(gen, n, scale=0.3),
                  rand(gen, m, n, dtype=dt))
    pre = torch.full((m, n), float("nan"), dtype=dt, device=device())
    y = vn.linear(dev(x), dev(w), dev(b), activation="gelu", residual=dev(r), pre=pre)
    want, z, ez = ref.linear(x, w, b, "gelu", r)
    within(y, want, ref.linear_bound(want, z, ez, dt, r), "y")
    within(pre, z, ez + ref.HALF[dt] * z.abs() * 1.01 + 1e-30, "pre")
    # the same bits again, and without the optional parts
    assert torch.equal(vn.linear(dev(x), dev(w), dev(b), activation="gelu", residual=dev(r)), y)
    want, z, ez = ref.linear(x, w, None, None, None)
    within(vn.linear(dev(x), dev(w)), want, ref.linear_bound(want, z, ez, dt, None), "x W^T")


@pytest.mark.parametrize("rows", [4, 200])
@pytest.mark.parametrize("act", [None, "none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype,out_dtype", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_linear_epilogues(dtype, out_dtype, act, rows):
    print("linear epilogue", dtype, out_dtype, act, rows, flush=True)
    dt, od = TYPES[dtype], TYPES[out_dtype]
    gen = torch.Generator().manual_seed(5)
    k, n = 96, 130
    # pre-activations from -8 to 8: both tails
    x, w = rand(gen, rows, k, scale=2.0, dtype=dt), rand(gen, n, k, scale=k ** -0.5, dtype=dt)
    b, r = rand(gen, n), rand(gen, rows, n, dtype=od)
    want, z, ez = ref.linear(x, w, b, act, r)
    y = vn.linear(dev(x), dev(w), dev(b), activation=act, residual=dev(r), out_dtype=od)
    assert y.dtype == od
    within(y, want, ref.linear_bound(want, z, ez, od, r), "y")
    # in place of the residual, as a residual stream is updated
    acc = dev(r).clone()
    assert vn.linear(dev(x), dev(w), dev(b), activation=act, residual=acc, out=acc) is acc
    assert torch.equal(acc, y)


def test_linear_layouts():
    """Leading axes, transposed and sliced views, unaligned starts, offsets in x."""
    gen = torch.Generator().manual_seed(9)
    for dt in (F32, BF16):
        x, w = rand(gen, 4, 3, 64, dtype=dt), rand(gen, 64, 48, scale=0.1, dtype=dt)
        want, z, ez = ref.linear(x.reshape(12, 64), w.t(), None, "relu", None)
        y = vn.linear(dev(x), dev(w).t(), activation="relu")
        assert y.shape == (4, 3, 48)
        within(y.reshape(12, 48), want, ref.linear_bound(want, z, ez, dt, None), "transposed weight")
        big = dev(rand(gen, 12 * 64 + 1, dtype=dt))
        big[1:] = dev(x.reshape(-1))
        assert torch.equal(vn.linear(big[1:].view(4, 3, 64), dev(w).t(), activation="relu"), y)
        wide = dev(rand(gen, 4, 3, 128, dtype=dt))
        wide[..., ::2] = dev(x)
        assert torch.equal(vn.linear(wide[..., ::2], dev(w).t(), activation="relu"), y)
        assert torch.equal(vn.linear(dev(x)[1, 2], dev(w).t(), activation="relu"), vn.linear(dev(x)[1, 2][None], dev(w).t(), activation="relu")[0])


def test_linear_nothing_to_sum_or_write():
    d = device()
    b, r = torch.randn(6, device=d), torch.randn(5, 6, device=d)
    y = vn.linear(torch.empty(5, 0, device=d), torch.empty(6, 0, device=d), b, activation="relu", residual=r)
    assert torch.equal(y, torch.relu(b)[None] + r)
    assert vn.linear(torch.empty(0, 8, device=d), torch.empty(6, 8, device=d)).shape == (0, 6)
    assert vn.linear(torch.empty(2, 8, device=d), torch.empty(0, 8, device=d)).shape == (2, 0)
    dx, dw, db = vn.linear_backward(torch.empty(0, 6, device=d), torch.empty(0, 8, device=d), torch.ones(6, 8, device=d))
    assert dx.shape == (0, 8) and not dw.any() and dw.shape == (6, 8) and not db.any() and db.shape == (6,)
    dx, dw, db = vn.linear_backward(torch.empty(3, 0, device=d), torch.ones(3, 8, device=d), torch.empty(0, 8, device=d))
    assert dx.shape == (3, 8) and not dx.any() and dw.shape == (0, 8) and db.shape == (0,)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_large_values_and_nonfinite(dtype):
    """Values near the type's ends keep their accuracy; a NaN stays in its row."""
    print("linear large", dtype, flush=True)
    dt = TYPES[dtype]
    gen = torch.Generator().manual_seed(3)
    m, k, n = 70, 130, 66
    x, w = rand(gen, m, k, dtype=dt), rand(gen, n, k, dtype=dt)
    x[3] *= 2.0 ** 100
    x[4] *= 2.0 ** -60
    w[5] *= 2.0 ** 20
    want, z, ez = ref.linear(x, w, None, None, None)
    within(vn.linear(dev(x), dev(w)), want, ref.linear_bound(want, z, ez, dt, None) , "scaled rows")
    top = torch.full((2, 64), torch.finfo(dt).max, dtype=dt)
    eye = torch.eye(64, dtype=dt)
    assert torch.equal(vn.linear(dev(top), dev(eye)).cpu(), top)
    x[7, 11] = float("nan")
    y = vn.linear(dev(x), dev(w)).cpu()
    assert torch.isnan(y[7]).all()
    keep = [i for i in range(m) if i != 7]
    within(y[keep], want[keep], ref.linear_bound(want, z, ez, dt, None)[keep], "other rows")


def test_linear_mid_size_sums_are_fp32():
    """A long reduction in bf16: as exact as fp32 sums of exact products are."""
    gen = torch.Generator().manual_seed(1)
    x, w = rand(gen, 300, 16384, dtype=BF16), rand(gen, 260, 16384, scale=1 / 128, dtype=BF16)
    want = x.double() @ w.double().t()
    y = vn.linear(dev(x), dev(w), out_dtype=F32).double().cpu()
    # rounding errors of partial sums add like a random walk: 6 standard deviations of
    # sqrt(k) * u * the partial sums' size, about that of the result
    assert float((y - want).norm() / want.norm()) <= 6 * math.sqrt(16384) * ref.U


BACK = [(1, 1, 1), (1, 256, 128), (3, 100, 70), (65, 130, 67), (64, 64, 64), (200, 784, 10), (129, 1000, 300),
        (700, 90, 513), (1030, 512, 260)]


@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", BACK, ids=str)
def test_linear_backward(shape, dtype, act):
    print("linear_backward", shape, dtype, act, flush=True)
    m, k, n = shape
    dt = TYPES[dtype]
    gen = torch.Generator().manual_seed(m + 5 * k + 9 * n)
    x, w = rand(gen, m, k, dtype=dt), rand(gen, n, k, scale=k ** -0.5, dtype=dt)
    dy, pre = rand(gen, m, n, dtype=dt), rand(gen, m, n, scale=2.0, dtype=dt)
    dx, dw, db = vn.linear_backward(dev(dy), dev(x), dev(w), activation=act, pre=None if act is None else dev(pre))
    dz = dy.double() * ref.slope(pre.double(), act)
    # dz within 24 units of |dy| (erf, exp, a division and their sums), rounded to the
    # operands' type; then sums of products as in the forward
    e_dz = (0 if act is None else 24 * 1.2) * ref.U * dy.double().abs()
    e = e_dz + (ref.HALF[dt] * 1.01 if dt == BF16 and act is not None else 0) * dz.abs()
    az, aw, ax = dz.abs() + e, w.double().abs(), x.double().abs()
    want = dz @ w.double()
    within(dx, want, e @ aw + (n + 12) * ref.U * (az @ aw) + ref.HALF[dt] * 1.01 * want.abs() + 1e-30, "dx")
    want = dz.t() @ x.double()
    within(dw, want, e.t() @ ax + (m + 12) * ref.U * (az.t() @ ax) + ref.HALF[dt] * 1.01 * want.abs() + 1e-30, "dw")
    within(db, dz.sum(0), e_dz.sum(0) + (m + 4) * ref.U * az.sum(0) + 1e-30, "db")
    again = vn.linear_backward(dev(dy), dev(x), dev(w), activation=act, pre=None if act is None else dev(pre))
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))


def test_linear_backward_options():
    gen = torch.Generator().manual_seed(2)
    x, w, dy, pre = rand(gen, 90, 70, dtype=BF16), rand(gen, 50, 70, dtype=BF16), rand(gen, 90, 50), rand(gen, 90, 50, dtype=BF16)
    args = [dev(t) for t in (dy, x, w)]
    full = vn.linear_backward(*args, activation="silu", pre=dev(pre), weight_gradient_dtype=F32)
    assert full[0].dtype == BF16 and full[1].dtype == F32 and full[2].dtype == F32
    for i in range(3):
        want = [False] * 3
        want[i] = True
        got = vn.linear_backward(*args, activation="silu", pre=dev(pre), input_gradient=want[0],
                                 weight_gradient=want[1], bias_gradient=want[2], weight_gradient_dtype=F32)
        assert all((g is not None) == k for g, k in zip(got, want))
        assert torch.equal(got[i], full[i])
    # fp32 dy with bf16 operands: db from the unrounded product, dw not rounded again
    dz = dy.double() * ref.slope(pre.double(), "silu")
    within(full[2], dz.sum(0), (24 * 1.2 + 94) * ref.U * dy.double().abs().sum(0) * 1.2, "db")
    b16 = dz.to(BF16).double()
    near = b16.t() @ x.double()
    # dz's own error can move a rounding: one step of bf16 for values near a tie
    off = (dz.abs() * 2.0 ** -7).t() @ x.double().abs() * 0.02 + 200 * ref.U * (dz.abs().t() @ x.double().abs())
    within(full[1], near, off, "dw")


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_linear_gradients_against_differences(act):
    """The layer's gradients against central differences of the 64-bit forward
    along random directions (h = 1e-4: the difference is within h^2 of the slope)."""
    gen = torch.Generator().manual_seed(8)
    m, k, n, h = 40, 30, 50, 1e-4
    x, w, b, c = rand(gen, m, k), rand(gen, n, k, scale=0.3), rand(gen, n), rand(gen, m, n)
    pre = torch.empty(m, n, device=device())
    vn.linear(dev(x), dev(w), dev(b), activation=act, pre=pre)
    grads = vn.linear_backward(dev(c), dev(x), dev(w), activation=act, pre=pre)

    def loss(t):
        return float((ref.linear(t[0], t[1], t[2], act, None)[0] * c.double()).sum())

    at = [x.double(), w.double(), b.double()]
    for i in range(3):
        d = rand(gen, *at[i].shape).double()
        up = [t + h * d if j == i else t for j, t in enumerate(at)]
        down = [t - h * d if j == i else t for j, t in enumerate(at)]
        slope = (loss(up) - loss(down)) / (2 * h)
        got = float((grads[i].double().cpu() * d).sum())
        size = float((grads[i].double().cpu() * d).abs().sum())
        assert abs(got - slope) <= (200 * ref.U + 100 * h * h) * size


# rows of every layout: below a lane's run, one off each width limit, odd widths, longer than the registers
NORMS = [(1, 1), (3, 7), (5, 8), (17, 100), (33, 128), (64, 129), (9, 512), (10, 513), (31, 1000), (7, 1024), (6, 1025),
         (5, 2048), (4, 2049), (300, 4096), (3, 4097), (2, 8192), (3, 8193), (2, 16384), (3, 16385), (2, 30011),
         (2500, 33), (4100, 260)]


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")], ids=str)
@pytest.mark.parametrize("shape", NORMS, ids=str)
def test_layer_norm(shape, types):
    print("layer_norm", shape, types, flush=True)
    m, n = shape
    dt, od = TYPES[types[0]], TYPES[types[1]]
    gen = torch.Generator().manual_seed(m + n)
    x, w, b = rand(gen, m, n, scale=3.0, mean=0.7, dtype=dt), rand(gen, n, scale=0.3, mean=1.0), rand(gen, n)
    y, mean, rstd = vn.layer_norm(dev(x), dev(w), dev(b), out_dtype=od, stats=True)
    assert y.dtype == od
    want = ref.layer_norm(x, w, b, 1e-5)
    for got, ok, bound, what in zip((y, mean, rstd), want, ref.layer_norm_bounds(x, w, b, *want, od), ("y", "mean", "rstd")):
        within(got, ok, bound, what)
    assert torch.equal(vn.layer_norm(dev(x), dev(w), dev(b), out_dtype=od), y)
    want = ref.layer_norm(x, None, None, 0.5)
    within(vn.layer_norm(dev(x), eps=0.5, out_dtype=od), want[0],
           ref.layer_norm_bounds(x, None, None, *want, od)[0], "without weight and bias")


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")], ids=str)
@pytest.mark.parametrize("shape", NORMS, ids=str)
def test_layer_norm_backward(shape, types):
    print("layer_norm_backward", shape, types, flush=True)
    m, n = shape
    gt, dt = TYPES[types[0]], TYPES[types[1]]
    gen = torch.Generator().manual_seed(m * 3 + n)
    x, w, dy = rand(gen, m, n, scale=3.0, mean=0.7, dtype=dt), rand(gen, n, scale=0.3, mean=1.0), rand(gen, m, n, dtype=gt)
    _, mean, rstd = (t.float() for t in ref.layer_norm(x, None, None, 1e-5))
    for weight in (w, None):
        got = vn.layer_norm_backward(dev(dy), dev(x), dev(mean), dev(rstd), dev(weight))
        want = ref.layer_norm_backward(dy, x, mean, rstd, weight)
        bounds = ref.layer_norm_backward_bounds(dy, x, mean, rstd, weight, want[0], m, dt)
        for g, o, e, what in zip(got, want, bounds, ("dx", "dweight", "dbias")):
            within(g, o, e, what)
    again = vn.layer_norm_backward(dev(dy), dev(x), dev(mean), dev(rstd))
    assert all(torch.equal(a, b) for a, b in zip(again, got))
    only = vn.layer_norm_backward(dev(dy), dev(x), dev(mean), dev(rstd), parameter_gradients=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], got[0])
    sums = vn.layer_norm_backward(dev(dy), dev(x), dev(mean), dev(rstd), input_gradient=False)
    assert sums[0] is None and torch.equal(sums[1], got[1]) and torch.equal(sums[2], got[2])


def test_layer_norm_edges():
    """Constant rows, large offsets, non-finite rows, layouts, nothing to do."""
    d = device()
    x = torch.full((3, 100), 5.0, device=d)
    y, mean, rstd = vn.layer_norm(x, stats=True)
    assert torch.equal(y, torch.zeros_like(y)) and torch.equal(mean, x[:, 0])
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=4 * ref.U)
    gen = torch.Generator().manual_seed(4)
    # a mean of 2^10 standard deviations: differences to the mean, not E[x^2] - mean^2
    far = rand(gen, 9, 1000, mean=1024.0)
    want = ref.layer_norm(far, None, None, 1e-5)
    got = vn.layer_norm(dev(far), stats=True)
    for g, o, e in zip(got, want, ref.layer_norm_bounds(far, None, None, *want, F32)):
        within(g, o, e, "far from zero")
    bad = rand(gen, 6, 300)
    bad[1, 7], bad[4, 2] = float("nan"), float("inf")
    y = vn.layer_norm(dev(bad)).cpu()
    assert torch.isnan(y[[1, 4]]).all() and torch.isfinite(y[[0, 2, 3, 5]]).all()
    x = rand(gen, 4, 5, 48)
    y = vn.layer_norm(dev(x))
    assert y.shape == x.shape
    assert torch.equal(vn.layer_norm(dev(x).transpose(0, 1)), y.transpose(0, 1))
    assert torch.equal(vn.layer_norm(dev(x)[1, 2]), y[1, 2])
    shifted = torch.empty(4 * 5 * 48 + 1, device=d)[1:].view(4, 5, 48)
    shifted.copy_(x)
    assert torch.equal(vn.layer_norm(shifted, out=shifted), y) and torch.equal(shifted, y)
    assert vn.layer_norm(torch.empty(0, 7, device=d)).shape == (0, 7)
    dx, dw, db = vn.layer_norm_backward(torch.empty(0, 7, device=d), torch.empty(0, 7, device=d), torch.empty(0, device=d),
                                        torch.empty(0, device=d))
    assert dx.shape == (0, 7) and not dw.any() and not db.any()
    with pytest.raises(ValueError):
        vn.layer_norm(torch.empty(3, 0, device=d))


def test_layer_norm_gradients_against_differences():
    gen = torch.Generator().manual_seed(6)
    m, n, h = 12, 90, 1e-4
    x, w, b, c = rand(gen, m, n), rand(gen, n, mean=1.0), rand(gen, n), rand(gen, m, n)
    _, mean, rstd = vn.layer_norm(dev(x), dev(w), dev(b), stats=True)
    grads = vn.layer_norm_backward(dev(c), dev(x), mean, rstd, dev(w))

    def loss(t):
        return float((ref.layer_norm(t[0], t[1], t[2], 1e-5)[0] * c.double()).sum())

    at = [x.double(), w.double(), b.double()]
    for i in range(3):
        d = rand(gen, *at[i].shape).double()
        up = [t + h * d if j == i else t for j, t in enumerate(at)]
        down = [t - h * d if j == i else t for j, t in enumerate(at)]
        slope = (loss(up) - loss(down)) / (2 * h)
        got = float((grads[i].double().cpu() * d).sum())
        size = float((grads[i].double().cpu() * d).abs().sum())
        assert abs(got - slope) <= (400 * ref.U + 100 * h * h) * size


SIZES = [(1,), (7,), (128,), (129,), (63, 63), (63,), (3, 5, 11), (0,), (4096,), (4097,), (70, 130), (100003,)]


def adamw_case(seed, sizes, gdt=F32, pdt=F32):
    gen = torch.Generator().manual_seed(seed)
    return [rand(gen, *s, dtype=pdt) for s in sizes], lambda: [rand(gen, *s, scale=0.01, dtype=gdt) for s in sizes]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gdt,pdt", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_adamw(gdt, pdt, bits):
    """Several steps over many sizes (over 64 tensors: two launches), the state's
    codes and the parameters bit for bit those of the definition in fp32."""
    print("adamw", gdt, pdt, bits, flush=True)
    sizes = SIZES * 6
    params, grads_of = adamw_case(11, sizes, TYPES[gdt], TYPES[pdt])
    # every third parameter at an address that is aligned to its element alone
    mine = []
    for i, p in enumerate(params):
        room = torch.zeros(p.numel() + 1, dtype=p.dtype, device=device())
        t = room[1:] if i % 3 == 0 else room[:p.numel()]
        t = t.view(p.shape)
        t.copy_(p)
        mine.append(t)
    wd = [0.0 if p.dim() < 2 else 0.1 for p in params]
    copies = [torch.zeros(p.shape, dtype=BF16, device=device()) if i % 2 else None for i, p in enumerate(params)] if pdt == "f32" else None
    hyper = dict(lr=3e-3, betas=(0.8, 0.95), eps=1e-6)
    grads = grads_of()
    opt = vn.AdamW(mine, [dev(g) for g in grads], weight_decay=wd, copies=copies, state_bits=bits, maximize=True, **hyper)
    state = [(torch.zeros(-(-p.numel() // 128) * 128), torch.zeros(-(-p.numel() // 128) * 128)) for p in params]
    for t in range(1, 4):
        opt.step(None if t == 1 else [dev(g) for g in grads])
        for i, (p, g) in enumerate(zip(params, grads)):
            n = p.numel()
            pad = lambda v: torch.nn.functional.pad(v.float().reshape(-1), (0, state[i][0].numel() - n))
            new, m, v = ref.adamw32(pad(p), pad(g), *state[i], t, hyper["lr"], hyper["betas"], hyper["eps"], wd[i], True)
            params[i] = new[:n].view(p.shape).to(p.dtype)
            assert torch.equal(mine[i].cpu(), params[i]), (t, i)
            if copies is not None and copies[i] is not None:
                assert torch.equal(copies[i].cpu(), params[i].to(BF16)), (t, i)
            at = slice(opt.offsets[i], opt.offsets[i] + m.numel())
            if bits == 32:
                assert torch.equal(opt.state["exp_avg"][at].cpu(), m) and torch.equal(opt.state["exp_avg_sq"][at].cpu(), v), (t, i)
            elif n:
                cm, cv, sm, sv = ref.quantize_state(m, v, t, opt.offsets[i])
                blocks = slice(at.start // 128, at.stop // 128)
                assert torch.equal(opt.state["exp_avg_scale"][blocks].cpu(), sm), (t, i)
                assert torch.equal(opt.state["exp_avg_sq_scale"][blocks].cpu(), sv), (t, i)
                assert torch.equal(opt.state["exp_avg"][at].view(torch.uint8).cpu(), cm), (t, i)
                assert torch.equal(opt.state["exp_avg_sq"][at].view(torch.uint8).cpu(), cv), (t, i)
                m, v = ref.dequantize(cm, sm, torch.float8_e4m3fn), ref.dequantize(cv, sv, torch.float8_e5m2)
            state[i] = (m, v)
        grads = grads_of()
    assert opt.state["step"] == 3
    for i, (m, v) in enumerate(opt.moments()):
        n = params[i].numel()
        assert torch.equal(m.cpu().reshape(-1), state[i][0][:n]) and torch.equal(v.cpu().reshape(-1), state[i][1][:n])


def test_adamw_against_64_bits():
    params, grads_of = adamw_case(1, [(301, 77), (5000,)])
    mine, m, v = [dev(p) for p in params], [0.0, 0.0], [0.0, 0.0]
    opt = vn.AdamW(mine, [dev(g) for g in grads_of()], lr=1e-2, weight_decay=0.1)
    p64 = [p.double() for p in params]
    for t in range(1, 21):
        grads = grads_of()
        opt.step([dev(g) for g in grads])
        for i, g in enumerate(grads):
            m[i] = 0.9 * m[i] + 0.1 * g.double()
            v[i] = 0.999 * v[i] + 0.001 * g.double() ** 2
            p64[i] = p64[i] * (1 - 1e-2 * 0.1) - 1e-2 * (m[i] / (1 - 0.9 ** t)) / ((v[i] / (1 - 0.999 ** t)).sqrt() + 1e-8)
    for i in range(2):
        # an update (at most lr * 10 in size) is within 3 t + 10 units, and a step rounds p twice
        bound = 20 * (2 * ref.U * p64[i].abs() + 70 * ref.U * 1e-2 * 10)
        within(mine[i], p64[i], bound, "p")


def test_adamw_8_bit_averages_follow():
    """Averages that move by less than a code's width a step still follow: after
    2000 steps of unit-variance gradients the second average, whose codes lie 25%
    apart and whose steps are 0.1%, is unbiased (within 5 standard errors of the
    simulated spread of 25% over 4096 elements, and the dither's own 4%), and
    after the gradients stop it decays: by a code whenever the offsets' even spread
    says, that is after 1000 (1/8 + 1/7 + 1/6 + 1/5) = 634 steps a halving where the
    exact average takes 693, which leaves 0.91 of it after 1000 steps (0.86 where
    the last few codes and the block's scale are simulated too)."""
    n = 4096
    gen = torch.Generator(device=device()).manual_seed(2)
    p, g = torch.zeros(n, device=device()), torch.zeros(n, device=device())
    opt = vn.AdamW([p], [g], state_bits=8, weight_decay=0.0)
    true = torch.zeros(n, dtype=torch.float64, device=device())
    for _ in range(2000):
        g.copy_(torch.randn(n, generator=gen, device=device()))
        opt.step()
        true = 0.999 * true + 0.001 * g.double() ** 2
    ratio = opt.moments()[0][1].double() / true
    assert abs(float(ratio.mean()) - 1) <= 0.04 + 5 * 0.25 / 64
    assert float(ratio.min()) > 0.2 and float(ratio.max()) < 4
    g.zero_()
    for _ in range(1000):
        opt.step()
    ratio = opt.moments()[0][1].double() / (true * 0.999 ** 1000)
    assert 0.75 <= float(ratio.mean()) <= 1.1


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_nonfinite_and_zero(bits):
    d = device()
    p = torch.ones(300, device=d)
    g = torch.zeros(300, device=d)
    opt = vn.AdamW([p], [g], state_bits=bits, weight_decay=0.0)
    opt.step()                      # zero gradients from a zero state: nothing moves
    assert torch.equal(p, torch.ones_like(p))
    g.fill_(0.5)
    g[5], g[140] = float("nan"), float("inf")
    opt.step()
    bad = ~torch.isfinite(p)
    assert bad[5] and bad[140] and int(bad.sum()) == 2
    g.fill_(0.5)
    opt.step()
    bad = ~torch.isfinite(p)
    if bits == 32:
        assert int(bad.sum()) == 2
    else:
        assert bad[:256].all() and not bad[256:].any()


def test_adamw_state_goes_on():
    """Stepping on from another optimizer's state gives the same bits."""
    params, grads_of = adamw_case(4, [(50, 30), (17,)])
    steps = [[dev(g) for g in grads_of()] for _ in range(4)]
    for bits in (32, 8):
        a, b = [dev(p) for p in params], [dev(p) for p in params]
        one = vn.AdamW(a, steps[0], state_bits=bits)
        for s in steps:
            one.step(s)
        two = vn.AdamW(b, steps[0], state_bits=bits)
        for s in steps[:2]:
            two.step(s)
        held = {k: v.clone() if torch.is_tensor(v) else v for k, v in two.state.items()}
        three = vn.AdamW(b, steps[2], state_bits=bits, state=held)
        for s in steps[2:]:
            three.step(s)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert three.state["step"] == 4


def test_binding_refusals():
    d = device()
    x, w = torch.zeros(4, 8, device=d), torch.zeros(5, 8, device=d)
    dy = torch.zeros(4, 5, device=d)
    with pytest.raises(ValueError, match="in_features"):
        vn.linear(x[:, :7], w)
    with pytest.raises(TypeError):
        vn.linear(x.half(), w.half())
    with pytest.raises(TypeError):
        vn.linear(x, w.bfloat16())
    with pytest.raises(TypeError):
        vn.linear(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="activation"):
        vn.linear(x, w, activation="tanh")
    with pytest.raises(ValueError, match="bias"):
        vn.linear(x, w, torch.zeros(6, device=d))
    with pytest.raises(ValueError, match="residual"):
        vn.linear(x, w, residual=dy.bfloat16())
    with pytest.raises(ValueError, match="pre"):
        vn.linear(x, w, pre=torch.zeros(5, 4, device=d).t())
    with pytest.raises(ValueError, match="out"):
        vn.linear(x, w, out=torch.zeros(4, 6, device=d))
    with pytest.raises(ValueError, match="needs pre"):
        vn.linear_backward(dy, x, w, activation="gelu")
    with pytest.raises(ValueError, match="dy"):
        vn.linear_backward(dy[:3], x, w)
    with pytest.raises(ValueError):
        vn.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError, match="weight"):
        vn.layer_norm(x, torch.ones(7, device=d))
    with pytest.raises(ValueError, match="mean"):
        vn.layer_norm_backward(x, x, torch.zeros(3, device=d), torch.zeros(4, device=d))
    with pytest.raises(TypeError):
        vn.layer_norm(x.double())
    with pytest.raises(ValueError, match="contiguous"):
        vn.AdamW([w.t()], [w.t()])
    with pytest.raises(ValueError, match="size"):
        vn.AdamW([w], [x])
    with pytest.raises(ValueError, match="one gradient"):
        vn.AdamW([w], [])
    with pytest.raises(ValueError, match="state_bits"):
        vn.AdamW([w], [w.clone()], state_bits=16)
    with pytest.raises(ValueError, match="weight_decay"):
        vn.AdamW([w], [w.clone()], weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError, match="copies"):
        vn.AdamW([w], [w.clone()], copies=[torch.zeros(5, 8, device=d)])
    with pytest.raises(ValueError, match="state"):
        vn.AdamW([w], [w.clone()], state=vn.AdamW([w], [w.clone()], state_bits=8).state)
    opt = vn.AdamW([w], [w.clone()])
    w.data = torch.zeros(500, 8, device=d)
    with pytest.raises(ValueError, match="other memory"):
        opt.step()


def step_of(d, dtype, gen):
    """A pre-norm residual layer's training step on fixed buffers: norm, projection
    with residual, gradients, optimizer with its count on the GPU."""
    w32 = torch.randn(130, 130, generator=gen).div(12).to(d)
    b, gw, gb = torch.zeros(130, device=d), torch.ones(130, device=d), torch.zeros(130, device=d)
    w = w32.to(dtype)
    x = torch.randn(70, 130, generator=gen).to(d).to(dtype)
    pre = torch.empty_like(x)
    params = [w32, b, gw, gb]
    grads = [torch.empty(130, 130, dtype=dtype, device=d)] + [torch.empty(130, device=d) for _ in range(3)]
    opt = vn.AdamW(params, grads, lr=1e-2, copies=[w, None, None, None] if dtype == BF16 else None, state_bits=8,
                   device_step=True)

    def step():
        h, mean, rstd = vn.layer_norm(x, gw, gb, stats=True)
        weight = w if dtype == BF16 else w32
        y = vn.linear(h, weight, b, activation="silu", residual=x, pre=pre)
        dx, dw, db = vn.linear_backward(y, h, weight, activation="silu", pre=pre)
        _, dg, dh = vn.layer_norm_backward(dx, x, mean, rstd, gw)
        for have, new in zip(grads, (dw, db, dg, dh)):
            have.copy_(new)
        opt.step()
        return y

    return step, params, opt


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_graph_replays_count_on(dtype):
    """A captured step replays as the eager steps go: the same parameters after
    each, with eager work and synchronizations between the replays."""
    d = device()
    eager, params_e, _ = step_of(d, dtype, torch.Generator().manual_seed(3))
    captured, params_g, opt = step_of(d, dtype, torch.Generator().manual_seed(3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured()
    torch.cuda.current_stream().wait_stream(side)
    eager()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(params_e, params_g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = captured()
    for i in range(4):
        graph.replay()
        want = eager()
        torch.cuda.synchronize()
        junk = torch.randn(1 << 20, device=d).sum().item()
        assert math.isfinite(junk)
        assert torch.equal(y, want), i
        assert all(torch.equal(a, b) for a, b in zip(params_e, params_g)), i
    assert int(opt.state["step"]) == 5


def test_other_streams():
    """Calls on a side stream, their temporaries freed while they run, give the
    bits of calls on the default stream."""
    d = device()
    gen = torch.Generator().manual_seed(12)
    x, w, dy = dev(rand(gen, 600, 520)), dev(rand(gen, 333, 520)), dev(rand(gen, 600, 333))
    pre = dev(rand(gen, 600, 333))

    def work():
        y = vn.linear(x, w, activation="gelu")
        g = vn.linear_backward(dy, x, w, activation="gelu", pre=pre)
        n, mean, rstd = vn.layer_norm(y, stats=True)
        return (y, n) + g + vn.layer_norm_backward(dy, y, mean, rstd)

    want = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(work())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


# (rows, in, out) whose products have enough tiles of 256 rows: both tile widths, rows and columns off the tiles,
# one stage of k and several, k off the stages, also in the k-major operands of the gradients
WIDE = [(5000, 72, 2048), (6200, 200, 2056), (6144, 64, 2048), (2049, 328, 5000), (8200, 8, 1544),
        (2049, 136, 3080), (2300, 64, 3328)]


@pytest.mark.parametrize("shape", WIDE, ids=str)
def test_linear_wide(shape):
    print("linear wide", shape, flush=True)
    m, k, n = shape
    gen = torch.Generator().manual_seed(m + k + n)
    x, w, b, r = (rand(gen, m, k, dtype=BF16), rand(gen, n, k, scale=k ** -0.5, dtype=BF16), rand(gen, n, scale=0.3),
                  rand(gen, m, n, dtype=BF16))
    pre = torch.full((m, n), float("nan"), dtype=BF16, device=device())
    y = vn.linear(dev(x), dev(w), dev(b), activation="silu", residual=dev(r), pre=pre)
    want, z, ez = ref.linear(x, w, b, "silu", r)
    within(y, want, ref.linear_bound(want, z, ez, BF16, r), "y")
    within(pre, z, ez + ref.HALF[BF16] * z.abs() * 1.01 + 1e-30, "pre")
    assert torch.equal(vn.linear(dev(x), dev(w), dev(b), activation="silu", residual=dev(r)), y)
    # a NaN past the end of a row's k, in the row that follows, stays in its row
    x[m // 2, 0] = float("nan")
    y = vn.linear(dev(x), dev(w)).cpu()
    assert torch.isnan(y[m // 2]).all() and int(torch.isnan(y).sum()) == n


# (rows, in, out): the input gradient on wide tiles, then the weight's
@pytest.mark.parametrize("shape", [(5000, 2056, 72), (6200, 2048, 264), (77, 2056, 5000), (331, 2048, 6152), (64, 4096, 4096),
                                   (2049, 3080, 72), (100, 3080, 2056)],
                         ids=str)
def test_linear_backward_wide(shape):
    print("linear_backward wide", shape, flush=True)
    m, k, n = shape
    gen = torch.Generator().manual_seed(m + k + n)
    x, w, dy = rand(gen, m, k, dtype=BF16), rand(gen, n, k, scale=k ** -0.5, dtype=BF16), rand(gen, m, n, dtype=BF16)
    dx, dw, db = vn.linear_backward(dev(dy), dev(x), dev(w), weight_gradient_dtype=F32)
    az, aw, ax = dy.double().abs(), w.double().abs(), x.double().abs()
    want = dy.double() @ w.double()
    within(dx, want, (n + 12) * ref.U * (az @ aw) + ref.HALF[BF16] * 1.01 * want.abs() + 1e-30, "dx")
    want = dy.double().t() @ x.double()
    within(dw, want, (m + 12) * ref.U * (az.t() @ ax) + ref.HALF[F32] * 1.01 * want.abs() + 1e-30, "dw")
    within(db, dy.double().sum(0), (m + 4) * ref.U * az.sum(0) + 1e-30, "db")
    again = vn.linear_backward(dev(dy), dev(x), dev(w), weight_gradient_dtype=F32)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")], ids=str)
def test_layer_norm_larger_than_the_caches(types):
    """Tensors that go past the caches: the first and the last rows against 64 bits, the column sums against fp32's."""
    print("layer_norm large", types, flush=True)
    gt, dt = TYPES[types[0]], TYPES[types[1]]
    m, n = 40003, 2049
    gen = torch.Generator(device=device()).manual_seed(m)
    x, dy = (torch.randn(m, n, generator=gen, device=device()).to(t) for t in (dt, gt))
    w, b = torch.randn(n, generator=gen, device=device()), torch.randn(n, generator=gen, device=device())
    y, mean, rstd = vn.layer_norm(x, w, b, stats=True)
    dx, dw, db = vn.layer_norm_backward(dy, x, mean, rstd, w)
    cpu = lambda t, rows: t[rows].cpu()
    for rows in (slice(0, 5), slice(m - 5, m)):
        xr, wr, br = cpu(x, rows), w.cpu(), b.cpu()
        want = ref.layer_norm(xr, wr, br, 1e-5)
        within(cpu(y, rows), want[0], ref.layer_norm_bounds(xr, wr, br, *want, dt)[0], "y")
        mr, rr, dr = cpu(mean, rows), cpu(rstd, rows), cpu(dy, rows)
        want = ref.layer_norm_backward(dr, xr, mr, rr, wr)
        within(cpu(dx, rows), want[0], ref.layer_norm_backward_bounds(dr, xr, mr, rr, wr, want[0], 5, dt)[0], "dx")
    sums = [torch.zeros(n, dtype=torch.float64, device=device()) for _ in range(4)]
    for i in range(0, m, 4096):
        g, h = dy[i:i + 4096].double(), (x[i:i + 4096].double() - mean[i:i + 4096, None].double()) * rstd[i:i + 4096, None].double()
        for s, t in zip(sums, ((g * h), g, (g * h).abs(), g.abs())):
            s += t.sum(0)
    sums = [s.cpu() for s in sums]
    within(dw, sums[0], (m + 8) * ref.U * sums[2], "dweight")
    within(db, sums[1], (m + 8) * ref.U * sums[3], "dbias")
