"""The dense operators in 64 bits on the CPU, and the error that each output may
have: derived from the number of fp32 operations behind it, u = 2^-24 each, and
the rounding of its type (half a step)."""

import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope(z, name):
    z = z.detach().clone().requires_grad_(True)
    if name == "relu":
        return (z > 0).double()
    if name in (None, "none"):
        return torch.ones_like(z)
    act(z, name).sum().backward()
    return z.grad


def linear(x, w, b, name, r):
    """(y, z, bound of z's error before rounding): products and sums in fp32 lose
    at most a unit for each of the k + 8 operations; the three-way split of fp32
    operands drops less than 4 u of a product."""
    x, w = x.double(), w.double()
    z = x @ w.t()
    size = x.abs() @ w.abs().t()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    y = act(z, name)
    if r is not None:
        y = y + r.double()
    return y, z, (x.shape[-1] + 12) * U * size


def linear_bound(y, z, ez, out_dtype, r):
    """z's error through a slope of at most 1.13; the activation itself within 16
    units of z's size (erf, exp and a division); the residual's sum; the rounding."""
    extra = 0 if r is None else r.double().abs()
    return 1.13 * ez + 16 * U * (z.abs() + 1) + 2 * U * extra + HALF[out_dtype] * y.abs() * 1.01 + 1e-30


def layer_norm(x, w, b, eps):
    x = x.double()
    var, mean = torch.var_mean(x, dim=-1, correction=0)
    rstd = (var + eps).rsqrt()
    xhat = (x - mean[..., None]) * rstd[..., None]
    y = xhat if w is None else xhat * w.double()
    return (y if b is None else y + b.double()), mean, rstd


def layer_norm_bounds(x, w, b, y, mean, rstd, out_dtype):
    """Bounds of (y, mean, rstd).  A mean is a sum of depth d = 40 + n / 8192
    (runs of 8, the lanes' tree, the waves) over n; the variance the same over
    squares; a statistic's error enters y through x - mean and through rstd."""
    x = x.double()
    n = x.shape[-1]
    d = 40 + n / 8192
    e_mean = (d + 2) * U * x.abs().mean(-1)
    # the variance, relative: its sum, the rounded differences and their squares
    # (d + 4 units), and the mean's error, which enters squared; rstd takes half of
    # that, plus the root and the division
    e_rstd = rstd * ((d + 8) * U + (e_mean * rstd) ** 2)
    ww = 1.0 if w is None else w.double().abs()
    bb = 0.0 if b is None else b.double().abs()
    dev = (x - mean[..., None]).abs()
    e_xhat = rstd[..., None] * (e_mean[..., None] + U * dev) + dev * e_rstd[..., None] + 3 * U * dev * rstd[..., None]
    e_y = ww * e_xhat + 3 * U * (y.abs() + bb) + HALF[out_dtype] * y.abs() * 1.01 + 1e-30
    return e_y, e_mean + 1e-30, e_rstd + 1e-30


def layer_norm_backward(dy, x, mean, rstd, w):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[..., None], rstd.double()[..., None]
    n = x.shape[-1]
    xhat = (x - mean) * rstd
    g = dy if w is None else dy * w.double()
    a, b = g.mean(-1, keepdim=True), (g * xhat).mean(-1, keepdim=True)
    dx = rstd * (g - a - xhat * b)
    flat = lambda t: t.reshape(-1, n)
    return dx, flat(dy * xhat).sum(0), flat(dy).sum(0)


def layer_norm_backward_bounds(dy, x, mean, rstd, w, dx, rows_depth, dtype):
    """xhat within 3 u of |x - mean| rstd plus u |x|; the row sums as in the
    forward; the column sums of depth rows_depth."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[..., None], rstd.double()[..., None]
    n = x.shape[-1]
    d = 40 + n / 8192
    xhat = ((x - mean) * rstd).abs()
    e_h = 4 * U * xhat
    g = (dy if w is None else dy * w.double()).abs()
    e_a = (d + 4) * U * g.mean(-1, keepdim=True)
    sb = (g * xhat).mean(-1, keepdim=True)
    e_b = (d + 8) * U * sb
    e_dx = rstd * (4 * U * (g + g.mean(-1, keepdim=True) + xhat * sb) + e_a + xhat * e_b + e_h * sb)
    flat = lambda t: t.reshape(-1, n).abs().sum(0)
    return (e_dx + HALF[dtype] * dx.abs() * 1.01 + 1e-30, (rows_depth + 8) * U * flat(dy.abs() * xhat) + 1e-30,
            (rows_depth + 4) * U * flat(dy) + 1e-30)


# ---- AdamW, in the fp32 operations of its definition -----------------------

BLOCK = 128


def exponent(x):
    return (x.abs().view(torch.int32) >> 23).to(torch.int64)


def pow2(e):
    """2^e for a whole e in the normal range, exactly."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def fp8_encode(x, mant, bias, scale_log2, theta, keep_positive):
    a = x.abs() * pow2(-scale_log2)
    e = (exponent(a) - 127).clamp(min=1 - bias)
    q = torch.floor(a * pow2(mant - e) + theta).to(torch.int64)
    code = ((e + bias - 1) << mant) + q
    if keep_positive:
        code = torch.where((x > 0) & (code == 0), torch.ones_like(code), code)
    return (code + torch.where(x < 0, 128, 0)).to(torch.uint8)


def fp8_scale(x, top):
    """The scale byte of each block of 128: the largest magnitude at exponent top."""
    return (exponent(x.abs().view(-1, BLOCK).amax(1)) - top).clamp(min=1)


def adamw32(p, g, m, v, t, lr, betas, eps, wd, maximize=False):
    """One step in fp32, operation by operation (tensors of fp32 on the CPU)."""
    b1, b2 = betas
    g = -g if maximize else g
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    # (torch's fp32 square root on the CPU is not always the nearest; through 64 bits it is)
    denom = v.double().sqrt().float() * (1.0 / math.sqrt(1.0 - b2 ** t)) + eps
    p = p * (1.0 - lr * wd) - (m / denom) * (lr / (1.0 - b1 ** t))
    return p, m, v


def quantize_state(m, v, t, first):
    """(codes of m, codes of v, scales of m, scales of v) of one tensor's padded
    state, whose first element is number `first` of the flat state."""
    at = first + torch.arange(m.numel(), dtype=torch.int64)
    theta = (((t * 0x9E3779B9 + at * 0xC13FA9A9) & 0xFFFFFFFF) >> 12).float() * 2.0 ** -20
    sm, sv = fp8_scale(m, 7), fp8_scale(v, 14)
    per = lambda s: s.repeat_interleave(BLOCK) - 127
    return (fp8_encode(m, 3, 7, per(sm), theta, False), fp8_encode(v, 2, 15, per(sv), theta, True),
            sm.to(torch.uint8), sv.to(torch.uint8))


def dequantize(codes, scale, kind):
    return (codes.view(kind).float().view(-1, BLOCK) * torch.exp2(scale.float() - 127)[:, None]).view(-1)
