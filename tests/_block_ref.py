"""Plain 64-bit forms of the transformer-block operators (test helpers), and
the error bounds of their kernels, derived from the arithmetic."""
import math

import torch

U32 = 2.0 ** -24                       # half a step of fp32
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}     # half a step, relative to the value
TINY = 2.0 ** -126


def row_stats(x, norm, eps):
    x = x.double()
    mean = x.mean(-1) if norm == "layer" else torch.zeros(x.shape[:-1], dtype=torch.float64, device=x.device)
    return mean, 1 / torch.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)


def norm_fwd(norm, x, gamma, beta, eps):
    x = x.double()
    mean, invstd = row_stats(x, norm, eps)
    g = 1.0 if gamma is None else gamma.double()
    b = 0.0 if beta is None else beta.double()
    return (x - mean[..., None]) * invstd[..., None] * g + b, mean, invstd


def norm_bwd(norm, x, dy, gamma, mean, invstd):
    """dx, dgamma, dbeta from the statistics that the backward is given."""
    x, dy = x.double(), dy.double()
    m = mean.double()[..., None] if norm == "layer" else 0.0
    xhat = (x - m) * invstd.double()[..., None]
    a = dy if gamma is None else dy * gamma.double()
    dx = a - xhat * (a * xhat).mean(-1, keepdim=True)
    if norm == "layer":
        dx = dx - a.mean(-1, keepdim=True)
    C = x.shape[-1]
    return dx * invstd.double()[..., None], (dy * xhat).reshape(-1, C).sum(0), dy.reshape(-1, C).sum(0)


# Longest chain of fp32 additions behind a row sum: 7 within a 16-byte item,
# 16 items of a thread, 5 shuffles, 32 warps of a block.
ROW_CHAIN = 60


def norm_fwd_bounds(norm, x, gamma, beta, eps, dtype):
    """Bounds on |y - exact|, |mean - exact| and |invstd - exact|.

    mean: ROW_CHAIN additions of terms |x| / C, the division's product (2).
    var: the same chain, each term (x - mean)^2 with 3 roundings; a mean off by
    dm adds dm^2, which is carried as given.  rsqrtf errs by at most 2 steps.
    y: the error of the mean, of x - mean, of invstd and of two products and a
    sum, then one rounding to the storage type."""
    x = x.double()
    y, mean, invstd = norm_fwd(norm, x, gamma, beta, eps)
    g = torch.ones((), dtype=torch.float64, device=x.device) if gamma is None else gamma.double().abs()
    b = torch.zeros((), dtype=torch.float64, device=x.device) if beta is None else beta.double().abs()
    dm = (ROW_CHAIN + 3) * U32 * x.abs().mean(-1) if norm == "layer" else torch.zeros_like(invstd)
    xc = (x - mean[..., None]).abs()
    # each difference is off by dm and half a step of itself
    rel_var = (ROW_CHAIN + 6) * U32 + (dm * dm) * invstd ** 2
    dis = invstd * (0.5 * rel_var + rel_var ** 2 + 5 * U32)
    dxhat = invstd[..., None] * (dm[..., None] + U32 * xc) + xc * dis[..., None] + xc * invstd[..., None] * 2 * U32
    dy = g * dxhat + 3 * U32 * (g * xc * invstd[..., None] + b)
    return dy + HALF[dtype] * (y.abs() + dy) + TINY, dm + U32 * mean.abs() + TINY, dis


def norm_bwd_bounds(norm, x, dy, gamma, mean, invstd, dtype, pdtype):
    """Bounds on dx, dgamma and dbeta, the statistics taken as given.

    xhat has 3 roundings, a one; m1 and m2 are row sums of such terms; dx is
    formed with 4 more.  A column sum adds at most 1024 terms in fp32 (at most
    128 in one thread's sequence, then 8 in order; 144 covers both and the
    terms' own roundings; where one thread takes all 1024 rows of its share the
    chain is 1024), the rest in fp64, then one rounding."""
    x, dy = x.double(), dy.double()
    m = mean.double()[..., None] if norm == "layer" else 0.0
    is_ = invstd.double()[..., None]
    xhat = ((x - m) * is_).abs()
    a = (dy if gamma is None else dy * gamma.double()).abs()
    dxh = 3 * U32 * xhat
    dm1 = (ROW_CHAIN + 3) * U32 * a.mean(-1, keepdim=True) if norm == "layer" else 0.0
    dm2 = (ROW_CHAIN + 7) * U32 * (a * xhat).mean(-1, keepdim=True)
    m2 = (a * xhat).mean(-1, keepdim=True)
    m1 = a.mean(-1, keepdim=True) if norm == "layer" else 0.0
    ref = norm_bwd(norm, x, dy, gamma, mean, invstd)
    e = is_ * (dm1 + xhat * dm2 + dxh * m2 + 6 * U32 * (a + m1 + xhat * m2))
    C = x.shape[-1]
    rows = x.numel() // C
    chain = min(1024, rows) + 16
    tg, tb = (dy.abs() * xhat).reshape(-1, C).sum(0), dy.abs().reshape(-1, C).sum(0)
    eg, eb = chain * U32 * tg, chain * U32 * tb
    return (e + HALF[dtype] * (ref[0].abs() + e) + TINY, eg + HALF[pdtype] * (ref[1].abs() + eg) + TINY,
            eb + HALF[pdtype] * (ref[2].abs() + eb) + TINY)


def act(name, z, param=1.0):
    """f(z) and f'(z) in 64 bits."""
    z = z.double()
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).double()
    if name == "leaky_relu":
        return torch.where(z > 0, z, param * z), torch.where(z > 0, 1.0, param).double()
    if name == "sigmoid":
        s = torch.special.expit(z)
        return s, s * torch.special.expit(-z)
    if name == "tanh":
        return torch.tanh(z), 4 * torch.special.expit(2 * z) * torch.special.expit(-2 * z)
    if name == "swish":
        s, c = torch.special.expit(param * z), torch.special.expit(-param * z)
        return z * s, s + param * z * s * c
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        u2 = 2 * k * (z + 0.044715 * z ** 3)
        s, c = torch.special.expit(u2), torch.special.expit(-u2)
        return z * s, s + z * s * c * 2 * k * (1 + 3 * 0.044715 * z * z)
    assert name == "gelu_erf", name
    p = 0.5 * torch.erfc(-z / math.sqrt(2))      # not 1 + erf, which is zero below -8.3
    return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def gated_fwd(name, x, w_gate, w_up, param=1.0):
    gate, up = x.double() @ w_gate.double().t(), x.double() @ w_up.double().t()
    return gate, up, act(name, gate, param)[0] * up


def gated_bwd(name, g, w_down, z, param=1.0):
    """dz = [d up f'(gate) | d f(gate)], h = f(gate) up, d = g w_down."""
    N = w_down.shape[1]
    gate, up = z.double()[:, :N], z.double()[:, N:]
    d = g.double() @ w_down.double()
    f, df = act(name, gate, param)
    return torch.cat([d * up * df, d * f], 1), f * up


def assert_within(got, ref, bound, what):
    got, ref, bound = got.double(), ref.double(), bound.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err = (got - ref).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for "
                             f"{float(ref[i])}, error {float(err[i]):.3g} over {float(bound[i]):.3g}")


# |f'| never exceeds this (sigmoid's quarter, the GELUs' and Swish's overshoot)
LIPSCHITZ = {"relu": 1.0, "leaky_relu": 1.0, "sigmoid": 0.25, "tanh": 1.0, "gelu_erf": 1.1290, "gelu_tanh": 1.1290,
             "swish": 1.0999}
# f and f' as the bf16 kernels evaluate them: tanh.approx is good to 2^-11, every other form to better than 2^-12;
# next to a zero of f' (whose terms cancel) an absolute 2^-20 on top.
F_REL, DF_ABS = 2.0 ** -11, 2.0 ** -20


def _acc(x, w, K):
    """Bound on an fp32 accumulation over k in any order: K additions, each off
    by at most a step of a partial sum below S = sum |x w|."""
    return K * 2.0 ** -23 * (x.double().abs() @ w.double().abs())


def gated_fwd_bounds(name, x, w_gate, w_up, param=1.0):
    """Bounds on z = [gate | up] and h: the accumulations' errors carried
    through f (Lipschitz) and the product, f's evaluation, one rounding."""
    K = x.shape[1]
    gate, up, h = gated_fwd(name, x, w_gate, w_up, param)
    eg, eu = _acc(x, w_gate.t(), K), _acc(x, w_up.t(), K)
    f = act(name, gate, param)[0].abs()
    ef = LIPSCHITZ[name] * eg + F_REL * f
    eh = ef * (up.abs() + eu) + f * eu + 2 * U32 * h.abs()
    half = HALF[torch.bfloat16]
    z, ez = torch.cat([gate, up], 1).abs(), torch.cat([eg, eu], 1)
    return ez + half * (z + ez) + TINY, eh + half * (h.abs() + eh) + TINY * (1 + up.abs())


def gated_bwd_bounds(name, g, w_down, z, param=1.0):
    """Bounds on dz and h for a z taken as given."""
    N, K = w_down.shape[1], g.shape[1]
    gate, up = z.double()[:, :N], z.double()[:, N:].abs()
    ed = _acc(g, w_down, K)
    d = (g.double() @ w_down.double()).abs()
    f, df = (v.abs() for v in act(name, gate, param))
    eg = ed * up * df + (d + ed) * up * (F_REL * df + DF_ABS)
    eu = ed * f + (d + ed) * F_REL * f
    ref, h = gated_bwd(name, g, w_down, z, param)
    half = HALF[torch.bfloat16]
    e = torch.cat([eg, eu], 1)
    eh = F_REL * h.abs()
    return (e + half * (ref.abs() + e) + TINY * (1 + torch.cat([d * up, d], 1)),
            eh + half * (h.abs() + eh) + TINY * (1 + up))


def assert_close_overall(got, ref, what, parts=1):
    """Norm of the error at most half a bf16 step of the norm of the result
    (the rms of a rounding is below half a step), times `parts` roundings: a
    fault in the order of operands or of K steps breaks every element."""
    err, norm = float((got.double() - ref).norm()), float(ref.norm())
    assert err <= parts * HALF[torch.bfloat16] * norm + TINY, (what, err / max(norm, TINY))
