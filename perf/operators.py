"""Cases of the normalisation and gated feed-forward operators, for timing and checking them.

Four operators and the block that a user builds from them:

  norm_fwd    y = gamma (x - mean) invstd + beta over the last axis (layer norm), or gamma x invstd (rms norm),
              with the row statistics that the backward pass keeps
  norm_bwd    dx, dgamma and dbeta from x, dy and the statistics
  gated_fwd   z = [x w_gate^T | x w_up^T], h = f(gate) up
  gated_bwd   d = g w_down; dz = [d up f'(gate) | d f(gate)] and the re-populated h = f(gate) up
  block       norm -> gated projections -> down projection, forward and backward, every gradient

`own` chooses between the plain form (elementary torch operations in 32 bits, rounded once at the end) and the
calls of this repository's package.
"""
import math

import torch

own = False

EPS = 1e-5
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the norms of eight decoding streams, one token each: latency
        {"name": "norm_fwd_decode", "op": "norm_fwd", "norm": "rms", "rows": 8, "C": 4096, "dtype": "bf16", "pdtype": "bf16"},
        # a training batch of 8 x 2048 tokens, d = 4096
        {"name": "norm_fwd_train", "op": "norm_fwd", "norm": "layer", "rows": 16384, "C": 4096, "dtype": "bf16", "pdtype": "f32"},
        # the same batch's backward pass
        {"name": "norm_bwd_train", "op": "norm_bwd", "norm": "layer", "rows": 16384, "C": 4096, "dtype": "bf16", "pdtype": "f32"},
        # full-precision channels-last feature maps of 1152 channels, an odd count of positions
        {"name": "norm_bwd_f32", "op": "norm_bwd", "norm": "layer", "rows": 12545, "C": 1152, "dtype": "f32", "pdtype": "f32"},
        # rows that are no multiple of a 16-byte vector
        {"name": "norm_bwd_odd_width", "op": "norm_bwd", "norm": "rms", "rows": 4099, "C": 1001, "dtype": "bf16", "pdtype": "bf16"},
        # one decoding stream: every weight read for a single token
        {"name": "gated_fwd_one_token", "op": "gated_fwd", "act": "swish", "M": 1, "N": 8192, "K": 4096, "z": False},
        # a batch of decoding streams
        {"name": "gated_fwd_decode", "op": "gated_fwd", "act": "swish", "M": 37, "N": 4096, "K": 4096, "z": False},
        # a prompt's chunk
        {"name": "gated_fwd_prompt", "op": "gated_fwd", "act": "gelu_tanh", "M": 411, "N": 8192, "K": 4096, "z": False},
        # a training micro-batch, z kept for the backward pass
        {"name": "gated_fwd_train", "op": "gated_fwd", "act": "swish", "M": 8192, "N": 8192, "K": 4096, "z": True},
        # a ragged micro-batch of a small model
        {"name": "gated_bwd_ragged", "op": "gated_bwd", "act": "gelu_erf", "M": 1023, "N": 2728, "K": 1024},
        # the training micro-batch's backward pass
        {"name": "gated_bwd_train", "op": "gated_bwd", "act": "swish", "M": 8192, "N": 8192, "K": 4096},
        # a whole pre-norm block's training step: output and every gradient
        {"name": "block_train", "op": "block", "norm": "rms", "act": "swish", "M": 4096, "N": 5464, "K": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult8(v):
    return max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "gated_fwd", "gated_bwd", "block"])
    act = rng.choice(["swish", "gelu_tanh", "gelu_erf", "relu"])
    if op in ("norm_fwd", "norm_bwd"):
        C = _log(rng, 64, 16384)
        if rng.random() < 0.75:
            C = _mult8(C)
        return {"op": op, "norm": rng.choice(["layer", "rms"]), "rows": _log(rng, 1, min(65536, (1 << 26) // C)), "C": C,
                "dtype": rng.choice(["bf16", "f32"]), "pdtype": rng.choice(["bf16", "f32"])}
    K, N = _mult8(_log(rng, 256, 4096)), _mult8(_log(rng, 256, 8192))
    if op == "gated_fwd":
        return {"op": op, "act": act, "M": _log(rng, 1, 8192), "N": N, "K": K, "z": rng.random() < 0.5}
    if op == "gated_bwd":
        return {"op": op, "act": act, "M": _log(rng, 16, 8192), "N": N, "K": K}
    # smooth activations: a jump of f' turns the rounding of the hidden layer into whole terms of the gradients
    act = rng.choice(["swish", "gelu_tanh", "gelu_erf"])
    return {"op": op, "norm": rng.choice(["layer", "rms"]), "act": act, "M": _log(rng, 64, 4096), "N": min(N, 4096), "K": min(K, 2048)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 12345)

    def normal(*shape, scale=1.0, shift=0.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale + shift).to(dtype)

    s = dict(case)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        dt, pdt, rows, C = _DTYPES[case["dtype"]], _DTYPES[case["pdtype"]], case["rows"], case["C"]
        # channels with offsets and scales of their own, as a residual stream has them
        chan = torch.rand(C, generator=gen, device="cuda") + 0.5
        off = torch.randn(C, generator=gen, device="cuda") * 0.5 + 0.25
        s["x"] = (torch.randn(rows, C, generator=gen, device="cuda") * chan + off).to(dt)
        s["gamma"] = normal(C, scale=0.2, shift=1.0, dtype=pdt)
        s["beta"] = normal(C, scale=0.1, dtype=pdt) if case["norm"] == "layer" else None
        if case["op"] == "norm_bwd":
            s["dy"] = normal(rows, C, dtype=dt)
            s["mean"], s["invstd"] = _row_stats(s["x"].float(), case["norm"])
        return s
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "gated_fwd":
        s["x"] = normal(M, K)
        s["w_gate"], s["w_up"] = normal(N, K, scale=K ** -0.5), normal(N, K, scale=K ** -0.5)
    elif case["op"] == "gated_bwd":
        s["g"], s["w_down"] = normal(M, K), normal(K, N, scale=K ** -0.5)
        s["z"] = normal(M, 2 * N)
    else:
        s["x"], s["g"] = normal(M, K).requires_grad_(), normal(M, K)
        s["gamma"] = normal(K, scale=0.2, shift=1.0).requires_grad_()
        s["beta"] = normal(K, scale=0.1).requires_grad_() if case["norm"] == "layer" else None
        s["w_gate_up"] = normal(2 * N, K, scale=K ** -0.5).requires_grad_()
        s["w_down"] = normal(K, N, scale=N ** -0.5).requires_grad_()
    return s


# ------------------------------------------------------------ plain forms

def _row_stats(x, norm):
    if norm == "rms":
        return None, torch.rsqrt((x * x).mean(-1) + EPS)
    mean = x.mean(-1)
    xc = x - mean[:, None]
    return mean, torch.rsqrt((xc * xc).mean(-1) + EPS)


def _xhat(x, mean, invstd):
    return (x if mean is None else x - mean[:, None]) * invstd[:, None]


def _normed(x, gamma, beta, mean, invstd):
    y = _xhat(x, mean, invstd) * gamma.float()
    return y if beta is None else y + beta.float()


def _norm_grads(x, dy, gamma, mean, invstd):
    xhat = _xhat(x, mean, invstd)
    gy = dy * gamma.float()
    rest = xhat * (gy * xhat).mean(-1, keepdim=True)
    if mean is not None:
        rest = rest + gy.mean(-1, keepdim=True)
    return (gy - rest) * invstd[:, None], (dy * xhat).sum(0), dy.sum(0)


def _act(act, g):
    """f(g) and f'(g)."""
    if act == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if act == "swish":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s + g * s * (1 - s)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    p = 0.5 * torch.erfc(-g / math.sqrt(2))
    return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _gated_grads(act, d, gate, up):
    f, df = _act(act, gate)
    return torch.cat([d * up * df, d * f], 1), f * up


def _plain(s):
    op = s["op"]
    if op == "norm_fwd":
        x = s["x"].float()
        mean, invstd = _row_stats(x, s["norm"])
        return {"y": _normed(x, s["gamma"], s["beta"], mean, invstd).to(s["x"].dtype), "mean": mean, "invstd": invstd}
    if op == "norm_bwd":
        dx, dgamma, dbeta = _norm_grads(s["x"].float(), s["dy"].float(), s["gamma"], s["mean"], s["invstd"])
        return {"dx": dx.to(s["x"].dtype), "dgamma": dgamma.to(s["gamma"].dtype),
                "dbeta": None if s["beta"] is None else dbeta.to(s["beta"].dtype)}
    if op == "gated_fwd":
        x = s["x"].float()
        gate, up = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
        h = (_act(s["act"], gate)[0] * up).bfloat16()
        return {"z": torch.cat([gate, up], 1).bfloat16() if s["z"] else None, "h": h}
    N = s["N"]
    if op == "gated_bwd":
        d, z = s["g"].float() @ s["w_down"].float(), s["z"].float()
        dz, h = _gated_grads(s["act"], d, z[:, :N], z[:, N:])
        return {"dz": dz.bfloat16(), "h": h.bfloat16()}
    with torch.no_grad():
        x, g, w1, w2 = s["x"].float(), s["g"].float(), s["w_gate_up"].float(), s["w_down"].float()
        mean, invstd = _row_stats(x, s["norm"])
        n = _normed(x, s["gamma"], s["beta"], mean, invstd)
        z = n @ w1.t()
        dz, h = _gated_grads(s["act"], g @ w2, z[:, :N], z[:, N:])
        dx, dgamma, dbeta = _norm_grads(x, dz @ w1, s["gamma"], mean, invstd)
        return {"out": (h @ w2.t()).bfloat16(), "dx": dx.bfloat16(), "dw_gate_up": (dz.t() @ n).bfloat16(),
                "dw_down": (g.t() @ h).bfloat16(), "dgamma": dgamma.bfloat16(),
                "dbeta": None if s["beta"] is None else dbeta.bfloat16()}


# ------------------------------------------------ the package's own calls

def _own(s):
    import memory_efficient_activation_b200 as mea

    op = s["op"]
    if op == "norm_fwd":
        y, mean, invstd = mea.norm_fwd(s["norm"], s["x"], s["gamma"], s["beta"], EPS)
        return {"y": y, "mean": mean, "invstd": invstd}
    if op == "norm_bwd":
        dx, dgamma, dbeta = mea.norm_bwd(s["norm"], s["x"], s["dy"], s["gamma"], s["mean"], s["invstd"],
                                         want_dbeta=s["beta"] is not None)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "gated_fwd":
        z, h = mea.matmul_gated_act_fwd(s["act"], s["x"], s["w_gate"], s["w_up"], want_z=s["z"])
        return {"z": z, "h": h}
    if op == "gated_bwd":
        dz, h = mea.matmul_gated_act_bwd(s["act"], s["g"], s["w_down"], s["z"])
        return {"dz": dz, "h": h}
    out = mea.GatedMLPFunction.apply(s["x"], s["w_gate_up"], s["w_down"], s["gamma"], s["beta"], s["act"], 1.0,
                                     s["norm"], EPS)
    leaves = [k for k in ("x", "w_gate_up", "w_down", "gamma", "beta") if s[k] is not None]
    grads = dict(zip(leaves, torch.autograd.grad(out, [s[k] for k in leaves], s["g"])))
    return {"out": out.detach(), "dx": grads["x"], "dw_gate_up": grads["w_gate_up"], "dw_down": grads["w_down"],
            "dgamma": grads["gamma"], "dbeta": grads.get("beta")}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    if case["op"] in ("norm_fwd", "norm_bwd"):
        e, p = (2 if case["dtype"] == "bf16" else 4), (2 if case["pdtype"] == "bf16" else 4)
        n, stats = case["rows"] * case["C"], (8 if case["norm"] == "layer" else 4) * case["rows"]
        vectors = (2 if case["norm"] == "layer" else 1) * case["C"] * p
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * n * e + vectors + stats, "flops": 8 * n}
        return {"bytes": 3 * n * e + case["C"] * p + vectors + stats, "flops": 14 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "gated_fwd":
        return {"bytes": 2 * (M * K + 2 * N * K + M * N * (3 if case["z"] else 1)), "flops": 4 * M * N * K}
    if case["op"] == "gated_bwd":
        return {"bytes": 2 * (M * K + K * N + 5 * M * N), "flops": 2 * M * N * K}
    return {"bytes": 2 * (4 * M * K + 6 * N * K + 2 * K), "flops": 18 * M * N * K}


# ------------------------------------------------ the definition in 64 bits

def _exact_act(act, g):
    """(f(g), f'(g)) in 64 bits: the normal distribution's cumulative function by erf, the logistic one by tanh."""
    if act == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g)), torch.where(g > 0, 1.0, 0.0).to(g.dtype)
    if act == "swish":
        s = torch.special.expit(g)
        return s * g, s * (1 + g * torch.special.expit(-g))
    if act == "gelu_tanh":
        a = (2 / math.pi) ** 0.5
        u = a * g + a * 0.044715 * g.pow(3)
        s = torch.special.expit(2 * u)                       # (1 + tanh u) / 2
        return g * s, s + g * 2 * s * torch.special.expit(-2 * u) * (a + 3 * a * 0.044715 * g.square())
    phi = torch.special.ndtr(g)
    return g * phi, torch.exp(-g.square() / 2) * g * (2 * math.pi) ** -0.5 + phi


def _exact_norm(x, gamma, beta, norm):
    mean = x.mean(1, keepdim=True) if norm == "layer" else x.new_zeros(x.shape[0], 1)
    invstd = ((x - mean).square().mean(1, keepdim=True) + EPS).pow(-0.5)
    y = (x - mean) * invstd * gamma.double()
    return (y if beta is None else y + beta.double()), mean, invstd


def _exact_norm_grads(x, dy, gamma, mean, invstd, norm):
    xhat = (x - mean) * invstd
    a = dy * gamma.double()
    C = x.shape[1]
    dx = a - xhat * ((a * xhat).sum(1, keepdim=True) / C)
    if norm == "layer":
        dx = dx - a.sum(1, keepdim=True) / C
    return dx * invstd, (xhat * dy).sum(0), dy.sum(0)


@torch.no_grad()
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        y, mean, invstd = _exact_norm(s["x"].double(), s["gamma"], s["beta"], s["norm"])
        return {"y": y, "mean": mean[:, 0] if s["norm"] == "layer" else None, "invstd": invstd[:, 0]}
    if op == "norm_bwd":
        mean = torch.zeros_like(s["invstd"]) if s["mean"] is None else s["mean"]
        dx, dgamma, dbeta = _exact_norm_grads(s["x"].double(), s["dy"].double(), s["gamma"], mean.double()[:, None],
                                              s["invstd"].double()[:, None], s["norm"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": None if s["beta"] is None else dbeta}
    if op == "gated_fwd":
        z = torch.mm(s["x"].double(), torch.cat([s["w_gate"], s["w_up"]]).double().t())
        return {"z": z if s["z"] else None, "h": _exact_act(s["act"], z[:, :s["N"]])[0] * z[:, s["N"]:]}
    N = case["N"]
    if op == "gated_bwd":
        z = s["z"].double()
        f, df = _exact_act(s["act"], z[:, :N])
        d = torch.mm(s["g"].double(), s["w_down"].double())
        return {"dz": torch.cat([df * z[:, N:] * d, f * d], 1), "h": z[:, N:] * f}
    x, g, w1, w2 = (s[k].detach().double() for k in ("x", "g", "w_gate_up", "w_down"))
    n, mean, invstd = _exact_norm(x, s["gamma"], s["beta"], s["norm"])
    z = torch.mm(n, w1.t())
    f, df = _exact_act(s["act"], z[:, :N])
    h, d = f * z[:, N:], torch.mm(g, w2)
    dz = torch.cat([df * z[:, N:] * d, f * d], 1)
    dx, dgamma, dbeta = _exact_norm_grads(x, torch.mm(dz, w1), s["gamma"], mean, invstd, s["norm"])
    return {"out": torch.mm(h, w2.t()), "dx": dx, "dw_gate_up": torch.mm(dz.t(), n), "dw_down": torch.mm(g.t(), h),
            "dgamma": dgamma, "dbeta": None if s["beta"] is None else dbeta}
