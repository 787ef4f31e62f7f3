"""Host-side checks of the row normalisation (no GPU): the 64-bit reference
against differences, the C ABI's refusals (fake addresses, refused before any
CUDA call) and the binding's argument checks."""
import os
import re

import pytest
import torch

import _block_ref as ref
import memory_efficient_activation_b200 as mea
from memory_efficient_activation_b200 import _capi, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20                                   # a fake, aligned device address
BF, F = _capi.MEA_BF16, _capi.MEA_F32


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _capi.lib()


def test_block_header_is_declared_and_exported(lib):
    src = open(os.path.join(ROOT, "include", "mea_block.h")).read()
    declared = re.findall(r"MEA_API\s+[\w\s\*]+?\b(mea_\w+)\s*\(", src)
    assert set(declared) == set(_capi.BLOCK_SIGNATURES) and len(declared) == len(set(declared))
    for fn in declared:
        assert hasattr(lib, fn), fn
    vals = dict(re.findall(r"\b(MEA_(?:LAYER|RMS)_NORM)\s*=\s*(\d+)", src))
    assert {k: int(v) for k, v in vals.items()} == {"MEA_LAYER_NORM": _capi.MEA_LAYER_NORM,
                                                    "MEA_RMS_NORM": _capi.MEA_RMS_NORM}


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_reference_gradient_against_differences(norm):
    torch.manual_seed(3)
    x, dy = torch.randn(3, 7, dtype=torch.float64), torch.randn(3, 7, dtype=torch.float64)
    gamma, beta = torch.randn(7, dtype=torch.float64), torch.randn(7, dtype=torch.float64)
    mean, invstd = ref.row_stats(x, norm, 1e-3)
    dx, dg, db = ref.norm_bwd(norm, x, dy, gamma, mean, invstd)
    h = 1e-6
    for t, grad in ((x, dx), (gamma, dg), (beta, db)):
        for i in range(t.numel()):
            old = float(t.view(-1)[i])
            t.view(-1)[i] = old + h
            up = float((ref.norm_fwd(norm, x, gamma, beta, 1e-3)[0] * dy).sum())
            t.view(-1)[i] = old - h
            dn = float((ref.norm_fwd(norm, x, gamma, beta, 1e-3)[0] * dy).sum())
            t.view(-1)[i] = old
            # central difference: h^2 truncation and 2^-52 / h rounding, both below 1e-7 here
            assert abs((up - dn) / (2 * h) - float(grad.view(-1)[i])) < 1e-7


def test_norm_fwd_validation(lib):
    def fwd(norm=0, dt=BF, pdt=F, rows=4, C=16, x=P, gamma=0, beta=0, eps=1e-5, y=2 * P, mean=3 * P, invstd=4 * P):
        return lib.mea_norm_fwd(norm, dt, pdt, rows, C, x, gamma or None, beta or None, eps, y, mean or None,
                                invstd or None, None)

    inv, uns = _capi.MEA_ERR_INVALID_ARG, _capi.MEA_ERR_UNSUPPORTED
    assert fwd(norm=2) == inv and fwd(dt=2) == inv and fwd(pdt=-1) == inv
    assert fwd(rows=-1) == inv and fwd(C=-1) == inv
    assert fwd(rows=1 << 31) == uns and fwd(C=1 << 31) == uns
    assert fwd(eps=-1.0) == inv and fwd(eps=float("nan")) == inv
    assert fwd(x=None) == inv and fwd(y=None) == inv
    assert fwd(y=P) == inv and fwd(y=P + 127) == inv                     # over x
    assert fwd(mean=P) == inv and fwd(invstd=2 * P) == inv               # statistics over x, over y
    assert fwd(gamma=2 * P) == inv and fwd(beta=4 * P) == inv
    assert fwd(rows=0) == _capi.MEA_OK and fwd(C=0) == _capi.MEA_OK      # nothing to do


def test_norm_bwd_validation(lib):
    need = lib.mea_norm_bwd_workspace_bytes(4, 16)
    assert need > 0

    def bwd(norm=0, dt=BF, pdt=F, rows=4, C=16, x=P, dy=2 * P, gamma=3 * P, mean=4 * P, invstd=5 * P, dx=6 * P,
            dgamma=7 * P, dbeta=8 * P, ws=9 * P, nb=need):
        return lib.mea_norm_bwd(norm, dt, pdt, rows, C, x, dy, gamma, mean, invstd, dx, dgamma, dbeta, ws, nb, None)

    inv, wsp = _capi.MEA_ERR_INVALID_ARG, _capi.MEA_ERR_WORKSPACE
    assert bwd(norm=-1) == inv and bwd(dt=7) == inv and bwd(pdt=2) == inv and bwd(rows=-2) == inv
    assert bwd(x=None) == inv and bwd(dy=None) == inv and bwd(dx=None) == inv
    assert bwd(mean=None) == inv and bwd(invstd=None) == inv
    assert bwd(dx=P + 2) == inv and bwd(dx=2 * P - 2) == inv             # partial overlaps
    assert bwd(ws=None) == wsp and bwd(nb=need - 1) == wsp and bwd(ws=9 * P + 8) == wsp
    assert bwd(dgamma=P) == inv and bwd(dbeta=3 * P) == inv and bwd(dbeta=7 * P) == inv and bwd(ws=6 * P) == inv
    assert bwd(dx=4 * P) == inv and bwd(dgamma=6 * P) == inv
    assert bwd(C=0) == _capi.MEA_OK


def test_workspace_is_a_function_of_the_shape(lib):
    ws = mea.norm_bwd_workspace_bytes
    assert ws(0, 16) == 0 and ws(16, 0) == 0 and ws(1 << 31, 8) == 0
    for rows, C in ((1, 1), (9, 33), (16384, 4096), (1 << 20, 144)):
        assert ws(rows, C) > 0 and ws(rows, C) % (8 * C) == 0
    # never more than 1024 rows in one fp32 sum
    assert ws(1 << 20, 144) >= (1 << 10) * 8 * 144


class _FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append(name)
            return 1 << 20 if name.endswith("_bytes") else 0
        return fn


def test_binding_checks_with_stand_in_library(monkeypatch):
    fake = _FakeLib()
    monkeypatch.setattr(_capi, "lib", lambda: fake)
    monkeypatch.setattr(mea, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(mea, "_stream", lambda t: 0)
    x = torch.zeros(2, 3, 16, dtype=torch.bfloat16)
    g, b = torch.ones(16), torch.zeros(16)
    y, mean, invstd = mea.norm_fwd("layer", x, g, b)
    assert y.shape == x.shape and mean.shape == invstd.shape == (2, 3) and mean.dtype == torch.float32
    assert mea.norm_fwd("rms", x, g.bfloat16())[1] is None
    assert mea.norm_fwd("layer", x, want_stats=False)[1:] == (None, None)
    dx, dg, db = mea.norm_bwd("layer", x, x, g, mean, invstd, want_dbeta=True)
    assert dx.shape == x.shape and dg.shape == db.shape == (16,) and dg.dtype == torch.float32
    assert mea.norm_bwd("rms", x, x, None, None, invstd)[1:] == (None, None)
    n = len(fake.calls)
    for call in (
        lambda: mea.norm_fwd("batch", x),
        lambda: mea.norm_fwd("layer", x, torch.ones(15)),
        lambda: mea.norm_fwd("layer", x, torch.ones(1, 16)),
        lambda: mea.norm_fwd("layer", x, g, b.bfloat16()),                 # two parameter types
        lambda: mea.norm_fwd("layer", x, out=torch.empty(6, 16)),          # fp32 out for bf16 x
        lambda: mea.norm_fwd("layer", torch.zeros(4, 0)),
        lambda: mea.norm_fwd("layer", torch.zeros(())),
        lambda: mea.norm_bwd("layer", x, x[:1], g, mean, invstd),
        lambda: mea.norm_bwd("layer", x, x.float(), g, mean, invstd),
        lambda: mea.norm_bwd("layer", x, x, g, None, invstd),
        lambda: mea.norm_bwd("layer", x, x, g, mean[:1], invstd),
        lambda: mea.norm_bwd("layer", x, x, g, mean, invstd.double()),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mea.norm_fwd("layer", x.half()), lambda: mea.norm_fwd("layer", x, g.double())):
        with pytest.raises(TypeError):
            call()
    assert [c for c in fake.calls[n:] if not c.endswith("_bytes")] == []


def test_binding_refuses_cpu_and_strided_tensors():
    with pytest.raises(ValueError):
        mea.norm_fwd("layer", torch.zeros(2, 8))
    with pytest.raises(ValueError):
        mea.norm_bwd("rms", torch.zeros(2, 8), torch.zeros(2, 8), None, None, torch.zeros(2))
    with pytest.raises(TypeError):
        mea.MemoryEfficientLayerNorm(8, dtype=torch.float16)
