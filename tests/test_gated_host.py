"""Host-side checks of the gated feed-forward block (no GPU): the 64-bit
reference against differences, refusals of the C ABI (fake addresses, refused
before any CUDA call) and of the binding."""
import pytest
import torch

import _block_ref as ref
import memory_efficient_activation_b200 as mea
from memory_efficient_activation_b200 import _capi, build
from test_norm_host import _FakeLib

P = 1 << 20
INV, UNS, OK = _capi.MEA_ERR_INVALID_ARG, _capi.MEA_ERR_UNSUPPORTED, _capi.MEA_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _capi.lib()


@pytest.mark.parametrize("act", ["sigmoid", "tanh", "gelu_erf", "gelu_tanh", "swish", "leaky_relu"])
def test_reference_gradient_against_differences(act):
    torch.manual_seed(5)
    M, N, K, D = 2, 3, 4, 5
    x, wg, wu, wd = (torch.randn(*s, dtype=torch.float64) for s in ((M, K), (N, K), (N, K), (D, N)))
    g, p = torch.randn(M, D, dtype=torch.float64), 1.3 if act == "swish" else 0.2

    def value():
        return float(((ref.gated_fwd(act, x, wg, wu, p)[2] @ wd.t()) * g).sum())

    gate, up, h = ref.gated_fwd(act, x, wg, wu, p)
    dz, h2 = ref.gated_bwd(act, g, wd, torch.cat([gate, up], 1), p)
    assert torch.allclose(h, h2, rtol=1e-14, atol=0)
    grads = ((x, dz @ torch.cat([wg, wu])), (wg, dz[:, :N].t() @ x), (wu, dz[:, N:].t() @ x), (wd, g.t() @ h))
    e = 1e-6
    for t, grad in grads:
        for i in range(t.numel()):
            old = float(t.view(-1)[i])
            t.view(-1)[i] = old + e
            a = value()
            t.view(-1)[i] = old - e
            b = value()
            t.view(-1)[i] = old
            # h^2 truncation and 2^-52 |value| / h rounding
            assert abs((a - b) / (2 * e) - float(grad.view(-1)[i])) < 1e-7


def test_gated_fwd_validation(lib):
    def fwd(act=6, M=4, N=16, K=8, x=P, wg=2 * P, wu=3 * P, z=4 * P, h=5 * P):
        return lib.mea_matmul_gated_act_fwd(act, M, N, K, x, wg, wu, 1.0, z, h, None)

    assert fwd(act=7) == INV and fwd(M=-1) == INV and fwd(N=-8) == INV and fwd(K=-8) == INV
    assert fwd(M=1 << 31) == UNS and fwd(N=1 << 31) == UNS and fwd(K=0) == UNS
    assert fwd(M=(1 << 31) - 1024) == UNS                      # a tile's last row number would pass 31 bits
    assert fwd(K=12) == UNS and fwd(N=12) == UNS
    assert fwd(x=None) == INV and fwd(wg=None) == INV and fwd(wu=None) == INV and fwd(z=None, h=None) == INV
    assert fwd(x=P + 8) == UNS and fwd(wg=2 * P + 2) == UNS and fwd(wu=3 * P + 4) == UNS
    assert fwd(z=4 * P + 8) == UNS and fwd(h=5 * P + 8) == UNS
    assert fwd(z=P) == INV and fwd(h=2 * P) == INV and fwd(h=3 * P + 16) == INV and fwd(h=4 * P + 64) == INV
    assert fwd(M=0) == OK and fwd(N=0) == OK


def test_gated_bwd_validation(lib):
    def bwd(act=6, M=4, N=16, K=8, g=P, w=2 * P, z=3 * P, dz=4 * P, h=5 * P):
        return lib.mea_matmul_gated_act_bwd(act, M, N, K, g, w, z, 1.0, dz, h, None)

    assert bwd(act=-1) == INV and bwd(M=-1) == INV and bwd(K=0) == UNS and bwd(K=4) == UNS and bwd(N=20) == UNS
    for k in ("g", "w", "z", "dz"):
        assert bwd(**{k: None}) == INV, k
    for i, k in enumerate(("g", "w", "z", "dz", "h")):
        assert bwd(**{k: (i + 1) * P + 2}) == UNS, k
    assert bwd(dz=P) == INV and bwd(dz=2 * P) == INV and bwd(dz=3 * P + 16) == INV
    assert bwd(h=P) == INV and bwd(h=3 * P) == INV and bwd(h=4 * P) == INV and bwd(h=2 * P + 32) == INV
    assert bwd(M=0) == OK and bwd(N=0) == OK


def test_binding_checks_with_stand_in_library(monkeypatch):
    fake = _FakeLib()
    monkeypatch.setattr(_capi, "lib", lambda: fake)
    monkeypatch.setattr(mea, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(mea, "_stream", lambda t: 0)
    bf = torch.bfloat16
    x, w, wd = torch.zeros(5, 8, dtype=bf), torch.zeros(32, 8, dtype=bf), torch.zeros(8, 16, dtype=bf)
    z, h = mea.matmul_gated_act_fwd("swish", x, w[:16], w[16:])
    assert z.shape == (5, 32) and h.shape == (5, 16)
    assert mea.matmul_gated_act_fwd("swish", x, w[:16], w[16:], want_z=False)[0] is None
    dz, hb = mea.matmul_gated_act_bwd("swish", x, wd, z, dz=z)
    assert dz is z and hb.shape == (5, 16)
    assert mea.matmul_gated_act_bwd("swish", x, wd, z, want_h=False)[1] is None
    n = len(fake.calls)
    for call in (
        lambda: mea.matmul_gated_act_fwd("swiss", x, w[:16], w[16:]),
        lambda: mea.matmul_gated_act_fwd("swish", x, w[:16], w[:8]),
        lambda: mea.matmul_gated_act_fwd("swish", x, wd, wd),
        lambda: mea.matmul_gated_act_fwd("swish", x[0], w[:16], w[16:]),
        lambda: mea.matmul_gated_act_fwd("swish", x, w[:16], w[16:], z=torch.empty(5, 16, dtype=bf)),
        lambda: mea.matmul_gated_act_fwd("swish", x, w[:16], w[16:], h=torch.empty(5, 16)),
        lambda: mea.matmul_gated_act_bwd("swish", x, wd, h),
        lambda: mea.matmul_gated_act_bwd("swish", x, w, z),
        lambda: mea.matmul_gated_act_bwd("swish", x, wd, z, dz=torch.empty(5, 32)),
        lambda: mea.MemoryEfficientGatedMLP(12, 16),
        lambda: mea.MemoryEfficientGatedMLP(8, 16, norm="batch"),
        lambda: mea.GatedMLPFunction.apply(x, w[:31], wd, None, None, "swish", 1.0, None, 1e-5),
    ):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        mea.matmul_gated_act_fwd("swish", x.float(), w[:16].float(), w[16:].float())
    assert len(fake.calls) == n


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(5, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mea.matmul_gated_act_fwd("swish", x, x, x)
    with pytest.raises(ValueError):
        mea.matmul_gated_act_bwd("swish", x, torch.zeros(8, 8, dtype=torch.bfloat16), torch.zeros(5, 16, dtype=torch.bfloat16))


def test_matmul_validation(lib):
    def mm(ta=0, tb=0, M=8, N=16, K=24, a=P, b=2 * P, c=3 * P):
        return lib.mea_matmul(ta, tb, M, N, K, a, b, c, None)

    assert mm(ta=1, tb=1) == UNS and mm(M=-1) == INV and mm(N=1 << 31) == UNS
    assert mm(a=None) == INV and mm(b=None) == INV and mm(c=None) == INV
    assert mm(a=P + 8) == UNS and mm(b=2 * P + 8) == UNS and mm(c=3 * P + 8) == UNS
    assert mm(N=12) == UNS and mm(K=12) == UNS and mm(ta=1, M=12) == UNS and mm(tb=1, K=12) == UNS
    assert mm(c=P) == INV and mm(c=2 * P + 16) == INV
    assert mm(M=0) == OK and mm(N=0) == OK


def test_matmul_binding_checks(monkeypatch):
    fake = _FakeLib()
    monkeypatch.setattr(_capi, "lib", lambda: fake)
    monkeypatch.setattr(mea, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(mea, "_stream", lambda t: 0)
    bf = torch.bfloat16
    a, b = torch.zeros(5, 8, dtype=bf), torch.zeros(8, 16, dtype=bf)
    assert mea.matmul(a, b).shape == (5, 16) and mea.matmul(b, b, True).shape == (16, 16)
    assert mea.matmul(a, torch.zeros(24, 8, dtype=bf), trans_b=True).shape == (5, 24)
    for call in (lambda: mea.matmul(a, a), lambda: mea.matmul(a, b, True), lambda: mea.matmul(a[0], b),
                 lambda: mea.matmul(a, b, out=torch.empty(5, 8, dtype=bf))):
        with pytest.raises(ValueError):
            call()
