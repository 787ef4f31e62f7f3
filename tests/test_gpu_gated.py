"""GPU parity of the gated feed-forward kernels (mea_matmul_gated_act_fwd /
_bwd) and of the block built on them with their 64-bit forms; the bounds are
derived in _block_ref.py."""
import pytest
import torch

import _block_ref as ref
import memory_efficient_activation_b200 as mea
from memory_efficient_activation_b200 import _capi

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ACTS = ["relu", "leaky_relu", "sigmoid", "tanh", "gelu_erf", "gelu_tanh", "swish"]


def _p(act):
    return {"leaky_relu": 0.01, "swish": 1.25}.get(act, 1.0)


def _normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(BF)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _fwd(act, M, N, K, seed, want_z=True, want_h=True):
    g = _gen(seed)
    x, wg, wu = _normal(g, M, K), _normal(g, N, K, scale=K ** -0.5), _normal(g, N, K, scale=K ** -0.5)
    z, h = mea.matmul_gated_act_fwd(act, x, wg, wu, _p(act), want_z=want_z, want_h=want_h)
    gate, up, rh = ref.gated_fwd(act, x, wg, wu, _p(act))
    bz, bh = ref.gated_fwd_bounds(act, x, wg, wu, _p(act))
    if want_z:
        rz = torch.cat([gate, up], 1)
        ref.assert_within(z, rz, bz, "z")
        ref.assert_close_overall(z, rz, "z")
    else:
        assert z is None
    if want_h:
        ref.assert_within(h, rh, bh, "h")
        ref.assert_close_overall(h, rh, "h")
    else:
        assert h is None
    return x, wg, wu, z, h


def _bwd(act, M, N, K, seed, want_h=True):
    g = _gen(seed)
    dout, wd, z = _normal(g, M, K), _normal(g, K, N, scale=K ** -0.5), _normal(g, M, 2 * N)
    dz, h = mea.matmul_gated_act_bwd(act, dout, wd, z, _p(act), want_h=want_h)
    rdz, rh = ref.gated_bwd(act, dout, wd, z, _p(act))
    bdz, bh = ref.gated_bwd_bounds(act, dout, wd, z, _p(act))
    ref.assert_within(dz, rdz, bdz, "dz")
    ref.assert_close_overall(dz, rdz, "dz")
    if want_h:
        ref.assert_within(h, rh, bh, "h")
    return dout, wd, z, dz, h


@pytest.fixture(autouse=True)
def no_expired_waits():
    yield
    assert _capi.lib().mea_matmul_error_word(1) == 0


@pytest.mark.parametrize("M,N,K", [(256, 128, 64), (256, 256, 128), (512, 256, 512)])
def test_gated_one_tile(M, N, K):
    _fwd("swish", M, N, K, 1)
    _bwd("swish", M, N, K, 2)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 136, 200), (33, 120, 72), (257, 264, 136)])
def test_gated_activations(act, M, N, K):
    _fwd(act, M, N, K, M + N + K)
    _bwd(act, M, N, K, M + N + K + 1)


@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 96, 127, 128, 129, 200, 255, 256, 257, 411, 1023])
@pytest.mark.parametrize("N,K", [(8, 8), (24, 1032), (328, 64), (1032, 520)])
def test_gated_token_counts(M, N, K):
    _fwd("swish", M, N, K, M * 7 + N)
    _bwd("gelu_tanh", M, N, K, M * 7 + N + 1)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (5, 8192, 1024), (37, 4096, 4096), (130, 2728, 1024), (300, 16384, 512),
                                   (4099, 1032, 136), (2500, 5464, 264), (9000, 520, 72)])
def test_gated_many_tiles(M, N, K):
    """Both accumulators in turn, groups of row tiles cut short, every pair at
    work."""
    _fwd("swish", M, N, K, M + N)
    _bwd("swish", M, N, K, M + N + 1)


@pytest.mark.parametrize("M,N,K", [(64, 9608, 72), (65, 9608, 72), (100, 9408, 72), (129, 4808, 72), (200, 4664, 72)])
def test_gated_either_side_of_the_kernels_border(M, N, K):
    """Few tokens with many and with few column tiles: both kernels."""
    _fwd("gelu_erf", M, N, K, M + N)


@pytest.mark.parametrize("act,param", [(a, _p(a)) for a in ACTS] + [("swish", 1.0), ("swish", -0.7), ("swish", 0.0)])
def test_gated_bwd_extreme_gates(act, param):
    """Gates far out on both sides, and a dense band around the zeros of f'."""
    g = _gen(16)
    M, N, K = 40, 264, 72
    dout, wd = _normal(g, M, K), _normal(g, K, N, scale=K ** -0.5)
    gate = torch.empty(M, N, device="cuda")
    gate[:20] = torch.linspace(-1.6, -0.6, 20 * N, device="cuda").view(20, N)
    far = torch.tensor([0.0, 5.0, 12.0, 13.5, 20.0, 60.0, 88.0, 100.0, 1e3, 1e6, 1e15, 1e30], device="cuda")
    gate[20:] = torch.cat([far, -far]).repeat(20 * N // 24)[:20 * N].view(20, N)
    z = torch.cat([gate, torch.ones(M, N, device="cuda")], 1).to(BF)
    dz, h = mea.matmul_gated_act_bwd(act, dout, wd, z, param)
    rdz, rh = ref.gated_bwd(act, dout, wd, z, param)
    bdz, bh = ref.gated_bwd_bounds(act, dout, wd, z, param)
    ref.assert_within(dz, rdz, bdz, "dz")
    ref.assert_within(h, rh, bh, "h")


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gated_outputs_skipped(M):
    a = _fwd("gelu_tanh", M, 264, 136, 5)
    b = _fwd("gelu_tanh", M, 264, 136, 5, want_z=False)
    c = _fwd("gelu_tanh", M, 264, 136, 5, want_h=False)
    assert torch.equal(a[4], b[4]) and torch.equal(a[3], c[3])
    d = _bwd("gelu_tanh", M, 264, 136, 6)
    e = _bwd("gelu_tanh", M, 264, 136, 6, want_h=False)
    assert torch.equal(d[3], e[3]) and e[4] is None


@pytest.mark.parametrize("M,N,K", [(1, 1032, 520), (70, 1032, 520), (1500, 1032, 520)])
def test_gated_in_place_halves_and_determinism(M, N, K):
    x, wg, wu, z, h = _fwd("swish", M, N, K, 7)
    w = torch.cat([wg, wu])
    for _ in range(3):
        z2, h2 = mea.matmul_gated_act_fwd("swish", x, w[:N], w[N:], _p("swish"))
        assert torch.equal(z, z2) and torch.equal(h, h2)
    zs, hs = mea.matmul_gated_act_fwd("swish", x, wg, wg, _p("swish"))          # one matrix for both
    assert torch.equal(zs[:, :N], zs[:, N:])
    g, wd, zin, dz, hb = _bwd("swish", M, N, K, 8)
    zc = zin.clone()
    dz2, hb2 = mea.matmul_gated_act_bwd("swish", g, wd, zc, _p("swish"), dz=zc)
    assert dz2 is zc and torch.equal(dz, dz2) and torch.equal(hb, hb2)


@pytest.mark.parametrize("M,N,K", [(1, 136, 72), (33, 136, 72), (129, 136, 72), (259, 264, 72)])
def test_gated_writes_nothing_beyond_its_outputs(M, N, K):
    def guarded(rows, cols):
        buf = torch.full((rows * cols + 128,), 7.0, dtype=BF, device="cuda")
        return buf, buf[64:64 + rows * cols].view(rows, cols)

    g = _gen(9)
    x, wg, wu = _normal(g, M, K), _normal(g, N, K), _normal(g, N, K)
    bz, z = guarded(M, 2 * N)
    bh, h = guarded(M, N)
    mea.matmul_gated_act_fwd("swish", x, wg, wu, z=z, h=h)
    bd, dz = guarded(M, 2 * N)
    bi, hi = guarded(M, N)
    mea.matmul_gated_act_bwd("swish", _normal(g, M, K), _normal(g, K, N), z, dz=dz, h=hi)
    for b in (bz, bh, bd, bi):
        assert (b[:64] == 7).all() and (b[-64:] == 7).all()


@pytest.mark.parametrize("M", [3, 200, 700])
def test_gated_bad_values_stay_in_their_row(M):
    x, wg, wu, z, h = _fwd("swish", M, 264, 136, 10)
    x2 = x.clone()
    x2[1, 4] = float("nan")
    z2, h2 = mea.matmul_gated_act_fwd("swish", x2, wg, wu, _p("swish"))
    keep = [i for i in range(M) if i != 1]
    assert torch.equal(z[keep], z2[keep]) and torch.equal(h[keep], h2[keep]) and z2[1].isnan().all()


def test_gated_no_tokens():
    w = torch.zeros(16, 8, dtype=BF, device="cuda")
    z, h = mea.matmul_gated_act_fwd("swish", torch.empty(0, 8, dtype=BF, device="cuda"), w, w)
    assert z.shape == (0, 32) and h.shape == (0, 16)
    dz, h = mea.matmul_gated_act_bwd("swish", torch.empty(0, 8, dtype=BF, device="cuda"), w.t().contiguous(), z)
    assert dz.shape == (0, 32) and h.shape == (0, 16)


@pytest.mark.parametrize("M", [2, 150, 900])
def test_gated_in_a_graph_and_on_two_streams(M):
    g = _gen(11)
    N, K = 520, 264
    x, wg, wu, wd = _normal(g, M, K), _normal(g, N, K), _normal(g, N, K), _normal(g, K, N)

    def step():
        z, h = mea.matmul_gated_act_fwd("swish", x, wg, wu)
        return (z, h) + mea.matmul_gated_act_bwd("swish", x, wd, z)

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(step())
    torch.cuda.synchronize()
    for o in [out] + outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def _block_ref(x, g, m):
    """The block in 64 bits: out and the gradients of x, w_gate_up, w_down,
    gamma, beta."""
    x, g = x.double().reshape(-1, x.shape[-1]), g.double().reshape(-1, g.shape[-1])
    w1, w2 = m.w_gate_up.detach().double(), m.w_down.detach().double()
    H = w2.shape[1]
    gamma = None if m.gamma is None else m.gamma.detach()
    if m.norm is None:
        n = x
    else:
        n, mean, invstd = ref.norm_fwd(m.norm, x, gamma, None if m.beta is None else m.beta.detach(), m.eps)
    gate, up, h = ref.gated_fwd(m.act, n, w1[:H], w1[H:], m.param)
    dz, _ = ref.gated_bwd(m.act, g, w2, torch.cat([gate, up], 1), m.param)
    grads = {"w_gate_up": dz.t() @ n, "w_down": g.t() @ h}
    dn = dz @ w1
    if m.norm is None:
        grads["x"] = dn
    else:
        grads["x"], grads["gamma"], grads["beta"] = ref.norm_bwd(m.norm, x, dn, gamma, mean, invstd)
    return h @ w2.t(), grads


@pytest.mark.parametrize("norm", [None, "layer", "rms"])
@pytest.mark.parametrize("act", ["swish", "gelu_erf"])
@pytest.mark.parametrize("batch,D,H", [((3, 50), 136, 264), ((2, 300), 256, 512), ((1, 1), 64, 128)])
def test_gated_block(norm, act, batch, D, H):
    """Norm, projections, product, down projection and the backward through
    all of them, as a model runs them.  Roundings to bf16 on the way to each
    result, each at most half a step of its own tensor and independent of the
    others': out 3 (n, h, out); dx 7 (n, z, dz, dn, dx and d gate's two factors
    z); weights as many: 8 half steps of the norm bound every one."""
    torch.manual_seed(12)
    m = mea.MemoryEfficientGatedMLP(D, H, act, norm=norm).cuda()
    with torch.no_grad():
        for p in (m.gamma, m.beta):
            if p is not None:
                p.add_(torch.randn_like(p) * 0.2)
    x = torch.randn(*batch, D, device="cuda").to(BF).requires_grad_()
    g = torch.randn(*batch, D, device="cuda").to(BF)
    out = m(x)
    out.backward(g)
    want, grads = _block_ref(x.detach(), g, m)
    ref.assert_close_overall(out.detach().reshape(-1, D), want, "out", 4)
    got = {"x": x.grad.reshape(-1, D), **{k: p.grad for k, p in m.named_parameters()}}
    assert set(got) == {k for k in grads if not (k == "beta" and norm == "rms")}
    for k, v in got.items():
        ref.assert_close_overall(v, grads[k], k, 8)
    with torch.no_grad():
        assert torch.equal(m(x), out)
    # frozen weights: only the input's gradient
    x2 = x.detach().clone().requires_grad_()
    m.requires_grad_(False)
    m(x2).backward(g)
    assert torch.equal(x2.grad, x.grad)


def test_gated_block_keeps_its_input_statistics_and_z_only():
    torch.manual_seed(14)
    m = mea.MemoryEfficientGatedMLP(256, 1024, norm="rms").cuda()
    x = torch.randn(2048, 256, device="cuda").to(BF).requires_grad_()
    m(x).sum().backward()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    out = m(x)
    kept = torch.cuda.memory_allocated() - before
    z, stats = 2048 * 2048 * 2, 2048 * 4
    assert kept <= z + stats + out.numel() * 2 + 4096, kept


def test_gated_block_training_step_in_a_graph():
    """Forward and backward captured; no eager graph of the same leaves is
    alive then (autograd ties a leaf's accumulation to the stream of the graph
    that made it, and would break the capture)."""
    torch.manual_seed(15)
    m = mea.MemoryEfficientGatedMLP(64, 128, norm="layer").cuda()
    x = torch.randn(96, 64, device="cuda").to(BF)
    g = torch.randn(96, 64, device="cuda").to(BF)
    params = list(m.parameters())

    def step():
        return torch.autograd.grad(m(x), params, g)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("M,N,K", [(8, 8, 8), (256, 256, 64), (264, 520, 72), (2056, 1032, 136), (4104, 2728, 264),
                                   (1, 40, 16), (37, 264, 200), (1000, 328, 1)])
def test_matmul_layouts(ta, tb, M, N, K):
    """Plain product in the three layouts, odd M (K with the first operand
    transposed): K additions in fp32 and one rounding."""
    if ta:
        M, K = -(-M // 8) * 8, K - 7 if K > 8 else K
    elif K % 8:
        K = 8
    g = _gen(M + N + K)
    a = _normal(g, *((K, M) if ta else (M, K)))
    b = _normal(g, *((N, K) if tb else (K, N)))
    c = mea.matmul(a, b, ta, tb)
    A, B = a.t() if ta else a, b.t() if tb else b
    want = A.double() @ B.double()
    e = K * 2.0 ** -23 * (A.double().abs() @ B.double().abs())
    ref.assert_within(c, want, e + 2.0 ** -8 * (want.abs() + e) + ref.TINY, "c")
    ref.assert_close_overall(c, want, "c")
    assert torch.equal(c, mea.matmul(a, b, ta, tb))


def test_matmul_empty_and_guarded():
    a, b = torch.empty(0, 16, dtype=BF, device="cuda"), torch.ones(16, 24, dtype=BF, device="cuda")
    assert mea.matmul(a, b).shape == (0, 24)
    z = mea.matmul(torch.empty(0, 16, dtype=BF, device="cuda"), torch.empty(0, 24, dtype=BF, device="cuda"), True)
    assert z.shape == (16, 24) and not z.any()
    buf = torch.full((37 * 40 + 128,), 7.0, dtype=BF, device="cuda")
    mea.matmul(torch.ones(37, 16, dtype=BF, device="cuda"), torch.ones(16, 40, dtype=BF, device="cuda"),
               out=buf[64:64 + 37 * 40].view(37, 40))
    assert (buf[:64] == 7).all() and (buf[-64:] == 7).all() and (buf[64:-64] == 16).all()


@pytest.mark.parametrize("norm", [None, "layer"])
def test_gated_block_of_no_tokens(norm):
    m = mea.MemoryEfficientGatedMLP(64, 128, norm=norm).cuda()
    x = torch.empty(0, 64, dtype=BF, device="cuda", requires_grad=True)
    out = m(x)
    out.backward(torch.empty_like(out))
    assert out.shape == (0, 64) and x.grad.shape == (0, 64)
    assert all(p.grad.shape == p.shape and not p.grad.any() for p in m.parameters())


@pytest.mark.parametrize("K", [72, 1288])
@pytest.mark.parametrize("alpha", [1.0, 1.25, 2.0, -2.0, 0.0])
def test_gated_bwd_swish_of_the_largest_gates(alpha, K):
    """alpha times the gate overflows fp32 or is infinite: f' is 1 or 0 there
    (as it is at 1e30 already), in the 256-row and in the few-token kernel.
    Where alpha times the gate is no number (0 times infinity) neither is f'."""
    g = _gen(17)
    M, N = 40, 264
    dout, wd = _normal(g, M, K), _normal(g, K, N, scale=K ** -0.5)
    far = torch.tensor([1e30, 1e37, 3e38, float("inf"), 2.0], device="cuda")
    gate = torch.cat([far, -far, far[:3]]).repeat(M * N // 13 + 1)[:M * N].view(M, N)
    up = torch.ones(M, N, device="cuda")
    dz, _ = mea.matmul_gated_act_bwd("swish", dout, wd, torch.cat([gate, up], 1).to(BF), alpha)
    z = torch.cat([gate.clamp(-1e30, 1e30), up], 1).to(BF)
    want, bound = ref.gated_bwd("swish", dout, wd, z, alpha)[0][:, :N], ref.gated_bwd_bounds("swish", dout, wd, z, alpha)[0][:, :N]
    number = ~(alpha * gate).isnan()
    ref.assert_within(dz[:, :N][number], want[number], bound[number], "d gate")
    assert dz[:, :N][~number].isnan().all()


@pytest.mark.parametrize("norm", [None, "rms"])
def test_gated_block_of_slices_off_a_16_byte_boundary(norm):
    """Input and gradient that start at odd elements of flat buffers (the
    gradient as the backward of a concatenation hands it over)."""
    torch.manual_seed(18)
    m = mea.MemoryEfficientGatedMLP(64, 128, norm=norm).cuda()
    x, g = torch.randn(7 * 64 + 1, device="cuda").to(BF), torch.randn(7 * 64 + 3, device="cuda").to(BF)
    whole, flat = x[1:].view(7, 64).clone().requires_grad_(), x.clone().requires_grad_()
    want = m(whole)
    want.backward(g[3:].view(7, 64).clone())
    grads = [p.grad for p in m.parameters()]
    m.zero_grad()
    out = m(flat[1:].view(7, 64))
    torch.cat([x[:3], out.flatten()]).backward(g)
    assert torch.equal(out, want) and torch.equal(flat.grad[1:].view(7, 64), whole.grad)
    assert all(torch.equal(p.grad, w) for p, w in zip(m.parameters(), grads))
    with torch.no_grad():
        assert torch.equal(m(x[1:].view(7, 64)), want)


def _matmul_check(ta, tb, M, N, K):
    g = _gen(M + N + K)
    a = _normal(g, *((K, M) if ta else (M, K)))
    b = _normal(g, *((N, K) if tb else (K, N)))
    c = mea.matmul(a, b, ta, tb)
    A, B = a.t() if ta else a, b.t() if tb else b
    want = A.double() @ B.double()
    e = K * 2.0 ** -23 * (A.double().abs() @ B.double().abs())
    ref.assert_within(c, want, e + 2.0 ** -8 * (want.abs() + e) + ref.TINY, "c")
    ref.assert_close_overall(c, want, "c")
    assert torch.equal(c, mea.matmul(a, b, ta, tb))


WIDTHS = [(4096, 4096, 136), (2296, 2040, 200), (8192, 5464, 64),      # 256 columns: 224 would take a round more
          (4096, 2736, 72), (2048, 5464, 72)]                          # 224 columns


@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("M,N,K", WIDTHS)
def test_matmul_of_both_tile_widths(ta, tb, M, N, K):
    _matmul_check(ta, tb, M, N, K)


@pytest.mark.parametrize("M,N,K", WIDTHS)
def test_gated_bwd_of_both_tile_widths(M, N, K):
    _bwd("gelu_tanh", M, N, K, M + N)


# Sums of 20 K blocks (1217 terms) and more over few tiles: K shared out over a
# cluster of two, four or eight blocks, one or two of them on an SM.

@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("M,N,K", [(8, 8, 1288), (1, 136, 4104), (128, 128, 8192), (200, 264, 6152), (264, 520, 1400),
                                   (512, 1032, 2056), (40, 1032, 2049), (1032, 264, 4099), (2048, 1032, 3080)])
def test_matmul_of_shared_sums(ta, tb, M, N, K):
    _matmul_check(ta, tb, -(-M // 8) * 8 if ta else M, N, K if ta else K // 8 * 8)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 264, 1288), (100, 264, 1288), (200, 520, 2056), (256, 136, 4104)])
def test_gated_bwd_of_shared_sums(act, M, N, K):
    dout, wd, z, dz, _ = _bwd(act, M, N, K, M + N + K)
    zc = z.clone()
    over, none = mea.matmul_gated_act_bwd(act, dout, wd, zc, _p(act), want_h=False, dz=zc)
    assert over is zc and none is None and torch.equal(dz, zc)


@pytest.mark.parametrize("act", ["swish", "gelu_tanh", "tanh"])
@pytest.mark.parametrize("M,N,K", [(300, 264, 2056), (515, 520, 2056), (700, 256, 4104), (1030, 72, 1288)])
def test_gated_fwd_of_shared_sums(act, M, N, K):
    """Several tiles of tokens, the last of them cut short."""
    a = _fwd(act, M, N, K, M + N)
    assert torch.equal(a[4], _fwd(act, M, N, K, M + N, want_z=False)[4])


@pytest.mark.parametrize("act,param", [(a, _p(a)) for a in ACTS] + [("swish", 1.0), ("swish", -0.7), ("swish", 0.0)])
def test_gated_bwd_extreme_gates_of_shared_sums(act, param):
    """As test_gated_bwd_extreme_gates, through the other epilogue."""
    g = _gen(19)
    M, N, K = 40, 264, 1288
    dout, wd = _normal(g, M, K), _normal(g, K, N, scale=K ** -0.5)
    gate = torch.empty(M, N, device="cuda")
    gate[:20] = torch.linspace(-1.6, -0.6, 20 * N, device="cuda").view(20, N)
    far = torch.tensor([0.0, 5.0, 12.0, 13.5, 20.0, 60.0, 88.0, 100.0, 1e3, 1e6, 1e15, 1e30], device="cuda")
    gate[20:] = torch.cat([far, -far]).repeat(20 * N // 24)[:20 * N].view(20, N)
    z = torch.cat([gate, torch.ones(M, N, device="cuda")], 1).to(BF)
    dz, h = mea.matmul_gated_act_bwd(act, dout, wd, z, param)
    rdz, rh = ref.gated_bwd(act, dout, wd, z, param)
    bdz, bh = ref.gated_bwd_bounds(act, dout, wd, z, param)
    ref.assert_within(dz, rdz, bdz, "dz")
    ref.assert_within(h, rh, bh, "h")


@pytest.mark.parametrize("M,N,K", [(33, 136, 1288), (131, 136, 1288), (259, 72, 1288)])
def test_shared_sums_write_nothing_beyond_their_outputs(M, N, K):
    def guarded(rows, cols):
        buf = torch.full((rows * cols + 128,), 7.0, dtype=BF, device="cuda")
        return buf, buf[64:64 + rows * cols].view(rows, cols)

    g = _gen(20)
    x, wg, wu, wd, z0 = _normal(g, M, K), _normal(g, N, K), _normal(g, N, K), _normal(g, K, N), _normal(g, M, 2 * N)
    bufs = [guarded(M, 2 * N), guarded(M, N), guarded(M, 2 * N), guarded(M, N), guarded(M, N), guarded(136, 264)]
    mea.matmul_gated_act_fwd("swish", x, wg, wu, z=bufs[0][1], h=bufs[1][1])
    mea.matmul_gated_act_bwd("swish", x, wd, z0, dz=bufs[2][1], h=bufs[3][1])
    mea.matmul(x, wd, out=bufs[4][1])
    mea.matmul(_normal(g, K, 136), _normal(g, K, 264), True, out=bufs[5][1])
    for b, _ in bufs:
        assert (b[:64] == 7).all() and (b[-64:] == 7).all()


@pytest.mark.parametrize("M", [2, 150, 300])
def test_shared_sums_in_a_graph_and_on_two_streams(M):
    g = _gen(21)
    N, K = 136, 2056
    x, wg, wu, wd, z0 = _normal(g, M, K), _normal(g, N, K), _normal(g, N, K), _normal(g, K, N), _normal(g, M, 2 * N)
    a, b = _normal(g, K, 136), _normal(g, K, 264)

    def step():
        return (mea.matmul_gated_act_fwd("swish", x, wg, wu) + mea.matmul_gated_act_bwd("swish", x, wd, z0) +
                (mea.matmul(x, wd), mea.matmul(x, wg, False, True), mea.matmul(a, b, True)))

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(step())
    torch.cuda.synchronize()
    for o in [out] + outs:
        assert all(torch.equal(p, q) for p, q in zip(o, want))


@pytest.mark.parametrize("norm", [None, "layer", "rms"])
@pytest.mark.parametrize("batch,D,H", [((2, 650), 64, 128), ((1, 40), 1288, 1400), ((5, 300), 1288, 136)])
def test_gated_block_of_shared_sums(norm, batch, D, H):
    """The block where the weights' gradients (many tokens of a small model)
    or the projections (few tokens) share their sums."""
    test_gated_block(norm, "swish", batch, D, H)


def test_gated_tensors_of_more_than_2_31_elements():
    """The last rows of a large batch are those of a small one (every sum over
    k has one order), and the last columns of a wide weight those of a narrow
    one."""
    g = _gen(22)
    M, N, K, n = 140000, 8192, 64, 4096
    x, wg, wu, wd = _normal(g, M, K), _normal(g, N, K), _normal(g, N, K), _normal(g, K, N)
    z, h = mea.matmul_gated_act_fwd("swish", x, wg, wu)
    zs, hs = mea.matmul_gated_act_fwd("swish", x[-n:], wg, wu)
    assert z.numel() > 2 ** 31 and torch.equal(z[-n:], zs) and torch.equal(h[-n:], hs)
    dz, hb = mea.matmul_gated_act_bwd("swish", x, wd, z, dz=z, h=h)
    dzs, hbs = mea.matmul_gated_act_bwd("swish", x[-n:], wd, zs)
    assert torch.equal(dz[-n:], dzs) and torch.equal(hb[-n:], hbs)
    del z, dz, zs, dzs
    M, N = 64, 1 << 24
    x, wg, wu = _normal(g, M, 8), _normal(g, N + 64, 8), _normal(g, N + 64, 8)
    z, h = mea.matmul_gated_act_fwd("swish", x, wg, wu)
    n = 8192
    zs, hs = mea.matmul_gated_act_fwd("swish", x, wg[-n:], wu[-n:])
    assert z.numel() > 2 ** 31 and torch.equal(h[:, -n:], hs)
    assert torch.equal(z[:, -n:], zs[:, n:]) and torch.equal(z[:, N + 64 - n:N + 64], zs[:, :n])


@pytest.mark.parametrize("act,param", [(a, _p(a)) for a in ACTS] + [("swish", 1.0), ("swish", -0.7), ("swish", 0.0), ("swish", 2.0)])
@pytest.mark.parametrize("M,N,K", [(40, 264, 8), (1040, 264, 8), (1040, 264, 1288)])
def test_gated_fwd_extreme_gates(act, param, M, N, K):
    """Gates that one product forms exactly, far out on both sides, through the
    forward's epilogues.  No sum stands behind them: f's evaluation and one
    rounding bound h."""
    far = torch.tensor([0.0, 0.5, 1.0, 5.0, 12.0, 13.5, 20.0, 60.0, 88.0, 100.0, 1e3, 1e6, 1e15, 1e30, 3e38], device="cuda")
    gates = torch.cat([far, -far, torch.linspace(-14, -0.5, 10, device="cuda")])
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    x[:, 0], x[:, 1] = gates.repeat(M // 40).to(BF), 1
    wg, wu = torch.zeros(N, K, dtype=BF, device="cuda"), torch.zeros(N, K, dtype=BF, device="cuda")
    wg[:, 0], wu[:, 1] = 1, 0.75
    z, h = mea.matmul_gated_act_fwd(act, x, wg, wu, param)
    gate, up, want = ref.gated_fwd(act, x, wg, wu, param)
    assert torch.equal(z.double(), torch.cat([gate, up], 1))
    bound = want.abs() * (ref.F_REL + ref.HALF[BF] * (1 + ref.F_REL)) + 2 * ref.TINY
    ref.assert_within(h, want, bound, "h")
