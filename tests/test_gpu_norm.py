"""GPU parity of the row normalisation (mea_norm_fwd, mea_norm_bwd) with its
64-bit form; the bounds are derived in _block_ref.py."""
import pytest
import torch

import _block_ref as ref
import memory_efficient_activation_b200 as mea

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NORMS = ["layer", "rms"]


def _inputs(rows, C, dtype, pdtype, seed, shift=0.0, offset=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(n, scale=1.0, mid=0.0, dt=DT[dtype]):
        buf = torch.empty(n + 8, dtype=dt, device="cuda")[offset:offset + n]
        return buf.copy_(torch.randn(n, generator=gen, device="cuda") * scale + mid)

    x, dy = normal(rows * C, 1.5, shift).view(rows, C), normal(rows * C).view(rows, C)
    return x, dy, normal(C, 0.3, 1.0, DT[pdtype]), normal(C, 0.2, 0.0, DT[pdtype])


def _check(norm, x, dy, gamma, beta, eps=1e-5):
    y, mean, invstd = mea.norm_fwd(norm, x, gamma, beta, eps)
    ry, rmean, rinv = ref.norm_fwd(norm, x, gamma, beta, eps)
    by, bmean, binv = ref.norm_fwd_bounds(norm, x, gamma, beta, eps, x.dtype)
    ref.assert_within(invstd, rinv, binv, "invstd")
    if norm == "layer":
        ref.assert_within(mean, rmean, bmean, "mean")
    else:
        assert mean is None
    ref.assert_within(y, ry, by, "y")
    pdt = torch.float32 if gamma is None else gamma.dtype
    got = mea.norm_bwd(norm, x, dy, gamma, mean, invstd, want_dgamma=True, want_dbeta=True)
    want = ref.norm_bwd(norm, x, dy, gamma, mean, invstd)
    bounds = ref.norm_bwd_bounds(norm, x, dy, gamma, mean, invstd, x.dtype, pdt)
    for name, g, w, b in zip(("dx", "dgamma", "dbeta"), got, want, bounds):
        ref.assert_within(g, w, b, name)
    return y, mean, invstd, got


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("dtype,pdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,C", [(1, 1), (3, 2), (5, 7), (1, 8), (33, 31), (2, 64), (37, 144), (9, 1001), (129, 1152),
                                    (7, 4096), (300, 4096), (5, 4104), (3, 5001), (17, 16384), (2, 40000)])
def test_norm_shapes(norm, dtype, pdtype, rows, C):
    x, dy, gamma, beta = _inputs(rows, C, dtype, pdtype, rows * 31 + C)
    _check(norm, x, dy, gamma, beta)


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,C", [(40001, 8), (20000, 24), (2500, 1000), (3000, 2056), (2100, 333), (1700, 8200)])
def test_norm_many_rows(norm, dtype, rows, C):
    """Several slabs of column sums, uneven shares, groups of every size."""
    x, dy, gamma, beta = _inputs(rows, C, dtype, "f32", rows + C)
    _check(norm, x, dy, gamma, beta)


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("dtype,pdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,C", [(2400, 264), (2369, 512), (2401, 2048), (300, 16384), (4099, 1001), (2100, 1003)])
def test_norm_streamed_rows(norm, dtype, pdtype, rows, C):
    """Rows enough for the streaming kernels (a warp to a row; rings of every
    width; single elements), each with both parameter types."""
    x, dy, gamma, beta = _inputs(rows, C, dtype, pdtype, rows * 3 + C)
    _check(norm, x, dy, gamma, beta)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,C", [(2, 131072), (2, 131073), (1, 300001)])
def test_norm_rows_longer_than_a_block_holds(dtype, rows, C):
    x, dy, gamma, beta = _inputs(rows, C, dtype, "f32", C)
    for norm in NORMS:
        _check(norm, x, dy, gamma, beta)


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_unaligned_tensors(dtype, offset):
    x, dy, gamma, beta = _inputs(21, 272, dtype, "f32", 5, offset=offset)
    assert x.data_ptr() % 16 or offset * x.element_size() % 16 == 0
    _check("layer", x, dy, gamma, beta)


@pytest.mark.parametrize("norm", NORMS)
def test_norm_without_parameters(norm):
    x, dy, gamma, beta = _inputs(19, 520, "bf16", "f32", 6)
    _check(norm, x, dy, None, None)
    _check(norm, x, dy, gamma, None)
    _check(norm, x, dy, None, beta)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_constant_rows_and_large_offsets(dtype):
    x, dy, gamma, beta = _inputs(12, 768, dtype, "f32", 7, shift=100.0)
    x[3] = 0.0
    x[4] = 2.5
    x[5] = 1e4
    y, mean, invstd, _ = _check("layer", x, dy, gamma, beta)
    assert torch.equal(y[4], beta.to(y.dtype)) and abs(float(invstd[4]) - 1e-5 ** -0.5) < 1e-4 * 1e-5 ** -0.5
    _check("rms", x, dy, gamma, beta)


@pytest.mark.parametrize("norm", NORMS)
def test_norm_bad_values_stay_in_their_row(norm):
    x, dy, gamma, beta = _inputs(9, 1024, "bf16", "f32", 8)
    clean = mea.norm_fwd(norm, x, gamma, beta)
    dxc = mea.norm_bwd(norm, x, dy, gamma, *clean[1:])[0]
    x[2, 5], x[6, 1000] = float("nan"), float("inf")
    y, mean, invstd = mea.norm_fwd(norm, x, gamma, beta)
    keep = [0, 1, 3, 4, 5, 7, 8]
    assert torch.equal(y[keep], clean[0][keep]) and y[2].isnan().all()
    dx = mea.norm_bwd(norm, x, dy, gamma, mean, invstd)[0]
    assert torch.equal(dx[keep], dxc[keep]) and dx[2].isnan().all()


@pytest.fixture(autouse=True)
def no_expired_waits():
    yield
    from memory_efficient_activation_b200 import _capi
    assert _capi.lib().mea_matmul_error_word(1) == 0


def test_norm_two_calls_at_once():
    """The same tensors normalised on two streams at the same time: the
    workspaces are per call."""
    x, dy, gamma, beta = _inputs(6000, 1024, "bf16", "bf16", 14)
    y, mean, invstd = mea.norm_fwd("layer", x, gamma, beta)
    want = mea.norm_bwd("layer", x, dy, gamma, mean, invstd, want_dbeta=True)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                got.append((mea.norm_fwd("layer", x, gamma, beta)[0],
                            mea.norm_bwd("layer", x, dy, gamma, mean, invstd, want_dbeta=True)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, y) and all(torch.equal(p, q) for p, q in zip(b, want))


def test_norm_no_rows():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(64, device="cuda")
    y, mean, invstd = mea.norm_fwd("layer", x, gamma)
    assert y.shape == x.shape and mean.shape == (0,)
    dx, dg, db = mea.norm_bwd("layer", x, x, gamma, mean, invstd, want_dbeta=True)
    assert dx.shape == x.shape and not dg.any() and not db.any()


@pytest.mark.parametrize("rows,C", [(700, 4096), (333, 1001), (2, 131072)])
def test_norm_dx_in_place_and_deterministic(rows, C):
    x, dy, gamma, beta = _inputs(rows, C, "bf16", "bf16", 9)
    y, mean, invstd = mea.norm_fwd("layer", x, gamma, beta)
    first = mea.norm_bwd("layer", x, dy, gamma, mean, invstd, want_dbeta=True)
    for target in ("x", "dy"):
        xc, dc = x.clone(), dy.clone()
        got = mea.norm_bwd("layer", xc, dc, gamma, mean, invstd, want_dbeta=True, out=xc if target == "x" else dc)
        for a, b in zip(first, got):
            assert torch.equal(a, b)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip((y, mean, invstd), mea.norm_fwd("layer", x, gamma, beta)))


def test_norm_writes_nothing_beyond_its_outputs():
    rows, C = 37, 1003
    x, dy, gamma, _ = _inputs(rows, C, "bf16", "f32", 10)
    buf = torch.full((rows * C + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[32:32 + rows * C].view(rows, C)
    _, mean, invstd = mea.norm_fwd("layer", x, gamma, out=out)
    assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()
    mea.norm_bwd("layer", x, dy, gamma, mean, invstd, out=out)
    assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()


def test_norm_on_a_side_stream_and_in_graphs():
    """Two graphs captured on one stream and replayed on two at once: their
    workspaces are their own."""
    cases = [_inputs(2000, 1024, "bf16", "f32", s) for s in (11, 12)]
    want = []
    for x, dy, gamma, beta in cases:
        y, mean, invstd = mea.norm_fwd("layer", x, gamma, beta)
        want.append((y, *mea.norm_bwd("layer", x, dy, gamma, mean, invstd, want_dbeta=True)))
    torch.cuda.synchronize()
    side, graphs, outs = torch.cuda.Stream(), [], []
    for x, dy, gamma, beta in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            y, mean, invstd = mea.norm_fwd("layer", x, gamma, beta)
            outs.append((y, *mea.norm_bwd("layer", x, dy, gamma, mean, invstd, want_dbeta=True)))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("cls,dtype", [(mea.MemoryEfficientLayerNorm, torch.float32),
                                       (mea.MemoryEfficientRMSNorm, torch.bfloat16)])
def test_norm_modules(cls, dtype):
    torch.manual_seed(13)
    m = cls(96, dtype=dtype).cuda()
    with torch.no_grad():
        for p in m.parameters():
            p.add_(torch.randn_like(p) * 0.2)
    x = torch.randn(4, 10, 96, device="cuda").bfloat16().requires_grad_()
    xt = x.transpose(0, 1)                                  # a strided input is copied, its gradient comes back strided
    dy = torch.randn(10, 4, 96, device="cuda").bfloat16()
    y = m(xt)
    y.backward(dy)
    mean, invstd = mea.norm_fwd(cls.norm, xt.detach().contiguous(), m.gamma)[1:]
    by = ref.norm_fwd_bounds(cls.norm, xt.detach(), m.gamma.detach(), None if m.beta is None else m.beta.detach(), 1e-5,
                             torch.bfloat16)[0]
    ref.assert_within(y.detach(), ref.norm_fwd(cls.norm, xt.detach(), m.gamma.detach(),
                                               None if m.beta is None else m.beta.detach(), 1e-5)[0], by, "y")
    want = ref.norm_bwd(cls.norm, xt.detach(), dy, m.gamma.detach(), mean, invstd)
    b = ref.norm_bwd_bounds(cls.norm, xt.detach(), dy, m.gamma.detach(), mean, invstd, torch.bfloat16, dtype)
    ref.assert_within(x.grad.transpose(0, 1), want[0], b[0], "dx")
    ref.assert_within(m.gamma.grad, want[1], b[1], "dgamma")
    assert m.gamma.grad.dtype == dtype
    if m.beta is not None:
        ref.assert_within(m.beta.grad, want[2], b[2], "dbeta")
    # a frozen parameter gets none
    m.gamma.requires_grad_(False)
    m.zero_grad()
    x.grad = None
    m(x).backward(torch.ones_like(x))
    assert m.gamma.grad is None and x.grad is not None


@pytest.mark.parametrize("dtype,rows,C", [("f32", 1100, 1001), ("bf16", 2200, 1001), ("bf16", 500, 5120),
                                          ("bf16", 200, 12288), ("f32", 300, 5120), ("bf16", 2500, 1024),
                                          ("bf16", 20, 1001), ("f32", 20, 4096)])
def test_norm_means_whose_square_overflows(dtype, rows, C):
    """Means beyond 1.85e19 beside deviations whose squares are finite: rows of
    two to seven warps in the streaming kernel, and the other kernels."""
    x, _, gamma, beta = _inputs(rows, C, dtype, "f32", rows + C)
    x[1::3] = (x[1::3].float() * 1e17 + 3e19).to(x.dtype)
    x[2::3] = (x[2::3].float() * 1e16 - 2.5e19).to(x.dtype)
    got = mea.norm_fwd("layer", x, gamma, beta)
    want = ref.norm_fwd("layer", x, gamma, beta, 1e-5)
    bounds = ref.norm_fwd_bounds("layer", x, gamma, beta, 1e-5, x.dtype)
    for name, g, w, b in zip(("y", "mean", "invstd"), got, want, bounds):
        ref.assert_within(g, w, b, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("rows,C", [(700, 272), (64, 1001), (3, 20000)])
def test_norm_dx_in_place_unaligned(rows, C, norm, dtype):
    """dx over x and over dy, single elements of tensors off a 16-byte
    boundary."""
    def fresh():
        x, dy, gamma, _ = _inputs(rows, C, dtype, "f32", rows + C, offset=1)
        assert x.data_ptr() % 16 and dy.data_ptr() % 16
        return x, dy, gamma

    x, dy, gamma = fresh()
    mean, invstd = mea.norm_fwd(norm, x, gamma)[1:]
    first = mea.norm_bwd(norm, x, dy, gamma, mean, invstd, want_dbeta=True, out=fresh()[0])
    for target in ("x", "dy"):
        x, dy, gamma = fresh()
        got = mea.norm_bwd(norm, x, dy, gamma, mean, invstd, want_dbeta=True, out=x if target == "x" else dy)
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_either_side_of_the_kernels_borders(dtype):
    """Sizes around every border between the kernels and between their numbers
    of items per thread: rows of one to more than 1024 threads' worth, few rows
    and enough to stream, whole vectors and single elements."""
    V = 8 if dtype == "bf16" else 4
    shapes = []
    for items in (1, 2, 32, 33, 64, 65, 128, 129, 256, 257, 512, 513, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193):
        small, large = max(1, (3 << 20) // (16 * items)), (5 << 20) // (16 * items)
        shapes += [(r, items * V) for r in (1, min(small, 3000), min(large, 6000))]
        if items > 4000:
            shapes += [(2400, items * V)]
    for C in (1, 3, 31, 33, 257, 511, 513, 1025, 2047, 2049, 4097, 8191, 8193, 16385):
        shapes += [(1, C), (max(1, min(3000, (1 << 20) // C)), C), (min(6000, (3 << 20) // C), C)]
    for rows, C in shapes:
        x, dy, gamma, beta = _inputs(rows, C, dtype, "f32", rows + C)
        for norm in NORMS:
            _check(norm, x, dy, gamma, beta)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("path", ["vectors", "odd width", "unaligned", "long rows"])
@pytest.mark.parametrize("rows", [1, 147, 149, 1023, 1025, 2049, 40001, 151553, 303105])
def test_norm_column_sums_count_every_row_once(rows, path, dtype):
    """Mean 0, invstd 1, elements and gradients of -3, -1, 1 and 3: every term
    is an odd integer and every partial sum below 2^24, so the sums are exact
    in any order, and a row lost or taken twice changes each of them."""
    C = {"vectors": 24, "odd width": 27, "unaligned": 24, "long rows": 16392 if dtype == "bf16" else 8200}[path]
    if path == "long rows":
        rows = min(rows, 2049)
    assert 9 * rows < 1 << 24
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def odd():
        buf = torch.empty(rows * C + 1, dtype=DT[dtype], device="cuda")[1 if path == "unaligned" else 0:][:rows * C]
        return buf.view(rows, C).copy_(torch.randint(-2, 2, (rows, C), generator=gen, device="cuda") * 2 + 1)

    x, dy = odd(), odd()
    mean, invstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    for norm in NORMS:
        _, dg, db = mea.norm_bwd(norm, x, dy, None, mean, invstd, want_dgamma=True, want_dbeta=True)
        assert torch.equal(dg.double(), (x.double() * dy.double()).sum(0))
        assert torch.equal(db.double(), dy.double().sum(0))


@pytest.mark.parametrize("rows,C", [(300000, 8192), (2200000, 1001), (66000, 32776)])
def test_norm_tensors_of_more_than_2_31_elements(rows, C):
    """The last rows of a large tensor are those of a small one of the same
    alignment, and the column sums count every row (exact integers)."""
    gen = torch.Generator(device="cuda").manual_seed(15)
    x, dy = (torch.empty(rows, C, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (x, dy):
        t.random_(-2, 2, generator=gen).mul_(2).add_(1)
    n = 8000
    assert x.numel() > 2 ** 31
    gamma = torch.randn(C, generator=gen, device="cuda")
    y, mean, invstd = mea.norm_fwd("layer", x, gamma)
    ys, ms, iss = mea.norm_fwd("layer", x[-n:].clone(), gamma)
    assert torch.equal(y[-n:], ys) and torch.equal(mean[-n:], ms) and torch.equal(invstd[-n:], iss)
    del y
    dx, _, _ = mea.norm_bwd("layer", x, dy, gamma, mean, invstd)
    dxs, _, _ = mea.norm_bwd("layer", x[-n:].clone(), dy[-n:].clone(), gamma, ms, iss)
    assert torch.equal(dx[-n:], dxs)
    del dx, dxs
    one, zero = torch.ones(rows, device="cuda"), torch.zeros(rows, device="cuda")
    _, dg, db = mea.norm_bwd("layer", x, dy, None, zero, one, want_dgamma=True, want_dbeta=True)
    eg, eb = torch.zeros(C, dtype=torch.double, device="cuda"), torch.zeros(C, dtype=torch.double, device="cuda")
    for i in range(0, rows, 20000):
        a, b = x[i:i + 20000].float(), dy[i:i + 20000].float()
        eg += (a * b).sum(0, dtype=torch.double)
        eb += b.sum(0, dtype=torch.double)
    assert torch.equal(dg.double(), eg.float().double()) and torch.equal(db.double(), eb)


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,C", [(2400, 1024), (4200, 1001), (40001, 24), (90001, 27), (600, 5120), (300, 16384), (3, 131073)])
def test_norm_bad_values_stay_in_their_row_of_a_large_tensor(rows, C, dtype, norm):
    """Rows beside one another in a block and in its stages; the column sums
    take the bad values of their own columns only (layer norm's and rms norm's
    normalised row is bad as a whole, so d gamma is; d beta is not)."""
    x, dy, gamma, beta = _inputs(rows, C, dtype, "f32", 16)
    clean = mea.norm_fwd(norm, x, gamma, beta)
    dxc, _, dbc = mea.norm_bwd(norm, x, dy, gamma, *clean[1:], want_dbeta=True)
    bad = sorted({1, rows // 2, rows - 1})
    x[bad[0], 0], x[bad[1], C // 2], x[bad[-1], C - 1] = float("nan"), float("inf"), float("-inf")
    y, mean, invstd = mea.norm_fwd(norm, x, gamma, beta)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(y[keep], clean[0][keep]) and y[bad[0]].isnan().all()
    dx, _, db = mea.norm_bwd(norm, x, dy, gamma, mean, invstd, want_dbeta=True)
    assert torch.equal(dx[keep], dxc[keep]) and dx[bad[0]].isnan().all() and torch.equal(db, dbc)
