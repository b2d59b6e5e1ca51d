"""The layer operators (norm, gated product, Newton-Schulz) on a B200 against
their 64-bit forms: sizes from one token up, ragged ones, both scale rules,
empty and non-finite rows, guards around every output, streams, graphs."""
import pytest

import layer_reference as R

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


def _ops():
    from blockwise_fp8_linear_fp8bw_b200 import ops
    return ops


def _gen(seed):
    return _t().Generator(device="cuda").manual_seed(seed)


def _normal(shape, seed, scale=1.0, dtype=None):
    torch = _t()
    v = torch.randn(*shape, generator=_gen(seed), device="cuda") * scale
    hit = torch.rand(*shape, generator=_gen(seed + 1), device="cuda") < 1e-3
    v = torch.where(hit, v * 50, v)
    return v.to(dtype or torch.bfloat16)


ROWS_COLS = [(1, 16), (1, 2048), (2, 128), (15, 144), (16, 1040), (17, 2048),
             (127, 256), (129, 4096), (300, 8192), (5, 8208), (640, 8208),
             (33, 16400), (700, 16400), (3, 32768), (1200, 272), (4100, 48),
             (90, 8192), (100, 6160), (1300, 1024), (1237, 1040), (5000, 256), (10005, 144)]


@pytest.mark.parametrize("rows,cols", ROWS_COLS)
@pytest.mark.parametrize("residual,f32,pow2", [(True, False, False),
                                               (False, True, False),
                                               (True, True, True)])
def test_norm(rows, cols, residual, f32, pow2):
    torch, ops = _t(), _ops()
    x = _normal((rows, cols), 10)
    r = _normal((rows, cols), 20, 2.0) if residual else None
    gamma = 1 + _normal((cols,), 30, 0.2, torch.float32)
    gamma = gamma if f32 else gamma.bfloat16()
    h, rstd, v, err = R.norm(x, r, gamma, 1e-6)
    out = ops.rmsnorm_quantize(x, gamma, r, 1e-6, colwise=True, pow2=pow2)
    assert torch.equal(out.h, h)
    assert bool(((out.rstd.double() - rstd).abs() <= R.NORM_REL * rstd).all())
    R.check_codes(out.q, out.s, v, err, 1, pow2, rows)
    R.check_codes(out.q_t, out.s_t, v, err, 0, pow2, rows)
    row = ops.rmsnorm_quantize(x, gamma, r, 1e-6, pow2=pow2)
    assert row.q_t is None and torch.equal(row.q, out.q) and torch.equal(row.s, out.s)
    y, h2, _ = ops.rmsnorm(x, gamma, r, 1e-6)
    assert torch.equal(h2, h)
    assert bool(((y.double() - v).abs() <= err + 2.0 ** -8 * v.abs() + 2.0 ** -134).all())
    ops.fp8bw_check_device_error()


@pytest.mark.parametrize("rows,cols", ROWS_COLS)
@pytest.mark.parametrize("residual,f32", [(True, False), (False, True)])
def test_norm_backward(rows, cols, residual, f32):
    torch, ops = _t(), _ops()
    h = _normal((rows, cols), 40, 2.0)
    dy = _normal((rows, cols), 50, 1e-3)
    dres = _normal((rows, cols), 60, 1e-3) if residual else None
    gamma = 1 + _normal((cols,), 70, 0.2, torch.float32)
    gamma = gamma if f32 else gamma.bfloat16()
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dh, tol, dg, gtol = R.norm_backward(dy, h, rstd, gamma, dres)
    a = ops.rmsnorm_backward(dy, h, rstd, gamma, dres)
    assert bool(((a[0].double() - dh).abs() <= tol).all())
    assert bool(((a[1].double() - dg).abs() <= gtol).all())
    b = ops.rmsnorm_backward(dy, h, rstd, gamma, dres)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])   # no atomics


def test_norm_backward_against_differences():
    torch, ops = _t(), _ops()
    rows, cols = 37, 528
    x = _normal((rows, cols), 80)
    gamma = 1 + _normal((cols,), 81, 0.2, torch.float32)
    dy = _normal((rows, cols), 82, 1.0)
    out = ops.rmsnorm_quantize(x, gamma, None, 1e-6)
    dh, dgamma = ops.rmsnorm_backward(dy, out.h, out.rstd, gamma)

    def loss(xd, gd):
        return (dy.double() * xd * (xd.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gd).sum()

    xd, gd, e = x.double(), gamma.double(), 1e-4
    for seed in range(4):
        dx = _normal((rows, cols), 90 + seed, 1.0, torch.float64)
        dg = _normal((cols,), 190 + seed, 1.0, torch.float64)
        # a central difference's own error: the third derivative times e^2,
        # a bounded function of values of order one, under 1e-6 of sum |dy|
        slack = 1e-6 * float(dy.double().abs().sum())
        num = (loss(xd + e * dx, gd) - loss(xd - e * dx, gd)) / (2 * e)
        assert abs(float(num - (dh.double() * dx).sum())) <= \
            2.0 ** -8 * float((dh.double() * dx).abs().sum()) + 50 * slack
        num = (loss(xd, gd + e * dg) - loss(xd, gd - e * dg)) / (2 * e)
        assert abs(float(num - (dgamma.double() * dg).sum())) <= \
            400 * R.U * float((dy.double() * xd).abs().sum()) * 50 + slack


GLU_SIZES = [(1, 16), (1, 6144), (7, 144), (16, 128), (17, 256), (128, 640),
             (129, 1360), (333, 272), (1000, 1024), (2050, 48), (1300, 2000),
             (4100, 640), (2500, 1040)]
# for the backward pass also widths whose end, over several rows of tiles per
# block, is 16 to 112 columns past a multiple of 128
GLU_BWD_SIZES = GLU_SIZES + [(6500, 464), (9000, 192), (4000, 720), (3000, 1296),
                             (7000, 112), (2700, 880), (130, 80), (40, 2032),
                             (15000, 192), (20001, 112), (40000, 48), (1100, 1360),
                             (1300, 1024)]


@pytest.mark.parametrize("rows,f", GLU_SIZES)
@pytest.mark.parametrize("pow2", [False, True])
def test_glu(rows, f, pow2):
    torch, ops = _t(), _ops()
    gu = _normal((rows, 2 * f), 100, 2.0)
    a, err = R.glu(gu)
    out = ops.swiglu_quantize(gu, colwise=True, pow2=pow2)
    R.check_codes(out.q, out.s, a, err, 1, pow2, rows)
    R.check_codes(out.q_t, out.s_t, a, err, 0, pow2, rows)
    row = ops.swiglu_quantize(gu, pow2=pow2)
    assert row.q_t is None
    assert torch.equal(row.q, out.q) and torch.equal(row.s, out.s)
    ops.fp8bw_check_device_error()


@pytest.mark.parametrize("rows,f", GLU_BWD_SIZES)
@pytest.mark.parametrize("pow2", [False, True])
def test_glu_backward(rows, f, pow2):
    ops = _ops()
    gu = _normal((rows, 2 * f), 110, 2.0)
    da = _normal((rows, f), 120, 1e-3)
    d, err = R.glu_backward(da, gu)
    out = ops.swiglu_backward_quantize(da, gu, pow2=pow2)
    R.check_codes(out.q, out.s, d, err, 1, pow2, rows)
    R.check_codes(out.q_t, out.s_t, d, err, 0, pow2, rows)
    ops.fp8bw_check_device_error()


def test_glu_backward_against_differences():
    """The 64-bit gradient the kernels are held to, against differences."""
    torch = _t()
    gu = _normal((5, 64), 130).double()
    da = _normal((5, 32), 131).double()
    d, _ = R.glu_backward(da, gu)
    e = 1e-5
    for seed in range(4):
        dx = _normal((5, 64), 140 + seed, 1.0, torch.float64)
        num = ((R.glu(gu + e * dx)[0] - R.glu(gu - e * dx)[0]) * da).sum() / (2 * e)
        scale = float((d * dx).abs().sum())
        assert abs(float(num - (d * dx).sum())) <= 1e-6 * scale


def test_zero_rows_and_large_gates():
    """All-zero rows and groups get scale 1; gates far out saturate the
    sigmoid; nothing becomes NaN."""
    torch, ops = _t(), _ops()
    x = _normal((40, 512), 150)
    x[3] = 0
    x[:, 128:256] = 0
    out = ops.rmsnorm_quantize(x, torch.ones(512, device="cuda"), None, 1e-6, colwise=True)
    assert not bool(out.q[3].any()) and bool((out.s[:, 3] == 1).all())
    assert not bool(out.q_t[128:256].any()) and bool((out.s_t[:, 128:256] == 1).all())
    assert abs(float(out.rstd[3]) - 1000.0) <= 1e-3
    gu = torch.zeros(32, 256, device="cuda").bfloat16()
    gu[:, :128] = torch.tensor([-3e38, -1000, -90, -88, -87, 0, 88, 1000] * 16,
                               device="cuda").bfloat16()
    gu[:, 128:] = 0.5
    a, err = R.glu(gu)
    # gate = -3e38: the product with a sigmoid of 0 is 0
    got = ops.swiglu_quantize(gu, colwise=True)
    R.check_codes(got.q, got.s, a, err, 1, False, 32)
    R.check_codes(got.q_t, got.s_t, a, err, 0, False, 32)
    d = ops.swiglu_backward_quantize(torch.ones(32, 128, device="cuda").bfloat16(), gu)
    assert not bool(torch.isnan(d.q.view(torch.float8_e4m3fn).float()).any())


@pytest.mark.parametrize("pow2", [False, True])
def test_values_near_the_end_of_fp32s_range(pow2):
    """Maxima between 2^126 and 2^128 (a reciprocal below the normal numbers), and
    products that leave the range before the sigmoid is applied."""
    torch, ops = _t(), _ops()
    gate = (_normal((48, 256), 170).float().abs() * 10 + 20).clamp(max=60)
    up = _normal((48, 256), 171).float().clamp(-3, 3) * 2.0 ** 120
    gate[:, ::17] = -100.0
    up[:, ::17] = 2.0 ** 126
    gu = torch.cat([gate, up], 1).bfloat16()
    a, err = R.glu(gu)
    assert 2.0 ** 126 < float(a.abs().max()) < 2.0 ** 128
    out = ops.swiglu_quantize(gu, colwise=True, pow2=pow2)
    R.check_codes(out.q, out.s, a, err, 1, pow2, 48)
    R.check_codes(out.q_t, out.s_t, a, err, 0, pow2, 48)
    gu[:, 256:] = _normal((48, 256), 172).clamp(-3, 3)
    da = up.bfloat16()
    d, err = R.glu_backward(da, gu)
    assert 2.0 ** 126 < float(d.abs().max()) < 2.0 ** 128
    out = ops.swiglu_backward_quantize(da, gu, pow2=pow2)
    R.check_codes(out.q, out.s, d, err, 1, pow2, 48)
    R.check_codes(out.q_t, out.s_t, d, err, 0, pow2, 48)
    x = _normal((48, 256), 173).clamp(-3, 3)
    gamma = torch.full((256,), 2.0 ** 125, device="cuda")
    _, _, v, err = R.norm(x, None, gamma, 1e-6)
    assert 2.0 ** 126 < float(v.abs().max()) < 2.0 ** 128
    n = ops.rmsnorm_quantize(x, gamma, None, 1e-6, colwise=True, pow2=pow2)
    R.check_codes(n.q, n.s, v, err, 1, pow2, 48)
    R.check_codes(n.q_t, n.s_t, v, err, 0, pow2, 48)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_stay_in_their_row(bad):
    torch, ops = _t(), _ops()
    x = _normal((48, 384), 160)
    ones = torch.ones(384, device="cuda")
    ref = ops.rmsnorm_quantize(x, ones)
    y = x.clone()
    y[5, 7] = bad
    got = ops.rmsnorm_quantize(y, ones)
    keep = [i for i in range(48) if i != 5]
    assert torch.equal(got.q[keep], ref.q[keep]) and torch.equal(got.s[:, keep], ref.s[:, keep])
    assert bool(torch.isnan(got.q[5].view(torch.float8_e4m3fn).float()).any())
    gu = _normal((48, 768), 161)
    ref, g2 = ops.swiglu_quantize(gu), gu.clone()
    g2[5, 7] = bad
    got = ops.swiglu_quantize(g2)
    assert torch.equal(got.q[keep], ref.q[keep])
    other = [i for i in range(384) if i >= 128]
    assert torch.equal(got.q[5, other], ref.q[5, other])


NS_SHAPES = [["16x16"], ["16x256", "256x16"], ["48x400", "272x272"], ["256x768"],
             ["768x256", "512x512", "16x2048"], ["1040x1296"], ["1296x1040"],
             ["640x640"] * 9, ["256x256"], ["112x1408", "2064x192", "16x64", "64x16", "240x272",
                               "256x3088", "1040x256", "128x128"]]


@pytest.mark.parametrize("shapes", NS_SHAPES, ids=lambda s: "+".join(s)[:40])
@pytest.mark.parametrize("steps,f32", [(5, True), (1, False), (2, True), (6, False)])
def test_newton_schulz(shapes, steps, f32):
    torch, ops = _t(), _ops()
    gs = []
    for i, s in enumerate(shapes):
        n, k = (int(v) for v in s.split("x"))
        g = _normal((n, k), 200 + i, 1e-3, torch.float32)
        gs.append(g if f32 else g.bfloat16())
    outs = ops.newton_schulz_batch(gs, steps=steps)
    ops.fp8bw_check_device_error()
    assert len(outs) == len(gs)
    for g, o in zip(gs, outs):
        ref = R.newton_schulz(g, steps, (3.4445, -4.7750, 2.0315), 1e-7)
        assert o.dtype == torch.bfloat16 and o.shape == g.shape
        assert float((o.double() - ref).norm()) <= R.ns_tolerance(steps) * float(ref.norm())
    again = ops.newton_schulz_batch(gs, steps=steps)
    assert all(torch.equal(a, b) for a, b in zip(outs, again))
    alone = ops.newton_schulz(gs[0], steps=steps)
    ref = R.newton_schulz(gs[0], steps, (3.4445, -4.7750, 2.0315), 1e-7)
    assert float((alone.double() - ref).norm()) <= R.ns_tolerance(steps) * float(ref.norm())


@pytest.mark.parametrize("shapes", [["1040x2064"], ["2320x1040", "512x272", "1040x1040"],
                                    ["1136x1712", "16x48", "1712x1136"],
                                    ["208x656", "144x144", "3088x256"]],
                         ids=lambda s: "+".join(s))
@pytest.mark.parametrize("steps", [2, 3, 5, 6, 7])
def test_newton_schulz_pairs_of_steps(shapes, steps):
    """Oblong matrices large enough to take some steps in pairs on their short
    side, alone and beside matrices that do not."""
    torch, ops = _t(), _ops()
    gs = [_normal(tuple(int(v) for v in s.split("x")), 250 + i, 1e-3, torch.float32)
          for i, s in enumerate(shapes)]
    outs = ops.newton_schulz_batch(gs, steps=steps)
    ops.fp8bw_check_device_error()
    for g, o in zip(gs, outs):
        ref = R.newton_schulz(g, steps, (3.4445, -4.7750, 2.0315), 1e-7)
        assert float((o.double() - ref).norm()) <= R.ns_tolerance(steps) * float(ref.norm())
    assert all(torch.equal(a, b) for a, b in zip(outs, ops.newton_schulz_batch(gs, steps=steps)))


@pytest.mark.parametrize("short", [1040, 240])
def test_newton_schulz_pairs_with_other_coefficients_and_spectra(short):
    torch, ops = _t(), _ops()
    g = _normal((short, 2064), 260, 1e-3, torch.float32)
    u = torch.linalg.qr(_normal((short, 4), 261, 1.0, torch.float32))[0]
    v = torch.linalg.qr(_normal((2064, 4), 262, 1.0, torch.float32))[0]
    low = g + 20.0 * u @ v.t()               # four directions some 250 times the rest
    for m, coeffs in ((low, (3.4445, -4.7750, 2.0315)), (g, (1.5, -0.5, 0.0)),
                      (g, (2.0, -1.5, 0.5)), (0.01 * g, (6.0, -9.0, 4.0))):
        ref = R.newton_schulz(m, 5, coeffs, 1e-7)
        got = ops.newton_schulz(m, coeffs=coeffs)
        if float(ref.abs().max()) > 4.0:
            # (6, -9, 4) diverges, to 1e45: outside what the operator promises,
            # which is a result that is not finite rather than a wrong one
            assert not bool(torch.isfinite(got.float()).all())
            continue
        assert float((got.double() - ref).norm()) <= R.ns_tolerance(5) * float(ref.norm())
    # a steep polynomial, whose product of two steps would not fit
    steep = (8.1566, -22.4833, 15.8789)
    ref = R.newton_schulz(g, 2, steep, 1e-7)
    got = ops.newton_schulz(g, steps=2, coeffs=steep)
    # B's norm is up to 5.7 here instead of 2.8, and a step multiplies by up to
    # 8.2 instead of 3.4
    assert float((got.double() - ref).norm()) <= 2 * R.ns_tolerance(2) * float(ref.norm())


def test_newton_schulz_singular_values_and_extremes():
    torch, ops = _t(), _ops()
    g = _normal((256, 640), 300, 1e-3, torch.float32)
    s = torch.linalg.svdvals(ops.newton_schulz(g).double())
    # the usual coefficients settle between 0.68 and 1.13
    assert 0.6 <= float(s.min()) and float(s.max()) <= 1.2
    # a few directions a thousand times larger than the rest keep the rest
    u = torch.linalg.qr(_normal((256, 4), 301, 1.0, torch.float32))[0]
    v = torch.linalg.qr(_normal((640, 4), 302, 1.0, torch.float32))[0]
    low = g + 40.0 * u @ v.t()
    ref = R.newton_schulz(low, 5, (3.4445, -4.7750, 2.0315), 1e-7)
    got = ops.newton_schulz(low)
    assert float((got.double() - ref).norm()) <= R.ns_tolerance(5) * float(ref.norm())
    # the norm is taken in 64 bits: any fp32 magnitude is fine
    big = ops.newton_schulz(g * 1e30, eps=0.0)
    small = ops.newton_schulz(g * 1e-30, eps=0.0)
    ref = R.newton_schulz(g, 5, (3.4445, -4.7750, 2.0315), 0.0)
    for o in (big, small):
        assert float((o.double() - ref).norm()) <= R.ns_tolerance(5) * float(ref.norm())
    z = torch.zeros(64, 128, device="cuda")
    assert not bool(ops.newton_schulz(z).any())
    # other coefficients (the cubic iteration) and a single step
    cubic = (1.5, -0.5, 0.0)
    got = ops.newton_schulz(g, steps=3, coeffs=cubic)
    ref = R.newton_schulz(g, 3, cubic, 1e-7)
    assert float((got.double() - ref).norm()) <= R.ns_tolerance(3) * float(ref.norm())


@pytest.mark.parametrize("shapes", [((64, 400), (256, 256)), ((400, 640), (528, 272))])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_newton_schulz_non_finite_matrix_beside_others(shapes, bad):
    """A matrix with a value that is not finite comes out not finite; the others of
    the call, and a matrix of zeros among them, do not notice."""
    torch, ops = _t(), _ops()
    a, b = (_normal(s, 310 + i, 1e-3, torch.float32) for i, s in enumerate(shapes))
    z = torch.zeros(48, 80, device="cuda")
    want = ops.newton_schulz_batch([a, z, b])
    broken = a.clone()
    broken[3, 5] = bad
    got = ops.newton_schulz_batch([broken, z, b])
    ops.fp8bw_check_device_error()
    assert not bool(torch.isfinite(got[0].float()).all())
    assert not bool(got[1].any()) and torch.equal(got[2], want[2])


def test_no_rows_and_empty_matrices():
    torch, ops = _t(), _ops()
    x = torch.empty(0, 256, device="cuda", dtype=torch.bfloat16)
    ones = torch.ones(256, device="cuda")
    out = ops.rmsnorm_quantize(x, ones, None, 1e-6, colwise=True)
    assert out.q.shape == (0, 256) and out.q_t.shape == (256, 0)
    dh, dg = ops.rmsnorm_backward(x, x, torch.empty(0, device="cuda"), ones)
    assert dh.shape == (0, 256) and not bool(dg.any())
    assert ops.swiglu_quantize(x).q.shape == (0, 128)
    assert ops.swiglu_backward_quantize(x[:, :128].contiguous(), x).q.shape == (0, 256)
    assert ops.newton_schulz_batch([]) == []
    e = torch.empty(0, 64, device="cuda")
    g = _normal((32, 64), 310, 1.0, torch.float32)
    outs = ops.newton_schulz_batch([e, g])
    assert outs[0].shape == (0, 64) and torch.equal(outs[1], ops.newton_schulz(g))


class _Guarded:
    """Outputs carved out of one buffer, 256 bytes of 0xA5 around each."""

    def __init__(self):
        self.bufs = []

    def __call__(self, shape, dtype):
        torch = _t()
        n = 1
        for d in shape:
            n *= d
        size = torch.empty((), dtype=dtype).element_size() * n
        buf = torch.full((size + 512 + (-size % 256),), 0xA5, dtype=torch.uint8, device="cuda")
        self.bufs.append((buf, size))
        return buf[256:256 + size].view(dtype).view(*shape)

    def check(self):
        for buf, size in self.bufs:
            assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + size:] == 0xA5).all())


@pytest.mark.parametrize("rows,cols", [(1, 272), (19, 1040), (131, 400), (300, 2064),
                                       (1111, 2064), (1100, 1200), (2400, 1280)])
def test_nothing_is_written_outside_the_outputs(rows, cols):
    torch, ops = _t(), _ops()
    g = _Guarded()
    u8, f32, b16 = torch.uint8, torch.float32, torch.bfloat16
    rp = (rows + 15) // 16 * 16
    cd = lambda a: (a + 127) // 128   # noqa: E731
    codes = lambda c: (g((rp, c), u8), g((cd(c), rp), f32), g((c, rp), u8),   # noqa: E731
                       g((cd(rp), c), f32))
    x, r = _normal((rows, cols), 400), _normal((rows, cols), 401)
    gamma = torch.ones(cols, device="cuda").bfloat16()
    h, rstd, y = g((rows, cols), b16), g((rows,), f32), g((rows, cols), b16)
    c = codes(cols)
    ops.fp8bw_rmsnorm_quantize(x, gamma, r, 1e-6, h, rstd, y, *c)
    ref = ops.rmsnorm_quantize(x, gamma, r, 1e-6, colwise=True)
    assert all(torch.equal(a, b) for a, b in zip((*c, h, rstd), ref))
    dh, dg = g((rows, cols), b16), g((cols,), f32)
    ws = g((ops.rmsnorm_backward_workspace(rows, cols),), u8)
    ops.fp8bw_rmsnorm_backward(x, h, rstd, gamma, r, dh, dg, ws)
    gu = _normal((rows, 2 * cols), 402)
    c = codes(cols)
    ops.fp8bw_swiglu_quantize(gu, *c)
    ops.fp8bw_swiglu_quantize(gu, *codes(cols)[:2])
    assert all(torch.equal(a, b) for a, b in zip(c, ops.swiglu_quantize(gu, colwise=True)))
    c = codes(2 * cols)
    ops.fp8bw_swiglu_backward_quantize(x, gu, *c)
    assert all(torch.equal(a, b) for a, b in zip(c, ops.swiglu_backward_quantize(x, gu)))
    grads = [_normal((rp, cols), 403, 1.0, f32), _normal((cols, 48), 404, 1.0, f32)]
    outs = [g(tuple(m.shape), b16) for m in grads]
    ws = g((ops.newton_schulz_workspace(grads),), u8)
    ops.fp8bw_newton_schulz(grads, outs, ws)
    assert all(torch.equal(a, b) for a, b in zip(outs, ops.newton_schulz_batch(grads)))
    g.check()
    ops.fp8bw_check_device_error()


def _step(ops, x, r, gamma, gu, da, g, stream):
    a = ops.rmsnorm_quantize(x, gamma, r, colwise=True, stream=stream)
    b = ops.rmsnorm_backward(x, a.h, a.rstd, gamma, r, stream=stream)
    c = ops.swiglu_quantize(gu, colwise=True, stream=stream)
    d = ops.swiglu_backward_quantize(da, gu, stream=stream)
    e = ops.newton_schulz_batch(g, stream=stream)
    return (*a, *b, *c, *d, *e)


def _step_inputs(seed):
    torch = _t()
    return (_normal((200, 528), seed), _normal((200, 528), seed + 1),
            torch.ones(528, device="cuda"), _normal((200, 512), seed + 2),
            _normal((200, 256), seed + 3),
            [_normal((272, 144), seed + 4, 1.0, torch.float32),
             _normal((64, 512), seed + 5, 1.0, torch.float32)])


def test_two_streams_and_the_stream_argument():
    torch, ops = _t(), _ops()
    ins = [_step_inputs(500), _step_inputs(600)]
    refs = [_step(ops, *i, None) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(3):
        # not the current stream: given by argument, as an object and as a
        # raw handle
        outs.append((_step(ops, *ins[0], streams[0]),
                     _step(ops, *ins[1], streams[1].cuda_stream)))
    torch.cuda.synchronize()
    for pair in outs:
        for got, ref in zip(pair, refs):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_two_graphs_replayed_together():
    torch, ops = _t(), _ops()
    ins = [_step_inputs(700), _step_inputs(800)]
    refs = [_step(ops, *i, None) for i in ins]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], []
    for i in ins:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            _step(ops, *i, None)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(_step(ops, *i, None))
        graphs.append(g)
        streams.append(s)
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, refs):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    # new inputs in the captured buffers
    fresh = _step_inputs(900)
    want = _step(ops, *fresh, None)
    for dst, src in zip(ins[0][:5], fresh[:5]):
        dst.copy_(src)
    for dst, src in zip(ins[0][5], fresh[5]):
        dst.copy_(src)
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want))
    del graphs


def test_codes_feed_the_gemms():
    """Codes of an odd number of tokens go into fprop, dgrad and wgrad as they
    are: the padding rows add nothing."""
    torch, ops = _t(), _ops()
    rows, k, n = 77, 528, 272
    x = _normal((rows, k), 1000)
    w = _normal((n, k), 1001, 0.02)
    out = ops.rmsnorm_quantize(x, torch.ones(k, device="cuda"), colwise=True)
    qw, sw, _ = ops.quantize_weight_block(w)
    y = ops.gemm_fprop(out.q, out.s, qw, sw)
    assert y.shape == (80, n) and not bool(y[rows:].any())
    deq = lambda q, s: q.view(torch.float8_e4m3fn).double() * \
        s.t().double().repeat_interleave(128, 1)[:, :q.shape[1]]   # noqa: E731
    wd = qw.view(torch.float8_e4m3fn).double() * \
        sw.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    a = deq(out.q, out.s)
    ref, bound = a @ wd.t(), a.abs() @ wd.abs().t()
    assert bool(((y.double() - ref).abs() <= 1e-3 * bound + 2.0 ** -8 * ref.abs()).all())
    dy = torch.zeros(80, n, device="cuda").bfloat16()
    dy[:rows] = _normal((rows, n), 1002, 1e-3)
    qdy_t, sdy_t = ops.quantize_colwise(dy)
    dw = ops.gemm_wgrad_f32(qdy_t, sdy_t, out.q_t, out.s_t)
    p, q = deq(qdy_t, sdy_t), deq(out.q_t, out.s_t)
    assert bool(((dw.double() - p @ q.t()).abs() <= 1e-3 * (p.abs() @ q.abs().t()) + 1e-30).all())


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows get what a call on them
    alone gives (row and column groups do not look beyond their 128 rows)."""
    torch, ops = _t(), _ops()
    rows, cols = 140_017, 16384
    start = 137_088                       # a multiple of 128
    g = _gen(500)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    gamma = torch.randn(cols, generator=g, device="cuda")
    assert x.numel() > 2 ** 31

    def same(big, tail, first):
        assert torch.equal(big.q[first:], tail.q) and torch.equal(big.s[:, first:], tail.s)
        assert torch.equal(big.q_t[:, first:], tail.q_t)
        assert torch.equal(big.s_t[first // 128:], tail.s_t)

    big, tail = (ops.rmsnorm_quantize(t, gamma, t, colwise=True) for t in (x, x[start:]))
    same(big, tail, start)
    assert torch.equal(big.h[start:], tail.h) and torch.equal(big.rstd[start:], tail.rstd)
    dh, dgamma = ops.rmsnorm_backward(x, big.h, big.rstd, gamma, x)
    tail_dh, _ = ops.rmsnorm_backward(x[start:], tail.h, tail.rstd, gamma, x[start:])
    assert torch.equal(dh[start:], tail_dh)
    want, size = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(2))
    for i in range(0, rows, 4096):
        t = x[i:i + 4096].double() * big.h[i:i + 4096].double() * big.rstd[i:i + 4096, None].double()
        want += t.sum(0)
        size += t.abs().sum(0)
    # as R.norm_backward: every term 2 roundings, and the additions
    assert bool(((dgamma.double() - want).abs() <= (2 + rows // 64 + 360) * R.U * size).all())
    del big, tail, dh, tail_dh
    same(ops.swiglu_quantize(x, colwise=True), ops.swiglu_quantize(x[start:], colwise=True), start)
    da = x[:, :cols // 2].contiguous()
    same(ops.swiglu_backward_quantize(da, x), ops.swiglu_backward_quantize(da[start:], x[start:]),
         start)
    x = x.view(-1)[:rows * 16352].view(rows, 16352)     # f = 8176: 112 past a multiple of 128
    da = x[:, :8176].contiguous()
    same(ops.swiglu_backward_quantize(da, x), ops.swiglu_backward_quantize(da[start:], x[start:]),
         start)
    ops.fp8bw_check_device_error()


def test_newton_schulz_offsets_past_32_bits():
    torch, ops = _t(), _ops()
    n, k = 2 ** 17, 16400
    g = torch.randn(n, k, generator=_gen(510), device="cuda", dtype=torch.bfloat16)
    a, b, c = 1.5, -0.6, 0.1
    out = ops.newton_schulz(g, steps=1, coeffs=(a, b, c))
    norm = sum(float(g[i:i + 8192].double().square().sum()) for i in range(0, n, 8192)) ** 0.5
    m = torch.zeros(k, k, device="cuda")
    for i in range(0, n, 16384):
        t = g[i:i + 16384].float() / norm
        m += t.t() @ t
    p = b * m + c * (m @ m)
    for rows in (slice(0, 64), slice(n - 64, n)):
        x = g[rows].double() / norm
        want = a * x + x @ p.double()
        err = float((out[rows].double() - want).norm())
        assert err <= R.ns_tolerance(1) * float(want.norm())
