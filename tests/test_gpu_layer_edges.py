"""The layer operators at the edges of what their interface allows: no eps, values at
the ends of fp32's range, rows that only pad, and what the block makes of them."""
import pytest

import layer_reference as R

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


def _ops():
    from blockwise_fp8_linear_fp8bw_b200 import ops
    return ops


def _normal(shape, seed, scale=1.0, dtype=None):
    torch = _t()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype or torch.bfloat16)


def _values(q):
    return q.view(_t().float8_e4m3fn).float()


def _padding_is_zero(out, rows):
    """Codes of the rows past `rows` are zero (either sign of it), their scales 1."""
    assert not bool(_values(out.q[rows:]).ne(0).any())
    assert bool((out.s[:, rows:] == 1).all())
    if out.q_t is not None:
        assert not bool(_values(out.q_t[:, rows:]).ne(0).any())


# a width and a length for each way that the rows are shared among threads
RAGGED = [(1, 16), (17, 2048), (77, 8208), (141, 4096), (143, 8192), (149, 8192),
          (701, 16400), (10005, 144), (1237, 1040)]


@pytest.mark.parametrize("rows,cols", RAGGED)
@pytest.mark.parametrize("pow2", [False, True])
def test_padding_rows_without_eps(rows, cols, pow2):
    """eps = 0 is allowed: a row of real values has a finite rstd, and the rows that
    only pad the codes are zero all the same."""
    torch, ops = _t(), _ops()
    x, r = _normal((rows, cols), 1), _normal((rows, cols), 2)
    gamma = 1 + _normal((cols,), 3, 0.2)
    h, rstd, v, err = R.norm(x, r, gamma, 0.0)
    for colwise in (False, True):
        out = ops.rmsnorm_quantize(x, gamma, r, 0.0, colwise=colwise, pow2=pow2)
        _padding_is_zero(out, rows)
        assert torch.equal(out.h, h)
        assert bool(((out.rstd.double() - rstd).abs() <= R.NORM_REL * rstd).all())
        R.check_codes(out.q, out.s, v, err, 1, pow2, rows)
    R.check_codes(out.q_t, out.s_t, v, err, 0, pow2, rows)
    ops.fp8bw_check_device_error()


@pytest.mark.parametrize("tokens", [1, 33, 48])
@pytest.mark.parametrize("pow2", [False, True])
def test_block_without_eps(tokens, pow2):
    """The block's gradients with eps = 0 are those with an eps too small to matter
    (2^-60 of a mean square of 2: half of fp32's rounding is 2^-24)."""
    torch = _t()
    from blockwise_fp8_linear_fp8bw_b200 import mlp
    x, r, dy, dh = (_normal((tokens, 272), 10 + i) for i in range(4))
    got = []
    for eps in (0.0, 2.0 ** -60):
        torch.manual_seed(7)
        m = mlp.BlockwiseFp8MLP(272, 400, eps=eps, device="cuda", pow2=pow2)
        xx = x.clone().requires_grad_()
        y, h = m(xx, r)
        torch.autograd.backward([y, h], [dy, dh])
        got.append((y.detach(), h.detach(), xx.grad, *(p.grad for p in m.parameters())))
    assert all(bool(torch.isfinite(t.float()).all()) for t in got[0])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def _check_norm(x, gamma, r, eps, pow2, rows):
    """Codes both ways and the bf16 output against the 64-bit norm; -> the codes."""
    torch, ops = _t(), _ops()
    _, _, v, err = R.norm(x, r, gamma, eps)
    out = ops.rmsnorm_quantize(x, gamma, r, eps, colwise=True, pow2=pow2)
    row = ops.rmsnorm_quantize(x, gamma, r, eps, pow2=pow2)
    assert torch.equal(out.q, row.q) and torch.equal(out.s, row.s)
    R.check_codes(out.q, out.s, v, err, 1, pow2, rows)
    R.check_codes(out.q_t, out.s_t, v, err, 0, pow2, rows)
    zero = v == 0
    assert not bool(_values(out.q[:rows])[zero].ne(0).any())
    assert not bool(_values(out.q_t[:, :rows]).t()[zero].ne(0).any())
    _padding_is_zero(out, rows)
    y, _, _ = ops.rmsnorm(x, gamma, r, eps)
    assert bool(((y.double() - v).abs() <= err + 2.0 ** -8 * v.abs() + 2.0 ** -134).all())
    # all outputs of one call are what the calls for each of them give
    both, every = torch.empty_like(y), [torch.empty_like(t) for t in (*out[:4], out.rstd)]
    ops.fp8bw_rmsnorm_quantize(x, gamma, r, eps, None if r is None else torch.empty_like(x),
                               every[4], both, *every[:4], pow2=pow2)
    assert torch.equal(both, y)
    assert all(torch.equal(a, b) for a, b in zip(every, (*out[:4], out.rstd)))
    ops.fp8bw_check_device_error()
    return out


@pytest.mark.parametrize("rows,cols", RAGGED)
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_nearly_empty_groups(rows, cols, pow2, residual):
    """A group, a row and a column of zeros and one value of 1e-37: the factor of the
    codes is beyond fp32's range, the codes are not."""
    torch = _t()
    x = _normal((rows, cols), 20)
    gamma = torch.full((cols,), 4.0, device="cuda")
    x[:, 3] = 0                                   # a column
    x[rows // 2, 3] = 1e-37
    if cols > 128:
        x[rows // 3, 128:256] = 0                 # a 1x128 group
        x[rows // 3, 130] = -1e-37
    if rows > 2:
        x[rows - 1] = 0                           # a row
        x[rows - 1, cols - 1] = 1e-37
    r = torch.zeros_like(x) if residual else None
    _check_norm(x, gamma, r, 1e-6, pow2, rows)


@pytest.mark.parametrize("rows,cols", RAGGED)
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("size,weight", [(2.0 ** 40, 2.0 ** 100), (2.0 ** -40, 2.0 ** -100),
                                         (2.0 ** -40, 2.0 ** 80), (2.0 ** 40, 2.0 ** -80)])
def test_norm_in_the_formulas_order(rows, cols, pow2, size, weight):
    """h rstd is of order one whatever h, so (h rstd) gamma is in fp32's range where
    h gamma is not (without eps). Every third column has such a weight."""
    torch = _t()
    x = _normal((rows, cols), 30, size)
    gamma = 1 + _normal((cols,), 31, 0.2, torch.float32)
    gamma[::3] *= weight
    _check_norm(x, gamma, None, 0.0, pow2, rows)
    gamma = (1 + _normal((cols,), 32, 0.2, torch.float32)) * weight
    _check_norm(x, gamma, None, 0.0, pow2, rows)


@pytest.mark.parametrize("rows,cols", [(1, 16), (17, 2048), (149, 8192), (10005, 144), (1237, 1040)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("pow2", [False, True])
def test_norm_weight_that_is_not_finite(rows, cols, bad, pow2):
    """It spoils its own column; the padding rows' codes stay zero."""
    torch, ops = _t(), _ops()
    x = _normal((rows, cols), 40)
    gamma = torch.ones(cols, device="cuda")
    gamma[5] = bad
    out = ops.rmsnorm_quantize(x, gamma, None, colwise=True, pow2=pow2)
    _padding_is_zero(out, rows)
    want = ops.rmsnorm_quantize(x, torch.ones_like(gamma), None, colwise=True, pow2=pow2)
    keep = [i for i in range(cols) if i != 5]
    assert torch.equal(out.q_t[keep], want.q_t[keep])
    assert torch.equal(out.s_t[:, keep], want.s_t[:, keep])
    assert torch.equal(out.rstd, want.rstd)
    v = _values(out.q_t)[5, :rows] * out.s_t[:, 5].repeat_interleave(128)[:rows]
    if pow2 and bad > 0:
        # the power-of-two rule gives a group with an infinity the scale 1, and
        # infinity times 1 saturates at E4M3's largest value
        assert bool((v.abs() == 448).all())
    else:
        assert not bool(torch.isfinite(v).any())


@pytest.mark.parametrize("pow2", [False, True])
def test_odd_groups_leave_their_neighbours_alone(pow2):
    """A row with values at the end of the range does not change what the rows and
    columns beside it get."""
    torch, ops = _t(), _ops()
    for rows, cols in RAGGED[1:]:
        x = _normal((rows, cols), 50)
        gamma = 1 + _normal((cols,), 51, 0.2)
        want = ops.rmsnorm_quantize(x, gamma, colwise=True, pow2=pow2)
        y = x.clone()
        y[5] = 0
        y[5, 7] = 1e-37
        got = ops.rmsnorm_quantize(y, gamma, colwise=True, pow2=pow2)
        keep = [i for i in range(rows) if i != 5]
        assert torch.equal(got.q[keep], want.q[keep])
        assert torch.equal(got.s[:, keep], want.s[:, keep])
        y = x.clone()
        y[:, 7] = 0
        g = gamma.clone()
        g[7] = 4.0
        y[rows // 2, 7] = 1e-37                   # (rstd is the same with or without it)
        z = y.clone()
        z[:, 7] = 0
        got, want = (ops.rmsnorm_quantize(t, g, colwise=True, pow2=pow2) for t in (y, z))
        keep = [i for i in range(cols) if i != 7]
        assert torch.equal(got.q_t[keep], want.q_t[keep])
        assert torch.equal(got.s_t[:, keep], want.s_t[:, keep])


def _every_gate(low, high):
    """Every bf16 value from low to high."""
    torch = _t()
    v = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16)
    v = v.view(torch.bfloat16)
    v = v[torch.isfinite(v.float()) & (v >= low) & (v <= high)]
    return v


@pytest.mark.parametrize("low,high", [(-80.0, -20.0), (-20.0, -2.0 ** -4), (2.0 ** -4, 100.0)])
def test_sigmoid_of_every_gate(low, high):
    """The scale of a group shows its largest value without a rounding to few bits.
    In units of u = 2^-24 relative: the approximate exponential 4 (2^-22), its argument's
    remainder to first order 1 and, at 80, 1.3 of second order, 1 + e 1, the approximate
    reciprocal 2, two products 1 each, the quotient 1."""
    torch, ops = _t(), _ops()
    gate = _every_gate(low, high)
    gu = torch.ones(gate.numel(), 256, device="cuda", dtype=torch.bfloat16)
    gu[:, :128] = gate[:, None]
    want = gate.double().abs() * torch.sigmoid(gate.double()) / 448.0
    for colwise in (False, True):
        got = ops.swiglu_quantize(gu, colwise=colwise).s[0, :gate.numel()].double()
        assert bool(((got - want).abs() <= 12.4 * R.U * want).all())
    # and of the gradient: dup = da gate sigmoid(gate), a product less
    da = torch.ones(gate.numel(), 128, device="cuda", dtype=torch.bfloat16)
    got = ops.swiglu_backward_quantize(da, gu).s[1, :gate.numel()].double()
    assert bool(((got - want).abs() <= 12.4 * R.U * want).all())


def test_gates_that_are_not_finite():
    """gate = inf: a is infinite, and its group's scale; -inf and NaN: NaN codes, and the
    rest of the group as without them."""
    torch, ops = _t(), _ops()
    inf = float("inf")
    gu = _normal((48, 512), 60)
    gu[7, 256 + 9] = 1.0
    for rows in (48, 4000):                       # both forms
        x = gu.repeat(rows // 48 + 1, 1)[:rows]
        ref = ops.swiglu_quantize(x, colwise=True)
        for bad, s in ((inf, inf), (-inf, None), (float("nan"), None)):
            y = x.clone()
            y[7, 9] = bad
            out = ops.swiglu_quantize(y, colwise=True)
            assert bool(torch.isnan(_values(out.q)[7, 9]))
            assert bool(torch.isnan(_values(out.q_t)[9, 7]))
            if s is not None:
                assert float(out.s[0, 7]) == inf and float(out.s_t[0, 9]) == inf
            q, keep = out.q.clone(), ref.q.clone()
            q[7, :128], keep[7, :128] = 0, 0
            assert torch.equal(q, keep)
            if s is None:
                v = _values(out.q)[7, :128] * out.s[0, 7]
                w = _values(ref.q)[7, :128] * ref.s[0, 7]
                v[9] = w[9]
                # (another largest value, another rounding)
                assert bool(((v - w).abs() <= 2.0 ** -4 * w.abs() + ref.s[0, 7] * 2.0 ** -9).all())


def _rule(v, pow2):
    """The quantisers' rule on fp32 values [rows, cols], 1x128 groups, rows padded to a
    multiple of 16; on the CPU, whose divisions are IEEE's. -> codes, scales."""
    torch = _t()
    v = torch.nn.functional.pad(v.cpu(), (0, 0, 0, -v.shape[0] % 16))
    rows, cols = v.shape
    w = torch.nn.functional.pad(v, (0, -cols % 128)).reshape(rows, -1, 128)
    amax = w.abs().amax(2)
    if pow2:
        m, e = torch.frexp(amax.double() / 448.0)
        e = torch.where(m > 0.5, e, e - 1).clamp(-127, 120)
        q, s = torch.ldexp(torch.ones_like(m), -e).float(), torch.ldexp(torch.ones_like(m), e).float()
        none = amax == 0
    else:
        # (a number divided by a tensor is its reciprocal times the number)
        q, s = torch.full_like(amax, 448.0) / amax, amax / torch.full_like(amax, 448.0)
        none = (amax == 0) | ~torch.isfinite(q)
    q, s = (torch.where(none, torch.ones_like(t), t) for t in (q, s))
    codes = (w * q[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(rows, -1)[:, :cols], s.t()


def _same_codes(out, v, pow2):
    torch = _t()
    q, s = _rule(v, pow2)
    assert torch.equal(out.q.cpu(), q) and torch.equal(out.s.cpu(), s)
    pad = torch.nn.functional.pad(v, (0, 0, 0, -v.shape[0] % 16))
    q, s = _rule(pad.t().contiguous(), pow2)
    cols = v.shape[1]
    assert torch.equal(out.q_t.cpu(), q[:cols]) and torch.equal(out.s_t.cpu(), s[:, :cols])


# the forms for few tiles, for ragged widths and for many tiles
@pytest.mark.parametrize("rows,f", [(33, 144), (777, 1360), (1300, 2000), (2500, 2048), (4100, 640)])
@pytest.mark.parametrize("pow2", [False, True])
def test_bits_of_the_quantisers_rule(rows, f, pow2):
    """Gates above 128 have a sigmoid of 1: the products of bf16 values are exact in
    fp32, and the codes and scales are bit by bit what the quantisers' rule makes of
    them, whatever their magnitude."""
    torch, ops = _t(), _ops()
    g = torch.Generator(device="cuda").manual_seed(70)

    def spread(r, c, low, high):
        e = torch.randint(low, high, (r, 1), generator=g, device="cuda").float()
        return torch.ldexp(torch.randn(r, c, generator=g, device="cuda"), e).bfloat16()
    gate = (128 + 128 * torch.rand(rows, f, generator=g, device="cuda")).bfloat16()
    up = spread(rows, f, -126, 110)
    v = gate.float() * up.float()
    out = ops.swiglu_quantize(torch.cat([gate, up], 1), colwise=True, pow2=pow2)
    _same_codes(out, v, pow2)
    row = ops.swiglu_quantize(torch.cat([gate, up], 1), pow2=pow2)
    assert torch.equal(row.q, out.q) and torch.equal(row.s, out.s)
    # backward: dgate = da up, dup = da gate (1 - sigmoid is 0)
    da, up = spread(rows, f, -60, 50), spread(rows, f, -60, 50)
    d = torch.cat([da.float() * up.float(), da.float() * gate.float()], 1)
    _same_codes(ops.swiglu_backward_quantize(da, torch.cat([gate, up], 1), pow2=pow2), d, pow2)


@pytest.mark.parametrize("cols", [16, 2048, 8192, 32768])
@pytest.mark.parametrize("residual", [False, True])
def test_the_range_of_the_norm(cols, residual):
    """Rows of a Euclidean norm from 2^-50 to 2^64 without eps, and beyond."""
    torch, ops = _t(), _ops()
    x = _normal((48, cols), 80, 1.0, torch.float32)
    x = x / x.double().norm(dim=1, keepdim=True).float()
    size = torch.linspace(-49.9, 63.9, 48, device="cuda", dtype=torch.float64).exp2()
    x = (x * size[:, None]).bfloat16()
    r = torch.zeros_like(x) if residual else None
    gamma = 1 + _normal((cols,), 81, 0.2)
    _, rstd, v, err = R.norm(x, r, gamma, 0.0)
    out = ops.rmsnorm_quantize(x, gamma, r, 0.0, colwise=True)
    assert bool(((out.rstd.double() - rstd).abs() <= R.NORM_REL * rstd).all())
    R.check_codes(out.q, out.s, v, err, 1, False, 48)
    R.check_codes(out.q_t, out.s_t, v, err, 0, False, 48)
    # beyond: zeros, and the rows beside them as they were
    y = x.clone()
    y[4] = (x[47].double() * 2).bfloat16()        # 2^64.9
    got = ops.rmsnorm_quantize(y, gamma, r, 0.0)
    assert float(got.rstd[4]) == 0 and not bool(_values(got.q[4]).ne(0).any())
    keep = [i for i in range(48) if i != 4]
    assert torch.equal(got.q[keep], out.q[keep]) and torch.equal(got.rstd[keep], out.rstd[keep])
    # with an eps that matters, any smaller row
    y = (x[:16].double() * 2.0 ** -70).bfloat16()
    h, rstd, v, err = R.norm(y, r[:16] if residual else None, gamma, 1e-6)
    got = ops.rmsnorm_quantize(y, gamma, r[:16] if residual else None, 1e-6)
    assert bool(((got.rstd.double() - rstd).abs() <= R.NORM_REL * rstd).all())
    R.check_codes(got.q, got.s, v, err, 1, False, 16)
