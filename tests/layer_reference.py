"""64-bit forms of the layer operators and the tolerances their fp32 kernels
are held to (torch double; no code of the library).

u = 2^-24 is fp32's relative rounding, 2^-8 bf16's, 2^-4 E4M3's (half a step).
"""
import torch

U = 2.0 ** -24


def groups(v, dim):
    """max |v| over 128-long groups along `dim`, spread back over v's shape."""
    w = v if dim == 1 else v.t()
    n, length = w.shape
    pad = -length % 128
    g = torch.nn.functional.pad(w.abs(), (0, pad)).reshape(n, -1, 128).amax(2)
    full = g.repeat_interleave(128, dim=1)[:, :length]
    return (g, full) if dim == 1 else (g, full)


def check_codes(q, s, v, err, dim, pow2, rows):
    """Row-wise (dim 1) or column-wise (dim 0) codes of the 64-bit v [rows,
    cols], each element of which the kernel may hold with an absolute error of
    `err` before it rounds to E4M3.

    The scale follows the group's maximum, which is off by at most the largest
    `err` of the group (and two roundings). A dequantised value is off by half
    a step of E4M3 at the code's magnitude, by `err`, and by the few roundings
    of the scaling; a saturated one (+-448) by the scale's own error."""
    codes = q.view(torch.float8_e4m3fn).double()
    rp = (rows + 15) // 16 * 16
    v = torch.nn.functional.pad(v, (0, 0, 0, rp - rows))
    err = torch.nn.functional.pad(err, (0, 0, 0, rp - rows))
    if dim == 0:
        v, err = v.t(), err.t()
    assert tuple(q.shape) == tuple(v.shape)
    g, _ = groups(v, 1)
    gerr, _ = groups(err, 1)
    sc = s.t().double()
    assert tuple(sc.shape) == tuple(g.shape)
    lo, hi = g - gerr, g + gerr
    empty = hi == 0
    assert bool((sc[empty] == 1.0).all())
    if pow2:
        live = ~empty & (lo > 2.0 ** -100)
        m, _ = torch.frexp(sc)
        assert bool((m[live] == 0.5).all())
        assert bool((448.0 * sc >= lo)[live].all())
        assert bool((224.0 * sc < hi)[live].all())
    else:
        # 448 / amax must be finite for the group rule to apply
        live = lo > 2.0 ** -100
        d = (sc - g / 448.0).abs()
        assert bool((d <= gerr / 448.0 + 4 * U * g / 448.0)[live].all())
    full = sc.repeat_interleave(128, dim=1)[:, :v.shape[1]]
    deq = codes * full
    # the spacing of E4M3 from the code's magnitude up (frexp: exact, where a
    # rounded log2 may fall short of a power of two); a code that was rounded
    # up to a power of two came from the finer spacing below, so this covers it
    step = torch.ldexp(torch.ones_like(codes),
                       torch.frexp(codes.abs().clamp_min(2.0 ** -6)).exponent - 4)
    rel = (g + gerr) / g.clamp_min(1e-300) - 1.0
    slack = rel.repeat_interleave(128, dim=1)[:, :v.shape[1]]
    tol = 0.5 * step * full + err + v.abs() * (4 * U + slack)
    bad = ~((deq - v).abs() <= tol)
    assert not bool(bad.any()), (
        "%d of %d codes off; first at %s: %s for %s (scale %s)"
        % (int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(),
           deq[bad][0].item(), v[bad][0].item(), full[bad][0].item()))
    # rows past the end: zero codes
    pad = codes[rows:] if dim == 1 else codes[:, rows:]
    assert not bool((pad != 0).any())


def norm(x, residual, gamma, eps):
    """-> (h bf16, rstd, v, err): the norm's 64-bit values and the error bound
    of the kernel's fp32 ones."""
    h = x if residual is None else (x.float() + residual.float()).bfloat16()
    hd = h.double()
    rstd = 1.0 / (hd.square().mean(1) + eps).sqrt()
    v = hd * rstd[:, None] * gamma.double()
    # the sum of squares: at most 64 + 5 + 16 additions of positive terms, half
    # of that error after the root; then a division, an addition, a root, a
    # reciprocal and two products
    return h, rstd, v, v.abs() * NORM_REL


NORM_REL = (85 / 2 + 6) * U


def norm_backward(dy, h, rstd, gamma, dres):
    """-> (dh, tol, dgamma, tol)."""
    dy, h, rstd, gamma = dy.double(), h.double(), rstd.double(), gamma.double()
    cols = h.shape[1]
    xh = h * rstd[:, None]
    g = dy * gamma
    m = (g * xh).mean(1, keepdim=True)
    dh = rstd[:, None] * (g - xh * m)
    # fp32: products and differences (8 roundings of each term) and the row
    # sum (at most 64 + 5 + 16 additions) of |g xh|
    mabs = (g * xh).abs().mean(1, keepdim=True)
    tol = rstd[:, None].abs() * (8 * U * (g.abs() + (xh * m).abs())
                                 + 90 * U * xh.abs() * mabs)
    if dres is not None:
        dh = dh + dres.double()
    tol = tol + 2 * U * dh.abs()
    tol = tol + 2.0 ** -8 * (dh.abs() + tol) + 2.0 ** -134   # the bf16 result
    terms = dy * xh
    # every term: 2 roundings; the additions: a thread's own rows, the 32
    # slices and what each slice adds up
    n = h.shape[0]
    adds = n // 64 + 8 + 32 + 320
    return dh, tol, terms.sum(0), (2 + adds) * U * terms.abs().sum(0)


def glu(gu):
    """-> (a, err): silu(gate) * up. The fast exponential is off by
    (2 + 1.5 |gate|) * 2 u relative, the quotient by 2 ulp (4 u), three
    products by u each; below -87 the sigmoid may be 0."""
    f = gu.shape[1] // 2
    gate, up = gu[:, :f].double(), gu[:, f:].double()
    a = gate * torch.sigmoid(gate) * up
    err = a.abs() * (12 + 3 * gate.abs()) * U + up.abs() * 2.0 ** -118
    return a, err


def glu_backward(da, gu):
    """-> (d, err) of [dgate | dup]."""
    f = gu.shape[1] // 2
    gate, up, da = gu[:, :f].double(), gu[:, f:].double(), da.double()
    sg, ns = torch.sigmoid(gate), torch.sigmoid(-gate)
    dgate = da * up * sg * (1 + gate * ns)
    dup = da * gate * sg
    e = (12 + 3 * gate.abs()) * U
    # 1 - sg carries sg's absolute error (at most e * sg) into gate * (1 - sg)
    egate = (da * up).abs() * (sg * (e * (1 + (gate * ns).abs())
                                     + gate.abs() * (e * sg * ns + U)) + 2.0 ** -118)
    eup = dup.abs() * e + da.abs() * 2.0 ** -118
    return torch.cat([dgate, dup], 1), torch.cat([egate, eup], 1)


def newton_schulz(g, steps, coeffs, eps):
    a, b, c = coeffs
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.norm() + eps)
    for _ in range(steps):
        m = x @ x.t()
        x = a * x + (b * m + c * (m @ m)) @ x
    return x.t() if tall else x


def ns_tolerance(steps):
    """Frobenius error relative to the result: bf16's half step, and per step
    the half steps (2^-11) of the three fp16 operands, of which B, with a norm
    of at most 2.8, multiplies X's."""
    return 2.0 ** -8 + steps * 3 * 2.8 * 2.0 ** -11
