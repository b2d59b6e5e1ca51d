"""The Newton-Schulz kernels against bounds that follow from their number formats
(ns_reference): as a whole and in every box of 32 x 32, where a warp that loses its
box, an operand in fewer bits or an iterate without its low half shows."""
import pytest

import ns_reference as N

pytestmark = pytest.mark.gpu

USUAL = (3.4445, -4.7750, 2.0315)


def _mods():
    import torch
    from blockwise_fp8_linear_fp8bw_b200 import ops
    return torch, ops


def _matrix(torch, n, k, seed, directions=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.randn(n, k, generator=gen, device="cuda") * 1e-3
    if directions:
        u = torch.linalg.qr(torch.randn(n, 4, generator=gen, device="cuda"))[0]
        v = torch.linalg.qr(torch.randn(k, 4, generator=gen, device="cuda"))[0]
        g = g + directions * u @ v.t()
    return g


# chains (short sides up to 256), tiles of 64, 128 and 256 columns, symmetric products
# with mirrored tiles, steps in pairs, ragged sides, several matrices at once
SHAPES = ["256x768", "768x240", "16x256", "272x272", "512x512", "512x1040", "1040x1296",
          "1296x1040", "1040x2064", "2320x1040", "2048x2048", "640x640,640x640,1136x1712",
          "112x1408,2064x192,256x256", "2048x2048,2048x4096,4096x2048,1040x2064"]


@pytest.mark.parametrize("shapes", SHAPES)
@pytest.mark.parametrize("steps", [1, 2, 5])
@pytest.mark.parametrize("directions", [0.0, 20.0])
def test_every_box(shapes, steps, directions):
    torch, ops = _mods()
    gs = [_matrix(torch, *(int(v) for v in s.split("x")), 10 + i, directions)
          for i, s in enumerate(shapes.split(","))]
    outs = ops.newton_schulz_batch(gs, steps=steps)
    ops.fp8bw_check_device_error()
    for g, o in zip(gs, outs):
        assert N.Bound(g, steps, USUAL).ok(o)


@pytest.mark.parametrize("shape", ["256x768", "768x256", "512x512", "1040x2064", "2064x1040",
                                   "2048x2048", "16x2048", "6144x256"])
def test_a_single_step_whose_products_count(shape):
    torch, ops = _mods()
    n, k = (int(v) for v in shape.split("x"))
    g = _matrix(torch, n, k, 30)
    coeffs = N.product_coefficients(n, k)
    assert N.Bound(g, 1, coeffs).ok(ops.newton_schulz(g, steps=1, coeffs=coeffs))
    ops.fp8bw_check_device_error()


@pytest.mark.parametrize("shapes", ["1040x2064", "2048x4096", "1136x1712,1712x1136"])
def test_products_of_pairs_repeat(shapes):
    """The last product of a pair of steps reads a second matrix through the staging
    that its mirror images leave through: 60 runs beside other work give the same bits."""
    torch, ops = _mods()
    gs = [_matrix(torch, *(int(v) for v in s.split("x")), 40 + i)
          for i, s in enumerate(shapes.split(","))]
    want = ops.newton_schulz_batch(gs)
    for g, o in zip(gs, want):
        assert N.Bound(g, 5, USUAL).ok(o)
    other = torch.cuda.Stream()
    noise = torch.randn(4096, 4096, device="cuda")
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(60):
        with torch.cuda.stream(other):
            noise.mul_(1.0001)
        assert all(torch.equal(a, b) for a, b in zip(want, ops.newton_schulz_batch(gs)))
    torch.cuda.synchronize()


def test_products_past_32_bits_of_offset():
    """2^31 elements, with coefficients for which the products weigh more than a X does
    (the largest eigenvalue of A is 1.1e-4 here): rows at the start, in the middle, next
    to element 2^31 and at the end."""
    torch, ops = _mods()
    n, k = 2 ** 17, 16400
    gen = torch.Generator(device="cuda").manual_seed(50)
    g = torch.randn(n, k, generator=gen, device="cuda", dtype=torch.bfloat16)
    a, b, c = N.product_coefficients(n, k)
    out = ops.newton_schulz(g, steps=1, coeffs=(a, b, c))
    ops.fp8bw_check_device_error()
    norm = sum(float(g[i:i + 8192].double().square().sum()) for i in range(0, n, 8192)) ** 0.5
    m = torch.zeros(k, k, device="cuda")
    for i in range(0, n, 16384):
        t = g[i:i + 16384].float() / norm
        m += t.t() @ t
    p = b * m + c * (m @ m)
    del m
    at = 2 ** 31 // k
    for first in (0, 48, n // 2, at - 40, at + 8, n - 64):
        x = g[first:first + 64].double() / norm
        part = x @ p.double()
        want = a * x + part
        # bf16 half a step; B's rounding (2^-11 of every entry, independent: about
        # 2^-11 of the term) and that of X and A (the same); fp32 accumulation of A's
        # 131072 terms on either side, random signs, 2^-24 sqrt(131072) = 2^-15.5
        tol = 2.0 ** -8 * float(want.norm()) + 4 * 2.0 ** -11 * float(part.norm())
        assert float(part.norm()) >= 20 * tol
        d = out[first:first + 64].double() - want
        assert float(d.norm()) <= tol
        # and box by box: twice the share of a box of a row of 513
        share = N.box_norms(d) / N.box_norms(want)
        assert float(share.max()) <= 2 * tol / float(want.norm())
