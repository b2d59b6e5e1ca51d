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
