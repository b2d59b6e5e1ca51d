"""The bounds that the Newton-Schulz kernels are held to, on the CPU: the number formats
keep them, and results with a mistake planted in the simulation do not."""
import pytest
import torch

import layer_reference as R
import ns_reference as N

USUAL = (3.4445, -4.7750, 2.0315)


def gaussian(n, k, seed, directions=0.0):
    gen = torch.Generator().manual_seed(seed)
    g = torch.randn(n, k, generator=gen, dtype=torch.float64) * 1e-3
    if directions:
        u = torch.linalg.qr(torch.randn(n, 4, generator=gen, dtype=torch.float64))[0]
        v = torch.linalg.qr(torch.randn(k, 4, generator=gen, dtype=torch.float64))[0]
        g = g + directions * u @ v.t()
    return g.float()


def lost(at, which, rows=slice(32, 64), cols=slice(64, 96)):
    """A 32 x 32 box of zeros in the `at`-th matrix called `which`."""
    seen = []

    def lose(name, m):
        if name == which:
            seen.append(0)
            if len(seen) - 1 == at:
                m = m.clone()
                m[rows, cols] = 0
        return m
    return lose


@pytest.mark.parametrize("shape", [(272, 528), (528, 272), (256, 256), (96, 400)])
@pytest.mark.parametrize("directions", [0.0, 20.0])
@pytest.mark.parametrize("steps", [1, 2, 5])
def test_the_formats_keep_the_bound(shape, directions, steps):
    g = gaussian(*shape, 1, directions)
    bound = N.Bound(g, steps, USUAL)
    for pairs in (False, True):
        assert bound.ok(N.simulate(g, steps, USUAL, 1e-7, pairs).bfloat16())
    # the kernels' normalisation is the formula's
    assert torch.equal(bound.exact, R.newton_schulz(g, steps, USUAL, 1e-7))


@pytest.mark.parametrize("pairs", [False, True])
def test_planted_mistakes_do_not(pairs):
    # (the pair matters where a few directions stand far above the rest)
    g, low = gaussian(272, 528, 2), gaussian(272, 528, 2, 20.0)
    ok, ok_low = N.Bound(g, 5, USUAL).ok, N.Bound(low, 5, USUAL).ok

    def run(m, **kw):
        return N.simulate(m, 5, USUAL, 1e-7, pairs, **kw).bfloat16()
    assert ok(run(g)) and ok_low(run(low))
    assert not ok(run(g, operand=torch.bfloat16))
    assert not ok_low(run(low, low=False))
    # (of the first A, whose off-diagonal entries are small yet, see the next test)
    for at, which in ((0, "result"), (2, "A"), (2, "P"), (1, "X")):
        assert not ok(run(g, lose=lost(at, which))), which
    if pairs:
        for which in ("T", "Q"):
            assert not ok(run(g, lose=lost(0, which))), which


@pytest.mark.parametrize("shape", [(256, 768), (768, 256), (512, 512)])
def test_a_single_step_whose_products_count(shape):
    """One step of the usual coefficients on a wide matrix is nearly a X: with these the
    product term is most of the result, and a lost box of any matrix shows."""
    g = gaussian(*shape, 3)
    coeffs = N.product_coefficients(*shape)
    bound = N.Bound(g, 1, coeffs)
    a_part = coeffs[0] * g.double() / (g.double().norm() + 1e-7)
    assert float((bound.exact - a_part).norm()) >= 50 * bound.off
    assert bound.ok(N.simulate(g, 1, coeffs, 1e-7).bfloat16())
    assert not bound.ok(a_part.bfloat16())
    for which in ("A", "P", "X"):
        assert not bound.ok(N.simulate(g, 1, coeffs, 1e-7, lose=lost(0, which)).bfloat16()), which
