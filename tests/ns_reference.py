"""What the Newton-Schulz kernels' number formats cost, simulated in 64 bits, and the
bounds that follow for their results (no code of the library).

Operands are fp16, the iterate is an fp16 pair hi + lo / 2048, everything else is
exact here. The kernels add fp32 accumulation (2^-24, nothing beside fp16's 2^-11),
so their rounding errors before the bf16 result are another draw of the same size as
the simulated ones: within twice those of the 64-bit result, and off by half a bf16
step (2^-8 relative) after it.
"""
import torch

XS, AS, QS, LS = 1024.0, 4096.0, 1024.0, 2048.0      # powers of two things are stored times


def product_coefficients(n, k):
    """(a, b, c) for which a step's products weigh more than a X does: a Gaussian
    n x k matrix of norm 1 has A = X X^T of norm top or so, and a + b s + c s^2 is
    0.5 for s = 0 and 2.5 for s = top."""
    r, c = min(n, k), max(n, k)
    top = (1 + (r / c) ** 0.5) ** 2 / r
    return 0.5, 3.0 / top, -1.0 / top ** 2


def simulate(g, steps, coeffs, eps, pairs=False, operand=torch.float16, low=True, lose=None):
    """The iteration in the kernels' number formats, without the rounding of the result.
    `pairs`: the first two and, from five steps on, the last two steps on the short
    side. Mistakes to plant: another `operand` format, no `low` half, and `lose`, a
    function (name of a matrix, matrix) -> matrix."""
    a, b, c = coeffs
    lose = lose or (lambda name, m: m)

    def op(name, m):
        return lose(name, m.to(operand).double())

    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = (x * (XS / (x.norm() + eps))).float().double()

    def split(v):
        hi = op("X", v)
        return hi, ((v - hi) * LS).to(torch.float16).double() / LS if low else torch.zeros_like(hi)

    def shift(i):
        return a + b + c if i >= 3 else a

    def poly(i, m):
        eye = torch.eye(m.shape[0], dtype=m.dtype, device=m.device)
        return op("P", c / AS * (m @ m) + b * m - (shift(i) - a) * AS * eye)

    hi, lo = split(x)
    i = 0
    while i < steps:
        two = pairs and i + 2 <= steps and (i == 0 or (steps >= 5 and i == steps - 2))
        m0 = op("A", hi @ hi.t() * (AS / XS ** 2))
        p0 = poly(i, m0)
        if two:
            t = op("T", p0 @ m0 / AS + shift(i) * m0)
            m1 = op("A", t @ p0 / AS + shift(i) * t)
            p1 = poly(i + 1, m1)
            q = op("Q", QS / AS ** 2 * (p0 @ p1) + shift(i + 1) * QS / AS * p0
                   + shift(i) * QS / AS * p1)
            x = shift(i) * shift(i + 1) * (hi + lo) + q @ hi / QS
        else:
            x = shift(i) * (hi + lo) + p0 @ hi / AS
        hi, lo = split(x)
        i += 2 if two else 1
    x = lose("result", x / XS)
    return x.t() if tall else x


def box_norms(m):
    """Norms of the 32 x 32 boxes of m."""
    n, k = m.shape
    m = torch.nn.functional.pad(m, (0, -k % 32, 0, -n % 32))
    return m.reshape(m.shape[0] // 32, 32, -1, 32).square().sum((1, 3)).sqrt()


class Bound:
    """Of a result for g: its distance from the 64-bit result, as a whole and in each
    box of 32 x 32."""

    def __init__(self, g, steps, coeffs, eps=1e-7):
        import layer_reference as R
        self.exact = R.newton_schulz(g, steps, coeffs, eps)
        sims = [simulate(g, steps, coeffs, eps, pairs) - self.exact for pairs in (False, True)]
        self.off = 2.0 ** -8 * float(self.exact.norm()) + 2 * max(float(s.norm()) for s in sims)
        self.box = 2.0 ** -8 * box_norms(self.exact) + 2 * max(float(box_norms(s).max())
                                                                for s in sims)

    def ok(self, got):
        d = got.double() - self.exact
        return float(d.norm()) <= self.off and bool((box_norms(d) <= self.box).all())
