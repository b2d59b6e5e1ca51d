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
