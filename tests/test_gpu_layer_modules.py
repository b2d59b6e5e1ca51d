"""The operators together, as a training step uses them: the feed-forward block
(forward, backward, inference) and the optimiser on its weights."""
import pytest

pytestmark = pytest.mark.gpu


def _mods():
    import torch
    from blockwise_fp8_linear_fp8bw_b200 import mlp, muon, ops
    return torch, ops, mlp, muon


def _block(torch, mlp, hidden=272, ffn=400, pow2=False, seed=0):
    torch.manual_seed(seed)
    m = mlp.BlockwiseFp8MLP(hidden, ffn, device="cuda", pow2=pow2)
    with torch.no_grad():
        m.gamma.copy_(1 + 0.2 * torch.randn(hidden, device="cuda"))
        m.w_gate_up.copy_(torch.randn(2 * ffn, hidden, device="cuda") * 0.06)
        m.w_down.copy_(torch.randn(hidden, ffn, device="cuda") * 0.05)
    return m


def _inputs(torch, tokens, hidden, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda: torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()   # noqa: E731
    return r(), r(), r(), r()


def _exact(torch, m, x, r, dy, dh, eps=1e-6):
    """The block without any rounding but h's, in 64 bits, and its gradients."""
    leaves = [t.detach().double().requires_grad_() for t in
              (m.gamma, m.w_gate_up, m.w_down)]
    gamma, w1, w2 = leaves
    h0 = x if r is None else (x.float() + r.float()).bfloat16()
    h = h0.double().requires_grad_()
    n = h * (h.square().mean(1, keepdim=True) + eps).rsqrt() * gamma
    gate, up = (n @ w1.t()).chunk(2, 1)
    y = (torch.nn.functional.silu(gate) * up) @ w2.t()
    loss = (y * dy.double()).sum() + (h * dh.double()).sum()
    return y, torch.autograd.grad(loss, [h] + leaves)


# E4M3 operands are off by at most 2^-4 relative, 0.036 rms; two per product and at
# most three products in a row, with a factor of up to two from the gate's slope:
# sqrt(6) * 0.036 * 2 = 0.18 of the norm. A missing term or a wrong sign is off by
# 1 or more.
QUANT = 0.25


def _near(got, want):
    got, want = got.detach().double(), want.detach()
    return float((got - want).norm()) <= QUANT * float(want.norm())


@pytest.mark.parametrize("tokens,hidden,ffn", [(1, 16, 16), (33, 272, 400), (256, 512, 256)])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("pow2", [False, True])
def test_block_forward_backward(tokens, hidden, ffn, residual, pow2):
    torch, ops, mlp, _ = _mods()
    m = _block(torch, mlp, hidden, ffn, pow2)
    x, r, dy, dh = _inputs(torch, tokens, hidden, 5)
    x.requires_grad_()
    r = r.requires_grad_() if residual else None
    y, h = m(x, r)
    torch.autograd.backward([y, h], [dy, dh])
    ops.fp8bw_check_device_error()
    # the operators one by one give the same bits
    n = ops.rmsnorm_quantize(x.detach(), m.gamma.detach(), None if r is None else r.detach(),
                             colwise=True, pow2=pow2)
    q1, s1, _ = ops.quantize_weight_block(m.w_gate_up.detach(), pow2=pow2)
    q2, s2, q2_t = ops.quantize_weight_block(m.w_down.detach(), pow2=pow2)
    gu = ops.gemm_fprop(n.q, n.s, q1, s1, pow2=pow2)
    a = ops.swiglu_quantize(gu, colwise=True, pow2=pow2)
    assert torch.equal(y, ops.gemm_fprop(a.q, a.s, q2, s2, pow2=pow2)[:tokens])
    assert torch.equal(h, n.h)
    pad = torch.zeros(n.q.shape[0], hidden, device="cuda").bfloat16()
    pad[:tokens] = dy
    qdy_t, sdy_t, qdy, sdy = ops.quantize_colwise(pad, with_rowwise=True, pow2=pow2)
    assert torch.equal(m.w_down.grad, ops.gemm_wgrad(qdy_t, sdy_t, a.q_t, a.s_t, pow2=pow2))
    d = ops.swiglu_backward_quantize(ops.gemm_dgrad(qdy, sdy, q2_t, s2, pow2=pow2), gu, pow2=pow2)
    assert torch.equal(m.w_gate_up.grad, ops.gemm_wgrad(d.q_t, d.s_t, n.q_t, n.s_t, pow2=pow2))
    # against the block in 64 bits
    ye, (dx, dgamma, dw1, dw2) = _exact(torch, m, x, r, dy, dh)
    assert _near(y, ye)
    if hidden >= 256:
        for got, want in ((x.grad, dx), (m.gamma.grad, dgamma), (m.w_gate_up.grad, dw1),
                          (m.w_down.grad, dw2)):
            assert _near(got, want)
    if residual:
        assert torch.equal(x.grad, r.grad)
    # no gradients: row-wise codes only, the same output; with kept codes too
    with torch.no_grad():
        y2, h2 = m(x, r)
        m.freeze()
        y3, _ = m(x, r)
    assert torch.equal(y2, y) and torch.equal(h2, h) and torch.equal(y3, y)


def test_main_grads_accumulate_and_frozen_weights():
    torch, _, mlp, _ = _mods()
    m = _block(torch, mlp)
    x, r, dy, dh = _inputs(torch, 48, 272, 9)
    m.w_gate_up.main_grad = torch.zeros(m.w_gate_up.shape, device="cuda")
    m.w_down.requires_grad_(False)
    for _ in range(2):
        y, h = m(x, r)
        torch.autograd.backward([y, h], [dy, dh])
    once = _block(torch, mlp)
    y, h = once(x, r)
    torch.autograd.backward([y, h], [dy, dh])
    assert m.w_gate_up.grad is None and m.w_down.grad is None
    # two equal gradients added in fp32: twice the one, whose bf16 form is off by 2^-8
    got, want = m.w_gate_up.main_grad / 2, once.w_gate_up.grad.float()
    assert bool(((got - want).abs() <= 2.0 ** -8 * got.abs()).all())


def test_gradients_of_one_output_alone_and_accumulated():
    torch, _, mlp, _ = _mods()
    m = _block(torch, mlp)
    x, r, dy, dh = _inputs(torch, 40, 272, 11)
    x.requires_grad_(), r.requires_grad_()
    zero = torch.zeros_like(dy)
    for use_y in (True, False):
        y, h = m(x, r)
        alone = torch.autograd.grad(y if use_y else h, [x, m.gamma], dy if use_y else dh)
        y, h = m(x, r)
        both = torch.autograd.grad([y, h], [x, m.gamma], [dy, zero] if use_y else [zero, dh])
        assert all(torch.equal(a, b) for a, b in zip(alone, both))
    # x and the residual receive the same gradient, but not the same memory
    for _ in range(2):
        y, h = m(x, r)
        torch.autograd.backward([y, h], [dy, dh])
    y, h = m(x, r)
    one = torch.autograd.grad([y, h], x, [dy, dh])[0]
    assert torch.equal(x.grad, one + one) and torch.equal(r.grad, one + one)


def test_block_refusals():
    torch, _, mlp, _ = _mods()
    m = _block(torch, mlp)
    x, r, _, _ = _inputs(torch, 16, 272, 1)
    for bad in (x.float(), x[:, :256], x.cpu()):
        with pytest.raises(ValueError, match="x: expected"):
            m(bad)
    with pytest.raises(ValueError, match="residual"):
        m(x, r[:8])
    with pytest.raises(ValueError, match="multiples of 16"):
        mlp.BlockwiseFp8MLP(100, 64)


def test_training_step_with_the_optimiser():
    """Two micro-batches into fp32 main-grads, then MuonH: the update is the
    orthogonalised momentum, the norm of every weight stays what it was."""
    torch, ops, mlp, muon = _mods()
    m = _block(torch, mlp)
    weights = [m.w_gate_up, m.w_down]
    for w in weights:
        w.main_grad = torch.zeros(w.shape, device="cuda")
    opt = muon.MuonH(weights, lr=0.01, momentum=0.9)
    before = [w.detach().clone() for w in weights]
    moments = [torch.zeros(w.shape, device="cuda", dtype=torch.float64) for w in weights]
    radius = [w.detach().double().norm() for w in weights]
    master = [w.detach().double() for w in weights]
    for step in range(2):
        for w in weights:
            w.main_grad.zero_()
        for micro in range(2):
            x, r, dy, dh = _inputs(torch, 40, 272, 20 + 2 * step + micro)
            y, h = m(x, r)
            torch.autograd.backward([y, h], [dy, dh])
        opt.step()
        for i, w in enumerate(weights):
            g = w.main_grad.double()
            moments[i] = 0.9 * moments[i] + g
            u = (g + 0.9 * moments[i]).float()
            o = ops.newton_schulz(u).double()
            n, k = w.shape
            master[i] = master[i] - 0.01 * max(1.0, n / k) ** 0.5 * o
            master[i] = master[i] * radius[i] / master[i].norm()
            # bf16 weights of an fp32 master: half a step, plus what fp32 rounding
            # of u (2^-23 per operation) moves the orthogonalised update by
            tol = 2.0 ** -8 * master[i].abs() + 0.01 * 2.0 ** -8 * 3
            assert bool(((w.detach().double() - master[i]).abs() <= tol).all())
            assert abs(float(w.detach().double().norm() / radius[i]) - 1) <= 2.0 ** -8
    assert all(not torch.equal(a, b) for a, b in zip(before, weights))


def test_optimiser_without_projection_and_its_refusals():
    torch, ops, _, muon = _mods()
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.nn.Parameter(torch.randn(64, 32, generator=g, device="cuda"))
    w.grad = torch.randn(64, 32, generator=g, device="cuda")
    start = w.detach().clone()
    opt = muon.MuonH([w], lr=0.1, nesterov=False, project=False)
    opt.step()
    want = start - 0.1 * 2.0 ** 0.5 * ops.newton_schulz(w.grad).float()
    assert bool(((w.detach() - want).abs() <= 2.0 ** -22 * (start.abs() + 0.2)).all())
    saved = opt.state_dict()
    other = muon.MuonH([torch.nn.Parameter(start.clone())], lr=0.1)
    other.load_state_dict(saved)
    with pytest.raises(ValueError, match="multiples"):
        muon.MuonH([torch.nn.Parameter(torch.zeros(24, 32))])
    with pytest.raises(ValueError, match="momentum"):
        muon.MuonH([w], momentum=1.0)


def test_step_in_a_graph():
    """The block's forward and backward captured and replayed with new inputs."""
    torch, _, mlp, _ = _mods()
    m = _block(torch, mlp)
    for w in (m.w_gate_up, m.w_down):
        w.main_grad = torch.zeros(w.shape, device="cuda")
    x, r, dy, dh = _inputs(torch, 80, 272, 31)
    x.requires_grad_()

    def step():
        y, h = m(x, r)
        return y.detach(), *torch.autograd.grad([y, h], [x, m.gamma], [dy, dh])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = step()
    fresh = _inputs(torch, 80, 272, 32)
    with torch.no_grad():
        for t, f in zip((x, r, dy, dh), fresh):
            t.copy_(f)
    for w in (m.w_gate_up, m.w_down):
        w.main_grad.zero_()
    g.replay()
    torch.cuda.synchronize()
    mains = [w.main_grad.clone() for w in (m.w_gate_up, m.w_down)]
    for w in (m.w_gate_up, m.w_down):
        w.main_grad.zero_()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.equal(a, w.main_grad) for a, w in zip(mains, (m.w_gate_up, m.w_down)))
    del g


@pytest.mark.parametrize("residual", [True, False])
def test_no_tokens(residual):
    """A block over an empty batch: empty results, zero gradients."""
    torch, _, mlp, _ = _mods()
    m = _block(torch, mlp)
    x, r, dy, _ = (t[:0] for t in _inputs(torch, 1, 272, 41))
    x.requires_grad_()
    y, h = m(x, r if residual else None)
    y.backward(dy)
    assert y.shape == h.shape == x.grad.shape == (0, 272)
    assert all(not p.grad.any() for p in m.parameters())
    with torch.no_grad():
        assert m(x)[0].shape == (0, 272)


def test_second_derivatives_are_refused():
    torch, _, mlp, _ = _mods()
    m = _block(torch, mlp)
    x, _, dy, _ = _inputs(torch, 16, 272, 42)
    x.requires_grad_()
    y, _ = m(x)
    dx, = torch.autograd.grad(y, x, dy.requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.float().sum().backward()


def test_optimiser_refuses_to_capture_its_first_step():
    """Its state would be set up anew in every replay. A later step replays as it
    runs eagerly."""
    torch, _, _, muon = _mods()
    torch.manual_seed(5)
    start = torch.randn(64, 96, device="cuda")
    grads = [torch.randn(64, 96, device="cuda") for _ in range(3)]
    w, v = (torch.nn.Parameter(start.clone()) for _ in range(2))
    w.grad, v.grad = grads[0].clone(), grads[0].clone()
    opt, eager = muon.MuonH([w], lr=0.1), muon.MuonH([v], lr=0.1)
    with pytest.raises(RuntimeError, match="one step before"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            opt.step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        opt.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        opt.step()
    for grad in grads:
        v.grad.copy_(grad)
        eager.step()
    for grad in grads[1:]:
        w.grad.copy_(grad)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, v)
    del g


def test_running_out_of_memory_raises_torchs_error():
    torch, ops, _, _ = _mods()
    gu = torch.zeros(1 << 14, 1 << 13, dtype=torch.bfloat16, device="cuda")
    torch.cuda.empty_cache()
    used = torch.cuda.memory_reserved()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((used + (16 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            ops.swiglu_quantize(gu)        # 64 MB of codes
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert not ops.swiglu_quantize(gu).q.any()
