"""The feed-forward block in calls that a user's program makes around it."""
import pytest

pytestmark = pytest.mark.gpu


def _mods():
    import torch
    from blockwise_fp8_linear_fp8bw_b200 import mlp
    return torch, mlp


def _block(torch, mlp, hidden=272, ffn=400, seed=0):
    torch.manual_seed(seed)
    return mlp.BlockwiseFp8MLP(hidden, ffn, device="cuda")


def _inputs(torch, shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(*shape, generator=g, device="cuda").bfloat16() for _ in range(3)]


@pytest.mark.parametrize("shape", [(33, 272), (48, 272), (1, 272), (3, 7, 272), (2, 16, 272)])
@pytest.mark.parametrize("residual", [False, True])
def test_the_output_may_be_changed_in_place(shape, residual):
    """As a residual stream is added into it, with and without gradients."""
    torch, mlp = _mods()
    m = _block(torch, mlp)
    x, r, dy = _inputs(torch, shape, 1)
    r = r if residual else None
    add = torch.ones(shape, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    grads, ys = [], []
    for in_place in (False, True):
        xx = x.clone().requires_grad_()
        y, h = m(xx, r)
        assert y.shape == h.shape == x.shape
        if in_place:
            y += add
        else:
            y = y + add
        y.backward(dy)
        ys.append(y.detach())
        grads.append([xx.grad, add.grad, *(p.grad for p in m.parameters())])
        add.grad = None
        m.zero_grad()
    assert torch.equal(*ys) and all(torch.equal(a, b) for a, b in zip(*grads))
    with torch.no_grad():
        y, _ = m(x, r)
        # (torch refuses to change a view made without gradients with them, as of any
        # module that brings its result into another shape)
        y = y if len(shape) == 2 else y.clone()
    y += add
    assert torch.equal(y.detach(), ys[0])


def test_a_captured_backward_pass_beside_an_eager_graph():
    """It is refused while a graph of the default stream holds the leaves, with the
    process and the device as they were, and works once that graph is gone."""
    torch, mlp = _mods()
    m = _block(torch, mlp)
    x, r, dy = _inputs(torch, (32, 272), 2)
    x.requires_grad_()
    for w in (m.w_gate_up, m.w_down):
        w.main_grad = torch.zeros(w.shape, device="cuda")

    def step():
        y, h = m(x, r)
        return torch.autograd.grad([y, h], [x, m.gamma], [dy, dy])

    s = torch.cuda.Stream()
    held = m(x, r)                                # on the default stream, kept
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = step()                             # eager, on another stream: fine
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="default stream still holds"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, step()))
    del held
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = step()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del g
