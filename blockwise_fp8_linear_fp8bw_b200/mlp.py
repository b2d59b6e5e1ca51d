"""A transformer layer's feed-forward block on the blockwise-FP8 path.

    h = x + residual                       (bf16 residual stream)
    y = W_down (silu(G) * U),   [G | U] = W_gate_up rmsnorm(h)

with the linears' operands coming as E4M3 codes straight from what produces
them (Puro-2B report, paperlayer.ai summary, Appendix C, "FP8 implementation
pipeline": the linears' GEMMs in E4M3, hidden and residual flow in bf16):

  forward   residual addition + norm -> row-wise (fprop) and column-wise
            (wgrad) codes; gate/up fprop -> bf16; gated product -> codes both
            ways; down fprop -> bf16
  backward  dY -> codes both ways; down dgrad -> bf16; the gated product's
            backward -> codes of d[G | U] both ways (nothing of it in bf16);
            gate/up dgrad -> bf16; the norm's backward, with the residual
            stream's gradient added; both weight gradients in one launch

The norm's and the gated product's outputs are rounded once, to E4M3. Any number
of tokens works: rows are padded to a multiple of 16 with zero codes.
"""
import torch
from torch.autograd.function import once_differentiable

from . import ops


def _pad_tokens(t):
    """`t` [tokens, n] with zero rows up to a multiple of 16."""
    extra = -t.shape[0] % 16
    t = t.contiguous()
    return torch.nn.functional.pad(t, (0, 0, 0, extra)) if extra else t


def _first_rows(t, n):
    """The first n rows of `t`, just made here, as a tensor of their own and not a view
    of it: what a Function returns may be changed in place, a view would not."""
    if t.shape[0] == n:
        return t
    return t.new_empty(0).set_(t.untyped_storage(), 0, (n, t.shape[1]), t.stride())


def _bf16_rows(t, k, name):
    if not t.is_cuda or t.dtype != torch.bfloat16 or t.shape[-1] != k:
        raise ValueError("%s: expected a bf16 CUDA tensor with %d features, got %s %s on %s"
                         % (name, k, t.dtype, tuple(t.shape), t.device))
    return (t if t.dim() == 2 else t.reshape(-1, k)).contiguous()


def _refuse_mixed_capture(ctx):
    """Under capture: raise if the gradient of one of the block's leaves is accumulated
    on the default stream, by a node that a graph made there still holds. Autograd would
    have the two streams wait for one another, which ends the capture and, from its
    worker thread, the process."""
    if not torch.cuda.is_current_stream_capturing():
        return
    for node, _ in ctx.next_functions:
        leaf = getattr(node, "variable", None)
        if leaf is not None and ops.accumulates_on_default_stream(leaf):
            raise RuntimeError(
                "BlockwiseFp8MLP: a graph made on the default stream still holds a %s leaf "
                "of this backward pass; let go of it, or warm up on the stream that captures"
                % (tuple(leaf.shape),))


class BlockwiseFp8MLPFunction(torch.autograd.Function):
    """(x, residual, gamma, w_gate_up, w_down) -> (y, h), or y alone without a
    residual (h is x then); see the module docstring. 2-D x and residual."""

    @staticmethod
    def forward(ctx, x, residual, gamma, w_gate_up, w_down, eps, pow2):
        n = ops.rmsnorm_quantize(x, gamma, residual, eps, colwise=True, pow2=pow2)
        (qw1, sw1, qw1_t), (qw2, sw2, qw2_t) = ops.quantize_weight_block_batch(
            [w_gate_up.contiguous(), w_down.contiguous()], pow2=pow2)
        gu = ops.gemm_fprop(n.q, n.s, qw1, sw1, pow2=pow2)
        a = ops.swiglu_quantize(gu, colwise=True, pow2=pow2)
        y = _first_rows(ops.gemm_fprop(a.q, a.s, qw2, sw2, pow2=pow2), x.shape[0])
        ctx.save_for_backward(n.h, n.rstd, gamma, n.q_t, n.s_t, gu, a.q_t, a.s_t,
                              qw1_t, sw1, qw2_t, sw2)
        ctx.weights = (w_gate_up, w_down)
        ctx.pow2 = pow2
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)     # no zeros for an unused y or h
        return (y, n.h) if ctx.has_residual else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        _refuse_mixed_capture(ctx)
        (h, rstd, gamma, qx_t, sx_t, gu, qa_t, sa_t, qw1_t, sw1, qw2_t,
         sw2) = ctx.saved_tensors
        pow2, weights = ctx.pow2, ctx.weights
        tokens = h.shape[0]
        if dy is None:
            dy = torch.zeros((tokens, weights[1].shape[0]), dtype=torch.bfloat16,
                             device=h.device)
        qdy_t, sdy_t, qdy, sdy = ops.quantize_colwise(
            _pad_tokens(dy), with_rowwise=True, pow2=pow2)
        da = ops.gemm_dgrad(qdy, sdy, qw2_t, sw2, pow2=pow2)
        d = ops.swiglu_backward_quantize(da, gu, pow2=pow2)
        dx = dgamma = None
        if ctx.needs_input_grad[0] or ctx.needs_input_grad[1] or ctx.needs_input_grad[2]:
            dn = ops.gemm_dgrad(d.q, d.s, qw1_t, sw1, pow2=pow2)[:tokens]
            dx, dgamma = ops.rmsnorm_backward(
                dn, h, rstd, gamma, None if dh is None else dh.contiguous())
            dgamma = dgamma.to(gamma.dtype)
        jobs = [(3, (d.q_t, d.s_t, qx_t, sx_t)), (4, (qdy_t, sdy_t, qa_t, sa_t))]
        grads = {3: None, 4: None}
        jobs = [(i, op) for i, op in jobs if ctx.needs_input_grad[i]]
        mains = [(i, op) for i, op in jobs if getattr(weights[i - 3], "main_grad", None) is not None]
        plain = [(i, op) for i, op in jobs if getattr(weights[i - 3], "main_grad", None) is None]
        if mains:
            ops.gemm_wgrad_f32_batch([op for _, op in mains],
                                     main_grads=[weights[i - 3].main_grad for i, _ in mains],
                                     pow2=pow2)
        if plain:
            for (i, _), dw in zip(plain, ops.gemm_wgrad_batch([op for _, op in plain],
                                                              pow2=pow2)):
                grads[i] = dw.to(weights[i - 3].dtype)
        # x and the residual have the same gradient; each gets memory of its own
        # (autograd may keep what it is given and add to it in place)
        dr = None
        if ctx.needs_input_grad[1]:
            dr = dx.clone() if ctx.needs_input_grad[0] else dx
        return (dx if ctx.needs_input_grad[0] else None, dr,
                dgamma if ctx.needs_input_grad[2] else None,
                grads[3], grads[4], None, None)


class BlockwiseFp8MLP(torch.nn.Module):
    """Pre-norm gated feed-forward block (hidden -> 2 x ffn -> hidden).

    `forward(x, residual)` returns (y, h): h is the bf16 sum that was normalised,
    the residual of the next block (x itself without a residual). bf16 weights
    `w_gate_up` [2 ffn, hidden] (gate rows first) and `w_down` [hidden, ffn], and
    the norm's `gamma`; a weight's fp32 `main_grad`, if it has one, receives its
    gradient as in BlockwiseFp8Linear.

    Without gradients only the row-wise codes are computed; `freeze()` then keeps
    the weights' codes for the calls that follow (until `unfreeze()`).

    A training step can be captured into a CUDA graph. Warm up on the stream that
    will capture, or let go of what eager steps returned before capturing: while a
    graph made on the default stream holds the leaves, autograd would synchronise with
    that stream, and the captured backward pass raises instead."""

    def __init__(self, hidden, ffn, eps=1e-6, device=None, pow2=False):
        super().__init__()
        if hidden % 16 or ffn % 16:
            raise ValueError("hidden and ffn must be multiples of 16")
        self.hidden, self.ffn, self.eps, self.pow2 = hidden, ffn, eps, pow2
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.gamma = torch.nn.Parameter(torch.ones(hidden, **bf16))
        w1, w2 = torch.empty(2 * ffn, hidden, **bf16), torch.empty(hidden, ffn, **bf16)
        torch.nn.init.normal_(w1, std=0.02)
        torch.nn.init.normal_(w2, std=0.02)
        self.w_gate_up = torch.nn.Parameter(w1)
        self.w_down = torch.nn.Parameter(w2)
        self._codes = None

    def _weight_codes(self):
        return ops.quantize_weight_block_batch(
            [self.w_gate_up.detach().contiguous(), self.w_down.detach().contiguous()],
            transposed=False, pow2=self.pow2)

    def freeze(self):
        """Keep the weights' codes (for inference: later changes of the weights
        are not seen before unfreeze())."""
        self._codes = self._weight_codes()

    def unfreeze(self):
        self._codes = None

    def _infer(self, x, residual):
        (qw1, sw1, _), (qw2, sw2, _) = self._codes or self._weight_codes()
        n = ops.rmsnorm_quantize(x, self.gamma.detach(), residual, self.eps, pow2=self.pow2)
        gu = ops.gemm_fprop(n.q, n.s, qw1, sw1, pow2=self.pow2)
        a = ops.swiglu_quantize(gu, pow2=self.pow2)
        y = ops.gemm_fprop(a.q, a.s, qw2, sw2, pow2=self.pow2)
        return _first_rows(y, x.shape[0]), n.h

    def forward(self, x, residual=None):
        shape = x.shape
        x2 = _bf16_rows(x, self.hidden, "x")
        r2 = None
        if residual is not None:
            if residual.shape != shape:
                raise ValueError("residual: expected %s, got %s"
                                 % (tuple(shape), tuple(residual.shape)))
            r2 = _bf16_rows(residual, self.hidden, "residual")
        leaves = (x2, r2, self.gamma, self.w_gate_up, self.w_down)
        if not torch.is_grad_enabled() or not any(
                t is not None and t.requires_grad for t in leaves):
            y, h = self._infer(x2, r2)
        elif r2 is None:
            y, h = BlockwiseFp8MLPFunction.apply(x2, None, self.gamma, self.w_gate_up,
                                                 self.w_down, self.eps, self.pow2), x2
        else:
            y, h = BlockwiseFp8MLPFunction.apply(x2, r2, self.gamma, self.w_gate_up,
                                                 self.w_down, self.eps, self.pow2)
        return (y, h) if len(shape) == 2 else (y.reshape(shape), h.reshape(shape))

    def extra_repr(self):
        return "hidden=%d, ffn=%d, eps=%g, pow2=%s" % (self.hidden, self.ffn, self.eps, self.pow2)


__all__ = ["BlockwiseFp8MLP", "BlockwiseFp8MLPFunction"]
