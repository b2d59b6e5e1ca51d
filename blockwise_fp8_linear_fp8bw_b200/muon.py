"""MuonH: the recipe's optimiser for the linears' weights -- momentum, an
orthogonalised update, and a projection of the weight back to its initial
Frobenius norm (Puro-2B report, arxiv-wiki summary, "Approach": Muon with a
hyperball projection to the initial Frobenius radius, weight decay 0).

    m <- momentum m + g,   u = g + momentum m  (Nesterov)  or m
    O = newton_schulz(u)                                   (this library)
    W <- W - lr sqrt(max(1, n / k)) O,   W <- W R / ||W||,  R = initial ||W||

The orthogonalisations of all weights run in batched launches (up to eight
matrices each). A weight's gradient is its fp32 `main_grad` if it has one (as the
linears of this library accumulate it), else its `.grad`; `zero_grad()` clears the
latter only, a main_grad is its owner's to clear. Momentum, the master copy of a
bf16 weight and the update are fp32. A weight whose initial norm is 0 stays 0 under
the projection.
"""
import torch

from . import ops


class MuonH(torch.optim.Optimizer):
    """Optimiser of 2-D weights [n, k] with sides that are multiples of 16, up to 2^17.

    `project=False` leaves the projection out (plain Muon)."""

    def __init__(self, params, lr=0.02, momentum=0.95, nesterov=True, steps=5,
                 coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7, project=True):
        if lr < 0 or not 0 <= momentum < 1:
            raise ValueError("lr must be >= 0 and momentum in [0, 1)")
        super().__init__(params, dict(lr=lr, momentum=momentum, nesterov=nesterov, steps=steps,
                                      coeffs=tuple(coeffs), eps=eps, project=project))

    def add_param_group(self, group):
        super().add_param_group(group)
        for p in self.param_groups[-1]["params"]:
            if p.dim() != 2 or p.shape[0] % 16 or p.shape[1] % 16 or max(p.shape) > 1 << 17:
                del self.param_groups[-1]
                raise ValueError("MuonH takes 2-D weights with sides that are multiples of "
                                 "16 and at most 2^17, got %s" % (tuple(p.shape),))

    def load_state_dict(self, state_dict):
        super().load_state_dict(state_dict)
        # the base class rounds a weight's state to the weight's type; it stays fp32
        saved = [i for group in state_dict["param_groups"] for i in group["params"]]
        params = [p for group in self.param_groups for p in group["params"]]
        for i, p in zip(saved, params):
            for key, value in state_dict["state"].get(i, {}).items():
                self.state[p][key] = value.detach().to(
                    device=p.device, dtype=torch.float32, copy=True)

    def _state_of(self, p, group):
        state = self.state[p]
        # (the state of a run whose weights were fp32 has no master)
        master = p.dtype != torch.float32 and "master" not in state
        if (not state or master) and torch.cuda.is_current_stream_capturing():
            # a replay would start from the captured state every time
            raise RuntimeError("MuonH: take one step before capturing one in a graph")
        if not state:
            w = p.detach().float()
            state["momentum"] = torch.zeros_like(w)
            state["radius"] = torch.linalg.vector_norm(w)
        if master:
            state["master"] = p.detach().float().clone()
        return state

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        work = []              # (group, [(weight, gradient)]) of one device
        for group in self.param_groups:
            todo = {}
            for p in group["params"]:
                g = getattr(p, "main_grad", None)
                g = p.grad if g is None else g
                if g is None:
                    continue
                # (before any state changes)
                if not p.is_cuda or g.device != p.device or g.shape != p.shape or g.is_sparse:
                    raise ValueError(
                        "MuonH steps CUDA weights with dense gradients of their shape and "
                        "device, got a weight %s on %s and a gradient %s on %s"
                        % (tuple(p.shape), p.device, tuple(g.shape), g.device))
                todo.setdefault(p.device, []).append((p, g))
            work += [(group, pairs) for pairs in todo.values()]
        for group, pairs in work:
            self._step_device(group, pairs)
        return loss

    def _step_device(self, group, pairs):
        params = [p for p, _ in pairs]
        states = [self._state_of(p, group) for p in params]
        grads = [g.detach().float() for _, g in pairs]
        moments = [s["momentum"] for s in states]
        torch._foreach_mul_(moments, group["momentum"])
        torch._foreach_add_(moments, grads)
        if group["nesterov"]:
            updates = torch._foreach_add(grads, moments, alpha=group["momentum"])
        else:
            updates = moments
        with torch.cuda.device(params[0].device):
            ortho = ops.newton_schulz_batch([u.contiguous() for u in updates],
                                            steps=group["steps"], coeffs=group["coeffs"],
                                            eps=group["eps"])
        for p, s, o in zip(params, states, ortho):
            n, k = p.shape
            w = s.get("master", p)
            w.add_(o, alpha=-group["lr"] * max(1.0, n / k) ** 0.5)
            if group["project"]:
                norm = torch.linalg.vector_norm(w)
                # a zero weight stays zero
                w.mul_(torch.where(norm > 0, s["radius"] / norm, torch.ones_like(norm)))
            if w is not p:
                p.copy_(w)


__all__ = ["MuonH"]
