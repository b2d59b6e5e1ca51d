"""MuonH's state and refusals, without a GPU."""
import pytest
import torch

from blockwise_fp8_linear_fp8bw_b200.muon import MuonH


def _state(opt, w, **more):
    gen = torch.Generator().manual_seed(1)
    opt.state[w] = {"momentum": torch.randn(w.shape, generator=gen),
                    "radius": torch.tensor(3.0), **more}


def test_a_bf16_weight_has_a_master_whatever_was_loaded(monkeypatch):
    """The state of a run with fp32 weights has none: the bf16 weight's own value starts
    it, and updates are not rounded to bf16 from step to step."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    old = torch.nn.Parameter(torch.randn(16, 32))
    saved = MuonH([old])
    _state(saved, old)
    w = torch.nn.Parameter(torch.randn(16, 32).bfloat16())
    opt = MuonH([w])
    opt.load_state_dict(saved.state_dict())
    state = opt._state_of(w, opt.param_groups[0])
    assert state["master"].dtype == torch.float32
    assert torch.equal(state["master"], w.detach().float())
    assert state["master"].data_ptr() != w.data_ptr()
    assert torch.equal(state["momentum"], saved.state[old]["momentum"])
    # and one that it has is kept
    state["master"].add_(1e-4)
    kept = state["master"].clone()
    assert torch.equal(opt._state_of(w, opt.param_groups[0])["master"], kept)
    fresh = torch.nn.Parameter(torch.randn(16, 32))
    assert "master" not in MuonH([fresh])._state_of(fresh, {})
