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


@pytest.mark.parametrize("make", [
    lambda w: torch.zeros(16, 32),                          # (the weight is on the CPU)
    lambda w: torch.zeros(32, 16),
    lambda w: torch.zeros(16, 32, device="meta"),
])
def test_what_a_step_cannot_take_is_refused_before_any_state_changes(make):
    first = torch.nn.Parameter(torch.randn(16, 32))
    w = torch.nn.Parameter(torch.randn(16, 32))
    opt = MuonH([first, w])
    _state(opt, w)
    before = {k: v.clone() for k, v in opt.state[w].items()}
    value = w.detach().clone()
    w.main_grad = make(w)
    with pytest.raises(ValueError, match="CUDA weights"):
        opt.step()
    assert torch.equal(w.detach(), value) and not opt.state[first]
    assert all(torch.equal(v, before[k]) for k, v in opt.state[w].items())


def test_sides_beyond_the_librarys_are_refused():
    w = torch.nn.Parameter(torch.empty((1 << 17) + 16, 16, device="meta"))
    with pytest.raises(ValueError, match="at most 2"):
        MuonH([w])
    MuonH([torch.nn.Parameter(torch.empty(1 << 17, 16, device="meta"))])


def test_no_state_is_set_up_under_capture(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    w = torch.nn.Parameter(torch.randn(16, 32).bfloat16())
    opt = MuonH([w])
    _state(opt, w)                                # without a master
    for _ in range(2):
        with pytest.raises(RuntimeError, match="one step before"):
            opt._state_of(w, {})
        opt.state.pop(w, None)                    # and without any
    _state(opt, w, master=torch.zeros(16, 32))
    opt._state_of(w, {})
