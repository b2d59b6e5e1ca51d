"""The layer operators without a GPU: the header's symbols, the argument
checks of the C ABI (fake pointers, refused before anything is read), and the
binding's own checks."""
import ctypes
import os
import re

import pytest
import torch

from blockwise_fp8_linear_fp8bw_b200 import _native, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8bw_layer.h")

E_NULL, E_SHAPE, E_ALIGN, E_DEVICE, E_ALIAS = -1, -2, -3, -4, -8
P = [0x10000000 * i for i in range(1, 14)]   # fake, aligned, never read


@pytest.fixture(scope="module")
def lib():
    return _native.load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(fp8bw_[a-z_0-9]+)\s*\(", text))
    assert names == set(_native.LAYER_SIGNATURES)
    assert not names & set(_native.SIGNATURES)
    for n in names:
        assert hasattr(lib, n)


def norm_args(rows=10, cols=64, eps=1e-6, **kw):
    a = dict(x=P[0], residual=P[1], gamma=P[2], f32=0, rows=rows, cols=cols, eps=eps,
             h=P[3], rstd=P[4], y=None, q=P[5], s=P[6], q_t=P[7], s_t=P[8], stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), E_SHAPE), (dict(rows=(1 << 30) + 1), E_SHAPE), (dict(cols=24), E_SHAPE),
    (dict(cols=-16), E_SHAPE), (dict(cols=32784), E_SHAPE), (dict(eps=-1.0), E_SHAPE),
    (dict(eps=float("nan")), E_SHAPE), (dict(x=None), E_NULL), (dict(gamma=None), E_NULL),
    (dict(h=None), E_NULL), (dict(residual=None), E_NULL), (dict(s=None), E_NULL),
    (dict(q=None), E_NULL), (dict(q_t=None), E_NULL), (dict(rstd=None), E_NULL),
    (dict(x=P[0] + 8), E_ALIGN), (dict(q=P[5] + 4), E_ALIGN), (dict(h=P[0]), E_ALIAS),
    (dict(q=P[6]), E_ALIAS), (dict(y=P[0] + 16), E_ALIAS), (dict(rstd=P[2] + 112), E_ALIAS),
    (dict(s_t=P[7] + 16 * 64 - 16), E_ALIAS),
])
@pytest.mark.parametrize("name", ["fp8bw_rmsnorm_quantize", "fp8bw_rmsnorm_quantize_pow2"])
def test_norm_refusals(lib, name, change, status):
    assert getattr(lib, name)(*norm_args(**change)) == status


def test_valid_arguments_reach_the_device_check(lib):
    # no GPU here: the first thing after the argument checks fails
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert lib.fp8bw_rmsnorm_quantize(*norm_args()) == E_DEVICE
    assert lib.fp8bw_rmsnorm_quantize(*norm_args(q=None, s=None, y=P[9])) == E_DEVICE
    assert lib.fp8bw_swiglu_quantize(P[0], 5, 32, P[1], P[2], None, None, None) == E_DEVICE
    assert lib.fp8bw_rmsnorm_backward(P[0], P[1], P[2], P[3], 1, None, 5, 64, P[4], P[5], P[6],
                                      1 << 20, None) == E_DEVICE


def test_norm_backward_refusals(lib):
    def call(dy=P[0], h=P[1], rstd=P[2], gamma=P[3], f32=0, dres=P[4], rows=10, cols=64, dh=P[5],
             dgamma=P[6], ws=P[7], size=1 << 20):
        return lib.fp8bw_rmsnorm_backward(dy, h, rstd, gamma, f32, dres, rows, cols, dh, dgamma,
                                          ws, size, None)
    need = lib.fp8bw_rmsnorm_backward_workspace(10, 64)
    assert need > 0 and need % 256 == 0
    assert lib.fp8bw_rmsnorm_backward_workspace(0, 64) == 0
    assert lib.fp8bw_rmsnorm_backward_workspace(10, 40) == E_SHAPE
    assert call(size=need - 1) == E_SHAPE and call(rows=-1) == E_SHAPE
    assert call(cols=32784) == E_SHAPE and call(cols=8) == E_SHAPE
    for kw in ("dy", "h", "rstd", "gamma", "dh", "dgamma", "ws"):
        assert call(**{kw: None}) == E_NULL, kw
        assert call(**{kw: P[9] + 4}) == E_ALIGN, kw
    assert call(dh=P[0]) == E_ALIAS and call(dh=P[4]) == E_ALIAS
    assert call(dgamma=P[2] + 32) == E_ALIAS and call(ws=P[5] + 64) == E_ALIAS


@pytest.mark.parametrize("name,da", [("fp8bw_swiglu_quantize", False),
                                     ("fp8bw_swiglu_quantize_pow2", False),
                                     ("fp8bw_swiglu_backward_quantize", True),
                                     ("fp8bw_swiglu_backward_quantize_pow2", True)])
def test_glu_refusals(lib, name, da):
    def call(gu=P[0], rows=10, f=64, q=P[1], s=P[2], q_t=P[3], s_t=P[4]):
        first = (P[5],) if da else ()
        return getattr(lib, name)(*first, gu, rows, f, q, s, q_t, s_t, None)
    assert call(rows=-1) == E_SHAPE and call(f=40) == E_SHAPE and call(f=-16) == E_SHAPE
    assert call(f=(1 << 22) + 16) == E_SHAPE
    assert call(rows=1 << 30, f=1 << 22) == E_SHAPE       # too many tiles
    assert call(gu=None) == E_NULL and call(q=None) == E_NULL and call(s=None) == E_NULL
    assert call(s_t=None) == E_NULL and call(q_t=None) == E_NULL
    assert call(gu=P[0] + 2) == E_ALIGN and call(s_t=P[4] + 8) == E_ALIGN
    assert call(q=P[0] + 64) == E_ALIAS and call(s=P[1] + 16) == E_ALIAS


def ns_jobs(*specs):
    arr = (_native.NsJob * max(1, len(specs)))()
    for i, sp in enumerate(specs):
        arr[i] = _native.NsJob(*sp)
    return ctypes.cast(arr, ctypes.c_void_p), arr


def test_newton_schulz_refusals(lib):
    ok = (P[0], 64, 128, P[1])
    ok2 = (P[2], 256, 64, P[3])
    p, keep = ns_jobs(ok, ok2)
    need = lib.fp8bw_newton_schulz_workspace(p, 2)
    assert need > 0

    def call(p=p, count=2, f32=1, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, ws=P[4],
             size=need):
        return lib.fp8bw_newton_schulz(p, count, f32, steps, a, b, c, eps, ws, size, None)
    assert call(count=9) == E_SHAPE and call(count=-1) == E_SHAPE
    assert call(steps=0) == E_SHAPE and call(steps=65) == E_SHAPE
    assert call(a=float("inf")) == E_SHAPE and call(c=float("nan")) == E_SHAPE
    assert call(eps=-1.0) == E_SHAPE and call(size=need - 1) == E_SHAPE
    assert call(p=None) == E_NULL and call(ws=None) == E_NULL
    assert call(ws=P[4] + 8) == E_ALIGN and call(ws=P[4] + 16) == E_ALIGN
    assert call(ws=P[0]) == E_ALIAS
    for spec, status in [((P[0], 72, 128, P[1]), E_SHAPE), ((P[0], 64, -16, P[1]), E_SHAPE),
                         ((P[0], (1 << 17) + 16, 16, P[1]), E_SHAPE),
                         ((None, 64, 128, P[1]), E_NULL), ((P[0], 64, 128, None), E_NULL),
                         ((P[0] + 8, 64, 128, P[1]), E_ALIGN), ((P[0], 64, 128, P[0]), E_ALIAS),
                         ((P[0], 64, 128, P[3] + 32), E_ALIAS),
                         ((P[0], 64, 128, P[2]), E_ALIAS)]:
        p2, keep2 = ns_jobs(spec, ok2)
        assert call(p=p2, size=1 << 30, ws=P[8]) == status, spec
    assert lib.fp8bw_newton_schulz_workspace(None, 0) == 0
    assert lib.fp8bw_newton_schulz_workspace(p, 9) == E_SHAPE


def test_binding_refuses_before_the_library():
    bf = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.rmsnorm_quantize(bf, torch.ones(64))
    with pytest.raises(ValueError, match="x: expected"):
        ops.rmsnorm_quantize(bf.float(), torch.ones(64))
    with pytest.raises(ValueError, match="gamma"):
        ops.rmsnorm_quantize(bf, torch.ones(32))
    with pytest.raises(ValueError, match="gamma"):
        ops.rmsnorm_quantize(bf, torch.ones(64, dtype=torch.float16))
    with pytest.raises(ValueError, match="residual"):
        ops.rmsnorm_quantize(bf, torch.ones(64), bf[:2])
    with pytest.raises(ValueError, match="gu"):
        ops.swiglu_quantize(torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="even"):
        ops.swiglu_quantize(torch.zeros(4, 33, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="da"):
        ops.swiglu_backward_quantize(bf, bf)
    with pytest.raises(ValueError, match="rstd"):
        ops.rmsnorm_backward(bf, bf, torch.ones(3), torch.ones(64))
    with pytest.raises(ValueError, match="CUDA"):
        ops.newton_schulz(torch.zeros(32, 32))


def test_optimiser_state_stays_fp32_and_groups_are_checked():
    """Loading a checkpoint does not round the fp32 state to a bf16 weight's type;
    groups added later are checked as the first ones are."""
    from blockwise_fp8_linear_fp8bw_b200.muon import MuonH
    g = torch.Generator().manual_seed(3)
    p = [torch.nn.Parameter(torch.randn(16, 32, generator=g).bfloat16()) for _ in range(2)]
    opt = MuonH(p)
    for w in p:
        opt.state[w] = {"momentum": torch.randn(16, 32, generator=g),
                        "radius": torch.randn((), generator=g),
                        "master": torch.randn(16, 32, generator=g)}
    saved = opt.state_dict()
    q = [torch.nn.Parameter(w.detach().clone()) for w in p]
    new = MuonH(q)
    new.load_state_dict(saved)
    for w, v in zip(p, q):
        for key, t in opt.state[w].items():
            assert new.state[v][key].dtype == torch.float32
            assert torch.equal(new.state[v][key], t)
            assert new.state[v][key].data_ptr() != t.data_ptr()
    for shape in ((16,), (24, 32), (16, 8)):
        with pytest.raises(ValueError, match="multiples of"):
            new.add_param_group({"params": [torch.nn.Parameter(torch.zeros(shape))]})
    assert len(new.param_groups) == 1


def test_binding_passes_errors_of_its_arguments_on():
    class Neither:
        def __bool__(self):
            raise LookupError("neither")

    gu = torch.zeros(16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.swiglu_quantize(gu, colwise=Neither())     # the tensor is refused first
    with pytest.raises(TypeError):
        ops.newton_schulz(torch.zeros(16, 16), steps="5")
