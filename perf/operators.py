"""Cases, plain forms and exact values of the operators that stand around the
blockwise-FP8 linears of a transformer layer:

  norm       residual addition + root-mean-square norm, leaving as E4M3 codes
             with 1x128 scales (row-wise, and column-wise for training)
  norm_bwd   its backward pass (input gradient and the norm weight's)
  glu        SiLU-gated product of a fused gate/up projection, leaving as E4M3
             codes (row-wise, and column-wise for training)
  glu_bwd    its backward pass, leaving as E4M3 codes of the gate/up gradient
  ns         orthogonalisation of weight updates by Newton-Schulz products

`run` computes an operator in its plain form (elementary torch operations in
32 bits) where `own` is false, and by the library's entry points where it is
true. E4M3 codes are returned as float8 numbers beside their fp32 scales.
"""
import math

import torch

own = False

_EPS = 1e-6
_NS = (3.4445, -4.7750, 2.0315)      # quintic iteration coefficients
_NS_EPS = 1e-7


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token entering a layer of hidden size 2048: latency
        {"name": "norm_token", "op": "norm", "tokens": 1, "cols": 2048,
         "residual": True, "colwise": False, "pow2": False, "gamma": "bf16"},
        # a short prompt chunk of ragged length, wide hidden size, no residual
        # (the first layer), power-of-two scales, fp32 norm weight
        {"name": "norm_chunk", "op": "norm", "tokens": 333, "cols": 5136,
         "residual": False, "colwise": False, "pow2": True, "gamma": "f32"},
        # a training micro-batch of 4 x 4096 tokens
        {"name": "norm_train", "op": "norm", "tokens": 16384, "cols": 2048,
         "residual": True, "colwise": True, "pow2": False, "gamma": "bf16"},
        # a packed batch whose token count is no multiple of anything
        {"name": "norm_bwd_ragged", "op": "norm_bwd", "tokens": 1037,
         "cols": 1040, "residual": False, "gamma": "f32"},
        {"name": "norm_bwd_train", "op": "norm_bwd", "tokens": 16384,
         "cols": 2048, "residual": True, "gamma": "bf16"},
        # a few decoded tokens in the feed-forward part
        {"name": "glu_tokens", "op": "glu", "tokens": 7, "f": 6144,
         "colwise": False, "pow2": False},
        {"name": "glu_train", "op": "glu", "tokens": 16384, "f": 6144,
         "colwise": True, "pow2": False},
        {"name": "glu_bwd_ragged", "op": "glu_bwd", "tokens": 777, "f": 1360,
         "pow2": False},
        {"name": "glu_bwd_train", "op": "glu_bwd", "tokens": 16384, "f": 6144,
         "pow2": False},
        # one small weight's update
        {"name": "ns_small", "op": "ns", "shapes": "256x768", "steps": 5,
         "grad": "bf16"},
        # the output projections (2048 x 2048) of eight layers
        {"name": "ns_square", "op": "ns",
         "shapes": ",".join(["2048x2048"] * 8), "steps": 5, "grad": "f32"},
        # the four linears of one layer (QKV, O, gate/up, down)
        {"name": "ns_layer", "op": "ns",
         "shapes": "4096x2048,2048x2048,12288x2048,2048x6144", "steps": 5,
         "grad": "f32"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v / step + 0.5) * step)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "glu", "glu_bwd", "ns"])
    if op in ("norm", "norm_bwd"):
        cols = _log_int(rng, 128, 8192, 16)
        tokens = min(_log_int(rng, 1, 16384), 16384 * 2048 // cols)
        case = {"op": op, "tokens": tokens, "cols": cols,
                "residual": rng.random() < 0.7,
                "gamma": rng.choice(["bf16", "f32"])}
        if op == "norm":
            case["colwise"] = rng.random() < 0.5
            # a power-of-two scale steps by two at its border: small cases
            # only, where no group's maximum is within rounding of one
            case["pow2"] = tokens * cols <= 1 << 21 and rng.random() < 0.3
        return case
    if op in ("glu", "glu_bwd"):
        f = _log_int(rng, 128, 16384, 16)
        tokens = min(_log_int(rng, 1, 16384), 16384 * 6144 // f)
        case = {"op": op, "tokens": tokens, "f": f,
                "pow2": tokens * f <= 1 << 21 and rng.random() < 0.3}
        if op == "glu":
            case["colwise"] = rng.random() < 0.5
        return case
    limit = _ns_flops([(4096, 2048), (2048, 2048), (12288, 2048),
                       (2048, 6144)], 5)
    steps = rng.choice([3, 5, 5, 6])
    shapes = []
    for _ in range(rng.choice([1, 1, 2, 4, 8])):
        s = (_log_int(rng, 64, 6144, 16), _log_int(rng, 64, 6144, 16))
        if _ns_flops(shapes + [s], steps) <= limit:
            shapes.append(s)
    if not shapes:
        shapes = [(_log_int(rng, 64, 2048, 16), _log_int(rng, 64, 2048, 16))]
    return {"op": "ns", "shapes": ",".join("%dx%d" % s for s in shapes),
            "steps": steps, "grad": rng.choice(["bf16", "f32"])}


def _shapes(case):
    return [tuple(int(v) for v in s.split("x"))
            for s in case["shapes"].split(",")]


def _ns_flops(shapes, steps):
    """Per step, with r <= c the sides: the symmetric products X X^T (r^2 c)
    and A A (r^3), each computed in one half, and B X (2 r^2 c)."""
    total = 0.0
    for n, k in shapes:
        r, c = min(n, k), max(n, k)
        total += steps * (3.0 * r * r * c + 1.0 * r * r * r)
    return total


def work(case):
    op = case["op"]
    if op == "norm":
        t, c = case["tokens"], case["cols"]
        g = -(-c // 128)
        rp = -(-t // 16) * 16
        b = 2 * t * c + c * (2 if case["gamma"] == "bf16" else 4) + 4 * t
        if case["residual"]:
            b += 2 * t * c + 2 * t * c          # residual in, sum out
        b += rp * c + 4 * g * rp
        if case["colwise"]:
            b += rp * c + 4 * (-(-rp // 128)) * c
        return {"bytes": b, "flops": 6 * t * c}
    if op == "norm_bwd":
        t, c = case["tokens"], case["cols"]
        b = (2 + 2 + 2) * t * c + 4 * t + c * 8
        if case["residual"]:
            b += 2 * t * c
        return {"bytes": b, "flops": 10 * t * c}
    if op == "glu":
        t, f = case["tokens"], case["f"]
        rp = -(-t // 16) * 16
        b = 4 * t * f + rp * f + 4 * (-(-f // 128)) * rp
        if case["colwise"]:
            b += rp * f + 4 * (-(-rp // 128)) * f
        return {"bytes": b, "flops": 8 * t * f}
    if op == "glu_bwd":
        t, f = case["tokens"], case["f"]
        rp = -(-t // 16) * 16
        b = 6 * t * f + 2 * rp * 2 * f
        b += 4 * (-(-2 * f // 128)) * rp + 4 * (-(-rp // 128)) * 2 * f
        return {"bytes": b, "flops": 16 * t * f}
    size = 2 if case["grad"] == "bf16" else 4
    elems = sum(n * k for n, k in _shapes(case))
    return {"bytes": elems * (size + 2),
            "flops": _ns_flops(_shapes(case), case["steps"])}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def spiked(*shape, scale=1.0, rate=1e-3, factor=50.0):
        """N(0, scale) with a few entries scaled up, as hidden states have."""
        v = normal(*shape) * scale
        hit = torch.rand(*shape, generator=g, device="cuda") < rate
        return torch.where(hit, v * factor, v).bfloat16()

    op = case["op"]
    if op in ("norm", "norm_bwd"):
        t, c = case["tokens"], case["cols"]
        gamma = 1.0 + 0.2 * normal(c)
        gamma = gamma.bfloat16() if case["gamma"] == "bf16" else gamma
        if op == "norm":
            return {"case": case, "x": spiked(t, c), "gamma": gamma,
                    "residual": spiked(t, c, scale=2.0)
                    if case["residual"] else None}
        h = spiked(t, c, scale=2.0)
        rstd = torch.rsqrt(h.double().square().mean(1) + _EPS).float()
        return {"case": case, "h": h, "rstd": rstd, "gamma": gamma,
                "dy": spiked(t, c, scale=1e-3, factor=100.0),
                "dres": spiked(t, c, scale=1e-3, factor=100.0)
                if case["residual"] else None}
    if op in ("glu", "glu_bwd"):
        t, f = case["tokens"], case["f"]
        gu = spiked(t, 2 * f, factor=20.0)
        if op == "glu":
            return {"case": case, "gu": gu}
        return {"case": case, "gu": gu,
                "da": spiked(t, f, scale=1e-3, factor=100.0)}
    grads = []
    for n, k in _shapes(case):
        # a bulk of noise and a few directions that stand out of it
        edge = math.sqrt(n) + math.sqrt(k)
        u = normal(n, 4) / math.sqrt(n)
        v = normal(4, k) / math.sqrt(k)
        m = 1e-3 * (normal(n, k) + 4.0 * edge * (u @ v))
        grads.append(m.bfloat16() if case["grad"] == "bf16" else m)
    return {"case": case, "grads": grads}


# ---------------------------------------------------------------- plain forms

def _plain_codes(y, dim, pow2):
    """E4M3 codes of fp32 y [rows, cols] in groups of 128 along `dim`, and
    their scales, in the layouts of the row-wise (dim 1: codes [rows, cols],
    scales [groups, rows]) and column-wise (dim 0: codes [cols, rows], scales
    [groups, cols]) quantisers."""
    v = y if dim == 1 else y.t()
    n, length = v.shape
    groups = -(-length // 128)
    v = torch.nn.functional.pad(v, (0, groups * 128 - length))
    v = v.reshape(n, groups, 128)
    amax = v.abs().amax(2)
    if pow2:
        m, e = torch.frexp(amax.double() / 448.0)
        e = torch.where(m > 0.5, e, e - 1).clamp(-127, 120)
        s = torch.ldexp(torch.ones_like(m), e).float()
        q = torch.ldexp(torch.ones_like(m), -e).float()
        bad = (amax == 0) | ~torch.isfinite(amax)
    else:
        s = amax / 448.0
        q = 448.0 / amax
        bad = (amax == 0) | ~torch.isfinite(q)
    s = torch.where(bad, torch.ones_like(s), s)
    q = torch.where(bad, torch.ones_like(q), q)
    codes = (v * q[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    codes = codes.reshape(n, groups * 128)[:, :length].contiguous()
    return codes, s.t().contiguous()


def _pad_rows(y):
    return torch.nn.functional.pad(y, (0, 0, 0, -y.shape[0] % 16))


def _plain_norm(st):
    c = st["case"]
    if st["residual"] is None:
        h = st["x"]
    else:
        h = (st["x"].float() + st["residual"].float()).bfloat16()
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + _EPS)
    y = _pad_rows(hf * rstd[:, None] * st["gamma"].float())
    out = {"rstd": rstd}
    if st["residual"] is not None:
        out["h"] = h
    out["q"], out["s"] = _plain_codes(y, 1, c["pow2"])
    if c["colwise"]:
        out["q_t"], out["s_t"] = _plain_codes(y, 0, c["pow2"])
    return out


def _plain_norm_bwd(st):
    h, dy = st["h"].float(), st["dy"].float()
    xhat = h * st["rstd"][:, None]
    g = dy * st["gamma"].float()
    dh = st["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if st["dres"] is not None:
        dh = dh + st["dres"].float()
    return {"dh": dh.bfloat16(), "dgamma": (dy * xhat).sum(0)}


def _plain_glu(st):
    c = st["case"]
    gate, up = st["gu"].float().chunk(2, 1)
    a = _pad_rows(gate / (1.0 + torch.exp(-gate)) * up)
    out = {}
    out["q"], out["s"] = _plain_codes(a, 1, c["pow2"])
    if c["colwise"]:
        out["q_t"], out["s_t"] = _plain_codes(a, 0, c["pow2"])
    return out


def _plain_glu_bwd(st):
    c = st["case"]
    gate, up = st["gu"].float().chunk(2, 1)
    da = st["da"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dgate = da * up * sig * (1.0 + gate * (1.0 - sig))
    dup = da * gate * sig
    d = _pad_rows(torch.cat([dgate, dup], 1))
    out = {}
    out["q"], out["s"] = _plain_codes(d, 1, c["pow2"])
    out["q_t"], out["s_t"] = _plain_codes(d, 0, c["pow2"])
    return out


def _plain_ns(st):
    a, b, c = _NS
    outs = []
    for grad in st["grads"]:
        tall = grad.shape[0] > grad.shape[1]
        x = grad.float().t() if tall else grad.float()
        x = x / (x.double().square().sum().sqrt().float() + _NS_EPS)
        for _ in range(st["case"]["steps"]):
            m = x @ x.t()
            x = a * x + (b * m + c * (m @ m)) @ x
        outs.append((x.t() if tall else x).bfloat16().contiguous())
    return outs


# ----------------------------------------------------------------- own calls

_ops = None


def _library():
    global _ops
    if _ops is None:
        from blockwise_fp8_linear_fp8bw_b200 import ops
        _ops = ops
    return _ops


def _own(st):
    ops = _library()
    c = st["case"]
    op = c["op"]
    e4m3 = torch.float8_e4m3fn
    if op == "norm":
        r = ops.rmsnorm_quantize(st["x"], st["gamma"], st["residual"], _EPS,
                                 colwise=c["colwise"], pow2=c["pow2"])
        out = {"rstd": r.rstd, "q": r.q.view(e4m3), "s": r.s}
        if st["residual"] is not None:
            out["h"] = r.h
        if c["colwise"]:
            out["q_t"], out["s_t"] = r.q_t.view(e4m3), r.s_t
        return out
    if op == "norm_bwd":
        dh, dgamma = ops.rmsnorm_backward(st["dy"], st["h"], st["rstd"],
                                          st["gamma"], st["dres"])
        return {"dh": dh, "dgamma": dgamma}
    if op == "glu":
        r = ops.swiglu_quantize(st["gu"], colwise=c["colwise"],
                                pow2=c["pow2"])
        out = {"q": r.q.view(e4m3), "s": r.s}
        if c["colwise"]:
            out["q_t"], out["s_t"] = r.q_t.view(e4m3), r.s_t
        return out
    if op == "glu_bwd":
        r = ops.swiglu_backward_quantize(st["da"], st["gu"], pow2=c["pow2"])
        return {"q": r.q.view(e4m3), "s": r.s, "q_t": r.q_t.view(e4m3),
                "s_t": r.s_t}
    return ops.newton_schulz_batch(st["grads"], steps=c["steps"], coeffs=_NS,
                                   eps=_NS_EPS)


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd,
            "glu": _plain_glu, "glu_bwd": _plain_glu_bwd,
            "ns": _plain_ns}[state["case"]["op"]](state)


# -------------------------------------------------------------- exact values

def _to_grid(v, digits, emin):
    """v rounded to `digits` significant binary digits, ties to even, with
    the spacing of exponent `emin` below it (all in 64 bits)."""
    exponent = torch.frexp(v).exponent.sub(1).clamp_min(emin).double()
    step = torch.exp2(exponent - (digits - 1))
    return torch.round(v / step) * step


def _exact_groups(y, along_rows, pow2):
    """Codes' values and scales of 64-bit y, one 128-long group at a time."""
    y = y.transpose(0, 1) if along_rows else y
    codes, scales = [], []
    for part in y.split(128, dim=1):
        top = part.abs().max(dim=1).values
        if pow2:
            s = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
        else:
            s = top / 448.0
        s = torch.where(top > 0, s, torch.ones_like(s))
        codes.append(_to_grid(part / s.unsqueeze(1), 4, -6).clamp(-448, 448))
        scales.append(s)
    return torch.cat(codes, dim=1), torch.stack(scales)


def _exact_out(y, colwise, pow2):
    rows = y.shape[0]
    full = y.new_zeros((rows + 15) // 16 * 16, y.shape[1])
    full[:rows] = y
    out = {}
    out["q"], out["s"] = _exact_groups(full, False, pow2)
    if colwise:
        out["q_t"], out["s_t"] = _exact_groups(full, True, pow2)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = st["x"].double()
        if st["residual"] is not None:
            h = _to_grid(h + st["residual"].double(), 8, -126)
        rstd = 1.0 / torch.sqrt((h * h).sum(dim=1) / h.shape[1] + _EPS)
        y = torch.einsum("tc,t,c->tc", h, rstd, st["gamma"].double())
        out = _exact_out(y, case["colwise"], case["pow2"])
        out["rstd"] = rstd
        if st["residual"] is not None:
            out["h"] = h
        return out
    if op == "norm_bwd":
        h, dy, w = st["h"].double(), st["dy"].double(), st["gamma"].double()
        rstd = st["rstd"].double()
        # y_c = w_c h_c rstd(h); d rstd / d h_c = -rstd^3 h_c / cols
        dot = torch.einsum("tc,tc,c->t", dy, h, w)
        dh = torch.einsum("tc,c,t->tc", dy, w, rstd)
        dh -= h * (rstd ** 3 * dot / h.shape[1]).unsqueeze(1)
        if st["dres"] is not None:
            dh += st["dres"].double()
        return {"dh": dh, "dgamma": torch.einsum("tc,tc,t->c", dy, h, rstd)}
    if op in ("glu", "glu_bwd"):
        f = case["f"]
        gate, up = st["gu"][:, :f].double(), st["gu"][:, f:].double()
        sig = torch.sigmoid(gate)
        if op == "glu":
            return _exact_out(gate * sig * up, case["colwise"], case["pow2"])
        da = st["da"].double()
        slope = sig + gate * sig * torch.sigmoid(-gate)
        d = torch.empty(case["tokens"], 2 * f, dtype=torch.float64,
                        device=da.device)
        d[:, :f] = da * up * slope
        d[:, f:] = da * gate * sig
        return _exact_out(d, True, case["pow2"])
    a, b, c = _NS
    outs = []
    for grad in st["grads"]:
        x = grad.double() / (torch.linalg.norm(grad.double()) + _NS_EPS)
        n, k = x.shape
        for _ in range(case["steps"]):
            # p(X) = X (a + b X^T X + c (X^T X)^2), grouped on the short side
            if n >= k:
                m = x.mT @ x
                x = torch.addmm(x @ (c * (m @ m)), x, b * m).add(x, alpha=a)
            else:
                m = x @ x.mT
                x = torch.addmm((c * (m @ m)) @ x, b * m, x).add(x, alpha=a)
        outs.append(x)
    return outs
