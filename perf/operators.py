"""The workloads of the layer-norm and gated feed-forward operators.

Five operators around the framework's normalised rows: layer norm forward and
backward, the gated feed-forward projection forward and backward in bf16, and
its MXFP8 form on quantised operands.  Each case is a dict of plain values;
``run`` computes it with elementary torch operations in fp32, or, where ``own``
is true, with the framework's operators.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one small batch of rows: latency of a decode or a tiny model's step
        dict(name="ln_fwd_64x1024_bf16", op="ln_fwd", T=64, D=1024, dtype="bf16", pad=0),
        # the hidden shape of the framework's headline workload
        dict(name="ln_fwd_8192x4096_bf16", op="ln_fwd", T=8192, D=4096, dtype="bf16", pad=0),
        # an odd row length in fp32: no row but the first starts on a 16-byte boundary
        dict(name="ln_fwd_3001x5003_fp32", op="ln_fwd", T=3001, D=5003, dtype="fp32", pad=0),
        # the backward at the headline shape
        dict(name="ln_bwd_8192x4096_bf16", op="ln_bwd", T=8192, D=4096, dtype="bf16", pad=0),
        # a ragged batch of short rows, cut out of wider ones, in fp16
        dict(name="ln_bwd_1037x1544_fp16", op="ln_bwd", T=1037, D=1544, dtype="fp16", pad=24),
        # one token: the weights' bytes are all there is
        dict(name="ffn_fwd_1x4096x14336", op="ffn_fwd", T=1, D=4096, F=14336, act="silu", save=False),
        # a training step's forward, which keeps the projections for the backward
        dict(name="ffn_fwd_8192x4096x14336_save", op="ffn_fwd", T=8192, D=4096, F=14336, act="silu", save=True),
        # a ragged chunk of a prompt in a small model
        dict(name="ffn_bwd_333x1032x2744_gelu", op="ffn_bwd", T=333, D=1032, F=2744, act="gelu_tanh"),
        # the training step's backward
        dict(name="ffn_bwd_8192x4096x14336", op="ffn_bwd", T=8192, D=4096, F=14336, act="silu"),
        # a decode batch on quantised operands
        dict(name="mx_ffn_16x4096x14336", op="mx_ffn", T=16, D=4096, F=14336, act="silu", out="bf16"),
        # a prompt chunk whose result goes to the next MXFP8 product
        dict(name="mx_ffn_8192x4096x14336_e4m3", op="mx_ffn", T=8192, D=4096, F=14336, act="silu", out="e4m3"),
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], uniform in its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi // step * step, max(step, -(-lo // step) * step, v // step * step))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ffn_fwd", "ffn_bwd", "mx_ffn"])
    if op in ("ln_fwd", "ln_bwd"):
        return dict(op=op, T=_log(rng, 16, 16384), D=_log(rng, 256, 8192, rng.choice([1, 8, 32])),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), pad=rng.choice([0, 0, 8, 24]))
    T, act = _log(rng, 1, 8192), rng.choice(["silu", "gelu", "gelu_tanh"])
    if op == "mx_ffn":
        return dict(op=op, T=T, D=_log(rng, 512, 4096, 128), F=_log(rng, 512, 14336, 32), act=act,
                    out=rng.choice(["bf16", "e4m3"]))
    D, F = _log(rng, 512, 4096, 8), _log(rng, 512, 14336, 8)
    if op == "ffn_fwd":
        return dict(op=op, T=T, D=D, F=F, act=act, save=rng.random() < 0.5)
    return dict(op=op, T=max(T, 64), D=D, F=F, act=act)


# ----------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * int(seed) + 17)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    x = torch.empty(*shape, dtype=torch.float32, device="cuda").normal_(0.0, scale, generator=g)
    return x.to(dtype)


def _rows(g, T, D, dtype, pad):
    """Activations with 1% of channels 50 times larger and an offset a channel, cut out of wider rows by `pad`."""
    x = torch.empty(T, D + pad, dtype=torch.float32, device="cuda").normal_(generator=g)
    x += 0.5 * torch.empty(D + pad, device="cuda").normal_(generator=g)
    wide = torch.rand(D + pad, device="cuda", generator=g) < 0.01
    x *= torch.where(wide, 50.0, 1.0)
    return x.to(dtype)[:, :D]


def _quantised(g, rows, cols, scale):
    """Random MXFP8 operand: E4M3 codes [rows, cols] and E8M0 scales of 32 in the block-scaled product's 128 x 4 tile layout."""
    v = torch.empty(rows, cols // 32, 32, device="cuda").normal_(0.0, scale, generator=g)
    m, e = torch.frexp(v.abs().amax(-1))
    e = e - 9 + (m > 0.875).to(e.dtype)                      # smallest e with amax <= 448 * 2^e
    codes = torch.ldexp(v, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8).reshape(rows, cols)
    up = -(-rows // 128) * 128
    s = torch.zeros(up, cols // 32, dtype=torch.uint8, device="cuda")
    s[:rows] = (e + 127).to(torch.uint8)
    s = s.view(up // 128, 4, 32, cols // 128, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return codes, s


def prepare(case, seed):
    g, op, T, D = _gen(seed), case["op"], case["T"], case["D"]
    s = dict(case)
    if op in ("ln_fwd", "ln_bwd"):
        dt = DTYPES[case["dtype"]]
        s["x"] = _rows(g, T, D, dt, case["pad"])
        s["gamma"] = (1.0 + 0.1 * torch.empty(D, device="cuda").normal_(generator=g)).to(dt)
        s["beta"] = _randn(g, D, scale=0.1, dtype=dt)
        s["eps"] = 1e-5
        if op == "ln_bwd":
            s["dy"] = _randn(g, T, D, scale=0.01 if dt != torch.float16 else 0.1, dtype=dt)
            v = s["x"].double()
            s["mean"] = v.mean(1).float()
            s["rstd"] = (v.var(1, unbiased=False) + s["eps"]).rsqrt().float()
        return s
    F = case["F"]
    if op == "mx_ffn":
        s["a_q"], s["a_s"] = _quantised(g, T, D, 1.0)
        s["g_q"], s["g_s"] = _quantised(g, F, D, 0.02)
        s["u_q"], s["u_s"] = _quantised(g, F, D, 0.02)
        return s
    s["x"] = _randn(g, T, D)
    s["w_gate"] = _randn(g, F, D, scale=0.02)
    s["w_up"] = _randn(g, F, D, scale=0.02)
    if op == "ffn_bwd":
        s["dh"] = _randn(g, T, F, scale=0.01)
        s["gate"] = (s["x"].float() @ s["w_gate"].float().t()).bfloat16()   # what the forward kept
        s["up"] = (s["x"].float() @ s["w_up"].float().t()).bfloat16()
    return s


# ------------------------------------------------------------ the plain forms

def _act(g, act):
    """act(g) and its derivative, fp32."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        phi = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    s = 1.0 / (1.0 + torch.exp(-2.0 * c * (g + 0.044715 * g * g * g)))      # (1 + tanh z) / 2
    return g * s, s + g * s * (1.0 - s) * 2.0 * c * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + s["eps"])
    y = d * rstd * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_ln_bwd(s):
    dt = s["x"].dtype
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["gamma"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return {"dx": dx.to(dt), "dgamma": (dy * xh).sum(0).to(dt), "dbeta": dy.sum(0).to(dt)}


def _plain_ffn_fwd(s):
    x = s["x"].float()
    gate = x @ s["w_gate"].float().t()
    up = x @ s["w_up"].float().t()
    out = {"h": (_act(gate, s["act"])[0] * up).bfloat16()}
    if s["save"]:
        out["gate"], out["up"] = gate.bfloat16(), up.bfloat16()
    return out


def _plain_ffn_bwd(s):
    x, dh, up = s["x"].float(), s["dh"].float(), s["up"].float()
    a, da = _act(s["gate"].float(), s["act"])
    dg, du = dh * up * da, dh * a
    dx = dg @ s["w_gate"].float() + du @ s["w_up"].float()
    return {"dx": dx.bfloat16(), "dw_gate": (dg.t() @ x).bfloat16(), "dw_up": (du.t() @ x).bfloat16()}


def _values(q, sc, rows, cols):
    """fp32 values of an MXFP8 operand."""
    tiles = sc.view(-1, cols // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, cols // 32)[:rows]
    e = tiles.to(torch.int32) - 127
    v = q.view(torch.float8_e4m3fn).float().view(rows, cols // 32, 32)
    return torch.ldexp(v, e.unsqueeze(-1)).view(rows, cols)


def _plain_mx_ffn(s):
    T, D, F = s["T"], s["D"], s["F"]
    a = _values(s["a_q"], s["a_s"], T, D)
    gate = a @ _values(s["g_q"], s["g_s"], F, D).t()
    up = a @ _values(s["u_q"], s["u_s"], F, D).t()
    h = _act(gate, s["act"])[0] * up
    if s["out"] == "bf16":
        return {"h": h.bfloat16()}
    b = h.view(T, F // 32, 32)
    m, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), -127).clamp(min=-127)
    codes = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(T, F)
    return {"h": codes, "scales": (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)}


def _own(s):
    from normalisation_row_bf16_b200 import ops
    op = s["op"]
    if op == "ln_fwd":
        y, mean, rstd = ops.layernorm_fwd(s["x"], s["gamma"], s["beta"], eps=s["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dx, dgamma, dbeta = ops.layernorm_bwd(s["x"], s["dy"], s["gamma"], s["mean"], s["rstd"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "ffn_fwd":
        h, gate, up = ops.gated_ffn_fwd(s["x"], s["w_gate"], s["w_up"], act=s["act"], save=s["save"])
        return {"h": h, "gate": gate, "up": up} if s["save"] else {"h": h}
    if op == "ffn_bwd":
        dx, dwg, dwu = ops.gated_ffn_bwd(s["dh"], s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], act=s["act"])
        return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}
    h, scales = ops.mxfp8_gated_ffn(s["a_q"], s["a_s"], s["g_q"], s["g_s"], s["u_q"], s["u_s"], s["T"], s["F"],
                                    s["D"], act=s["act"], out=s["out"], scale_layout=ops.SCALES_ROWMAJOR)
    if s["out"] == "bf16":
        return {"h": h}
    return {"h": h.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def run(state):
    if own:
        return _own(state)
    plain = {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "ffn_fwd": _plain_ffn_fwd, "ffn_bwd": _plain_ffn_bwd,
             "mx_ffn": _plain_mx_ffn}
    return plain[state["op"]](state)


# ------------------------------------------------------------------- the work

def work(case):
    T, D, op = case["T"], case["D"], case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        es = 4 if case["dtype"] == "fp32" else 2
        if op == "ln_fwd":
            return {"bytes": es * (2 * T * D + 2 * D) + 8 * T, "flops": 8 * T * D}
        return {"bytes": es * (3 * T * D + 3 * D) + 8 * T, "flops": 14 * T * D}
    F = case["F"]
    if op == "ffn_fwd":
        return {"bytes": 2 * (T * D + 2 * F * D + T * F * (3 if case["save"] else 1)), "flops": 4 * T * D * F}
    if op == "ffn_bwd":
        return {"bytes": 2 * (3 * T * F + 2 * T * D + 4 * F * D), "flops": 8 * T * D * F}
    h = 2 * T * F if case["out"] == "bf16" else T * F + T * F // 32
    return {"bytes": (T + 2 * F) * (D + D // 32) + h, "flops": 4 * T * D * F}


# ------------------------------------------------------ the results in 64 bits

def _exact_act(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if act == "gelu":
        cdf = torch.special.ndtr(g)
        return g * cdf, cdf + g * torch.exp(-g.square() / 2) * (2 * math.pi) ** -0.5
    k = (2 / math.pi) ** 0.5
    t = torch.tanh(k * (g + 0.044715 * g.pow(3)))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 0.134145 * g.square())


def _exact_mx(q, sc, rows, cols):
    """Decoded from the fields of each code, and the scale's byte looked up by its place in the tile layout."""
    c = q.view(rows, cols).to(torch.int64)
    mag, ex = (c & 7).double(), (c >> 3) & 15
    v = torch.where(ex == 0, mag * 2.0 ** -9, (8 + mag) * torch.exp2(ex.double() - 10))
    v = torch.where(c >= 128, -v, v)
    r = torch.arange(rows, device=q.device)[:, None]
    k = torch.arange(cols // 32, device=q.device)[None, :]
    at = ((r // 128) * (cols // 128) + k // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + k % 4
    return v * torch.exp2(sc[at].double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "ln_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + s["eps"]) ** -0.5
        return {"y": (x - mean[:, None]) * rstd[:, None] * s["gamma"].double() + s["beta"].double(), "mean": mean,
                "rstd": rstd}
    if op == "ln_bwd":
        dy, r = s["dy"].double(), s["rstd"].double()
        n = (s["x"].double() - s["mean"].double()[:, None]) * r[:, None]
        a = dy * s["gamma"].double()
        D = case["D"]
        dx = (D * a - a.sum(1)[:, None] - n * (a * n).sum(1)[:, None]) * (r / D)[:, None]
        return {"dx": dx, "dgamma": torch.einsum("td,td->d", dy, n), "dbeta": dy.sum(0)}
    if op == "ffn_fwd":
        x = s["x"].double()
        gate, up = torch.mm(x, s["w_gate"].double().t()), torch.mm(x, s["w_up"].double().t())
        h = _exact_act(gate, s["act"])[0] * up
        return {"h": h, "gate": gate, "up": up} if s["save"] else {"h": h}
    if op == "ffn_bwd":
        a, da = _exact_act(s["gate"].double(), s["act"])
        dh, x = s["dh"].double(), s["x"].double()
        du, dg = dh * a, dh * da * s["up"].double()
        dx = torch.mm(dg, s["w_gate"].double()).addmm_(du, s["w_up"].double())
        return {"dx": dx, "dw_gate": torch.mm(dg.t(), x), "dw_up": torch.mm(du.t(), x)}
    T, D, F = case["T"], case["D"], case["F"]
    a = _exact_mx(s["a_q"], s["a_s"], T, D)
    gate = torch.mm(a, _exact_mx(s["g_q"], s["g_s"], F, D).t())
    up = torch.mm(a, _exact_mx(s["u_q"], s["u_s"], F, D).t())
    h = _exact_act(gate, s["act"])[0] * up
    if case["out"] == "bf16":
        return {"h": h}
    del gate, up
    b = h.view(T, F // 32, 32)
    amax = b.abs().amax(-1)
    e = torch.ceil(torch.log2(amax / 448)).clamp(-127, 127)
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, torch.where(amax <= 224 * torch.exp2(e), e - 1, e)).clamp(-127, 127)
    v = b * torch.exp2(-e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)   # spacing of E4M3 there
    return {"h": (torch.round(v / step) * step).view(T, F), "scales": torch.exp2(e)}
