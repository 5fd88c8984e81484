"""The block operators' measured cases: layer norm, the linear layer with its
epilogues and gradients, and 8-bit activation checkpoints.

Where ``own`` is false, ``run`` computes an operator in its plain form:
elementary torch operations in 32 bits, rounded once at the end.  Where it is
true, ``run`` makes the calls a training step makes of the library.
``exact`` gives the same outputs from the definitions in 64 bits.

Sizes are those of the workloads' transformer blocks (d 768, 1280 and 12288
with ffn 5120 and 49152, 1024 to 2048 tokens a sequence) and of the ragged
unit (odd row and column counts); weights are stored [in, out] as in the GPT
blocks, or [out, in].
"""
import math

import torch

own = False

GROUP = 32            # elements that share one exponent in an 8-bit checkpoint
EPS = 1e-5


def listed():
    return [
        # the latency of one token through a GPT-2 Large block's norm
        dict(name="ln_fwd_token", op="ln_fwd", rows=1, cols=1280, dtype="bf16", params="bf16", ckpt=False, pad=0),
        # minGPT-175B block, two sequences of 2048, with the norm's input kept in 8 bits for the backward pass
        dict(name="ln_fwd_175b_ckpt", op="ln_fwd", rows=4096, cols=12288, dtype="bf16", params="bf16", ckpt=True, pad=0),
        # GPT-2 Large block, micro-batch 4 x 1024, with the residual branch's gradient added, fp32 gradients
        dict(name="ln_bwd_gpt2_large", op="ln_bwd", rows=4096, cols=1280, dtype="bf16", params="bf16", grads="f32", ckpt=False, add=True, pad=0),
        # minGPT-175B block: the backward pass from the 8-bit checkpoint, bf16 gradients
        dict(name="ln_bwd_175b_ckpt", op="ln_bwd", rows=4096, cols=12288, dtype="bf16", params="bf16", grads="bf16", ckpt=True, add=True, pad=0),
        # one token through a GPT-2 Large block's first MLP product (evaluation with the gathered weights)
        dict(name="lin_fwd_token", op="lin_fwd", tokens=1, inf=1280, outf=5120, layout="in_out", act="gelu_tanh", bias=True, residual=False, ckpt=False, out="bf16", pad=0),
        # the ragged unit's odd matrix, [out, in], residual added, fp32 result; no row is 16-byte aligned
        dict(name="lin_fwd_ragged", op="lin_fwd", tokens=1031, inf=1283, outf=5121, layout="out_in", act="none", bias=True, residual=True, ckpt=False, out="f32", pad=0),
        # GPT-2 Large block, micro-batch 4 x 1024: first MLP product, pre-activation kept in 8 bits
        dict(name="lin_fwd_gpt2_large", op="lin_fwd", tokens=4096, inf=1280, outf=5120, layout="in_out", act="gelu_tanh", bias=True, residual=False, ckpt=True, out="bf16", pad=0),
        # minGPT-175B block, two sequences of 2048: second MLP product onto the residual stream
        dict(name="lin_fwd_175b", op="lin_fwd", tokens=4096, inf=49152, outf=12288, layout="in_out", act="none", bias=True, residual=True, ckpt=False, out="bf16", pad=0),
        # GPT-2 Large block: gradients of the second MLP product, through the GELU by the 8-bit checkpoint, fp32 gradients
        dict(name="lin_bwd_gpt2_large", op="lin_bwd", tokens=4096, inf=5120, outf=1280, layout="in_out", act="gelu_tanh", x8=False, z8=True, add=False, grads="f32", pad=0),
        # minGPT-175B block, one sequence of 2048: gradients of the first MLP product, its input from an 8-bit checkpoint, bf16 gradients
        dict(name="lin_bwd_175b", op="lin_bwd", tokens=2048, inf=12288, outf=49152, layout="in_out", act="none", x8=True, z8=False, add=False, grads="bf16", pad=0),
        # a few tokens of an odd width into a checkpoint and back: latency and a ragged last group
        dict(name="act8_ragged", op="act8", rows=37, cols=1283, dtype="f32", act="none", pad=1),
        # a GPT-2 Large block's pre-activation, micro-batch 8 x 1024, into 8 bits and back through the GELU (recomputing the second product's input)
        dict(name="act8_gpt2_large", op="act8", rows=8192, cols=5120, dtype="bf16", act="gelu_tanh", pad=0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width over the range: a multiple of 64, of 8, or any number."""
    n = _spread(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    n = max(step, n - n % step)
    return n if n != 3072 else n + step


def draw(rng):
    op = rng.choice(("ln_fwd", "ln_bwd", "lin_fwd", "lin_bwd", "act8"))
    pad = rng.choice((0, 0, 8, 3))      # elements between a row's end and the next row, for inputs cut from wider tensors
    if op in ("ln_fwd", "ln_bwd", "act8"):
        c = dict(op=op, rows=_spread(rng, 1, 8192), cols=_width(rng, 64, 12288), dtype=rng.choice(("bf16", "bf16", "f32")), pad=pad)
        c["rows"] = min(c["rows"], 4096 * 12288 // c["cols"])
        if op == "act8":
            c.update(act=rng.choice(("none", "gelu_tanh", "gelu_erf", "relu")))
            return c
        c.update(params=rng.choice(("bf16", "f32")), ckpt=rng.random() < 0.5)
        if op == "ln_bwd":
            c.update(grads=rng.choice(("bf16", "f32")), add=rng.random() < 0.5)
        return c
    c = dict(op=op, tokens=_spread(rng, 1, 8192), inf=_width(rng, 64, 16384), outf=_width(rng, 64, 16384),
             layout=rng.choice(("in_out", "out_in")), act=rng.choice(("none", "gelu_tanh", "gelu_erf", "relu")), pad=pad)
    c["tokens"] = max(1, min(c["tokens"], 2048 * 12288 * 49152 // (c["inf"] * c["outf"])))
    if op == "lin_fwd":
        c.update(bias=rng.random() < 0.8, residual=rng.random() < 0.5, ckpt=rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "f32")))
    else:
        c.update(x8=rng.random() < 0.5, z8=rng.random() < 0.5, add=rng.random() < 0.5, grads=rng.choice(("bf16", "f32")))
    return c


# ---- inputs -----------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


class _Maker:
    """Seeded inputs on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, shape, std, dtype, mean=0.0):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=self.g).to(dtype)

    def matrix(self, rows, cols, std, dtype, pad=0):
        return self.normal((rows, cols + pad), std, dtype)[:, :cols]

    def activations(self, rows, cols, dtype, pad=0, std=1.0):
        """Activations as a transformer block has them: a few channels far larger than the rest, each with an offset."""
        scale = torch.ones(cols + pad, device="cuda")
        big = torch.rand(cols + pad, device="cuda", generator=self.g) < 0.01
        scale[big] = 8.0
        x = torch.empty((rows, cols + pad), device="cuda").normal_(0.0, std, generator=self.g)
        x.mul_(scale).add_(torch.empty(cols + pad, device="cuda").normal_(0.0, 0.2 * std, generator=self.g) * scale)
        return x.to(dtype)[:, :cols]


def _packed(x):
    """An 8-bit checkpoint of x as it lies in memory: int8 values in rows of a
    multiple of 32 bytes, and one exponent byte to each group of 32."""
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    full = torch.zeros((rows, groups * GROUP), device=x.device)
    full[:, :cols] = x
    full = full.view(rows, groups, GROUP)
    top = full.abs().amax(dim=2)
    e = (torch.frexp(top)[1] - 1).clamp(-120, 127)
    e = torch.where(top == 0, torch.full_like(e, -120), e)
    q = torch.ldexp(full, (6 - e).unsqueeze(2)).round_().clamp_(-127, 127).to(torch.int8)
    return q.view(rows, groups * GROUP), (e + 127).to(torch.uint8)


def prepare(case, seed):
    c, m, op = case, _Maker(seed), case["op"]
    s = {"case": c}
    if op in ("ln_fwd", "ln_bwd"):
        dt, pt = _TYPES[c["dtype"]], _TYPES[c["params"]]
        rows, cols = c["rows"], c["cols"]
        x = m.activations(rows, cols, dt, c["pad"])
        s["gamma"] = m.normal((cols,), 0.1, pt, 1.0)
        if op == "ln_fwd":
            s["x"], s["beta"] = x, m.normal((cols,), 0.1, pt)
        else:
            xf = x.float()
            s["mean"] = xf.mean(dim=1)
            s["rstd"] = torch.rsqrt(xf.var(dim=1, unbiased=False) + EPS)
            s["dy"] = m.matrix(rows, cols, 1e-2, dt, c["pad"])
            s["add"] = m.matrix(rows, cols, 1e-2, dt) if c["add"] else None
            if c["ckpt"]:
                s["q"], s["e"] = _packed(xf)
            else:
                s["x"] = x
    elif op == "act8":
        s["x"] = m.activations(c["rows"], c["cols"], _TYPES[c["dtype"]], c["pad"])
    else:
        T, I, O = c["tokens"], c["inf"], c["outf"]
        w = m.matrix(I, O, 0.9 / math.sqrt(I), torch.bfloat16) if c["layout"] == "in_out" else m.matrix(O, I, 0.9 / math.sqrt(I), torch.bfloat16)
        s["w"] = w
        x = m.activations(T, I, torch.bfloat16, c["pad"])
        if op == "lin_fwd":
            s["x"] = x
            s["bias"] = m.normal((O,), 0.1, torch.bfloat16) if c["bias"] else None
            s["residual"] = m.matrix(T, O, 1.0, torch.bfloat16) if c["residual"] else None
        else:
            s["dy"] = m.matrix(T, O, 1e-2, torch.bfloat16, c["pad"])
            s["add"] = m.matrix(T, I, 1e-2, torch.bfloat16) if c["add"] else None
            if c["x8"]:
                s["q"], s["e"] = _packed(x.float())
            else:
                s["x"] = x
            if c["act"] != "none":
                z = m.activations(T, I, torch.bfloat16, 0)
                if c["z8"]:
                    s["zq"], s["ze"] = _packed(z.float())
                else:
                    s["z"] = z
    if own:
        _with_handles(s)
    return s


def _with_handles(s):
    """What a training program keeps between calls: the compute handle with its
    workspace, output buffers, and views of the checkpoints."""
    from fully_sharded_unit_gb300 import binding as B

    c, op = s["case"], s["case"]["op"]

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op in ("ln_fwd", "ln_bwd"):
        rows, cols, dt = c["rows"], c["cols"], _TYPES[c["dtype"]]
        s["c"] = B.Compute(B.fsdp_layer_norm_workspace_bytes(rows, cols))
        if op == "ln_fwd":
            s["y"], s["mean"], s["rstd"] = empty((rows, cols), dt), empty(rows, torch.float32), empty(rows, torch.float32)
            if c["ckpt"]:
                s["k"], s["kv"] = B.Act8(rows, cols), empty((rows, cols), torch.bfloat16)
        else:
            s["dx"] = empty((rows, cols), dt)
            s["dgamma"], s["dbeta"] = empty(cols, _TYPES[c["grads"]]), empty(cols, _TYPES[c["grads"]])
            s["input"] = B.Act8(rows, cols, q=s["q"], exps=s["e"]) if c["ckpt"] else s["x"]
    elif op == "act8":
        s["c"] = B.Compute(0)
        s["k"], s["kv"] = B.Act8(c["rows"], c["cols"]), empty((c["rows"], c["cols"]), torch.bfloat16)
    else:
        T, I, O = c["tokens"], c["inf"], c["outf"]
        s["c"] = B.Compute(B.fsdp_linear_workspace_bytes(T, I, O))
        if op == "lin_fwd":
            s["y"] = empty((T, O), _TYPES[c["out"]])
            s["k"] = B.Act8(T, O) if c["ckpt"] else None
            s["kv"] = empty((T, O), torch.bfloat16) if c["ckpt"] else None
        else:
            s["dx"], s["dw"], s["db"] = empty((T, I), torch.bfloat16), empty(tuple(s["w"].shape), _TYPES[c["grads"]]), empty(O, _TYPES[c["grads"]])
            s["input"] = B.Act8(T, I, q=s["q"], exps=s["e"]) if c["x8"] else s["x"]
            s["preact"] = None
            if c["act"] != "none":
                s["preact"] = B.Act8(T, I, q=s["zq"], exps=s["ze"]) if c["z8"] else s["z"]


# ---- the plain forms ----------------------------------------------------------

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


def _read8(q, e, cols):
    """The values an 8-bit checkpoint stands for, in 32 bits."""
    rows, groups = e.shape
    v = torch.ldexp(q.view(rows, groups, GROUP).float(), (e.to(torch.int32) - 133).unsqueeze(2))
    return v.view(rows, groups * GROUP)[:, :cols]


def _through8(x):
    q, e = _packed(x)
    return _read8(q, e, x.shape[1])


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "ln_fwd":
        dt = _TYPES[c["dtype"]]
        x = s["x"].float()
        mean = x.sum(dim=1, keepdim=True) / c["cols"]
        d = x - mean
        rstd = 1.0 / torch.sqrt((d * d).sum(dim=1, keepdim=True) / c["cols"] + EPS)
        r = {"y": (d * rstd * s["gamma"].float() + s["beta"].float()).to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
        if c["ckpt"]:
            r["kept"] = _through8(x).to(torch.bfloat16)
        return r
    if op == "ln_bwd":
        dt, gt = _TYPES[c["dtype"]], _TYPES[c["grads"]]
        x = _read8(s["q"], s["e"], c["cols"]) if c["ckpt"] else s["x"].float()
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = (x - s["mean"][:, None]) * rstd
        g = dy * s["gamma"].float()
        dx = rstd * (g - g.sum(dim=1, keepdim=True) / c["cols"] - xh * ((g * xh).sum(dim=1, keepdim=True) / c["cols"]))
        if c["add"]:
            dx = dx + s["add"].float()
        return {"dx": dx.to(dt), "dgamma": (dy * xh).sum(dim=0).to(gt), "dbeta": dy.sum(dim=0).to(gt)}
    if op == "act8":
        return {"kept": _act(_through8(s["x"].float()), c["act"]).to(torch.bfloat16)}
    w = s["w"].float()
    w = w if c["layout"] == "in_out" else w.t()
    if op == "lin_fwd":
        z = s["x"].float() @ w
        if c["bias"]:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if c["residual"]:
            y = y + s["residual"].float()
        r = {"y": y.to(_TYPES[c["out"]])}
        if c["ckpt"]:
            r["kept"] = _through8(z).to(torch.bfloat16)
        return r
    gt = _TYPES[c["grads"]]
    dy = s["dy"].float()
    dx = dy @ w.t()
    if c["act"] != "none":
        dx = dx * _act_slope(_read8(s["zq"], s["ze"], c["inf"]) if c["z8"] else s["z"].float(), c["act"])
    if c["add"]:
        dx = dx + s["add"].float()
    x = _read8(s["q"], s["e"], c["inf"]) if c["x8"] else s["x"].float()
    dw = x.t() @ dy if c["layout"] == "in_out" else dy.t() @ x
    return {"dx": dx.to(torch.bfloat16), "dw": dw.to(gt), "db": dy.sum(dim=0).to(gt)}


def _own(s):
    c, op, h = s["case"], s["case"]["op"], s["c"]
    if op == "ln_fwd":
        r = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
        h.layer_norm_forward(s["x"], s["gamma"], s["beta"], EPS, s["y"], s["mean"], s["rstd"], ckpt=s.get("k"))
        if c["ckpt"]:
            h.act8_unpack(s["k"], s["kv"])
            r["kept"] = s["kv"]
        return r
    if op == "ln_bwd":
        h.layer_norm_backward(s["dy"], s["input"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"], add=s["add"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "act8":
        h.act8_pack(s["x"], s["k"])
        h.act8_unpack(s["k"], s["kv"], activation=c["act"])
        return {"kept": s["kv"]}
    if op == "lin_fwd":
        r = {"y": s["y"]}
        h.linear_forward(s["x"], s["w"], s["y"], bias=s["bias"], activation=c["act"], residual=s["residual"], preact=s["k"], weight_layout=c["layout"])
        if c["ckpt"]:
            h.act8_unpack(s["k"], s["kv"])
            r["kept"] = s["kv"]
        return r
    h.linear_grad_input(s["dy"], s["w"], s["dx"], activation=c["act"], preact=s["preact"], add=s["add"], weight_layout=c["layout"])
    h.linear_grad_weight(s["input"], s["dy"], s["dw"], dbias=s["db"], weight_layout=c["layout"])
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without --------------------------------------------

_SIZE = {"bf16": 2, "f32": 4}


def work(case):
    c, op = case, case["op"]
    if op in ("ln_fwd", "ln_bwd", "act8"):
        n, b = c["rows"] * c["cols"], _SIZE[c["dtype"]]
        kept = c["rows"] * -(-c["cols"] // GROUP) * (GROUP + 1)      # a checkpoint: 32 bytes and an exponent to a group
        if op == "act8":
            return {"bytes": n * b + kept + 2 * n, "flops": 8 * n}
        p = _SIZE[c["params"]]
        if op == "ln_fwd":
            return {"bytes": 2 * n * b + 2 * c["cols"] * p + 8 * c["rows"] + ((kept + 2 * n) if c["ckpt"] else 0), "flops": 8 * n}
        return {"bytes": n * b * (2 + c["add"]) + (kept if c["ckpt"] else n * b) + c["cols"] * (p + 2 * _SIZE[c["grads"]]) + 8 * c["rows"], "flops": 14 * n}
    T, I, O = c["tokens"], c["inf"], c["outf"]
    if op == "lin_fwd":
        kept = T * -(-O // GROUP) * (GROUP + 1) + 2 * T * O if c["ckpt"] else 0
        return {"bytes": 2 * (T * I + I * O) + T * O * (_SIZE[c["out"]] + 2 * c["residual"]) + 2 * O * c["bias"] + kept, "flops": 2 * T * I * O}
    kept = T * -(-I // GROUP) * (GROUP + 1)
    z = 0 if c["act"] == "none" else kept if c["z8"] else 2 * T * I
    return {"bytes": 2 * (T * O + I * O + T * I * (1 + c["add"])) + (kept if c["x8"] else 2 * T * I) + z + (I * O + O) * _SIZE[c["grads"]], "flops": 4 * T * I * O}


# ---- 64 bits ------------------------------------------------------------------

def _exact_read(q, e, cols):
    scale = torch.exp2(e.double() - 133.0).repeat_interleave(GROUP, dim=1)
    return (q.double() * scale)[:, :cols]


def _exact_keep(x):
    rows, cols = x.shape
    more = -cols % GROUP
    x = torch.cat([x, x.new_zeros(rows, more)], dim=1).unflatten(1, (-1, GROUP))
    top = x.abs().max(dim=2, keepdim=True).values
    step = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -120))) - 6.0)
    return (torch.clamp(torch.round(x / step), -127, 127) * step).flatten(1)[:, :cols]


def _exact_gelu(z, act):
    """(activation, derivative) in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
    if act == "gelu_erf":
        p = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(8.0 / math.pi)        # tanh(u) = 2 sigmoid(2u) - 1
    p = torch.sigmoid(k * (z + 0.044715 * z ** 3))
    return z * p, p + z * p * (1 - p) * k * (1 + 0.134145 * z * z)


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "ln_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        r = {"y": torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], s["gamma"].double()), "mean": mean, "rstd": rstd}
        if c["ckpt"]:
            r["kept"] = _exact_keep(x)
        return r
    if op == "ln_bwd":
        x = _exact_read(s["q"], s["e"], c["cols"]) if c["ckpt"] else s["x"].double()
        dy, r = s["dy"].double(), s["rstd"].double()[:, None]
        n = (x - s["mean"].double()[:, None]) * r
        h = dy * s["gamma"].double()
        dx = (h - h.mean(dim=1, keepdim=True) - n * (h * n).mean(dim=1, keepdim=True)) * r
        if c["add"]:
            dx += s["add"].double()
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, n), "dbeta": dy.sum(0)}
    if op == "act8":
        return {"kept": _exact_gelu(_exact_keep(s["x"].double()), c["act"])[0]}
    spec = "io" if c["layout"] == "in_out" else "oi"
    w = s["w"].double()
    if op == "lin_fwd":
        z = torch.einsum("ti,%s->to" % spec, s["x"].double(), w)
        del w
        if c["bias"]:
            z += s["bias"].double()
        y = _exact_gelu(z, c["act"])[0]
        if c["residual"]:
            y = y + s["residual"].double()
        return {"y": y, "kept": _exact_keep(z)} if c["ckpt"] else {"y": y}
    dy = s["dy"].double()
    dx = torch.einsum("to,%s->ti" % spec, dy, w)
    del w
    if c["act"] != "none":
        dx *= _exact_gelu(_exact_read(s["zq"], s["ze"], c["inf"]) if c["z8"] else s["z"].double(), c["act"])[1]
    if c["add"]:
        dx += s["add"].double()
    x = _exact_read(s["q"], s["e"], c["inf"]) if c["x8"] else s["x"].double()
    return {"dx": dx, "dw": torch.einsum("ti,to->%s" % spec, x, dy), "db": dy.sum(0)}
