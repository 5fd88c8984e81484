"""The measured cases of the operators around a training step's ends: log
probabilities of given tokens (forward, backward, and both in one pass), the
residual norm (norms before and after a block, with its gate and residual
scale), and AdamW over many tensors with moments in 32 or 8 bits.

Where ``own`` is false, ``run`` computes an operator in its plain form:
elementary torch operations in 32 bits, rounded once at the end.  Where it is
true, ``run`` makes the calls a training program makes of the library.
``exact`` gives the same outputs from the definitions in 64 bits.

Sizes are those of the workloads' transformer blocks (d 128, 1280 and 12288,
1024 to 2048 tokens a sequence), of their vocabulary of 50257 tokens, and of
the ragged unit (odd widths, a tensor of one element).
"""
import math

import torch

own = False

EPS = 1e-6
GROUP = 32            # elements that share one exponent in 8-bit moments
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
VOCAB = 50257


def listed():
    return [
        # eight sequences' next tokens: every row read for its 20 most likely tokens
        dict(name="logprob_tokens", op="lp_fwd", rows=8, vocab=VOCAB, dtype="bf16", pad=0, top=20, scale=1.25),
        # evaluation of 8 x 1024 tokens: log probability, entropy and five alternatives; rows of an odd width start anywhere
        dict(name="logprob_eval", op="lp_fwd", rows=8192, vocab=VOCAB, dtype="bf16", pad=0, top=5, scale=1.0),
        # gradient of a policy loss with an entropy bonus, 2 x 1024 tokens, F32 logits in rows padded to 50304
        dict(name="logprob_grad", op="lp_bwd", rows=2048, vocab=VOCAB, dtype="f32", pad=47, entropy=True, scale=1.0),
        # the training loss of a micro-batch of 8 x 1024 tokens: log probabilities and the logits' gradient in one call
        dict(name="logprob_loss", op="lp_loss", rows=8192, vocab=VOCAB, dtype="bf16", pad=0, entropy=False, scale=1.0),
        # the latency of one token at a GPT-2 Large block's end
        dict(name="resnorm_token", op="rn_fwd", rows=1, cols=1280, dtype="bf16", params="bf16", post=True, gate=True, pad=0),
        # minGPT-175B width, two sequences of 2048: norm of the block's result, gate, residual, the next block's norm
        dict(name="resnorm_175b", op="rn_fwd", rows=4096, cols=12288, dtype="bf16", params="bf16", post=True, gate=True, pad=0),
        # its gradients at GPT-2 Large width, micro-batch 4 x 1024
        dict(name="resnorm_grad_gpt2_large", op="rn_bwd", rows=4096, cols=1280, dtype="bf16", params="bf16", grads="f32", post=True, gate=True, pad=0),
        # its gradients at minGPT-175B width
        dict(name="resnorm_grad_175b", op="rn_bwd", rows=4096, cols=12288, dtype="bf16", params="bf16", grads="bf16", post=True, gate=False, pad=0),
        # its gradients at the ragged unit's odd width: no row is 16-byte aligned
        dict(name="resnorm_grad_ragged", op="rn_bwd", rows=1031, cols=5121, dtype="bf16", params="f32", grads="f32", post=False, gate=True, pad=0),
        # the reduced ragged unit's tensors (odd sizes, one of one element): latency
        dict(name="adamw_ragged", op="adamw", model="ragged", blocks=1, state="8bit", grads="f32", copy=False, tight=True),
        # twelve GPT-2 Large blocks, moments in 32 bits
        dict(name="adamw_gpt2_large_32bit", op="adamw", model="d1280", blocks=12, state="f32", grads="f32", copy=True, tight=False),
        # all 36 GPT-2 Large blocks (708 million parameters), moments in 8 bits, bf16 gradients, bf16 copies written for the next gather
        dict(name="adamw_gpt2_large_8bit", op="adamw", model="d1280", blocks=36, state="8bit", grads="bf16", copy=True, tight=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width over the range: a multiple of 64, of 8, or any number."""
    n = _spread(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    return max(step, n - n % step)


def draw(rng):
    op = rng.choice(("lp_fwd", "lp_bwd", "lp_loss", "rn_fwd", "rn_bwd", "adamw"))
    if op.startswith("lp"):
        c = dict(op=op, rows=_spread(rng, 1, 8192), vocab=_width(rng, 64, 131072), dtype=rng.choice(("bf16", "bf16", "f32")),
                 pad=rng.choice((0, 0, 7, 8)), scale=rng.choice((1.0, 1.0, 0.7, 1.5)))
        c["rows"] = max(1, min(c["rows"], 4096 * VOCAB // c["vocab"]))
        c.update(top=rng.choice((0, 1, 5, 20, 32))) if op == "lp_fwd" else c.update(entropy=rng.random() < 0.5)
        return c
    if op.startswith("rn"):
        c = dict(op=op, rows=_spread(rng, 1, 8192), cols=_width(rng, 64, 12288), dtype=rng.choice(("bf16", "bf16", "f32")),
                 params=rng.choice(("bf16", "f32")), post=rng.random() < 0.7, gate=rng.random() < 0.5, pad=rng.choice((0, 0, 8, 3)))
        c["rows"] = min(c["rows"], 2048 * 12288 // c["cols"])
        if op == "rn_bwd":
            c.update(grads=rng.choice(("bf16", "f32")))
        return c
    return dict(op=op, model=rng.choice(("ragged", "d128", "d1280")), blocks=rng.randint(1, 12), state=rng.choice(("f32", "8bit", "8bit")),
                grads=rng.choice(("bf16", "f32")), copy=rng.random() < 0.5, tight=rng.random() < 0.5)


# ---- inputs -----------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


class _Maker:
    """Seeded inputs on the GPU."""

    def __init__(self, seed):
        self.seed = seed
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, shape, std, dtype, mean=0.0):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=self.g).to(dtype)

    def uniform(self, shape):
        return torch.rand(shape, device="cuda", generator=self.g)

    def matrix(self, rows, cols, std, dtype, pad=0):
        return self.normal((rows, cols + pad), std, dtype)[:, :cols]

    def activations(self, rows, cols, dtype, pad=0):
        """Activations as a transformer block has them: a few channels far larger than the rest."""
        scale = torch.ones(cols + pad, device="cuda")
        scale[self.uniform(cols + pad) < 0.01] = 8.0
        return self.normal((rows, cols + pad), 1.0, torch.float32).mul_(scale).to(dtype)[:, :cols]


def _shapes(model, blocks):
    """The tensors of a model's blocks, in registration order: (elements, weight decay or not)."""
    if model == "ragged":
        unit = [(1031, 40), (40,), (40,), (40, 129), (7, 13), (1,)]
    else:
        d = int(model[1:])
        f = 4 * d
        unit = [(d,), (d,), (d, 3 * d), (3 * d,), (d, d), (d,), (d,), (d,), (d, f), (f,), (f, d), (d,)]
    return [(math.prod(s), len(s) > 1) for _ in range(blocks) for s in unit]


def _logits(m, c):
    """Logits as a model gives them: one likely token in most rows, ties (bf16), one token in 64 masked with -inf."""
    rows, v = c["rows"], c["vocab"]
    z = torch.empty((rows, v + c["pad"]), device="cuda").normal_(0.0, 2.0, generator=m.g)
    tokens = (m.uniform(rows) * v).long().clamp_(max=v - 1)
    z[torch.arange(rows, device="cuda"), tokens] += 12.0 * m.uniform(rows)
    z[:, :v:64] = -math.inf
    return z.to(_TYPES[c["dtype"]])[:, :v], tokens


def prepare(case, seed):
    c, m, op = case, _Maker(seed), case["op"]
    s = {"case": c}
    if op.startswith("lp"):
        rows = c["rows"]
        s["z"], tokens = _logits(m, c)
        tokens[tokens % 64 == 0] += 1 if c["vocab"] > 1 else 0          # not a masked one
        s["tokens"] = tokens.clamp_(max=c["vocab"] - 1)
        s["tokens"][m.uniform(rows) < 0.06] = -1                       # padding
        if op != "lp_fwd":
            s["a"] = m.normal((rows,), 0.2, torch.float32, -1.0) / rows
            s["a"][s["tokens"] < 0] = 0.0
            s["b"] = m.normal((rows,), 1e-3, torch.float32, -1e-2) / rows if c["entropy"] else None
            if c["entropy"]:
                s["b"][s["tokens"] < 0] = 0.0
        if op == "lp_bwd":          # what the forward kept
            top = s["z"].amax(dim=1).double()
            ln = torch.empty(rows, dtype=torch.float64, device="cuda")
            h = torch.empty(rows, dtype=torch.float64, device="cuda")
            for at in range(0, rows, 1024):
                d = (s["z"][at:at + 1024].double() - top[at:at + 1024, None]) * c["scale"]
                e = torch.exp(d)
                total = e.sum(dim=1)
                ln[at:at + 1024] = torch.log(total)
                h[at:at + 1024] = ln[at:at + 1024] - (e * d.clamp(min=-1e30)).sum(dim=1) / total
            s["stats"] = torch.stack((top, ln), dim=1).float()
            s["h"] = h.float() if c["entropy"] else None
    elif op.startswith("rn"):
        dt, pt, rows, cols = _TYPES[c["dtype"]], _TYPES[c["params"]], c["rows"], c["cols"]
        s["residual"] = m.activations(rows, cols, dt, c["pad"])
        s["block"] = m.matrix(rows, cols, 0.5, dt, c["pad"])
        s["post"] = m.normal((cols,), 0.1, pt, 1.0) if c["post"] else None
        s["gate"] = m.normal((cols,), 0.1, pt, 0.5) if c["gate"] else None
        s["gamma"] = m.normal((cols,), 0.1, pt, 1.0)
        s["alpha"] = 0.875
        if op == "rn_bwd":          # what the forward kept
            out, rstd, post_rstd = _resnorm(s)
            s["out"], s["rstd"] = torch.empty((rows, cols + c["pad"]), dtype=dt, device="cuda")[:, :cols].copy_(out), rstd
            s["post_rstd"] = post_rstd
            s["dy"] = m.matrix(rows, cols, 1e-2, dt, c["pad"])
            s["dout"] = m.matrix(rows, cols, 1e-2, dt, c["pad"])
    else:
        _optimizer(s, m)
    if own:
        _with_handles(s)
    return s


def _optimizer(s, m):
    """Flat buffers as a training program has them.  Parameters and gradients lie
    one behind the other (``tight``: as the unsharded unit has them, so that tensors
    begin anywhere) or on multiples of 32 elements; moments are on multiples of 32."""
    c = s["case"]
    sizes = _shapes(c["model"], c["blocks"])
    n = torch.tensor([k for k, _ in sizes])
    room = (n + GROUP - 1) // GROUP * GROUP
    begin = torch.cumsum(room, 0) - room
    flat = torch.cumsum(n, 0) - n if c["tight"] else begin
    s["sizes"], s["flat"], s["begin"] = n.tolist(), flat.tolist(), begin.tolist()
    s["decay"] = [1.0 if d else 0.0 for _, d in sizes]
    length, padded = int(flat[-1] + n[-1]), int(room.sum())
    s["param"] = m.normal((length,), 0.02, torch.float32)
    s["grad"] = (m.normal((length,), 1e-3, torch.float32) * torch.where(m.uniform(length) < 1e-3, 100.0, 1.0)).to(_TYPES[c["grads"]])
    s["copy"] = torch.zeros(length, dtype=torch.bfloat16, device="cuda") if c["copy"] else None
    s["step"], s["seed"] = 1000, m.seed + 7
    # what the plain form needs to treat all tensors at once
    n, begin, flat = n.cuda(), begin.cuda(), flat.cuda()
    number = torch.arange(len(sizes), device="cuda")
    of = torch.repeat_interleave(number, n)
    place = torch.arange(int(n.sum()), device="cuda") - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
    s["index"] = {"of": of.to(torch.int32), "place": place, "flat": flat[of] + place, "at": begin[of] + place, "padded": padded}
    at = s["index"]["at"]
    m1 = torch.zeros(padded, device="cuda")
    m1[at] = m.normal((at.numel(),), 3e-4, torch.float32)
    m2 = torch.zeros(padded, device="cuda")
    m2[at] = m.normal((at.numel(),), 1e-3, torch.float32).square_() * 0.6
    if c["state"] == "f32":
        s["m"], s["v"] = m1, m2
    else:
        s["m"], s["v"] = _keep8(m1, True, 0.5), _keep8(m2, False, 0.5)


# 8-bit moments: (codes, exponent bytes).  An element of a group with exponent
# byte B stands for f * 2^(B - 127), f the small float that its code spells: 3 bits
# below the leading one and 4 (signed) or 5 (unsigned) bits of exponent, the
# largest exponent for [1, 2).

def _keep8(x, signed, chance):
    """x (a multiple of 32 long) in 8 bits: up or down to a neighbour, up where what is cut off plus ``chance`` reaches a step."""
    g = x.view(-1, GROUP)
    top = g.abs().amax(dim=1)
    b = ((top.view(torch.int32) + 0xFFFFF) >> 23).clamp(1, 253)
    y = torch.ldexp(g.abs().double(), (127 - b).double()[:, None]).view(-1)
    low = -14 if signed else -30
    e = torch.where(y > 0, torch.frexp(y)[1] - 1, low).clamp(min=low)
    code = torch.floor(torch.ldexp(y, (3 - e).double()) + chance).long()
    code = (code + ((e - low) << 3)).clamp(max=127 if signed else 255)
    code = torch.where((x < 0) & (code > 0), code + 128, code) if signed else torch.where(x > 0, code.clamp(min=1), code)
    return code.to(torch.uint8), b.to(torch.uint8)


def _read8(q, b, signed):
    """The values that 8-bit moments stand for, in 32 bits."""
    k = q.to(torch.int32)
    low = (k & 127) if signed else k
    e, f = low >> 3, low & 7
    v = torch.ldexp(torch.where(e > 0, f + 8, f).float(), (e.clamp(min=1) - (18 if signed else 34)).float())
    v = torch.where(k > 127, -v, v) if signed else v
    return torch.ldexp(v.view(-1, GROUP), (b.to(torch.int32) - 127).float()[:, None]).view(-1)


def _with_handles(s):
    """What a training program keeps between calls: the compute handle with its
    workspace, output buffers, and the optimizer's list of tensors."""
    from fully_sharded_unit_gb300 import binding as B

    c, op = s["case"], s["case"]["op"]

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op.startswith("lp"):
        rows, v = c["rows"], c["vocab"]
        s["c"] = B.Compute(0)
        s["logprob"] = empty(rows, torch.float32)
        if op == "lp_fwd":
            s["entropy"] = empty(rows, torch.float32)
            if c["top"]:
                s["top_tokens"], s["top_logprobs"] = empty((rows, c["top"]), torch.int64), empty((rows, c["top"]), torch.float32)
        else:
            s["dz"] = empty((rows, v + c["pad"]), _TYPES[c["dtype"]])[:, :v]
    elif op.startswith("rn"):
        rows, cols, dt = c["rows"], c["cols"], _TYPES[c["dtype"]]
        s["c"] = B.Compute(B.fsdp_residual_norm_workspace_bytes(rows, cols))
        if op == "rn_fwd":
            s["out"], s["y"] = empty((rows, cols), dt), empty((rows, cols), dt)
            s["rstd"], s["post_rstd"] = empty(rows, torch.float32), empty(rows, torch.float32) if c["post"] else None
        else:
            gt = _TYPES[c["grads"]]
            s["dresidual"], s["dblock"], s["dgamma"] = empty((rows, cols), dt), empty((rows, cols), dt), empty(cols, gt)
            s["dpost"] = empty(cols, gt) if c["post"] else None
            s["dgate"] = empty(cols, gt) if c["gate"] else None
    else:
        s["c"] = B.Compute(0)
        p, g = ([t[a:a + n] for a, n in zip(s["flat"], s["sizes"])] for t in (s["param"], s["grad"]))
        copies = [s["copy"][a:a + n] for a, n in zip(s["flat"], s["sizes"])] if c["copy"] else None
        if c["state"] == "f32":
            m, v = ([t[a:a + n] for a, n in zip(s["begin"], s["sizes"])] for t in (s["m"], s["v"]))
        else:
            padded = s["index"]["padded"]
            s["m8"], s["v8"] = (B.State8(padded, signed=k == "m", codes=s[k][0], exps=s[k][1]) for k in "mv")
            s["m_out"], s["v_out"] = empty(padded, torch.bfloat16), empty(padded, torch.bfloat16)
            m, v = ([t.piece(a, n) for a, n in zip(s["begin"], s["sizes"])] for t in (s["m8"], s["v8"]))
        s["list"] = B.AdamWTensors(p, g, m, v, copies=copies, decay_scale=s["decay"])


# ---- the plain forms ----------------------------------------------------------

def _soft(z, scale):
    """(scale (z - max), its exponentials, their sum) of each row."""
    top = z.amax(dim=1, keepdim=True)
    d = (z - torch.where(top == -math.inf, torch.zeros_like(top), top)) * scale
    e = torch.exp(d)
    return d, e, e.sum(dim=1, keepdim=True)


def _entropy(d, e, total):
    return torch.log(total[:, 0]) - (e * torch.where(e > 0, d, torch.zeros_like(d))).sum(dim=1) / total[:, 0]


def _given(d, total, tokens):
    got = torch.gather(d, 1, tokens.clamp(min=0)[:, None])[:, 0] - torch.log(total[:, 0])
    return torch.where(tokens < 0, torch.zeros_like(got), got)


def _ranked(z, k):
    """The k largest of each row, the lowest index first among equals."""
    bits = (z + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    at = torch.arange(z.shape[1], device=z.device)
    return torch.topk((order << 32) | (0xFFFFFFFF - at), k, dim=1)[1]


def _logits_grad(s, d, p, ln, h):
    """p: probabilities; ln: log of the sum; h: entropies."""
    c, a, b = s["case"], s["a"][:, None], s["b"]
    dz = -a * p
    if b is not None:
        lp = torch.where(p > 0, d - ln, torch.zeros_like(d))
        dz = dz - b[:, None] * p * (lp + h[:, None])
    rows = torch.arange(c["rows"], device=dz.device)
    dz[rows, s["tokens"].clamp(min=0)] += torch.where(s["tokens"] < 0, torch.zeros_like(s["a"]), s["a"])
    return dz * c["scale"]


def _resnorm(s):
    """(residual stream, rstd of it, rstd of the block's result), in 32 bits."""
    o, r = s["block"].float(), None
    if s["post"] is not None:
        r = 1.0 / torch.sqrt((o * o).sum(dim=1, keepdim=True) / o.shape[1] + EPS)
        o = o * r * s["post"].float()
    if s["gate"] is not None:
        o = o * s["gate"].float()
    x = s["alpha"] * s["residual"].float() + o
    rstd = 1.0 / torch.sqrt((x * x).sum(dim=1) / x.shape[1] + EPS)
    return x, rstd, None if r is None else r[:, 0]


def _chance(s):
    """The 32 random bits of each element, of which the moments take 16 each."""
    mask, i = 0xFFFFFFFF, s["index"]
    key = _keys(s)[i["of"].long()]
    x = (i["place"] & mask) ^ key ^ ((i["place"] >> 32) * 0x85157AF5 & mask)
    x = (x ^ (x >> 16)) * 0xD36F86A9 & mask
    x = (x ^ (x >> 15)) * 0xC242E759 & mask
    return x ^ (x >> 16)


def _keys(s):
    """A 32-bit key for each tensor, from the step's seed and the tensor's number."""
    keys = [((s["seed"] * 0x9E3779B97F4A7C15 + (t + 1) * 0xD1B54A32D192ED03) & (2 ** 64 - 1)) >> 32 for t in range(len(s["sizes"]))]
    return torch.tensor(keys, device="cuda")


def _plain_adamw(s):
    c, i = s["case"], s["index"]
    at, flat = i["at"], i["flat"]
    decay = torch.tensor([1.0 - HP["lr"] * HP["weight_decay"] * d for d in s["decay"]], dtype=torch.float64).float().cuda()[i["of"].long()]
    m, v = (s["m"], s["v"]) if c["state"] == "f32" else (_read8(*s["m"], True), _read8(*s["v"], False))
    g, p = s["grad"][flat].float(), s["param"][flat]
    m1 = HP["beta1"] * m[at] + (1.0 - HP["beta1"]) * g
    v1 = HP["beta2"] * v[at] + (1.0 - HP["beta2"]) * (g * g)
    t = s["step"]
    size = HP["lr"] / (1.0 - HP["beta1"] ** t)
    p = p * decay - size * (m1 / (torch.sqrt(v1 / (1.0 - HP["beta2"] ** t)) + HP["eps"]))
    s["param"][flat] = p
    if c["copy"]:
        s["copy"][flat] = p.to(torch.bfloat16)
    r = {"param": s["param"]}
    if c["copy"]:
        r["copy"] = s["copy"]
    if c["state"] == "f32":
        s["m"][at], s["v"][at] = m1, v1
        r["m"], r["v"] = s["m"], s["v"]
        return r
    bits = torch.zeros(i["padded"], dtype=torch.int64, device="cuda")
    bits[at] = _chance(s)
    new = torch.zeros(i["padded"], device="cuda")
    new[at] = m1
    q, b = _keep8(new, True, (bits & 0xFFFF).double() / 65536)
    s["m"][0].copy_(q), s["m"][1].copy_(b)
    new[at] = v1
    q, b = _keep8(new, False, (bits >> 16).double() / 65536)
    s["v"][0].copy_(q), s["v"][1].copy_(b)
    r["m"], r["v"] = _read8(*s["m"], True).to(torch.bfloat16), _read8(*s["v"], False).to(torch.bfloat16)
    return r


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op.startswith("lp"):
        z = s["z"].float()
        d, e, total = _soft(z, c["scale"])
        if op == "lp_fwd":
            r = {"logprob": _given(d, total, s["tokens"]), "entropy": _entropy(d, e, total)}
            if c["top"]:
                r["top_tokens"] = _ranked(z, c["top"])
                r["top_logprobs"] = torch.gather(d, 1, r["top_tokens"]) - torch.log(total)
            return r
        if op == "lp_bwd":
            d = (z - s["stats"][:, :1]) * c["scale"]
            p = torch.exp(d - s["stats"][:, 1:])
            return {"dz": _logits_grad(s, d, p, s["stats"][:, 1:], s["h"]).to(s["z"].dtype)}
        r = {"logprob": _given(d, total, s["tokens"])}
        h = _entropy(d, e, total) if c["entropy"] else None
        r["dz"] = _logits_grad(s, d, e / total, torch.log(total), h).to(s["z"].dtype)
        return r
    if op == "rn_fwd":
        dt = s["residual"].dtype
        x, rstd, post_rstd = _resnorm(s)
        r = {"out": x.to(dt), "y": (x * rstd[:, None] * s["gamma"].float()).to(dt), "rstd": rstd}
        if c["post"]:
            r["post_rstd"] = post_rstd
        return r
    if op == "rn_bwd":
        dt, gt, n = s["residual"].dtype, _TYPES[c["grads"]], c["cols"]
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = s["out"].float() * rstd
        g = dy * s["gamma"].float()
        t = s["dout"].float() + rstd * (g - xh * ((g * xh).sum(dim=1, keepdim=True) / n))
        r = {"dresidual": (s["alpha"] * t).to(dt), "dgamma": (dy * xh).sum(dim=0).to(gt)}
        u, e = s["block"].float(), t
        if c["post"]:
            u = u * s["post_rstd"][:, None]
            e = e * s["post"].float()
        if c["gate"]:
            e = e * s["gate"].float()
        both = (t * u).sum(dim=0)
        if c["post"]:
            r["dpost"] = (both * s["gate"].float() if c["gate"] else both).to(gt)
            e = s["post_rstd"][:, None] * (e - u * ((e * u).sum(dim=1, keepdim=True) / n))
        if c["gate"]:
            r["dgate"] = (both * s["post"].float() if c["post"] else both).to(gt)
        r["dblock"] = e.to(dt)
        return r
    return _plain_adamw(s)


def _own(s):
    c, op, h = s["case"], s["case"]["op"], s["c"]
    if op == "lp_fwd":
        h.token_logprobs_forward(s["z"], s["tokens"], s["logprob"], entropy=s["entropy"], top_tokens=s.get("top_tokens"),
                                 top_logprobs=s.get("top_logprobs"), scale=c["scale"])
        r = {"logprob": s["logprob"], "entropy": s["entropy"]}
        if c["top"]:
            r.update(top_tokens=s["top_tokens"], top_logprobs=s["top_logprobs"])
        return r
    if op == "lp_bwd":
        h.token_logprobs_backward(s["z"], s["tokens"], s["stats"], s["dz"], dlogprob=s["a"], entropy=s["h"], dentropy=s["b"], scale=c["scale"])
        return {"dz": s["dz"]}
    if op == "lp_loss":
        h.token_logprobs_loss(s["z"], s["tokens"], s["logprob"], s["dz"], dlogprob=s["a"], dentropy=s["b"], scale=c["scale"])
        return {"logprob": s["logprob"], "dz": s["dz"]}
    if op == "rn_fwd":
        h.residual_norm_forward(s["residual"], s["out"], block=s["block"], post_gamma=s["post"], gate=s["gate"], residual_scale=s["alpha"],
                                y=s["y"], gamma=s["gamma"], eps=EPS, rstd=s["rstd"], post_rstd=s["post_rstd"])
        r = {"out": s["out"], "y": s["y"], "rstd": s["rstd"]}
        if c["post"]:
            r["post_rstd"] = s["post_rstd"]
        return r
    if op == "rn_bwd":
        h.residual_norm_backward(s["dy"], s["dout"], s["out"], s["block"], s["dresidual"], s["dblock"], gamma=s["gamma"], rstd=s["rstd"],
                                 dgamma=s["dgamma"], post_gamma=s["post"], post_rstd=s["post_rstd"], dpost_gamma=s["dpost"], gate=s["gate"],
                                 dgate=s["dgate"], residual_scale=s["alpha"])
        r = {"dresidual": s["dresidual"], "dblock": s["dblock"], "dgamma": s["dgamma"]}
        if c["post"]:
            r["dpost"] = s["dpost"]
        if c["gate"]:
            r["dgate"] = s["dgate"]
        return r
    h.adamw_tensors(s["list"], HP, s["step"], seed=s["seed"])
    r = {"param": s["param"]}
    if c["copy"]:
        r["copy"] = s["copy"]
    if c["state"] == "f32":
        r.update(m=s["m"], v=s["v"])
        return r
    h.state8_unpack(s["m8"], s["m_out"])
    h.state8_unpack(s["v8"], s["v_out"])
    r.update(m=s["m_out"], v=s["v_out"])
    return r


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without --------------------------------------------

_SIZE = {"bf16": 2, "f32": 4}


def work(case):
    c, op = case, case["op"]
    if op.startswith("lp"):
        n, b, rows = c["rows"] * c["vocab"], _SIZE[c["dtype"]], c["rows"]
        if op == "lp_fwd":
            return {"bytes": n * b + rows * (16 + 12 * c["top"]), "flops": 7 * n}
        return {"bytes": 2 * n * b + rows * (16 + 8 * (op == "lp_bwd") + 8 * c["entropy"]), "flops": (5 + 5 * (op == "lp_loss") + 3 * c["entropy"]) * n}
    if op.startswith("rn"):
        n, b, p = c["rows"] * c["cols"], _SIZE[c["dtype"]], _SIZE[c["params"]] * c["cols"] * (1 + c["post"] + c["gate"])
        if op == "rn_fwd":
            return {"bytes": 4 * n * b + p + 8 * c["rows"], "flops": 10 * n}
        return {"bytes": 6 * n * b + p + _SIZE[c["grads"]] * c["cols"] * (1 + c["post"] + c["gate"]) + 8 * c["rows"], "flops": 22 * n}
    n = sum(k for k, _ in _shapes(c["model"], c["blocks"]))
    states = 16 if c["state"] == "f32" else 4 * (1 + 1 / GROUP) + 2 * (1 + 1 / GROUP) + 4     # 8 bits: updated, then read as bf16 values
    return {"bytes": n * (8 + _SIZE[c["grads"]] + states + 2 * c["copy"]), "flops": 16 * n}


# ---- 64 bits ------------------------------------------------------------------

def _exact_logits(s):
    """Rows in pieces: 64 bits of a whole matrix of logits are many GB."""
    c, op, k = s["case"], s["case"]["op"], s["case"]["scale"]
    parts = []
    for at in range(0, c["rows"], 512):
        rows = slice(at, at + 512)
        z, tokens = s["z"][rows].double() * k, s["tokens"][rows]
        lse = torch.logsumexp(z, dim=1, keepdim=True)
        if op == "lp_bwd":
            lse = s["stats"][rows, :1].double() * k + s["stats"][rows, 1:].double()
        lp = z - lse
        p = lp.exp()
        some = tokens >= 0
        r = {"logprob": torch.where(some, lp.gather(1, tokens.clamp(min=0)[:, None])[:, 0], 0.0)}
        plogp = torch.xlogy(p, p)
        h = -plogp.sum(dim=1)
        if op == "lp_fwd":
            r["entropy"] = h
            if c["top"]:
                r["top_tokens"] = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :c["top"]].clone()
                r["top_logprobs"] = lp.gather(1, r["top_tokens"])
        else:
            a = s["a"][rows].double()[:, None]
            one = torch.zeros_like(p).scatter_(1, tokens.clamp(min=0)[:, None], some.double()[:, None])
            dz = a * (one - p)
            if c["entropy"]:
                if op == "lp_bwd":
                    h, plogp = s["h"][rows].double(), torch.where(p > 0, p * lp, 0.0)
                dz -= s["b"][rows].double()[:, None] * (plogp + p * h[:, None])
            r = {"dz": (dz * k).float()} if op == "lp_bwd" else {"logprob": r["logprob"], "dz": (dz * k).float()}
        parts.append(r)
    return {name: torch.cat([r[name] for r in parts]) for name in parts[0]}


def _exact_resnorm(s):
    c, n = s["case"], s["case"]["cols"]
    o, h = s["block"].double(), s["residual"].double()
    post, gate = (torch.ones(n, dtype=torch.float64, device="cuda") if s[k] is None else s[k].double() for k in ("post", "gate"))
    gamma = s["gamma"].double()
    if c["op"] == "rn_fwd":
        r2 = torch.rsqrt(o.square().mean(dim=1) + EPS)
        x = torch.addcmul(h * s["alpha"], o * r2[:, None] if c["post"] else o, post * gate)
        r1 = torch.rsqrt(x.square().mean(dim=1) + EPS)
        r = {"out": x, "y": torch.einsum("rc,r,c->rc", x, r1, gamma), "rstd": r1}
        return dict(r, post_rstd=r2) if c["post"] else r
    dy, x, r1 = s["dy"].double(), s["out"].double(), s["rstd"].double()
    g = dy * gamma
    along = torch.einsum("rc,rc->r", g, x) / n
    t = s["dout"].double() + g * r1[:, None] - x * (r1 ** 3 * along)[:, None]
    r = {"dresidual": t * s["alpha"], "dgamma": torch.einsum("rc,rc,r->c", dy, x, r1)}
    e = t * (post * gate)
    if c["post"]:
        r2 = s["post_rstd"].double()
        sums = torch.einsum("rc,rc,r->c", t, o, r2)
        r["dpost"] = sums * gate
        r["dblock"] = e * r2[:, None] - o * (r2 ** 3 * torch.einsum("rc,rc->r", e, o) / n)[:, None]
    else:
        sums = torch.einsum("rc,rc->c", t, o)
        r["dblock"] = e
    if c["gate"]:
        r["dgate"] = sums * post
    return r


def _exact_small(x, least, half):
    """|x| < 2 as small floats with three bits below the leading one and exponents from ``least`` on; half: what is added before cutting."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** least))) - 3)
    return torch.floor(x / step + half) * step


def _exact_adamw(s):
    c, i, t = s["case"], s["index"], s["step"]
    where = i["at"]

    def moment(x, least, half=None, keep=False):
        if not keep:
            q, b = x
            sign = torch.where(q.view(-1, GROUP) > 127, -1.0, 1.0).double() if least == -14 else 1.0
            k = (q & 127 if least == -14 else q).view(-1, GROUP).double()
            e = torch.floor(k / 8)
            f = torch.where(e > 0, (k - 8 * e) / 8 + 1, k / 8) * torch.exp2(e.clamp(min=1) + (least - 1))
            return (sign * f * torch.exp2(b.double() - 127)[:, None]).flatten()[where]
        full, chance = (torch.zeros(i["padded"], dtype=torch.float64, device="cuda").index_copy_(0, where, w).view(-1, GROUP) for w in (x, half))
        top = full.abs().amax(dim=1, keepdim=True)
        unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -126))))
        unit = torch.where(top > 1.875 * unit, 2 * unit, unit)
        kept = _exact_small(full.abs() / unit, least, chance)
        if least != -14:
            kept = torch.where((full > 0) & (kept == 0), 2.0 ** (least - 3), kept)
        return (kept * unit * torch.sign(full)).flatten()

    m, v = (s["m"].double()[where], s["v"].double()[where]) if c["state"] == "f32" else (moment(s["m"], -14), moment(s["v"], -30))
    g = s["grad"].double()[i["flat"]]
    m = torch.lerp(g, m, HP["beta1"])
    v = torch.lerp(g.square(), v, HP["beta2"])
    p = s["param"].double()
    wd = torch.tensor(s["decay"], dtype=torch.float64, device="cuda")[i["of"].long()] * HP["weight_decay"]
    old = p[i["flat"]]
    step = m / (1 - HP["beta1"] ** t) / (torch.sqrt(v / (1 - HP["beta2"] ** t)) + HP["eps"])
    p[i["flat"]] = old - HP["lr"] * (wd * old + step)
    r = {"param": p}
    if c["copy"]:
        r["copy"] = torch.zeros_like(p).index_copy_(0, i["flat"], p[i["flat"]])
    if c["state"] == "f32":
        for name, x in (("m", m), ("v", v)):
            r[name] = torch.zeros(i["padded"], dtype=torch.float64, device="cuda").index_copy_(0, where, x)
        return r
    word = _chance(s)
    r["m"] = moment(m, -14, (word % 65536).double() / 65536, keep=True)
    r["v"] = moment(v, -30, torch.floor(word.double() / 65536) / 65536, keep=True)
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("lp"):
        return _exact_logits(s)
    return _exact_resnorm(s) if case["op"].startswith("rn") else _exact_adamw(s)
