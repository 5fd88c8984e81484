"""The operators at a step's ends together with the block operators: a training step of a small
language model (embedding, a block between two norms with gate and residual scale, logits, loss,
gradients, AdamW over all tensors), against 64-bit autograd, and the same step from a graph."""
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS, ALPHA = 1e-5, 0.9
HP = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.01)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


class Model:
    """y0 = norm(E[tokens]); o = gelu(y0 W1 + b1) W2; h, y = norms of E[tokens] and o; logits = y W3."""

    def __init__(self, vocab, d, ffn, rows, moments, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.rows, self.vocab, self.d = rows, vocab, d
        shapes = dict(emb=(vocab, d), n0=(d,), w1=(d, ffn), b1=(ffn,), w2=(ffn, d), post=(d,), gate=(d,), n1=(d,), w3=(d, vocab))
        std = dict(emb=1.0, w1=d ** -0.5, w2=ffn ** -0.5, w3=2 * d ** -0.5)
        self.p = {k: torch.empty(s, device="cuda").normal_(0, std.get(k, 0.1), generator=g) + (len(s) == 1) for k, s in shapes.items()}
        self.b = {k: v.to(BF) for k, v in self.p.items()}       # what the operators compute with
        self.g = {k: torch.zeros_like(v) for k, v in self.p.items()}
        m = [B.State8(v.numel(), True) if moments == "8bit" else torch.zeros_like(v) for v in self.p.values()]
        v = [B.State8(t.numel(), False) if moments == "8bit" else torch.zeros_like(t) for t in self.p.values()]
        self.list = B.AdamWTensors(list(self.p.values()), list(self.g.values()), m, v, copies=list(self.b.values()),
                                   decay_scale=[float(len(s) > 1) for s in shapes.values()])
        self.c = B.Compute(max(B.fsdp_linear_workspace_bytes(rows, d, ffn), B.fsdp_linear_workspace_bytes(rows, d, vocab, weight_aligned=False),
                               B.fsdp_residual_norm_workspace_bytes(rows, d)))
        e = lambda *s, t=BF: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.y0, self.z, self.a, self.o, self.h, self.y, self.dy, self.dh, self.do, self.dx = e(rows, d), e(rows, ffn), e(rows, ffn), e(rows, d), e(rows, d), e(rows, d), e(rows, d), e(rows, d), e(rows, d), e(rows, d)
        self.x, self.x0, self.r0, self.r1, self.r2 = e(rows, d), e(rows, d), e(rows, t=F32), e(rows, t=F32), e(rows, t=F32)
        self.logits, self.lp = e(rows, vocab), e(rows, t=F32)

    def step(self, tokens, targets, weights):
        c, b, g = self.c, self.b, self.g
        torch.index_select(b["emb"], 0, tokens, out=self.x)
        c.residual_norm_forward(self.x, self.x0, y=self.y0, gamma=b["n0"], eps=EPS, rstd=self.r0)
        c.linear_forward(self.y0, b["w1"], self.a, bias=b["b1"], activation="gelu_tanh", preact=self.z)
        c.linear_forward(self.a, b["w2"], self.o)
        c.residual_norm_forward(self.x, self.h, block=self.o, post_gamma=b["post"], gate=b["gate"], residual_scale=ALPHA, y=self.y,
                                gamma=b["n1"], eps=EPS, rstd=self.r1, post_rstd=self.r2)
        c.linear_forward(self.y, b["w3"], self.logits)
        c.token_logprobs_loss(self.logits, targets, self.lp, self.logits, dlogprob=weights)     # in place
        c.linear_grad_weight(self.y, self.logits, g["w3"])
        c.linear_grad_input(self.logits, b["w3"], self.dy)
        c.residual_norm_backward(self.dy, None, self.h, self.o, self.dh, self.do, gamma=b["n1"], rstd=self.r1, dgamma=g["n1"], post_gamma=b["post"],
                                 post_rstd=self.r2, dpost_gamma=g["post"], gate=b["gate"], dgate=g["gate"], residual_scale=ALPHA)
        c.linear_grad_weight(self.a, self.do, g["w2"])
        c.linear_grad_input(self.do, b["w2"], self.a, activation="gelu_tanh", preact=self.z)
        c.linear_grad_weight(self.y0, self.a, g["w1"], dbias=g["b1"])
        c.linear_grad_input(self.a, b["w1"], self.dy)
        c.residual_norm_backward(self.dy, self.dh, self.x0, None, self.dx, None, gamma=b["n0"], rstd=self.r0, dgamma=g["n0"])
        mine = tokens[None, :, None] == torch.arange(self.vocab, device="cuda")[:, None, None]
        g["emb"].copy_(torch.where(mine, self.dx.float(), 0.0).sum(dim=1))

    def update(self, n, seed):
        self.c.adamw_tensors(self.list, HP, n, seed=seed)


def _data(vocab, rows, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    tokens, targets = (torch.randint(0, vocab, (rows,), device="cuda", generator=g) for _ in range(2))
    targets[::5] = -1
    return tokens, targets, torch.where(targets < 0, 0.0, -1.0 / int((targets >= 0).sum()))


def _rms(x):
    return x * torch.rsqrt(x.square().mean(dim=1, keepdim=True) + EPS)


@pytest.mark.parametrize("vocab,d,ffn,rows", [(300, 64, 136, 96), (1031, 40, 129, 70)])
def test_gradients(vocab, d, ffn, rows):
    """Each of the eight bf16 matrices between the operators is off by 2^-9 of itself at random; the products and norms
    behind them carry that on with weights of about one, so a gradient is off by sqrt(12) 2^-9 = 0.7 %; 2 % are
    allowed (3 % of the bias's sum over rows, which loses by cancellation)."""
    m = Model(vocab, d, ffn, rows, "f32")
    tokens, targets, weights = _data(vocab, rows, 1)
    m.step(tokens, targets, weights)
    p = {k: v.double().requires_grad_() for k, v in m.b.items()}
    x = p["emb"][tokens]
    o = torch.nn.functional.gelu((_rms(x) * p["n0"]) @ p["w1"] + p["b1"], approximate="tanh") @ p["w2"]
    h = ALPHA * x + p["gate"] * (_rms(o) * p["post"])
    lp = torch.log_softmax((_rms(h) * p["n1"]) @ p["w3"], dim=1)
    lp = torch.where(targets < 0, 0.0, lp.gather(1, targets.clamp(min=0)[:, None])[:, 0])
    (lp * weights).sum().backward()
    assert (m.lp.double() - lp).norm() <= 0.01 * lp.norm()
    for k, v in p.items():
        assert (m.g[k].double() - v.grad).norm() <= (0.03 if k == "b1" else 0.02) * v.grad.norm(), k
    assert m.c.status() == 0
    m.c.close()


@pytest.mark.parametrize("moments", ["f32", "8bit"])
def test_steps_run_alike_eagerly_and_from_a_graph(moments):
    vocab, d, ffn, rows = 500, 64, 128, 64
    runs = []
    for how in ("eager", "graph"):
        m = Model(vocab, d, ffn, rows, moments, seed=3)
        tokens, targets, weights = _data(vocab, rows, 2)
        m.step(tokens, targets, weights)
        if how == "graph":
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                m.step(tokens, targets, weights)
        for n in range(1, 4):
            t2, g2, w2 = _data(vocab, rows, 10 + n)
            tokens.copy_(t2), targets.copy_(g2), weights.copy_(w2)
            graph.replay() if how == "graph" else m.step(tokens, targets, weights)
            m.update(n, seed=100 + n)      # its constants are the step's: not from the graph
        torch.cuda.synchronize()
        assert all(bool(torch.isfinite(v).all()) for v in m.p.values())
        runs.append({k: v.clone() for k, v in m.p.items()})
        assert m.c.status() == 0
        m.c.close()
    for k in runs[0]:
        assert torch.equal(runs[0][k], runs[1][k]), k
    # every parameter moved
    m = Model(vocab, d, ffn, rows, moments, seed=3)
    for k, v in m.p.items():
        assert not torch.equal(v, runs[0][k]), k
    m.c.close()


def test_two_handles_on_two_streams():
    """Calls of two handles that may overlap give what each gives alone."""
    z = torch.randn((300, 5003), device="cuda").to(BF)
    t = torch.randint(0, 5003, (300,), device="cuda")
    a = torch.full((300,), -1.0, device="cuda")
    x, o = torch.randn((900, 1280), device="cuda").to(BF), torch.randn((900, 1280), device="cuda").to(BF)
    w = torch.ones(1280, dtype=BF, device="cuda")

    def make():
        c = B.Compute(B.fsdp_residual_norm_workspace_bytes(900, 1280))
        out = [torch.empty(300, device="cuda"), torch.empty_like(z), torch.empty_like(x), torch.empty_like(x), torch.empty(1280, device="cuda")]
        r = torch.rand(900, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) + 0.5
        return c, out, r

    def calls(c, out, r):
        c.token_logprobs_loss(z, t, out[0], out[1], dlogprob=a)
        c.residual_norm_backward(x, o, o, x, out[2], out[3], gamma=w, rstd=r, dgamma=out[4])

    c, want, r = make()
    calls(c, want, r)
    torch.cuda.synchronize()
    c.close()
    pairs = [make() for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, p in zip(streams, pairs):
            with torch.cuda.stream(s):
                calls(*p)
    torch.cuda.synchronize()
    for c, out, _ in pairs:
        assert all(torch.equal(u, v) for u, v in zip(out, want))
        c.close()
