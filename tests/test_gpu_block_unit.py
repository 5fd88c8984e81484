"""The block operators together, inside a unit's step: gradients of the MLP unit
against 64-bit autograd, and a training run whose loss falls.  And gradients of
single operators against differences of the forward pass."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from conftest import ROOT
from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


def _example():
    spec = importlib.util.spec_from_file_location("train_mlp_unit", os.path.join(ROOT, "examples", "train_mlp_unit.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("d,ffn,tokens,grad_dtype", [(128, 512, 96, "f32"), (72, 264, 200, "bf16"), (40, 129, 33, "f32")])
def test_unit_gradients(d, ffn, tokens, grad_dtype):
    """A checkpoint errs by at most 2^-7 of its group's largest value, uniformly:
    1.4 % of the tensor (a group's largest value is about three times its rms);
    both checkpoints, the slope that reads one of them, and the bf16 roundings of
    h, dz and dy (0.3 % each) give less than 5 % together."""
    m = _example().MlpUnit(d, ffn, tokens, 2, grad_dtype, std=0.1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.empty((tokens, d), device="cuda").normal_(generator=gen).to(BF)
    dy = torch.empty((tokens, d), device="cuda").normal_(generator=gen).to(BF)
    m.unit.allgather(m.gathered)
    y = m.forward(x).clone()
    dx = m.backward(dy, 1).clone()
    got = [g.clone() for g in m._views(m.grads[1])]
    xd = x.double().requires_grad_()
    p = [v.double().detach().requires_grad_() for v in m.params]
    n = torch.nn.functional.layer_norm(xd, (d,), p[0], p[1], 1e-5)
    want_y = torch.nn.functional.gelu(n @ p[2] + p[3], approximate="tanh") @ p[4] + p[5] + xd
    want_y.backward(dy.double())
    assert (y.double() - want_y).norm() <= 0.02 * want_y.norm()
    for name, a, b in zip(("dx", "ln w", "ln b", "w1", "b1", "w2", "b2"), [dx] + got, [xd.grad] + [v.grad for v in p]):
        assert (a.double() - b).norm() <= 0.05 * b.norm(), name
    assert m.close() == 0


def test_training_run_learns():
    m = _example().MlpUnit(128, 512, 256, 2)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    batches = [torch.empty((256, 128), device="cuda").normal_(generator=gen).to(BF) for _ in range(2)]
    targets = [b.roll(1, dims=1) for b in batches]
    hp = dict(lr=3e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    losses = [m.step(batches, targets, hp).item() for _ in range(60)]
    assert losses[-1] < 0.5 * losses[0], losses[::10]
    assert m.close() == 0


def test_layer_norm_gradient_against_differences():
    """L = sum(y r) in F32.  The difference quotient errs by h^2/6 times the third
    derivative along the direction (at most about 10 of the sizes below) and by
    the rounding of y, 2^-22 of sum |y r|, over 2h."""
    rows, cols, h = 5, 64, 2.0 ** -6
    rng = np.random.default_rng(0)
    t = lambda *s: torch.from_numpy(rng.normal(size=s)).float().cuda()  # noqa: E731
    x, gamma, beta, r = t(rows, cols), t(cols) + 2, t(cols), t(rows, cols)
    c = B.Compute(B.fsdp_layer_norm_workspace_bytes(rows, cols))
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)

    def loss(x, gamma, beta):
        c.layer_norm_forward(x, gamma, beta, 0.1, y, mean, rstd)
        return (y.double() * r.double()).sum().item()

    loss(x, gamma, beta)
    size = (y.double() * r.double()).abs().sum().item()
    c.layer_norm_backward(r, x, gamma, mean, rstd, dx, dg, db)
    for i, grad in enumerate((dx, dg, db)):
        args = [x, gamma, beta]
        for _ in range(4):
            d = t(*grad.shape)
            up, down = ([a + s * h * d if j == i else a for j, a in enumerate(args)] for s in (1, -1))
            slope = (loss(*up) - loss(*down)) / (2 * h)
            want = (grad.double() * d.double()).sum().item()
            assert abs(slope - want) <= h * h / 6 * 10 * size / rows + 2.0 ** -22 * size / h, (i, slope, want)
    c.close()


@pytest.mark.parametrize("act", ["gelu_tanh", "gelu_erf"])
def test_linear_gradient_against_differences(act):
    """L = sum(act(x W + b) r), y in F32; x and its steps are bf16 numbers.  The
    gradient goes through dz in F32 rounded to bf16 (2^-8), the quotient errs by
    h^2/6 of the third derivative (at most 1 an element times (dW)^3) and rounding."""
    T, I, O_, h = 9, 40, 72, 2.0 ** -4
    rng = np.random.default_rng(1)
    x = torch.from_numpy(np.rint(rng.normal(size=(T, I)) * 16) / 16).to(BF).cuda()
    w = torch.from_numpy(rng.normal(size=(I, O_)) * 0.1).to(BF).cuda()
    b, r = (torch.from_numpy(rng.normal(size=s)).float().cuda() for s in ((O_,), (T, O_)))
    c = B.Compute(B.fsdp_linear_workspace_bytes(T, 72, 72))
    y, z = torch.empty((T, O_), device="cuda"), torch.empty((T, O_), device="cuda")

    def loss(v):
        c.linear_forward(v, w, y, bias=b, activation=act, preact=z)
        return (y.double() * r.double()).sum().item()

    loss(x)
    size = (y.double() * r.double()).abs().sum().item()
    # dz = r * act'(z), through an identity weight; then dx = dz W^T
    eye = torch.eye(O_, device="cuda").to(BF)
    dz, dx = torch.empty((T, O_), dtype=BF, device="cuda"), torch.empty((T, I), device="cuda")
    rb = r.to(BF)
    r = rb.float()
    c.linear_grad_input(rb, eye, dz, activation=act, preact=z.clone())
    c.linear_grad_input(dz, w, dx)
    for _ in range(6):
        d = torch.from_numpy(rng.integers(-1, 2, size=(T, I))).float().cuda()
        slope = (loss((x.float() + h * d).to(BF)) - loss((x.float() - h * d).to(BF))) / (2 * h)
        want = (dx.double() * d.double()).sum().item()
        step = (d.double() @ w.double()).abs()
        bound = 2.0 ** -8 * (dz.double().abs() * step).sum().item() + h * h / 6 * (step ** 3 * r.double().abs()).sum().item() \
            + 2.0 ** -22 * size / h
        assert abs(slope - want) <= bound, (slope, want, bound)
    c.close()
