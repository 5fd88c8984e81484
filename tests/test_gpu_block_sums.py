"""How exactly the linear layer adds up: sums of one sign, in which an
accumulator that cuts off instead of rounding errs the same way in every step."""
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


def _positive(gen, rows, cols):
    """Values in (0, 2), every row by a factor of its own in [1, 2), so that sums
    of products lie anywhere between two powers of two."""
    out = torch.empty((rows, cols), dtype=BF, device="cuda")
    factor = 1 + torch.rand((rows, 1), device="cuda", generator=gen)
    step = max(1, (1 << 27) // rows)
    for c in range(0, cols, step):
        part = out[:, c:c + step]
        part.copy_(torch.rand(part.shape, device="cuda", generator=gen) * factor)
    return out


def test_a_kept_checkpoint_comes_from_sums_as_exact_as_fp32_results():
    """z is known to ez, the error that an F32 result of these products may have
    (slices of 768 products are 48 steps, each off by at most a unit of 2^-23; the
    slices' additions round to nearest), so a kept element lies within half a step
    and ez of the exact sum.  Cut off in each of 2500 steps without slices, the sums
    put elements near a boundary beyond it."""
    T, I, O_ = 300, 40000, 8192
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x, w = _positive(gen, T, I), _positive(gen, O_, I)
    c = B.Compute(B.fsdp_linear_workspace_bytes(T, I, O_))
    k, y, v = B.Act8(T, O_), torch.empty((T, O_), dtype=BF, device="cuda"), torch.empty((T, O_), device="cuda")
    c.linear_forward(x, w, y, preact=k, weight_layout="out_in")
    c.act8_unpack(k, v)
    assert c.status() == 0
    c.close()
    z = torch.cat([x.double() @ part.double().t() for part in w.split(1024)], dim=1)
    ez = (48 * 2.0 ** -23 + (I / 768 + 20) * 2.0 ** -24) * z
    step = torch.exp2(k.exps.double() - 133).repeat_interleave(32, dim=1)
    off = (v.double() - z).abs()
    allowed = torch.where(z + ez >= 127 * step, step, step / 2) + ez
    assert bool((off <= allowed).all()), ((off - allowed) / step).max().item()


@pytest.mark.parametrize("kind", ["forward", "grad_weight"])
def test_long_bf16_sums_do_not_drift(kind):
    """The drift may be 2^-13, a thirty-second of BF16's own rounding (up to 2^-8):
    a unit of 2^-23 of the sum in each of 1024 steps of 16 products.  The rounding
    is to nearest and the sums lie anywhere, so it averages out over the elements;
    four deviations of its mean are added.  300000 products in one go are 18750 such
    steps, and were off by up to 1.7e-3."""
    T, I, O_ = 300, 300000, 8192
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x, w = _positive(gen, T, I), _positive(gen, O_, I)
    got = torch.empty((T, O_), dtype=BF, device="cuda")
    some = slice(0, O_, 32)
    want = torch.cat([x.double() @ part.double().t() for part in w[some].split(64)], dim=1)
    if kind == "forward":
        c = B.Compute(B.fsdp_linear_workspace_bytes(T, I, O_))
        c.linear_forward(x, w, got, weight_layout="out_in")
    else:
        c = B.Compute(B.fsdp_linear_workspace_bytes(I, T, O_))
        c.linear_grad_weight(x.t().contiguous(), w.t().contiguous(), got)
    assert c.status() == 0
    c.close()
    rel = (got[:, some].double() - want) / want
    assert rel.abs().max().item() <= 2.0 ** -8 + 2.0 ** -13 + 2.0 ** -18
    mean = rel.mean().abs().item()
    assert mean <= 2.0 ** -13 + 4 * 2.0 ** -8 / 3 ** 0.5 / rel.numel() ** 0.5, mean


@pytest.mark.parametrize("data,stated", [("random signs", 7e-7), ("one sign", 1.3e-6), ("one large product", 1.3e-5)])
@pytest.mark.parametrize("k", [768, 7680])
def test_fp32_sums_are_as_exact_as_the_header_states(data, stated, k):
    """Twice the header's measured figure, as norms: slices of 2048 products err by
    three times it for random signs, uncut sums of 7680 by ten."""
    T, O_ = 512, 4096
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    if data == "one sign":
        x, w = _positive(gen, T, k), _positive(gen, O_, k)
    else:
        x, w = (torch.empty((n, k), device="cuda").normal_(generator=gen) for n in (T, O_))
        if data == "one large product":
            x, w = x.abs(), w.abs()
            x[:, 0] = w[:, 0] = 512
        x, w = x.to(BF), w.to(BF)
    y = torch.empty((T, O_), device="cuda")
    c = B.Compute(B.fsdp_linear_workspace_bytes(T, k, O_))
    c.linear_forward(x, w, y, weight_layout="out_in")
    assert c.status() == 0
    c.close()
    want = x.double() @ w.double().t()
    off = ((y.double() - want).norm() / want.norm()).item()
    assert off <= 2 * stated, off


@pytest.mark.parametrize("k", [256, 512, 768, 1280, 3000])
def test_a_kept_checkpoint_of_random_signs(k):
    """Elements land on the wrong side of a rounding boundary in proportion to the
    sums' error, which slices keep within about twice that of fp32 sums (measured
    ones: 8e-9 sqrt(k) of the result).  As a norm, where each of these is one step
    off, the kept values' error is then within sqrt(2), and 1.5 with what the
    sample of a few thousand of them adds, of that from fp32 sums."""
    T, O_ = 4096, 2560
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    x, w = (torch.empty((n, k), device="cuda").normal_(generator=gen).to(BF) for n in (T, O_))
    c = B.Compute(B.fsdp_linear_workspace_bytes(T, k, O_))
    kept, y, v = B.Act8(T, O_), torch.empty((T, O_), dtype=BF, device="cuda"), torch.empty((T, O_), device="cuda")
    c.linear_forward(x, w, y, preact=kept, weight_layout="out_in")
    c.act8_unpack(kept, v)
    assert c.status() == 0
    c.close()

    def quantised(z):
        top = z.unflatten(1, (-1, 32)).abs().amax(dim=2, keepdim=True)
        step = torch.exp2(torch.floor(torch.log2(top)) - 6)
        return ((z.unflatten(1, (-1, 32)) / step).round().clamp(-127, 127) * step).flatten(1)

    z = x.double() @ w.double().t()
    exact = quantised(z)
    noise = 8e-9 * k ** 0.5 * z.square().mean().sqrt() * torch.empty_like(z).normal_(generator=gen)
    off = lambda a: ((a - exact).norm() / exact.norm()).item()  # noqa: E731
    assert off(v.double()) <= 1.5 * off(quantised(z + noise)), (off(v.double()), off(quantised(z + noise)))
