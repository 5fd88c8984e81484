"""8-bit moments at values that a code stands for, and next to those halfway between codes."""
import numpy as np
import pytest
import torch

import test_gpu_adamw_tensors as A
from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
f = np.float32


@pytest.fixture(scope="module")
def c():
    from conftest import library
    library()
    h = B.Compute(0)
    yield h
    h.close()


@pytest.mark.parametrize("off", [0, 1])
def test_every_code_is_the_rules(c, off):
    """Any values: one code for each, or one of two where value and random bits add up to a code exactly."""
    n = 2 ** 21 + 13
    rng = np.random.default_rng(2)
    with np.errstate(over="ignore"):   # few bits, so that many sums are a code exactly, and a few infinities
        g = (rng.normal(size=n) * np.exp(rng.normal(size=n) * 3)).astype(np.float16).astype(f)
    p, gt = (torch.zeros(n + off, device="cuda")[off:] for _ in range(2))
    gt.copy_(torch.from_numpy(g))
    m, v = (B.State8(n, s, torch.zeros(n + off, dtype=torch.uint8, device="cuda")[off:]) for s in (True, False))
    c.adamw_tensors(B.AdamWTensors([p], [gt], [m], [v]), dict(A.HP, lr=0.0, beta1=0.0, beta2=0.0), 1, seed=5)
    rm, rv = A.random_bits(n, 0, 5)
    for state, x, r in ((m, g, rm), (v, g * g, rv)):
        A.same(state.exps, A.encode(x, state.signed, r)[1], "exponents")
        A.same_codes(state.codes, x, state.signed, r, "codes")


@pytest.mark.parametrize("signed", [True, False])
def test_codes_pack_to_themselves(c, signed):
    """Every code beside one in the upper half of its exponent, which fixes the group's byte."""
    codes = np.arange(256, dtype=np.uint8).repeat(252)
    codes = codes[codes != 128] if signed else codes       # there is no negative zero
    groups = np.zeros((-(-len(codes) // 31), 32), np.uint8)
    flat = np.zeros(groups.shape[0] * 31, np.uint8)
    flat[:len(codes)] = codes
    groups[:, 1:] = flat.reshape(-1, 31)
    groups[:, 0] = 127 if signed else 255                  # 1.875, the largest of an exponent byte
    exps = (np.arange(len(groups)) % 252 + 1).astype(np.uint8)
    exps[exps < 36] += 36                                  # what the smallest code stands for is a float of full accuracy
    n = groups.size
    s = B.State8(n, signed, torch.from_numpy(groups.reshape(-1).copy()).cuda(), torch.from_numpy(exps).cuda())
    x, t = torch.empty(n, device="cuda"), B.State8(n, signed)
    c.state8_unpack(s, x)
    c.state8_pack(x, t)
    A.same(t.exps, exps, "exponents")
    A.same(t.codes, groups.reshape(-1), "codes")


@pytest.mark.parametrize("signed", [True, False])
def test_pack_next_to_halves(c, signed):
    """The smallest codes are whole numbers of one step: the values a last place above, at and below each half between two of
    them go up, to the even one and down."""
    least, first = (-17, 1) if signed else (-33, 2)         # an unsigned element that is not 0 is at least the first code
    k = np.arange(first if not signed else 0, 8) + 0.5
    half = np.ldexp(k, least).astype(f)
    x = np.concatenate([np.nextafter(half, f(0)), half, np.nextafter(half, f(4))])
    want = np.concatenate([np.floor(k), np.rint(k), np.ceil(k)]).astype(np.uint8)
    for top in (1.0, 2.0 ** -40, 2.0 ** 14, 2.0 ** 60):
        group = np.zeros(32, f)
        group[:len(x)] = x * f(top)
        group[31] = top
        s = B.State8(32, signed)
        c.state8_pack(torch.from_numpy(group).cuda(), s)
        A.same(s.codes[:len(x)], want, f"codes under {top}")
