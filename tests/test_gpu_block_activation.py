"""The activations' fp32 evaluation against 64 bits, at the accuracy that
include/fsdp_unit.h states."""
import math

import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


def _exact(z, act):
    """(activation, slope)"""
    if act == "gelu_erf":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(8 / math.pi)
    p = torch.sigmoid(k * (z + 0.044715 * z ** 3))
    return z * p, p + z * p * (1 - p) * k * (1 + 3 * 0.044715 * z * z)


@pytest.mark.parametrize("act", ["gelu_tanh", "gelu_erf"])
def test_gelu_in_f32(act):
    """2^-21 |z| and, for the slope, 2^-17: the comments beside the functions derive
    them.  Values of every size from 2^-8 to 2^6, both signs."""
    n, rows = 512, 3000
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    z = torch.empty((rows, n), device="cuda").normal_(generator=gen)
    z *= torch.exp2(torch.randint(-8, 5, (rows, 1), device="cuda", generator=gen).float())
    c = B.Compute(B.fsdp_linear_workspace_bytes(rows, n, n))
    k, v, y = B.Act8(rows, n), torch.empty_like(z), torch.empty_like(z)
    c.act8_pack(z, k)
    c.act8_unpack(k, v)
    c.act8_unpack(k, y, activation=act)
    assert bool(((y.double() - _exact(v.double(), act)[0]).abs() <= 2.0 ** -21 * v.double().abs()).all())
    # ones through an identity: the slope itself
    one, eye, d = torch.ones((rows, n), dtype=BF, device="cuda"), torch.eye(n, device="cuda").to(BF), torch.empty_like(z)
    c.linear_grad_input(one, eye, d, activation=act, preact=z)
    assert c.status() == 0
    c.close()
    assert (d.double() - _exact(z.double(), act)[1]).abs().max().item() <= 2.0 ** -17
