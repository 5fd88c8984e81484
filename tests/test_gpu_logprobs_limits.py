"""Log probabilities where a term's form changes: largest logits on both sides of |z| scale log2(e) = 2^20."""
import math

import numpy as np
import pytest
import torch

import test_gpu_logprobs as L
from block_harness import U, inside
from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def c():
    from conftest import library
    library()
    h = B.Compute(0)
    yield h
    h.close()


def _rows(vocab, scale, sign):
    """Logits a few last places apart around sign 2^20 / (scale log2 e), rising, falling, in any order, and with either side
    at a row's ends alone.  A place is 2^-24 to 2^-23 of the limit, 0.04 to 0.09 in scale z."""
    limit = np.float32(2.0 ** 20 / (scale * math.log2(math.e)))
    up = (limit.view(np.int32) + np.arange(-24, 24) * 2).astype(np.int32).view(np.float32)
    z = np.sort(np.resize(up, vocab))
    rng = np.random.default_rng(vocab)
    ends = np.sort(rng.permutation(z))
    rows = np.stack([z, z[::-1], rng.permutation(z), np.roll(ends, vocab // 2), np.where(np.arange(vocab) < vocab - 2, up[20], up[27]),
                     np.where(np.arange(vocab) < 2, up[27], up[20])])
    return torch.from_numpy(np.ascontiguousarray(sign * rows, dtype=np.float32)).cuda()


@pytest.mark.parametrize("scale", [1.0, 1e3, 1e5])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("vocab", [97, 8192, 50257])
def test_largest_logits_on_both_sides_of_the_limit(c, vocab, scale, sign):
    """The logits are floats and the definition is taken at them.  A term's argument is off by 2^-23 of itself (below 2^-23 * 8 here) and
    by 2^-24 of what is up to 2^-4 of the largest: inside _eps, which allows for arguments of the size of ln S."""
    z = _rows(vocab, scale, sign)
    rows = len(z)
    t = torch.randint(0, vocab, (rows,), device="cuda")
    lp, st, h = L._check_forward(c, z, t, scale, 5)
    a = torch.ones(rows, device="cuda")
    for b in (None, a):
        want, tol = L._wanted_grad(z, t, scale, a, b)
        tol = tol + U[F32] * np.abs(want)
        dz = torch.empty_like(z)
        c.token_logprobs_backward(z, t, st, dz, dlogprob=a, entropy=h if b is not None else None, dentropy=b, scale=scale)
        inside(dz, want, tol, "backward")
        lp2, h2, st2 = torch.empty_like(lp), torch.empty_like(h), torch.empty_like(st)
        c.token_logprobs_loss(z, t, lp2, dz, dlogprob=a, dentropy=b, entropy=h2, stats=st2, scale=scale)
        L._check_rows(L._reference(z, t, scale), vocab, lp2, st2, h2)
        inside(dz, want, tol, "loss")
    assert c.status() == 0
