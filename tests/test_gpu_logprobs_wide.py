"""The loss on rows that take blocks of 1024 threads, alone and in pairs, and rows in shared memory that hold what is not finite.
Checks and bounds are those of test_gpu_logprobs."""
import math

import numpy as np
import pytest
import torch

import test_gpu_logprobs as L
from block_harness import U, Guarded, inside
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


@pytest.mark.parametrize("rows,vocab,dtype,pad", [(170, 50257, F32, 0), (160, 128256, BF, 0), (160, 60007, BF, 1), (160, 40000, F32, 4)])
@pytest.mark.parametrize("entropy", [False, True])
def test_loss(c, rows, vocab, dtype, pad, entropy):
    z, t = L._logits(rows, vocab, dtype, seed=3)
    t[1] = -1
    z[2] = -math.inf
    z[3, 5] = math.nan
    z[4, vocab - 1] = math.inf
    z[rows - 1, 1:] = -math.inf
    gz, dz = Guarded(rows, vocab, dtype, pad, offset=pad % 3, like=z), Guarded(rows, vocab, dtype, pad, offset=pad % 3)
    a, b = torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda") if entropy else None
    lp, st, h = torch.empty(rows, device="cuda"), torch.empty((rows, 2), device="cuda"), torch.empty(rows, device="cuda")
    for out in (dz, gz):     # and in place
        c.token_logprobs_loss(gz.t, t, lp, out.t, dlogprob=a, dentropy=b, entropy=h, stats=st)
        if out is dz:
            L._check_rows(L._reference(z, t, 1.0), vocab, lp, st, h)
            want, tol = L._wanted_grad(z, t, 1.0, a, b)
            inside(dz.t, want, np.nan_to_num(tol + U[dtype] * np.abs(want)), "dlogits")
        out.check()
    assert torch.equal(gz.t.nan_to_num(7.0), dz.t.nan_to_num(7.0))
    assert c.status() == 0
