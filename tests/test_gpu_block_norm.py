"""The layer norm's gradients where a row's mean is far larger than its
deviation."""
import numpy as np
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B
from oracle import block_oracle as O

from block_harness import U32, inside, np64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


@pytest.mark.parametrize("cols", [40, 256, 768, 1280, 2048, 4096, 5120, 8192, 12288, 16384, 20480, 129, 5121])
@pytest.mark.parametrize("mean", [1.0, 100.0, -1000.0, 10000.0])
@pytest.mark.parametrize("kind", ["f32", "bf16", "act8"])
def test_backward_of_rows_with_a_large_mean(cols, mean, kind):
    """x - mean is rounded once and its product with rstd once, so x-hat is known to
    2.01 u of itself, however large the mean; dgamma of one row adds one rounded
    product.  (With mean * rstd rounded by itself x-hat was off by u |mean| rstd.)"""
    rng = np.random.default_rng(cols)
    x = torch.from_numpy(rng.normal(mean, 1.0, (1, cols))).to(BF if kind == "bf16" else F32).cuda()
    dy = torch.from_numpy(rng.normal(0, 1, (1, cols))).to(BF if kind == "bf16" else F32).cuda()
    gamma = torch.from_numpy(rng.normal(1, 0.2, cols)).float().cuda()
    X = np64(x)
    m, r = torch.from_numpy(X.mean(1)).float().cuda(), torch.from_numpy(1 / np.sqrt(X.var(1) + 1e-5)).float().cuda()
    c = B.Compute(B.fsdp_layer_norm_workspace_bytes(1, cols))
    source = x
    if kind == "act8":
        source = B.Act8(1, cols)
        c.act8_pack(x, source)
        X = O.act8_unpack(source.q.cpu().numpy(), source.exps.cpu().numpy(), cols)
    dx = torch.empty((1, cols), device="cuda")
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    c.layer_norm_backward(dy, source, gamma, m, r, dx, dg, db)
    assert c.status() == 0
    c.close()
    DY, G, M, R = np64(dy), np64(gamma), np64(m), np64(r)
    DX, DG, DB = O.layer_norm_grad(DY, X, G, M, R)
    xh = np.abs((X - M[:, None]) * R[:, None])
    exh = 2.01 * U32 * xh
    inside(dg, DG, (np.abs(DY) * (exh + 1.01 * U32 * xh))[0] + 1e-38, "dgamma")
    assert np.array_equal(np64(db), DB)
    gm = np.abs(DY * G)
    row = (cols / 1024 + 128) * U32
    c1, c2 = gm.mean(1)[:, None], (gm * xh).mean(1)[:, None]
    e1, e2 = row * c1, row * c2 + (gm * exh).mean(1)[:, None]
    inside(dx, DX, R[:, None] * (4 * U32 * (gm + c1 + xh * c2) + e1 + xh * e2 + exh * c2) + 3 * U32 * np.abs(DX), "dx")
