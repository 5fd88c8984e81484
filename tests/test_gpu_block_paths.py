"""The linear layer at shapes whose products take every path of the product
kernels (tests/test_product_plan.py says which), with the whole epilogue, against
64-bit products."""
import math

import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

from block_harness import U, U32, Guarded
from plan_harness import PRODUCTS

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


@pytest.fixture
def rand():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)

    def normal(rows, cols, std=1.0, dtype=BF, pad=0, offset=0):
        t = torch.empty((rows, cols), device="cuda").normal_(0, std, generator=gen).to(dtype)
        return Guarded(rows, cols, dtype, pad, offset, t).t if pad or offset else t

    return normal


def _place(N):
    """Rows that start anywhere where the width is odd."""
    return (3, 1) if N % 2 else (0, 0)


def _near(got, want, tol, what):
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), (what, int((off > tol).sum()), (off / tol).max().item())


def _rounded(want, e, dtype):
    return U[dtype] * (want.abs() + e) + e


def _sum_error(a, b, k, exact):
    """Products of one size: up to a unit of 2^-23 of the magnitudes' sum in each step
    of 16 of a slice, and the slices' and parts' additions; the magnitudes' sum is
    at most the rows' and columns' norms' product."""
    size = a.double().norm(dim=1)[:, None] * b.double().norm(dim=0)[None]
    longest = 768 if exact else 16384
    return ((min(k, longest) / 16 + 2) * 2.0 ** -23 + (k / longest + 80) * 2.0 ** -24) * size


def _activation(z, act):
    """(value, slope) in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu_erf":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(8 / math.pi)
    p = torch.sigmoid(k * (z + 0.044715 * z ** 3))
    return z * p, p + z * p * (1 - p) * k * (1 + 3 * 0.044715 * z * z)


def _read8(c, k):
    v = torch.empty((k.rows, k.cols), device="cuda")
    c.act8_unpack(k, v)
    return v.double()


def _keeps(c, k, z, ez):
    """Half a step, or a whole one at the top of a group; exponents as the group's
    largest has them; zeros in the pads of a short group."""
    cols = k.cols
    E = k.exps.double() - 127
    step = torch.exp2(E - 6).repeat_interleave(32, dim=1)[:, :cols]
    tol = torch.where(z.abs() + ez >= 127 * step, step, step / 2) + ez
    _near(_read8(c, k), z, tol, "kept")
    fold = lambda a: torch.nn.functional.pad(a, (0, -cols % 32)).unflatten(1, (-1, 32)).amax(dim=2)  # noqa: E731
    top, et = fold(z.abs()), fold(ez)
    assert bool((torch.exp2(E) <= top + et).all()) and bool((top - et < torch.exp2(E + 1)).all())
    assert not bool(k.q[:, cols:].any())


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("act,res,keep,odt", [("gelu_tanh", None, "act8", BF), ("gelu_erf", "same", "bf16", BF), ("relu", "other", "f32", F32)])
def test_forward(rand, M, N, K, layout, act, res, keep, odt):
    pad, offset = _place(N)
    x = rand(M, K, 1.0, BF, pad, offset)
    w = rand(*((K, N) if layout == "in_out" else (N, K)), K ** -0.5, BF, pad, offset)
    W = w if layout == "in_out" else w.t()
    bias = rand(1, N, 0.5, F32 if res else BF)[0]
    y = Guarded(M, N, odt, pad, offset)
    residual = None
    if res == "same":
        y.t.copy_(rand(M, N, 1.0, odt))
        residual = y.t
    elif res == "other":
        residual = rand(M, N, 1.0, BF, pad, offset)
    R = 0 if residual is None else residual.double()
    pre = B.Act8(M, N) if keep == "act8" else Guarded(M, N, BF if keep == "bf16" else F32, pad, offset)
    if keep == "act8":
        pre.q.fill_(99)
    c = B.Compute(B.fsdp_linear_workspace_bytes(M, K, N, weight_aligned=w))
    c.linear_forward(x, w, y.t, bias=bias, activation=act, residual=residual, preact=pre if keep == "act8" else pre.t, weight_layout=layout)
    assert c.status() == 0
    y.check()
    z = x.double() @ W.double() + bias.double()
    ez = _sum_error(x, W, K, keep != "bf16") + 2 * U32 * z.abs()
    Y = _activation(z, act)[0] + R
    ey = ez if act == "relu" else 1.13 * ez + 2.0 ** -18 * z.abs()
    ey = ey + 2 * U32 * (Y.abs() + (R.abs() if res else 0))
    _near(y.t, Y, _rounded(Y, ey, odt), "y")
    if keep == "act8":
        _keeps(c, pre, z, ez)
    else:
        pre.check()
        _near(pre.t, z, _rounded(z, ez, pre.t.dtype), "z")
    c.close()


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("act,keep,add,odt", [("gelu_tanh", "act8", "same", BF), ("gelu_erf", "bf16", None, BF), ("relu", "f32", "other", F32)])
def test_grad_input(rand, M, N, K, layout, act, keep, add, odt):
    pad, offset = _place(N)
    dy = rand(M, K, 1.0, BF, pad, offset)
    w = rand(*((N, K) if layout == "in_out" else (K, N)), K ** -0.5, BF, pad, offset)
    W = w if layout == "in_out" else w.t()             # N x K
    z = rand(M, N, 1.5, F32 if keep == "f32" else BF, pad, offset)
    c = B.Compute(B.fsdp_linear_workspace_bytes(M, N, K, weight_aligned=w))
    pre, Z = z, z.double()
    if keep == "act8":
        pre = B.Act8(M, N)
        c.act8_pack(z, pre)
        Z = _read8(c, pre)
    dx = Guarded(M, N, odt, pad, offset)
    extra = None
    if add == "same":
        dx.t.copy_(rand(M, N, 1.0, odt))
        extra = dx.t
    elif add == "other":
        extra = rand(M, N, 1.0, BF, pad, offset)
    A = 0 if extra is None else extra.double()
    c.linear_grad_input(dy, w, dx.t, activation=act, preact=pre, add=extra, weight_layout=layout)
    assert c.status() == 0
    c.close()
    dx.check()
    P = dy.double() @ W.double().t()
    ep = _sum_error(dy, W.t(), K, odt == F32)
    DX = P * _activation(Z, act)[1] + A
    ed = 1.13 * ep + (P.abs() + ep) * (2.0 ** -24 if act == "relu" else 2.0 ** -17) + 2 * U32 * (DX.abs() + (A.abs() if add else 0))
    _near(dx.t, DX, _rounded(DX, ed, odt), "dx")


@pytest.mark.parametrize("M,N,K", [p for p in PRODUCTS if p[0] > 256])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("x8,gdt,accumulate", [(False, F32, True), (True, BF, False), (False, BF, True)])
def test_grad_weight(rand, M, N, K, layout, x8, gdt, accumulate):
    pad, offset = _place(N)
    I, O_ = (M, N) if layout == "in_out" else (N, M)
    x, dy = rand(K, I, 1.0, BF, pad, offset), rand(K, O_, K ** -0.5, BF, pad, offset)
    c = B.Compute(B.fsdp_linear_workspace_bytes(K, I, O_))
    source, X = x, x
    if x8:
        source = B.Act8(K, I)
        c.act8_pack(x, source)
        X = _read8(c, source)
    old, oldb = rand(M, N, 1.0, gdt), rand(1, O_, 1.0, gdt)
    dw, db = Guarded(M, N, gdt, 0, offset, old), Guarded(1, O_, gdt, 0, 1, oldb)
    c.linear_grad_weight(source, dy, dw.t, dbias=db.t[0], weight_layout=layout, accumulate=accumulate)
    assert c.status() == 0
    c.close()
    dw.check()
    db.check()
    DW = X.double().t() @ dy.double()
    ew = _sum_error(X.t(), dy, K, gdt == F32)
    if layout == "out_in":
        DW, ew = DW.t(), ew.t()
    DB, eb = dy.double().sum(0), (K / 8 + 64) * U32 * dy.double().abs().sum(0)
    if accumulate:
        DW, DB = DW + old.double(), DB + oldb.double()[0]
    _near(dw.t, DW, _rounded(DW, ew + 2 * U32 * DW.abs(), gdt), "dw")
    _near(db.t[0], DB, _rounded(DB, eb + 2 * U32 * DB.abs(), gdt), "db")
