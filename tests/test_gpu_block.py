"""Block operators against the 64-bit oracle, through the C ABI."""
import numpy as np
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B
from oracle import block_oracle as O

from block_harness import U, U32, Guarded, act_bound, inside, np64, product_bound, slope_bound

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


@pytest.fixture
def handle():
    c = B.Compute(64 << 20)
    yield c
    assert c.status() == 0
    c.close()


def _normal(seed, shape, std=1.0, dtype=F32, mean=0.0):
    return torch.from_numpy(np.random.default_rng(seed).normal(mean, std, shape)).to(dtype).cuda()


# ---- 8-bit checkpoints ---------------------------------------------------------

def _same_pack(x, k):
    q, b = O.act8_pack(np64(x))
    assert np.array_equal(k.exps.cpu().numpy(), b)
    assert np.array_equal(k.q.cpu().numpy(), q)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (3, 31, 0, 0), (2, 32, 8, 8), (5, 33, 3, 1), (7, 256, 0, 0),
                                                  (4, 264, 8, 0), (3, 264, 5, 0), (2, 1283, 1, 3), (300, 40, 0, 0),
                                                  (70, 1025, 2, 1), (9, 1056, 3, 2), (130, 37, 0, 0)])
def test_act8_pack_and_unpack(handle, dtype, rows, cols, pad, offset):
    x = Guarded(rows, cols, dtype, pad, offset, _normal(rows + cols, (rows, cols), 3.0, dtype)).t
    k = B.Act8(rows, cols)
    k.q.fill_(99)
    handle.act8_pack(x, k)
    _same_pack(x, k)
    want = O.act8_unpack(k.q.cpu().numpy(), k.exps.cpu().numpy(), cols)
    for odt in (BF, F32):
        for act in ("none", "relu", "gelu_tanh", "gelu_erf"):
            out = Guarded(rows, cols, odt, pad, offset)
            handle.act8_unpack(k, out.t, activation=act)
            out.check()
            a = O.activation(want, act)
            if act in ("none", "relu"):
                assert np.array_equal(np64(out.t), a)       # every value is a bf16 number
            else:
                e = act_bound(want, 0.0, act)
                inside(out.t, a, U[odt] * (np.abs(a) + e) + e, act)


def test_act8_special_values(handle):
    x = torch.zeros((3, 160), device="cuda")
    x[0, 5] = float("inf")
    x[0, 37] = float("nan")
    x[0, 64:96] = 2.0 ** -130                                  # subnormal: below the smallest step
    x[0, 96:128] = torch.linspace(-1, 1, 32) * 3.0e38
    x[0, 128:] = 1.9999
    x[1, :32] = -0.0
    x[1, 32:64] = 2.0 ** -119 * torch.linspace(0.1, 1, 32)
    x[1, 64:96] = torch.arange(32) + 0.5                       # ties at a step of 0.25 are exact, at the top too
    x[2] = torch.linspace(-127.5, 127.5, 160) / 64
    k = B.Act8(3, 160)
    handle.act8_pack(x, k)
    _same_pack(x, k)
    out = torch.empty((3, 160), dtype=BF, device="cuda")
    handle.act8_unpack(k, out)
    assert bool(torch.isnan(out[0, :64]).all()) and not bool(torch.isnan(out[0, 64:]).any())


def test_act8_zero_rows(handle):
    k = B.Act8(0, 40)
    handle.act8_pack(torch.empty((0, 40), device="cuda"), k)
    handle.act8_unpack(k, torch.empty((0, 40), device="cuda"))


# ---- layer norm ------------------------------------------------------------------

def _norm_bounds(x, gamma, beta, y, mean, rstd, odt):
    """The rows' sums are made of at most C/1024 + 64 additions in turn and a
    tree of 10 and 32 partial sums behind them."""
    C = x.shape[1]
    g = (C / 1024 + 128) * U32
    em = g * np.abs(x).mean(1) + U32 * np.abs(mean)
    d = np.abs(x - mean[:, None])
    # variance: relative g + 4u, and the mean's error enters squared (its first-order term sums to 0)
    er = (g + 8 * U32) * rstd + rstd ** 3 * em ** 2 + rstd ** 2 * em * 2 * U32 * C ** 0.5
    ey = np.abs(gamma) * (rstd[:, None] * (em[:, None] + 2 * U32 * (np.abs(x) + np.abs(mean)[:, None])) + d * (er + 4 * U32 * rstd)[:, None]) \
        + 4 * U32 * (np.abs(y) + np.abs(beta))
    return em, er, U[odt] * (np.abs(y) + ey) + ey


NORM_SHAPES = [(1, 1, 0, 0), (2, 7, 0, 0), (3, 32, 0, 0), (1, 768, 0, 0), (9, 129, 0, 0), (5, 1280, 0, 0), (33, 1280, 8, 0),
               (4, 1283, 3, 1), (3, 4104, 0, 8), (7, 4104, 1, 0), (2, 12288, 0, 0), (2, 12289, 0, 0), (2, 16392, 0, 0), (1, 70000, 0, 0),
               (700, 64, 0, 0), (2000, 40, 0, 0)]


@pytest.mark.parametrize("rows,cols,pad,offset", NORM_SHAPES)
@pytest.mark.parametrize("xdt,ydt,pdt", [(BF, BF, BF), (F32, BF, BF), (F32, F32, F32), (BF, F32, F32)])
def test_layer_norm_forward(handle, rows, cols, pad, offset, xdt, ydt, pdt):
    x = Guarded(rows, cols, xdt, pad, offset, _normal(cols, (rows, cols), 2.0, xdt, 0.7)).t
    gamma, beta = _normal(1, cols, 0.3, pdt, 1.0), _normal(2, cols, 0.3, pdt)
    y = Guarded(rows, cols, ydt, pad, offset)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    k = B.Act8(rows, cols)
    handle.layer_norm_forward(x, gamma, beta, 1e-5, y.t, mean, rstd, ckpt=k)
    y.check()
    X, G, Bt = np64(x), np64(gamma), np64(beta)
    Y, M, R = O.layer_norm(X, G, Bt, 1e-5)
    em, er, ey = _norm_bounds(X, G, Bt, Y, M, R, ydt)
    inside(mean, M, em + 1e-30, "mean")
    inside(rstd, R, er, "rstd")
    inside(y.t, Y, ey, "y")
    if rows * cols <= 40000:
        _same_pack(x, k)
    first = y.t.clone()
    handle.layer_norm_forward(x, gamma, beta, 1e-5, y.t, mean, rstd)
    assert torch.equal(first, y.t)


def test_layer_norm_constant_rows_and_not_finite_rows(handle):
    x = torch.full((4, 96), 3.0, device="cuda")
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3] = torch.arange(96, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    gamma, beta = torch.ones(96, device="cuda"), torch.full((96,), 0.25, device="cuda")
    handle.layer_norm_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    assert bool((y[0] == 0.25).all())           # a constant row: beta
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[2]).all())
    assert bool(torch.isfinite(y[3]).all())


def _norm_grad_case(handle, rows, cols, pad, offset, xdt, ydt, pdt, gdt, ckpt, add, accumulate):
    x = Guarded(rows, cols, xdt, pad, offset, _normal(cols, (rows, cols), 2.0, xdt, 0.7)).t
    dy = Guarded(rows, cols, ydt, pad, offset, _normal(cols + 1, (rows, cols), 0.5, ydt)).t
    gamma = _normal(3, cols, 0.3, pdt, 1.0)
    X = np64(x)
    M = X.mean(1)
    R = 1 / np.sqrt(X.var(1) + 1e-5)
    mean, rstd = torch.from_numpy(M).float().cuda(), torch.from_numpy(R).float().cuda()
    M, R = np64(mean), np64(rstd)
    source = x
    if ckpt:
        source = B.Act8(rows, cols)
        handle.act8_pack(x, source)
        X = O.act8_unpack(source.q.cpu().numpy(), source.exps.cpu().numpy(), cols)
    dx = Guarded(rows, cols, xdt, pad, offset)
    extra = None
    if add == "other":
        extra = Guarded(rows, cols, BF, pad, offset, _normal(5, (rows, cols), 0.5, BF)).t
    elif add == "same":
        dx.t.copy_(_normal(5, (rows, cols), 0.5, xdt))
        extra = dx.t
    E = np64(extra) if extra is not None else None
    g0, b0 = _normal(8, cols, 1.0, gdt), _normal(9, cols, 1.0, gdt)
    dg = Guarded(1, cols, gdt, 0, 3, g0[None])
    db = Guarded(1, cols, gdt, 0, 1, b0[None])
    handle.layer_norm_backward(dy, source, gamma, mean, rstd, dx.t, dg.t[0], db.t[0], add=extra, accumulate=accumulate)
    for o in (dx, dg, db):
        o.check()
    DY, G = np64(dy), np64(gamma)
    DX, DG, DB = O.layer_norm_grad(DY, X, G, M, R, E)
    xh = np.abs((X - M[:, None]) * R[:, None])
    exh = 4 * U32 * (np.abs(X) + np.abs(M)[:, None]) * R[:, None]
    gm = np.abs(DY * G)
    row = (cols / 1024 + 128) * U32
    c1, c2 = gm.mean(1)[:, None], (gm * xh).mean(1)[:, None]
    e1 = row * c1
    e2 = row * c2 + (gm * exh).mean(1)[:, None]
    edx = R[:, None] * (4 * U32 * (gm + c1 + xh * c2) + e1 + xh * e2 + exh * c2) + 2 * U32 * np.abs(DX)
    inside(dx.t, DX, U[xdt] * (np.abs(DX) + edx) + edx, "dx")
    more = (rows + 64) * U32
    edg = more * (np.abs(DY) * xh).sum(0) + (np.abs(DY) * exh).sum(0)
    edb = more * np.abs(DY).sum(0)
    if accumulate:
        DG, DB = DG + np64(g0), DB + np64(b0)
    inside(dg.t[0], DG, U[gdt] * (np.abs(DG) + edg) + edg + 2 * U32 * np.abs(DG) + 1e-30, "dgamma")
    inside(db.t[0], DB, U[gdt] * (np.abs(DB) + edb) + edb + 2 * U32 * np.abs(DB) + 1e-30, "dbeta")


@pytest.mark.parametrize("rows,cols,pad,offset", NORM_SHAPES)
@pytest.mark.parametrize("ckpt,add", [(False, None), (True, "other"), (False, "same")])
@pytest.mark.parametrize("xdt,ydt,pdt,gdt", [(BF, BF, BF, F32), (F32, BF, F32, BF), (F32, F32, F32, F32)])
def test_layer_norm_backward(handle, rows, cols, pad, offset, xdt, ydt, pdt, gdt, ckpt, add):
    _norm_grad_case(handle, rows, cols, pad, offset, xdt, ydt, pdt, gdt, ckpt, add, accumulate=add == "other")


def test_layer_norm_zero_rows(handle):
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    s = torch.empty(0, device="cuda")
    gamma = torch.ones(64, dtype=BF, device="cuda")
    handle.layer_norm_forward(e, gamma, gamma, 1e-5, e, s, s)
    dg, db = torch.full((64,), 5.0, device="cuda"), torch.full((64,), 6.0, device="cuda")
    handle.layer_norm_backward(e, e, gamma, s, s, e, dg, db, accumulate=True)
    assert bool((dg == 5).all()) and bool((db == 6).all())
    handle.layer_norm_backward(e, e, gamma, s, s, e, dg, db)
    assert not bool(dg.any()) and not bool(db.any())


# ---- linear layer ------------------------------------------------------------------

def _weight(seed, I, O_, layout, pad=0, offset=0):
    w = _normal(seed, (I, O_), I ** -0.5, BF)
    stored = w if layout == "in_out" else w.t()
    return Guarded(*stored.shape, BF, pad, offset, stored).t, np64(w)


def _keeps(z, ez, k):
    """A checkpoint of z, known to ez, holds it to half a step (a whole one at the top of a group)."""
    v = O.act8_unpack(k.q.cpu().numpy(), k.exps.cpu().numpy(), z.shape[1])
    cols = z.shape[1]
    E = k.exps.cpu().numpy().astype(int) - 127
    rep = lambda a: a.repeat(32, axis=1)[:, :cols]  # noqa: E731
    step = rep(np.exp2(E - 6.0))
    assert np.all(np.abs(v - z) <= np.where(np.abs(z) + ez >= 127 * step, step, step / 2) + ez)
    more = -cols % 32
    fold = lambda a: np.pad(a, ((0, 0), (0, more))).reshape(a.shape[0], -1, 32).max(2)  # noqa: E731
    top, et = fold(np.abs(z)), fold(ez)
    assert np.all((np.exp2(E) <= top + et) | (E == -120)) and np.all(top - et < np.exp2(E + 1.0))


LIN_SHAPES = [(1, 1, 1), (1, 64, 128), (2, 40, 129), (7, 129, 40), (17, 256, 264), (33, 72, 256), (64, 640, 72), (128, 128, 128),
              (129, 264, 130), (200, 513, 384), (300, 64, 520), (5, 1283, 700), (1, 1280, 640)]


@pytest.mark.parametrize("T,I,O_", LIN_SHAPES)
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("act,res,keep,odt", [("none", None, None, BF), ("gelu_tanh", None, "act8", BF),
                                              ("gelu_erf", "bf16", "bf16", F32), ("relu", "same", "f32", F32)])
def test_linear_forward(handle, T, I, O_, layout, act, res, keep, odt):
    pad, offset = (0, 0) if (T + I) % 2 else (3, 1)
    x = Guarded(T, I, BF, pad, offset, _normal(T, (T, I), 1.0, BF)).t
    w, W = _weight(I, I, O_, layout, pad, offset)
    bias = None if act == "none" else _normal(4, O_, 0.5, BF if res else F32)
    y = Guarded(T, O_, odt, pad, offset)
    residual = None
    if res == "bf16":
        residual = _normal(6, (T, O_), 1.0, BF)
    elif res == "same":
        y.t.copy_(_normal(6, (T, O_), 1.0, odt))
        residual = y.t
    RES = np64(residual) if residual is not None else None
    pre = None if keep is None else B.Act8(T, O_) if keep == "act8" else Guarded(T, O_, BF if keep == "bf16" else F32, pad, offset)
    handle.linear_forward(x, w, y.t, bias=bias, activation=act, residual=residual,
                          preact=pre.t if isinstance(pre, Guarded) else pre, weight_layout=layout)
    y.check()
    X = np64(x)
    Y, Z = O.linear(X, W, None if bias is None else np64(bias), act, RES)
    ez = product_bound(X, W, I) + 2 * U32 * np.abs(Z)
    ey = act_bound(Z, ez, act) + 2 * U32 * (np.abs(Y) + (0 if RES is None else np.abs(RES)))
    inside(y.t, Y, U[odt] * (np.abs(Y) + ey) + ey, "y")
    if keep == "act8":
        _keeps(Z, ez, pre)
    elif keep:
        pre.check()
        inside(pre.t, Z, U[pre.t.dtype] * (np.abs(Z) + ez) + ez, "z")


@pytest.mark.parametrize("T,I,O_", LIN_SHAPES)
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("act,keep,add,odt", [("none", None, None, BF), ("gelu_tanh", "act8", None, BF),
                                              ("gelu_erf", "f32", "other", F32), ("relu", "bf16", "same", BF)])
def test_linear_grad_input(handle, T, I, O_, layout, act, keep, add, odt):
    pad, offset = (0, 0) if (T + I) % 2 else (3, 1)
    dy = Guarded(T, O_, BF, pad, offset, _normal(T, (T, O_), 1.0, BF)).t
    w, W = _weight(I, I, O_, layout, pad, offset)
    z = None
    if keep:
        z = Guarded(T, I, F32 if keep == "f32" else BF, pad, offset, _normal(11, (T, I), 1.5)).t
    Z = np64(z) if keep else None
    if keep == "act8":
        k = B.Act8(T, I)
        handle.act8_pack(z, k)
        z, Z = k, O.act8_unpack(k.q.cpu().numpy(), k.exps.cpu().numpy(), I)
    dx = Guarded(T, I, odt, pad, offset)
    extra = None
    if add == "other":
        extra = _normal(6, (T, I), 1.0, BF)
    elif add == "same":
        dx.t.copy_(_normal(6, (T, I), 1.0, odt))
        extra = dx.t
    E = np64(extra) if extra is not None else None
    handle.linear_grad_input(dy, w, dx.t, activation=act, preact=z, add=extra, weight_layout=layout)
    dx.check()
    DY = np64(dy)
    DX = O.linear_grad_input(DY, W, act, Z, E)
    ep = product_bound(DY, W.T, O_)
    P = np.abs(DY @ W.T)
    ed = 1.13 * ep + (P + ep) * slope_bound(act) + 2 * U32 * (np.abs(DX) + (0 if E is None else np.abs(E)))
    inside(dx.t, DX, U[odt] * (np.abs(DX) + ed) + ed, "dx")


@pytest.mark.parametrize("T,I,O_", LIN_SHAPES)
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("x8,gdt,bias,accumulate", [(False, F32, True, False), (True, BF, True, True), (True, F32, False, True)])
def test_linear_grad_weight(handle, T, I, O_, layout, x8, gdt, bias, accumulate):
    pad, offset = (0, 0) if (T + I) % 2 else (3, 1)
    x = Guarded(T, I, BF, pad, offset, _normal(T, (T, I), 1.0, BF)).t
    dy = Guarded(T, O_, BF, pad, offset, _normal(T + 1, (T, O_), 1.0, BF)).t
    X, DY = np64(x), np64(dy)
    if x8:
        k = B.Act8(T, I)
        handle.act8_pack(x, k)
        x, X = k, O.act8_unpack(k.q.cpu().numpy(), k.exps.cpu().numpy(), I)
    shape = (I, O_) if layout == "in_out" else (O_, I)
    old = _normal(12, shape, 1.0, gdt)
    dw = Guarded(*shape, gdt, 0, 3, old)
    oldb = _normal(13, (1, O_), 1.0, gdt)
    db = Guarded(1, O_, gdt, 0, 1, oldb)
    handle.linear_grad_weight(x, dy, dw.t, dbias=db.t[0] if bias else None, weight_layout=layout, accumulate=accumulate)
    dw.check()
    db.check()
    DW, DB = O.linear_grad_weight(X, DY)
    ew = product_bound(X.T, DY, T)
    eb = (T + 64) * U32 * np.abs(DY).sum(0)
    if layout == "out_in":
        DW, ew = DW.T, ew.T
    if accumulate:
        DW, DB = DW + np64(old), DB + np64(oldb)[0]
    ew, eb = ew + 2 * U32 * np.abs(DW), eb + 2 * U32 * np.abs(DB)
    inside(dw.t, DW, U[gdt] * (np.abs(DW) + ew) + ew, "dw")
    if bias:
        inside(db.t[0], DB, U[gdt] * (np.abs(DB) + eb) + eb, "db")
    else:
        assert torch.equal(db.t, oldb)


def test_linear_zero_tokens(handle):
    x, dy, w = (torch.empty(s, dtype=BF, device="cuda") for s in ((0, 64), (0, 72), (64, 72)))
    handle.linear_forward(x, w, dy)
    handle.linear_grad_input(dy, w, x)
    dw, db = torch.full((64, 72), 2.0, device="cuda"), torch.full((72,), 3.0, device="cuda")
    handle.linear_grad_weight(x, dy, dw, dbias=db, accumulate=True)
    assert bool((dw == 2).all()) and bool((db == 3).all())
    handle.linear_grad_weight(x, dy, dw, dbias=db)
    assert not bool(dw.any()) and not bool(db.any())


def test_linear_not_finite_inputs_stay_in_their_rows(handle):
    T, I, O_ = 130, 72, 136
    x = _normal(1, (T, I), 1.0, BF)
    x[3, 5], x[129, 0] = float("inf"), float("nan")
    w = _normal(2, (I, O_), 0.2, BF)
    y = torch.empty((T, O_), dtype=BF, device="cuda")
    handle.linear_forward(x, w, y, activation="relu")
    rows = ~torch.isfinite(y).all(dim=1)
    assert rows.nonzero().flatten().tolist() == [3, 129]
    assert bool(torch.isnan(y[129]).all())


# ---- what a caller relies on ---------------------------------------------------------

def _chain(c, x, w, b, gamma, beta, dy, stream=None):
    T, I = x.shape
    O_ = w.shape[1]
    n, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    k, kz = B.Act8(T, I), B.Act8(T, O_)
    y, dw, db = torch.empty((T, O_), dtype=BF, device="cuda"), torch.empty_like(w, dtype=F32), torch.empty(O_, device="cuda")
    dn, dx = torch.empty_like(x), torch.empty_like(x)
    dg, dbt = torch.empty(I, device="cuda"), torch.empty(I, device="cuda")

    def go():
        c.layer_norm_forward(x, gamma, beta, 1e-5, n, mean, rstd, ckpt=k, stream=stream)
        c.linear_forward(n, w, y, bias=b, activation="gelu_tanh", preact=kz, stream=stream)
        c.linear_grad_weight(n, dy, dw, dbias=db, stream=stream)
        c.linear_grad_input(dy, w, dn, stream=stream)
        c.layer_norm_backward(dn, k, gamma, mean, rstd, dx, dg, dbt, add=x, stream=stream)

    return go, (n, mean, rstd, k.q, k.exps, kz.q, kz.exps, y, dw, db, dn, dx, dg, dbt)


def _chain_inputs():
    T, I, O_ = 300, 256, 520
    return (_normal(1, (T, I), 1.0, BF), _normal(2, (I, O_), 0.06, BF), _normal(3, O_, 0.1, BF), _normal(4, I, 0.1, BF, 1.0),
            _normal(5, I, 0.1, BF), _normal(6, (T, O_), 0.1, BF))


def test_same_bits_on_another_stream_and_from_a_graph():
    args = _chain_inputs()
    ws = max(B.fsdp_linear_workspace_bytes(300, 256, 520), B.fsdp_layer_norm_workspace_bytes(300, 256))
    c = B.Compute(ws, allocator=B.TorchAllocator())
    go, outs = _chain(c, *args)
    go()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    go2, outs2 = _chain(c, *args, stream=side)
    side.wait_stream(torch.cuda.current_stream())
    go2()
    side.synchronize()
    for a, b in zip(want, outs2):
        assert torch.equal(a, b)
    for o in outs2:
        o.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        go2()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs2):
        assert torch.equal(a, b)
    assert c.status() == 0
    c.close()


def _code(f):
    with pytest.raises(B.FsdpError) as e:
        f()
    return e.value.code


def test_refusals_change_nothing(handle):
    x = _normal(1, (4, 64), 1.0, BF)
    y = torch.full((4, 64), 9.0, dtype=BF, device="cuda")
    s, g = torch.full((4,), 9.0, device="cuda"), torch.ones(64, device="cuda")
    w = _normal(2, (64, 64), 0.1, BF)
    dw = torch.full((64, 64), 9.0, device="cuda")
    bad = B.FSDP_E_INVALID_ARG
    ln = lambda **k: B.fsdp_layer_norm_forward(handle.handle, *[k.get(n, d) for n, d in (("x", x), ("gamma", g), ("beta", g), ("eps", 1e-5), ("y", y), ("mean", s), ("rstd", s))], ckpt=k.get("ckpt"))  # noqa: E731
    assert _code(lambda: ln(eps=-1.0)) == bad
    assert _code(lambda: ln(eps=float("nan"))) == bad
    assert _code(lambda: ln(y=y[:3])) == bad
    assert _code(lambda: ln(ckpt=B.Act8(4, 65))) == bad
    assert _code(lambda: ln(ckpt=x)) == bad
    assert _code(lambda: handle.linear_forward(x.float(), w, y)) == bad
    assert _code(lambda: handle.linear_forward(x, w.float(), y)) == bad
    assert _code(lambda: handle.linear_forward(x, w[:, :63], y)) == bad
    assert _code(lambda: handle.linear_forward(x, w, y, activation=9)) == bad
    assert _code(lambda: handle.linear_forward(x, w, y, weight_layout=2)) == bad
    assert _code(lambda: handle.linear_forward(x, w, y, residual=y[:2])) == bad
    assert _code(lambda: handle.linear_grad_input(x, w, y, activation="relu")) == bad
    assert _code(lambda: handle.linear_grad_weight(x, y[:3], dw)) == bad
    assert _code(lambda: handle.linear_grad_weight(x.float(), y, dw)) == bad
    assert _code(lambda: handle.act8_pack(x, B.Act8(4, 32))) == bad
    assert _code(lambda: handle.act8_unpack(x, y)) == bad
    assert _code(lambda: handle.set_wait_limit(0.0)) == bad
    small = B.Compute(0)
    assert _code(lambda: small.linear_grad_weight(x, y, dw, dbias=g)) == B.FSDP_E_CAPACITY
    assert "bytes of workspace" in B.fsdp_last_error()
    assert _code(lambda: small.layer_norm_backward(x, x, g, s, s, y, g, g)) == B.FSDP_E_CAPACITY
    small.close()
    # raw views: null data, short ld, misaligned data, an ACT8 ld that is not the format's
    lib, ok = B.lib(), B._mat(x)

    def m(t, **changes):
        v = B.Matrix.from_buffer_copy(B._mat(t))
        for field, value in changes.items():
            setattr(v, field, value)
        return bytes(v)

    out = m(y)
    call = lambda a, b: lib.fsdp_act8_unpack(handle.handle, a, 0, b, None)  # noqa: E731
    k = B.Act8(4, 64)
    assert call(m(k, data=None), out) == bad and call(m(k, exps=None), out) == bad
    assert call(m(k, ld=128), out) == bad and call(m(k, data=k.q.data_ptr() + 8), out) == B.FSDP_E_ALIGN
    assert call(m(k), m(y, ld=63)) == bad and call(m(k), m(y, data=y.data_ptr() + 1)) == B.FSDP_E_ALIGN
    assert call(m(k, cols=0, ld=0), m(y, cols=0)) == bad and call(m(k, rows=-1), m(y, rows=-1)) == bad
    assert lib.fsdp_act8_unpack(None, m(k), 0, out, None) == bad and lib.fsdp_act8_unpack(handle.handle, None, 0, out, None) == bad
    assert lib.fsdp_linear_forward(handle.handle, ok, B._mat(w), 0, None, 0, 0, None, None, None, None) == bad
    torch.cuda.synchronize()
    assert bool((y == 9).all()) and bool((s == 9).all()) and bool((dw == 9).all()) and bool((g == 1).all())


def test_a_copy_that_never_arrives_is_reported():
    """The give-up path: the first stage's copies are withheld, the waits behind
    them run out, and the handle works again after its status has been read."""
    c = B.Compute(B.fsdp_linear_workspace_bytes(512, 256, 512))
    x, w = _normal(1, (512, 256), 1.0, BF), _normal(2, (256, 512), 0.1, BF)
    y, again = (torch.empty((512, 512), dtype=BF, device="cuda") for _ in range(2))
    c.linear_forward(x, w, y)
    assert c.status() == 0
    c.set_wait_limit(0.02, withhold_next=1)
    c.linear_forward(x, w, again)
    assert c.status() == B.FSDP_KSTATUS_WAIT_TIMEOUT
    assert c.status() == 0
    c.set_wait_limit()
    c.linear_forward(x, w, again)
    assert c.status() == 0 and torch.equal(y, again)
    c.close()


@pytest.mark.parametrize("rows,cols", [(1300, 520), (700, 4104), (1400, 1280), (5000, 768), (1300, 2880), (1300, 4096), (1000, 5000),
                                       (700, 6000), (700, 8192), (320, 16384), (320, 20480), (160, 20488)])
def test_layer_norm_many_rows(handle, rows, cols):
    """Enough rows for a block to walk several of them."""
    x = _normal(cols, (rows, cols), 2.0, BF, 0.7)
    gamma, beta = _normal(1, cols, 0.3, BF, 1.0), _normal(2, cols, 0.3, BF)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    k = B.Act8(rows, cols)
    handle.layer_norm_forward(x, gamma, beta, 1e-5, y, mean, rstd, ckpt=k)
    X, G, Bt = np64(x), np64(gamma), np64(beta)
    Y, M, R = O.layer_norm(X, G, Bt, 1e-5)
    em, er, ey = _norm_bounds(X, G, Bt, Y, M, R, BF)
    inside(mean, M, em, "mean")
    inside(rstd, R, er, "rstd")
    inside(y, Y, ey, "y")
    other = B.Act8(rows, cols)
    handle.act8_pack(x, other)
    assert torch.equal(k.q, other.q) and torch.equal(k.exps, other.exps)
    for ckpt, add in ((False, "other"), (True, None)):
        _norm_grad_case(handle, rows, cols, 0, 0, BF, BF, BF, F32, ckpt, add, False)


@pytest.mark.parametrize("rows,cols,pad,offset", [(1000, 31, 3, 1), (1000, 257, 0, 0), (700, 1283, 3, 1), (400, 2050, 2, 6), (320, 4099, 0, 0),
                                                  (320, 6151, 1, 0), (160, 12287, 3, 5), (40, 16383, 2, 1), (700, 1280, 3, 0)])
def test_layer_norm_many_rows_anywhere(handle, rows, cols, pad, offset):
    for xdt, ydt, pdt in ((BF, BF, BF), (F32, BF, F32)):
        test_layer_norm_forward(handle, rows, cols, pad, offset, xdt, ydt, pdt)
    for (xdt, ydt, pdt), ckpt, add in (((BF, BF, BF), False, "same"), ((BF, BF, F32), True, "other"), ((F32, F32, BF), False, "other")):
        _norm_grad_case(handle, rows, cols, pad, offset, xdt, ydt, pdt, F32, ckpt, add, False)


@pytest.mark.parametrize("T,I,O_,kind", [(300, 16384, 512, "fwd"), (20000, 264, 512, "dw"), (300, 40000, 8192, "fwd")])
def test_long_fp32_sums_do_not_drift(handle, T, I, O_, kind):
    """All products positive, so that an accumulator which cuts off instead of
    rounding errs the same way in every step.  A slice of 768 products is 48
    steps, each off by at most a unit of 2^-23 of the sum; the slices' own
    additions round to nearest."""
    c = B.Compute(B.fsdp_linear_workspace_bytes(T, I, O_))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    x = torch.rand((T, I), device="cuda", generator=gen).to(BF)
    if kind == "fwd":
        w = torch.rand((I, O_), device="cuda", generator=gen).to(BF)
        got, want, k = torch.empty((T, O_), device="cuda"), x.double() @ w.double(), I
        c.linear_forward(x, w, got)
    else:
        dy = torch.rand((T, O_), device="cuda", generator=gen).to(BF)
        got, want, k = torch.empty((I, O_), device="cuda"), x.double().t() @ dy.double(), T
        c.linear_grad_weight(x, dy, got)
    assert c.status() == 0
    off = ((got.double() - want).abs() / want).max().item()
    assert off <= 48 * 2.0 ** -23 + (k / 768 + 20) * 2.0 ** -24, off
    c.close()
