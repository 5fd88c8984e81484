"""The residual norm, forward and backward, against the definitions in 64 bits.

Bounds.  Sums of n squares or products in fp32, whatever their order, are off by (n / 32 + 40) 2^-24 of
the sum of magnitudes where a thread adds at most n / 32 + 8 of them (a warp has a row at least) and the rest
goes by trees; U is the rounding of an output's type."""
import numpy as np
import pytest
import torch

from block_harness import U, Guarded, inside, np64
from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


def _compute(rows, cols):
    return B.Compute(B.fsdp_residual_norm_workspace_bytes(rows, cols))


def _inputs(rows, cols, dtype, params, post, gate, pad, seed=0, mixed=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def mat(std=1.0, dt=dtype):
        return Guarded(rows, cols, dt, pad, offset=pad % 3, like=torch.empty((rows, cols), device="cuda").normal_(0, std, generator=g))

    def vec(mean):
        return torch.empty(cols, device="cuda").normal_(mean, 0.2, generator=g).to(params)

    other = {BF: F32, F32: BF}[dtype] if mixed else dtype
    return dict(h=mat(), o=mat(0.7, other), post=vec(1.0) if post else None, gate=vec(0.5) if gate else None, gamma=vec(1.0), dy=mat(1.0, other), dout=mat(0.5))


def _forward64(h, o, post, gate, gamma, alpha):
    h = np64(h)
    r2 = None
    b = np.zeros_like(h)
    if o is not None:
        b = np64(o)
        if post is not None:
            r2 = 1 / np.sqrt((b * b).mean(axis=1) + EPS)
            b = b * r2[:, None] * np64(post)
        if gate is not None:
            b = b * np64(gate)
    s = alpha * h + b
    r1 = 1 / np.sqrt((s * s).mean(axis=1) + EPS)
    y = None if gamma is None else s * r1[:, None] * np64(gamma)
    return s, y, r1, r2, b


def _tree(n):
    return (n / 32 + 48) * 2.0 ** -24


def _check(rows, cols, dtype, params, post, gate, pad, out=None, mixed=False, has_block=True, has_gamma=True, alpha=0.75):
    out = out or dtype
    i = _inputs(rows, cols, dtype, params, post, gate, pad, mixed=mixed)
    c = _compute(rows, cols)
    h, o = i["h"].t, i["o"].t if has_block else None
    gamma = i["gamma"] if has_gamma else None
    s, y = Guarded(rows, cols, out, pad, offset=pad % 3), Guarded(rows, cols, out, pad + 1, offset=1) if has_gamma else None
    rstd, post_rstd = torch.empty(rows, device="cuda") if has_gamma else None, torch.empty(rows, device="cuda") if post else None
    c.residual_norm_forward(h, s.t, block=o, post_gamma=i["post"], gate=i["gate"], residual_scale=alpha, y=y.t if y else None, gamma=gamma, eps=EPS,
                            rstd=rstd, post_rstd=post_rstd)
    ws, wy, r1, r2, b = _forward64(h, o, i["post"], i["gate"], gamma, alpha)
    e = _tree(cols)
    size = np.abs(alpha * np64(h)) + np.abs(b)
    near = size * 2.0 ** -22 + np.abs(b) * e
    inside(s.t, ws, near + U[out] * np.abs(ws), "out")
    if post:
        inside(post_rstd, r2, r2 * e, "post_rstd")
    if has_gamma:
        err = e + 2.0 ** -22 + (near * np.abs(ws)).mean(axis=1) * r1 ** 2     # of rstd, relative
        inside(rstd, r1, r1 * err, "rstd")
        w = np.abs(np64(gamma)) * r1[:, None]
        inside(y.t, wy, w * near + np.abs(wy) * (err[:, None] + 2.0 ** -22 + U[out]), "y")
    for m in (s, y, i["h"], i["o"]):
        if m is not None:
            m.check()
    return i, c, s, rstd, post_rstd


def _check_backward(i, c, s, rstd, post_rstd, params, grads, out, pad, alpha=0.75, has_block=True, has_gamma=True, has_dout=True, accumulate=False):
    rows, cols = s.t.shape
    dy, dout = i["dy"].t if has_gamma else None, i["dout"].t if has_dout else None
    o = i["o"].t if has_block else None
    post, gate, gamma = i["post"], i["gate"], i["gamma"] if has_gamma else None
    dh, db = Guarded(rows, cols, out, pad + 3, offset=1), Guarded(rows, cols, out, pad, offset=pad % 3) if has_block else None
    vec = {k: Guarded(1, cols, grads, offset=n) if v is not None else None for n, (k, v) in enumerate((("gamma", gamma), ("post", post), ("gate", gate)))}
    old = {}
    for k, v in vec.items():
        if v is not None:
            v.t.copy_(torch.arange(cols, device="cuda") % 5 - 2.0)
            old[k] = np64(v.t[0]) if accumulate else 0.0
    at = lambda k: vec[k].t[0] if vec[k] is not None else None  # noqa: E731
    c.residual_norm_backward(dy, dout, s.t if has_gamma else None, o, dh.t, db.t if db else None, gamma=gamma, rstd=rstd, dgamma=at("gamma"),
                             post_gamma=post, post_rstd=post_rstd, dpost_gamma=at("post"), gate=gate, dgate=at("gate"), residual_scale=alpha, accumulate=accumulate)
    n = cols
    e = _tree(n)
    t = np64(dout) if dout is not None else np.zeros((rows, cols))
    et = np.abs(t) * 2.0 ** -23
    if has_gamma:
        r1 = np64(rstd)[:, None]
        xh, g = np64(s.t) * r1, np64(dy) * np64(gamma)
        c1 = (g * xh).mean(axis=1, keepdims=True)
        ec1 = np.abs(g * xh).mean(axis=1, keepdims=True) * (e + 2.0 ** -21)
        t = t + r1 * (g - xh * c1)
        et = et + r1 * (np.abs(g) + np.abs(xh * c1)) * 2.0 ** -21 + r1 * np.abs(xh) * ec1 + np.abs(t) * 2.0 ** -23
    inside(dh.t, alpha * t, alpha * et + U[out] * np.abs(alpha * t), "dresidual")
    dh.check()
    if has_gamma:
        want = (np64(dy) * xh).sum(axis=0) + old["gamma"]
        size = np.abs(np64(dy) * xh).sum(axis=0) + np.abs(old["gamma"])
        inside(at("gamma"), want, size * (rows + 8) * 2.0 ** -23 + U[grads] * np.abs(want), "dgamma")
    if has_block:
        r2 = np64(post_rstd)[:, None] if post is not None else 1.0
        u = np64(o) * r2
        k = (np64(post) if post is not None else 1.0) * (np64(gate) if gate is not None else 1.0)
        ee = t * k
        want, tol = ee, np.abs(k) * et + np.abs(ee) * 2.0 ** -22
        if post is not None:
            c2 = (ee * u).mean(axis=1, keepdims=True)
            # the sum goes as (dout + rstd g) k u less rstd c1 xh k u
            parts = np.abs(k * u) * (np.abs(np64(dout)) if dout is not None else 0.0)
            if has_gamma:
                parts = parts + np.abs(k * u) * r1 * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(axis=1, keepdims=True))
            ec2 = parts.mean(axis=1, keepdims=True) * (2 * e + 2.0 ** -19)
            want = r2 * (ee - u * c2)
            tol = r2 * (tol + np.abs(u) * ec2 + np.abs(u * c2) * 2.0 ** -21)
        inside(db.t, want, tol + U[out] * np.abs(want), "dblock")
        db.check()
        both, size = (t * u).sum(axis=0), (np.abs(t * u) * (rows + 16) * 2.0 ** -23 + et * np.abs(u)).sum(axis=0)
        for name, by in (("post", gate), ("gate", post)):
            if vec[name] is not None:
                f = np64(by) if by is not None else 1.0
                want = both * f + old[name]
                inside(at(name), want, size * np.abs(f) + (2.0 ** -22 + U[grads]) * (np.abs(want) + np.abs(both * f)), "d" + name)
    for v in vec.values():
        if v is not None:
            v.check()


SIZES = [(1, 1), (3, 7), (2, 8), (5, 40), (33, 72), (700, 128), (1, 1280), (9, 1283), (340, 1280), (6, 2560), (3, 5121), (320, 4096), (160, 12288), (2, 12288), (3, 12296), (2, 20488),
         (2, 33001), (2, 49992), (3, 70001)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,params,post,gate,pad", [(BF, BF, True, True, 0), (BF, BF, True, False, 8), (BF, F32, False, True, 0), (F32, F32, True, True, 0),
                                                        (BF, BF, True, True, 3), (F32, BF, False, False, 1)])
def test_both_directions(rows, cols, dtype, params, post, gate, pad):
    i, c, s, rstd, post_rstd = _check(rows, cols, dtype, params, post, gate, pad)
    _check_backward(i, c, s, rstd, post_rstd, params, F32, dtype, pad)
    c.close()


@pytest.mark.parametrize("rows,cols", [(5, 40), (13, 1283), (400, 1280), (170, 12288)])
@pytest.mark.parametrize("kw", [dict(has_block=False), dict(has_gamma=False), dict(mixed=True), dict(out=F32), dict(out=BF)])
def test_options(rows, cols, kw):
    for dtype in (BF, F32):
        post = kw.get("has_block", True)
        i, c, s, rstd, post_rstd = _check(rows, cols, dtype, BF, post, post, 0, **kw)
        more = {k: v for k, v in kw.items() if k.startswith("has")}
        for has_dout in (True, False) if kw.get("has_gamma", True) else (True,):
            for grads, acc in ((F32, True), (BF, False), (BF, True)):
                _check_backward(i, c, s, rstd, post_rstd, BF, grads, kw.get("out", dtype), 0, has_dout=has_dout, accumulate=acc, **more)
        c.close()


def test_without_a_norm_after_the_block():
    for post, gate in ((False, False), (False, True), (True, False)):
        i, c, s, rstd, post_rstd = _check(300, 768, BF, BF, post, gate, 0)
        _check_backward(i, c, s, rstd, post_rstd, BF, F32, BF, 0)
        c.close()


def test_zero_rows_and_rows_of_zeros():
    c = _compute(4, 64)
    z, w = torch.zeros((4, 64), dtype=BF, device="cuda"), torch.ones(64, dtype=BF, device="cuda")
    s, y, r1, r2 = torch.empty_like(z), torch.empty_like(z), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    c.residual_norm_forward(z, s, block=z.clone(), post_gamma=w, gate=w, y=y, gamma=w, eps=EPS, rstd=r1, post_rstd=r2)
    assert not bool(s.any()) and not bool(y.any())
    assert torch.allclose(r1, torch.full_like(r1, EPS ** -0.5), rtol=1e-6) and torch.equal(r1, r2)
    none, e = z[:0], torch.empty(0, device="cuda")
    g = [torch.full((64,), 3.0, device="cuda") for _ in range(3)]
    c.residual_norm_forward(none, none, block=none, post_gamma=w, gate=w, y=none, gamma=w, rstd=e, post_rstd=e)
    kw = dict(gamma=w, rstd=e, dgamma=g[0], post_gamma=w, post_rstd=e, dpost_gamma=g[1], gate=w, dgate=g[2])
    c.residual_norm_backward(none, none, none, none, none, none, accumulate=True, **kw)
    assert all(bool((v == 3).all()) for v in g)
    c.residual_norm_backward(none, none, none, none, none, none, **kw)
    assert not any(bool(v.any()) for v in g)
    c.close()


def test_values_that_are_not_finite():
    """They stay in their rows, and in the columns' sums."""
    for cols in (128, 1283, 12288):
        i = _inputs(6, cols, BF, BF, True, True, 0)
        c = _compute(6, cols)
        i["h"].t[1, 5], i["o"].t[3, 7] = float("inf"), float("nan")
        s, y, r1, r2 = torch.empty_like(i["h"].t), torch.empty_like(i["h"].t), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
        c.residual_norm_forward(i["h"].t, s, block=i["o"].t, post_gamma=i["post"], gate=i["gate"], y=y, gamma=i["gamma"], eps=EPS, rstd=r1, post_rstd=r2)
        assert bool(torch.isfinite(y[[0, 2, 4, 5]].float()).all()) and bool(torch.isnan(y[3]).all())
        assert bool(torch.isnan(y[1, 5])) and not bool(y[1, :5].any()) and torch.isinf(s[1]).sum() == 1
        c.close()


def test_same_results_twice_on_another_stream_and_in_a_graph():
    rows, cols = 500, 1280
    i, c, s, rstd, post_rstd = _check(rows, cols, BF, BF, True, True, 0)
    dh, db = torch.empty((rows, cols), dtype=BF, device="cuda"), torch.empty((rows, cols), dtype=BF, device="cuda")
    g = [torch.empty(cols, device="cuda") for _ in range(3)]

    def back():
        c.residual_norm_backward(i["dy"].t, i["dout"].t, s.t, i["o"].t, dh, db, gamma=i["gamma"], rstd=rstd, dgamma=g[0], post_gamma=i["post"],
                                 post_rstd=post_rstd, dpost_gamma=g[1], gate=i["gate"], dgate=g[2], residual_scale=0.75)

    back()
    want = [v.clone() for v in (dh, db, *g)]
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for run in ("eager", "stream", "graph", "replay"):
        for v in (dh, db, *g):
            v.zero_()
        torch.cuda.synchronize()
        if run == "eager":
            back()
        elif run == "stream":
            with torch.cuda.stream(st):
                back()
        elif run == "graph":
            with torch.cuda.graph(graph):
                back()
            graph.replay()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dh, db, *g), want)), run
    c.close()


def test_gradient_against_differences():
    """L = sum(out q + y r) in F32, along random directions of all inputs.  The quotient errs by h^2/6 of
    the third derivative (at most about 10 of the sizes below) and by rounding, 2^-22 of the sizes over 2h."""
    rows, cols, step, alpha = 4, 64, 2.0 ** -6, 0.75
    rng = np.random.default_rng(0)
    t = lambda *s: torch.from_numpy(rng.normal(size=s)).float().cuda()  # noqa: E731
    args = [t(rows, cols), t(rows, cols), t(cols) * 0.2 + 1, t(cols) * 0.2 + 1, t(cols) * 0.2 + 1]   # h, o, post, gate, gamma
    q, r = t(rows, cols), t(rows, cols)
    c = _compute(rows, cols)
    s, y, r1, r2 = torch.empty_like(q), torch.empty_like(q), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")

    def loss(h, o, post, gate, gamma):
        c.residual_norm_forward(h, s, block=o, post_gamma=post, gate=gate, residual_scale=alpha, y=y, gamma=gamma, eps=0.1, rstd=r1, post_rstd=r2)
        return (s.double() * q.double() + y.double() * r.double()).sum().item()

    loss(*args)
    size = ((s.double() * q.double()).abs() + (y.double() * r.double()).abs()).sum().item()
    grads = [torch.empty_like(a) for a in args]
    c.residual_norm_backward(r, q, s, args[1], grads[0], grads[1], gamma=args[4], rstd=r1, dgamma=grads[4], post_gamma=args[2], post_rstd=r2,
                             dpost_gamma=grads[2], gate=args[3], dgate=grads[3], residual_scale=alpha)
    for n, grad in enumerate(grads):
        for _ in range(4):
            d = t(*grad.shape)
            up, down = (loss(*[a + sign * step * d if m == n else a for m, a in enumerate(args)]) for sign in (1, -1))
            want = (grad.double() * d.double()).sum().item()
            assert abs((up - down) / (2 * step) - want) <= step * step / 6 * 10 * size / rows + 2.0 ** -22 * size / step, n
    c.close()
