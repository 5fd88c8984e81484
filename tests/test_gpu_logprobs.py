"""Token log probabilities, their alternatives and the logits' gradient, against the
definitions in 64 bits.

Bounds.  With d2 = (z - max) scale log2 e, a term 2^d2 is off by 2^-22 (the exponential) and
2^-23 |d2| ln 2 (two roundings of its argument); weighted by the terms the second is below 2^-23 (H + ln S).
A row has 128 threads at least.  A thread adds n terms (2^-24 each) and rescales its sums at most once a
group of 16 or 32 and 21 times on the way to the block's (2^-22 each, and as much again for the distance moved).  `_eps` adds
these up; ln S is off by that and by its own roundings."""
import math

import numpy as np
import pytest
import torch

from block_harness import U, Guarded, inside, np64
from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = math.inf


@pytest.fixture(scope="module")
def c():
    from conftest import library
    library()
    h = B.Compute(0)
    yield h
    h.close()


def _logits(rows, vocab, dtype, seed=0, std=3.0, masked=0.1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.empty((rows, vocab), device="cuda").normal_(0, std, generator=g)
    if vocab > 4:
        z[torch.rand((rows, vocab), device="cuda", generator=g) < masked] = -INF
    z[:, 0] = 0.5
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    return z.to(dtype), t


def _reference(z, t, scale):
    """(log probabilities of all, p, entropy, ln S, max) in 64 bits; the header's rules for odd rows."""
    z = np64(z)
    top = z.max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        d = (z - np.where(top == -INF, 0.0, top)) * scale
        e = np.exp(d)
        s = e.sum(axis=1, keepdims=True)
        lp = d - np.log(s)
        p = e / s
        h = -np.where(p > 0, p * lp, 0.0).sum(axis=1)
        dead = (s == 0)[:, 0]
        bad = ~np.isfinite(s[:, 0])
    lp[dead], p[dead], h[dead] = -INF, 0.0, 0.0
    lp[bad], p[bad], h[bad] = np.nan, np.nan, np.nan
    t = t.cpu().numpy()
    given = np.where(t < 0, 0.0, np.take_along_axis(lp, np.clip(t, 0, z.shape[1] - 1)[:, None], 1)[:, 0])
    given = np.where(t >= z.shape[1], np.nan, given)
    ln_s = np.log(s[:, 0], where=s[:, 0] > 0, out=np.full(len(s), -INF))
    ln_s[bad] = np.nan
    return lp, p, h, ln_s, top[:, 0], given


def _eps(vocab, h, ln_s):
    n = -(-vocab // 128) + 8
    return 2.0 ** -22 * (1 + h + np.abs(ln_s) + 2 * (n / 16 + 22)) + 2.0 ** -24 * (n + 40)


def _close(got, want, tol, what):
    got = np64(got)
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True), what
    inside(np.where(odd, 0.0, got), np.where(odd, 0.0, want), np.where(np.isfinite(tol), tol, 0.0), what)


def _ranked(z, k):
    return torch.sort(z.double(), dim=1, descending=True, stable=True)[1][:, :k]


def _check_rows(ref, vocab, lp, st, h):
    """Log probabilities, stats and entropies against _reference's; which rows are finite."""
    _, _, wh, ln_s, m, given = ref
    eps = _eps(vocab, np.nan_to_num(wh), np.nan_to_num(ln_s, neginf=0.0))
    _close(h, wh, 2 * eps * (1 + np.abs(wh)), "entropy")
    with np.errstate(invalid="ignore"):
        tol = eps + 2.0 ** -22 * (np.abs(np.nan_to_num(given, neginf=0.0)) + np.abs(np.nan_to_num(ln_s, neginf=0.0)))
    _close(lp, given, tol, "logprob")
    good = np.isfinite(wh)
    assert np.array_equal(np64(st)[good, 0], m[good])
    _close(st[:, 1][torch.from_numpy(good).cuda()], ln_s[good], (eps + 2.0 ** -22 * np.abs(ln_s))[good], "ln S")
    return good, eps


def _check_forward(c, z, t, scale, top):
    rows, vocab = z.shape
    lp, st, h = torch.empty(rows, device="cuda"), torch.empty((rows, 2), device="cuda"), torch.empty(rows, device="cuda")
    tt, tl = (torch.empty((rows, top), dtype=torch.int64, device="cuda"), torch.empty((rows, top), device="cuda")) if top else (None, None)
    c.token_logprobs_forward(z, t, lp, entropy=h, stats=st, top_tokens=tt, top_logprobs=tl, scale=scale)
    ref = _reference(z, t, scale)
    want, ln_s = ref[0], ref[3]
    good, eps = _check_rows(ref, vocab, lp, st, h)
    if top:
        g = torch.from_numpy(good).cuda()
        assert torch.equal(tt[g], _ranked(z, top)[g])
        assert bool((tt[~g] == -1).all()) and bool(torch.isnan(tl[~g]).all())
        w = np.take_along_axis(want[good], tt[g].cpu().numpy(), 1)
        _close(tl[g], w, np.broadcast_to((eps + 2.0 ** -22 * np.abs(ln_s))[good][:, None], w.shape) + 2.0 ** -22 * np.abs(np.nan_to_num(w, neginf=0.0)), "top")
    return lp, st, h


def _wanted_grad(z, t, scale, a, b, h=None):
    lp, p, wh, ln_s, _, _ = _reference(z, t, scale)
    rows, vocab = lp.shape
    t = t.cpu().numpy()
    a = np.where(t < 0, 0.0, np.zeros(rows) if a is None else np64(a))
    b = np.zeros(rows) if b is None else np64(b)
    h = wh if h is None else np64(h)
    one = np.zeros_like(p)
    some = (t >= 0) & (t < vocab)
    one[np.nonzero(some)[0], t[some]] = 1.0
    with np.errstate(all="ignore"):
        l = np.where(p > 0, lp, 0.0)
        dz = scale * (a[:, None] * (one - p) - b[:, None] * p * (l + h[:, None]))
        eps = _eps(vocab, np.nan_to_num(wh), np.nan_to_num(ln_s, neginf=0.0))[:, None] + 2.0 ** -21 * (1 + np.abs(l))
        size = scale * (np.abs(a[:, None]) * (one + p) + np.abs(b[:, None]) * p * (np.abs(l) + h[:, None] + 1))
    dz[(a == 0) & (b == 0) | np.isneginf(ln_s)] = 0.0
    dz[(t >= vocab) & np.isfinite(a) & (a != 0)] = np.nan
    return dz, size * eps


CASES = [(1, 1, BF, 0, 1.0, 1), (3, 2, F32, 0, 1.0, 2), (5, 40, BF, 3, 0.7, 32), (2, 257, F32, 1, 1.5, 5), (7, 1283, BF, 0, 1.0, 20),
         (4, 4096, BF, 8, 1.0, 1), (3, 4099, F32, 0, 2.0, 32), (9, 50257, BF, 0, 1.0, 20), (3, 50257, F32, 47, 1.25, 7),
         (2, 70001, BF, 5, 0.25, 3), (1300, 4099, BF, 0, 1.0, 20), (600, 2053, F32, 3, 1.0, 32)]


@pytest.mark.parametrize("rows,vocab,dtype,pad,scale,top", CASES)
def test_forward(c, rows, vocab, dtype, pad, scale, top):
    z, t = _logits(rows, vocab, dtype)
    t[rows // 2:rows // 2 + (rows > 2)] = -1
    gz = Guarded(rows, vocab, dtype, pad, offset=pad % 3, like=z)
    _check_forward(c, gz.t, t, scale, min(top, vocab))
    _check_forward(c, gz.t, t, scale, 0)
    gz.check()
    assert c.status() == 0


@pytest.mark.parametrize("rows,vocab,dtype,pad,scale,top", CASES)
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient(c, rows, vocab, dtype, pad, scale, top, out, entropy):
    z, t = _logits(rows, vocab, dtype, seed=1)
    t[0] = -1
    gz = Guarded(rows, vocab, dtype, pad, offset=pad % 3, like=z)
    a, b = torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda") if entropy else None
    lp, st, h = _check_forward(c, gz.t, t, scale, 0)
    want, tol = _wanted_grad(z, t, scale, a, b)
    tol = tol + U[out] * np.abs(want)
    for pad_out in (pad, pad + 1):
        dz = Guarded(rows, vocab, out, pad_out, offset=pad_out % 5)
        c.token_logprobs_backward(gz.t, t, st, dz.t, dlogprob=a, entropy=h if entropy else None, dentropy=b, scale=scale)
        inside(dz.t, want, tol, "dlogits")
        dz.check()
        both = Guarded(rows, vocab, out, pad_out, offset=pad_out % 5)
        lp2, h2, st2 = torch.empty_like(lp), torch.empty_like(h), torch.empty_like(st)
        c.token_logprobs_loss(gz.t, t, lp2, both.t, dlogprob=a, dentropy=b, entropy=h2, stats=st2, scale=scale)
        _check_rows(_reference(z, t, scale), vocab, lp2, st2, h2)   # rows may be split otherwise than in the forward pass
        inside(both.t, want, tol, "dlogits in one call")
        both.check()
    if entropy:
        c.token_logprobs_backward(gz.t, None, st, dz.t, entropy=h, dentropy=b, scale=scale)
        want, tol = _wanted_grad(z, torch.full_like(t, -1), scale, None, b)
        inside(dz.t, want, tol + U[out] * np.abs(want), "the entropy's gradient alone")
    if out == dtype:   # in place
        got, lp2 = dz.t.clone(), torch.empty_like(lp)
        c.token_logprobs_backward(gz.t, t, st, got, dlogprob=a, entropy=h if entropy else None, dentropy=b, scale=scale)
        one = Guarded(rows, vocab, dtype, pad, offset=pad % 3, like=z)
        c.token_logprobs_backward(one.t, t, st, one.t, dlogprob=a, entropy=h if entropy else None, dentropy=b, scale=scale)
        assert torch.equal(one.t, got)
        one.check()
        one = Guarded(rows, vocab, dtype, pad, offset=pad % 3, like=z)
        c.token_logprobs_loss(one.t, t, lp2, one.t, dlogprob=a, dentropy=b, scale=scale)
        want, tol = _wanted_grad(z, t, scale, a, b)
        inside(one.t, want, tol + U[dtype] * np.abs(want), "in place")
        _check_rows(_reference(z, t, scale), vocab, lp2, st, h)
        one.check()
    gz.check()
    assert c.status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [5, 1283, 50257])
def test_odd_rows(c, dtype, vocab):
    """Masked rows, rows of the type's lowest and highest values, infinities, NaN, equal logits."""
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    z, _ = _logits(12, vocab, dtype, seed=2)
    z[0] = -INF
    z[1] = low
    z[2], z[2, 3] = low, 1.0
    z[3, vocab - 1] = INF
    z[4, vocab - 2] = math.nan
    z[5] = 0.0
    z[6] = -0.0
    z[6, 2::2] = 0.0
    z[7], z[7, vocab - 1] = -INF, high
    z[8], z[8, 1] = high, -INF
    z[9, vocab // 2] = 60.0
    t = torch.full((12,), vocab - 1, device="cuda")
    t[10], t[11] = -5, 0
    k = min(vocab, 32)
    lp, st, h = _check_forward(c, z, t, 1.0, k)
    for a, b in ((torch.ones(12, device="cuda"), None), (torch.ones(12, device="cuda"), torch.ones(12, device="cuda"))):
        dz = torch.empty_like(z)
        want, tol = _wanted_grad(z, t, 1.0, a, b)
        c.token_logprobs_loss(z, t, torch.empty_like(lp), dz, dlogprob=a, dentropy=b)
        inside(dz, want, np.nan_to_num(tol + U[dtype] * np.abs(want)), "loss")
        c.token_logprobs_backward(z, t, st, dz, dlogprob=a, entropy=h, dentropy=b)
        inside(dz, want, np.nan_to_num(tol + U[dtype] * np.abs(want)), "backward")
    a = torch.zeros(12, device="cuda")
    c.token_logprobs_backward(z, t, st, dz, dlogprob=a)
    assert bool((dz == 0).all())   # whatever the logits
    assert c.status() == 0


def test_a_token_outside_the_vocabulary(c):
    z, t = _logits(4, 100, BF)
    t[1], t[2] = 100, 2 ** 40
    lp, st, dz = torch.empty(4, device="cuda"), torch.empty((4, 2), device="cuda"), torch.empty_like(z)
    c.token_logprobs_forward(z, t, lp, stats=st)
    assert torch.isnan(lp).tolist() == [False, True, True, False]
    assert c.status() == B.FSDP_KSTATUS_BAD_TOKEN and c.status() == 0
    a = torch.ones(4, device="cuda")
    c.token_logprobs_backward(z, t, st, dz, dlogprob=a)
    assert torch.isnan(dz).all(dim=1).tolist() == torch.isnan(dz).any(dim=1).tolist() == [False, True, True, False]
    assert c.status() == B.FSDP_KSTATUS_BAD_TOKEN
    c.token_logprobs_loss(z, t, lp, dz, dlogprob=a)
    assert torch.isnan(dz).all(dim=1).tolist() == [False, True, True, False]
    assert c.status() == B.FSDP_KSTATUS_BAD_TOKEN and c.status() == 0


@pytest.mark.parametrize("dtype,each", [(BF, 8), (F32, 4)])
def test_alternatives_that_one_list_holds(c, dtype, each):
    """Logits placed so that the largest ones all belong to a few threads: more candidates than
    there is room for, in rising, falling and equal order."""
    vocab = 4000000
    i = torch.arange(vocab, device="cuda")
    mine = (i // each) % 512 < 3
    z = torch.zeros((3, vocab), device="cuda")
    z[0] = torch.where(mine, 1.0 + (i % 4096) * 2.0 ** -6, 0.0)
    z[1] = torch.where(mine, 5.0, 0.0)
    z[2] = -(i * 8.0 / vocab)
    z = z.to(dtype)
    for row in range(3):
        _check_forward(c, z[row:row + 1], torch.zeros(1, dtype=torch.int64, device="cuda"), 1.0, 32)
    z = torch.linspace(0, 4, vocab, device="cuda").to(dtype)[None].contiguous()
    _check_forward(c, z, torch.zeros(1, dtype=torch.int64, device="cuda"), 1.0, 32)


@pytest.mark.parametrize("dtype,vocab", [(BF, 1200000), (F32, 700001)])
def test_rows_that_no_cluster_holds(c, dtype, vocab):
    z, t = _logits(2, vocab, dtype, seed=6, std=1.0)
    a = torch.tensor([1.0, -2.0], device="cuda")
    lp, st, h = _check_forward(c, z, t, 1.0, 3)
    want, tol = _wanted_grad(z, t, 1.0, a, a)
    dz = torch.empty_like(z)
    c.token_logprobs_loss(z, t, lp, dz, dlogprob=a, dentropy=a)
    inside(dz, want, tol + U[dtype] * np.abs(want), "loss")
    c.token_logprobs_backward(z, t, st, dz, dlogprob=a, entropy=h, dentropy=a)
    inside(dz, want, tol + U[dtype] * np.abs(want), "backward")


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 3e5, 1e7, 1e25, 1e30])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scales(c, dtype, scale):
    """From nearly uniform to one-hot; logits of either sign and size.  d may be off by 2^-23 of itself; as x e^-x and
    x^2 e^-x are below 0.4 and 0.6, that is below 2^-22 of scale (|a| + |b| (1 + H)), H up to 7.2."""
    z, t = _logits(6, 1283, dtype, seed=9)
    z[1] -= 300.0
    z[2] += 300.0
    z[3] *= 1e-20
    t[:] = z.float().argmax(dim=1)
    lp, st, h = torch.empty(6, device="cuda"), torch.empty((6, 2), device="cuda"), torch.empty(6, device="cuda")
    c.token_logprobs_forward(z, t, lp, entropy=h, stats=st, scale=scale)
    _check_rows(_reference(z, t, scale), 1283, lp, st, h)
    a = torch.ones(6, device="cuda")
    dz = torch.empty_like(z)
    want, tol = _wanted_grad(z, t, scale, a, a)
    with np.errstate(over="ignore"):
        want, tol = np.clip(want, -1e38, 1e38), tol + U[dtype] * np.abs(want)
    for call in (lambda: c.token_logprobs_loss(z, t, lp, dz, dlogprob=a, dentropy=a, scale=scale),
                 lambda: c.token_logprobs_backward(z, t, st, dz, dlogprob=a, entropy=h, dentropy=a, scale=scale)):
        call()
        inside(dz, want, tol + scale * 2.0 ** -18, "gradient")


def test_no_rows_and_no_tokens(c):
    z, t = _logits(0, 100, BF)
    e = torch.empty(0, device="cuda")
    c.token_logprobs_forward(z, t, e, entropy=e)
    c.token_logprobs_loss(z, t, e, z, dlogprob=e)
    c.token_logprobs_backward(z, t, torch.empty((0, 2), device="cuda"), z, dlogprob=e)
    z, t = _logits(6, 999, F32)
    h, h2, lp = (torch.empty(6, device="cuda") for _ in range(3))
    tt, tl = torch.empty((6, 4), dtype=torch.int64, device="cuda"), torch.empty((6, 4), device="cuda")
    c.token_logprobs_forward(z, None, None, entropy=h, top_tokens=tt, top_logprobs=tl)
    c.token_logprobs_forward(z, t, lp, entropy=h2)
    assert torch.equal(h, h2) and torch.equal(tt, _ranked(z, 4))


def test_many_rows(c):
    """More rows than blocks run at once.  A row alone is split over more threads: both are within eps."""
    z, t = _logits(3001, 300, BF, seed=4)
    lp, _, h = _check_forward(c, z, t, 1.0, 5)
    one = torch.empty(1, device="cuda")
    for r in (0, 1500, 3000):
        c.token_logprobs_forward(z[r:r + 1], t[r:r + 1], one)
        if torch.isfinite(lp[r]):
            assert abs(one.item() - lp[r].item()) <= 2 * _eps(300, 6.0, 6.0) + 2.0 ** -22 * (abs(lp[r].item()) + 6)
        else:
            assert one.item() == lp[r].item()


def test_offsets_beyond_32_bits(c):
    """A row that begins past 2^32 bytes and past 2^31 elements."""
    stride, vocab = 2 ** 31 + 6, 1000
    buf = torch.zeros(stride + vocab, dtype=BF, device="cuda")
    z = torch.as_strided(buf, (2, vocab), (stride, 1))
    src, t = _logits(2, vocab, BF, seed=5)
    z.copy_(src)
    lp, st, _ = _check_forward(c, z, t, 1.0, 9)
    a = torch.ones(2, device="cuda")
    c.token_logprobs_backward(z, t, st, z, dlogprob=a)
    want, tol = _wanted_grad(src, t, 1.0, a, None)
    inside(z, want, tol + U[BF] * np.abs(want), "in place")
    assert not bool(buf[vocab:stride].any())


def test_gradient_against_differences(c):
    """L = sum(a logprob + b H) in F32.  The quotient errs by h^2/6 of the third derivative along the
    direction (below 8 (|a| + 4 |b|) for p <= 1 and directions of size <= 1, four directions' spread) and by
    the forward's rounding over 2h."""
    rows, vocab, step = 3, 37, 2.0 ** -6
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    z = torch.empty((rows, vocab), device="cuda").normal_(generator=g)
    t = torch.tensor([0, 36, -1], device="cuda")
    a, b = (torch.empty(rows, device="cuda").normal_(generator=g) for _ in range(2))
    lp, h, dz = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(z)

    def loss(z):
        c.token_logprobs_forward(z, t, lp, entropy=h, scale=1.5)
        return (a.double() * lp.double() + b.double() * h.double()).sum().item()

    c.token_logprobs_loss(z, t, lp, dz, dlogprob=a, dentropy=b, scale=1.5)
    size = (a.abs() + 4 * b.abs()).sum().item()
    for _ in range(5):
        d = torch.rand((rows, vocab), device="cuda", generator=g) * 2 - 1
        slope = (loss(z + step * d) - loss(z - step * d)) / (2 * step)
        want = (dz.double() * d.double()).sum().item()
        assert abs(slope - want) <= step ** 2 / 6 * 8 * 1.5 ** 3 * size + 2.0 ** -18 * size / step


def test_captured_and_on_another_stream(c):
    z, t = _logits(5, 5003, BF, seed=8)
    a = torch.ones(5, device="cuda")
    lp, dz = torch.empty(5, device="cuda"), torch.empty_like(z)
    c.token_logprobs_loss(z, t, lp, dz, dlogprob=a)
    want = (lp.clone(), dz.clone())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lp.zero_(), dz.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.token_logprobs_loss(z, t, lp, dz, dlogprob=a)
    s.synchronize()
    assert torch.equal(lp, want[0]) and torch.equal(dz, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.token_logprobs_loss(z, t, lp, dz, dlogprob=a)
    for _ in range(2):
        lp.zero_(), dz.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lp, want[0]) and torch.equal(dz, want[1])
