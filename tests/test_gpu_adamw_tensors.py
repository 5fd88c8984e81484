"""AdamW over many tensors: against the unit's AdamW and against numpy's fp32 operations in the
documented order, bit for bit; 8-bit moments against the format's definition."""
import numpy as np
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
f = np.float32


@pytest.fixture(scope="module")
def c():
    from conftest import library
    library()
    h = B.Compute(0)
    yield h
    h.close()


# ---- the format ----

def decode(codes, exps, signed):
    k = codes.astype(np.int64)
    low = k & 127 if signed else k
    e, m = low >> 3, low & 7
    v = np.ldexp(np.where(e > 0, 8 + m, m).astype(np.float64), np.maximum(e, 1) - (18 if signed else 34))
    v = np.where(k > 127, -v, v) if signed else v
    byte = np.repeat(exps.astype(np.int64), 32)[:len(k)]
    return np.where(byte == 255, np.nan, np.where(byte == 0, 0.0, np.ldexp(v, byte - 127)))


def encode(x, signed, bits=None):
    """Codes and exponent bytes of float32 x; ``bits``: 16 random bits an element, or nearest even."""
    n = len(x)
    mag = np.abs(x) if signed else np.where(np.isnan(x), x, np.maximum(x, f(0)))
    groups = -(-n // 32)
    pad = np.zeros(groups * 32, f)
    pad[:n] = mag
    g = pad.reshape(-1, 32)
    bad = ~np.isfinite(g).all(axis=1)
    top = np.where(bad, f(0), np.nan_to_num(g, nan=0, posinf=0).max(axis=1)).astype(f).view(np.uint32).astype(np.int64)
    exps = np.where(bad, 255, np.clip((top + 0xFFFFF) >> 23, 1, 253))
    e = np.repeat(exps, 32)[:n]
    y = np.ldexp(np.where(e == 255, 0.0, np.nan_to_num(mag, nan=0, posinf=0)).astype(np.float64), 127 - np.minimum(e, 253))
    least, most = (-14, 127) if signed else (-30, 255)
    ex = np.maximum(np.where(y > 0, np.frexp(y)[1] - 1, least), least)
    k = np.ldexp(y, 3 - ex)                                   # 8 .. 16, below 8 under the least exponent
    k = np.rint(k * 2 ** 20) / 2 ** 20                        # the 20 bits below
    k = np.rint(k) if bits is None else np.floor(k + bits / 65536)
    code = np.minimum(k.astype(np.int64) + ((ex - least) << 3), most)
    code = np.where((x < 0) & (code > 0), code | 128, code) if signed else np.where(mag > 0, np.maximum(code, 1), 0)
    return np.where(e == 255, 0, code).astype(np.uint8), exps.astype(np.uint8)


def same_codes(got, x, signed, bits, what):
    """encode()'s codes; where value and random bits add up to a code exactly, that or the one below."""
    got, (want, exps) = got.cpu().numpy(), encode(x, signed, bits)
    e = np.repeat(exps.astype(np.int64), 32)[:len(x)]
    y = np.ldexp(np.where(e == 255, 0.0, np.abs(np.nan_to_num(x, nan=0, posinf=0, neginf=0))).astype(np.float64), 127 - np.minimum(e, 253))
    k = np.ldexp(y, 3 - np.maximum(np.where(y > 0, np.frexp(y)[1] - 1, -30), -14 if signed else -30)) + bits / 65536
    tie = (k == np.rint(k)) & (y > 0)
    low, up = got.astype(np.int64) & (127 if signed else 255), want.astype(np.int64) & (127 if signed else 255)
    assert len(x) < 1000 or tie.mean() <= 0.01, what
    ok = (got == want) | (tie & (low == up - 1))
    assert ok.all(), f"{what}: {np.flatnonzero(~ok)[:5]} of {ok.size}"


def random_bits(n, number, seed, first=0):
    key = ((seed * 0x9E3779B97F4A7C15 + (number + 1) * 0xD1B54A32D192ED03) % 2 ** 64) >> 32
    i = np.arange(first, first + n, dtype=np.uint64)
    x = (i & np.uint64(0xFFFFFFFF)).astype(np.uint32) ^ np.uint32(key) ^ ((i >> np.uint64(32)).astype(np.uint32) * np.uint32(0x85157AF5))
    x ^= x >> np.uint32(16)
    x *= np.uint32(0xD36F86A9)
    x ^= x >> np.uint32(15)
    x *= np.uint32(0xC242E759)
    x ^= x >> np.uint32(16)
    return (x & np.uint32(0xFFFF)).astype(np.int64), (x >> np.uint32(16)).astype(np.int64)


def adamw(p, g, m, v, step, lr_scale=1.0, decay_scale=1.0, grad_scale=None, hp=HP):
    """One step in fp32, one rounding an operation; constants formed in 64 bits and rounded once."""
    lr, wd = hp["lr"] * lr_scale, hp["weight_decay"] * decay_scale
    with np.errstate(all="ignore"):
        g = g if grad_scale is None else g * f(grad_scale)
        m = f(hp["beta1"]) * m + f(1 - hp["beta1"]) * g
        v = f(hp["beta2"]) * v + f(1 - hp["beta2"]) * (g * g)
        denom = np.sqrt(v / f(1 - hp["beta2"] ** step)) + f(hp["eps"])
        return p * f(1 - lr * wd) - f(lr / (1 - hp["beta1"] ** step)) * (m / denom), m, v


def same(a, b, what):
    a = a.cpu().numpy() if isinstance(a, torch.Tensor) else a
    assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f"), f"{what}: {np.flatnonzero(a != b)[:5]} of {a.size}"


def host(t):
    return t.detach().float().cpu().numpy()


def _tensor(n, off, dtype=F32, std=1.0, seed=0, fill=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    buf = torch.full((n + off + 40,), -77, dtype=dtype, device="cuda")
    t = buf[off:off + n]
    t.copy_(torch.empty(n, device="cuda").normal_(0, std, generator=g) if fill is None else fill)
    return t, buf


def _untouched(t, buf, off):
    n = t.numel()
    assert bool((buf[:off] == buf.new_full((), -77)).all()) and bool((buf[off + n:] == buf.new_full((), -77)).all())


SIZES = [1, 0, 31, 32, 33, 64, 127, 1000, 2047, 2048, 2049, 4096, 5121, 20000, 7 * 13, 65536 + 17]


@pytest.mark.parametrize("moments", ["f32", "8bit"])
@pytest.mark.parametrize("grad", [F32, BF])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_step(c, moments, grad, off):
    ps, gs, ms, vs, cs, bufs, want = [], [], [], [], [], [], []
    for j, n in enumerate(SIZES):
        p, b0 = _tensor(n, off, seed=4 * j)
        g, b1 = _tensor(n, off, grad, 1e-3, seed=4 * j + 1)
        k, b2 = _tensor(n, off, BF, fill=torch.zeros(n, device="cuda"))
        bufs += [(p, b0), (g, b1), (k, b2)]
        m0 = torch.randn(n, generator=torch.Generator().manual_seed(j)).numpy() * f(3e-4)
        v0 = (torch.randn(n, generator=torch.Generator().manual_seed(j + 99)).numpy() * f(1e-3)) ** 2
        if moments == "f32":
            m, b3 = _tensor(n, off, fill=torch.from_numpy(m0).cuda())
            v, b4 = _tensor(n, off, fill=torch.from_numpy(v0).cuda())
            bufs += [(m, b3), (v, b4)]
        else:
            cm, em = encode(m0, True)
            cv, ev = encode(v0, False)
            m0, v0 = decode(cm, em, True).astype(f), decode(cv, ev, False).astype(f)
            state = []
            for codes, exps in ((cm, em), (cv, ev)):
                x, bx = _tensor(n, off, torch.uint8, fill=torch.from_numpy(codes).cuda())
                e, be = _tensor(len(exps), off, torch.uint8, fill=torch.from_numpy(exps).cuda())
                bufs += [(x, bx), (e, be)]
                state.append((x, e))
            m, v = B.State8(n, True, *state[0]), B.State8(n, False, *state[1])
        ps.append(p), gs.append(g), ms.append(m), vs.append(v), cs.append(k if j % 3 else None)
        want.append((host(p), host(g), m0, v0))
    lr, decay = [1.0 + 0.5 * (j % 2) for j in range(len(SIZES))], [float(j % 4 != 1) for j in range(len(SIZES))]
    tensors = B.AdamWTensors(ps, gs, ms, vs, copies=cs, lr_scale=lr, decay_scale=decay)
    scale = torch.tensor([0.37], device="cuda")
    for step, seed in ((7, 12345), (8, 2 ** 63 + 5)):
        c.adamw_tensors(tensors, HP, step, seed=seed, grad_scale=scale if step == 8 else None)
        for j, n in enumerate(SIZES):
            p0, g0, m0, v0 = want[j]
            p1, m1, v1 = adamw(p0, g0, m0, v0, step, lr[j], decay[j], f(0.37) if step == 8 else None)
            same(ps[j], p1, f"param {j}")
            if cs[j] is not None:
                assert torch.equal(cs[j], ps[j].to(BF)), j
            if moments == "f32":
                same(ms[j], m1, f"m {j}")
                same(vs[j], v1, f"v {j}")
            else:
                rm, rv = random_bits(n, j, seed)
                for got, x, signed, r in ((ms[j], m1, True, rm), (vs[j], v1, False, rv)):
                    same(got.exps, encode(x, signed, r)[1], f"exponents {j} {signed}")
                    same_codes(got.codes, x, signed, r, f"codes {j} {signed}")
                m1, v1 = (decode(s.codes.cpu().numpy(), s.exps.cpu().numpy(), s.signed).astype(f) for s in (ms[j], vs[j]))
            want[j] = (p1, g0, m1, v1)
    for t, buf in bufs:
        _untouched(t, buf, off)


def test_the_units_adamw_has_the_same_bits(c):
    shapes = [(33, 47), (100,), (1,)]
    u = B.Unit(shapes, "flat", 3, "f32")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    params = [torch.empty(s, device="cuda").normal_(0, 0.1, generator=gen) for s in shapes]
    u.load(params)
    p = torch.cat([x.reshape(-1) for x in params])
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    g = torch.empty_like(p)
    at, views = 0, []
    for s in shapes:
        n = int(np.prod(s))
        views.append(slice(at, at + n))
        at += n
    tensors = B.AdamWTensors([p[s] for s in views], [g[s] for s in views], [m[s] for s in views], [v[s] for s in views])
    for step in range(1, 4):
        grads = [torch.empty_like(p).normal_(0, 1e-2, generator=gen) for _ in range(3)]
        u.reduce_scatter(grads)
        g.copy_(u.read_global("grad"))
        u.adamw_step(HP)
        c.adamw_tensors(tensors, HP, step)
        for mine, name in ((p, "param"), (m, "exp_avg"), (v, "exp_avg_sq")):
            assert torch.equal(mine, u.read_global(name)), (step, name)
    u.close()


def test_more_tensors_than_one_launch_takes(c):
    n = 1203
    sizes = [1 + (7 * j) % 70 for j in range(n)]
    ps = [torch.full((k,), float(j % 9), device="cuda") for j, k in enumerate(sizes)]
    gs = [torch.full((k,), 1e-3 * (j % 5 - 2), device="cuda") for j, k in enumerate(sizes)]
    ms, vs = [B.State8(k, True) for k in sizes], [B.State8(k, False) for k in sizes]
    p0 = [host(p) for p in ps]
    c.adamw_tensors(B.AdamWTensors(ps, gs, ms, vs), HP, 1, seed=9)
    for j in range(0, n, 41):
        p1, m1, v1 = adamw(p0[j], host(gs[j]), np.zeros(sizes[j], f), np.zeros(sizes[j], f), 1)
        same(ps[j], p1, j)
        rm, rv = random_bits(sizes[j], j, 9)
        same_codes(ms[j].codes, m1, True, rm, j)
        same_codes(vs[j].codes, v1, False, rv, j)


def test_skipped_and_empty(c):
    p, g = torch.randn(100, device="cuda"), torch.randn(100, device="cuda")
    m, v, k = B.State8(100, True), B.State8(100, False), torch.zeros(100, dtype=BF, device="cuda")
    tensors = B.AdamWTensors([p], [g], [m], [v], copies=[k])
    skip, before = torch.ones(1, dtype=torch.int32, device="cuda"), p.clone()
    c.adamw_tensors(tensors, HP, 1, skip=skip)
    assert torch.equal(p, before) and not bool(m.codes.any()) and not bool(v.exps.any()) and not bool(k.any())
    skip.zero_()
    c.adamw_tensors(tensors, HP, 1, skip=skip)
    assert not torch.equal(p, before) and bool(k.any())
    c.adamw_tensors(B.AdamWTensors([], [], [], []), HP, 1)
    e = torch.empty(0, device="cuda")
    c.adamw_tensors(B.AdamWTensors([e], [e], [e], [e]), HP, 1)


@pytest.mark.parametrize("moments", ["f32", "8bit"])
def test_gradients_that_are_not_finite(c, moments):
    n = 96
    p, g = torch.ones(n, device="cuda"), torch.full((n,), 1e-3, device="cuda")
    g[3], g[70] = float("inf"), float("nan")
    m, v = (B.State8(n, True), B.State8(n, False)) if moments == "8bit" else (torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"))
    c.adamw_tensors(B.AdamWTensors([p], [g], [m], [v]), HP, 1)
    want, m1, v1 = adamw(np.ones(n, f), host(g), np.zeros(n, f), np.zeros(n, f), 1)
    same(p, want, "param")
    if moments == "8bit":
        assert m.exps.tolist()[0] == m.exps.tolist()[2] == v.exps.tolist()[0] == v.exps.tolist()[2] == 255 != m.exps.tolist()[1]
        out = torch.empty(n, device="cuda")
        for s in (m, v):
            c.state8_unpack(s, out)
            assert torch.isnan(out).tolist() == [True] * 32 + [False] * 32 + [True] * 32


@pytest.mark.parametrize("signed", [True, False])
@pytest.mark.parametrize("n", [1, 31, 33, 64, 5000, 262144 + 5])
def test_pack_and_unpack(c, signed, n):
    rng = np.random.default_rng(n)
    x = (rng.normal(size=n) * np.exp(rng.normal(size=n) * 8)).astype(f)
    if n > 1000:
        x[:32], x[32:64], x[64], x[96], x[128] = 0, rng.normal(size=32) * 1e-38, np.inf, np.nan, 3e38
        x[160:192], x[192], x[200] = 1e-45, 1.875, 1.8750001
        x[256:288] = -np.abs(x[256:288])
    s = B.State8(n, signed)
    c.state8_pack(torch.from_numpy(x).cuda(), s)
    codes, exps = encode(x, signed)
    same(s.exps, exps, "exponents")
    same(s.codes, codes, "codes")
    want = decode(codes, exps, signed)
    for dt in (F32, BF):
        out = torch.empty(n + 1, dtype=dt, device="cuda")[1:]
        c.state8_unpack(s, out)
        w = torch.from_numpy(want.astype(f)).to(dt).float().numpy()
        same(host(out), w, dt)
    fine = np.isfinite(want)
    mag = x if signed else np.maximum(x, 0)
    unit = np.ldexp(1.0, np.repeat(exps.astype(int), 32)[:n] - 127)
    tol = np.maximum(np.abs(mag) * 2.0 ** -4, unit * 2.0 ** (-18 if signed else -33))
    inside = fine & (np.repeat(exps, 32)[:n] < 253)
    assert bool((np.abs(want - mag)[inside] <= tol[inside]).all())


def test_codes_survive(c):
    """Every code with every exponent byte that occurs reads as the definition says, and packs to itself
    where its group's largest element is in the upper half of the codes' range."""
    for signed in (True, False):
        codes = np.tile(np.arange(256, dtype=np.uint8), 254)
        codes = codes[(codes & 127) > 0] if signed else codes
        n = len(codes) // 32 * 32
        codes = codes[:n].copy()
        exps = (np.arange(n // 32) % 252 + 1).astype(np.uint8)
        s = B.State8(n, signed, torch.from_numpy(codes).cuda(), torch.from_numpy(exps).cuda())
        out = torch.empty(n, device="cuda")
        c.state8_unpack(s, out)
        same(out, decode(codes, exps, signed).astype(f), "values")


def test_rounding_at_random_keeps_the_mean(c):
    """A moving average that moves by less than a rounding step follows the 32-bit one: 256 equal elements,
    400 steps.  Each rounding's mean is the value, up to 2^-17 of a step.  Its deviation is at most half a
    step, 2^-4 v; v grows in proportion to the steps, so the squares sum to a third of 400 of the last, and the
    mean of 256 has a deviation of 2^-4 / 16 * 20 * 0.58 v at most, of which six are allowed."""
    n, g = 256, 1e-3
    p, grad = torch.zeros(n, device="cuda"), torch.full((n,), g, device="cuda")
    m, v = B.State8(n, True), B.State8(n, False)
    tensors = B.AdamWTensors([p], [grad], [m], [v])
    hp = dict(HP, lr=0.0)
    for step in range(1, 401):
        c.adamw_tensors(tensors, hp, step, seed=step)
    out = torch.empty(n, device="cuda")
    c.state8_unpack(v, out)
    want = g * g * (1 - 0.999 ** 400)
    assert abs(out.double().mean().item() - want) <= 6 * 2.0 ** -4 / 16 * 20 * 0.58 * want
    assert out.double().mean().item() > 0.5 * want      # to nearest it stops near 0.016 g^2 of 0.33
    c.state8_unpack(m, out)
    assert abs(out.double().mean().item() - g) <= 6 * 2.0 ** -4 / 16 * 2.3 * g   # sqrt(1 / (1 - 0.9^2)) steps' worth


def test_elements_beyond_32_bits(c):
    n, tail = 2 ** 32 + 96, 160
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=BF, device="cuda")
    m, v = B.State8(n, True), B.State8(n, False)
    first = n - tail
    g[first:] = torch.linspace(-1e-2, 1e-2, tail, device="cuda").to(BF)
    c.adamw_tensors(B.AdamWTensors([p], [g], [m], [v]), HP, 3, seed=1)
    p1, m1, v1 = adamw(np.zeros(tail, f), host(g[first:]), np.zeros(tail, f), np.zeros(tail, f), 3)
    same(p[first:], p1, "param")
    rm, rv = random_bits(tail, 0, 1, first)
    same_codes(m.codes[first:], m1, True, rm, "m")
    same_codes(v.codes[first:], v1, False, rv, "v")
    assert not bool(m.codes[:first].any()) and not bool(p[:first].any())
    out = torch.empty(n, dtype=BF, device="cuda")
    c.state8_unpack(m, out)
    same(host(out[first:]), decode(m.codes[first:].cpu().numpy(), m.exps[first // 32:].cpu().numpy(), True).astype(f), "values")


def test_captured_and_on_another_stream(c):
    n = 5000
    g = torch.randn(n, device="cuda")
    results = []
    for how in ("eager", "stream", "graph"):
        p, m, v = torch.ones(n, device="cuda"), B.State8(n, True), B.State8(n, False)
        tensors = B.AdamWTensors([p], [g], [m], [v])
        torch.cuda.synchronize()
        if how == "eager":
            c.adamw_tensors(tensors, HP, 2, seed=4)
        elif how == "stream":
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                c.adamw_tensors(tensors, HP, 2, seed=4)
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                c.adamw_tensors(tensors, HP, 2, seed=4)
            graph.replay()
        torch.cuda.synchronize()
        results.append((p, m.codes, m.exps, v.codes, v.exps))
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))
