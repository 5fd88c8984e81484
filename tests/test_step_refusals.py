"""What the operators at a training step's ends refuse: what the binding sees (without a GPU too),
and what the library checks before anything is enqueued."""
import ctypes

import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

BF, F32, I64 = torch.bfloat16, torch.float32, torch.int64
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


def _refused(f, code=B.FSDP_E_INVALID_ARG):
    with pytest.raises(B.FsdpError) as e:
        f()
    assert e.value.code == code, str(e.value)
    return str(e.value)


def test_host_tensors_are_refused():
    h, x, v, t = B.ComputeHandle(), torch.zeros((4, 8)), torch.zeros(4), torch.zeros(4, dtype=I64)
    for call in (lambda: B.fsdp_token_logprobs_forward(h, x, t, v), lambda: B.fsdp_token_logprobs_backward(h, x, t, v, x, dlogprob=v),
                 lambda: B.fsdp_token_logprobs_loss(h, x, t, v, x, dlogprob=v), lambda: B.fsdp_residual_norm_forward(h, x, x),
                 lambda: B.fsdp_residual_norm_backward(h, x, x, x, x, x, x), lambda: B.State8(10, True, device="cpu"),
                 lambda: B.AdamWTensors([v], [v], [v], [v]), lambda: B.fsdp_state8_pack(h, v, v), lambda: B.fsdp_adamw_tensors(h, [v], HP, 1),
                 lambda: B.AdamWTensors([v], [], [v], [v]), lambda: B.AdamWTensors([v], [None], [v], [v]), lambda: B.AdamWTensors([None], [v], [v], [v])):
        _refused(call)
    _refused(lambda: B.fsdp_residual_norm_forward(h, None, x))
    _refused(lambda: B.fsdp_token_logprobs_forward(h, None, t, v))


def test_workspace():
    assert B.fsdp_residual_norm_workspace_bytes(0, 8) == 0
    assert B.fsdp_residual_norm_workspace_bytes(10, 8) >= 10 * 2 * 8 * 4
    for rows, cols in ((-1, 8), (1, 0), (1, 2 ** 41)):
        _refused(lambda: B.fsdp_residual_norm_workspace_bytes(rows, cols))
    assert B.lib().fsdp_residual_norm_workspace_bytes(1, 1, None) == B.FSDP_E_INVALID_ARG


def test_null_handles():
    l = B.lib()
    m = B.Matrix(None, None, 0, 8, 8, 0)
    r = ctypes.byref(m)
    assert l.fsdp_token_logprobs_forward(None, r, None, 1.0, None, None, None, 0, None, None, None) == B.FSDP_E_INVALID_ARG
    assert l.fsdp_token_logprobs_backward(None, r, None, 1.0, None, None, None, None, r, None) == B.FSDP_E_INVALID_ARG
    assert l.fsdp_token_logprobs_loss(None, r, None, 1.0, None, None, None, None, None, r, None) == B.FSDP_E_INVALID_ARG
    assert l.fsdp_residual_norm_forward(None, r, None, None, None, None, 0, 1.0, 0.0, r, None, None, None, None) == B.FSDP_E_INVALID_ARG
    assert l.fsdp_residual_norm_backward(None, r, None, r, None, None, None, None, 0, 1.0, None, None, r, None, None, None, None, 0, 0, None) == B.FSDP_E_INVALID_ARG
    assert l.fsdp_state8_pack(None, 0, None, 0, None, None, None) == B.FSDP_E_INVALID_ARG
    assert l.fsdp_state8_unpack(None, 0, None, None, 0, None, 0, None) == B.FSDP_E_INVALID_ARG
    assert l.fsdp_adamw_tensors(None, None, 0, ctypes.byref(B._hp(HP)), 1, 0, None, None, None) == B.FSDP_E_INVALID_ARG


@pytest.mark.gpu
def test_logits():
    c = B.Compute(0)
    z, t, v = torch.zeros((4, 8), device="cuda"), torch.zeros(4, dtype=I64, device="cuda"), torch.zeros(4, device="cuda")
    s, tt, tl = torch.zeros((4, 2), device="cuda"), torch.zeros((4, 3), dtype=I64, device="cuda"), torch.zeros((4, 3), device="cuda")
    forward, back, loss = c.token_logprobs_forward, c.token_logprobs_backward, c.token_logprobs_loss
    for call in (lambda: forward(z, t, None), lambda: forward(z, None, v), lambda: forward(z, t.int(), v), lambda: forward(z, t[:3], v), lambda: forward(z, t, v[:3]),
                 lambda: forward(z, t, v, scale=0.0), lambda: forward(z, t, v, scale=float("nan")), lambda: forward(z, t, v, scale=-1.0),
                 lambda: forward(z, t, v, scale=1e39), lambda: forward(z.half(), t, v), lambda: forward(z.t(), t, v), lambda: forward(z, t, v, stats=v),
                 lambda: forward(z, t, v, top_tokens=tt), lambda: forward(z, t, v, top_tokens=tt, top_logprobs=tl[:, :2]),
                 lambda: forward(z[:, :2], t, v, top_tokens=tt, top_logprobs=tl),
                 lambda: forward(z.repeat(1, 9), t, v, top_tokens=tt.repeat(1, 11), top_logprobs=tl.repeat(1, 11)),
                 lambda: back(z, t, s, z), lambda: back(z, None, s, z, dlogprob=v), lambda: back(z, t, None, z, dlogprob=v), lambda: back(z, t, s, z, dentropy=v),
                 lambda: back(z, t, s, z[:, :7], dlogprob=v), lambda: back(z, t, s, None, dlogprob=v), lambda: back(z, t, s, z.double(), dlogprob=v),
                 lambda: loss(z, t, None, z, dlogprob=v), lambda: loss(z, None, v, z, dlogprob=v), lambda: loss(z, t, v, z), lambda: loss(z, t, v, None, dlogprob=v),
                 lambda: forward(B.Act8(4, 8), t, v), lambda: forward(z[:, :0], t, v)):
        _refused(call)
    raw = torch.zeros(64, dtype=torch.uint8, device="cuda")
    m = B.Matrix(z.data_ptr(), None, 4, 8, 8, 0)
    at = raw.data_ptr()
    assert B.lib().fsdp_token_logprobs_forward(c.handle, ctypes.byref(m), at + 4, 1.0, at, None, None, 0, None, None, None) == B.FSDP_E_ALIGN
    assert B.lib().fsdp_token_logprobs_forward(c.handle, ctypes.byref(m), at, 1.0, at + 2, None, None, 0, None, None, None) == B.FSDP_E_ALIGN
    assert B.lib().fsdp_token_logprobs_forward(c.handle, ctypes.byref(m), at, 1.0, at, None, None, -1, None, None, None) == B.FSDP_E_INVALID_ARG
    big = B.Matrix(z.data_ptr(), None, 1, 2 ** 30 + 1, 2 ** 30 + 1, 0)
    assert B.lib().fsdp_token_logprobs_forward(c.handle, ctypes.byref(big), at, 1.0, at, None, None, 0, None, None, None) == B.FSDP_E_INVALID_ARG
    c.close()


@pytest.mark.gpu
def test_residual_norm():
    x, w, r, g = torch.zeros((4, 8), device="cuda"), torch.zeros(8, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(8, device="cuda")
    c = B.Compute(B.fsdp_residual_norm_workspace_bytes(4, 8))
    fw, bw = c.residual_norm_forward, c.residual_norm_backward
    y = x.clone()
    for call in (lambda: fw(x, None), lambda: fw(x, x[:, :7]), lambda: fw(x, y, y=y, rstd=r), lambda: fw(x, y, gamma=w, rstd=r), lambda: fw(x, y, y=y, gamma=w),
                 lambda: fw(x, y, rstd=r), lambda: fw(x, y, post_rstd=r), lambda: fw(x, y, post_gamma=w, post_rstd=r), lambda: fw(x, y, gate=w),
                 lambda: fw(x, y, block=x, post_gamma=w), lambda: fw(x, y, block=x, post_gamma=w, gate=w.to(BF), post_rstd=r), lambda: fw(x, y, residual_scale=float("inf")),
                 lambda: fw(x, y, residual_scale=1e39), lambda: fw(x, y, eps=-1.0), lambda: fw(x, y, eps=float("nan")), lambda: fw(x, y, block=x, gate=w[:7]),
                 lambda: fw(x, y, y=y, gamma=w, rstd=r[:3]), lambda: fw(B.Act8(4, 8), y), lambda: fw(x, y, block=x.half()),
                 lambda: bw(None, None, x, x, y, y), lambda: bw(x, None, x, None, y, None), lambda: bw(None, x, None, x, y, None), lambda: bw(None, x, None, None, y, y),
                 lambda: bw(x, None, None, None, y, None, gamma=w, rstd=r, dgamma=g), lambda: bw(x, None, x, None, y, None, gamma=w, rstd=r),
                 lambda: bw(x, None, x, None, y, None, gamma=w, dgamma=g), lambda: bw(None, x, None, x, y, y, gate=w), lambda: bw(None, x, None, x, y, y, dgate=g),
                 lambda: bw(None, x, None, x, y, y, post_gamma=w, dpost_gamma=g), lambda: bw(None, x, None, x, y, y, gate=w, dgate=g, post_gamma=w, post_rstd=r, dpost_gamma=g.to(BF)),
                 lambda: bw(None, x, None, None, None, None)):
        _refused(call)
    small = B.Compute(16)
    assert "workspace" in _refused(lambda: small.residual_norm_backward(None, x, None, x, y, y), B.FSDP_E_CAPACITY)
    small.close()
    c.close()


@pytest.mark.gpu
def test_adamw():
    c = B.Compute(0)
    p, g = torch.zeros(40, device="cuda"), torch.zeros(40, device="cuda")
    m8, v8 = B.State8(40, True), B.State8(40, False)
    T = B.AdamWTensors
    for call in (lambda: T([p], [g[:39]], [p], [p]), lambda: T([p.to(BF)], [g], [p], [p]), lambda: T([p], [g.half()], [p], [p]), lambda: T([p], [g], [v8], [m8]),
                 lambda: T([p], [g], [m8], [p]), lambda: T([p], [g], [B.State8(39, True)], [v8]), lambda: T([p], [g], [p], [p], copies=[p]), lambda: T([p], [g], [p], [p], lr_scale=[]),
                 lambda: T([p[::2]], [g[:20]], [p[:20]], [p[:20]]), lambda: m8.piece(16, 8), lambda: m8.piece(32, 9), lambda: m8.piece(-32, 9),
                 lambda: B.State8(40, True, torch.zeros(39, dtype=torch.uint8, device="cuda")), lambda: B.State8(40, True, p), lambda: c.state8_pack(g[:39], m8),
                 lambda: c.state8_pack(g.to(BF), m8), lambda: c.state8_unpack(m8, g.half()), lambda: c.state8_unpack(p, g), lambda: c.state8_unpack(m8, g[:39])):
        _refused(call)
    ok = T([p], [g], [m8], [v8])
    one, flag = torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in (lambda: c.adamw_tensors(ok, HP, 0), lambda: c.adamw_tensors(ok, dict(HP, lr=-1.0), 1), lambda: c.adamw_tensors(ok, dict(HP, beta2=1.0), 1),
                 lambda: c.adamw_tensors(ok, HP, 1, grad_scale=one.double()), lambda: c.adamw_tensors(ok, HP, 1, grad_scale=torch.ones(2, device="cuda")),
                 lambda: c.adamw_tensors(ok, HP, 1, grad_scale=one.cpu()), lambda: c.adamw_tensors(ok, HP, 1, skip=one), lambda: c.adamw_tensors([ok], HP, 1),
                 lambda: c.adamw_tensors(T([p], [g], [m8], [v8], lr_scale=[-1.0]), HP, 1), lambda: c.adamw_tensors(T([p], [g], [m8], [v8], decay_scale=[float("nan")]), HP, 1),
                 lambda: c.adamw_tensors(T([p], [g], [m8], [v8], lr_scale=[1e300]), dict(HP, lr=1e300), 1), lambda: c.adamw_tensors(T([p], [g], [None], [p]), HP, 1)):
        _refused(call)
    e = (B.AdamWTensor * 1)()
    ctypes.memmove(e, ok.array, ctypes.sizeof(e))
    hp = ctypes.byref(B._hp(HP))
    call = lambda n=1, a=e: B.lib().fsdp_adamw_tensors(c.handle, a, n, hp, 1, 0, None, None, None)  # noqa: E731
    for field, value, code in (("param", p.data_ptr() + 2, B.FSDP_E_ALIGN), ("grad", g.data_ptr() + 1, B.FSDP_E_ALIGN), ("copy_bf16", p.data_ptr() + 1, B.FSDP_E_ALIGN),
                               ("exp_avg_exps", None, B.FSDP_E_INVALID_ARG), ("numel", -1, B.FSDP_E_INVALID_ARG), ("numel", 2 ** 41, B.FSDP_E_INVALID_ARG),
                               ("grad_dtype", 2, B.FSDP_E_INVALID_ARG), ("moments", 2, B.FSDP_E_INVALID_ARG)):
        old = getattr(e[0], field)
        setattr(e[0], field, value)
        assert call() == code, field
        setattr(e[0], field, old)
    assert call(-1) == B.FSDP_E_INVALID_ARG and call(1, None) == B.FSDP_E_INVALID_ARG and call(0, None) == B.FSDP_OK
    assert B.lib().fsdp_state8_pack(c.handle, 2, p.data_ptr(), 1, p.data_ptr(), p.data_ptr(), None) == B.FSDP_E_INVALID_ARG
    assert B.lib().fsdp_state8_unpack(c.handle, 0, p.data_ptr(), p.data_ptr(), 1, p.data_ptr(), 2, None) == B.FSDP_E_INVALID_ARG
    c.close()


@pytest.mark.gpu
def test_a_handle_of_another_device_is_refused():
    x, v, t = torch.zeros((8, 8), device="cuda"), torch.zeros(8, device="cuda"), torch.zeros(8, dtype=I64, device="cuda")
    s = B.State8(8, True)
    h = B.ComputeHandle()
    h.device = x.get_device() + 1
    for f in (lambda: B.fsdp_token_logprobs_forward(h, x, t, v), lambda: B.fsdp_token_logprobs_loss(h, x, t, v, x, dlogprob=v),
              lambda: B.fsdp_residual_norm_forward(h, x, x), lambda: B.fsdp_state8_pack(h, v, s), lambda: B.fsdp_state8_unpack(h, s, v),
              lambda: B.fsdp_adamw_tensors(h, B.AdamWTensors([v], [v], [v], [v]), HP, 1)):
        assert "handle" in _refused(f)
