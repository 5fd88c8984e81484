"""What the binding's block operators refuse before anything reaches the library:
arguments whose faults the C side cannot see.  The refusals are errors, not
assertions, so that they stand in an optimised interpreter too."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from conftest import ROOT
from fully_sharded_unit_gb300 import binding as B

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


def _refused(f):
    with pytest.raises(B.FsdpError) as e:
        f()
    assert e.value.code == B.FSDP_E_INVALID_ARG
    return str(e.value)


def _calls(x, vec, stat):
    """Each entry point with `x` for its matrices and `vec`, `stat` for its vectors."""
    h = B.ComputeHandle()
    return [lambda: B.fsdp_layer_norm_forward(h, x, vec, vec, 1e-5, x, stat, stat),
            lambda: B.fsdp_layer_norm_backward(h, x, x, vec, stat, stat, x, vec, vec),
            lambda: B.fsdp_linear_forward(h, x, x, x, bias=vec),
            lambda: B.fsdp_linear_grad_input(h, x, x, x),
            lambda: B.fsdp_linear_grad_weight(h, x, x, x, dbias=vec),
            lambda: B.fsdp_act8_pack(h, x, x),
            lambda: B.fsdp_act8_unpack(h, x, x)]


def test_host_tensors_are_refused():
    for call in _calls(torch.zeros((8, 8), dtype=BF), torch.zeros(8, dtype=BF), torch.zeros(8)):
        assert "CUDA tensor" in _refused(call)
    _refused(lambda: B._vec(torch.zeros(8), 8))
    _refused(lambda: B._stat(torch.zeros(8), 8))
    _refused(lambda: B._mat(torch.zeros(8)))
    _refused(lambda: B._mat(torch.zeros((2, 2, 2))))
    _refused(lambda: B._mat("x"))
    _refused(lambda: B.Act8(4, 40, device="cpu"))


def test_refusals_stand_in_an_optimised_interpreter():
    code = textwrap.dedent("""
        import torch
        from fully_sharded_unit_gb300 import binding as B
        assert False                      # not looked at
        x, v = torch.zeros((8, 8), dtype=torch.bfloat16), torch.zeros(8)
        n = 0
        for f in (lambda: B._mat(x), lambda: B._vec(v, 8), lambda: B._vec(v, 9), lambda: B._same(0, 1, "a and b"),
                  lambda: B.Act8(4, 40, device="cpu"), lambda: B.fsdp_act8_pack(B.ComputeHandle(), x, x)):
            try:
                f()
            except B.FsdpError:
                n += 1
        print("refused", n)
    """)
    r = subprocess.run([sys.executable, "-O", "-c", code], cwd=ROOT, capture_output=True, text=True,
                       env=dict(os.environ, PYTHONPATH=ROOT))
    assert r.stdout.strip() == "refused 6", r.stdout + r.stderr


@pytest.mark.gpu
def test_device_tensors_that_do_not_fit_are_refused():
    x, v, s = torch.zeros((8, 8), dtype=BF, device="cuda"), torch.zeros(8, dtype=BF, device="cuda"), torch.zeros(8, device="cuda")
    for call in _calls(x.half(), v, s):
        assert "float16" in _refused(call)
    wide = torch.zeros((8, 16), dtype=BF, device="cuda")[:, ::2]
    for call in _calls(wide, v, s):
        assert "contiguous" in _refused(call)
    norm, norm_grad, linear, _, weight, _, _ = _calls(x, v.half(), s)
    for call in (norm, norm_grad, linear, weight):
        _refused(call)
    for call in (_calls(x, v[:7], s)[0], _calls(x, v, s[:7])[0], _calls(x, v, v)[0], _calls(x, v, s[::2])[1], _calls(x, s.cpu(), s)[2]):
        _refused(call)
    h = B.ComputeHandle()
    _refused(lambda: B.fsdp_layer_norm_forward(h, x, v, v.float(), 1e-5, x, s, s))
    _refused(lambda: B.fsdp_layer_norm_backward(h, x, x, v, s, s, x, v, v.float()))
    _refused(lambda: B.fsdp_linear_grad_weight(h, x, x, x, dbias=s))
    q, e = torch.zeros((8, 32), dtype=torch.int8, device="cuda"), torch.zeros((8, 1), dtype=torch.uint8, device="cuda")
    B.Act8(8, 8, q=q, exps=e)
    for bad in (dict(q=q[:4], exps=e), dict(q=q.view(torch.uint8), exps=e), dict(q=q.cpu(), exps=e), dict(q=q, exps=e.repeat(1, 2)),
                dict(q=q, exps=e.view(torch.int8))):
        _refused(lambda: B.Act8(8, 8, **bad))


@pytest.mark.gpu
def test_a_handle_of_another_device_is_refused():
    """The handle here says that it is of a device which the tensors are not on."""
    x, v, s = torch.zeros((8, 8), dtype=BF, device="cuda"), torch.zeros(8, dtype=BF, device="cuda"), torch.zeros(8, device="cuda")
    k = B.Act8(8, 8)
    h = B.ComputeHandle()
    h.device = x.get_device() + 1
    for f in (lambda: B.fsdp_layer_norm_forward(h, x, v, v, 1e-5, x, s, s), lambda: B.fsdp_act8_unpack(h, k, x),
              lambda: B.fsdp_linear_grad_weight(h, x, x, x), lambda: B._vec(v, 8, h.device)):
        assert "handle" in _refused(f)
    c = B.Compute(0)
    assert c.handle.device == x.get_device() == k.device
    c.act8_pack(x, k)
    c.close()
