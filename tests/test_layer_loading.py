"""What the package needs to load: the codec neither torch nor the layer's binding, the layer not
the binding; and a binding compiled against another torch is neither kept nor loaded."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

import __graft_entry__

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
qbuild = __graft_entry__._build_module()


def python(code):
    r = subprocess.run([sys.executable, "-W", "always", "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout, r.stderr


def test_codec_without_torch():
    out, _ = python("""
import sys
sys.modules["torch"] = None
import embedding_communication_codecs_gb300 as q
print(q.qc_code_words(32, 4), q.lib.qc_version() is not None, "int8_matmul" in dir(q))
""")
    assert out.split() == ["4", "True", "True"]


def test_importing_the_package_loads_neither_torch_nor_the_layer():
    out, _ = python("""
import sys
import embedding_communication_codecs_gb300 as q
print("torch" in sys.modules, "embedding_communication_codecs_gb300.layer" in sys.modules)
q.int8_matmul, q.layer.qc_swiglu_encode
print("torch" in sys.modules, q.int8_matmul is q.layer.int8_matmul, hasattr(q, "no_such_name"))
""")
    assert out.split() == ["False", "False", "True", "True", "False"]


def test_layer_without_its_binding():
    out, err = python("""
import sys
sys.modules["embedding_communication_codecs_gb300._qcbind"] = None
import embedding_communication_codecs_gb300 as q
import torch
for call in (lambda: q.rowwise_int8(torch.zeros(4, 8)),
             lambda: q.int8_matmul(torch.zeros((4, 8), dtype=torch.int8), torch.zeros(4), torch.zeros((2, 8), dtype=torch.int8),
                                   torch.zeros(2))):
    try:
        call()
    except ValueError as e:
        print("CUDA tensor" in str(e))
""")
    assert out.split() == ["True", "True"] and "ctypes" in err and "RuntimeWarning" in err


def test_a_binding_of_another_torch_is_rebuilt_and_not_loaded(tmp_path, monkeypatch):
    qbuild.build_library()
    assert qbuild.up_to_date() and qbuild.bind_fits()
    text = open(qbuild.BIND_STAMP).read()
    other = tmp_path / "stamp"
    other.write_text(text.replace("__version__ = '", "__version__ = '9"))
    monkeypatch.setattr(qbuild, "BIND_STAMP", str(other))
    assert qbuild.library_up_to_date() and not qbuild.bind_fits() and not qbuild.up_to_date()
    _, err = python(f"""
import embedding_communication_codecs_gb300.build as b
b.BIND_STAMP = {str(other)!r}
import embedding_communication_codecs_gb300 as q
import sys
q.int8_matmul
assert "embedding_communication_codecs_gb300._qcbind" not in sys.modules
""")
    assert "another torch" in err
    other.write_text("")
    assert not qbuild.bind_fits()


@pytest.mark.parametrize("call", ["rowwise_int8_dequant", "int8_matmul"])
@pytest.mark.parametrize("current", [0, 1])
def test_the_calls_that_were_the_bindings_alone(call, current, monkeypatch):
    """As for the other calls: made from Python, on the tensors' device and its current stream."""
    from tests import test_layer_devices as devices
    from torch._subclasses.fake_tensor import FakeTensorMode
    monkeypatch.setattr(devices, "IN_PYTHON", [call])
    with FakeTensorMode():
        devices.test_the_tensors_device_is_made_current(call, current, monkeypatch)


@pytest.mark.gpu
def test_same_bits_without_the_binding(monkeypatch):
    import torch

    import embedding_communication_codecs_gb300 as q
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, w = (torch.randn(s, generator=gen, device="cuda") for s in ((70, 264), (48, 264)))
    dy = torch.randn((70, 48), generator=gen, device="cuda").to(torch.bfloat16)
    b = torch.randn(48, generator=gen, device="cuda")

    def everything():
        (xc, xs), (wc, ws) = q.rowwise_int8(x), q.rowwise_int8(w)
        out = [xc, xs, q.rowwise_int8_dequant(xc, xs), q.rowwise_int8_dequant(xc, xs, dtype=torch.float32),
               q.int8_matmul(xc, xs, wc, ws, b), q.int8_matmul(xc[:1], xs[:1], wc, ws, dtype=torch.float32),
               q.int8_input_grad(dy, wc, ws), *q.int8_weight_grad(dy, xc, xs, with_bias=True)]
        saved = q.swiglu_encode(x)
        return out + list(saved) + [q.swiglu_backward(x[:, :132].contiguous(), saved[2], saved[3])]
    bound = everything()
    assert type(q.layer._qcbind).__name__ == "module"
    monkeypatch.setattr(q.layer, "_qcbind", q.layer._Declines())
    for i, (a, c) in enumerate(zip(bound, everything())):
        assert torch.equal(a, c), i
