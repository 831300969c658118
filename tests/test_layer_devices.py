"""A call of the 8-bit layer runs on its tensors' device: operands on two devices are refused,
and where the tensors' device is not the current one, it is made current around the call.

CPU only: the tensors are torch's fake ones, which have a device and no memory; nothing is
launched."""
from __future__ import annotations

import contextlib

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import embedding_communication_codecs_gb300 as q
from embedding_communication_codecs_gb300 import layer

T, N, K = 6, 20, 36
I8, F32, BF16 = torch.int8, torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def fake():
    with FakeTensorMode():
        yield


def at(device):
    """The tensors of every call, by name, all on cuda:0 but those named in `device`."""
    def t(name, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=f"cuda:{device.get(name, 0)}")
    return dict(
        x=t("x", (T, K), F32), xc=t("xc", (T, K), I8), xs=t("xs", (T,), F32), wc=t("wc", (N, K), I8), ws=t("ws", (N,), F32),
        bias=t("bias", (N,), F32), dy=t("dy", (T, N), BF16), y=t("y", (T, N), F32), dx=t("dx", (T, K), F32),
        dw=t("dw", (N, K), F32), db=t("db", (N,), F32), gu=t("gu", (T, 2 * K), F32), dh=t("dh", (T, K), F32),
        sc=t("sc", (T, 2 * K), I8), ss=t("ss", (T, 2), F32), hc=t("hc", (T, K), I8), hs=t("hs", (T,), F32),
        work=t("work", (1 << 20,), torch.uint8))


CALLS = {
    "rowwise_int8_dequant": (("xc", "xs"), lambda a: q.rowwise_int8_dequant(a["xc"], a["xs"])),
    "int8_matmul": (("xc", "xs", "wc", "ws", "bias"), lambda a: q.int8_matmul(a["xc"], a["xs"], a["wc"], a["ws"], a["bias"])),
    "int8_input_grad": (("dy", "wc", "ws"), lambda a: q.int8_input_grad(a["dy"], a["wc"], a["ws"])),
    "int8_weight_grad": (("dy", "xc", "xs"), lambda a: q.int8_weight_grad(a["dy"], a["xc"], a["xs"])),
    "int8_weight_grad into": (("dy", "xc", "xs", "dw", "db"),
                              lambda a: q.int8_weight_grad(a["dy"], a["xc"], a["xs"], into=(a["dw"], a["db"]))),
    "swiglu_backward": (("dh", "sc", "ss"), lambda a: q.swiglu_backward(a["dh"], a["sc"], a["ss"])),
    "qc_rowwise_int8": (("x", "xc", "xs"), lambda a: q.qc_rowwise_int8(a["x"], q.QC_DTYPE_F32, K, T, K, a["xc"], a["xs"])),
    "qc_rowwise_int8_dequant": (("xc", "xs", "dx"),
                                lambda a: q.qc_rowwise_int8_dequant(a["xc"], a["xs"], T, K, a["dx"], q.QC_DTYPE_F32, K)),
    "qc_int8_matmul": (("xc", "xs", "wc", "ws", "bias", "y", "work"),
                       lambda a: q.qc_int8_matmul(a["xc"], a["xs"], a["wc"], a["ws"], a["bias"], T, N, K, a["y"], q.QC_DTYPE_F32, N,
                                                  a["work"], 1 << 20)),
    "qc_int8_input_grad": (("dy", "wc", "ws", "dx", "work"),
                           lambda a: q.qc_int8_input_grad(a["dy"], N, a["wc"], a["ws"], T, N, K, a["dx"], q.QC_DTYPE_F32, K, a["work"],
                                                          1 << 20)),
    "qc_int8_weight_grad": (("dy", "xc", "xs", "dw", "db", "work"),
                            lambda a: q.qc_int8_weight_grad(a["dy"], N, a["xc"], a["xs"], T, N, K, a["dw"], q.QC_DTYPE_F32, a["db"], 0,
                                                            a["work"], 1 << 20)),
    "qc_swiglu_encode": (("gu", "hc", "hs", "sc", "ss"),
                         lambda a: q.qc_swiglu_encode(a["gu"], q.QC_DTYPE_F32, 2 * K, T, K, a["hc"], a["hs"], a["sc"], a["ss"])),
    "qc_swiglu_backward": (("dh", "sc", "ss", "gu"),
                           lambda a: q.qc_swiglu_backward(a["dh"], q.QC_DTYPE_F32, K, a["sc"], a["ss"], T, K, a["gu"], 2 * K)),
}


@pytest.mark.parametrize("call,other", [(c, n) for c, (names, _) in CALLS.items() for n in names])
def test_operands_on_two_devices_are_refused(call, other):
    with pytest.raises(ValueError, match="cuda:1"):
        CALLS[call][1](at({other: 1}))


SINGLE = {"rowwise_int8": (("x",), lambda a: q.rowwise_int8(a["x"])), "swiglu_encode": (("gu",), lambda a: q.swiglu_encode(a["gu"]))}


# the calls that Python can make as well as the binding
IN_PYTHON = [c for c in [*CALLS, *SINGLE] if c not in ("rowwise_int8_dequant", "int8_matmul")]


@pytest.mark.parametrize("call", IN_PYTHON)
@pytest.mark.parametrize("current", [0, 1])
def test_the_tensors_device_is_made_current(call, current, monkeypatch):
    """What goes through Python (the binding's own guard is in its source): the C call is
    made with the tensors' device current, on that device's current stream."""
    names, run = {**CALLS, **SINGLE}[call]
    now = [current]
    seen = []

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        yield
        now[0] = before

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_workspace"):
                return lambda *a: 0
            return lambda *a: seen.append((now[0], a[-1])) or q.QC_OK

    class Declines:
        def __getattr__(self, name):
            return lambda *a: None

    class Stream:
        def __init__(self):
            self.cuda_stream = 1000 + now[0]

    monkeypatch.setattr(layer, "lib", Lib())
    monkeypatch.setattr(layer, "_qcbind", Declines())
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 256)
    run(at({n: 1 for n in names}))
    assert seen == [(1, 1001)] and now[0] == current


@pytest.mark.parametrize("call", [c for c in [*CALLS, *SINGLE] if not c.startswith("qc_")])
def test_a_stream_of_another_device_is_refused(call):
    names, _ = {**CALLS, **SINGLE}[call]

    class Stream:
        device = torch.device("cuda:0")
        cuda_stream = 7
    a = at({n: 1 for n in names})
    args = [a[n] for n in names if n not in ("dw", "db")]
    kw = {"into": (a["dw"], a["db"])} if "dw" in names else {}
    with pytest.raises(ValueError, match="stream"):
        getattr(q, call.split()[0])(*args, stream=Stream(), **kw)
