"""What the 8-bit layer refuses: the Python calls by tensor (ValueError), the C calls by
status.  CPU only: nothing is launched, the C calls' addresses are never followed."""
from __future__ import annotations

import pytest
import torch

import embedding_communication_codecs_gb300 as q

T, N, K = 6, 20, 36
I8 = torch.int8


def codes(r, d):
    return torch.zeros((r, d), dtype=I8), torch.zeros(r)


XC, XS = codes(T, K)
WC, WS = codes(N, K)
DY = torch.zeros((T, N), dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [
    lambda: q.rowwise_int8(torch.zeros(4, 8)),
    lambda: q.rowwise_int8_dequant(XC, XS),
    lambda: q.int8_matmul(XC, XS, WC, WS),
    lambda: q.int8_input_grad(DY, WC, WS),
    lambda: q.int8_weight_grad(DY, XC, XS),
    lambda: q.swiglu_encode(torch.zeros(4, 8)),
    lambda: q.swiglu_backward(torch.zeros(4, 8), torch.zeros((4, 16), dtype=I8), torch.zeros((4, 2))),
])
def test_all_right_but_on_the_host(call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        call()


@pytest.mark.parametrize("call,msg", [
    (lambda: q.rowwise_int8(torch.zeros(8)), "2-D"),
    (lambda: q.rowwise_int8(torch.zeros((4, 8), dtype=torch.float16)), "dtype"),
    (lambda: q.rowwise_int8(torch.zeros(8, 4).t()), "dense along"),
    (lambda: q.rowwise_int8(torch.zeros(8).expand(4, 8)), "overlap"),
    (lambda: q.rowwise_int8_dequant(XC, XS[:5]), "row_scale"),
    (lambda: q.rowwise_int8_dequant(XC, XS.double()), "row_scale"),
    (lambda: q.rowwise_int8_dequant(XC, XS, dtype=torch.float16), "dtype"),
    (lambda: q.rowwise_int8_dequant(XC.to(torch.uint8), XS), "row_codes"),
    (lambda: q.int8_matmul(XC, XS, WC[:, :-1].contiguous(), WS), "rows of 35"),
    (lambda: q.int8_matmul(XC, XS, WC[:, :-1], WS), "contiguous"),
    (lambda: q.int8_matmul(XC, XS, WC, WS[:-1]), "w_scale"),
    (lambda: q.int8_matmul(XC, XS, WC, WS, bias=torch.zeros(N - 1)), "bias"),
    (lambda: q.int8_matmul(XC, XS, WC, WS, bias=torch.zeros(N, dtype=torch.bfloat16)), "bias"),
    (lambda: q.int8_matmul(XC, XS, WC, WS, dtype=torch.int32), "dtype"),
    (lambda: q.int8_matmul(XC.reshape(-1), XS, WC, WS), "2-D"),
    (lambda: q.int8_input_grad(DY.float(), WC, WS), "dy has dtype"),
    (lambda: q.int8_input_grad(DY[:, :-1].contiguous(), WC, WS), "dy has rows of 19"),
    (lambda: q.int8_input_grad(DY.t().contiguous().t(), WC, WS), "dense along"),
    (lambda: q.int8_weight_grad(DY[:-1], XC, XS), "dy has 5 rows"),
    (lambda: q.int8_weight_grad(DY, XC, XS, into=(torch.zeros((N, K), dtype=torch.bfloat16), None)), "dw"),
    (lambda: q.int8_weight_grad(DY, XC, XS, into=(torch.zeros((N, K)), torch.zeros(N + 1))), "dbias"),
    (lambda: q.swiglu_encode(torch.zeros(4, 7)), "even"),
    (lambda: q.swiglu_backward(torch.zeros(4, 8), torch.zeros((4, 8), dtype=I8), torch.zeros((4, 2))), "saved_codes"),
    (lambda: q.swiglu_backward(torch.zeros(4, 8), torch.zeros((4, 16), dtype=I8), torch.zeros((4,))), "saved_scale"),
])
def test_refused_tensors(call, msg):
    with pytest.raises(ValueError, match=msg):
        call()


@pytest.mark.parametrize("call,msg", [
    (lambda: q.qc_rowwise_int8(torch.zeros(4, 8), q.QC_DTYPE_F32, 9, 4, 8, torch.zeros(32, dtype=I8), torch.zeros(4)), "x"),
    (lambda: q.qc_rowwise_int8(torch.zeros(4, 8), q.QC_DTYPE_F32, 8, 4, 8, torch.zeros(31, dtype=I8), torch.zeros(4)), "codes spans"),
    (lambda: q.qc_int8_matmul(XC, XS, WC, WS, None, T, N, K, torch.zeros((T, N)), q.QC_DTYPE_BF16, N, None, 0), "y has dtype"),
    (lambda: q.qc_int8_matmul(XC, XS, WC, WS, None, T, N, K, torch.zeros((T, N)), q.QC_DTYPE_F32, N, torch.zeros(8, dtype=torch.uint8), 9), "workspace spans"),
    (lambda: q.qc_int8_weight_grad(DY, N, XC, XS, T, N, K, torch.zeros(N * K - 1), q.QC_DTYPE_F32, None, 0, None, 0), "dw spans"),
    (lambda: q.qc_swiglu_backward(torch.zeros(T, K), q.QC_DTYPE_F32, K, torch.zeros(2 * T * K, dtype=I8), torch.zeros(2 * T - 1), T, K, torch.zeros(T, 2 * K), 2 * K), "saved_scale spans"),
])
def test_c_names_check_their_tensors(call, msg):
    with pytest.raises(ValueError, match=msg):
        call()


A, B, C, D, E, W = (0x10000000 * (i + 1) for i in range(6))   # addresses that are never followed
BIG = 1 << 40


def mm(**kw):
    a = dict(xc=A, xs=B, wc=C, ws=D, bias=None, T=T, N=N, K=K, y=E, dt=0, ys=N, w=W, wb=BIG)
    a.update(kw)
    return q.lib.qc_int8_matmul(a["xc"], a["xs"], a["wc"], a["ws"], a["bias"], a["T"], a["N"], a["K"], a["y"], a["dt"],
                                a["ys"], a["w"], a["wb"], 0)


def test_matmul_statuses():
    assert mm(dt=2) == q.QC_ERR_INVALID_ARG
    assert mm(N=0) == q.QC_ERR_INVALID_ARG and mm(K=0) == q.QC_ERR_INVALID_ARG
    assert mm(K=(1 << 20) + 1) == q.QC_ERR_UNSUPPORTED and mm(T=(1 << 30) + 1) == q.QC_ERR_UNSUPPORTED
    assert mm(ys=N - 1) == q.QC_ERR_INVALID_ARG and mm(ys=1 << 50) == q.QC_ERR_UNSUPPORTED
    assert mm(xc=None) == q.QC_ERR_NULL and mm(y=None) == q.QC_ERR_NULL
    assert mm(xs=B + 2) == q.QC_ERR_ALIGNMENT and mm(y=E + 2) == q.QC_ERR_ALIGNMENT
    assert mm(y=A) == q.QC_ERR_INVALID_ARG and b"overlaps" in q.lib.qc_last_error()
    assert mm(T=0, xc=None, y=None) == q.QC_OK
    assert q.lib.qc_int8_matmul_workspace(0, 0, 0) == 0


def test_input_grad_statuses():
    def ig(**kw):
        a = dict(dy=A, dys=N, wc=C, ws=D, T=T, N=N, K=K, dx=E, dt=0, dxs=K, w=W, wb=BIG)
        a.update(kw)
        return q.lib.qc_int8_input_grad(a["dy"], a["dys"], a["wc"], a["ws"], a["T"], a["N"], a["K"], a["dx"], a["dt"],
                                        a["dxs"], a["w"], a["wb"], 0)
    assert ig(dys=N - 1) == q.QC_ERR_INVALID_ARG and ig(dxs=K - 1) == q.QC_ERR_INVALID_ARG
    assert ig(dy=A + 1) == q.QC_ERR_ALIGNMENT and ig(dx=None) == q.QC_ERR_NULL
    assert ig(dx=C) == q.QC_ERR_INVALID_ARG and ig(dt=-1) == q.QC_ERR_INVALID_ARG
    assert ig(T=0, dy=None) == q.QC_OK


def test_weight_grad_statuses():
    def wg(**kw):
        a = dict(dy=A, dys=N, xc=C, xs=D, T=T, N=N, K=K, dw=E, dt=0, db=None, fl=0, w=W, wb=BIG)
        a.update(kw)
        return q.lib.qc_int8_weight_grad(a["dy"], a["dys"], a["xc"], a["xs"], a["T"], a["N"], a["K"], a["dw"], a["dt"],
                                         a["db"], a["fl"], a["w"], a["wb"], 0)
    assert wg(fl=1) == q.QC_ERR_INVALID_ARG
    assert wg(fl=q.QC_ACCUMULATE_INTO_OUT, dt=1) == q.QC_ERR_INVALID_ARG
    assert wg(db=E) == q.QC_ERR_INVALID_ARG and wg(db=B + 1) == q.QC_ERR_ALIGNMENT
    assert wg(dw=None) == q.QC_ERR_NULL and wg(dys=N - 1) == q.QC_ERR_INVALID_ARG
    assert wg(T=0, fl=q.QC_ACCUMULATE_INTO_OUT, dy=None) == q.QC_OK
    assert wg(N=1 << 20, K=1 << 20, dys=1 << 20, T=1, dw=None) == q.QC_ERR_NULL   # 2^40 weights are within the limits


def test_row_and_gate_statuses():
    L = q.lib
    assert L.qc_rowwise_int8(A, 0, 8, 4, 0, B, C, 0) == q.QC_ERR_INVALID_ARG
    assert L.qc_rowwise_int8(A, 0, 7, 4, 8, B, C, 0) == q.QC_ERR_INVALID_ARG
    assert L.qc_rowwise_int8(A, 5, 8, 4, 8, B, C, 0) == q.QC_ERR_INVALID_ARG
    assert L.qc_rowwise_int8(A + 2, 0, 8, 4, 8, B, C, 0) == q.QC_ERR_ALIGNMENT
    assert L.qc_rowwise_int8(A, 0, 8, 4, 8, A, C, 0) == q.QC_ERR_INVALID_ARG
    assert L.qc_rowwise_int8(A, 0, 8, 1 << 31, 8, B, C, 0) == q.QC_ERR_UNSUPPORTED
    assert L.qc_rowwise_int8(None, 0, 8, 0, 8, None, None, 0) == q.QC_OK
    assert L.qc_rowwise_int8_dequant(A, B, 4, 8, C, 0, 7, 0) == q.QC_ERR_INVALID_ARG
    assert L.qc_rowwise_int8_dequant(A, B, 4, 8, A, 0, 8, 0) == q.QC_ERR_INVALID_ARG
    assert L.qc_swiglu_encode(A, 0, 15, 4, 8, B, C, D, E, 0) == q.QC_ERR_INVALID_ARG
    assert L.qc_swiglu_encode(A, 0, 16, 4, 8, B, C, B, E, 0) == q.QC_ERR_INVALID_ARG
    assert L.qc_swiglu_encode(A, 0, 16, 4, 8, B, C, D, None, 0) == q.QC_ERR_NULL
    assert L.qc_swiglu_backward(A, 1, 8, B, C, 4, 8, D, 15, 0) == q.QC_ERR_INVALID_ARG
    assert L.qc_swiglu_backward(A, 1, 8, B, C, 4, 8, A, 16, 0) == q.QC_ERR_INVALID_ARG
    assert L.qc_swiglu_backward(None, 1, 8, None, None, 0, 8, None, 16, 0) == q.QC_OK
