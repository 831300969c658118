"""int8_weight_grad(into=...) and the arguments that it leaves without a meaning."""
from __future__ import annotations

import pytest
import torch

import embedding_communication_codecs_gb300 as q

T, N, K = 6, 20, 36
DY, XC, XS = torch.zeros((T, N), dtype=torch.bfloat16), torch.zeros((T, K), dtype=torch.int8), torch.zeros(T)
DW, DB = torch.zeros((N, K)), torch.zeros(N)


@pytest.mark.parametrize("kw,msg", [
    (dict(into=(DW, None), dtype=torch.bfloat16), "dtype"),
    (dict(into=(DW, DB), dtype=torch.bfloat16), "dtype"),
    (dict(into=(DW, None), with_bias=True), "with_bias"),
])
def test_contradictions_are_refused(kw, msg):
    with pytest.raises(ValueError, match=msg):
        q.int8_weight_grad(DY, XC, XS, **kw)


@pytest.mark.parametrize("kw", [dict(into=(DW, DB)), dict(into=(DW, DB), with_bias=True), dict(into=(DW, None)),
                                dict(into=(DW, DB), dtype=torch.float32)])
def test_the_rest_goes_on_to_the_device_check(kw):
    with pytest.raises(ValueError, match="CUDA tensor"):
        q.int8_weight_grad(DY, XC, XS, **kw)
