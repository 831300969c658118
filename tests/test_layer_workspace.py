"""The forward product's scratch memory: codes that are read where they lie take no copies."""
from __future__ import annotations

import pytest
import torch

import embedding_communication_codecs_gb300 as q

A, B, C, D, E, W = (0x10000000 * (i + 1) for i in range(6))   # addresses that are never followed
SIZES = [(17, 28672, 4096), (48, 11000, 4096), (128, 1024, 1024), (300, 4096, 4096), (500, 4096, 4096), (600, 4096, 4096), (40, 64, 100),
         (1000, 1024, 1024), (8, 512, 512), (40, 300, 16384)]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_sizes(T, N, K):
    anywhere = q.qc_int8_matmul_workspace(T, N, K)
    in_place = q.qc_int8_matmul_codes_workspace(A, C, T, N, K)
    assert in_place <= anywhere
    for x, w in ((A + 1, C), (A, C + 8), (A + 4, C + 4)):
        assert q.qc_int8_matmul_codes_workspace(x, w, T, N, K) <= anywhere
    if K % 16:
        assert in_place == q.qc_int8_matmul_codes_workspace(A + 1, C, T, N, K)
    elif T <= 384:
        # at most the partial sums of a cut contraction, in whole 32s
        assert in_place <= 2 * 152 * 128 * 128 * 4 and in_place % 4096 == 0
    assert q.qc_int8_matmul_codes_workspace(A, C, 5, 0, 0) == 0


def status(x, w, nbytes, T, N, K):
    """With a missing y: QC_ERR_NULL says that the workspace was found large enough."""
    return q.lib.qc_int8_matmul(x, B, w, D, None, T, N, K, None, q.QC_DTYPE_F32, N, W, nbytes, 0)


@pytest.mark.parametrize("T,N,K", [s for s in SIZES if s[0] > 16])
def test_what_the_call_asks_for(T, N, K):
    for x, w in ((A, C), (A + 1, C), (A, C + 8)):
        need = q.qc_int8_matmul_codes_workspace(x, w, T, N, K)
        assert status(x, w, need, T, N, K) == q.QC_ERR_NULL
        if need:
            assert status(x, w, need - 1, T, N, K) == q.QC_ERR_INVALID_ARG
            assert b"workspace" in q.lib.qc_last_error()
    assert status(A + 1, C, q.qc_int8_matmul_workspace(T, N, K), T, N, K) == q.QC_ERR_NULL


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 8])
@pytest.mark.parametrize("T,N,K", [(17, 4096, 4096), (48, 11000, 4096), (500, 4096, 4096), (500, 300, 4112), (40, 300, 16384), (40, 300, 4097)])
def test_the_call_stays_inside_it(T, N, K, shift):
    gen = torch.Generator(device="cuda").manual_seed(T + K)

    def codes(rows):
        base = torch.randint(-16, 17, (rows * K + 16,), generator=gen, device="cuda", dtype=torch.int8)
        return base[shift:shift + rows * K].view(rows, K)
    x, w = codes(T), codes(N)
    one_t, one_n = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
    need = q.qc_int8_matmul_codes_workspace(x, w, T, N, K)
    room = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    y = torch.empty((T, N), device="cuda")
    q.qc_int8_matmul(x, one_t, w, one_n, None, T, N, K, y, q.QC_DTYPE_F32, N, room[:need] if need else None, need)
    assert torch.equal(y.double(), x.double() @ w.double().t())
    assert bool((room[need:] == 0x5A).all())
    assert torch.equal(q.int8_matmul(x, one_t, w, one_n, dtype=torch.float32), y)


@pytest.mark.gpu
def test_aligned_codes_allocate_no_copies():
    T, N, K = 48, 11000, 4096
    x = torch.ones((T, K), dtype=torch.int8, device="cuda")
    w = torch.ones((N, K), dtype=torch.int8, device="cuda")
    one_t, one_n = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    y = q.int8_matmul(x, one_t, w, one_n)
    assert torch.cuda.max_memory_allocated() - before <= y.numel() * 2 + (2 << 20)
