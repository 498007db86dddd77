"""Calls whose waits between warps run out, from a few cycles on: they end, say so, and leave what runs
behind them on the GPU alone.

A call with an armed bound may also come through, where nothing had to be waited for that long: then
its status is clear and its result is the usual one.  The calls queued behind it are compared bit for
bit; no wait of the host lies between them, so that they take over shared memory and tensor memory
as soon as the block that gave up frees them.
"""
import pytest
import torch

import linear_attention_layer_causal_b200 as gdn
import ops_ref as ref

LIMITS = (1, 40, 200, 600, 1500, 4000)


def operands(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    a, sa = ref.quant(torch.randn(M, K, generator=g).cuda(), 1)
    w, sw = ref.quant(torch.randn(N, K, generator=g).cuda(), 128)
    return a, sa, w, sw


def workspace(M, N, K):
    return torch.empty(gdn.matmul_fp8_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")


def given_up(ws, got, want):
    status = gdn.prefill_status(ws)[0]
    assert status in (gdn.GDN_OK, gdn.GDN_ERR_TIMEOUT)
    if status == gdn.GDN_OK:
        assert torch.equal(got, want)
    return status == gdn.GDN_ERR_TIMEOUT


# few rows (a cluster's blocks, with one block of k each and with several) and many; K so short that
# every load is on its way before a role gives up, and longer
@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (1, 12352, 2048), (5, 300, 512), (16, 4096, 1024), (33, 1000, 512), (60, 640, 4096),
                                   (100, 1000, 768), (3000, 4096, 128), (3000, 4096, 256), (3000, 4096, 512), (2100, 2400, 1536)])
def test_products_that_give_up(M, N, K):
    a, sa, w, sw = operands(M, N, K, 1)
    small = operands(3, 520, 640, 2)
    want, want_small = gdn.matmul_fp8(a, sa, w, sw), gdn.matmul_fp8(*small)
    times = 0
    for limit in LIMITS:
        wss, got, behind = [workspace(M, N, K) for _ in range(4)], [], []
        for ws in wss:
            gdn.wait_limit_next_call(limit)
            got.append(gdn.matmul_fp8(a, sa, w, sw, workspace=ws))
            behind.append((gdn.matmul_fp8(*small), gdn.matmul_fp8(a, sa, w, sw)))
        for ws, g, (s, b) in zip(wss, got, behind):
            times += given_up(ws, g, want)
            assert torch.equal(s, want_small) and torch.equal(b, want)
    assert times > 0  # a bound of a cycle is below any copy's time
