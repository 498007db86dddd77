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


def mixer(lens, P, S, dtype, segments, gate, seed):
    cfg = gdn.SsmConfig(2, 6, P, S, act_dtype=dtype, segments=segments)
    g = torch.Generator().manual_seed(seed)
    act = torch.bfloat16 if dtype == "bf16" else torch.float32
    N, B, C = sum(lens), len(lens), cfg.conv_dim
    cu = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    xbc, dt, z = (torch.randn(*s, generator=g).cuda().to(act) for s in ((N, C), (N, 6), (N, 6, P)))
    kw = dict(conv_b=0.1 * torch.randn(C, generator=g).cuda(), dt_bias=torch.randn(6, generator=g).cuda() - 3,
              D=torch.randn(6, generator=g).cuda(), z=z if gate else None,
              initial_state=0.1 * torch.randn(B, 6, P, S, generator=g).cuda(), initial_conv=torch.randn(B, 3, C, generator=g).cuda().to(act))
    conv_w, A_log = 0.5 * torch.randn(C, 4, generator=g).cuda(), torch.rand(6, generator=g).cuda()

    def call(ws=None):
        out = gdn.ssm_prefill(cfg, xbc, dt, cu, conv_w, A_log, return_final_state=True, workspace=ws, **kw)
        return torch.cat([out["y"].float().flatten(), out["final_state"].flatten()])
    return call, gdn.ssm_prefill_workspace_size(cfg, B, N)


# one chunk (the loading warp never waits), a few, many, and sequences of both kinds in one batch
@pytest.mark.gpu
@pytest.mark.parametrize("lens,segments", [([37], 1), ([64, 1, 0], 1), ([200], 1), ([130, 20], 2), ([1500], 1), ([1500, 64], 5)])
@pytest.mark.parametrize("P,S,dtype,gate", [(64, 64, "bf16", True), (64, 128, "f32", True), (128, 64, "bf16", False), (128, 128, "bf16", True)])
def test_prompts_that_give_up(lens, segments, P, S, dtype, gate):
    call, need = mixer(lens, P, S, dtype, segments, gate, 5)
    small = operands(3, 520, 640, 2)
    want, want_small = call(), gdn.matmul_fp8(*small)
    times = 0
    for limit in LIMITS:
        wss, got, behind = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(3)], [], []
        for ws in wss:
            gdn.wait_limit_next_call(limit)
            got.append(call(ws))
            behind.append((gdn.matmul_fp8(*small), call()))
        for ws, g, (s, b) in zip(wss, got, behind):
            times += given_up(ws, g, want)
            assert torch.equal(s, want_small) and torch.equal(b, want)
    assert times > 0 or max(lens) <= 200  # its waits sleep some microseconds before they look at the bound


@pytest.mark.gpu
def test_a_call_without_work_takes_the_armed_bound():
    """The bound is for the next call, whatever that has to do: the one after it runs unbounded again."""
    a, sa, w, sw = operands(100, 1000, 768, 1)
    want, ws = gdn.matmul_fp8(a, sa, w, sw), workspace(100, 1000, 768)
    call, need = mixer([1500], 64, 64, "bf16", 1, True, 5)
    cfg = gdn.SsmConfig(2, 6, 64, 64)
    none = torch.empty(0, cfg.conv_dim, dtype=torch.bfloat16, device="cuda")
    want_y, ws_y = call(), torch.empty(need, dtype=torch.uint8, device="cuda")
    empty = [lambda: gdn.matmul_fp8(a[:0], sa[:0], w, sw), lambda: gdn.matmul_fp8(a, sa, w[:0], sw[:0]),
             lambda: gdn.ssm_prefill(cfg, none, none[:, :6], torch.zeros(1, dtype=torch.int32, device="cuda"),
                                     torch.zeros(cfg.conv_dim, 4, device="cuda"), torch.zeros(6, device="cuda"))]
    for nothing in empty:
        gdn.wait_limit_next_call(1)
        nothing()
        got = gdn.matmul_fp8(a, sa, w, sw, workspace=ws)
        assert gdn.prefill_status(ws) == (gdn.GDN_OK, 0) and torch.equal(got, want)
        gdn.wait_limit_next_call(1)
        nothing()
        got = call(ws_y)
        assert gdn.prefill_status(ws_y) == (gdn.GDN_OK, 0) and torch.equal(got, want_y)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 300, 256), (16, 128, 1024), (1000, 4096, 256)])
def test_every_call_that_gave_up_says_so(M, N, K):
    """Many short calls with a bound of a cycle, each with status words that an earlier call left set: whatever
    block's wait runs out first, a wrong result never comes with a clear status."""
    a, sa, w, sw = operands(M, N, K, 3)
    want = gdn.matmul_fp8(a, sa, w, sw)
    words = torch.full((300, gdn.matmul_fp8_workspace_size(M, N, K)), 255, dtype=torch.uint8, device="cuda")
    outs = []
    for ws in words:
        gdn.wait_limit_next_call(1)
        outs.append(gdn.matmul_fp8(a, sa, w, sw, workspace=ws))
    words = words[:, :8].contiguous().view(torch.int32).tolist()
    for (status, detail), out in zip(words, outs):
        assert status in (0, 1) and detail == 0
        assert status == 1 or torch.equal(out, want)
