"""Hang detection on the GPU, without hanging it: every pipeline wait of the
tcgen05 kernels gives up after a limit and reports GPT2_ERR_TIMEOUT in a
device status word.  With the limit set to one nanosecond every wait that is
not already satisfied (after the hardware's own short suspension inside one
try-wait) gives up, so a long GEMM takes the abort path (copies and
MMAs in flight are drained, tensor memory is freed, the kernel returns);
afterwards, with the default limit, the same call on the same context
computes the right result."""
import numpy as np
import pytest
import torch

import decoder_only_transformer_step_b200 as gp

pytestmark = pytest.mark.gpu

DEV_ERR_TIMEOUT = 4


def _operands(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    A = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    B = torch.randn(N, K, generator=g).to(torch.bfloat16).cuda()
    return A, B


@pytest.mark.parametrize("bn", [256, 128])
def test_timeout_is_reported_and_the_context_recovers(bn):
    # single-CTA tiles with a 1024-k-block loop (about 0.3 ms of MMAs per
    # tile): the epilogue's wait for the accumulator cannot complete inside
    # the hardware's own suspension of a single try-wait
    M, N, K = 256, 256, 65536
    A, B = _operands(M, N, K, 7 + bn)
    C = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        gp.gpt2_set_wait_timeout_ns(1)
        gp.gpt2_op_gemm_bf16_status(A, 0, K, B, 0, K, C, 0, N, M, N, K, bn=bn, splits=1, status=status)
        torch.cuda.synchronize()
    finally:
        gp.gpt2_set_wait_timeout_ns(0)
    assert int(status.item()) & DEV_ERR_TIMEOUT
    status.zero_()
    gp.gpt2_op_gemm_bf16_status(A, 0, K, B, 0, K, C, 0, N, M, N, K, bn=bn, splits=1, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ref = A.float() @ B.float().t()
    assert (C.float() - ref).abs().max().item() <= 1e-2 * ref.abs().max().item()


def test_a_choice_whose_blocks_do_not_meet_in_time_is_no_token():
    # 8 blocks share a row.  The whole history lies in the last one's ids, thousands of them and one again and again,
    # so that block 0 has long been waiting when it reports; with the limit at one nanosecond it gives up.
    rows, V, H = 4, 262144, 262143
    g = torch.Generator().manual_seed(5)
    z = torch.randn(rows, V, generator=g).cuda()
    h = torch.full((rows, H), V - 1, dtype=torch.int32)
    h[:, :H // 2] = torch.randint(7 * V // 8, V, (rows, H // 2), generator=g, dtype=torch.int32)
    n0 = H - 1
    hist, n = h.cuda(), torch.full((rows,), n0, dtype=torch.int32, device="cuda")
    rules = gp.LogitRules(history=hist, history_len=n, presence=torch.ones(rows, device="cuda"), append=True)

    def call():
        out = torch.zeros(rows, V, device="cuda")
        nxt = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
        pos = torch.arange(rows, dtype=torch.int32, device="cuda")
        n.fill_(n0)
        hist[:, n0] = -7
        gp.gpt2_op_logit_rules(z, V, out, V, rows, V, rules, nxt, pos)
        torch.cuda.synchronize()
        return out, nxt.tolist(), pos.tolist(), n.tolist(), hist[:, n0].tolist()
    try:
        gp.gpt2_set_wait_timeout_ns(1)
        out, nxt, pos, length, last = call()
    finally:
        gp.gpt2_set_wait_timeout_ns(0)
    out2, nxt2, pos2, length2, last2 = call()
    want = z.clone()
    for r in range(rows):
        want[r, h[r, :n0].long().unique().cuda()] -= 1
    assert torch.equal(out2, want) and torch.equal(out, want)     # the logits do not wait for one another
    assert nxt2 == want.argmax(1).tolist() == last2
    assert pos2 == [r + 1 for r in range(rows)] and length2 == [n0 + 1] * rows
    assert -1 in nxt
    for r in range(rows):
        if nxt[r] == -1:
            assert (pos[r], length[r], last[r]) == (r, n0, -7)
        else:
            assert (nxt[r], pos[r], length[r], last[r]) == (nxt2[r], r + 1, n0 + 1, nxt2[r])


@pytest.mark.parametrize("hd,B", [(128, 256), (64, 100)])     # two row tiles, one
def test_prefix_attention_whose_waits_run_out_is_nan_and_the_context_recovers(hd, B):
    # the queries are read from pinned host memory: megabytes over the bus, for which the tensor cores' warps and the
    # copies of the keys wait tens of microseconds
    P = 40000 if hd == 128 else 60000
    g = torch.Generator().manual_seed(hd)
    q = torch.randn(B, hd, generator=g).bfloat16().pin_memory()
    pk, pv = (torch.randn(1, P, hd, generator=g).bfloat16().cuda() for _ in range(2))
    n = gp.gpt2_op_prefix_attention_scratch_bytes(B, 1, 1, hd, P, 0)
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(q):
        o = torch.zeros(B, hd, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(B, 1, device="cuda")
        torch.cuda.synchronize()
        rc = gp._lib().gpt2_op_prefix_attention_bf16(q.data_ptr(), hd, pk.data_ptr(), pv.data_ptr(), P, P, None, None, None,
                                                     0, o.data_ptr(), hd, lse.data_ptr(), scratch.data_ptr(), n, B, 1, 1,
                                                     hd, torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        return o, lse[:, 0]
    o, lse = call(q.cuda())
    try:
        gp.gpt2_set_wait_timeout_ns(1)
        o1, lse1 = call(q)
    finally:
        gp.gpt2_set_wait_timeout_ns(0)
    gone = torch.isnan(lse1)
    assert bool(gone.any())
    assert bool(torch.isnan(o1[gone]).all())
    assert torch.equal(o1[~gone], o[~gone]) and torch.equal(lse1[~gone], lse[~gone])
    o2, lse2 = call(q)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    z = q.cuda().double() @ pk[0].double().t() / hd**0.5
    assert bool(((o.double() - torch.softmax(z, 1) @ pv[0].double()).abs() <= 2e-2).all())
