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
