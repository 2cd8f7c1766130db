"""Refusals and sizes of the serving operators (4-bit weights, attention over a
shared prefix, rules on logits), all decided on the host: no GPU needed."""
import ctypes

import pytest

import decoder_only_transformer_step_b200 as gp
from decoder_only_transformer_step_b200 import build_lib

INVALID = gp.ERRORS_BY_NAME["GPT2_ERR_INVALID_ARG"]
SHAPE = gp.ERRORS_BY_NAME["GPT2_ERR_UNSUPPORTED_SHAPE"]
WORKSPACE = gp.ERRORS_BY_NAME["GPT2_ERR_WORKSPACE"]
A = 1 << 20  # an aligned address that no call below gets to read


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return gp._lib()


def test_q4_sizes(L):
    assert gp.gpt2_op_q4_packed_bytes(5, 64) == 5 * 32
    assert gp.gpt2_op_q4_scale_count(5, 64, 32) == 2 * 8
    assert gp.gpt2_op_q4_scale_count(8, 128, 128) == 8
    for n, k, g in [(0, 64, 32), (5, 0, 32), (5, 48, 32), (5, 96, 64), (5, 64, 16), (5, 64, 0), (-1, 64, 32)]:
        assert gp.gpt2_op_q4_scale_count(n, k, g) == 0
    assert gp.gpt2_op_q4_packed_bytes(70000, 65536) == 70000 * 32768  # past 32 bits


def test_q4_model_bytes(L):
    cfg = gp.GPT2_124M.c()
    mats = [(3 * 768, 768), (768, 768), (4 * 768, 768), (768, 4 * 768)]
    pad = lambda b: (b + 255) // 256 * 256  # noqa: E731
    for g in (32, 64, 128):
        one = lambda n, k: pad(n * k // 2) + pad(k // g * n * 2)  # noqa: E731
        assert gp.gpt2_q4_bytes(cfg, g) == 12 * sum(one(*m) for m in mats) + one(50304, 768)
    assert gp.gpt2_q4_bytes(cfg, 48) == 0
    assert gp.gpt2_q4_bytes(gp.GPT2_1558M.c(), 128) == 0      # d 1600 is no multiple of 128
    assert gp.gpt2_q4_bytes(gp.GPT2_1558M.c(), 64) > 0
    assert gp.gpt2_q4_bytes(gp.GPT2_TINY.c(), 32) == 0        # fp32 mode


def test_quantize_refusals(L):
    def q(w=A, w32=1, ldw=64, N=4, K=64, g=32, p=A, s=A):
        return L.gpt2_op_q4_quantize(w, w32, ldw, N, K, g, p, s, None)
    assert q(w=None) == q(p=None) == q(s=None) == INVALID
    assert q(w=A + 4) == q(p=A + 8) == q(s=A + 2) == INVALID
    assert q(N=-1) == q(K=-64) == q(ldw=32) == INVALID
    assert q(K=48) == q(g=48) == q(g=0) == q(ldw=68) == q(K=0) == SHAPE
    assert q(N=0) == 0

    def d(p=A, s=A, N=4, K=64, g=32, o=A, ldo=64):
        return L.gpt2_op_q4_dequantize(p, s, N, K, g, o, 0, ldo, None)
    assert d(p=None) == d(s=None) == d(o=None) == d(o=A + 4) == d(ldo=32) == d(N=-2) == INVALID
    assert d(K=80, ldo=80) == d(ldo=65) == d(g=16) == SHAPE
    assert d(N=0) == 0


def test_gemv_refusals(L):
    def f(x=A, ldx=64, p=A, s=A, b=None, o=A, o32=0, ldo=8, rows=1, N=8, K=64, g=32):
        return L.gpt2_op_gemv_q4(x, ldx, p, s, b, o, o32, ldo, rows, N, K, g, None)
    assert f(x=None) == f(p=None) == f(s=None) == f(o=None) == INVALID
    assert f(rows=17) == f(rows=-1) == f(N=-1) == f(ldx=32) == f(ldo=7) == INVALID
    assert f(x=A + 8) == f(p=A + 4) == f(s=A + 2) == f(b=A + 1) == f(o=A + 1) == f(o=A + 2, o32=1) == INVALID
    assert f(K=48) == f(g=40) == f(ldx=68) == f(K=0) == SHAPE
    assert f(K=32768 + 32, ldx=40000) == SHAPE
    assert f(rows=0) == f(N=0) == 0


def test_prefix_refusals_and_scratch(L):
    size = gp.gpt2_op_prefix_attention_scratch_bytes
    assert size(2, 4, 4, 64, 100, 10) > 0
    for a in [(0, 4, 4, 64, 1, 1), (2, 4, 3, 64, 1, 1), (2, 4, 4, 32, 1, 1), (2, 4, 4, 64, -1, 1), (2, 4, 4, 64, 1, -1)]:
        assert size(*a) == 0
    assert size(1, 1, 1, 64, 0, 0) > 0

    def f(q=A, ldq=256, pk=A, pv=A, P=8, cap=8, k=A, v=A, n=A, m=4, o=A, ldo=256, lse=None, s=A, sb=1 << 40, B=2, Hq=4,
          Hkv=4, hd=64):
        return L.gpt2_op_prefix_attention_bf16(q, ldq, pk, pv, P, cap, k, v, n, m, o, ldo, lse, s, sb, B, Hq, Hkv, hd,
                                               None)
    assert f(q=None) == f(pk=None) == f(pv=None) == f(k=None) == f(v=None) == f(n=None) == f(o=None) == f(s=None) == INVALID
    assert f(cap=7) == f(P=-1) == f(m=-1) == f(B=-1) == f(Hkv=0) == f(Hq=0) == INVALID
    assert f(ldq=255) == f(ldo=128) == f(ldq=257) == f(ldo=257) == INVALID
    assert f(q=A + 2) == f(o=A + 2) == f(pk=A + 8) == f(v=A + 8) == f(lse=A + 2) == f(s=A + 8) == INVALID
    assert f(hd=32) == f(Hq=6, Hkv=4) == SHAPE
    assert f(sb=size(2, 4, 4, 64, 8, 4) - 1) == WORKSPACE
    assert f(B=0) == 0


def test_logit_rules_refusals(L):
    def f(z=A, ld=100, o=A, ldo=100, rows=2, V=100, nxt=A, pos=None, null=False, **r):
        c = gp.gpt2_logit_rules(**r)
        return L.gpt2_op_logit_rules(z, ld, o, ldo, rows, V, None if null else ctypes.byref(c), nxt, pos, None)
    assert f(z=None) == f(o=None) == f(null=True) == f(ld=99) == f(ldo=99) == f(rows=-1) == f(V=-1) == INVALID
    assert f(ldo=101) == INVALID                                   # in place with another pitch
    assert f(nxt=None, pos=A) == INVALID
    assert f(history=A) == f(history=A, history_len=A) == INVALID  # no lengths, no pitch
    assert f(append=1) == f(nxt=None, history=A, history_len=A, history_ld=4, append=1) == INVALID
    assert f(n_bias=3) == f(n_bias=-1) == f(n_bias=2, bias_ids=A) == INVALID
    assert f(allowed=A, allowed_ld=3) == f(presence=A + 2) == f(z=A + 1) == INVALID
    assert f(n_bias=4096, bias_ids=A, bias_values=A) == SHAPE
    assert f(history=A, history_len=A, history_ld=262144) == SHAPE
    assert f(V=262145, ld=400000, ldo=400000) == SHAPE
    assert f(rows=0) == f(V=0) == 0


def test_model_calls_refuse_a_null_context(L):
    assert L.gpt2_q4_pack(None, A, 1 << 30, 64, None) == INVALID
    assert L.gpt2_decode_step_ex(None, A, 1 << 30, 1, 1, A, A, None, A, None) == INVALID
    assert L.gpt2_rules_next(None, A, 1, ctypes.byref(gp.gpt2_logit_rules()), A, None, None) == INVALID
    cfg = gp.GPT2_124M.c()
    assert gp.gpt2_decode_scratch_bytes(cfg, 16, 100, 500) == gp.gpt2_op_prefix_attention_scratch_bytes(16, 12, 12, 64, 500, 100)
    for a in [(17, 100, 500), (16, 100, 925), (16, 0, 500), (16, 100, 0)]:
        assert gp.gpt2_decode_scratch_bytes(cfg, *a) == 0


def test_binding_refuses_host_short_and_mistyped_buffers(L):
    import torch
    x = torch.zeros(64, dtype=torch.bfloat16)
    p, s = torch.zeros(8 * 32, dtype=torch.uint8), torch.zeros(16, dtype=torch.bfloat16)
    o = torch.zeros(8, dtype=torch.bfloat16)
    with pytest.raises(gp.Gpt2Error, match="not on the current CUDA device"):
        gp.gpt2_op_gemv_q4(x, 64, p, s, None, o, 0, 8, 1, 8, 64, 32)
    with pytest.raises(gp.Gpt2Error, match="x is torch.float32"):
        gp.gpt2_op_gemv_q4(x.float(), 64, p, s, None, o, 0, 8, 1, 8, 64, 32)
    with pytest.raises(gp.Gpt2Error, match="is missing"):
        gp.gpt2_op_gemv_q4(None, 64, p, s, None, o, 0, 8, 1, 8, 64, 32)
    with pytest.raises(gp.Gpt2Error, match="belong together"):
        gp.LogitRules(bias_ids=torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(gp.Gpt2Error, match="needs history_len"):
        gp.LogitRules(history=torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(gp.Gpt2Error, match="rules are for"):
        gp.LogitRules(presence=torch.zeros(2), frequency=torch.zeros(3))


def test_binding_refuses_views_that_repeat_elements():
    # an expanded tensor counts more elements than its memory holds
    import torch
    one = torch.zeros(1, dtype=torch.bfloat16)
    with pytest.raises(gp.Gpt2Error, match="holds 1 elements, 64 are needed"):
        gp._buf("f", "bias", one.expand(64), torch.bfloat16, -1, 64)
    with pytest.raises(gp.Gpt2Error, match="holds 8 elements, 32 are needed"):
        gp._buf("f", "x", torch.zeros(8).expand(4, 8), torch.float32, -1, 32)
    rows = torch.zeros(4, 16)
    assert gp._buf("f", "x", rows[:, :8], torch.float32, -1, 56) == rows.data_ptr()
    assert gp._buf("f", "x", rows, torch.float32, -1, 64) == rows.data_ptr()
    assert gp._buf("f", "x", rows.t(), torch.float32, -1, 64) == rows.data_ptr()
    with pytest.raises(gp.Gpt2Error, match="scratch holds 1 elements, 4096 are needed"):
        gp._scratch("f", torch.zeros(1, dtype=torch.uint8).expand(4096), torch.uint8, -1)


def test_sizes_near_the_end_of_32_bits_are_refused(L):
    # offsets of parts and tiles are formed from them by additions in 32 bits
    big = 2**31 - 1
    assert gp.gpt2_op_prefix_attention_scratch_bytes(1, 1, 1, 16, 2**30, 0) > 0
    assert gp.gpt2_op_prefix_attention_scratch_bytes(1, 1, 1, 16, big, 0) == 0
    assert gp.gpt2_op_prefix_attention_scratch_bytes(1, 1, 1, 16, 0, big) == 0
    call = lambda P, m: L.gpt2_op_prefix_attention_bf16(  # noqa: E731
        A, 16, A, A, P, big, A, A, A, m, A, 16, None, A, 1 << 40, 1, 1, 1, 16, None)
    assert call(big, 0) == call(0, big) == SHAPE
    assert gp.gpt2_op_q4_scale_count(2**30, 32, 32) > 0
    assert gp.gpt2_op_q4_scale_count(big, 32, 32) == 0
    assert L.gpt2_op_q4_quantize(A, 1, 32, big, 32, 32, A, A, None) == SHAPE
    assert L.gpt2_op_q4_dequantize(A, A, big, 32, 32, A, 0, 32, None) == SHAPE
    assert L.gpt2_op_gemv_q4(A, 32, A, A, None, A, 0, big, 1, big, 32, 32, None) == SHAPE


def test_shared_memory_accessed_in_wide_words_states_its_alignment():
    # a misaligned 16-byte access would fault: the array's address must not hang on how large the static part is
    import os
    import re
    csrc = os.path.join(os.path.dirname(gp.__file__), "csrc")
    for name in ("q4.cu", "prefix.cu", "rules.cu"):
        arrays = re.findall(r"extern __shared__ ([^;]*);", open(os.path.join(csrc, name)).read())
        assert arrays
        for a in arrays:
            aligned = re.match(r"__align__\((\d+)\)", a)
            # (smem_raw: its user rounds the address up to 1024 bytes)
            assert a.endswith("smem_raw[]") or (aligned and int(aligned.group(1)) >= 16), (name, a)


def test_binding_refuses_views_whose_elements_lie_elsewhere(monkeypatch):
    import torch
    # host tensors pass for the current device's, and no call leaves the binding
    calls = []
    T = gp._torch()
    for name in ("quantize", "dequantize", "gemv", "prefix", "rules"):
        monkeypatch.setattr(T, name, lambda *a: calls.append(a) or 0)
    monkeypatch.setattr(gp, "_where", lambda *a: (-1, None))
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    N, K, g, rows = 8, 64, 32, 4
    ok = dict(x=torch.zeros(rows, K, dtype=bf), w=torch.zeros(N, K), packed=torch.zeros(N, K // 2, dtype=u8),
              scales=torch.zeros(K // g, N, dtype=bf), bias=torch.zeros(N, dtype=bf), out=torch.zeros(rows, N, dtype=bf),
              deq=torch.zeros(N, K, dtype=bf))

    def gemv(ldx=K, ldo=N, **kw):
        a = {**ok, **kw}
        gp.gpt2_op_gemv_q4(a["x"], ldx, a["packed"], a["scales"], a["bias"], a["out"], 0, ldo, rows, N, K, g)

    def quantize(ldw=K, **kw):
        a = {**ok, **kw}
        gp.gpt2_op_q4_quantize(a["w"], 1, ldw, N, K, g, a["packed"], a["scales"])

    def dequantize(ldo=K, **kw):
        a = {**ok, **kw}
        gp.gpt2_op_q4_dequantize(a["packed"], a["scales"], N, K, g, a["deq"], 0, ldo)

    B, H, hd, P, cap, M = 2, 3, 16, 5, 9, 4
    at = dict(q=torch.zeros(B, H, hd, dtype=bf), pk=torch.zeros(H, cap, hd, dtype=bf), k=torch.zeros(B, H, M, hd, dtype=bf),
              v=torch.zeros(B, H, M, hd, dtype=bf), len=torch.zeros(B, dtype=i32), o=torch.zeros(B, H, hd, dtype=bf),
              lse=torch.zeros(B, H), s=torch.zeros(1 << 16, dtype=u8))

    def prefix(ldq=H * hd, ldo=H * hd, **kw):
        a = {**at, **kw}
        gp.gpt2_op_prefix_attention_bf16(a["q"], ldq, a["pk"], a["pk"], P, cap, a["k"], a["v"], a["len"], M, a["o"], ldo,
                                         a["lse"], a["s"], B, H, H, hd)

    z = torch.zeros(4, 100)

    def rules(logits=z, out=z, ld=100, nxt=torch.zeros(4, dtype=i32), pos=None):
        gp.gpt2_op_logit_rules(logits, ld, out, ld, 4, 100, gp.LogitRules(), nxt, pos)

    wide = torch.zeros(rows, 2 * K, dtype=bf)
    good = [lambda: gemv(), lambda: gemv(x=wide[:, :K], ldx=2 * K), lambda: gemv(x=wide.view(-1)), lambda: quantize(),
            lambda: quantize(w=torch.zeros(N, K + 8)[:, :K], ldw=K + 8), lambda: dequantize(), lambda: prefix(),
            lambda: prefix(pk=at["pk"][:, :P]), lambda: prefix(q=torch.zeros(B, 50, dtype=bf)[:, :48], ldq=50),
            lambda: rules(), lambda: rules(logits=torch.zeros(4, 128)[:, :100], out=torch.zeros(4, 128), ld=128)]
    for i, f in enumerate(good):
        f()
        assert len(calls) == i + 1
    bad = [lambda: gemv(x=torch.zeros(K, rows, dtype=bf).t()),                       # transposed
           lambda: gemv(x=wide[:, :K]),                                              # another pitch
           lambda: gemv(x=wide[:, ::2]), lambda: gemv(packed=torch.zeros(K // 2, N, dtype=u8).t()),
           lambda: gemv(packed=torch.zeros(N, K, dtype=u8)[:, :K // 2]),
           lambda: gemv(scales=torch.zeros(N, K // g, dtype=bf).t()), lambda: gemv(bias=torch.zeros(N, 2, dtype=bf)[:, 0]),
           lambda: gemv(out=torch.zeros(N, rows, dtype=bf).t()), lambda: quantize(w=torch.zeros(K, N).t()),
           lambda: quantize(w=torch.zeros(2 * N, K)[::2]), lambda: dequantize(deq=torch.zeros(K, N, dtype=bf).t()),
           lambda: prefix(q=torch.zeros(H, B, hd, dtype=bf).transpose(0, 1)),
           lambda: prefix(pk=torch.zeros(cap, H, hd, dtype=bf).transpose(0, 1)),     # positions before heads
           lambda: prefix(k=torch.zeros(B, M, H, hd, dtype=bf).transpose(1, 2)),
           lambda: prefix(v=torch.zeros(B, H, 2 * M, hd, dtype=bf)[:, :, :M]),       # a longer cache's first positions
           lambda: prefix(len=torch.zeros(2 * B, dtype=i32)[::2]), lambda: prefix(lse=torch.zeros(H, B).t()),
           lambda: rules(logits=torch.zeros(100, 4).t()), lambda: rules(out=torch.zeros(4, 200)[:, ::2]),
           lambda: rules(nxt=torch.zeros(8, dtype=i32)[::2]), lambda: rules(pos=torch.zeros(8, dtype=i32)[::2])]
    for f in bad:
        with pytest.raises(gp.Gpt2Error, match="is a view with strides"):
            f()
    assert len(calls) == len(good)


def test_calls_with_nothing_to_do_take_the_null_of_empty_tensors(L):
    # (an empty tensor's address is NULL; sizes that are wrong stay wrong)
    q = lambda N, K=64, ldw=64: L.gpt2_op_q4_quantize(None, 1, ldw, N, K, 32, None, None, None)  # noqa: E731
    d = lambda N: L.gpt2_op_q4_dequantize(None, None, N, 64, 32, None, 0, 64, None)  # noqa: E731
    assert q(0) == d(0) == 0 and q(1) == d(1) == q(0, ldw=32) == INVALID and q(0, K=48) == SHAPE
    g = lambda rows, N, K=64: L.gpt2_op_gemv_q4(None, 64, None, None, None, None, 0, 8, rows, N, K, 32, None)  # noqa: E731
    assert g(0, 8) == g(2, 0) == 0 and g(1, 1) == g(17, 0) == INVALID and g(0, 8, K=48) == SHAPE
    p = lambda B, hd=64: L.gpt2_op_prefix_attention_bf16(  # noqa: E731
        None, 256, None, None, 8, 8, None, None, None, 4, None, 256, None, None, 0, B, 4, 4, hd, None)
    assert p(0) == 0 and p(1) == INVALID and p(0, hd=32) == SHAPE
    r = lambda rows, V, **k: L.gpt2_op_logit_rules(  # noqa: E731
        None, 100, None, 100, rows, V, ctypes.byref(gp.gpt2_logit_rules(**k)), None, None, None)
    assert r(0, 100) == r(2, 0) == r(0, 100, n_bias=3) == r(0, 100, append=1) == 0 and r(2, 100) == INVALID


def test_a_history_without_room_is_none(monkeypatch):
    # also as a view, whose address is not NULL: nothing counts and nothing is added
    import torch
    monkeypatch.setattr(gp, "_buf", lambda where, name, t, *a: None if t is None else t.data_ptr() or None)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    n = torch.zeros(3, dtype=torch.int32)
    for h in (torch.zeros(3, 0, dtype=torch.int32), torch.zeros(3, 8, dtype=torch.int32)[:, 4:4]):
        r = gp.LogitRules(history=h, history_len=n, presence=torch.ones(3), append=True)
        assert r.c.history is None and r.c.history_ld == 0 and r.c.append == 0 and r.rows == 3
    r = gp.LogitRules(history=torch.zeros(3, 8, dtype=torch.int32), history_len=n, append=True)
    assert r.c.history and r.c.history_ld == 8 and r.c.append == 1
    b = torch.zeros(3, 4)[:, 2:2]
    r = gp.LogitRules(bias_ids=b.int(), bias_values=b)
    assert r.c.bias_values is None and r.c.n_bias == 0
    assert gp.LogitRules(append=True).c.append == 1      # no history at all: the call refuses it


def test_a_mask_without_words_is_refused_not_taken_for_none():
    import torch
    for a in (torch.zeros(2, 0, dtype=torch.int32), torch.zeros(2, 8, dtype=torch.int32)[:, 3:3]):
        with pytest.raises(gp.Gpt2Error, match="allowed has no words"):
            gp.LogitRules(allowed=a)


def test_where_a_call_runs():
    from types import SimpleNamespace as S

    def fail():
        raise RuntimeError("an error of the CUDA runtime")
    T = S(current_device=lambda: 1, available=lambda: True, stream_of=lambda dev: 700 + dev)
    assert gp._where(None, T) == (1, 701)
    assert gp._where(S(device_index=1, cuda_stream=9), T) == (1, 9)
    with pytest.raises(gp.Gpt2Error, match="stream is on CUDA device 0, the current device is 1"):
        gp._where(S(device_index=0, cuda_stream=9), T)
    # no GPU: device 0, on which no host buffer lies; with a GPU an error is not taken for that
    assert gp._where(None, S(current_device=fail, available=lambda: False)) == (0, None)
    with pytest.raises(RuntimeError, match="CUDA runtime"):
        gp._where(None, S(current_device=fail, available=lambda: True))
    with pytest.raises(RuntimeError, match="CUDA runtime"):
        gp._where(None, S(current_device=lambda: 0, available=lambda: True, stream_of=lambda dev: fail()))


def test_model_calls_refuse_short_mistyped_and_host_buffers(monkeypatch):
    import torch
    from types import SimpleNamespace as S
    i32, u8 = torch.int32, torch.uint8
    tok, pos, z = torch.zeros(3, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(3, 128)
    cache, none = torch.zeros(4096, dtype=u8), gp.LogitRules()
    ctx = S(vocab_padded=128)          # what gpt2_create leaves on its context
    with pytest.raises(gp.Gpt2Error, match="not on the current CUDA device"):
        gp.gpt2_rules_next(ctx, z, 3, none, tok, pos)
    with pytest.raises(gp.Gpt2Error, match="not on the current CUDA device"):
        gp.gpt2_q4_pack(ctx, cache, 64)
    with pytest.raises(gp.Gpt2Error, match="not on the current CUDA device"):
        gp.gpt2_decode_step_ex(ctx, cache, 3, 4, tok, pos, None, z)
    # host tensors pass for the current device's, and no call leaves the binding
    calls = []
    monkeypatch.setattr(gp, "_where", lambda *a: (-1, None))
    lib = S(**{n: (lambda *a: calls.append(a) or 0) for n in ("gpt2_rules_next", "gpt2_q4_pack", "gpt2_decode_step_ex")},
            gpt2_strerror=gp._lib().gpt2_strerror)
    monkeypatch.setattr(gp, "_lib", lambda: lib)
    step = lambda tok=tok, pos=pos, z=z, cache=cache, b=3: gp.gpt2_decode_step_ex(ctx, cache, b, 4, tok, pos, None, z)  # noqa: E731
    nxt = lambda z=z, tok=tok, pos=pos, b=3: gp.gpt2_rules_next(ctx, z, b, none, tok, pos)  # noqa: E731
    pack = lambda q: gp.gpt2_q4_pack(ctx, q, 64)  # noqa: E731
    for f in (step, nxt, lambda: nxt(pos=None), lambda: pack(cache)):
        f()
    assert len(calls) == 4
    short = torch.zeros(2, dtype=i32)
    for f, what in [(lambda: step(tok=short), "tokens holds 2"), (lambda: step(pos=short), "pos holds 2"),
                    (lambda: step(z=z[:, :127].contiguous()), "logits holds 381"), (lambda: step(b=4), "holds 3"),
                    (lambda: step(tok=tok.long()), "tokens is torch.int64"), (lambda: step(z=z.double()), "logits is"),
                    (lambda: step(cache=cache.float()), "cache is"), (lambda: step(z=torch.zeros(3, 256)[:, :128]), "strides"),
                    (lambda: step(pos=None), "pos is missing"), (lambda: nxt(tok=short), "next_tokens holds 2"),
                    (lambda: nxt(pos=short), "pos holds 2"), (lambda: nxt(z=z[:2].clone()), "logits holds 256"),
                    (lambda: nxt(tok=tok.long()), "next_tokens is"), (lambda: nxt(z=z.half()), "logits is"),
                    (lambda: nxt(tok=torch.zeros(6, dtype=i32)[::2]), "strides"), (lambda: pack(cache.float()), "q4 is"),
                    (lambda: pack(cache[::2]), "strides"), (lambda: pack(cache[:0]), "q4 holds 0")]:
        with pytest.raises(gp.Gpt2Error, match=what):
            f()
    assert len(calls) == 4
