"""The serving operators in the model, together: decode steps behind a shared
prefix, with 4-bit weights, under rules, against the fp64 oracle on the same
weights (the 4-bit ones dequantised), and inside one CUDA graph."""
import numpy as np
import pytest
import torch

import decoder_only_transformer_step_b200 as gp
from decoder_only_transformer_step_b200 import inputs
from oracle import Config, kv_cache_empty, decode_step, prefill
import oracle
from oracle_fixtures import TINY, params_for

pytestmark = pytest.mark.gpu

HD64 = Config(n_layer=2, d_model=128, n_head=2, n_ctx=128, vocab=1024)


def make_model(oc, mode, batch=8):
    model = gp.GPT2(gp.ModelConfig(oc.n_layer, oc.d_model, oc.n_head, oc.n_ctx, oc.vocab - 12, oc.vocab, batch, mode))
    flat = oracle.flatten(params_for(oc, seed=71), oc).astype(np.float32)
    model.master.copy_(torch.from_numpy(flat))
    model.refresh_shadow()
    return model, oracle.unflatten(flat.astype(np.float64), oc)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def rel_err(z, ref):
    return float(np.abs(z - ref).max() / np.abs(ref).max())


def rounded(model, oc, group):
    """The oracle's parameters with the step's matrices as their 4-bit values; the
    head apart, since the embedding keeps its own."""
    def q(w):
        N, K = w.shape
        t = torch.from_numpy(w.astype(np.float32)).cuda().contiguous()
        p = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
        s = torch.empty(K // group, (N + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda")
        gp.gpt2_op_q4_quantize(t, 1, K, N, K, group, p, s)
        out = torch.empty(N, K, device="cuda")
        gp.gpt2_op_q4_dequantize(p, s, N, K, group, out, 1, K)
        return out.cpu().numpy().astype(np.float64)
    full = {n: model.view(model.master, n) for n, *_ in model.layout}
    flat = model.master.clone()
    for n, off, r, c in model.layout:
        if n.split(".")[-1] in ("w_qkv", "w_o", "w_fc", "w_mp"):
            flat[off:off + r * c] = torch.from_numpy(q(full[n].cpu().numpy()).ravel()).float().cuda()
    return oracle.unflatten(flat.cpu().numpy().astype(np.float64), oc), q(full["wte"].cpu().numpy())


def oracle_step(p, head, oc, cache, tok, pos):
    """decode_step with the LM head `head` (None: tied)."""
    if head is None:
        return decode_step(p, oc, cache, tok, pos)
    # the tied logits h wte^T give the hidden state back (wte has full column
    # rank: least squares, exact to fp64), which the other head then reads
    h = np.linalg.lstsq(p["wte"], decode_step(p, oc, cache, tok, pos).T, rcond=None)[0].T
    return h @ head.T


@pytest.mark.parametrize("oc", [TINY, HD64], ids=["hd16", "hd64"])
@pytest.mark.parametrize("mode", [1, 0])
@pytest.mark.parametrize("P", [1, 37])
def test_rows_behind_a_prefix_match_the_oracle_on_whole_sequences(oc, mode, P):
    batch, max_len = 5, 20
    model, p64 = make_model(oc, mode)
    prompt, _ = inputs.uniform_tokens(1, oc.n_ctx, oc.vocab - 12, seed=72)
    pre = gp.KVCache(model, 1, P + 2)
    pre.prefill(i32(prompt), i32([P]))
    cache = gp.KVCache(model, batch, max_len, prefix=pre, prefix_len=P)
    ref = kv_cache_empty(oc, batch, P + max_len)
    whole = np.repeat(prompt, batch, 0)
    prefill(p64, oc, ref, whole, np.full(batch, P, np.int32))
    pos = np.zeros(batch, np.int32)
    before = pre.buf.clone()
    for step in range(8):
        tok = inputs.uniform_tokens(batch, 1, oc.vocab - 12, seed=200 + step)[0][:, 0]
        z = cache.step(i32(tok), i32(pos)).cpu().numpy().astype(np.float64)
        z_ref = decode_step(p64, oc, ref, tok, pos + P)
        assert rel_err(z, z_ref) <= (1e-4 if mode == 1 else 2e-2), step
        pos = pos + 1
        if step == 3:
            pos[1] = 0                                  # a row that starts over
    torch.cuda.synchronize()
    assert model.status() == 0
    planes = 2 * oc.n_layer * ((oc.n_head * (P + 2) * (oc.d_model // oc.n_head) * (4 if mode else 2) + 255) // 256 * 256)
    assert torch.equal(before[:planes], pre.buf[:planes])   # the prefix is only read


# wide enough that the products stream their weights (the narrow ones above read them directly)
WIDE = Config(n_layer=1, d_model=1280, n_head=20, n_ctx=64, vocab=2560)


@pytest.mark.parametrize("oc,group,batch", [(HD64, g, b) for g in (32, 64, 128) for b in (1, 8, 13)] +
                         [(WIDE, g, b) for g in (32, 128) for b in (3, 16)],
                         ids=lambda v: "wide" if v is WIDE else "narrow" if v is HD64 else str(v))
def test_decode_with_4_bit_weights_matches_the_oracle_on_their_values(oc, group, batch):
    model, _ = make_model(oc, 0, batch=16)
    q4 = gp.Q4Weights(model, group)
    p64, head = rounded(model, oc, group)
    cache = gp.KVCache(model, batch, 16, q4=q4)
    ref = kv_cache_empty(oc, batch, 16)
    for step in range(6 if oc is HD64 else 3):
        tok = inputs.uniform_tokens(batch, 1, oc.vocab - 12, seed=300 + step)[0][:, 0]
        pos = np.full(batch, step, np.int32)
        z = cache.step(i32(tok), i32(pos)).cpu().numpy().astype(np.float64)
        z_ref = oracle_step(p64, head, oc, ref, tok, pos)
        assert rel_err(z, z_ref) <= 2e-2, step          # the bf16 mode's tolerance
    torch.cuda.synchronize()
    assert model.status() == 0


def test_without_options_it_is_the_plain_step_bit_by_bit():
    oc = HD64
    model, _ = make_model(oc, 0)
    tok, pos = i32([3, 4, 5]), i32([0, 0, 0])
    a, b = gp.KVCache(model, 3, 10), gp.KVCache(model, 3, 10)
    z = a.step(tok, pos).clone()
    gp.gpt2_decode_step_ex(model.ctx, b.buf, 3, 10, tok, pos, gp.gpt2_decode_opts(), b.logits)
    assert torch.equal(z, b.logits)


def test_everything_together_in_one_graph_repeats_the_eager_loop():
    oc = HD64
    batch, max_len, P, steps = 4, 24, 50, 20
    model, _ = make_model(oc, 0)
    q4 = gp.Q4Weights(model, 64)
    prompt, _ = inputs.uniform_tokens(1, oc.n_ctx, oc.vocab - 12, seed=73)
    pre = gp.KVCache(model, 1, P)
    pre.prefill(i32(prompt), i32([P]))
    words = (oc.vocab - 12 + 31) // 32
    allowed = torch.from_numpy(np.random.default_rng(74).integers(-2**31, 2**31, (batch, words)).astype(np.int32)).cuda()

    def loop(graph):
        cache = gp.KVCache(model, batch, max_len, prefix=pre, prefix_len=P, q4=q4)
        hist = torch.full((batch, P + steps), -1, dtype=torch.int32, device="cuda")
        hist[:, :P] = i32(prompt)[0, :P]
        rules = gp.LogitRules(history=hist, history_len=i32([P] * batch), gen_start=i32([P] * batch),
                              repetition=torch.full((batch,), 1.2, device="cuda"),
                              presence=torch.full((batch,), 3.0, device="cuda"), allowed=allowed, append=True)
        cache.tokens.copy_(i32([1, 2, 3, 4]))

        def one():
            cache.step()
            cache.greedy_advance(rules)
        if not graph:
            for _ in range(steps):
                one()
        else:
            one()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                one()
            for _ in range(steps - 1):
                g.replay()
        torch.cuda.synchronize()
        return hist.cpu().numpy(), cache.pos.tolist(), cache.logits.clone()

    a, pos, za = loop(False)
    b, pos2, zb = loop(True)
    np.testing.assert_array_equal(a, b)
    assert pos == pos2 == [steps] * batch and torch.equal(za, zb)
    assert model.status() == 0
    bits = allowed.cpu().numpy().view(np.uint32)
    for r in range(batch):
        for t in a[r, P:].tolist():
            assert (int(bits[r, t // 32]) >> (t % 32)) & 1   # only allowed ids
    assert all(len(set(a[r, P:])) > 5 for r in range(batch))  # the presence penalty keeps it moving


def test_refusals_of_the_model_calls():
    oc = HD64
    model, _ = make_model(oc, 0)
    pre = gp.KVCache(model, 1, 30)
    with pytest.raises(ValueError):
        gp.Q4Weights(model, 48)
    with pytest.raises(ValueError):
        gp.KVCache(model, 2, 100, prefix=pre, prefix_len=29)       # 129 positions
    with pytest.raises(ValueError):
        gp.KVCache(model, 2, 10, prefix=pre, prefix_len=31)
    with pytest.raises(ValueError):
        gp.KVCache(model, 2, 10, prefix_len=3)
    with pytest.raises(ValueError):
        gp.KVCache(model, 2, 10, prefix=gp.KVCache(model, 2, 30), prefix_len=3)
    c = gp.KVCache(model, 2, 10, prefix=pre, prefix_len=20)
    with pytest.raises(ValueError):
        c.prefill(None, None)
    bad = gp.ERRORS_BY_NAME

    def code(**kw):
        o = gp.gpt2_decode_opts(**{n: getattr(c.opts, n) for n, _ in gp.gpt2_decode_opts._fields_})
        for k, v in kw.items():
            setattr(o, k, v)
        try:
            gp.gpt2_decode_step_ex(model.ctx, c.buf, 2, 10, c.tokens, c.pos, o, c.logits)
        except gp.Gpt2Error as e:
            return e.code
        return 0
    assert code() == 0
    assert code(prefix_len=31) == code(prefix_len=-1) == code(prefix_bytes=100) == bad["GPT2_ERR_INVALID_ARG"]
    assert code(prefix_cap=129) == code(prefix=c.opts.prefix + 16) == code(scratch=None) == bad["GPT2_ERR_INVALID_ARG"]
    assert code(scratch_bytes=c.opts.scratch_bytes - 1) == bad["GPT2_ERR_WORKSPACE"]
    assert code(q4=c.opts.prefix, q4_group=48) == bad["GPT2_ERR_INVALID_ARG"]
    assert code(q4=c.opts.prefix, q4_group=64, q4_bytes=16) == bad["GPT2_ERR_WORKSPACE"]
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(gp.Gpt2Error):
        gp.gpt2_q4_pack(model.ctx, small, 64)
    f32, _ = make_model(TINY, 1)
    with pytest.raises(ValueError):
        gp.Q4Weights(f32, 32)
    # a position out of range is reported, as by the plain step
    c.pos.fill_(10)
    c.step()
    assert model.status() == bad["GPT2_ERR_POSITION_RANGE"]


def test_prompts_fed_by_steps_behind_a_prefix_as_documented():
    # step, pos += 1, ..., step, greedy_advance: the rows end where a prefill of their whole sequences ends
    oc, batch, P, n = TINY, 3, 21, 6
    model, _ = make_model(oc, 1)
    whole, _ = inputs.uniform_tokens(batch, oc.n_ctx, oc.vocab - 12, seed=75)
    whole[:, :P] = whole[0, :P]
    plain = gp.KVCache(model, batch, P + 20)
    plain.prefill(i32(whole), i32([P + n] * batch))
    first = plain.logits[:, : oc.vocab - 12].clone()
    pre = gp.KVCache(model, 1, P)
    pre.prefill(i32(whole[:1]), i32([P]))
    cache = gp.KVCache(model, batch, 20, prefix=pre, prefix_len=P)
    hist = torch.full((batch, 16), -1, dtype=torch.int32, device="cuda")
    length = torch.zeros(batch, dtype=torch.int32, device="cuda")
    rules = gp.LogitRules(history=hist, history_len=length, append=True)
    prompt = i32(whole[:, P:P + n])
    for i in range(n):
        cache.step(prompt[:, i].contiguous())
        if i + 1 < n:
            cache.pos += 1
    z = cache.logits[:, : oc.vocab - 12].clone()
    assert float((z - first).abs().max()) <= 1e-4 * float(first.abs().max())      # the fp32 mode's tolerance
    cache.greedy_advance(rules)
    assert cache.pos.tolist() == [n] * batch and length.tolist() == [1] * batch   # the prompt is nobody's choice
    for _ in range(5):
        cache.step()
        cache.greedy_advance(rules)
        plain.step()
        plain.greedy_advance()
        assert float((cache.logits - plain.logits)[:, : oc.vocab - 12].abs().max()) <= 2e-4 * float(first.abs().max())
        assert torch.equal(cache.tokens, plain.tokens)
    assert cache.pos.tolist() == [n + 5] * batch and hist[:, :6].tolist() == hist[:, :6].clamp(0).tolist()
    assert model.status() == 0


def test_prefill_beside_4_bit_weights_is_that_of_the_models_own():
    oc = HD64
    model, _ = make_model(oc, 0)
    tok, lens = i32(inputs.uniform_tokens(2, oc.n_ctx, oc.vocab - 12, seed=76)[0]), i32([9, 30])
    a, b = gp.KVCache(model, 2, 40), gp.KVCache(model, 2, 40, q4=gp.Q4Weights(model, 64))
    a.prefill(tok, lens)
    b.prefill(tok, lens)
    assert torch.equal(a.logits, b.logits) and torch.equal(a.tokens, b.tokens)
    assert not torch.equal(a.step(), b.step())
