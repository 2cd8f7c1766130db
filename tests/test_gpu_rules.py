"""Rules on logits against the same steps in numpy: every step is one fp32
operation, so logits and choices agree bit by bit; and against 64 bits, where
a logit is off by at most half a step (2^-24) of each of the four values on its
way."""
import numpy as np
import pytest
import torch

import decoder_only_transformer_step_b200 as gp

pytestmark = pytest.mark.gpu
F = np.float32


def reference(z, V, r, ft=np.float32):
    """(rules applied, choice) by the definition, each step rounded to ft."""
    out = z[:, :V].astype(ft).copy()
    rows = out.shape[0]
    for i in range(rows):
        c_all, c_gen = np.zeros(V, np.int64), np.zeros(V, np.int64)
        if r.get("history") is not None:
            H = r["history"].shape[1]
            n = int(np.clip(r["history_len"][i], 0, H))
            g0 = int(r["gen_start"][i]) if r.get("gen_start") is not None else 0
            for j in range(n):
                t = int(r["history"][i, j])
                if 0 <= t < V:
                    c_all[t] += 1
                    c_gen[t] += j >= g0
        rep, pres, freq = (ft(r[k][i]) if r.get(k) is not None else ft(d)
                           for k, d in (("repetition", 1), ("presence", 0), ("frequency", 0)))
        with np.errstate(invalid="ignore", over="ignore"):
            out[i] = np.where(c_all > 0, np.where(out[i] > 0, out[i] / rep, out[i] * rep), out[i])
            out[i] = np.where(c_gen > 0, (out[i] - freq * c_gen.astype(ft)) - pres, out[i])
            if r.get("bias_ids") is not None:
                bias = {int(t): ft(v) for t, v in zip(r["bias_ids"][i], r["bias_values"][i])}
                for t, v in bias.items():
                    if 0 <= t < V:
                        out[i, t] = out[i, t] + v
        if r.get("allowed") is not None:
            bits = (r["allowed"][i].view(np.uint32)[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
            out[i] = np.where(bits == 1, out[i], ft(-np.inf))
    nxt = []
    for i in range(rows):
        nan = np.flatnonzero(np.isnan(out[i]))
        nxt.append(int(nan[0]) if len(nan) else int(np.argmax(out[i])))
    return out, np.array(nxt, np.int32)


def random_rules(rng, rows, V, hist, n_bias, mask, parts="hgrpfba"):
    r = {}
    if "h" in parts and hist:
        r["history"] = np.minimum((V + 3) * rng.random((rows, hist)) ** 2, V + 1).astype(np.int32) - 1  # -1 and V among them
        r["history_len"] = rng.integers(-1, hist + 2, rows).astype(np.int32)
        if "g" in parts:
            r["gen_start"] = rng.integers(0, hist + 1, rows).astype(np.int32)
        r["repetition"] = (1 + rng.random(rows)).astype(F) if "r" in parts else None
        r["presence"] = rng.random(rows).astype(F) if "p" in parts else None
        r["frequency"] = rng.random(rows).astype(F) if "f" in parts else None
    if "b" in parts and n_bias:
        r["bias_ids"] = rng.integers(-2, V + 1, (rows, n_bias)).astype(np.int32)
        r["bias_values"] = (5 * rng.standard_normal((rows, n_bias))).astype(F)
    if "a" in parts and mask:
        r["allowed"] = rng.integers(0, 1 << 32, (rows, (V + 31) // 32 + 1), dtype=np.uint32).view(np.int32)
    return r


def on_device(r, **kw):
    return gp.LogitRules(**{k: torch.from_numpy(v).cuda() for k, v in r.items() if v is not None}, **kw)


def run(z, V, r, ldo=None, in_place=False, **kw):
    rows, ld = z.shape
    ldo = ld if in_place else ldo or V
    zt = torch.from_numpy(z).cuda()
    out = zt if in_place else torch.full((rows, ldo), 123.0, device="cuda")
    nxt = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    rules = on_device(r, **kw)
    gp.gpt2_op_logit_rules(zt, ld, out, ldo, rows, V, rules, nxt, pos)
    torch.cuda.synchronize()
    assert pos.tolist() == list(range(1, rows + 1))
    if not in_place:
        np.testing.assert_array_equal(zt.cpu().numpy(), z)
    return out.cpu().numpy(), nxt.cpu().numpy(), rules


@pytest.mark.parametrize("rows,V,ld", [(1, 1, 1), (3, 31, 40), (2, 513, 513), (5, 5000, 5003), (40, 1000, 1024),
                                       (150, 777, 777), (300, 300, 301), (1, 200001, 200001), (2, 262144, 262144)])
@pytest.mark.parametrize("hist,n_bias,mask", [(0, 0, 1), (1, 1, 0), (90, 40, 1), (3000, 700, 1)])
def test_rules_bit_by_bit(rows, V, ld, hist, n_bias, mask):
    rng = np.random.default_rng(rows + V + hist)
    z = (3 * rng.standard_normal((rows, ld))).astype(F)
    r = random_rules(rng, rows, V, hist, n_bias, mask)
    want, nxt = reference(z, V, r)
    in_place = (rows + hist) % 2 == 0
    out, got, _ = run(z, V, r, ldo=V + rows % 3, in_place=in_place)
    np.testing.assert_array_equal(out[:, :V], want)
    np.testing.assert_array_equal(got, nxt)
    assert np.array_equal(out[:, V:], z[:, V:]) if in_place else (out[:, V:] == 123).all()
    exact, _ = reference(z, V, r, np.float64)
    fin = np.isfinite(exact)
    # half a step for each operation, of values no larger than |z| rep, freq c, pres, bias
    size = 2 * np.abs(z[:, :V].astype(np.float64)) + hist + 1 + 25
    assert (np.abs(want[fin] - exact[fin]) <= 5 * 2.0**-24 * size[fin]).all()


@pytest.mark.parametrize("parts", ["", "h", "hr", "hgp", "hf", "b", "a", "hgrpf", "ba"])
def test_each_rule_alone(parts):
    rng = np.random.default_rng(11)
    z = rng.standard_normal((6, 900)).astype(F)
    r = random_rules(rng, 6, 900, 60, 25, 1, parts)
    want, nxt = reference(z, 900, r)
    out, got, _ = run(z, 900, r)
    np.testing.assert_array_equal(out, want)
    np.testing.assert_array_equal(got, nxt)


def test_ties_nan_infinities_and_rows_with_nothing_left():
    V = 2000
    rng = np.random.default_rng(12)
    z = rng.standard_normal((8, V)).astype(F)
    allowed = np.full((8, (V + 31) // 32), -1, np.int32)
    z[0, [17, 900, 1999]] = 50.0                  # tie: lowest id
    z[1, [700, 40]] = np.nan                      # first NaN
    z[2, 3] = np.nan
    allowed[2, 0] &= ~(1 << 3)                    # a masked NaN is gone
    z[3, :] = -np.inf                             # nothing above -inf: id 0
    allowed[4, :] = 0                             # the mask leaves nothing
    z[5, 100] = np.inf
    allowed[5, 3] &= ~(1 << 4)                    # a masked +inf is gone
    z[6, :] = np.finfo(F).min                     # all at the type's lowest value
    allowed[6, : V // 64] = 0
    z[7, 5] = -0.0
    z[7, 6:] = -1
    z[7, :5] = -1
    z[7, 9] = 0.0                                 # -0 and 0 are equal: the lower id
    r = dict(allowed=allowed)
    want, nxt = reference(z, V, r)
    out, got, _ = run(z, V, r)
    np.testing.assert_array_equal(out, want)
    np.testing.assert_array_equal(got, nxt)
    assert got.tolist()[:2] == [17, 40] and got[3] == 0 and got[4] == 0 and got[7] == 5


def test_the_same_id_many_times_and_the_last_bias_counts():
    z = np.ones((2, 64), F)
    r = dict(history=np.full((2, 5000), 7, np.int32), history_len=np.array([5000, 4999], np.int32),
             gen_start=np.array([4, 0], np.int32), frequency=np.array([0.125, 0.25], F),
             presence=np.array([0.5, 0.0], F), repetition=np.array([2.0, 1.0], F),
             bias_ids=np.array([[7, 9, 9, 7], [9, 9, 9, 9]], np.int32),
             bias_values=np.array([[1, 2, 3, 4], [-1, -2, -3, 100]], F))
    out, nxt, _ = run(z, 64, r)
    assert out[0, 7] == F(0.5 - 0.125 * 4996 - 0.5 + 4) and out[0, 9] == 4 and out[1, 9] == 101 and out[1, 7] == F(1 - 0.25 * 4999)
    assert nxt.tolist() == [9, 9]


def test_append_in_a_captured_loop():
    # each step penalises what the steps before chose: the choices walk down the logits
    rows, V, H = 3, 4096, 6
    rng = np.random.default_rng(13)
    z0 = rng.standard_normal((rows, V)).astype(F)
    zt, out = torch.from_numpy(z0).cuda(), torch.empty(rows, V, device="cuda")
    hist = torch.full((rows, H), -1, dtype=torch.int32, device="cuda")
    n = torch.zeros(rows, dtype=torch.int32, device="cuda")
    rules = gp.LogitRules(history=hist, history_len=n, presence=torch.full((rows,), 100.0, device="cuda"), append=True)
    nxt = torch.zeros(rows, dtype=torch.int32, device="cuda")
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    gp.gpt2_op_logit_rules(zt, V, out, V, rows, V, rules, nxt, pos)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            gp.gpt2_op_logit_rules(zt, V, out, V, rows, V, rules, nxt, pos)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    order = np.argsort(-z0, axis=1, kind="stable")
    np.testing.assert_array_equal(hist.cpu().numpy(), order[:, :H])   # full after six, the seventh is not added
    assert n.tolist() == [H] * rows and pos.tolist() == [7] * rows
    np.testing.assert_array_equal(nxt.cpu().numpy(), order[:, H])


def test_without_a_choice():
    z = torch.randn(4, 500, device="cuda")
    out = torch.empty_like(z)
    pres = torch.ones(4, device="cuda")
    gp.gpt2_op_logit_rules(z, 500, out, 500, 4, 500, gp.LogitRules(presence=pres))
    assert torch.equal(z, out)                                       # no history: nothing to penalise
    with pytest.raises(gp.Gpt2Error):
        gp.gpt2_op_logit_rules(z, 500, out, 500, 4, 500, gp.LogitRules(presence=pres[:3].clone()))


@pytest.mark.parametrize("rows", [6, 450])               # a row's 8 blocks, one block a row
@pytest.mark.parametrize("parts", ["h", "b", "hgrpfb"])
@pytest.mark.parametrize("append", [False, True])
def test_nothing_left_beside_a_history_and_biases_is_id_0(rows, parts, append):
    V = 2000
    rng = np.random.default_rng(15)
    z = rng.standard_normal((rows, V)).astype(F)
    allowed = np.full((rows, (V + 31) // 32), -1, np.int32)
    allowed[0::3] = 0                                     # the mask leaves nothing
    z[1::3] = -np.inf                                     # the logits leave nothing; the other rows choose
    r = dict(allowed=allowed)
    if "h" in parts:
        r["history"] = rng.integers(17, V, (rows, 40)).astype(np.int32)   # no id 0
        r["history_len"] = rng.integers(5, 39, rows).astype(np.int32)
    if "g" in parts:
        r["gen_start"] = np.full(rows, 3, np.int32)
        for k in ("repetition", "presence", "frequency"):
            r[k] = (1 + rng.random(rows)).astype(F)
    if "b" in parts:
        r["bias_ids"] = rng.integers(17, V, (rows, 9)).astype(np.int32)
        r["bias_values"] = rng.standard_normal((rows, 9)).astype(F)
    append = append and "h" in parts
    want, nxt = reference(z, V, r)
    out, got, rules = run(z, V, r, append=append)
    np.testing.assert_array_equal(out, want)
    np.testing.assert_array_equal(got, nxt)
    assert not got[0::3].any() and not got[1::3].any()
    if append:
        n = r["history_len"]
        np.testing.assert_array_equal(rules.tensors["history_len"].cpu().numpy(), n + 1)
        assert (rules.tensors["history"].cpu().numpy()[np.arange(rows), n] == nxt).all()
