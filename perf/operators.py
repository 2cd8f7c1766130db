"""The operators of the serving step that are measured: 4-bit weights with
group scales (quantising them, and the matrix-vector products that read them),
attention of a decode batch whose rows share one prefix, and rules on logits
(penalties, biases, grammar masks) with the greedy choice.

``listed()`` and ``draw(rng)`` give cases, ``prepare(case, seed)`` a case's
inputs on the GPU, ``run(state)`` one pass: in plain torch operations, or,
where ``own`` is true, through this library.  ``exact(case, seed)`` is the
same result from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
HEADROOM = 1 << 28  # elements of one fp32 / fp64 temporary in the chunked forms


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # QKV projection of the 1558M configuration (d 1600) for one conversation: latency counts
        dict(name="gemv-1x4800x1600", op="gemv", rows=1, N=4800, K=1600, group=64, out_fp32=False, bias=True),
        # its MLP output projection for a full cache of 16 rows: long rows, few columns
        dict(name="gemv-16x1600x6400", op="gemv", rows=16, N=1600, K=6400, group=128, out_fp32=False, bias=True),
        # its LM head for 8 rows: fp32 logits
        dict(name="gemv-8x50304x1600", op="gemv", rows=8, N=50304, K=1600, group=32, out_fp32=True, bias=False),
        # one large layer of a bigger network, an odd number of columns
        dict(name="gemv-5x28673x8192", op="gemv", rows=5, N=28673, K=8192, group=128, out_fp32=False, bias=False),
        # loading weights: the fc matrix of the 350M configuration from its fp32 master
        dict(name="quantize-4096x1024", op="quantize", N=4096, K=1024, group=64, w_fp32=True),
        # and the token embedding of the 1558M one from bf16
        dict(name="quantize-50304x1600", op="quantize", N=50304, K=1600, group=32, w_fp32=False),
        # three short chats behind one system prompt, 124M heads
        dict(name="prefix-3x12x200", op="prefix", B=3, Hq=12, Hkv=12, hd=64, P=200, max_len=64),
        # a full cache of the 1558M configuration, most of the context shared
        dict(name="prefix-16x25x768", op="prefix", B=16, Hq=25, Hkv=25, hd=64, P=768, max_len=256),
        # the 4096-position configuration with a long shared document
        dict(name="prefix-16x12x3500", op="prefix", B=16, Hq=12, Hkv=12, hd=64, P=3500, max_len=596),
        # grouped heads of 128, many rows behind a long prefix
        dict(name="prefix-40x32x32768", op="prefix", B=40, Hq=32, Hkv=8, hd=128, P=32768, max_len=512),
        # every rule on a full cache
        dict(name="rules-16x50257", op="rules", rows=16, V=50257, ld=50304, hist=1024, n_bias=64, mask=True),
        # a large batch of long histories
        dict(name="rules-384x50257", op="rules", rows=384, V=50257, ld=50304, hist=4096, n_bias=300, mask=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "quantize", "prefix", "prefix", "rules"])
    if op == "gemv" or op == "quantize":
        group = rng.choice([32, 64, 128])
        K = group * _log(rng, 1, 28672 // group)
        most = 50304 * 1600 if op == "quantize" else 28673 * 8192
        N = _log(rng, 1, min(65536, most // K))
        if op == "quantize":
            return dict(op=op, N=N, K=K, group=group, w_fp32=rng.random() < 0.5)
        return dict(op=op, rows=rng.randint(1, 16), N=N, K=K, group=group, out_fp32=rng.random() < 0.4,
                    bias=rng.random() < 0.5)
    if op == "prefix":
        while True:
            Hkv, G = rng.choice([1, 2, 4, 8, 12, 16, 25]), rng.choice([1, 1, 2, 3, 4, 8])
            hd, B = rng.choice([64, 64, 128]), _log(rng, 1, 64)
            P = _log(rng, 1, 131072) if rng.random() < 0.95 else 0
            max_len = _log(rng, 1, 2048)
            c = dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, hd=hd, P=P, max_len=max_len)
            if B * Hkv * G * (P + max_len) * hd <= 40 * 32 * (32768 + 512) * 128 and \
                    Hkv * (P + B * max_len) * hd <= 8 * (32768 + 40 * 512) * 128:
                return c
    V = _log(rng, 500, 262144)
    ld = V + rng.choice([0, 0, 1, 7, 47, 128])
    rows = max(1, min(_log(rng, 1, 512), 384 * 50257 // V))
    return dict(op=op, rows=rows, V=V, ld=ld, hist=_log(rng, 1, 16384 if rows <= 64 else 4096),
                n_bias=rng.choice([0, 1, 17, 64, 300]), mask=rng.random() < 0.7)


def work(case):
    c = case
    if c["op"] == "gemv":
        b = c["N"] * c["K"] // 2 + 2 * c["N"] * (c["K"] // c["group"]) + 2 * c["rows"] * c["K"]
        b += c["rows"] * c["N"] * (4 if c["out_fp32"] else 2) + (2 * c["N"] if c["bias"] else 0)
        return {"bytes": b, "flops": 2 * c["rows"] * c["N"] * c["K"]}
    if c["op"] == "quantize":
        n = c["N"] * c["K"]
        # the weights in, nibbles and scales out; then those in and the values they stand for out
        return {"bytes": n * (4 if c["w_fp32"] else 2) + 2 * (n // 2 + 2 * n // c["group"]) + 2 * n, "flops": 4 * n}
    if c["op"] == "prefix":
        own_keys = sum(_lens(c))
        b = 4 * c["Hkv"] * c["hd"] * (c["P"] + own_keys) + 4 * c["B"] * c["Hq"] * c["hd"] + 4 * c["B"] * c["Hq"]
        return {"bytes": b, "flops": 4 * c["Hq"] * c["hd"] * (c["B"] * c["P"] + own_keys)}
    n = c["rows"] * c["V"]
    b = 8 * n + 4 * c["rows"] * c["hist"] + 8 * c["rows"] * c["n_bias"] + 4 * c["rows"]
    return {"bytes": b + (n // 8 if c["mask"] else 0), "flops": 6 * n}


def _lens(c):
    """Own positions of each row: spread over 0 .. max_len, both ends among them."""
    if c["B"] == 1:
        return [c["max_len"]]
    return [(b * 7 % c["B"]) * c["max_len"] // (c["B"] - 1) for b in range(c["B"])] if c["B"] % 7 else \
        [b * c["max_len"] // (c["B"] - 1) for b in range(c["B"])]


# ----------------------------------------------------------------- inputs ---

def _chunks(n, width):
    step = max(1, HEADROOM // max(1, width))
    return [(i, min(n, i + step)) for i in range(0, n, step)]


def _pitch(N):
    return (N + 7) // 8 * 8


def _q4(w, group):
    """Whole numbers -7..7 (fp32) and scales (bf16 [N, K/group]) of w [N, K]."""
    N, K = w.shape
    w = w.float().view(N, K // group, group)
    top = w.abs().amax(2)
    s = (top / torch.full_like(top, 7.0)).bfloat16()
    sf = s.float()[:, :, None]
    q = torch.round(w / torch.where(sf == 0, torch.ones_like(sf), sf)).clamp(-7, 7)
    return torch.where(sf == 0, torch.zeros_like(q), q).view(N, K), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = case

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, device=DEV).normal_(0, std, generator=g).to(dtype)

    def uniform(*shape):
        return torch.empty(shape, device=DEV).uniform_(generator=g)

    s = dict(case=c)
    if c["op"] == "gemv":
        N, K, group = c["N"], c["K"], c["group"]
        # weights as a trained layer's (std 0.02), quantised: byte j of a row holds k = 2j (low half) and 2j + 1
        s["packed"] = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(K // group, _pitch(N), dtype=torch.bfloat16, device=DEV)
        for a, b in _chunks(N, 4 * K):
            q, sc = _q4(normal(b - a, K, std=0.02), group)
            n = (q + 8).to(torch.uint8)
            s["packed"][a:b] = n[:, 0::2] | (n[:, 1::2] << 4)
            s["scales"][:, a:b] = sc.t()
        s["x"] = normal(c["rows"], K, dtype=torch.bfloat16)  # as a LayerNorm leaves them
        s["bias"] = normal(N, std=0.1, dtype=torch.bfloat16) if c["bias"] else None
        s["out"] = torch.empty(c["rows"], N, dtype=torch.float32 if c["out_fp32"] else torch.bfloat16, device=DEV)
    elif c["op"] == "quantize":
        N, K = c["N"], c["K"]
        s["w"] = normal(N, K, std=0.02, dtype=torch.float32 if c["w_fp32"] else torch.bfloat16)
        s["packed"] = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(K // c["group"], _pitch(N), dtype=torch.bfloat16, device=DEV)
        s["out"] = torch.empty(N, K, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "prefix":
        B, Hq, Hkv, hd, P, M = (c[k] for k in ("B", "Hq", "Hkv", "hd", "P", "max_len"))
        bf = torch.bfloat16
        s["q"] = normal(B, Hq, hd, std=1.5, dtype=bf)
        s["pk"], s["pv"] = normal(Hkv, P, hd, dtype=bf), normal(Hkv, P, hd, dtype=bf)
        s["k"], s["v"] = normal(B, Hkv, M, hd, dtype=bf), normal(B, Hkv, M, hd, dtype=bf)
        s["len"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)
        s["out"] = torch.empty(B, Hq, hd, dtype=bf, device=DEV)
        s["lse"] = torch.empty(B, Hq, dtype=torch.float32, device=DEV)
    else:
        rows, V, ld, H = c["rows"], c["V"], c["ld"], c["hist"]
        s["logits"] = normal(rows, ld, std=3.0)
        # ids crowd at the low end of the vocabulary, as a tokenizer's frequent ones do
        s["history"] = (V * uniform(rows, H) ** 3).int().clamp_(0, V - 1)
        s["hist_len"] = (uniform(rows) * (H + 1)).int().clamp_(0, H)
        s["gen_start"] = (uniform(rows) * s["hist_len"]).int()
        one = uniform(rows) < 0.25  # rows that ask for no penalty
        s["repetition"] = torch.where(one, torch.ones_like(one, dtype=torch.float32), 1 + 0.3 * uniform(rows))
        s["presence"] = torch.where(one, 0.0, 0.6 * uniform(rows))
        s["frequency"] = torch.where(one, 0.0, 0.4 * uniform(rows))
        n = c["n_bias"]
        s["bias_ids"] = (V * uniform(rows, n)).int().clamp_(0, V - 1) if n else None
        s["bias_values"] = normal(rows, n, std=4.0) if n else None
        # a grammar that allows about an eighth of the ids
        s["allowed"] = None
        if c["mask"]:
            W = (V + 31) // 32
            bits = (uniform(rows, W * 32) < 0.125).view(rows, W, 32).long()
            words = (bits << torch.arange(32, device=DEV)).sum(2)
            s["allowed"] = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
        s["out"] = torch.empty(rows, V, device=DEV)
        s["next"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------- plain forms ---

def _plain_gemv(s):
    c = s["case"]
    N, K, group = c["N"], c["K"], c["group"]
    x = s["x"].float()
    y = torch.empty(c["rows"], N, device=DEV)
    for a, b in _chunks(N, K):
        p = s["packed"][a:b]
        q = torch.stack((p & 15, p >> 4), 2).view(b - a, K // group, group).float() - 8
        w = q * s["scales"][:, a:b].t().float()[:, :, None]
        y[:, a:b] = x @ w.view(b - a, K).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["out"].dtype)


def _plain_quantize(s):
    group = s["case"]["group"]
    q, sc = _q4(s["w"], group)
    n = (q + 8).to(torch.uint8)
    packed = n[:, 0::2] | (n[:, 1::2] << 4)
    q = torch.stack((packed & 15, packed >> 4), 2).view(-1, group).float() - 8
    return {"w": (q * sc.float().view(-1, 1)).view(s["w"].shape).bfloat16(), "scales": sc}


def _plain_prefix(s):
    c = s["case"]
    B, Hq, Hkv, hd, P, M = (c[k] for k in ("B", "Hq", "Hkv", "hd", "P", "max_len"))
    G = Hq // Hkv
    q = s["q"].float().view(B, Hkv, G, hd) / math.sqrt(hd)
    qp = q.permute(1, 0, 2, 3).reshape(Hkv, B * G, hd)
    zp = (qp @ s["pk"].float().transpose(1, 2)).view(Hkv, B, G, P).permute(1, 0, 2, 3)
    zo = q @ s["k"].float().transpose(2, 3)
    live = torch.arange(M, device=DEV)[None, :] < s["len"][:, None]
    zo = torch.where(live[:, None, None, :], zo, torch.full_like(zo, -math.inf))
    z = torch.cat((zp, zo), 3)
    m = z.amax(3, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m0)
    l = p.sum(3, keepdim=True)
    op = p[..., :P].permute(1, 0, 2, 3).reshape(Hkv, B * G, P) @ s["pv"].float()
    oo = p[..., P:] @ torch.where(live[:, None, :, None], s["v"].float(), torch.zeros_like(s["v"], dtype=torch.float32))
    o = (op.view(Hkv, B, G, hd).permute(1, 0, 2, 3) + oo) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m0 + torch.log(l)).view(B, Hq)
    return {"o": o.reshape(B, Hq, hd).bfloat16(), "lse": lse}


def _plain_rules(s):
    c = s["case"]
    rows, V, H = c["rows"], c["V"], c["hist"]
    z = s["logits"][:, :V]
    at = torch.arange(H, device=DEV)[None, :]
    h = s["history"].long()
    ones = torch.ones(rows, H, device=DEV)
    in_all = torch.where(at < s["hist_len"][:, None], ones, 0 * ones)
    in_gen = torch.where(at >= s["gen_start"][:, None], in_all, 0 * ones)
    seen = torch.zeros(rows, V, device=DEV).scatter_add_(1, h, in_all) > 0
    count = torch.zeros(rows, V, device=DEV).scatter_add_(1, h, in_gen)
    rep = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - s["frequency"][:, None] * count
    z = z - torch.where(count > 0, s["presence"][:, None], torch.zeros_like(z))
    if s["bias_ids"] is not None:
        n = c["n_bias"]
        order = torch.arange(1, n + 1, device=DEV).expand(rows, n)  # the last entry of an id counts
        last = torch.zeros(rows, V, dtype=torch.int64, device=DEV).scatter_reduce_(1, s["bias_ids"].long(), order, "amax")
        table = torch.cat((torch.zeros(rows, 1, device=DEV), s["bias_values"]), 1)
        z = torch.where(last > 0, z + table.gather(1, last), z)
    if s["allowed"] is not None:
        bits = (s["allowed"][:, :, None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
        z = torch.where(bits.view(rows, -1)[:, :V] > 0, z, torch.full_like(z, -math.inf))
    top = z.amax(1, keepdim=True)
    ids = torch.arange(V, dtype=torch.int32, device=DEV)[None, :]
    return {"z": z, "next": torch.where(z == top, ids, torch.full_like(ids, V)).amin(1)}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"gemv": _plain_gemv, "quantize": _plain_quantize, "prefix": _plain_prefix, "rules": _plain_rules}[c["op"]](s)
    import decoder_only_transformer_step_b200 as gp
    if c["op"] == "gemv":
        gp.gpt2_op_gemv_q4(s["x"], c["K"], s["packed"], s["scales"], s["bias"], s["out"], int(c["out_fp32"]), c["N"],
                           c["rows"], c["N"], c["K"], c["group"])
        return s["out"]
    if c["op"] == "quantize":
        N, K, group = c["N"], c["K"], c["group"]
        gp.gpt2_op_q4_quantize(s["w"], int(c["w_fp32"]), K, N, K, group, s["packed"], s["scales"])
        gp.gpt2_op_q4_dequantize(s["packed"], s["scales"], N, K, group, s["out"], 0, K)
        return {"w": s["out"], "scales": s["scales"][:, :N].t()}
    if c["op"] == "prefix":
        B, Hq, Hkv, hd, P, M = (c[k] for k in ("B", "Hq", "Hkv", "hd", "P", "max_len"))
        if "scratch" not in s:  # a workspace of the batch, kept as a decode loop keeps it
            n = gp.gpt2_op_prefix_attention_scratch_bytes(B, Hq, Hkv, hd, P, M)
            s["scratch"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        gp.gpt2_op_prefix_attention_bf16(s["q"], Hq * hd, s["pk"], s["pv"], P, P, s["k"], s["v"], s["len"], M, s["out"],
                                         Hq * hd, s["lse"], s["scratch"], B, Hq, Hkv, hd)
        return {"o": s["out"], "lse": s["lse"]}
    if "rules" not in s:  # the rules of the batch, kept as a decode loop keeps them
        s["rules"] = gp.LogitRules(history=s["history"], history_len=s["hist_len"], gen_start=s["gen_start"],
                                   repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                                   bias_ids=s["bias_ids"], bias_values=s["bias_values"], allowed=s["allowed"])
    gp.gpt2_op_logit_rules(s["logits"], c["ld"], s["out"], c["V"], c["rows"], c["V"], s["rules"], s["next"])
    return {"z": s["out"], "next": s["next"]}


# ------------------------------------------------------------------- exact ---

def exact(case, seed):
    s, c = prepare(case, seed), case
    d = torch.float64
    if c["op"] == "gemv":
        N, K, group = c["N"], c["K"], c["group"]
        x, y = s["x"].to(d), torch.empty(c["rows"], N, dtype=d, device=DEV)
        for a, b in _chunks(N, 2 * K):
            by = s["packed"][a:b].to(torch.int16)
            w = torch.empty(b - a, K, dtype=d, device=DEV)
            w[:, 0::2] = (by % 16 - 8).to(d)
            w[:, 1::2] = (by // 16 - 8).to(d)
            w *= s["scales"][:, a:b].to(d).t().repeat_interleave(group, 1)
            y[:, a:b] = x @ w.t()
        return y if s["bias"] is None else y + s["bias"].to(d)
    if c["op"] == "quantize":
        w = s["w"].to(d).reshape(-1, c["group"])
        sc = (w.abs().max(1, keepdim=True).values / 7).bfloat16().to(d)
        q = torch.where(sc > 0, torch.round(w / sc), 0 * w).clamp(-7, 7)
        return {"w": (q * sc).view(s["w"].shape), "scales": sc.view(c["N"], -1)}
    if c["op"] == "prefix":
        B, Hq, Hkv, hd, P = (c[k] for k in ("B", "Hq", "Hkv", "hd", "P"))
        G, lens = Hq // Hkv, _lens(c)
        o = torch.zeros(B, Hq, hd, dtype=d, device=DEV)
        lse = torch.full((B, Hq), -math.inf, dtype=d, device=DEV)
        for h in range(Hkv):
            pk, pv = s["pk"][h].to(d), s["pv"][h].to(d)
            for b in range(B):
                if P + lens[b] == 0:
                    continue
                k = torch.cat((pk, s["k"][b, h, : lens[b]].to(d)))
                v = torch.cat((pv, s["v"][b, h, : lens[b]].to(d)))
                z = s["q"][b, h * G:(h + 1) * G].to(d) @ k.t() / math.sqrt(hd)
                o[b, h * G:(h + 1) * G] = torch.softmax(z, 1) @ v
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(z, 1)
        return {"o": o, "lse": lse}
    z = s["logits"][:, : c["V"]].to(d)
    for r in range(c["rows"]):
        n, g0 = int(s["hist_len"][r]), int(s["gen_start"][r])
        h = s["history"][r, :n].long()
        ids = torch.unique(h)
        v = z[r, ids]
        rep, pres, freq = (float(s[k][r]) for k in ("repetition", "presence", "frequency"))
        z[r, ids] = torch.where(v > 0, v / rep, v * rep)
        ids, times = torch.unique(h[g0:], return_counts=True)
        z[r, ids] -= freq * times.to(d) + pres
        if c["n_bias"]:
            entries = dict(zip(s["bias_ids"][r].tolist(), s["bias_values"][r].tolist()))
            at = torch.tensor(list(entries), device=DEV)
            z[r, at] += torch.tensor(list(entries.values()), dtype=d, device=DEV)
        if c["mask"]:
            words = s["allowed"][r].long() & 0xFFFFFFFF
            bit = torch.arange(c["V"], device=DEV)
            z[r] = torch.where((words[bit // 32] >> (bit % 32)) % 2 == 1, z[r], torch.full_like(z[r], -math.inf))
    return {"z": z, "next": None}
