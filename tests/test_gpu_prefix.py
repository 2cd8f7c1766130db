"""Attention over a shared prefix and each row's own positions against its
definition in 64 bits.

Tolerance of o: the probabilities are rounded to bf16 before the second
product, half a step (2^-8 relative) each, so o is off by at most
2^-8 sum p |v|; the fp32 sums and exponentials add less than 2^-14 of the same
(2^-22 a step over the longest chain of steps here), a score off by s changes
a probability by a share 2 s at most, and o itself is rounded once, 2^-8 |o|.
lse: a score's hd products are exact, their sum off by 2^-23 of their
magnitudes each time; the sum of the exponentials as above.
"""
import math

import numpy as np
import pytest
import torch

import decoder_only_transformer_step_b200 as gp

pytestmark = pytest.mark.gpu


def make(B, Hq, Hkv, hd, P, max_len, lens, seed, cap=None, ldq=None, ldo=None, q_std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rnd(*s):
        return torch.empty(s, device="cuda").normal_(generator=g).bfloat16()
    cap = cap or P
    ldq, ldo = ldq or Hq * hd, ldo or Hq * hd
    s = dict(B=B, Hq=Hq, Hkv=Hkv, hd=hd, P=P, cap=cap, max_len=max_len, ldq=ldq, ldo=ldo, lens=lens)
    s["q"] = rnd(B, ldq) * q_std
    s["pk"], s["pv"] = rnd(Hkv, cap, hd), rnd(Hkv, cap, hd)
    s["k"], s["v"] = rnd(B, Hkv, max_len, hd), rnd(B, Hkv, max_len, hd)
    s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["o"] = torch.full((B, ldo), 55.0, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.full((B, Hq), 9.0, device="cuda")
    n = gp.gpt2_op_prefix_attention_scratch_bytes(B, Hq, Hkv, hd, P, max_len)
    s["scratch"] = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN where nothing is written
    return s


def call(s, stream=None):
    gp.gpt2_op_prefix_attention_bf16(s["q"], s["ldq"], s["pk"], s["pv"], s["P"], s["cap"], s["k"], s["v"], s["len"],
                                     s["max_len"], s["o"], s["ldo"], s["lse"], s["scratch"], s["B"], s["Hq"], s["Hkv"],
                                     s["hd"], stream=stream)


def check(s):
    B, Hq, Hkv, hd, P = (s[k] for k in ("B", "Hq", "Hkv", "hd", "P"))
    G = Hq // Hkv
    q = s["q"][:, : Hq * hd].double().view(B, Hq, hd)
    o = s["o"][:, : Hq * hd].double().view(B, Hq, hd)
    for b in range(B):
        n = max(0, min(s["max_len"], s["lens"][b]))
        if P + n == 0:
            assert bool((o[b] == 0).all()) and bool((s["lse"][b] == -math.inf).all())
            continue
        k = torch.cat((s["pk"][:, :P].double(), s["k"][b, :, :n].double()), 1).repeat_interleave(G, 0)
        v = torch.cat((s["pv"][:, :P].double(), s["v"][b, :, :n].double()), 1).repeat_interleave(G, 0)
        z = torch.einsum("hd,hjd->hj", q[b], k) / math.sqrt(hd)
        mag = torch.einsum("hd,hjd->hj", q[b].abs(), k.abs()).amax(1) / math.sqrt(hd)
        p = torch.softmax(z, 1)
        want = torch.einsum("hj,hjd->hd", p, v)
        sc = (hd + 4) * 2.0**-23 * mag  # how far a score may be off
        tol = (2.0**-8 + 2.0**-14 + 4 * sc[:, None]) * torch.einsum("hj,hjd->hd", p, v.abs()) + 2.0**-8 * want.abs()
        err = (o[b] - want).abs()
        assert bool((err <= tol).all()), (b, float((err / tol).max()))
        lse = torch.logsumexp(z, 1)
        assert bool(((s["lse"][b].double() - lse).abs() <= 2 * sc + 2.0**-18 + 2.0**-22 * lse.abs()).all()), b
    assert bool((s["o"][:, Hq * hd:] == 55).all())


@pytest.mark.parametrize("hd", [16, 64, 128])
@pytest.mark.parametrize("P", [0, 1, 31, 129, 700])
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 2, 2), (3, 4, 2), (5, 3, 1), (17, 8, 8), (9, 40, 2)])
def test_prefix_attention_against_64_bits(hd, P, B, Hq, Hkv):
    max_len = 70
    lens = [(37 * b) % (max_len + 1) for b in range(B)]       # 0 and others
    lens[-1] = max_len
    s = make(B, Hq, Hkv, hd, P, max_len, lens, seed=P + B, cap=P + 3, ldq=Hq * hd + 6, ldo=Hq * hd + 2)
    # what lies behind the keys that count is not read
    s["pk"][:, P:] = float("nan")
    s["pv"][:, P:] = float("inf")
    for b, n in enumerate(lens):
        s["k"][b, :, n:] = float("nan")
        s["v"][b, :, n:] = float("-inf")
    call(s)
    check(s)


@pytest.mark.parametrize("B,Hq,Hkv,hd,P,max_len", [(33, 32, 8, 128, 3000, 40), (64, 8, 1, 64, 2049, 9),
                                                   (200, 4, 4, 64, 511, 33), (2, 64, 1, 128, 5000, 600),
                                                   (16, 12, 12, 64, 3500, 596), (1, 1, 1, 64, 40000, 1),
                                                   (5, 6, 3, 16, 3000, 50), (64, 8, 8, 16, 1100, 30), (16, 25, 25, 64, 768, 256),
                                                   (3, 12, 12, 64, 300, 1024), (8, 4, 4, 128, 200, 1500)])
def test_many_rows_and_long_prefixes(B, Hq, Hkv, hd, P, max_len):
    s = make(B, Hq, Hkv, hd, P, max_len, [(b * 13) % (max_len + 1) for b in range(B)], seed=B)
    call(s)
    check(s)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv", [(17, 3, 3), (32, 2, 2), (43, 3, 1), (64, 2, 1), (65, 4, 2), (40, 32, 8), (256, 1, 1),
                                      (129, 4, 2), (100, 8, 1)])
@pytest.mark.parametrize("P", [1024, 1151, 4000])
def test_many_rows_on_the_tensor_cores(hd, B, Hq, Hkv, P):
    # one row tile, two even and uneven ones, several row groups; a last block of keys of any length
    s = make(B, Hq, Hkv, hd, P, 20, [(b * 7) % 21 for b in range(B)], seed=P + B, cap=P + 5, ldq=Hq * hd + 2, ldo=Hq * hd + 4)
    s["pk"][:, P:] = float("nan")
    s["pv"][:, P:] = float("inf")
    call(s)
    check(s)


@pytest.mark.parametrize("hd,B,Hq,Hkv,P", [(64, 48, 1, 1, 29400), (64, 65, 2, 1, 11007), (64, 128, 2, 2, 11001),
                                           (64, 43, 3, 1, 10950), (64, 300, 1, 1, 4750), (64, 257, 2, 1, 3000),
                                           (128, 96, 1, 1, 7424), (128, 129, 2, 2, 5500), (128, 40, 32, 8, 4500),
                                           (128, 128, 1, 1, 5569), (128, 100, 8, 1, 1024), (128, 520, 1, 1, 1500)])
def test_much_work_on_the_tensor_cores(hd, B, Hq, Hkv, P):
    s = make(B, Hq, Hkv, hd, P, 20, [(b * 7) % 21 for b in range(B)], seed=P + B, cap=P + 5, ldq=Hq * hd + (B % 2) * 2,
             ldo=Hq * hd + 4)
    s["pk"][:, P:] = float("nan")
    s["pv"][:, P:] = float("inf")
    call(s)
    check(s)


def test_maxima_that_keep_growing():
    # keys ordered so that every block raises the maxima: the running sums are rescaled again and again
    s = make(40, 4, 1, 128, 3000, 0, [0] * 40, seed=8, q_std=3.0)
    s["q"] = s["q"].abs()
    s["pk"] = (s["pk"].abs() * torch.linspace(0.0, 1.5, 3000, device="cuda")[None, :, None]).bfloat16()
    call(s)
    check(s)
    s = make(80, 4, 1, 128, 3000, 0, [0] * 80, seed=9, q_std=3.0)   # the same on the tensor cores
    s["q"] = s["q"].abs()
    s["pk"] = (s["pk"].abs() * torch.linspace(0.0, 1.5, 3000, device="cuda")[None, :, None]).bfloat16()
    call(s)
    check(s)


def test_sharp_scores_and_lengths_out_of_range():
    # scores of +-60: one key takes nearly all weight; lengths below 0 and past max_len are clamped
    s = make(4, 4, 4, 64, 257, 40, [-5, 0, 41, 1 << 30], seed=1, q_std=8.0)
    call(s)
    check(s)


def test_no_keys_at_all_and_null_parts():
    s = make(2, 4, 4, 64, 0, 0, [0, 0], seed=2)
    s["pk"] = s["pv"] = s["k"] = s["v"] = s["len"] = None
    call(s)
    assert bool((s["o"] == 0).all()) and bool((s["lse"] == -math.inf).all())


def test_without_own_positions_or_lse():
    s = make(3, 4, 4, 64, 300, 0, [0, 0, 0], seed=3)
    s["lse"] = None
    call(s)
    s["lse"] = torch.zeros(3, 4, device="cuda")
    o = s["o"].clone()
    call(s)
    assert torch.equal(o, s["o"])
    check(s)


def test_it_repeats_bitwise_and_in_a_graph_whose_lengths_grow():
    s = make(5, 12, 12, 64, 600, 300, [0, 7, 100, 299, 300], seed=4)
    call(s)
    o, lse = s["o"].clone(), s["lse"].clone()
    s["scratch"].fill_(0xFF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(s, stream=side)
    side.synchronize()
    assert torch.equal(o, s["o"]) and torch.equal(lse, s["lse"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(s)
    s["lens"] = [1, 8, 101, 300, 300]
    s["len"].copy_(torch.tensor(s["lens"], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    check(s)


def test_a_cache_whose_offsets_pass_32_bits():
    # 2^31 elements and more before the last head's keys and the last row's own
    B, H, hd, cap = 1, 9, 128, 1 << 21
    k = torch.zeros(H, cap, hd, dtype=torch.bfloat16, device="cuda")
    s = make(B, H, H, hd, 200, 1, [0], seed=5)
    k[:, :200] = s["pk"]
    s["pk"] = s["pv"] = k
    s["cap"] = cap
    call(s)
    check(s)
    own = torch.zeros(9, 1, cap, hd, dtype=torch.bfloat16, device="cuda")
    s = make(9, 1, 1, hd, 0, 4, [0, 1, 0, 2, 0, 3, 0, 0, 100], seed=6)
    own[:, :, :100] = torch.randn(9, 1, 100, hd, device="cuda").bfloat16()
    s["k"] = s["v"] = own
    s["max_len"] = cap
    s["scratch"] = torch.empty(gp.gpt2_op_prefix_attention_scratch_bytes(9, 1, 1, hd, 0, cap), dtype=torch.uint8,
                               device="cuda")
    call(s)
    check(s)


@pytest.mark.parametrize("hd,B,Hq,Hkv,P", [(64, 128, 12, 12, 16321), (64, 150, 24, 24, 16001), (64, 64, 75, 75, 22001),
                                           (64, 25, 150, 30, 12001), (64, 257, 20, 20, 5601),
                                           (128, 50, 37, 37, 14999), (128, 130, 40, 40, 6001), (128, 300, 25, 25, 2500),
                                           (128, 24, 150, 75, 15000)])
def test_long_parts_on_the_tensor_cores(hd, B, Hq, Hkv, P):
    # so many key/value heads that a block takes 1024 keys and more: 20 to 344 steps, the ring of tiles used again and
    # again; one row tile and two, several row groups, odd and even numbers of steps, a last step of any length
    s = make(B, Hq, Hkv, hd, P, 3, [b % 4 for b in range(B)], seed=P + B, cap=P + 1, ldq=Hq * hd + (B % 2) * 2)
    s["pk"][:, P:] = float("nan")
    s["pv"][:, P:] = float("inf")
    call(s)
    check(s)


@pytest.mark.parametrize("hd,B,P", [(128, 128, 5633), (128, 256, 2817), (64, 128, 11001), (64, 200, 7100)])
@pytest.mark.parametrize("grow", [3.0, 9.0, 20.0])
def test_maxima_that_grow_at_every_step_of_long_parts(hd, B, P, grow):
    # one block a head takes the whole prefix.  The scores of the even rows grow by a factor 2^grow a step of 64 keys
    # (above 2^8 every step rescales what came before, below it every few steps), those of the odd rows fall
    H = 75
    s = make(B, H, H, hd, P, 0, [0] * B, seed=B + P)
    u = torch.where(torch.arange(hd, device="cuda") % 3 == 0, -1.0, 1.0)
    top = grow * math.log(2) * P / 64                              # the largest score
    c = math.sqrt(top / math.sqrt(hd))
    sign = torch.where(torch.arange(B, device="cuda") % 2 == 0, 1.0, -1.0)
    s["q"] = (sign[:, None, None] * c * u + 0.1 * s["q"].float().view(B, H, hd)).bfloat16().view(B, H * hd)
    ramp = torch.linspace(0.0, c, P, device="cuda")
    s["pk"] = (ramp[None, :, None] * u + 0.1 * s["pk"].float()).bfloat16()
    call(s)
    check(s)


@pytest.mark.parametrize("hd,keys", [(16, 640), (64, 512), (128, 256)])
@pytest.mark.parametrize("over", [0, 1])
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 12, 12), (16, 25, 25), (7, 34, 2), (33, 32, 32)])
def test_both_sides_of_the_choice_of_kernel(hd, keys, over, B, Hq, Hkv):
    # a block for all keys of its rows up to so many keys (and 55 MB in all), parts that are joined beyond
    m = 90
    s = make(B, Hq, Hkv, hd, keys + over - m, m, [(b * 41) % (m + 1) for b in range(B - 1)] + [m], seed=B + hd)
    call(s)
    check(s)
