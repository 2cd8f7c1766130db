"""4-bit weights with group scales against their definition: the quantiser
bit by bit against the same fp32 steps in numpy, the matrix-vector products
against 64 bits.

Tolerance of the products: operands are exact, sums are fp32.  A term passes
at most `depth` additions (inside the tensor core's 16-term sums, along a
group's products, over the groups, warps and blocks), each off by at most one
fp32 step (2^-23) of a partial sum that sum |s q x| bounds; the result is
rounded once to its type (half a step)."""
import numpy as np
import pytest
import torch

import decoder_only_transformer_step_b200 as gp

pytestmark = pytest.mark.gpu


def pitch(N):
    return (N + 7) // 8 * 8


def buffers(N, K, group):
    packed = torch.full((N, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((K // group, pitch(N)), 7.0, dtype=torch.bfloat16, device="cuda")
    return packed, scales


def bf16_np(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().float().numpy()


def reference_quantise(w, group):
    """(q int, s fp32 [N, K/group]) by the definition, in fp32 as it says."""
    N, K = w.shape
    g = w.astype(np.float32).reshape(N, K // group, group)
    s = bf16_np(np.abs(g).max(2) / np.float32(7))
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.clip(np.rint(g / s[:, :, None]), -7, 7)
    q = np.where(s[:, :, None] == 0, 0, q)
    return q.astype(np.int64).reshape(N, K), s


def unpack(packed):
    p = packed.cpu().numpy().astype(np.int64)
    q = np.empty((p.shape[0], p.shape[1] * 2), np.int64)
    q[:, 0::2], q[:, 1::2] = p & 15, p >> 4
    return q - 8


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("w32", [0, 1])
@pytest.mark.parametrize("N,k", [(1, 1), (3, 2), (33, 5), (130, 9)])
def test_quantize_is_its_definition(group, w32, N, k):
    K, ldw = k * group, k * group + 24
    rng = np.random.default_rng(N * 100 + k)
    w = (rng.standard_normal((N, ldw)) * 0.02).astype(np.float32)
    w[0, :group] = 0                                         # an empty group
    w[-1, :group] = np.linspace(-7, 7, group) * 0.25         # quotients at and next to halves
    w[-1, 0] = 1.75
    if N > 2:
        w[1, :group] *= np.float32(1e-41)                    # subnormal weights, a subnormal scale
        w[2, :group] *= np.float32(1e38)
    t = torch.from_numpy(w).cuda()
    if not w32:
        t = t.bfloat16()
        w = t.float().cpu().numpy()
    packed, scales = buffers(N, K, group)
    gp.gpt2_op_q4_quantize(t, w32, ldw, N, K, group, packed, scales)
    q, s = reference_quantise(w[:, :K], group)
    np.testing.assert_array_equal(unpack(packed), q)
    np.testing.assert_array_equal(scales.float().cpu().numpy()[:, :N], s.T)
    assert (scales[:, N:] == 0).all()
    # the error of a weight is at most half a scale (plus what the clamp of a
    # scale rounded down by half a bf16 step cuts off: 7 * 2^-9 scales)
    big = np.repeat(s, group, 1).astype(np.float64)
    ok = np.abs(w[:, :K].astype(np.float64) - q * big) <= big * (0.5 + 7 * 2**-8)
    assert ok[np.repeat(s > 1e-37, group, 1)].all()
    for out32 in (0, 1):
        out = torch.full((N, K + 8), 3.0, dtype=torch.float32 if out32 else torch.bfloat16, device="cuda")
        gp.gpt2_op_q4_dequantize(packed, scales, N, K, group, out, out32, K + 8)
        want = torch.from_numpy((q * np.repeat(s, group, 1)).astype(np.float32))
        assert torch.equal(out[:, :K].cpu(), want if out32 else want.bfloat16())
        assert (out[:, K:] == 3).all()


def test_groups_with_infinity_or_nan_stay_visible():
    w = torch.randn(4, 96, device="cuda")
    w[1, 40], w[2, 70] = float("inf"), float("nan")
    packed, scales = buffers(4, 96, 32)
    gp.gpt2_op_q4_quantize(w, 1, 96, 4, 96, 32, packed, scales)
    s = scales[:, :4].float().cpu()
    assert torch.isinf(s[1, 1]) and torch.isnan(s[2, 2]) and int(torch.isfinite(s).sum()) == 10
    x = torch.ones(1, 96, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(1, 4, device="cuda")
    gp.gpt2_op_gemv_q4(x, 96, packed, scales, None, y, 1, 4, 1, 4, 96, 32)
    assert torch.isfinite(y[0]).tolist() == [True, False, False, True]


def gemv_case(rows, N, K, group, out32, bias, seed, ldx=None, ldo=None):
    rng = np.random.default_rng(seed)
    ldx, ldo = ldx or K, ldo or N
    nib = rng.integers(0, 16, size=(N, K)).astype(np.uint8)
    packed = torch.from_numpy(nib[:, 0::2] | (nib[:, 1::2] << 4)).cuda()
    sc = np.zeros((K // group, pitch(N)), np.float32)
    sc[:, :N] = bf16_np(0.01 * np.exp(rng.standard_normal((K // group, N))))
    sc[:, N:] = np.nan                                        # never read into a result
    scales = torch.from_numpy(sc).cuda().bfloat16()
    x = torch.full((rows, ldx), float("nan"), dtype=torch.bfloat16, device="cuda")
    xv = bf16_np(rng.standard_normal((rows, K)))
    x[:, :K] = torch.from_numpy(xv).cuda().bfloat16()
    b = bf16_np(rng.standard_normal(N)) if bias else None
    out = torch.full((rows, ldo), 77.0, dtype=torch.float32 if out32 else torch.bfloat16, device="cuda")
    bt = torch.from_numpy(b).cuda().bfloat16() if bias else None
    gp.gpt2_op_gemv_q4(x, ldx, packed, scales, bt, out, out32, ldo, rows, N, K, group)
    W = torch.from_numpy(nib.astype(np.float64) - 8).cuda() * scales[:, :N].double().t().repeat_interleave(group, 1)
    x64 = torch.from_numpy(xv).cuda().double()
    y = x64 @ W.t()
    mag = x64.abs() @ W.abs().t()
    if bias:
        y, mag = y + bt.double(), mag + bt.double().abs()
    depth = (group // 32) * 17 + K / group + 16 + 8 + 3
    got = out[:, :N].double()
    tol = depth * 2.0**-23 * mag + (2.0**-24 if out32 else 2.0**-8) * y.abs() * (1 + 2.0**-7)
    assert bool(((got - y).abs() <= tol).all()), float(((got - y).abs() / tol).max())
    assert bool((out[:, N:] == 77).all())
    return packed, scales, x, out


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", [1, 3, 8, 9, 16])
@pytest.mark.parametrize("N,K", [(1, 128), (15, 256), (17, 384), (130, 1280), (2305, 896), (40, 6400)])
def test_gemv_against_64_bits(group, rows, N, K):
    gemv_case(rows, N, K, group, out32=(rows + N) % 2, bias=rows % 2, seed=rows * 7 + N, ldx=K + 8 * (rows % 3),
              ldo=N + rows % 4)


@pytest.mark.parametrize("N,K,group,rows", [(9, 32, 32, 2), (5, 96, 32, 16), (21, 160, 32, 1), (64, 1600, 64, 16),
                                            (7, 64, 64, 5), (100, 28672, 128, 16), (33, 32768, 32, 16),
                                            (300, 32768, 64, 8), (5000, 8192, 128, 4), (2000, 20480, 32, 9),
                                            # several tiles a block one after the other
                                            (40001, 64, 32, 3), (20011, 1600, 64, 12), (30000, 2048, 128, 1),
                                            (50304, 768, 32, 16), (17000, 12800, 64, 16)])
def test_gemv_odd_lengths_and_inputs_split_over_a_cluster(N, K, group, rows):
    gemv_case(rows, N, K, group, out32=1, bias=0, seed=N + K)


def test_gemv_repeats_bitwise_on_streams_and_in_a_graph():
    packed, scales, x, out = gemv_case(8, 2000, 1600, 64, 1, 0, 3)
    first = out.clone()
    s = torch.cuda.Stream()
    other = torch.zeros_like(out)
    s.wait_stream(torch.cuda.current_stream())
    gp.gpt2_op_gemv_q4(x, 1600, packed, scales, None, other, 1, 2000, 8, 2000, 1600, 64, stream=s)
    s.synchronize()
    assert torch.equal(other, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            gp.gpt2_op_gemv_q4(x, 1600, packed, scales, None, other, 1, 2000, 8, 2000, 1600, 64)
    other.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(other, first)


def test_weights_quantised_just_before_are_the_ones_read():
    # the product may not run ahead of the quantiser on the same stream
    N, K, group = 4096, 1024, 64
    packed, scales = buffers(N, K, group)
    x = torch.randn(4, K, device="cuda").bfloat16()
    outs = [torch.empty(4, N, device="cuda") for _ in range(6)]
    ws = [torch.randn(N, K, device="cuda") * (i + 1) for i in range(6)]
    torch.cuda.synchronize()
    for w, o in zip(ws, outs):
        gp.gpt2_op_q4_quantize(w, 1, K, N, K, group, packed, scales)
        gp.gpt2_op_gemv_q4(x, K, packed, scales, None, o, 1, N, 4, N, K, group)
    deq = torch.empty(N, K, device="cuda")
    for w, o in zip(ws, outs):
        gp.gpt2_op_q4_quantize(w, 1, K, N, K, group, packed, scales)
        gp.gpt2_op_q4_dequantize(packed, scales, N, K, group, deq, 1, K)
        y, mag = x.double() @ deq.double().t(), x.double().abs() @ deq.double().abs().t()
        assert bool(((o.double() - y).abs() <= 80 * 2.0**-23 * mag).all())


@pytest.mark.parametrize("scale", [1.0, 0.02, 3e-38, 1e37])
def test_bf16_weights_at_and_around_halves(scale):
    # every bf16 significand against every scale significand: quotients at exact halves among them
    K, group = 256, 32
    rng = np.random.default_rng(21)
    w = (rng.integers(-255, 256, size=(4096, K)) / 128.0).astype(np.float32)
    w[:, ::group] = 7 * (rng.integers(128, 256, size=(4096, K // group)) / 128.0) / 2   # sets the scale
    t = (torch.from_numpy(w) * scale).bfloat16().cuda()
    packed, scales = buffers(4096, K, group)
    gp.gpt2_op_q4_quantize(t, 0, K, 4096, K, group, packed, scales)
    q, s = reference_quantise(t.float().cpu().numpy(), group)
    np.testing.assert_array_equal(scales.float().cpu().numpy(), s.T)
    np.testing.assert_array_equal(unpack(packed), q)


@pytest.mark.parametrize("N,K,group", [(100, 512, 64), (3000, 1536, 32), (2100, 5376, 128)])
@pytest.mark.parametrize("rows", [4, 11])
def test_rows_of_any_magnitude_and_rows_that_are_not_finite(N, K, group, rows):
    # each row has a scale of its own, from the type's largest values to its subnormal ones; inside a row the
    # magnitudes span 2^40.  The tolerance is that of gemv_case, for the order of sums only: nothing else rounds.
    rng = np.random.default_rng(N)
    nib = rng.integers(1, 16, size=(N, K)).astype(np.uint8)
    packed = torch.from_numpy(nib[:, 0::2] | (nib[:, 1::2] << 4)).cuda()
    scales = torch.zeros(K // group, pitch(N), device="cuda").bfloat16()
    scales[:, :N] = torch.from_numpy(2.0 ** rng.integers(-12, -8, (K // group, N))).cuda()
    x = torch.from_numpy(rng.standard_normal((rows, K)) * 2.0 ** rng.integers(-40, 1, (rows, K)))
    x = (x * torch.tensor([[3e37], [1e-37], [3e-39], [1.0]][:4] + [[2e5]] * (rows - 4))).bfloat16().cuda()
    y = torch.empty(rows, N, device="cuda")
    gp.gpt2_op_gemv_q4(x, K, packed, scales, None, y, 1, N, rows, N, K, group)
    W = torch.from_numpy(nib.astype(np.float64) - 8).cuda() * scales[:, :N].double().t().repeat_interleave(group, 1)
    want, mag = x.double() @ W.t(), x.double().abs() @ W.abs().t()
    depth = (group // 32) * 17 + K / group + 16 + 8 + 3
    # (results below the smallest normal number are held in steps of 2^-149; x's two powers of two round once each)
    tol = depth * 2.0**-23 * mag + 2.0**-24 * want.abs() + 2.0**-148
    # -8 sum x starts a group's sum: its terms are in mag up to a factor 8 / |q| <= 8
    tol = tol + depth * 2.0**-23 * 8 * (x.double().abs() @ (W.abs() / (torch.from_numpy(nib.astype(np.float64) - 8).abs().cuda() + (torch.from_numpy(nib).cuda() == 8))).t())
    assert bool(((y.double() - want).abs() <= tol).all()), float(((y.double() - want).abs() / tol).max())
    x[1, 5], x[2, 7] = float("inf"), float("nan")
    z = torch.empty_like(y)
    gp.gpt2_op_gemv_q4(x, K, packed, scales, None, z, 1, N, rows, N, K, group)
    assert not bool(torch.isfinite(z[1:3]).any())
    keep = [r for r in range(rows) if r not in (1, 2)]
    assert torch.equal(z[keep], y[keep])


@pytest.mark.parametrize("N,K,group", [(100, 512, 64), (130, 1280, 32), (1500, 6400, 128),     # read directly
                                       (4200, 1536, 32), (2100, 5376, 64), (2100, 5376, 128),
                                       (20000, 512, 32), (20000, 512, 64), (20000, 512, 128)])  # streamed
@pytest.mark.parametrize("rows", [1, 7, 16])
@pytest.mark.parametrize("size", [-133, -126, -100, -70, -60, 60, 100, 118, 126])
def test_scales_of_any_magnitude(N, K, group, rows, size):
    # Scales near 2^size, x such that the results are ordinary numbers where x's range allows it.  An addition is
    # off by at most a step (2^-23) of sum |s (|q| + 8) |x|| (the streamed form starts a group at -8 sum x) and, where
    # the streamed form's sums are subnormal, by half of 2^-149 in its own unit, which is at most 2^19 max |x| of the row
    rng = np.random.default_rng(1000 + N + size)
    nib = rng.integers(0, 16, size=(N, K)).astype(np.uint8)
    packed = torch.from_numpy(nib[:, 0::2] | (nib[:, 1::2] << 4)).cuda()
    scales = torch.zeros(K // group, pitch(N), device="cuda").bfloat16()
    one = 2.0 ** (size + rng.integers(-2 if size > -130 else 0, 2, (K // group, N)))
    scales[:, :N] = torch.from_numpy(one).cuda()
    x = torch.from_numpy(rng.standard_normal((rows, K)) * 2.0 ** np.clip(-size, -100, 100)).bfloat16().cuda()
    y = torch.empty(rows, N, device="cuda")
    gp.gpt2_op_gemv_q4(x, K, packed, scales, None, y, 1, N, rows, N, K, group)
    s64 = scales[:, :N].double().t().repeat_interleave(group, 1)
    q = torch.from_numpy(nib.astype(np.float64) - 8).cuda()
    want, mag = x.double() @ (s64 * q).t(), x.double().abs() @ (s64 * (q.abs() + 8)).t()
    depth = (group // 32) * 17 + K / group + 16 + 8 + 3
    tol = depth * 2.0**-23 * mag + 2.0**-24 * want.abs() + depth * 2.0**-131 * x.double().abs().amax(1, keepdim=True) + 2.0**-148
    assert bool(torch.isfinite(y).all())
    assert bool(((y.double() - want).abs() <= tol).all()), float(((y.double() - want).abs() / tol).max())
    if size >= -100:  # (the last two terms are the smallest part of it there)
        assert bool((want.abs().amax(1) > 2.0**4 * tol.amax(1)).all())


@pytest.mark.parametrize("N,K,group", [(20000, 1536, 32), (20000, 384, 64), (20003, 1536, 128)])
@pytest.mark.parametrize("rows", [4, 11])
def test_streamed_rows_of_any_magnitude(N, K, group, rows):
    test_rows_of_any_magnitude_and_rows_that_are_not_finite(N, K, group, rows)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", [1, 8, 9, 16])
@pytest.mark.parametrize("N,K", [(2368, 1664), (4736, 768), (4752, 768), (9472, 128), (9488, 128), (160, 4096), (160, 8192),
                                 (90, 12288), (33, 16384)])
def test_gemv_on_both_sides_of_the_choice_of_kernel(N, K, group, rows):
    gemv_case(rows, N, K, group, out32=1, bias=1, seed=N + K + rows)
