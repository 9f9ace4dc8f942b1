"""The 4-bit weight calls on the GPU where the formulas are delicate: negative gates of the GELU,
weights that are no numbers, batches without tokens, waits that run out."""
import ctypes
import math

import pytest
import torch

import expert_routed_ffn_softmax_b200 as moe
import w4_reference as ref
from expert_routed_ffn_softmax_b200 import _abi

pytestmark = pytest.mark.gpu


def synced():
    assert moe.sync_status() == 0


def cut_of(T, K, N, geglu):
    """{CTAs of a unit's K, strips, units, blocks a chunk, fragments, take-over} of a product of group 32
    with zero points."""
    cut = (ctypes.c_int * 6)()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert moe.load().moe_debug_w4_cut(T, K, N, 32, _abi.MOE_FLAG_W4_ZEROS, geglu, sms, cut) == 0
    return list(cut)


# ----------------------------------------------------------------------------- GELU
def identity(E, H, group=64):
    """E identity matrices [H, H]: code 9 on the diagonal, 8 (the value 0) elsewhere, scales 1."""
    codes = torch.full((E, H, H), 8, dtype=torch.uint8)
    codes[:, torch.arange(H), torch.arange(H)] = 9
    scales = torch.ones((E, H, ref.groups(H, group)), dtype=torch.bfloat16)
    return moe.w4_pack(ref.nibbles(codes).cuda(), scales.cuda(), group=group)


def gates(T, H):
    """bf16 values over [-9, 4], -2, -3 and -4 among them."""
    x = torch.linspace(-9, 4, T * H, dtype=torch.float64).to(torch.bfloat16)
    x[:6] = torch.tensor([-2.0, -3.0, -4.0, -1.0, 0.0, -0.0])
    return x[torch.randperm(T * H, generator=torch.Generator().manual_seed(T))].view(T, H)


def geglu(x):
    """gelu_tanh(x) * x in float64, without a sum that cancels."""
    a = x.double()
    return a / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))) * a


def check_gelu(y, x):
    # With identity matrices every product is exact and y is h: one rounding to bf16 (half a step,
    # 2^-8) of a value in fp32.  Its exponent is at most 2 * 0.8 * (9 + 0.0447 * 9^3) = 67 in size and
    # carries five roundings of 2^-24 relative and one step of a two-unit exp: 67 * 5 * 2^-24 + 2^-22
    # < 2^-15; the product and the quotient add four more units.  2^-14 covers them.
    want = geglu(x)
    off = (y.cpu().double() - want).abs() / want.abs().clamp(min=1e-30)
    assert float(off.max()) <= ref.HALF_BF16 + 2.0 ** -14, float(off.max())


@pytest.mark.parametrize("T,H", [(1, 1024), (8, 128), (9, 128), (16, 64)])
def test_dense_gelu_of_negative_gates(T, H):
    m, x = identity(1, H), gates(T, H)
    check_gelu(moe.dense_ffn_w4(x.cuda(), m, m, m), x)
    synced()


@pytest.mark.parametrize("T,H", [(1, 1024), (3, 192), (16, 64)])
def test_layer_gelu_of_negative_gates(T, H):
    """One expert a token, weight 1."""
    m, x = identity(4, H), gates(T, H)
    wr = torch.zeros((H, 4), dtype=torch.bfloat16)
    check_gelu(moe.forward_w4(x.cuda(), wr.cuda(), m, m, m, 1), x)
    synced()


def test_gelu_far_from_zero():
    """Gates whose exponentials overflow or vanish: 0 on the left, the gate itself on the right."""
    m = identity(1, 64)
    x = torch.zeros((3, 64), dtype=torch.bfloat16)
    x[0, :5] = torch.tensor([-12.0, -40.0, -1e13, -1e18, -64.0])
    x[1, :5] = torch.tensor([12.0, 40.0, 1e13, 1e18, 64.0])
    y = moe.dense_ffn_w4(x.cuda(), m, m, m).cpu()
    assert float(y[0].abs().max()) < 1e-30 and float(y[2].abs().max()) == 0
    want = x[1].double() ** 2
    assert bool(((y[1].double() - want).abs() <= ref.HALF_BF16 * want).all())
    synced()


# ----------------------------------------------------------------------------- the quantiser
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantise_damaged_group_is_nan(group, zeros, bad):
    """A NaN or an infinity makes all of its group NaN, and nothing else: as the formulas have it."""
    E, K, N = 2, 192, 80
    g = torch.Generator().manual_seed(group)
    w = (torch.randn((E, K, N), generator=g) * 0.02 + 0.03).to(torch.bfloat16)   # codes above 8 mostly
    clean = moe.w4_dequantize(moe.w4_quantize(w.cuda(), group=group, zeros=zeros)).cpu()
    assert bool(clean.isfinite().all())
    at = [(0, 0, 0), (0, 31, 1), (1, 130, 79), (1, 191, 40), (0, 66, 16)]
    want = clean.clone()
    for e, k, n in at:
        w[e, k, n] = bad
        want[e, k // group * group:(k // group + 1) * group, n] = float("nan")
    q = moe.w4_quantize(w.cuda(), group=group, zeros=zeros)
    got = moe.w4_dequantize(q).cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0))
    # codes and zero points of such a group are 8
    rec = q.data.cpu()[0, 0, 0]
    assert rec[:16].tolist()[0:4] == [0x88] * 4
    if zeros:
        assert int(rec[512 + (64 if group == 32 else 32)]) == 8
    synced()


@pytest.mark.parametrize("group", [32, 128])
def test_quantise_range_past_fp32(group):
    """hi - lo that no fp32 holds: the scale is infinite, the group NaN."""
    w = torch.zeros((1, 128, 16))
    w[0, 0, 3], w[0, 1, 3] = 3e38, -3e38
    w[0, 64, 5] = 3e38
    q = moe.w4_quantize(w.to(torch.bfloat16).cuda(), group=group, zeros=True)
    d = moe.w4_dequantize(q).cpu()
    assert bool(d[0, :group, 3].isnan().all())
    keep = torch.ones_like(d, dtype=torch.bool)
    keep[0, :group, 3] = False
    assert bool(d[keep].isfinite().all()) and float(d[0, 64, 5]) > 2.9e38
    synced()


# ----------------------------------------------------------------------------- no tokens
def test_layer_without_tokens_counts_none():
    """Empty batches: counts and offsets are zeros, whatever the memory held."""
    E = 16
    m = identity(E, 64)
    wr = torch.zeros((64, E), dtype=torch.bfloat16, device="cuda")
    used = [torch.full((n,), 7, dtype=torch.int32, device="cuda") for n in (E, E + 1, 5) * 4]
    del used
    y, aux = moe.forward_w4(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), wr, m, m, m, 2, aux=True)
    assert y.shape == (0, 64) and aux["topk_weights"].shape == (0, 2) and aux["perm"].shape == (0,)
    assert aux["expert_counts"].tolist() == [0] * E
    assert aux["expert_offsets"].tolist() == [0] * (E + 1)
    assert aux["router_stats"].tolist() == [0] * 5


# ----------------------------------------------------------------------------- waits that run out
def random_weights(K, N, seed):
    """Random codes of group 32 under one scale and zero point, made on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    return moe.w4_pack(codes, torch.full((N, K // 32), 0.01, dtype=torch.bfloat16, device="cuda"),
                       torch.full((N, K // 32), 7, dtype=torch.uint8, device="cuda"), group=32)


def gives_up(call):
    """With the wait limit at next to nothing the call's waits run out: it returns, the error is
    reported once, and the next calls are right again."""
    want = call()
    synced()
    lib = moe.load()
    for _ in range(3):
        assert lib.moe_debug_set_wait_limit_ns(1) == 0
        try:
            call()
            status = moe.sync_status()
        finally:
            assert lib.moe_debug_set_wait_limit_ns(0) == 0
        assert status == _abi.MOE_ERR_TIMEOUT
        synced()
        assert torch.equal(call(), want)
    synced()


def test_linear_gives_up_while_units_are_taken_over():
    """A unit of 128 rows over K = 16384 takes some 90 us, during which the joining warps wait; each CTA
    has asked for its next unit by then."""
    T, K, N = 16, 16384, 131072
    assert cut_of(T, K, N, 0)[1::4] == [8, 1]
    w = random_weights(K, N, 1)
    x = torch.randn((T, K), device="cuda").to(torch.bfloat16)
    gives_up(lambda: moe.linear_w4(x, w))


def test_dense_gives_up_in_clusters_that_started_early():
    """The second product's first clusters start while the first product runs, and wait for its h."""
    T, H, I = 16, 16384, 5760
    assert cut_of(T, I, H, 0)[0] == 2 and cut_of(T, H, I, 1)[0] == 2
    g, u, d = random_weights(H, I, 1), random_weights(H, I, 2), random_weights(I, H, 3)
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    gives_up(lambda: moe.dense_ffn_w4(x, g, u, d))


# ----------------------------------------------------------------------------- the binding
def test_dense_ffn_takes_dequantised_matrices():
    """The documented way to larger batches: one matrix of w4_dequantize is what dense_ffn takes.  The
    two round alike (h and y to bf16), but for sums in another order and dense_ffn's weights, each
    rounded once: three half steps."""
    H, I = 256, 192
    g = torch.Generator(device="cuda").manual_seed(1)
    q = [moe.w4_quantize((torch.randn(s, generator=g, device="cuda") * 0.05).to(torch.bfloat16), zeros=True)
         for s in ((H, I), (H, I), (I, H))]
    x = torch.randn((64, H), generator=g, device="cuda").to(torch.bfloat16)
    y = moe.dense_ffn(x, *[moe.w4_dequantize(m)[0] for m in q]).double()
    z = torch.cat([moe.dense_ffn_w4(x[i:i + 16], *q) for i in range(0, 64, 16)]).double()
    assert float((y - z).norm() / z.norm()) < 3 * ref.HALF_BF16
    synced()


def test_pack_refuses_what_is_no_tensor():
    c = torch.zeros((32, 64), dtype=torch.uint8, device="cuda")
    s = torch.ones((32, 2), dtype=torch.bfloat16, device="cuda")
    for bad in ((c, None, None), (c, 1.0, None), (c, s, 8), (c.unsqueeze(0), s.unsqueeze(0), [8])):
        with pytest.raises(TypeError):
            moe.w4_pack(*bad)
