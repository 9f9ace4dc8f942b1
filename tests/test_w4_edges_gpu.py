"""The 4-bit weight calls on the GPU where the formulas are delicate: negative gates of the GELU."""
import math

import pytest
import torch

import expert_routed_ffn_softmax_b200 as moe
import w4_reference as ref

pytestmark = pytest.mark.gpu


def synced():
    assert moe.sync_status() == 0


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
