"""The 4-bit weight calls over their whole reach: every batch size, every way of cutting a product,
byte offsets past 32 bits, routing weights beside moe_route's."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import expert_routed_ffn_softmax_b200 as moe
import w4_reference as ref
from expert_routed_ffn_softmax_b200 import _abi
from w4_cuts import CUTS

pytestmark = pytest.mark.gpu

FORMS = [(32, False), (32, True), (64, False), (64, True), (128, False), (128, True)]


def synced():
    assert moe.sync_status() == 0


def gpu_matrix(K, N, group, zeros, seed, E=1):
    """(W4Weights, float64 values [E, K, N] on the GPU) of random codes, zero points and scales."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    G = ref.groups(K, group)
    codes = torch.randint(0, 16, (E, N, K), generator=g, device="cuda", dtype=torch.uint8)
    zp = torch.randint(0, 16, (E, N, G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    scales = ((torch.rand((E, N, G), generator=g, device="cuda") - 0.3) * 0.01).to(torch.bfloat16)
    w = moe.w4_pack(ref.nibbles(codes), scales, zp, group=group)
    wide = lambda t: t.double().repeat_interleave(group, -1)[..., :K]  # noqa: E731
    v = codes.double()
    v -= 8.0 if zp is None else wide(zp)
    v *= wide(scales)
    return w, v.transpose(1, 2)


def rows(T, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)


def check(got, y, err):
    ref.check(got, y.cpu(), err.cpu())


# ----------------------------------------------------------------------------- products
@pytest.mark.parametrize("T", [4, 5, 6, 10, 11, 12, 14, 15])
@pytest.mark.parametrize("group,zeros", FORMS)
def test_linear_the_other_batch_sizes(T, group, zeros):
    w, v = gpu_matrix(704, 144, group, zeros, seed=T)
    x = rows(T, 704, T)
    y, err = ref.linear(x, v[0], group)
    check(moe.linear_w4(x, w), y, err)
    check(moe.linear_w4(x, w, fp32=True), y, err)
    synced()


@pytest.mark.parametrize("row", CUTS, ids=lambda r: "-".join(map(str, r)))
def test_every_cut(row):
    """Each cut on this device's SMs, in fp32 and bf16, and the same bits from the same call."""
    geglu, cluster, strips, frag, steal, T, K, N, group, zeros = row
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cut = (ctypes.c_int * 6)()
    lib = moe.load()
    assert lib.moe_debug_w4_cut(T, K, N, group, _abi.MOE_FLAG_W4_ZEROS if zeros else 0, geglu, sms, cut) == 0
    assert sms != 148 or (cut[0], cut[1], cut[4], cut[5]) == (cluster, strips, frag, steal)
    x = rows(T, K, N)
    if geglu:
        (g, vg), (u, vu) = gpu_matrix(K, N, group, zeros, 1), gpu_matrix(K, N, group, zeros, 2)
        d, vd = gpu_matrix(N, K, group, zeros, 3)
        y, err = ref.ffn(x, vg[0], vu[0], vd[0], group)
        got = moe.dense_ffn_w4(x, g, u, d)
        check(got, y, err)
        assert torch.equal(moe.dense_ffn_w4(x, g, u, d), got)
    else:
        w, v = gpu_matrix(K, N, group, zeros, 1)
        y, err = ref.linear(x, v[0], group)
        got = moe.linear_w4(x, w, fp32=True)
        check(got, y, err)
        assert torch.equal(moe.linear_w4(x, w, fp32=True), got)
        assert torch.equal(moe.linear_w4(x, w), got.to(torch.bfloat16))
    synced()


# ----------------------------------------------------------------------------- far offsets
def one_filled(E, K, N, code=0x88):
    """W4Weights of group 64 with scales 1 and every code 8: the value 0."""
    shape = (E, N // 16, K // 64, 544)
    data = torch.full(shape, code, dtype=torch.uint8, device="cuda")
    data[..., 512:] = torch.tensor([0x80, 0x3F], dtype=torch.uint8, device="cuda").repeat(16)
    return moe.W4Weights(data, E, K, N, 64, False)


def test_linear_past_4_gib():
    K, N = 16384, 520016
    w = one_filled(1, K, N)
    assert w.data.numel() > 1 << 32
    w.data[0, -1, -1, :512] = 0x99                         # last strip, last block: the value 1
    w.data[0, (1 << 32) // (544 * 256) + 1, 0, :512] = 0xAA   # the strip past 2^32 bytes: 2
    x = torch.zeros((2, K), dtype=torch.bfloat16, device="cuda")
    x[0, -1] = 2.0
    x[1] = 1.0
    y = moe.linear_w4(x, w, fp32=True)
    want = torch.zeros_like(y)
    want[0, -16:], want[1, -16:] = 2, 64
    far = 16 * ((1 << 32) // (544 * 256) + 1)
    want[1, far:far + 16] = 128
    assert torch.equal(y, want)
    synced()


def test_weights_past_4_gib():
    """Quantise, pack and dequantise: the last of 260 matrices is as it is alone."""
    E, K, N = 260, 4096, 8192
    w = torch.zeros((E, K, N), dtype=torch.bfloat16, device="cuda")
    w[-1] = rows(K, N, 1)
    w[3] = rows(K, N, 2)
    for zeros in (False, True):
        q = moe.w4_quantize(w, group=64, zeros=zeros)
        assert q.data[:-1].numel() > 1 << 32
        for e in (-1, 3):
            assert torch.equal(q.data[e], moe.w4_quantize(w[e], group=64, zeros=zeros).data[0])
        assert torch.equal(q.data[4], q.data[258])
    del w
    back = moe.w4_dequantize(q)
    for e in (-1, 3, 4):
        part = moe.W4Weights(q.data[e].unsqueeze(0), 1, K, N, 64, True)
        assert torch.equal(back[e], moe.w4_dequantize(part)[0])
    del back, q
    codes = torch.full((E, N, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    codes[-1] = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8)
    scales = torch.ones((E, N, K // 64), dtype=torch.bfloat16, device="cuda")
    scales[-1] = rows(N, K // 64, 3)
    assert codes[:-1].numel() > 1 << 32
    p = moe.w4_pack(codes, scales, group=64)
    assert torch.equal(p.data[-1], moe.w4_pack(codes[-1], scales[-1], group=64).data[0])
    assert torch.equal(p.data[0], p.data[258])
    synced()


def test_layer_past_4_gib():
    """The last of 256 experts of more than 16 MiB a projection is as the last of 4."""
    T, H, E, I = 5, 4096, 256, 8192
    few = [gpu_matrix(*s, 64, False, 5 + i)[0] for i, s in enumerate(((H, I), (H, I), (I, H)))]
    x = rows(T, H, 9)
    y = []
    for n in (4, E):
        q = []
        for m in few:
            w = one_filled(n, m.K, m.N)
            w.data[-1] = m.data[0]
            q.append(w)
        if n == E:
            assert q[0].data[:-1].numel() > 1 << 32 and q[2].data[:-1].numel() > 1 << 32
        wr = torch.zeros((H, n), dtype=torch.bfloat16, device="cuda")
        bias = torch.zeros(n, device="cuda")
        bias[-1] = 5.0
        y.append(moe.forward_w4(x, wr, *q, 1, bias=bias))
        del q
    assert torch.equal(y[0], y[1]) and float(y[0].abs().max()) > 0
    synced()


# ----------------------------------------------------------------------------- the router
@pytest.mark.parametrize("T,H,E,k,spread,bias", [
    (1, 2816, 128, 8, 0.02, False), (16, 2816, 128, 8, 0.02, True), (9, 256, 256, 8, 0.5, False),
    (16, 64, 4, 4, 2.0, True), (5, 4096, 12, 3, 0.001, False), (16, 16384, 64, 8, 0.01, False)])
@pytest.mark.parametrize("renorm", [True, False])
def test_layer_weights_are_within_1e6_of_route(T, H, E, k, spread, bias, renorm):
    """The softmax in fp32 of fp64 differences d: exp(d) is off by |d| exp(d) 2^-24 <= 0.37 * 2^-24 for
    rounding d and two units for the exponential, the sum and the quotient by as much again: under
    2^-20 < 1e-6 for weights of at most 1."""
    q = [one_filled(E, *s) for s in ((H, 64), (H, 64), (64, H))]
    g = torch.Generator(device="cuda").manual_seed(E)
    wr = (torch.randn((H, E), generator=g, device="cuda") * spread).to(torch.bfloat16)
    b = torch.randn(E, generator=g, device="cuda") if bias else None
    x = rows(T, H, T)
    x[0] = 0                                  # every logit equal (but for the bias): the exact path
    _, aux = moe.forward_w4(x, wr, *q, k, bias=b, renorm=renorm, aux=True)
    ids, w = moe.route(x, wr, k, bias=b, renorm=renorm)
    assert torch.equal(aux["topk_ids"], ids)
    assert float((aux["topk_weights"].double() - w.double()).abs().max()) <= 1e-6
    exact = oracle.route(x.cpu(), wr.cpu(), k, bias=None if b is None else b.cpu(), renorm=renorm)[1]
    assert np.abs(aux["topk_weights"].cpu().numpy().astype(np.float64) - exact).max() <= 1e-6
    synced()


# ----------------------------------------------------------------------------- the limits
def test_linear_at_the_limits():
    for T, K, N in ((16, 64, 1048576), (1, 64, 1048576), (16, 16384, 16), (1, 16384, 16)):
        w, v = gpu_matrix(K, N, 64, True, 7)
        x = rows(T, K, 1)
        y, err = ref.linear(x, v[0], 64)
        check(moe.linear_w4(x, w, fp32=True), y, err)
    synced()


def test_dense_at_the_limits():
    T, H, I = 16, 16384, 8192
    m = [gpu_matrix(*s, 32, True, i) for i, s in enumerate(((H, I), (H, I), (I, H)))]
    x = (rows(T, H, 1).float() * 0.1).to(torch.bfloat16)
    y, err = ref.ffn(x, *[v[0] for _, v in m], 32)
    check(moe.dense_ffn_w4(x, *[w for w, _ in m]), y, err)
    synced()


def test_layer_at_the_limits():
    """The widest layer: every token on both of its experts' 134 M weights a projection."""
    T, H, I, E, k = 16, 16384, 8192, 4, 2
    m = [gpu_matrix(*s, 64, False, i, E) for i, s in enumerate(((H, I), (H, I), (I, H)))]
    x = (rows(T, H, 1).float() * 0.1).to(torch.bfloat16)
    wr = rows(H, E, 2)
    y, aux = moe.forward_w4(x, wr, *[w for w, _ in m], k, aux=True)
    ids, wts = moe.route(x, wr, k)
    assert torch.equal(aux["topk_ids"], ids)
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    err = torch.zeros_like(want)
    for e in range(E):
        o, eo = ref.ffn(x, *[v[e] for _, v in m], 64)
        w = (wts * (ids == e)).sum(1, keepdim=True).double()
        want += w * o
        err += w * eo + 1e-6 * (o.abs() + eo) + 4 * ref.U32 * w * o.abs()
    check(y, want, err)
    synced()


def test_many_small_matrices():
    """4096 matrices of one record a strip: pack, quantise and back."""
    E, K, N = 4096, 64, 16
    codes = torch.randint(0, 256, (E, N, K // 2), device="cuda", dtype=torch.uint8)
    scales = torch.rand((E, N, 1), device="cuda").to(torch.bfloat16)
    d = moe.w4_dequantize(moe.w4_pack(codes, scales, group=64))
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    assert torch.equal(d, ((c - 8) * scales.double()).transpose(1, 2).to(torch.bfloat16))
    q = moe.w4_quantize(d, group=64, zeros=True)
    assert torch.equal(q.data[4095], moe.w4_quantize(d[4095], group=64, zeros=True).data[0])
    synced()


# ----------------------------------------------------------------------------- odd values and places
def small_layer(T, k=3, seed=0):
    H, I, E = 256, 128, 16
    q = [gpu_matrix(*s, 64, True, seed + i, E)[0] for i, s in enumerate(((H, I), (H, I), (I, H)))]
    return rows(T, H, seed), rows(H, E, seed + 9), q, k


@pytest.mark.parametrize("T", [2, 7, 9, 16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_that_are_no_numbers_stay_apart(T, bad):
    """A damaged token reaches neither the other tokens of the layer and the dense MLP nor an id out of
    range; the call's status stays OK."""
    x, wr, q, k = small_layer(T)
    d = [gpu_matrix(*s, 64, True, 30 + i)[0] for i, s in enumerate(((256, 192), (256, 192), (192, 256)))]
    clean, dense = moe.forward_w4(x, wr, *q, k), moe.dense_ffn_w4(x, *d)
    x2 = x.clone()
    x2[T // 2, 5] = bad
    y, aux = moe.forward_w4(x2, wr, *q, k, aux=True)
    z = moe.dense_ffn_w4(x2, *d)
    keep = torch.arange(T) != T // 2
    ids = aux["topk_ids"]
    assert bool(((ids >= 0) & (ids < 16)).all()) and int(aux["expert_counts"].sum()) == T * k
    ids2, _ = moe.route(x2, wr, k)
    assert torch.equal(ids, ids2)
    # units of the same height: a token's sums are in the same order, whoever shares its experts
    assert torch.equal(y[keep], clean[keep]) and torch.equal(z[keep], dense[keep])
    assert bool(y[T // 2].isnan().any()) and bool(z[T // 2].isnan().any())
    synced()


def test_bias_that_masks_experts():
    """Experts at the lowest fp32 value or at -infinity are not chosen while others are left."""
    x, wr, q, k = small_layer(8)
    for low in (torch.finfo(torch.float32).min, float("-inf")):
        b = torch.zeros(16, device="cuda")
        b[2::2] = low
        b[1] = low
        y, aux = moe.forward_w4(x, wr, *q, k, bias=b, aux=True)
        ids, w = moe.route(x, wr, k, bias=b)
        assert torch.equal(aux["topk_ids"], ids) and bool((b[ids.long()] == 0).all())
        assert float((aux["topk_weights"] - w).abs().max()) <= 1e-6
        assert bool(y.isfinite().all())
    synced()


def test_activations_below_the_normal_range():
    """Subnormal bf16 activations count."""
    w, v = gpu_matrix(256, 64, 64, False, 3)
    x = (rows(9, 256, 1).double() * 2.0 ** -129).to(torch.bfloat16)
    assert 0 < float(x.abs().max()) < 2.0 ** -125
    big = moe.W4Weights(w.data.clone(), 1, 256, 64, 64, False)
    big.data[..., 512:] = torch.tensor([0x80, 0x5F], dtype=torch.uint8, device="cuda").repeat(16)   # 2^64
    c = moe.w4_dequantize(big).double()
    y, err = ref.linear(x, c[0], 64)
    check(moe.linear_w4(x, big, fp32=True), y, err)
    synced()


def test_rows_around_the_outputs_stay():
    """out= in the middle of a buffer: the layer and the dense MLP write their rows only."""
    x, wr, q, k = small_layer(5)
    d = [gpu_matrix(*s, 64, True, 30 + i)[0] for i, s in enumerate(((256, 192), (256, 192), (192, 256)))]
    for call in (lambda o: moe.forward_w4(x, wr, *q, k, out=o), lambda o: moe.dense_ffn_w4(x, *d, out=o)):
        buf = torch.full((12, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        want = call(None)
        assert call(buf[4:9]).data_ptr() == buf[4:9].data_ptr()
        assert torch.equal(buf[4:9], want) and bool((buf[:4] == 7).all()) and bool((buf[9:] == 7).all())
    synced()


def test_layer_with_outputs_on_another_stream():
    x, wr, q, k = small_layer(6)
    want, aux = moe.forward_w4(x, wr, *q, k, aux=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, aux2 = moe.forward_w4(x, wr, *q, k, aux=True, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and all(torch.equal(aux[n], aux2[n]) for n in aux)
    synced()
