"""The 4-bit weight calls on the GPU against their definitions in float64 (w4_reference.py), every
element within a bound derived there from the fp32 arithmetic and the outputs' rounding."""
import threading

import numpy as np
import pytest
import torch

import oracle
import expert_routed_ffn_softmax_b200 as moe
import w4_reference as ref
from expert_routed_ffn_softmax_b200 import _abi

pytestmark = pytest.mark.gpu


def to_gpu(codes, scales, zp, group):
    return moe.w4_pack(ref.nibbles(codes).cuda(), scales.cuda(),
                       None if zp is None else zp.cuda(), group=group)


def matrix(E, K, N, group, zeros, seed, extreme=False):
    """(W4Weights, float64 values [E, K, N])."""
    c = ref.make_checkpoint(E, K, N, group, zeros, seed, extreme)
    return to_gpu(*c, group), ref.values(*c, group)


def rows(T, K, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, K), generator=g).to(torch.bfloat16)


def synced():
    assert moe.sync_status() == 0


FORMS = [(32, False), (32, True), (64, False), (64, True), (128, False), (128, True)]


# ----------------------------------------------------------------------------- the weights
@pytest.mark.parametrize("E,K,N", [(1, 64, 16), (3, 192, 80), (2, 704, 64), (1, 128, 272)])
@pytest.mark.parametrize("group,zeros", FORMS)
def test_pack_writes_the_documented_layout(E, K, N, group, zeros):
    c = ref.make_checkpoint(E, K, N, group, zeros, seed=K + N)
    w = to_gpu(*c, group)
    assert np.array_equal(w.data.cpu().numpy(), ref.packed_bytes(*c, group))
    back = moe.w4_dequantize(w).cpu()
    assert torch.equal(back, ref.values(*c, group).to(torch.bfloat16))
    synced()


@pytest.mark.parametrize("E,K,N", [(1, 64, 16), (2, 192, 80), (1, 704, 208)])
@pytest.mark.parametrize("group,zeros", FORMS)
def test_quantize_takes_the_documented_steps(E, K, N, group, zeros):
    g = torch.Generator().manual_seed(K)
    w = (torch.randn((E, K, N), generator=g) * 0.02).to(torch.bfloat16)
    w[0, :32, 0] = 0
    w[0, :, 1] = w[0, :, 1].abs()
    w[0, :, 2] *= 2.0 ** 100
    w[0, :, 3] *= 2.0 ** -120            # scales near the bottom of bf16
    w[0, 5, 4] = 3.0                     # an outlier
    q = moe.w4_quantize(w.cuda(), group=group, zeros=zeros)
    codes, scales, zp = ref.quantize(w, group, zeros)
    assert np.array_equal(q.data.cpu().numpy(),
                          ref.packed_bytes(codes, scales, zp if zeros else None, group))
    synced()


def test_quantize_rounds_ties_to_even():
    """Weights at half-integer multiples of the scale, all exact in bf16, at three scales."""
    K, N = 128, 16
    w = torch.zeros((1, K, N), dtype=torch.float64)
    steps = torch.tensor([7.0] + [j + 0.5 for j in range(-7, 7)] + [-7.0])
    for n in range(N):
        scale = (1.0, 1.5, 1.25)[n % 3] * 2.0 ** (n - 12)
        w[0, :, n] = scale * steps.repeat(K // 16)
    assert torch.equal(w.to(torch.bfloat16).double(), w)
    w = w.to(torch.bfloat16)
    for group in (32, 64, 128):
        codes, scales, _ = ref.quantize(w, group, False)
        assert torch.equal(codes[0, :, 1:15].double(), 8 + torch.round(steps[1:15].double()).expand(N, 14))
        q = moe.w4_quantize(w.cuda(), group=group)
        assert np.array_equal(q.data.cpu().numpy(), ref.packed_bytes(codes, scales, None, group))


def test_quantize_ragged_tiles():
    """Matrices that end inside a tile of 64 rows x 128 elements, several of them."""
    g = torch.Generator().manual_seed(6)
    for E, K, N in ((2, 64, 16), (3, 192, 48), (1, 320, 1040)):
        w = torch.randn((E, K, N), generator=g).to(torch.bfloat16)
        for zeros in (False, True):
            codes, scales, zp = ref.quantize(w, 128, zeros)
            q = moe.w4_quantize(w.cuda(), group=128, zeros=zeros)
            assert np.array_equal(q.data.cpu().numpy(),
                                  ref.packed_bytes(codes, scales, zp if zeros else None, 128))
            assert torch.equal(moe.w4_dequantize(q).cpu(),
                               ref.values(codes, scales, zp if zeros else None, 128).to(torch.bfloat16))


def test_one_matrix_may_leave_the_leading_axis_out():
    c, s, z = ref.make_checkpoint(1, 128, 32, 64, True, seed=1)
    a = moe.w4_pack(ref.nibbles(c)[0].cuda(), s[0].cuda(), z[0].cuda(), group=64)
    assert a.shape == (1, 128, 32) and torch.equal(a.data, to_gpu(c, s, z, 64).data)
    w = torch.randn(128, 32).to(torch.bfloat16).cuda()
    assert torch.equal(moe.w4_quantize(w).data, moe.w4_quantize(w.unsqueeze(0)).data)


# ----------------------------------------------------------------------------- linear
@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 13, 16])
@pytest.mark.parametrize("group,zeros", FORMS)
def test_linear_every_batch_size(T, group, zeros):
    K, N = 704, 144
    w, v = matrix(1, K, N, group, zeros, seed=T)
    x = rows(T, K, T)
    y, err = ref.linear(x, v[0], group)
    ref.check(moe.linear_w4(x.cuda(), w), y, err)
    ref.check(moe.linear_w4(x.cuda(), w, fp32=True), y, err)
    synced()


@pytest.mark.parametrize("T,K,N", [(1, 64, 16), (16, 64, 16), (5, 128, 48), (3, 2816, 2816),
                                   (16, 2112, 2816), (8, 16384, 64), (16, 16384, 80),
                                   (2, 64, 65536), (1, 8192, 4112), (11, 192, 20000)])
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
def test_linear_sizes(T, K, N, group, zeros):
    w, v = matrix(1, K, N, group, zeros, seed=N)
    x = rows(T, K, N)
    y, err = ref.linear(x, v[0], group)
    ref.check(moe.linear_w4(x.cuda(), w, fp32=True), y, err)
    ref.check(moe.linear_w4(x.cuda(), w), y, err)
    synced()


@pytest.mark.parametrize("T,K,N", [
    # K shared by 2, 4 and 8 CTAs, with odd last strips and uneven shares of K; rows kept in shared
    # memory and fragments; more units than run at once
    (1, 704, 2816), (4, 1088, 4112), (6, 4160, 1040), (8, 8256, 528), (2, 16320, 112),
    (12, 16384, 2064), (9, 1984, 4112), (16, 704, 2832), (13, 8192, 4096), (5, 576, 50000),
    (8, 4160, 20016), (10, 1024, 32784)])
def test_linear_cuts(T, K, N):
    w, v = matrix(1, K, N, 64, False, seed=K + N)
    x = rows(T, K, N)
    y, err = ref.linear(x, v[0], 64)
    ref.check(moe.linear_w4(x.cuda(), w, fp32=True), y, err)
    synced()


def test_linear_same_call_same_bits():
    """Sums are joined in a fixed order, whichever CTA takes a unit."""
    for T, K, N in ((1, 2816, 65536), (16, 2816, 40000), (8, 8192, 1024), (3, 704, 2816)):
        w, _ = matrix(1, K, N, 128, False, seed=T)
        x = rows(T, K, T).cuda()
        first = moe.linear_w4(x, w, fp32=True)
        for _ in range(20):
            assert torch.equal(moe.linear_w4(x, w, fp32=True), first)


def test_linear_one_hot_rows_give_the_weights():
    """A one-hot activation reads one weight: every position, exactly."""
    K, N = 192, 48
    for group, zeros in FORMS:
        w, v = matrix(1, K, N, group, zeros, seed=9, extreme=True)
        for k0 in range(0, K, 16):
            x = torch.zeros((16, K), dtype=torch.bfloat16)
            x[torch.arange(16), k0 + torch.arange(16)] = 1
            y = moe.linear_w4(x.cuda(), w, fp32=True).cpu()
            assert torch.equal(y.double(), v[0, k0:k0 + 16])


def test_linear_large_and_tiny_values():
    """Codes at the ends of their range, activations over 30 orders of magnitude."""
    K, N = 256, 64
    w, v = matrix(1, K, N, 32, True, seed=2, extreme=True)
    x = rows(6, K, 3) * (10.0 ** torch.linspace(-18, 12, 6)).unsqueeze(1).to(torch.bfloat16)
    y, err = ref.linear(x, v[0], 32)
    ref.check(moe.linear_w4(x.cuda(), w, fp32=True), y, err)


def test_linear_non_finite_rows_stay_apart():
    """Infinities and NaN of one row do not reach another, at any batch size."""
    K, N = 704, 64
    w, v = matrix(1, K, N, 64, False, seed=4)
    for T in (2, 7, 9, 16):
        x = rows(T, K, T)
        clean = moe.linear_w4(x.cuda(), w).cpu()
        for bad in (float("inf"), float("nan")):
            x2 = x.clone()
            x2[T // 2, 5] = bad
            y = moe.linear_w4(x2.cuda(), w).cpu()
            keep = torch.arange(T) != T // 2
            assert torch.equal(y[keep], clean[keep])
            assert not torch.isfinite(y[T // 2]).all()


def test_linear_empty_batch_and_rows_behind_the_last():
    w, v = matrix(1, 128, 48, 64, False, seed=5)
    assert moe.linear_w4(rows(0, 128, 0).cuda(), w).shape == (0, 48)
    buf = torch.full((20, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    x = rows(5, 128, 1)
    out = moe.linear_w4(x.cuda(), w, out=buf[8:13])
    assert out.data_ptr() == buf[8:13].data_ptr()
    assert bool((buf[:8] == 7).all()) and bool((buf[13:] == 7).all())
    y, err = ref.linear(x, v[0], 64)
    ref.check(buf[8:13], y, err)


def test_linear_past_32_bits():
    """A matrix of more than 2^31 packed bytes: rows near its end are the right ones."""
    K, N = 16384, 268400
    n = moe.load().moe_w4_packed_bytes(1, K, N, 64, 0)
    assert n > 1 << 31
    data = torch.zeros((1, N // 16, K // 64, 544), dtype=torch.uint8, device="cuda")
    data[..., :512] = 0x88                                       # code 8: the value 0
    one = torch.tensor([0x80, 0x3F], dtype=torch.uint8, device="cuda")   # bf16 1.0
    data[..., 512:] = one.repeat(16)
    w = _abi.W4Weights(data, 1, K, N, 64, False)
    last = data[0, -1, -1]                                        # last strip, last block
    last[:512] = 0x99                                             # code 9: the value 1
    x = torch.zeros((2, K), dtype=torch.bfloat16, device="cuda")
    x[0, -1] = 2.0
    x[1, -64:] = 1.0
    y = moe.linear_w4(x, w, fp32=True)
    assert bool((y[:, :-16] == 0).all())
    assert bool((y[0, -16:] == 2).all()) and bool((y[1, -16:] == 64).all())
    synced()


# ----------------------------------------------------------------------------- dense MLP
@pytest.mark.parametrize("T,H,I,group,zeros", [
    (1, 64, 64, 32, False), (16, 64, 64, 128, True), (1, 2816, 2112, 64, False),
    (8, 2816, 2112, 32, True), (16, 2816, 2112, 128, False), (5, 192, 1088, 64, True),
    (9, 4096, 128, 32, False), (3, 128, 8192, 128, True), (8, 192, 8192, 64, False),
    (8, 8192, 192, 64, True), (13, 1088, 2752, 128, False), (2, 16384, 64, 64, False)])
def test_dense_ffn(T, H, I, group, zeros):
    g, vg = matrix(1, H, I, group, zeros, seed=1)
    u, vu = matrix(1, H, I, group, zeros, seed=2)
    d, vd = matrix(1, I, H, group, zeros, seed=3)
    x = rows(T, H, T + H)
    y, err = ref.ffn(x, vg[0], vu[0], vd[0], group)
    got = moe.dense_ffn_w4(x.cuda(), g, u, d)
    ref.check(got, y, err)
    rel = float((got.cpu().double() - y).norm() / y.norm())
    # two roundings to bf16, each uniform in half a step: well under one half step together
    assert rel < ref.HALF_BF16, rel
    assert torch.equal(got, moe.dense_ffn_w4(x.cuda(), g, u, d))
    synced()


def test_dense_ffn_empty_batch():
    g, _ = matrix(1, 64, 128, 64, False, seed=1)
    d, _ = matrix(1, 128, 64, 64, False, seed=2)
    assert moe.dense_ffn_w4(rows(0, 64, 0).cuda(), g, g, d).shape == (0, 64)


# ----------------------------------------------------------------------------- the routed layer
def layer_inputs(T, H, E, I, group, zeros, seed=0, bias=False):
    g, vg = matrix(E, H, I, group, zeros, seed + 1)
    u, vu = matrix(E, H, I, group, zeros, seed + 2)
    d, vd = matrix(E, I, H, group, zeros, seed + 3)
    gen = torch.Generator().manual_seed(seed + 4)
    wr = (torch.randn((H, E), generator=gen) * 0.05).to(torch.bfloat16)
    b = torch.randn(E, generator=gen) if bias else None
    return (g, u, d), (vg, vu, vd), wr, b


LAYER_CASES = [
    # T, H, E, I, k, group, zeros, bias, renorm
    (1, 64, 4, 64, 1, 64, False, False, True), (1, 256, 8, 128, 8, 32, True, True, True),
    (2, 128, 12, 192, 3, 128, False, False, False), (5, 704, 16, 64, 4, 64, True, False, True),
    (8, 256, 128, 128, 8, 64, False, True, True), (9, 192, 64, 64, 8, 32, False, False, True),
    (16, 256, 8, 128, 2, 128, True, True, False), (16, 128, 256, 64, 8, 64, True, False, True),
    (13, 320, 132 + 4, 192, 5, 32, True, True, True), (7, 2816, 32, 704, 8, 64, False, False, True),
    (16, 4096, 4, 64, 4, 64, False, False, True),
    # taller units of gate | up, and of W_down with an odd tail: many rows an expert, and few
    (16, 128, 8, 2432, 4, 64, False, False, True), (12, 4800, 16, 64, 8, 32, True, False, True),
    (16, 64, 256, 448, 8, 128, False, False, True), (16, 2048, 128, 64, 8, 64, False, False, True),
    (8, 128, 8, 2432, 4, 32, True, True, False)]


@pytest.mark.parametrize("T,H,E,I,k,group,zeros,bias,renorm", LAYER_CASES)
def test_layer(T, H, E, I, k, group, zeros, bias, renorm):
    q, v, wr, b = layer_inputs(T, H, E, I, group, zeros, seed=T * H, bias=bias)
    x = rows(T, H, T)
    y, aux = moe.forward_w4(x.cuda(), wr.cuda(), *q, k, bias=None if b is None else b.cuda(),
                            renorm=renorm, aux=True)
    synced()
    ids, wts, _ = oracle.route(x, wr, k, bias=b, renorm=renorm)
    assert np.array_equal(aux["topk_ids"].cpu().numpy(), ids)
    assert np.abs(aux["topk_weights"].cpu().numpy().astype(np.float64) - wts).max() <= 1e-5
    counts, offsets, perm = oracle.dispatch(ids, E)[:3]
    assert np.array_equal(aux["expert_counts"].cpu().numpy(), counts)
    assert np.array_equal(aux["expert_offsets"].cpu().numpy(), offsets)
    assert np.array_equal(aux["perm"].cpu().numpy(), perm)
    assert moe.router_stats(aux)["path"] == "fp64"
    ref.check(y, *ref.layer(x, ids, wts, *v, group))
    again = moe.forward_w4(x.cuda(), wr.cuda(), *q, k, bias=None if b is None else b.cuda(),
                           renorm=renorm)
    assert torch.equal(y, again)
    synced()


def test_layer_ties_take_the_lower_expert():
    """Equal logits everywhere (zero rows, duplicated router columns): ids as the oracle's."""
    T, H, E, I, k = 6, 256, 16, 64, 5
    q, v, wr, _ = layer_inputs(T, H, E, I, 64, False, seed=8)
    wr[:, 1::2] = wr[:, 0::2]
    x = rows(T, H, 1)
    x[2] = 0
    y, aux = moe.forward_w4(x.cuda(), wr.cuda(), *q, k, aux=True)
    synced()
    ids, wts, _ = oracle.route(x, wr, k)
    assert np.array_equal(aux["topk_ids"].cpu().numpy(), ids)
    assert moe.router_stats(aux)["exact_recomputes"] >= 1
    ref.check(y, *ref.layer(x, ids, wts, *v, 64))
    assert bool((y[2] == 0).all())


def test_layer_all_tokens_on_the_same_experts():
    """Every token the same: each chosen expert holds all 16 rows."""
    T, H, E, I, k = 16, 256, 32, 128, 8
    q, v, wr, _ = layer_inputs(T, H, E, I, 32, True, seed=11)
    x = rows(1, H, 2).expand(T, H).contiguous()
    y = moe.forward_w4(x.cuda(), wr.cuda(), *q, k)
    ids, wts, _ = oracle.route(x, wr, k)
    assert len(np.unique(ids)) == k
    ref.check(y, *ref.layer(x, ids, wts, *v, 32))
    assert bool((y == y[0]).all())
    synced()


def test_layer_empty_batch():
    q, _, wr, _ = layer_inputs(1, 64, 4, 64, 64, False)
    y, aux = moe.forward_w4(rows(0, 64, 0).cuda(), wr.cuda(), *q, 2, aux=True)
    assert y.shape == (0, 64) and aux["topk_ids"].shape == (0, 2)


def test_layer_agrees_with_the_bf16_layer_on_dequantised_weights():
    """The way to larger batches: the bf16 layer on the dequantised weights gives the same y up
    to the rounding of the weights, of h and of the expert outputs to bf16 (4 half steps)."""
    T, H, E, I, k = 8, 512, 16, 256, 4
    gen = torch.Generator().manual_seed(3)
    w = [(torch.randn(s, generator=gen) * 0.05).to(torch.bfloat16).cuda()
         for s in ((E, H, I), (E, H, I), (E, I, H))]
    wr = (torch.randn((H, E), generator=gen) * 0.05).to(torch.bfloat16).cuda()
    x = rows(T, H, 5).cuda()
    q = [moe.w4_quantize(t, group=32, zeros=True) for t in w]
    y4 = moe.forward_w4(x, wr, *q, k)
    yb = moe.forward(x, wr, *[moe.w4_dequantize(t) for t in q], k)
    assert float((y4.double() - yb.double()).norm() / yb.double().norm()) < 4 * ref.HALF_BF16
    synced()


# ----------------------------------------------------------------------------- as they are used
def decode_block(x, wr, experts, dense, head, k):
    """A decode step's feed-forward half: routed experts and dense MLP side by side, then a
    projection."""
    y = moe.forward_w4(x, wr, *experts, k) + moe.dense_ffn_w4(x, *dense)
    return moe.linear_w4(y, head, fp32=True)


def block_inputs(T=4, H=256, E=16, I=128, Id=192, V=1008, k=4, seed=0):
    experts, _, wr, _ = layer_inputs(T, H, E, I, 64, True, seed=seed)
    dense = [matrix(1, *s, 64, True, seed + 20 + i)[0] for i, s in enumerate(((H, Id), (H, Id), (Id, H)))]
    head = matrix(1, H, V, 128, False, seed + 30)[0]
    return rows(T, H, seed).cuda(), wr.cuda(), experts, dense, head, k


def test_operators_together_match_their_definitions():
    T, H, E, I, k = 4, 256, 16, 128, 4
    experts, v, wr, _ = layer_inputs(T, H, E, I, 64, True, seed=40)
    dm = [matrix(1, *s, 64, True, 60 + i) for i, s in enumerate(((H, 192), (H, 192), (192, H)))]
    head, hv = matrix(1, H, 1008, 128, False, 70)
    x = rows(T, H, 40)
    ids, wts, _ = oracle.route(x, wr, k)
    y1, e1 = ref.layer(x, ids, wts, *v, 64)
    y2, e2 = ref.ffn(x, *[m[1][0] for m in dm], 64)
    y, err = y1 + y2, ref.rounded(y1, e1, torch.bfloat16) + ref.rounded(y2, e2, torch.bfloat16)
    err = ref.rounded(y, err, torch.bfloat16)
    z, ez = ref.linear(y, hv[0], 128)
    got = decode_block(x.cuda(), wr.cuda(), experts, [m[0] for m in dm], head, k)
    ref.check(got, z, ez * 2 + err @ hv[0].abs())
    synced()


def test_captured_and_replayed():
    """The block in a CUDA graph: replays on new inputs give the eager results, and two graphs
    replayed in turn do not disturb each other."""
    a, b = block_inputs(seed=1), block_inputs(T=11, seed=2)
    graphs = []
    for args in (a, b):
        decode_block(*args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = decode_block(*args)
        graphs.append((g, out))
    for seed in range(3):
        for args in (a, b):
            args[0].copy_(rows(*args[0].shape, 100 + seed).cuda())
        want = [decode_block(*args).clone() for args in (a, b)]
        for g, out in graphs:
            out.fill_(-1)
        for g, _ in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        for (g, out), w in zip(graphs, want):
            assert torch.equal(out, w)
    synced()


def test_two_streams_at_once():
    """Calls in flight on two streams (default workspaces) give the results of calls alone."""
    a, b = block_inputs(seed=3), block_inputs(T=16, seed=4)
    want = [decode_block(*args).clone() for args in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(20):
        for i, args in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                outs[i].append(decode_block(*args))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])
    synced()


def test_two_threads_at_once():
    a, b = block_inputs(seed=5), block_inputs(T=9, seed=6)
    want = [decode_block(*args).clone() for args in (a, b)]
    torch.cuda.synchronize()
    bad = []

    def work(args, w):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                if not torch.equal(decode_block(*args), w):
                    bad.append(args[0].shape)
    ts = [threading.Thread(target=work, args=p) for p in zip((a, b), want)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad
    synced()


def test_waits_that_run_out_are_reported():
    """With the wait limit at next to nothing the layer's hand-overs run out: the call returns, the
    error is reported once, and the next call is right again."""
    T, H, E, I, k = 8, 256, 64, 128, 4
    q, _, wr, _ = layer_inputs(T, H, E, I, 64, False, seed=90)
    x, wr = rows(T, H, 90).cuda(), wr.cuda()
    want = moe.forward_w4(x, wr, *q, k)
    synced()
    lib = moe.load()
    assert lib.moe_debug_set_wait_limit_ns(1) == 0
    try:
        moe.forward_w4(x, wr, *q, k)
        status = moe.sync_status()
    finally:
        assert lib.moe_debug_set_wait_limit_ns(0) == 0
    assert status == _abi.MOE_ERR_TIMEOUT
    synced()
    assert torch.equal(moe.forward_w4(x, wr, *q, k), want)
    synced()


def test_stream_argument():
    """stream=: the call and what it allocates belong to that stream."""
    x, wr, experts, dense, head, k = block_inputs(seed=7)
    want = [moe.linear_w4(x, head), moe.dense_ffn_w4(x, *dense), moe.forward_w4(x, wr, *experts, k)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [moe.linear_w4(x, head, stream=s), moe.dense_ffn_w4(x, *dense, stream=s),
           moe.forward_w4(x, wr, *experts, k, stream=s)]
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_caller_owned_workspace():
    x, wr, experts, dense, head, k = block_inputs(seed=8)
    L = moe.load()
    n = L.moe_w4_workspace_size(4, 256, 16, 128, k, _abi.MOE_FLAG_W4_ZEROS)
    ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")   # contents are scratch
    want = moe.forward_w4(x, wr, *experts, k)
    for _ in range(2):
        assert torch.equal(moe.forward_w4(x, wr, *experts, k, workspace_buf=ws[:n]), want)
    assert bool((ws[n:] == 0xA5).all())
    with pytest.raises(moe.MoEError):
        moe.forward_w4(x, wr, *experts, k, workspace_buf=ws[:n - 256])
    synced()


def test_binding_refuses():
    x, wr, experts, dense, head, k = block_inputs(seed=9)
    other = matrix(1, 256, 192, 32, True, 1)[0]
    no = pytest.raises
    with no(moe.MoEError):
        moe.linear_w4(rows(17, 256, 0).cuda(), head)
    with no(ValueError):
        moe.linear_w4(x[:, :128].contiguous(), head)           # another K
    with no(ValueError):
        moe.linear_w4(x.t().contiguous().t(), head)            # not contiguous
    with no(TypeError):
        moe.linear_w4(x.float(), head)
    with no(TypeError):
        moe.linear_w4(x, head.data)
    with no(ValueError):
        moe.linear_w4(x, experts[0])                           # several matrices
    with no((TypeError, ValueError)):
        moe.linear_w4(x, head, out=torch.empty((4, 1008), device="cuda"))
    with no(ValueError):
        moe.dense_ffn_w4(x, dense[0], other, dense[2])         # another group
    with no(ValueError):
        moe.dense_ffn_w4(x, dense[0], dense[1], dense[1])      # not [I, H]
    with no(moe.MoEError):
        moe.dense_ffn_w4(x, *dense, out=x)
    with no(ValueError):
        moe.forward_w4(x, wr, dense[0], dense[1], dense[2], k)  # not E matrices
    with no(moe.MoEError):
        moe.forward_w4(x, wr, *experts, 17)
    with no(TypeError):
        moe.forward_w4(x, wr, *experts, k, bias=torch.zeros(16, dtype=torch.float64, device="cuda"))
    with no(moe.MoEError):
        moe.w4_quantize(torch.zeros((64, 24), dtype=torch.bfloat16, device="cuda"))
    with no(moe.MoEError):
        moe.w4_quantize(torch.zeros((64, 16), dtype=torch.bfloat16, device="cuda"), group=16)
    c, s, z = ref.make_checkpoint(1, 128, 32, 64, True, seed=1)
    with no(ValueError):
        moe.w4_pack(ref.nibbles(c).cuda(), s[:, :, :1].contiguous().cuda(), group=64)
    with no(ValueError):
        moe.w4_pack(ref.nibbles(c).cuda(), s.cpu().cuda(), z[:, :16].contiguous().cuda(), group=64)
    synced()
